"""What the decayed linear-attention operators and the query/key rotation are measured on.

Three operators, each reached through ``linear_attention_delta_gdn_b200.binding``:

  linear   linear attention with one fixed decay per head over whole sequences,
               S_t = a_h S_{t-1} + k_t v_t^T,   o_t = S_t^T q_t,   a_h = exp(log_decay_h),
           forward, or forward and backward, dense [B, T, H, D] or packed by cu_seqlens
  step     the same recurrence for one token of each request, on the states of a pool that the requests' slots name
  rotate   RMS norm of every query and key head and the position rotation (one to three axes) in one pass,
           forward, or forward and backward

``run`` computes them with elementary torch operations in 32 bits (decay factors and angles in 64) where ``own`` is
false, and makes the framework's calls where it is true.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _linear(name, dtype, H, Dk, Dv, lengths="", B=1, T=0, decay="slopes", state=False, grad=False):
    return {"name": name, "op": "linear", "dtype": dtype, "H": H, "Dk": Dk, "Dv": Dv, "B": B, "T": T, "lengths": lengths,
            "decay": decay, "state": state, "grad": grad}


def _step(name, dtype, B, H, Dk, Dv, pool, idle=0):
    return {"name": name, "op": "step", "dtype": dtype, "B": B, "H": H, "Dk": Dk, "Dv": Dv, "pool": pool, "idle": idle}


def _rotate(name, dtype, B, T, Hq, Hk, D, pairs, axes=1, interleaved=False, norm=True, far=0, grad=False):
    return {"name": name, "op": "rotate", "dtype": dtype, "B": B, "T": T, "Hq": Hq, "Hk": Hk, "D": D, "pairs": pairs, "axes": axes,
            "interleaved": interleaved, "norm": norm, "far": far, "grad": grad}


def listed():
    return [
        # the prompt of one chat turn, an odd length: latency
        _linear("prompt-b1t77", "bf16", 16, 128, 128, B=1, T=77),
        # prefill of a batch at the training layer's shape
        _linear("prompt-b4t4096", "bf16", 16, 128, 128, B=4, T=4096),
        # a long document that continues from a stored state
        _linear("prompt-b1t65536-s0", "bf16", 16, 128, 128, B=1, T=65536, state=True),
        # prompts of several requests packed back to back, one of them empty and one of a single token
        _linear("prompt-packed", "bf16", 8, 64, 128, lengths="1000,1,4097,0,333,2048,77,5001", state=True),
        # one layer's training step, forward and backward
        _linear("train-b4t4096", "bf16", 16, 128, 128, B=4, T=4096, grad=True),
        # the same on packed documents with narrow heads and both state gradients
        _linear("train-packed-d64", "bf16", 12, 64, 64, lengths="1531,64,2900,7,1201,3333", state=True, grad=True),
        # a 32-bit training step, as for a check of a model's numerics
        _linear("train-f32-b2t1001", "f32", 4, 64, 64, B=2, T=1001, state=True, grad=True),
        # one request answering: latency
        _step("step-b1", "bf16", 1, 16, 128, 128, pool=8),
        # a full serving batch with some idle rows, the states bandwidth-bound
        _step("step-b256", "bf16", 256, 16, 128, 128, pool=320, idle=5),
        # queries and keys of a prefill at the training layer's shape
        _rotate("rotate-b4t4096", "bf16", 4, 4096, 16, 16, 128, pairs=64),
        # queries and keys of one serving step, far into long documents
        _rotate("rotate-step-b64", "bf16", 64, 1, 16, 4, 128, pairs=32, interleaved=True, far=900000),
        # video tokens (time, height, width), shared key heads, a training step
        _rotate("rotate-video-train", "bf16", 2, 3999, 16, 4, 128, pairs=64, axes=3, grad=True),
    ]


def _about(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    kind = rng.choice(("prompt", "prompt", "packed", "train", "train", "step", "rotate", "rotate"))
    dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
    if kind in ("prompt", "packed", "train"):
        H, Dk, Dv = rng.choice((1, 2, 4, 8, 12, 16, 20, 32)), rng.choice((16, 32, 64, 128, 128)), rng.choice((16, 32, 64, 128, 128))
        grad = kind == "train" or (kind == "packed" and rng.random() < 0.5)
        rows = (1 << 18 if grad else 1 << 20) // (1 if dtype == "bf16" else 4)   # tokens x heads at most
        c = dict(decay=rng.choice(("slopes", "slopes", "slow", "none", "strong")), state=rng.random() < 0.5, grad=grad)
        if kind == "packed" or (kind == "train" and rng.random() < 0.4):
            left, lens = rows // H, []
            for _ in range(rng.randint(1, 24)):
                n = rng.choice((0, 1)) if rng.random() < 0.1 else min(left, _about(rng, 2, 16384))
                left -= n
                lens.append(n)
            if not any(lens):
                lens.append(65)
            c["lengths"] = ",".join(map(str, lens))
        else:
            B = _about(rng, 1, 16)
            c.update(B=B, T=_about(rng, 1, min(65536, max(1, rows // (H * B)))))
        c = _linear("", dtype, H, Dk, Dv, **c)
    elif kind == "step":
        H, D = rng.choice((1, 4, 8, 16, 32)), rng.choice((16, 32, 64, 128, 128))
        B = _about(rng, 1, max(1, 4096 // H))
        c = _step("", dtype, B, H, D, rng.choice((D, 64, 128)), pool=B + rng.randint(1, 40), idle=rng.choice((0, 0, 1, B // 8)))
    else:
        Hk = rng.choice((1, 2, 4, 8, 16))
        Hq, D = Hk * rng.choice((1, 1, 2, 4)), rng.choice((16, 32, 64, 128, 128))
        B = _about(rng, 1, 64)
        grad = rng.random() < 0.5
        T = _about(rng, 1, max(1, (1 << 19) // ((Hq + Hk) * B)))
        c = _rotate("", dtype, B, T, Hq, Hk, D, pairs=rng.choice((D // 2, D // 2, D // 4, D // 8)), axes=rng.choice((1, 1, 2, 3)),
                    interleaved=rng.random() < 0.5, norm=rng.random() < 0.8, far=rng.choice((0, 0, 30000, 2000000)), grad=grad)
    del c["name"]
    return c


# ------------------------------------------------------------------ what a user's program has in hand

def _lengths(c):
    return [int(x) for x in c["lengths"].split(",")] if c["lengths"] else [c["T"]] * c["B"]


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dt = _DT[c["dtype"]]

    def normal(*shape, scale=1.0, to=dt):
        return torch.randn(shape, generator=g, device="cuda").mul_(scale).to(to)

    def decays(H, kind):
        h = torch.arange(1, H + 1, device="cuda", dtype=torch.float32)
        jitter = 0.75 + 0.5 * torch.rand(H, generator=g, device="cuda")
        if kind == "none":      # plain linear attention
            return torch.zeros(H, device="cuda")
        if kind == "slow":      # horizons of hundreds to thousands of tokens
            return -jitter * torch.exp2(-6 - 6 * h / H)
        if kind == "strong":    # horizons of a token or less
            return -jitter * 40 * h / H
        return -jitter * torch.exp2(-8 * h / H)

    s = {"case": c}
    if c["op"] == "linear":
        H, Dk, Dv, lens = c["H"], c["Dk"], c["Dv"], _lengths(c)
        lead = (sum(lens),) if c["lengths"] else (c["B"], c["T"])
        s["q"], s["k"] = normal(*lead, H, Dk, scale=Dk ** -0.5), normal(*lead, H, Dk)
        s["v"] = normal(*lead, H, Dv)
        s["g"] = decays(H, c["decay"])
        if c["lengths"]:
            s["cu"] = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda")
            s["Tmax"] = max(lens)
        s["S0"] = normal(len(lens), H, Dk, Dv, to=torch.float32) if c["state"] else None
        if c["grad"]:
            s["do"] = normal(*lead, H, Dv)
            s["dST"] = normal(len(lens), H, Dk, Dv, scale=0.1, to=torch.float32) if c["state"] else None
    elif c["op"] == "step":
        B, H, Dk, Dv = c["B"], c["H"], c["Dk"], c["Dv"]
        s["q"], s["k"], s["v"] = normal(B, H, Dk, scale=Dk ** -0.5), normal(B, H, Dk), normal(B, H, Dv)
        s["g"] = decays(H, "slopes")
        s["S"] = normal(c["pool"], H, Dk, Dv, to=torch.float32)
        slots = torch.randperm(c["pool"], generator=g, device="cuda")[:B].to(torch.int32)
        if c["idle"]:
            slots[torch.randperm(B, generator=g, device="cuda")[:c["idle"]]] = -1
        s["slots"] = slots
    else:
        B, T, Hq, Hk, D, P, A = (c[n] for n in ("B", "T", "Hq", "Hk", "D", "pairs", "axes"))
        s["q"], s["k"] = normal(B, T, Hq, D, scale=3.0), normal(B, T, Hk, D, scale=0.5)
        s["inv_freq"] = torch.exp(-math.log(10000.0) / P * torch.arange(P, device="cuda", dtype=torch.float64)).float()
        first = torch.randint(0, c["far"] + 1, (B, 1), generator=g, device="cuda")
        t = torch.arange(T, device="cuda").expand(B, T)
        if A == 1:
            s["pos"] = (first + t).contiguous()
        else:   # frames of 24 x 40 patches; with two axes rows of 40
            per = (960, 40, 1)[3 - A:]
            of = (1 << 40, 24, 40)[3 - A:] if A == 3 else (1 << 40, 40)
            s["pos"] = torch.stack([(t // p) % n + (first if i == 0 else 0) for i, (p, n) in enumerate(zip(per, of))]).to(torch.int32).contiguous()
        # a quarter of the pairs for the first axis, the others' share of the rest in turn
        own_pairs = [P] if A == 1 else [P // 4] + [(P - P // 4 + i) // (A - 1) for i in range(A - 1)]
        s["axes"] = None if A == 1 else torch.cat([torch.full((n,), i, dtype=torch.int32) for i, n in enumerate(own_pairs)])[:P].contiguous().cuda()
        s["wq"] = 1 + normal(D, scale=0.1, to=torch.float32) if c["norm"] else None
        s["wk"] = 1 + normal(D, scale=0.1, to=torch.float32) if c["norm"] else None
        if c["grad"]:
            s["dyq"], s["dyk"] = normal(B, T, Hq, D), normal(B, T, Hk, D)
    return s


_EPS = 1e-6


def run(state):
    s, c = state, state["case"]
    if own:
        return _framework(s, c)
    return {"linear": _plain_linear, "step": _plain_step, "rotate": _plain_rotate}[c["op"]](s, c)


def _framework(s, c):
    from linear_attention_delta_gdn_b200 import binding as b
    if c["op"] == "step":
        return b.gdn2_linear_decode_step(s["q"], s["k"], s["v"], s["g"], s["S"], slots=s["slots"]), s["S"]
    if c["op"] == "rotate":
        norm = dict(q_weight=s["wq"], k_weight=s["wk"], eps=_EPS if c["norm"] else None, interleaved=c["interleaved"])
        q, k = b.gdn2_qk_norm_rope_fwd(s["q"], s["k"], s["pos"], s["inv_freq"], s["axes"], **norm)
        if not c["grad"]:
            return q, k
        d = b.gdn2_qk_norm_rope_bwd(s["q"], s["k"], s["dyq"], s["dyk"], s["pos"], s["inv_freq"], s["axes"], **norm)
        return [q, k, d["dq"], d["dk"]] + ([d["dq_weight"], d["dk_weight"]] if c["norm"] else [])
    x = (s["q"], s["k"], s["v"], s["g"])
    if c["lengths"]:
        out = list(b.gdn2_linear_varlen_fwd(*x, s["cu"], s["Tmax"], s["S0"]))
        d = b.gdn2_linear_varlen_bwd(*x, s["do"], s["cu"], s["Tmax"], s["S0"], s["dST"], want_dS0=c["state"]) if c["grad"] else {}
    else:
        out = list(b.gdn2_linear_fwd(*x, s["S0"]))
        d = b.gdn2_linear_bwd(*x, s["do"], s["S0"], s["dST"], want_dS0=c["state"]) if c["grad"] else {}
    return out + [d[n] for n in ("dq", "dk", "dv", "dS0") if d.get(n) is not None]


# ------------------------------------------------------------------ plain forms

_C = 128   # tokens of a chunk of the plain form


def _decay(g, steps):
    """exp(g_h * steps) in 32 bits from a product in 64; steps >= 0, one more dimension in front for the heads."""
    return torch.exp(g.double().view(-1, *([1] * steps.dim())) * steps.double()).float()


def _rows(x, idx, real):
    """Packed [Ttot, H, D] -> padded [N, H, T, D] in 32 bits, zeros behind each sequence's end."""
    return torch.where(real[:, :, None, None], x.float()[idx], 0.0).transpose(1, 2)


def _mix(q, k, v, g, start, lead):
    """sum over j <= i of a^(i-j) (q_i . k_j) v_j, plus a^(i+lead) q_i start; [N, H, T, D], T a multiple of the chunk."""
    N, H, T, _ = q.shape
    q, k, v = (x.reshape(N, H, T // _C, _C, x.shape[-1]) for x in (q, k, v))
    i = torch.arange(_C, device=q.device)
    far = (i[:, None] - i[None, :])
    w = torch.where(far >= 0, _decay(g, far.clamp(min=0)), 0.0)
    o = ((q @ k.transpose(-1, -2)) * w[None, :, None]) @ v
    local = (k * _decay(g, _C - 1 - i)[None, :, None, :, None]).transpose(-1, -2) @ v   # [N, H, NC, Dk, Dv]
    n = torch.arange(T // _C, device=q.device)
    far = (n[:, None] - n[None, :] - 1)
    join = torch.where(far >= 0, _decay(g, far.clamp(min=0) * _C), 0.0)
    before = (join[None] @ local.flatten(-2)).view_as(local)
    o = o + _decay(g, i + 1)[None, :, None, :, None] * (q @ before)
    if start is not None:
        o = o + _decay(g, n[:, None] * _C + i[None, :] + lead)[None, :, :, :, None] * (q @ start[:, :, None])
    return o.view(N, H, T, -1)


def _plain_linear(s, c):
    q, k, v, g, S0 = s["q"], s["k"], s["v"], s["g"], s["S0"]
    lead = q.shape[:-2]
    H, dt = c["H"], q.dtype
    q, k, v = (x.reshape(-1, H, x.shape[-1]) for x in (q, k, v))
    if c["lengths"]:
        begin, lens, Tmax = s["cu"][:-1].long(), (s["cu"][1:] - s["cu"][:-1]).long(), s["Tmax"]
    else:
        begin, Tmax = torch.arange(c["B"], device=q.device) * c["T"], c["T"]
        lens = torch.full((c["B"],), c["T"], device=q.device)
    t = torch.arange(-(-Tmax // _C) * _C, device=q.device)[None]
    real = t < lens[:, None]
    fwd = torch.where(real, begin[:, None] + t, 0)
    rev = torch.where(real, begin[:, None] + lens[:, None] - 1 - t, 0)

    def back(y, idx):
        out = torch.empty((q.shape[0], H, y.shape[-1]), dtype=dt, device=q.device)
        out[idx[real]] = y.transpose(1, 2)[real].to(dt)
        return out.view(*lead, H, y.shape[-1])

    q1, k1, v1 = (_rows(x, fwd, real) for x in (q, k, v))
    left = torch.where(real, lens[:, None] - 1 - t, 0)      # tokens behind this one
    fade = torch.exp(g.double()[None, :, None] * left[:, None].double()).float()[..., None]
    whole = torch.exp(g.double()[None, :] * lens[:, None].double()).float()[..., None, None]
    o = _mix(q1, k1, v1, g, S0, 1)
    ST = (k1 * fade).transpose(-1, -2) @ v1
    if S0 is not None:
        ST = ST + whole * S0
    out = [back(o, fwd), ST]
    if c["grad"]:
        do, dST = s["do"].reshape(-1, H, v.shape[-1]), s["dST"]
        do1 = _rows(do, fwd, real)
        dq = _mix(do1, v1, k1, g, None if S0 is None else S0.transpose(-1, -2), 1)
        q2, k2, v2, do2 = (_rows(x, rev, real) for x in (q, k, v, do))
        dk = _mix(v2, do2, q2, g, None if dST is None else dST.transpose(-1, -2), 0)
        dv = _mix(k2, q2, do2, g, dST, 0)
        out += [back(dq, fwd), back(dk, rev), back(dv, rev)]
        if S0 is not None:
            age = torch.exp(g.double()[None, :, None] * (t + 1)[:, None].double()).float()[..., None]
            out.append((q1 * age).transpose(-1, -2) @ do1 + whole * dST)
    return out


def _plain_step(s, c):
    rows = (s["slots"] >= 0).nonzero()[:, 0]
    slot = s["slots"][rows].long()
    q, k, v = (s[n][rows].float() for n in "qkv")
    S = torch.exp(s["g"])[None, :, None, None] * s["S"][slot] + k[..., None] * v[..., None, :]
    o = torch.zeros((c["B"], c["H"], c["Dv"]), dtype=s["q"].dtype, device=S.device)
    o[rows] = (q[..., None] * S).sum(-2).to(o.dtype)
    s["S"][slot] = S
    return o, s["S"]


def _angles(s):
    p = s["pos"] if s["axes"] is not None else s["pos"][None]                   # [A, B, T]
    which = s["axes"].long() if s["axes"] is not None else torch.zeros(s["inv_freq"].numel(), dtype=torch.long, device=p.device)
    a = p[which].double() * s["inv_freq"].double()[:, None, None]               # [P, B, T]
    return a.permute(1, 2, 0)[:, :, None]


def _turn(x, cos, sin, interleaved):
    P = cos.shape[-1]
    a, b = (x[..., 0:2 * P:2], x[..., 1:2 * P:2]) if interleaved else (x[..., :P], x[..., P:2 * P])
    a, b = a * cos - b * sin, a * sin + b * cos
    y = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((y, x[..., 2 * P:]), -1)


def _plain_rotate(s, c):
    a = _angles(s)
    cos, sin = a.cos().float(), a.sin().float()

    def forward(x, w):
        x = x.float()
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + _EPS) if w is not None else None
        return _turn(x if w is None else x * r * w, cos, sin, c["interleaved"]), r

    def backward(x, r, w, dy):
        d = _turn(dy.float(), cos, -sin, c["interleaved"])
        if w is None:
            return d, None
        n = x.float() * r
        dn = d * w
        return (dn - n * (dn * n).mean(-1, keepdim=True)) * r, (d * n).sum((0, 1, 2))

    q, rq = forward(s["q"], s["wq"])
    k, rk = forward(s["k"], s["wk"])
    out = [q.to(s["q"].dtype), k.to(s["q"].dtype)]
    if c["grad"]:
        dq, dwq = backward(s["q"], rq, s["wq"], s["dyq"])
        dk, dwk = backward(s["k"], rk, s["wk"], s["dyk"])
        out += [dq.to(s["q"].dtype), dk.to(s["q"].dtype)] + ([dwq, dwk] if c["norm"] else [])
    return out


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "linear":
        lens, H, Dk, Dv = _lengths(c), c["H"], c["Dk"], c["Dv"]
        tok, st = sum(lens) * H, 4 * len(lens) * H * Dk * Dv
        n = tok * (2 * Dk + 2 * Dv) * e + st * (2 if c["state"] else 1)
        if c["grad"]:   # also dout read, dq, dk, dv written; dST read, dS0 written
            n += tok * (2 * Dk + 2 * Dv) * e + (2 * st if c["state"] else 0)
        # state update and read-out: 4 Dk Dv; backward: dq, dk, dv, the gradient state's update and the state again
        return {"bytes": n, "flops": tok * Dk * Dv * (14 if c["grad"] else 4)}
    if c["op"] == "step":
        rows = (c["B"] - c["idle"]) * c["H"]
        return {"bytes": rows * (8 * c["Dk"] * c["Dv"] + (2 * c["Dk"] + c["Dv"]) * e) + c["B"] * c["H"] * c["Dv"] * e, "flops": rows * 5 * c["Dk"] * c["Dv"]}
    x = c["B"] * c["T"] * (c["Hq"] + c["Hk"]) * c["D"]
    pos = c["B"] * c["T"] * c["axes"] * (8 if c["axes"] == 1 else 4)
    return {"bytes": x * e * (4 if c["grad"] else 2) + pos, "flops": x * (16 if c["grad"] else 6)}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    s, c = prepare(case, seed), case
    f = {n: t.double() for n, t in s.items() if isinstance(t, torch.Tensor) and t.is_floating_point()}
    if c["op"] == "step":
        S, o = f["S"], torch.zeros((c["B"], c["H"], c["Dv"]), dtype=torch.float64, device="cuda")
        for r, slot in enumerate(s["slots"].tolist()):
            if slot >= 0:
                S[slot] = S[slot] * f["g"].exp().view(-1, 1, 1) + torch.einsum("hk,hv->hkv", f["k"][r], f["v"][r])
                o[r] = torch.einsum("hk,hkv->hv", f["q"][r], S[slot])
        return o, S
    if c["op"] == "rotate":
        return _exact_rotate(s, c, f)
    lens, H = _lengths(c), c["H"]
    if (sum(lens) if c["lengths"] else c["T"]) > 140000:
        return None
    a = f["g"].exp().view(1, H, 1, 1)
    names = ("o", "dq", "dk", "dv")
    out = {n: torch.empty_like(f[x]) for n, x in zip(names, "vqkv")}
    states = []
    for b in range(len(lens) if c["lengths"] else 1):
        at = slice(int(s["cu"][b]), int(s["cu"][b + 1])) if c["lengths"] else slice(None)
        part = lambda x: x[at][None] if c["lengths"] else x   # [batch, token, H, D]
        q, k, v = part(f["q"]), part(f["k"]), part(f["v"])
        T, n = q.shape[1], q.shape[0]
        one = slice(b, b + 1) if c["lengths"] else slice(None)
        S = f["S0"][one].clone() if c["state"] else torch.zeros((n, H, c["Dk"], c["Dv"]), dtype=torch.float64, device="cuda")
        do = part(f["do"]) if c["grad"] else None
        o, dq, dk, dv = (part(out[x]) for x in names)
        for t in range(T):
            S = a * S + k[:, t, :, :, None] * v[:, t, :, None, :]
            o[:, t] = (q[:, t, :, None, :] @ S)[:, :, 0]
            if c["grad"]:
                dq[:, t] = (S @ do[:, t, :, :, None])[..., 0]
        got = [S]
        if c["grad"]:
            G = f["dST"][one].clone() if c["state"] else torch.zeros_like(S)
            for t in range(T - 1, -1, -1):
                G = G + q[:, t, :, :, None] * do[:, t, :, None, :]
                dk[:, t] = (G @ v[:, t, :, :, None])[..., 0]
                dv[:, t] = (k[:, t, :, None, :] @ G)[:, :, 0]
                G = a * G
            got.append(G)
        states.append(got)
    ends = [torch.cat(x) for x in zip(*states)]
    return [out["o"], ends[0]] + ([out["dq"], out["dk"], out["dv"]] + ([ends[1]] if c["state"] else []) if c["grad"] else [])


def _exact_rotate(s, c, f):
    pos = s["pos"].double() if s["axes"] is not None else s["pos"].double()[None]
    which = s["axes"].tolist() if s["axes"] is not None else [0] * c["pairs"]
    turn = torch.stack([torch.polar(torch.ones_like(pos[0]), pos[x] * w) for x, w in zip(which, f["inv_freq"])], -1)[:, :, None]
    P, D = c["pairs"], c["D"]
    first = list(range(0, 2 * P, 2)) if c["interleaved"] else list(range(P))
    second = [x + 1 for x in first] if c["interleaved"] else [x + P for x in first]

    def rotated(x, by):
        y, z = x.clone(), torch.complex(x[..., first], x[..., second]) * by
        y[..., first], y[..., second] = z.real, z.imag
        return y

    outs, grads, weights = [], [], []
    for x, w, dy in ((f["q"], f.get("wq"), f.get("dyq")), (f["k"], f.get("wk"), f.get("dyk"))):
        r = (x.pow(2).sum(-1, keepdim=True) / D + _EPS).pow(-0.5) if c["norm"] else None
        outs.append(rotated(x * r * w if c["norm"] else x, turn))
        if c["grad"]:
            d = rotated(dy, turn.conj())
            if c["norm"]:   # y = x r w: dx = r w d - x r^3 sum(w d x) / D
                weights.append((d * x * r).sum((0, 1, 2)))
                d = r * w * d - x * r.pow(3) * (w * d * x).sum(-1, keepdim=True) / D
            grads.append(d)
    return outs + grads + weights
