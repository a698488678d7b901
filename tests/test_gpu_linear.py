"""Linear attention with a decay per head on the GPU against the fp64 oracle: whole sequences, packed sequences, the
single-token step on a pool of states, and their runs together.

Tolerances (relative L2 per head), from the roundings on the way:
  fp32   outputs and states 1e-5: products of two-term operands are off by 2^-21 at most, sums of 64 terms by
         64 * 2^-24 = 4e-6, a decay power by 2 ulp plus 2^-24 of its exponent (below 100 where it matters, 4e-6)
  bf16   outputs 3 * 2^-8 = 1.2e-2: the pair weights, the state and the output each round once, half a step is 2^-8
         states (fp32) 2e-5: a term of the state's products is two bf16 numbers, off by 2^-18 = 4e-6, then a sum of 128
         terms (128 * 2^-24 = 8e-6) and the decay powers (4e-6)
The single-token step has fp32 arithmetic throughout: states 1e-6 (a handful of roundings), outputs as its test derives.
"""
import numpy as np
import pytest
import torch

from conftest import worst_head_rel_l2
from linear_attention_delta_gdn_b200 import binding
from linear_attention_delta_gdn_b200.inputs import to_f64
from oracle import linear as lin

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
TOL = {"f32": 1e-5, "bf16": 3 * 2.0 ** -8}
TOL_STATE = {"f32": 1e-5, "bf16": 2e-5}


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from linear_attention_delta_gdn_b200 import build
    build.build()
    binding.gdn2_device_status()
    yield
    assert binding.gdn2_device_status() == binding.GDN2_OK, binding.last_error()


def make(lead, N, H, Dk, Dv, dtype, seed, decays=None):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)
    x = {"q": r(*lead, H, Dk) * Dk ** -0.5, "k": r(*lead, H, Dk), "v": r(*lead, H, Dv), "do": r(*lead, H, Dv)}
    x = {n: t.to(DT[dtype]) for n, t in x.items()}
    x["g"] = -torch.exp2(-8.0 * torch.arange(1, H + 1) / H) if decays is None else torch.tensor(decays, dtype=torch.float32)
    x["S0"], x["dST"] = r(N, H, Dk, Dv), r(N, H, Dk, Dv)
    return x, {n: t.cuda() for n, t in x.items()}


def check_tokens(got, want, dtype, what):
    assert np.all(np.isfinite(got)), what
    err = worst_head_rel_l2(got, want)
    assert err <= TOL[dtype], (what, err)


def check_states(got, want, dtype, what):
    # 32 bits hold nothing below 2^-149 and full precision only from 2^-126: a head whose elements all lie below that (a
    # state behind a decay of e^-150, 7e-66) is off by at most 2^-126 an element instead.
    tiny = np.abs(want).max(axis=(2, 3), keepdims=True) < 2.0 ** -126
    assert np.all(np.abs(np.where(tiny, got, 0.0)) <= 2.0 ** -126), what
    err = worst_head_rel_l2(np.where(tiny, 0.0, got), np.where(tiny, 0.0, want), state=True)
    assert err <= TOL_STATE[dtype], (what, err)


def check_dense(x, d, dtype, S0=True, dST=True):
    f = {n: to_f64(t) for n, t in x.items()}
    o, ST = binding.gdn2_linear_fwd(d["q"], d["k"], d["v"], d["g"], d["S0"] if S0 else None)
    g = binding.gdn2_linear_bwd(d["q"], d["k"], d["v"], d["g"], d["do"], d["S0"] if S0 else None, d["dST"] if dST else None)
    torch.cuda.synchronize()
    a = {"S0": f["S0"]} if S0 else {}
    b = {"dST": f["dST"]} if dST else {}
    o_ref, ST_ref = lin.fwd(f["q"], f["k"], f["v"], f["g"], **a)
    ref = lin.bwd(f["q"], f["k"], f["v"], f["g"], f["do"], **a, **b)
    check_tokens(to_f64(o), o_ref, dtype, "o")
    check_states(to_f64(ST), ST_ref, dtype, "ST")
    for n in ("dq", "dk", "dv"):
        check_tokens(to_f64(g[n]), ref[n], dtype, n)
    check_states(to_f64(g["dS0"]), ref["dS0"], dtype, "dS0")


# lengths around the chunk borders of both paths (64, 128), one token, several chunks with a ragged end
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 2, 63, 64, 65, 127, 128, 129, 200, 256, 511])
def test_lengths(dtype, T):
    x, d = make((2, T), 2, 3, 64, 64, dtype, 100 + T)
    check_dense(x, d, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Dk", [16, 32, 64, 128])
@pytest.mark.parametrize("Dv", [16, 32, 64, 128])
def test_head_sizes(dtype, Dk, Dv):
    x, d = make((1, 300), 1, 3, Dk, Dv, dtype, Dk * 1000 + Dv)
    check_dense(x, d, dtype)


# no decay, the usual slopes, horizons of a token or less, one that is 0 in 32 bits, no memory at all
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
def test_decays(dtype, D):
    x, d = make((1, 333), 1, 8, D, D, dtype, 7, [0.0, -1e-7, -0.004, -0.5, -3.0, -20.0, -150.0, -float("inf")])
    check_dense(x, d, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("S0,dST", [(False, False), (True, False), (False, True)])
def test_missing_states_read_as_zero(dtype, S0, dST):
    x, d = make((2, 150), 2, 2, 128, 64, dtype, 8)
    check_dense(x, d, dtype, S0, dST)


# enough chunks a head and few enough heads that a sequence is cut into segments, and many heads where it is not
@pytest.mark.parametrize("dtype,B,T,H,Dk,Dv", [("bf16", 1, 5000, 2, 128, 128), ("bf16", 1, 2600, 1, 64, 32),
                                               ("bf16", 3, 300, 60, 64, 64), ("f32", 1, 2100, 2, 32, 64)])
def test_long_and_wide(dtype, B, T, H, Dk, Dv):
    x, d = make((B, T), B, H, Dk, Dv, dtype, 9, list(-np.logspace(-4, 0, H)))
    check_dense(x, d, dtype)


def test_no_tokens_hands_the_state_on():
    x, d = make((2, 0), 2, 3, 64, 64, "bf16", 10)
    o, ST = binding.gdn2_linear_fwd(d["q"], d["k"], d["v"], d["g"], d["S0"])
    g = binding.gdn2_linear_bwd(d["q"], d["k"], d["v"], d["g"], d["do"], d["S0"], d["dST"])
    assert o.shape == (2, 0, 3, 64) and torch.equal(ST, d["S0"]) and torch.equal(g["dS0"], d["dST"])
    _, ST = binding.gdn2_linear_fwd(d["q"], d["k"], d["v"], d["g"])
    assert not ST.any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [40, 3000])
def test_state_in_place(dtype, T):
    """ST may be S0 and dS0 may be dST."""
    x, d = make((1, T), 1, 2, 64, 64, dtype, 11)
    o, ST = binding.gdn2_linear_fwd(d["q"], d["k"], d["v"], d["g"], d["S0"])
    g = binding.gdn2_linear_bwd(d["q"], d["k"], d["v"], d["g"], d["do"], d["S0"], d["dST"])
    S, G = d["S0"].clone(), d["dST"].clone()
    o2, _ = binding.gdn2_linear_fwd(d["q"], d["k"], d["v"], d["g"], S, ST=S)
    g2 = binding.gdn2_linear_bwd(d["q"], d["k"], d["v"], d["g"], d["do"], d["S0"], G, grads={"dS0": G})
    assert torch.equal(S, ST) and torch.equal(o2, o) and torch.equal(G, g["dS0"])
    assert all(torch.equal(g2[n], g[n]) for n in ("dq", "dk", "dv"))


# ------------------------------------------------------------------ packed sequences

def packed_case(lengths, H, Dk, Dv, dtype, seed, tail=0):
    total = sum(lengths) + tail
    x, d = make((total,), len(lengths), H, Dk, Dv, dtype, seed)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32)
    return x, d, cu.cuda()


@pytest.mark.parametrize("dtype,Dk,Dv", [("f32", 64, 64), ("bf16", 128, 128), ("bf16", 64, 64), ("bf16", 32, 128)])
@pytest.mark.parametrize("lengths", [[100, 1, 0, 64, 37, 200, 65, 128, 0], [0], [1], [2500, 3, 700]])
def test_packed(dtype, Dk, Dv, lengths):
    H = 2
    x, d, cu = packed_case(lengths, H, Dk, Dv, dtype, 20)
    Tmax = max(lengths)
    o, ST = binding.gdn2_linear_varlen_fwd(d["q"], d["k"], d["v"], d["g"], cu, Tmax, d["S0"])
    g = binding.gdn2_linear_varlen_bwd(d["q"], d["k"], d["v"], d["g"], d["do"], cu, Tmax, d["S0"], d["dST"])
    assert binding.gdn2_device_status() == binding.GDN2_OK, binding.last_error()
    f = {n: to_f64(t) for n, t in x.items()}
    for i, n in enumerate(lengths):
        at = slice(sum(lengths[:i]), sum(lengths[:i + 1]))
        part = {m: f[m][at][None] for m in ("q", "k", "v", "do")}
        o_ref, ST_ref = lin.fwd(part["q"], part["k"], part["v"], f["g"], f["S0"][i:i + 1])
        ref = lin.bwd(part["q"], part["k"], part["v"], f["g"], part["do"], f["S0"][i:i + 1], f["dST"][i:i + 1])
        check_tokens(to_f64(o)[at][None], o_ref, dtype, ("o", i))
        check_states(to_f64(ST)[i:i + 1], ST_ref, dtype, ("ST", i))
        for m in ("dq", "dk", "dv"):
            check_tokens(to_f64(g[m])[at][None], ref[m], dtype, (m, i))
        check_states(to_f64(g["dS0"])[i:i + 1], ref["dS0"], dtype, ("dS0", i))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_packed_equals_each_sequence_alone_bit_for_bit(dtype):
    lengths, H, Dk, Dv = [130, 77, 256], 2, 64, 128
    x, d, cu = packed_case(lengths, H, Dk, Dv, dtype, 21)
    o, ST = binding.gdn2_linear_varlen_fwd(d["q"], d["k"], d["v"], d["g"], cu, max(lengths), d["S0"])
    g = binding.gdn2_linear_varlen_bwd(d["q"], d["k"], d["v"], d["g"], d["do"], cu, max(lengths), d["S0"], d["dST"])
    for i in range(len(lengths)):
        at = slice(sum(lengths[:i]), sum(lengths[:i + 1]))
        one = [d[n][at][None].contiguous() for n in ("q", "k", "v")] + [d["g"]]
        o1, ST1 = binding.gdn2_linear_fwd(*one, d["S0"][i:i + 1])
        g1 = binding.gdn2_linear_bwd(*one, d["do"][at][None].contiguous(), d["S0"][i:i + 1], d["dST"][i:i + 1])
        assert torch.equal(o[at], o1[0]) and torch.equal(ST[i:i + 1], ST1)
        assert all(torch.equal(g[n][at], g1[n][0]) for n in ("dq", "dk", "dv")) and torch.equal(g["dS0"][i:i + 1], g1["dS0"])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lengths", [[70, 129, 30], [1500, 1, 900]])
def test_a_neighbour_full_of_nan_changes_nothing_and_rows_behind_stay(dtype, lengths):
    H, Dk, Dv, tail = 2, 64, 64, 40
    x, d, cu = packed_case(lengths, H, Dk, Dv, dtype, 22, tail)
    args = lambda: (d["q"], d["k"], d["v"], d["g"])

    def run():
        mark = lambda t: torch.full_like(t, 7.0)
        o, ST = binding.gdn2_linear_varlen_fwd(*args(), cu, max(lengths), d["S0"], o=mark(d["v"]))
        g = binding.gdn2_linear_varlen_bwd(*args(), d["do"], cu, max(lengths), d["S0"], d["dST"],
                                           grads={"dq": mark(d["q"]), "dk": mark(d["k"]), "dv": mark(d["v"])})
        return [o, g["dq"], g["dk"], g["dv"]], [ST, g["dS0"]]

    tokens, states = run()
    for t in tokens:
        assert bool((t[sum(lengths):] == 7.0).all())
    bad = slice(lengths[0], lengths[0] + lengths[1])
    for n in ("q", "k", "v", "do"):
        d[n][bad] = float("nan")
        d[n][sum(lengths):] = float("inf")
    tokens2, states2 = run()
    keep = [slice(0, lengths[0]), slice(lengths[0] + lengths[1], sum(lengths))]
    for a, b in zip(tokens, tokens2):
        assert all(torch.equal(a[s], b[s]) for s in keep) and bool((b[sum(lengths):] == 7.0).all())
        assert bool(b[bad].isnan().any())
    for a, b in zip(states, states2):
        assert torch.equal(a[0], b[0]) and torch.equal(a[2], b[2])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_inconsistent_lengths_are_reported(dtype):
    H, D = 2, 64
    x, d, cu = packed_case([70, 30], H, D, D, dtype, 23)
    binding.gdn2_device_status()
    run = lambda cu, Tmax: binding.gdn2_linear_varlen_fwd(d["q"], d["k"], d["v"], d["g"], cu, Tmax, d["S0"])
    o, ST = run(cu, 64)      # cut at 64 tokens
    assert binding.gdn2_device_status() == binding.GDN2_ERR_INVALID and "Tmax" in binding.last_error()
    f = {n: to_f64(t) for n, t in x.items()}
    o_ref, ST_ref = lin.fwd(*(f[n][None, :64] for n in "qkv"), f["g"], f["S0"][:1])
    check_tokens(to_f64(o)[None, :64], o_ref, dtype, "cut o")
    check_states(to_f64(ST)[:1], ST_ref, dtype, "cut ST")
    for bad in ([0, 70, 200], [0, 70, 20], [-5, 70, 100]):
        _, ST = run(torch.tensor(bad, dtype=torch.int32).cuda(), 100)
        assert binding.gdn2_device_status() == binding.GDN2_ERR_INVALID and "cu_seqlens" in binding.last_error()
        dropped = 0 if bad[0] < 0 else 1
        assert torch.equal(ST[dropped], d["S0"][dropped])
    assert binding.gdn2_device_status() == binding.GDN2_OK


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_no_room_for_tokens_hands_the_states_on_and_reports(dtype):
    x, d, cu = packed_case([5, 0], 2, 64, 64, dtype, 24)
    args = (d["q"], d["k"], d["v"], d["g"])
    empty = torch.zeros(3, dtype=torch.int32, device="cuda")
    for lengths, status in ((empty, binding.GDN2_OK), (cu, binding.GDN2_ERR_INVALID)):
        o, ST = binding.gdn2_linear_varlen_fwd(*args, lengths, 0, d["S0"], o=torch.full_like(d["v"], 7.0))
        g = binding.gdn2_linear_varlen_bwd(*args, d["do"], lengths, 0, d["S0"], d["dST"])
        assert binding.gdn2_device_status() == status
        assert torch.equal(ST, d["S0"]) and torch.equal(g["dS0"], d["dST"]) and bool((o == 7.0).all())


# a state that grows: a head's 128-token power stays finite in 32 bits (e^0.3 per token: e^38)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [100, 128])
def test_growing_states(dtype, T):
    x, d = make((1, T), 1, 3, 64, 64, dtype, 25, [0.3, 0.05, 0.0])
    check_dense(x, d, dtype)


# more segments than a block has items, and a bound on the length far above the lengths
def test_many_segments_and_a_loose_bound():
    lengths = [9000, 0, 333, 129]
    x, d, cu = packed_case(lengths, 1, 64, 64, "bf16", 26)
    args = (d["q"], d["k"], d["v"], d["g"])
    o, ST = binding.gdn2_linear_varlen_fwd(*args, cu, 60000, d["S0"])
    g = binding.gdn2_linear_varlen_bwd(*args, d["do"], cu, 60000, d["S0"], d["dST"])
    assert binding.gdn2_device_status() == binding.GDN2_OK
    f = {n: to_f64(t) for n, t in x.items()}
    for i in range(len(lengths)):
        at = slice(sum(lengths[:i]), sum(lengths[:i + 1]))
        part = {m: f[m][at][None] for m in ("q", "k", "v", "do")}
        o_ref, ST_ref = lin.fwd(part["q"], part["k"], part["v"], f["g"], f["S0"][i:i + 1])
        ref = lin.bwd(part["q"], part["k"], part["v"], f["g"], part["do"], f["S0"][i:i + 1], f["dST"][i:i + 1])
        check_tokens(to_f64(o)[at][None], o_ref, "bf16", ("o", i))
        check_states(to_f64(ST)[i:i + 1], ST_ref, "bf16", ("ST", i))
        for m in ("dq", "dk", "dv"):
            check_tokens(to_f64(g[m])[at][None], ref[m], "bf16", (m, i))
        check_states(to_f64(g["dS0"])[i:i + 1], ref["dS0"], "bf16", ("dS0", i))


# ------------------------------------------------------------------ the single-token step

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Dk,Dv", [(16, 16), (16, 128), (32, 64), (64, 32), (128, 16), (128, 128), (64, 128)])
@pytest.mark.parametrize("B", [1, 3, 40])
def test_step(dtype, Dk, Dv, B):
    H, pool = 8, B + 5
    x, d = make((B,), pool, H, Dk, Dv, dtype, 30 + B, [0.0, -0.01, -0.1, -1.0, -5.0, -50.0, -150.0, -float("inf")])
    slots = torch.randperm(pool, generator=torch.Generator().manual_seed(B))[:B].to(torch.int32)
    if B > 1:
        slots[1] = -1
    S = d["S0"].clone()
    o = binding.gdn2_linear_decode_step(d["q"], d["k"], d["v"], d["g"], S, slots.cuda())
    f = {n: to_f64(t) for n, t in x.items()}
    want = f["S0"].copy()
    got_S, got = to_f64(S), to_f64(o)
    for b, s in enumerate(slots.tolist()):
        if s < 0:
            assert not got[b].any()
            continue
        o_ref, S_ref = lin.fwd(f["q"][b][None, None], f["k"][b][None, None], f["v"][b][None, None], f["g"], want[s:s + 1])
        before, want[s] = want[s].copy(), S_ref[0]
        # o_j sums Dk products q_i S_ij whose terms may cancel, so its error goes by the sum of their sizes: Dk roundings
        # of the sum, and 4 of each term (the product, a S + k v's two, the decay factor's), each 2^-24 of that sum at most
        size = np.einsum("hk,hkv->hv", np.abs(f["q"][b]), np.exp(f["g"])[:, None, None] * np.abs(before) +
                         np.abs(f["k"][b])[..., None] * np.abs(f["v"][b])[:, None, :])
        allowed = (Dk + 4) * 2.0 ** -24 * size + (2.0 ** -8 * np.abs(o_ref[0, 0]) if dtype == "bf16" else 0.0)
        assert np.all(np.abs(got[b] - o_ref[0, 0]) <= allowed), b
        assert worst_head_rel_l2(got_S[s][None], S_ref, state=True) <= 1e-6, b
    untouched = [i for i in range(pool) if i not in slots.tolist()]
    assert torch.equal(S[untouched], d["S0"][untouched])


def test_step_without_slots_and_bad_slots():
    x, d = make((3,), 5, 2, 64, 64, "bf16", 31)
    args = (d["q"], d["k"], d["v"], d["g"])
    S = d["S0"].clone()
    o = binding.gdn2_linear_decode_step(*args, S)
    S2 = d["S0"].clone()
    o2 = binding.gdn2_linear_decode_step(*args, S2, torch.arange(3, dtype=torch.int32).cuda())
    assert torch.equal(o, o2) and torch.equal(S, S2) and torch.equal(S[3:], d["S0"][3:])
    assert binding.gdn2_device_status() == binding.GDN2_OK
    for slots, alive in (([4, 9, 0], [0, 2]), ([2, 2, 1], [0, 2]), ([1, 3, 1], [0, 1]), ([5, -1, 2], [2])):
        S3 = d["S0"].clone()
        o3 = binding.gdn2_linear_decode_step(*args, S3, torch.tensor(slots, dtype=torch.int32).cuda())
        assert binding.gdn2_device_status() == binding.GDN2_ERR_INVALID and "slots" in binding.last_error()
        for b in range(3):
            assert bool(o3[b].any()) == (b in alive), (slots, b)
        named = [slots[b] for b in alive]
        for i in range(5):
            assert torch.equal(S3[i], d["S0"][i]) == (i not in named), (slots, i)
    assert binding.gdn2_device_status() == binding.GDN2_OK


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_prompt_then_steps_equals_the_whole_sequence(dtype):
    """A packed prefill into a pool of states, then single tokens, against one long sequence a request."""
    lengths, steps, H, Dk, Dv = [200, 1, 77], 5, 4, 128, 64
    g = -torch.exp2(-8.0 * torch.arange(1, H + 1) / H)
    whole = [make((1, n + steps), 1, H, Dk, Dv, dtype, 40 + i)[0] for i, n in enumerate(lengths)]
    cat = lambda n: torch.cat([w[n][0, :l] for w, l in zip(whole, lengths)]).cuda()
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32).cuda()
    gd = g.cuda()
    o, ST = binding.gdn2_linear_varlen_fwd(cat("q"), cat("k"), cat("v"), gd, cu, max(lengths))
    pool = torch.zeros(6, H, Dk, Dv, device="cuda")
    slots = torch.tensor([4, 0, 3], dtype=torch.int32).cuda()
    pool[slots.long()] = ST
    out = []
    for s in range(steps):
        at = [torch.stack([w[n][0, l + s] for w, l in zip(whole, lengths)]).cuda() for n in "qkv"]
        out.append(binding.gdn2_linear_decode_step(*at, gd, pool, slots))
    for i, (w, n) in enumerate(zip(whole, lengths)):
        f = {m: to_f64(w[m]) for m in "qkv"}
        o_ref, S_ref = lin.fwd(f["q"], f["k"], f["v"], to_f64(g))
        got = np.concatenate([to_f64(o)[sum(lengths[:i]):sum(lengths[:i + 1])], np.stack([to_f64(t[i]) for t in out])])
        check_tokens(got[None], o_ref, dtype, i)
        check_states(to_f64(pool[int(slots[i])])[None], S_ref, dtype, i)


@pytest.mark.parametrize("dtype,packed", [("f32", False), ("bf16", False), ("bf16", True)])
def test_autograd(dtype, packed):
    lengths = [90, 130]
    x, d, cu = packed_case(lengths, 2, 64, 64, dtype, 50, tail=6)
    if not packed:
        x, d = make((2, 130), 2, 2, 64, 64, dtype, 51)
    leaves = [d[n].requires_grad_() for n in ("q", "k", "v", "S0")]
    o, ST = binding.decay_linear_attention(*leaves[:3], d["g"], leaves[3], *((cu, max(lengths)) if packed else ()))
    got = torch.autograd.grad((o * d["do"]).sum() + (ST * d["dST"]).sum(), leaves)
    det = [t.detach() for t in leaves]
    if packed:
        want = binding.gdn2_linear_varlen_bwd(*det[:3], d["g"], d["do"], cu, max(lengths), det[3], d["dST"])
        n = sum(lengths)
        assert not o[n:].any() and all(not t[n:].any() for t in got[:3])
    else:
        want = binding.gdn2_linear_bwd(*det[:3], d["g"], d["do"], det[3], d["dST"])
        n = None
    for t, m in zip(got, ("dq", "dk", "dv")):
        assert torch.equal(t[:n], want[m][:n]), m
    assert torch.equal(got[3], want["dS0"])
    # only the final state is used; only q needs a gradient
    o, ST = binding.decay_linear_attention(*leaves[:3], d["g"], leaves[3], *((cu, max(lengths)) if packed else ()))
    (dk,) = torch.autograd.grad(ST.sum(), [leaves[1]])
    assert bool(dk.isfinite().all()) and bool(dk.any())


def test_second_derivatives_are_refused():
    x, d = make((1, 40), 1, 2, 64, 64, "f32", 52)
    q = d["q"].requires_grad_()
    o, _ = binding.decay_linear_attention(q, d["k"], d["v"], d["g"])
    (dq,) = torch.autograd.grad((o * o).sum(), q, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        dq.sum().backward()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_another_stream_a_graph_and_two_at_once(dtype):
    x, d = make((1, 1500), 1, 2, 128, 128, dtype, 60)
    y, e = make((1, 700), 1, 2, 128, 128, dtype, 61)
    call = lambda t: (lambda o, g: [*o, g["dq"], g["dk"], g["dv"], g["dS0"]])(
        binding.gdn2_linear_fwd(t["q"], t["k"], t["v"], t["g"], t["S0"]),
        binding.gdn2_linear_bwd(t["q"], t["k"], t["v"], t["g"], t["do"], t["S0"], t["dST"]))
    want, want2 = call(d), call(e)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s, t in zip(streams, (d, e)):
        with torch.cuda.stream(s):
            for _ in range(3):
                r = call(t)
            got.append(r)
    torch.cuda.synchronize()
    for a, b in zip(got, (want, want2)):
        assert all(torch.equal(p, q) for p, q in zip(a, b))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = call(d)
    for n in ("q", "k", "v", "do"):
        d[n].copy_(torch.flip(d[n], (1,)).contiguous())
    graph.replay()
    fresh = call(d)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(held, fresh))
    assert not torch.equal(held[0], want[0])


def test_step_in_a_graph():
    x, d = make((4,), 6, 4, 128, 128, "bf16", 62)
    S, slots = d["S0"].clone(), torch.tensor([1, 5, -1, 2], dtype=torch.int32).cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = binding.gdn2_linear_decode_step(d["q"], d["k"], d["v"], d["g"], S, slots)
    ref = S.clone()
    for new in ([1, 5, -1, 2], [0, -1, 3, 5]):
        slots.copy_(torch.tensor(new, dtype=torch.int32))
        graph.replay()
        want = binding.gdn2_linear_decode_step(d["q"], d["k"], d["v"], d["g"], ref, slots)
        assert torch.equal(o, want) and torch.equal(S, ref)
