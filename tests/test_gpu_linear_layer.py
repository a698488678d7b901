"""The layer of projections, query/key norm with rotation and linear attention, forward, backward and token by token,
against the same layer written out in 64 bits.

Tolerances (relative L2). fp32: a projection's sum of up to 256 products 1e-6, the norm with rotation 1e-6, linear
attention 2e-6; the products of q and k and of P and v take two of them each and the way back as many again: y and S_T
1e-5, gradients 2e-5. bf16: half a step, 2^-8, for every rounding a value passes: q and k twice each (projection, rotation),
v, the pairs' weights, the copy of the state, o and y once: 9 * 2^-8. The gradients add those of dy's way: do, dq, dk, dv,
the three before the projections and the gradient itself: 16 * 2^-8.
"""
import numpy as np
import pytest
import torch

from conftest import rel_l2
from linear_attention_delta_gdn_b200 import binding

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
TOL_Y = {"f32": 1e-5, "bf16": 9 * 2.0 ** -8}
TOL_G = {"f32": 2e-5, "bf16": 16 * 2.0 ** -8}
PARAMS = ("W_qk", "W_v", "W_out", "q_weight", "k_weight")


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from linear_attention_delta_gdn_b200 import build
    build.build()
    binding.gdn2_device_status()
    yield
    assert binding.gdn2_device_status() == binding.GDN2_OK, binding.last_error()


def layer_of(dtype, d_model, H, Dk, Dv, **kw):
    from linear_attention_delta_gdn_b200.layer import DecayLinearAttentionLayer
    torch.manual_seed(3)
    layer = DecayLinearAttentionLayer(d_model, H, Dk, Dv, dtype=DT[dtype], device="cuda", **kw)
    with torch.no_grad():
        for w in (layer.q_weight, layer.k_weight):
            w.mul_(1 + 0.2 * torch.randn_like(w))
    return layer


def written_out(layer, w, x, S0, positions):
    """One sequence x [T, d_model] in 64 bits on the CPU with parameters w; positions [axes, T]. Returns (y, S_T)."""
    H, Dk, Dv, T = layer.H, layer.Dk, layer.Dv, x.shape[0]
    q, k = (x @ w["W_qk"]).view(T, 2, H, Dk).unbind(1)
    v = (x @ w["W_v"]).view(T, H, Dv)
    f = layer.inv_freq.double().cpu()
    axes = torch.zeros(len(f), dtype=torch.long) if layer.axes is None else layer.axes.long().cpu()
    t = (positions.double().cpu()[axes] * f[:, None]).T[:, None]
    n = len(f)

    def turned(z, weight):
        z = z / torch.sqrt((z * z).mean(-1, keepdim=True) + layer.eps) * weight
        a, b = z[..., :n], z[..., n:2 * n]
        return torch.cat([a * t.cos() - b * t.sin(), a * t.sin() + b * t.cos(), z[..., 2 * n:]], -1)

    q, k = turned(q, w["q_weight"]), turned(k, w["k_weight"])
    a = torch.exp(layer.log_decay.double().cpu())[:, None, None]
    S, o = S0, []
    for i in range(T):
        S = a * S + k[i, :, :, None] * v[i, :, None, :]
        o.append((S * q[i, :, :, None]).sum(1))
    return torch.stack(o).flatten(1) @ w["W_out"], S


CASES = {"dense": dict(d_model=96, H=3, Dk=64, Dv=64), "wide": dict(d_model=64, H=2, Dk=128, Dv=32, pairs=20),
         "axes": dict(d_model=64, H=2, Dk=64, Dv=128, sections=(8, 12, 12)),
         "packed": dict(d_model=80, H=2, Dk=128, Dv=128), "packed-axes": dict(d_model=64, H=1, Dk=32, Dv=16, sections=(3, 5))}


def set_up(name, dtype):
    layer = layer_of(dtype, **CASES[name])
    g = torch.Generator().manual_seed(11)
    lengths = [150, 1, 0, 67] if "packed" in name else [133, 133]
    tail = 5 if "packed" in name else 0
    n, total, A = len(lengths), sum(lengths) + tail, 1 if layer.axes is None else int(layer.axes.max()) + 1
    x = torch.randn(total, layer.d_model, generator=g).to(DT[dtype])
    S0 = torch.randn(n, layer.H, layer.Dk, layer.Dv, generator=g) * 0.1
    pos = torch.randint(0, 500, (A, total), generator=g, dtype=torch.int32)
    dy = torch.randn(total, layer.d_model, generator=g).to(DT[dtype])
    dST = torch.randn(S0.shape, generator=g) * 0.1
    return layer, lengths, x, S0, pos, dy, dST


def run(layer, name, lengths, x, S0, pos):
    """The layer's call: (y [Ttot, d_model], S_T)."""
    p = pos if layer.axes is not None else pos[0]
    if "packed" in name:
        cu = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32).cuda()
        return layer(x, S0, p.contiguous(), cu, max(lengths))
    B, T = len(lengths), lengths[0]
    y, ST = layer(x.view(B, T, -1), S0, p.reshape(*p.shape[:-1], B, T))
    return y.flatten(0, 1), ST


def loss64(layer, w, lengths, x, S0, pos, dy, dST):
    """<dy, y> + <dST, S_T>, y and S_T, in 64 bits."""
    at, ys, Ss = 0, [], []
    for i, n in enumerate(lengths):
        y, S = written_out(layer, w, x[at:at + n], S0[i], pos[:, at:at + n]) if n else (x[:0] @ w["W_qk"][:, :0] @ w["W_out"][:0], S0[i])
        ys.append(y)
        Ss.append(S)
        at += n
    y, S = torch.cat(ys), torch.stack(Ss)
    return (y * dy[:at]).sum() + (S * dST).sum(), y, S


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("name", list(CASES))
def test_layer_and_its_gradients(name, dtype):
    layer, lengths, x, S0, pos, dy, dST = set_up(name, dtype)
    n = sum(lengths)
    xd, Sd = x.cuda().requires_grad_(), S0.cuda().requires_grad_()
    y, ST = run(layer, name, lengths, xd, Sd, pos.cuda())
    ((y * dy.cuda())[:n].float().sum() + (ST * dST.cuda()).sum()).backward()
    w = {m: getattr(layer, m).detach().double().cpu().requires_grad_() for m in PARAMS}
    x64, S64 = x.double().requires_grad_(), S0.double().requires_grad_()
    L, y_ref, S_ref = loss64(layer, w, lengths, x64, S64, pos, dy.double(), dST.double())
    L.backward()
    far = lambda a, b: rel_l2(a.detach().double().cpu().numpy(), b.detach().numpy())
    assert far(y[:n], y_ref) <= TOL_Y[dtype] and far(ST, S_ref) <= TOL_Y[dtype]
    assert not y[n:].any()   # rows behind the last sequence
    for m in PARAMS:
        assert far(getattr(layer, m).grad, w[m].grad) <= TOL_G[dtype], m
    assert far(xd.grad, x64.grad) <= TOL_G[dtype] and far(Sd.grad, S64.grad) <= TOL_G[dtype]


@pytest.mark.parametrize("name", ["dense", "packed-axes"])
def test_gradients_against_differences(name):
    """The loss's change along a direction of all parameters and inputs, in 64 bits, against the gradients' product with it.
    The third derivative over a step of 1e-5 leaves about 1e-8 of it; the product is off by 2e-5 of the gradients' length times
    the direction's."""
    layer, lengths, x, S0, pos, dy, dST = set_up(name, "f32")
    n = sum(lengths)
    xd, Sd = x.cuda().requires_grad_(), S0.cuda().requires_grad_()
    y, ST = run(layer, name, lengths, xd, Sd, pos.cuda())
    ((y * dy.cuda())[:n].sum() + (ST * dST.cuda()).sum()).backward()
    g = torch.Generator().manual_seed(5)
    leaves = {m: getattr(layer, m) for m in PARAMS} | {"x": xd, "S0": Sd}
    v = {m: torch.randn(t.shape, generator=g, dtype=torch.float64) for m, t in leaves.items()}
    at = lambda s: {m: t.detach().double().cpu() + s * v[m] for m, t in leaves.items()}

    def loss(s):
        p = at(s)
        return float(loss64(layer, p, lengths, p["x"], p["S0"], pos, dy.double(), dST.double())[0])

    h = 1e-5
    slope = (loss(h) - loss(-h)) / (2 * h)
    grads = {m: t.grad.double().cpu() for m, t in leaves.items()}
    got = sum(float((grads[m] * v[m]).sum()) for m in leaves)
    room = sum(2e-5 * float(grads[m].norm() * v[m].norm()) for m in leaves) + 1e-6 * abs(slope)
    assert abs(got - slope) <= room, (got, slope, room)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_prompts_then_steps(dtype):
    """A packed prefill, its states into a pool, then single tokens, against each whole sequence written out."""
    layer = layer_of(dtype, 64, 2, 128, 64)
    g = torch.Generator().manual_seed(2)
    lengths, steps = [140, 1, 30], 4
    xs = [torch.randn(n + steps, 64, generator=g).to(DT[dtype]) for n in lengths]
    starts = [0, 70000, 12]
    pos = [torch.arange(s, s + len(x), dtype=torch.int32) for s, x in zip(starts, xs)]
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32).cuda()
    with torch.no_grad():
        y, ST = layer(torch.cat([x[:n] for x, n in zip(xs, lengths)]).cuda(), None,
                      torch.cat([p[:n] for p, n in zip(pos, lengths)]).cuda(), cu, max(lengths))
    pool = torch.zeros(5, 2, 128, 64, device="cuda")
    slots = torch.tensor([3, 0, -1, 4], dtype=torch.int32).cuda()   # an idle row among them
    pool[slots[slots >= 0].long()] = ST
    rows = [0, 1, None, 2]
    out = []
    for s in range(steps):
        x = torch.stack([torch.zeros(64, dtype=DT[dtype]) if r is None else xs[r][lengths[r] + s] for r in rows]).cuda()
        p = torch.tensor([0 if r is None else int(pos[r][lengths[r] + s]) for r in rows], dtype=torch.int32).cuda()
        out.append(layer.step(x, p, pool, slots))
    w = {m: getattr(layer, m).detach().double().cpu() for m in PARAMS}
    for i, r in enumerate(rows):
        if r is None:
            assert not any(o[i].any() for o in out)
            continue
        y_ref, S_ref = written_out(layer, w, xs[r].double(), torch.zeros(2, 128, 64, dtype=torch.float64), pos[r][None])
        a = int(cu[r])
        got = torch.cat([y[a:a + lengths[r]], torch.stack([o[i] for o in out])])
        assert rel_l2(got.double().cpu().numpy(), y_ref.numpy()) <= TOL_Y[dtype]
        assert rel_l2(pool[slots[i]].double().cpu().numpy(), S_ref.numpy()) <= TOL_Y[dtype]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_training_step_in_a_graph(dtype):
    """Forward and backward captured after a warm-up on the capturing stream, replayed on new inputs."""
    layer = layer_of(dtype, 96, 2, 64, 32)
    x = torch.randn(2, 150, 96, device="cuda").to(DT[dtype])
    pos = torch.arange(150, dtype=torch.int32, device="cuda").expand(2, 150).contiguous()
    S0 = torch.randn(2, 2, 64, 32, device="cuda")
    dy = torch.randn(2, 150, 96, device="cuda").to(DT[dtype])

    def step():
        y, ST = layer(x, S0, pos)
        return [y.detach(), ST.detach(), *torch.autograd.grad((y * dy).sum() + ST.sum(), list(layer.parameters()))]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        held = step()
    for seed in (1, 2):
        torch.manual_seed(seed)
        x.copy_(torch.randn(2, 150, 96))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        for a, b in zip(got, step()):
            assert torch.equal(a, b)
