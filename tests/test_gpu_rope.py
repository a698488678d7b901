"""The query/key norm with rotation on the GPU against the fp64 oracle.

Tolerances (relative L2): the arithmetic is fp32, one output rounding: bf16 2^-8; fp32 1e-6 (the norm's sum of 128
terms is a tree of 7 levels, the rotation three roundings, sine and cosine 2 ulp). Weight gradients (fp32) are sums
over R rows whose terms have any sign: 1e-6 times sqrt(R / 100) at most here, 1e-5.
"""
import numpy as np
import pytest
import torch

from conftest import rel_l2
from linear_attention_delta_gdn_b200 import binding
from linear_attention_delta_gdn_b200.inputs import to_f64
from oracle import linear as lin

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
TOL = {"f32": 1e-6, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from linear_attention_delta_gdn_b200 import build
    build.build()
    binding.gdn2_device_status()
    yield
    assert binding.gdn2_device_status() == binding.GDN2_OK, binding.last_error()


def check(dtype, B, T, Hq, Hk, D, pairs, num_axes=1, interleaved=False, norm=True, weights=True, far=0, pos64=False, seed=1):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)
    q, k = (r(B, T, Hq, D) * 3).to(DT[dtype]), (r(B, T, Hk, D) * 0.3).to(DT[dtype])
    dyq, dyk = r(B, T, Hq, D).to(DT[dtype]), r(B, T, Hk, D).to(DT[dtype])
    pos = torch.randint(-5, 6, (num_axes, B, T), generator=g) + far
    pos = pos.to(torch.int64 if pos64 else torch.int32)
    f = torch.exp(-9.2 * torch.arange(pairs) / pairs).float()
    axes = torch.randint(0, num_axes, (pairs,), generator=g, dtype=torch.int32)
    wq, wk = (1 + 0.2 * r(D), 1 + 0.2 * r(D)) if norm and weights else (None, None)
    cu = lambda t: None if t is None else t.cuda()
    kw = dict(axes=cu(axes) if num_axes > 1 else None, q_weight=cu(wq), k_weight=cu(wk), eps=1e-6 if norm else None,
              interleaved=interleaved)
    p = pos.cuda() if num_axes > 1 else pos[0].cuda()
    qo, ko = binding.gdn2_qk_norm_rope_fwd(q.cuda(), k.cuda(), p, f.cuda(), **kw)
    d = binding.gdn2_qk_norm_rope_bwd(q.cuda(), k.cuda(), dyq.cuda(), dyk.cuda(), p, f.cuda(), **kw)
    ax = axes.numpy() if num_axes > 1 else np.zeros(pairs, int)
    for x, y, w, out, dx, dw in ((q, dyq, wq, qo, d["dq"], d["dq_weight"]), (k, dyk, wk, ko, d["dk"], d["dk_weight"])):
        a = dict(weight=None if w is None else to_f64(w), eps=kw["eps"], interleaved=interleaved)
        assert rel_l2(to_f64(out), lin.rope_fwd(to_f64(x), pos.numpy(), f.numpy(), ax, **a)) <= TOL[dtype]
        dx_ref, dw_ref = lin.rope_bwd(to_f64(x), to_f64(y), pos.numpy(), f.numpy(), ax, **a)
        assert rel_l2(to_f64(dx), dx_ref) <= TOL[dtype]
        if w is not None:
            assert rel_l2(to_f64(dw), dw_ref) <= 1e-5
        else:
            assert dw is None


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,pairs", [(16, 8), (16, 2), (16, 1), (32, 16), (32, 7), (64, 32), (64, 12), (128, 64), (128, 32),
                                     (128, 61), (128, 16)])
def test_head_sizes_and_pairs(dtype, interleaved, D, pairs):
    check(dtype, 2, 9, 6, 2, D, pairs, interleaved=interleaved)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,Hq,Hk", [(1, 1, 1, 1), (64, 1, 16, 4), (1, 1301, 3, 1), (3, 777, 5, 5), (2, 4000, 2, 2)])
def test_shapes(dtype, B, T, Hq, Hk):
    check(dtype, B, T, Hq, Hk, 64, 32)


@pytest.mark.parametrize("num_axes", [2, 3, 4])
@pytest.mark.parametrize("pos64", [False, True])
def test_axes(num_axes, pos64):
    check("f32", 2, 50, 4, 2, 128, 64, num_axes=num_axes, pos64=pos64)


@pytest.mark.parametrize("norm,weights", [(False, False), (True, False)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_without_norm_or_weight(dtype, norm, weights):
    check(dtype, 2, 33, 4, 2, 128, 64, norm=norm, weights=weights)


@pytest.mark.parametrize("far,pos64", [(1 << 20, False), ((1 << 31) - 10, False), (-(1 << 30), False), (1 << 40, True)])
def test_far_positions(far, pos64):
    """The angle keeps its error at any position (pos * 2^-64 turns: 4e-7 rad at 2^40, below the bf16 rounding and the
    weight gradients' 1e-5 there)."""
    check("bf16" if pos64 else "f32", 1, 16, 2, 2, 64, 32, far=far, pos64=pos64)


def test_zero_rows_and_no_tokens():
    z = torch.zeros(1, 3, 2, 64, device="cuda")
    pos, f, w = torch.arange(3, dtype=torch.int32, device="cuda")[None], torch.rand(32).cuda(), torch.ones(64).cuda()
    qo, ko = binding.gdn2_qk_norm_rope_fwd(z, z, pos, f, q_weight=w, k_weight=w)
    d = binding.gdn2_qk_norm_rope_bwd(z, z, z + 1, z + 1, pos, f, q_weight=w, k_weight=w)
    assert not qo.any() and bool(d["dq"].isfinite().all()) and not d["dq_weight"].any()
    e = torch.zeros(2, 0, 2, 64, device="cuda")
    pos = torch.zeros(2, 0, dtype=torch.int32, device="cuda")
    qo, _ = binding.gdn2_qk_norm_rope_fwd(e, e, pos, f, q_weight=w, k_weight=w)
    d = binding.gdn2_qk_norm_rope_bwd(e, e, e, e, pos, f, q_weight=w, k_weight=w)
    assert qo.shape == e.shape and not d["dq_weight"].any() and not d["dk_weight"].any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_slices_of_a_projection_and_in_place(dtype):
    B, T, Hq, Hk, D = 2, 19, 4, 2, 64
    z = torch.randn(B, T, (Hq + 2 * Hk) * D, device="cuda").to(DT[dtype])
    q, k = z[..., :Hq * D].view(B, T, Hq, D), z[..., Hq * D:(Hq + Hk) * D].view(B, T, Hk, D)
    pos, f, w = torch.arange(T, device="cuda").expand(B, T).contiguous(), torch.rand(32).cuda(), torch.rand(64).cuda()
    dq, dk = torch.randn(B, T, Hq, D, device="cuda").to(DT[dtype]), torch.randn(B, T, Hk, D, device="cuda").to(DT[dtype])
    a = dict(q_weight=w, k_weight=w)
    got = binding.gdn2_qk_norm_rope_fwd(q, k, pos, f, **a)
    want = binding.gdn2_qk_norm_rope_fwd(q.contiguous(), k.contiguous(), pos, f, **a)
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    got, ref = (binding.gdn2_qk_norm_rope_bwd(*x, dq, dk, pos, f, **a) for x in ((q, k), (q.contiguous(), k.contiguous())))
    assert all(torch.equal(got[n], ref[n]) for n in got)
    qc, kc = q.contiguous(), k.contiguous()
    binding.gdn2_qk_norm_rope_fwd(qc, kc, pos, f, q_out=qc, k_out=kc, **a)
    assert torch.equal(qc, want[0]) and torch.equal(kc, want[1])


def test_an_axis_outside_turns_nothing_and_is_reported():
    x, w = torch.randn(1, 5, 2, 64, device="cuda"), None
    pos, f = torch.arange(1, 11, dtype=torch.int32, device="cuda").view(2, 1, 5), torch.ones(32).cuda()
    axes = torch.zeros(32, dtype=torch.int32, device="cuda")
    axes[3], axes[7] = 2, -1
    qo, _ = binding.gdn2_qk_norm_rope_fwd(x, x, pos, f, axes, eps=None)
    assert binding.gdn2_device_status() == binding.GDN2_ERR_INVALID and "axes" in binding.last_error()
    for c in (3, 35, 7, 39):
        assert torch.equal(qo[..., c], x[..., c])
    assert not torch.equal(qo[..., 4], x[..., 4])
    assert binding.gdn2_device_status() == binding.GDN2_OK


def test_autograd_and_graph():
    B, T, Hq, Hk, D = 2, 40, 4, 2, 128
    g = torch.Generator().manual_seed(5)
    r = lambda *s: torch.randn(s, generator=g).cuda()
    q, k, wq, wk = r(B, T, Hq, D).requires_grad_(), r(B, T, Hk, D).requires_grad_(), r(D).requires_grad_(), r(D).requires_grad_()
    pos, f = torch.arange(T, device="cuda").expand(B, T).contiguous(), torch.rand(48, generator=g).cuda()
    dq, dk = r(B, T, Hq, D), r(B, T, Hk, D)
    qo, ko = binding.qk_norm_rope(q, k, pos, f, q_weight=wq, k_weight=wk)
    got = torch.autograd.grad((qo * dq).sum() + (ko * dk).sum(), (q, k, wq, wk))
    det = [t.detach() for t in (q, k, wq, wk)]
    call = lambda: binding.gdn2_qk_norm_rope_bwd(*det[:2], dq, dk, pos, f, q_weight=det[2], k_weight=det[3])
    want = call()
    for t, n in zip(got, ("dq", "dk", "dq_weight", "dk_weight")):
        assert torch.equal(t, want[n]), n
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = call()
    dq.mul_(-1.5)
    graph.replay()
    fresh = call()
    assert all(torch.equal(held[n], fresh[n]) for n in held) and not torch.equal(held["dq"], want["dq"])
