"""Linear attention with a decay per head and the query/key norm with rotation, without a GPU: the oracle's gradients
against differences, the identity that makes the backward three forward passes, workspace sizes, and the refusals of
the C entry points and of the binding (nothing is launched for any of them)."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import linear as lin

P = 1 << 20   # an address that passes the checks; every call here is refused before anything could read it


@pytest.fixture(scope="module")
def L():
    from linear_attention_delta_gdn_b200 import build, binding
    build.build()
    return binding.lib()


# ------------------------------------------------------------------ the oracle

@pytest.mark.parametrize("T", [1, 5])
def test_oracle_gradients_against_differences(T):
    rng = np.random.default_rng(3)
    B, H, Dk, Dv = 2, 2, 3, 4
    x = {"q": rng.normal(size=(B, T, H, Dk)), "k": rng.normal(size=(B, T, H, Dk)), "v": rng.normal(size=(B, T, H, Dv)),
         "S0": rng.normal(size=(B, H, Dk, Dv))}
    g = np.array([-0.3, -1.1])
    do, dST = rng.normal(size=(B, T, H, Dv)), rng.normal(size=(B, H, Dk, Dv))

    def loss():
        o, S = lin.fwd(x["q"], x["k"], x["v"], g, x["S0"])
        return (o * do).sum() + (S * dST).sum()

    got = lin.bwd(x["q"], x["k"], x["v"], g, do, x["S0"], dST)
    h = 1e-6   # the loss is a polynomial of degree 3 at most: a central difference is exact but for rounding
    for n in x:
        for i in np.ndindex(x[n].shape):
            keep = x[n][i]
            x[n][i] = keep + h
            up = loss()
            x[n][i] = keep - h
            down = loss()
            x[n][i] = keep
            assert abs((up - down) / (2 * h) - got["d" + n][i]) < 1e-7, (n, i)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_rotation_oracle_gradients_against_differences(interleaved, norm):
    rng = np.random.default_rng(4)
    B, T, H, D, pairs = 1, 2, 2, 8, 3
    x, dy, w = rng.normal(size=(B, T, H, D)), rng.normal(size=(B, T, H, D)), rng.normal(size=D)
    pos, f, axes = rng.integers(0, 50, (2, B, T)), rng.random(pairs).astype(np.float32), np.array([0, 1, 1])
    kw = dict(weight=w if norm else None, eps=1e-6 if norm else None, interleaved=interleaved)
    dx, dw = lin.rope_bwd(x, dy, pos, f, axes, **kw)
    h = 1e-6
    for arr, want in ((x, dx),) + (((w, dw),) if norm else ()):
        for i in np.ndindex(arr.shape):
            keep = arr[i]
            arr[i] = keep + h
            up = (lin.rope_fwd(x, pos, f, axes, **kw) * dy).sum()
            arr[i] = keep - h
            down = (lin.rope_fwd(x, pos, f, axes, **kw) * dy).sum()
            arr[i] = keep
            assert abs((up - down) / (2 * h) - want[i]) < 1e-7, i


def test_oracle_backward_is_the_forward_with_operands_exchanged():
    """dq is the pass with (dout, v, k), dk and dv the ones on reversed tokens: the identity the kernels rest on."""
    rng = np.random.default_rng(5)
    B, T, H, Dk, Dv = 1, 9, 2, 3, 5
    q, k = rng.normal(size=(2, B, T, H, Dk))
    v, do = rng.normal(size=(2, B, T, H, Dv))
    g = np.array([-0.2, -2.0])
    S0, dST = rng.normal(size=(2, B, H, Dk, Dv))
    want = lin.bwd(q, k, v, g, do, S0, dST)
    t = lambda S: S.swapaxes(-1, -2)
    rev = lambda x: x[:, ::-1]
    np.testing.assert_allclose(lin.fwd(do, v, k, g, t(S0))[0], want["dq"], atol=1e-12)
    # behind the end the gradient state is not decayed before the last token takes it: a^(T-1-i) instead of a^(i+1)
    undo = np.exp(-g)[None, :, None, None]
    np.testing.assert_allclose(rev(lin.fwd(rev(v), rev(do), rev(q), g, t(dST) * undo)[0]), want["dk"], atol=1e-12)
    np.testing.assert_allclose(rev(lin.fwd(rev(k), rev(q), rev(do), g, dST * undo)[0]), want["dv"], atol=1e-12)


# ------------------------------------------------------------------ sizes and refusals of the C entry points

def test_workspace_sizes(L):
    f = L.gdn2_linear_workspace_size
    for dt in (0, 1):
        for op in (0, 2):
            a, b = f(op, 2, 300, 4, 64, 128, dt), f(op, 2, 3000, 4, 64, 128, dt)
            assert a % 256 == 0 and a <= b
        assert f(1, 2, 300, 4, 64, 64, dt) == 0 and f(3, 2, 300, 4, 64, 64, dt) == 0   # no such op
        assert f(0, 0, 300, 4, 64, 64, dt) == 0 and f(0, 2, 300, 4, 48, 64, dt) == 0
    assert f(0, 1, 64, 1, 64, 64, 7) == 0
    assert L.gdn2_qk_norm_rope_workspace_size(128) > 0 and L.gdn2_qk_norm_rope_workspace_size(96) == 0


def _fwd(L, q=P, k=P, v=P, g=P, S0=None, o=P, ST=None, B=1, T=8, H=1, Dk=64, Dv=64, dt=0, ws=P, wsb=1 << 40):
    return L.gdn2_linear_fwd(q, k, v, g, S0, o, ST, B, T, H, Dk, Dv, dt, ws, wsb, None)


def _bwd(L, q=P, k=P, v=P, g=P, S0=None, do=P, dST=None, dq=P, dk=P, dv=P, dS0=None, B=1, T=8, H=1, Dk=64, Dv=64, dt=0, ws=P,
         wsb=1 << 40):
    return L.gdn2_linear_bwd(q, k, v, g, S0, do, dST, dq, dk, dv, dS0, B, T, H, Dk, Dv, dt, ws, wsb, None)


def test_sequence_calls_refuse_bad_arguments(L):
    for call, names in ((_fwd, ("q", "k", "v", "o")), (_bwd, ("q", "k", "v", "do", "dq", "dk", "dv"))):
        for n in names:
            assert call(L, **{n: None}) == 1 and b"NULL" in L.gdn2_last_error(), n
            assert call(L, **{n: P + 8}) == 1 and b"16-byte" in L.gdn2_last_error(), n
        assert call(L, g=None) == 1 and b"log_decay" in L.gdn2_last_error()
        assert call(L, g=P + 2) == 1
        assert call(L, S0=P + 4) == 1
        assert call(L, B=0) == 1 and call(L, H=0) == 1 and call(L, T=-1) == 1
        assert call(L, dt=2) == 1
        assert call(L, Dk=96) == 2 and call(L, Dv=256) == 2
        assert call(L, ws=None) == 3 and b"workspace" in L.gdn2_last_error()
        assert call(L, wsb=255) == 3
        assert call(L, ws=P + 16) == 1 and b"256-byte" in L.gdn2_last_error()
        assert call(L, B=1 << 20, T=1 << 20) == 1 and b"too large" in L.gdn2_last_error()
    assert _fwd(L, ST=P + 4) == 1 and _bwd(L, dST=P + 4) == 1 and _bwd(L, dS0=P + 4) == 1


def test_packed_calls_refuse_bad_arguments(L):
    def fwd(cu=P, N=2, Tmax=8, Ttot=10, H=1, Dk=64, Dv=64, dt=0):
        return L.gdn2_linear_varlen_fwd(P, P, P, P, cu, N, Tmax, Ttot, None, P, None, H, Dk, Dv, dt, P, 1 << 40, None)

    def bwd(cu=P, N=2, Tmax=8, Ttot=10, H=1, Dk=64, Dv=64, dt=0):
        return L.gdn2_linear_varlen_bwd(P, P, P, P, cu, N, Tmax, Ttot, None, P, None, P, P, P, None, H, Dk, Dv, dt, P, 1 << 40,
                                        None)
    for call in (fwd, bwd):
        assert call(cu=None) == 1 and b"cu_seqlens" in L.gdn2_last_error()
        assert call(cu=P + 1) == 1
        assert call(N=0) == 1 and call(Tmax=-1) == 1 and call(Ttot=-1) == 1
        assert call(Ttot=1 << 31) == 1 and b"too large" in L.gdn2_last_error()
        assert call(Dk=8) == 2 and call(dt=5) == 1


def test_decode_step_refuses_bad_arguments(L):
    def step(q=P, k=P, v=P, g=P, S=P, slots=P, n=4, o=P, B=2, H=1, Dk=64, Dv=64, dt=0):
        return L.gdn2_linear_decode_step(q, k, v, g, S, slots, n, o, B, H, Dk, Dv, dt, None)
    for n in ("q", "k", "v", "S", "o"):
        assert step(**{n: None}) == 1 and step(**{n: P + 8}) == 1
    assert step(g=None) == 1 and step(slots=P + 2) == 1
    assert step(n=0) == 1 and step(slots=None, n=1) == 1 and b"states" in L.gdn2_last_error()
    assert step(B=0) == 1 and step(Dk=24) == 2 and step(dt=9) == 1


def test_rotation_refuses_bad_arguments(L):
    def fwd(q=P, k=P, qs=256, ks=128, pos=P, pb=4, A=1, f=P, ax=None, pairs=32, norm=1, eps=1e-6, wq=None, wk=None, qo=P, ko=P,
            B=1, T=4, Hq=4, Hk=2, D=64, dt=0):
        return L.gdn2_qk_norm_rope_fwd(q, k, qs, ks, pos, pb, A, f, ax, pairs, 0, norm, eps, wq, wk, qo, ko, B, T, Hq, Hk, D, dt,
                                       None)
    for n in ("q", "k", "pos", "f", "qo", "ko"):
        assert fwd(**{n: None}) == 1, n
    assert fwd(q=P + 8) == 1 and fwd(wq=P + 4) == 1 and fwd(pos=P + 4, pb=8) == 1 and fwd(ax=P + 2) == 1
    assert fwd(qs=255) == 1 and fwd(qs=254) == 1 and fwd(ks=130, dt=1) == 1 and b"16 bytes" in L.gdn2_last_error()
    assert fwd(pb=2) == 1 and fwd(A=0) == 1
    assert fwd(pairs=0) == 1 and fwd(pairs=33) == 1
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        assert fwd(eps=eps) == 1
    assert fwd(B=0) == 1 and fwd(T=-1) == 1 and fwd(Hk=0) == 1 and fwd(D=48) == 2 and fwd(dt=4) == 1

    def bwd(ws=P, wsb=1 << 30, wq=P, wk=P, dq=P, dyq=P, norm=1):
        return L.gdn2_qk_norm_rope_bwd(P, P, 256, 128, dyq, P, P, 4, 1, P, None, 32, 0, norm, 1e-6, P, P, dq, P, wq, wk, 1, 4, 4, 2,
                                       64, 0, ws, wsb, None)
    assert bwd(ws=None) == 3 and bwd(wsb=16) == 3 and bwd(ws=P + 16) == 1
    assert bwd(dq=None) == 1 and bwd(dyq=None) == 1 and bwd(wq=P + 4) == 1


# ------------------------------------------------------------------ refusals of the binding

def test_binding_refuses_bad_tensors():
    from linear_attention_delta_gdn_b200 import binding as b
    x, g = torch.zeros(1, 4, 2, 16), torch.zeros(2)
    with pytest.raises(ValueError, match="CUDA"):
        b.gdn2_linear_fwd(x, x, x, g)
    with pytest.raises(ValueError, match="k must be"):
        b.gdn2_linear_fwd(x, x[:, :3], x, g)
    with pytest.raises(ValueError, match="log_decay"):
        b.gdn2_linear_fwd(x, x, x, g.double())
    with pytest.raises(ValueError, match="log_decay"):
        b.gdn2_linear_fwd(x, x, x, torch.zeros(3))
    with pytest.raises(TypeError):
        b.gdn2_linear_fwd(x.half(), x.half(), x.half(), g)
    with pytest.raises(ValueError, match="dout"):
        b.gdn2_linear_bwd(x, x, x, g, x[..., :8])
    with pytest.raises(ValueError, match="must be"):
        b.gdn2_linear_fwd(x[0], x[0], x[0], g)
    with pytest.raises(ValueError, match="cu_seqlens"):
        b.gdn2_linear_varlen_fwd(x[0], x[0], x[0], g, torch.zeros(3), 4)
    with pytest.raises(ValueError, match="gradient"):
        b.decay_linear_attention(x, x, x, g.requires_grad_())
    with pytest.raises(ValueError, match="together"):
        b.decay_linear_attention(x[0], x[0], x[0], torch.zeros(2), cu_seqlens=torch.zeros(2, dtype=torch.int32))
    s = torch.zeros(1, 2, 16)
    with pytest.raises(ValueError, match="num_slots"):
        b.gdn2_linear_decode_step(s, s, s, torch.zeros(2), torch.zeros(4, 2, 16, 8))
    with pytest.raises(ValueError, match="CUDA"):
        b.gdn2_linear_decode_step(s, s, s, torch.zeros(2), torch.zeros(4, 2, 16, 16))
    with pytest.raises(ValueError, match="CUDA"):
        b.gdn2_qk_norm_rope_fwd(x, x, torch.zeros(1, 4, dtype=torch.int32), torch.zeros(8))


def test_rotation_argument_checks():
    from linear_attention_delta_gdn_b200 import binding as b
    x, pos, f = torch.zeros(2, 4, 2, 16), torch.zeros(2, 4, dtype=torch.int32), torch.zeros(8)
    check = lambda q=x, k=x, p=pos, fr=f, ax=None, wq=None, wk=None, eps=1e-6: b._rope(q, k, p, fr, ax, wq, wk, eps, False)
    check()
    assert check(q=torch.zeros(2, 4, 6, 16)[:, :, 2:4])[1][2] == 6 * 16    # a slice's token stride
    for bad in (dict(q=x[0]), dict(k=x[:, :3]), dict(k=x.double()), dict(p=pos[:1]), dict(fr=f.double()), dict(wq=torch.ones(16), eps=None),
                dict(p=pos.expand(3, 2, 4)), dict(wq=torch.ones(8)), dict(ax=torch.zeros(7, dtype=torch.int32)),
                dict(q=torch.zeros(2, 4, 16, 2).transpose(2, 3)), dict(q=torch.zeros(4, 2, 2, 16).transpose(0, 1))):
        with pytest.raises(ValueError):
            check(**bad)
    with pytest.raises(TypeError):
        check(p=pos.float())
    assert b.rope_axes((2, 3, 3), "cpu").tolist() == [0, 0, 1, 1, 1, 2, 2, 2]


def test_layer_refusals():
    from linear_attention_delta_gdn_b200.layer import DecayLinearAttentionLayer
    with pytest.raises(ValueError, match="add up"):
        DecayLinearAttentionLayer(32, 2, 16, 16, pairs=8, sections=(2, 3))
    layer = DecayLinearAttentionLayer(32, 2, 16, 16, sections=(3, 5), dtype=torch.float32)
    assert layer.axes.tolist() == [0] * 3 + [1] * 5 and layer.inv_freq.shape == (8,)
    with pytest.raises(ValueError, match="positions"):
        layer(torch.zeros(1, 4, 32))
    layer = DecayLinearAttentionLayer(32, 2, 16, 16, dtype=torch.float32)
    with pytest.raises(ValueError, match="positions"):
        layer(torch.zeros(4, 32), cu_seqlens=torch.tensor([0, 4], dtype=torch.int32), Tmax=4)
    with pytest.raises(ValueError, match="CUDA"):
        layer(torch.zeros(1, 4, 32))
