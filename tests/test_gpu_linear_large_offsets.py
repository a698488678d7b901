"""Linear attention, its step and the rotation on tensors of more than 2^31 elements: what is checked lies behind that offset."""
import pytest
import torch

from linear_attention_delta_gdn_b200 import binding
from linear_attention_delta_gdn_b200.inputs import to_f64
from oracle import linear as lin
from test_gpu_linear import DT, built, check_states, check_tokens, make  # noqa: F401 (built: the module's fixture)

pytestmark = pytest.mark.gpu
H, D = 16, 128
FRONT = 2 ** 31 // (H * D) + 5   # token rows in front


def behind(t):
    """t's rows behind FRONT others, which are not set."""
    big = torch.empty((FRONT + t.shape[0], *t.shape[1:]), dtype=t.dtype, device="cuda")
    big[FRONT:] = t
    return big


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [300, 1000])
def test_packed_rows(dtype, T):
    """(Against the oracle: where a sequence is cut into segments goes by the rows of the tensor, too.)"""
    x, d = make((T,), 1, H, D, D, dtype, 95)
    cu = torch.tensor([FRONT, FRONT + T], dtype=torch.int32).cuda()
    f = {n: to_f64(t) for n, t in x.items()}
    q, k, v, do = (f[n][None] for n in ("q", "k", "v", "do"))
    o_ref, ST_ref = lin.fwd(q, k, v, f["g"], f["S0"])
    ref = lin.bwd(q, k, v, f["g"], do, f["S0"], f["dST"])
    big = [behind(d[n]) for n in ("q", "k", "v")]
    o, ST = binding.gdn2_linear_varlen_fwd(*big, d["g"], cu, T, d["S0"])
    check_tokens(to_f64(o[FRONT:])[None], o_ref, dtype, "o")
    check_states(to_f64(ST), ST_ref, dtype, "ST")
    del o
    g = binding.gdn2_linear_varlen_bwd(*big, d["g"], behind(d["do"]), cu, T, d["S0"], d["dST"])
    for n in ("dq", "dk", "dv"):
        check_tokens(to_f64(g[n][FRONT:])[None], ref[n], dtype, n)
    check_states(to_f64(g["dS0"]), ref["dS0"], dtype, "dS0")
    assert binding.gdn2_device_status() == binding.GDN2_OK


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_pool_of_states(dtype):
    B, slots = 3, 2 ** 31 // (H * D * D) + 4
    _, d = make((B,), B, H, D, D, dtype, 96)
    S = d["S0"].clone()
    o = binding.gdn2_linear_decode_step(d["q"], d["k"], d["v"], d["g"], S)
    pool = torch.empty(slots, H, D, D, device="cuda")
    pool[-B:] = d["S0"]
    o2 = binding.gdn2_linear_decode_step(d["q"], d["k"], d["v"], d["g"], pool, torch.arange(slots - B, slots, dtype=torch.int32, device="cuda"))
    assert torch.equal(o2, o) and torch.equal(pool[-B:], S)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rotation_rows(dtype):
    T = 37
    g = torch.Generator().manual_seed(97)
    q, k, dq, dk = (torch.randn(T, h, D, generator=g).to(DT[dtype]).cuda() for h in (H, 1, H, 1))
    pos, f = torch.arange(T, device="cuda"), torch.rand(64, generator=g).cuda()
    w = torch.rand(D, generator=g).cuda()
    small = binding.gdn2_qk_norm_rope_fwd(q[None], k[None], pos[None], f, q_weight=w, k_weight=w)
    ref = binding.gdn2_qk_norm_rope_bwd(q[None], k[None], dq[None], dk[None], pos[None], f, q_weight=w, k_weight=w)
    zero = lambda t: torch.zeros((1, FRONT + T, *t.shape[1:]), dtype=t.dtype, device="cuda")
    big = [zero(t) for t in (q, k)]
    p = torch.zeros(1, FRONT + T, dtype=torch.int64, device="cuda")
    for b, t in zip(big + [p], (q, k, pos)):
        b[0, FRONT:] = t
    out = binding.gdn2_qk_norm_rope_fwd(*big, p, f, q_weight=w, k_weight=w)
    assert all(torch.equal(x[:, FRONT:], y) for x, y in zip(out, small))
    del out
    dy = [zero(t) for t in (dq, dk)]
    for b, t in zip(dy, (dq, dk)):
        b[0, FRONT:] = t
    got = binding.gdn2_qk_norm_rope_bwd(*big, *dy, p, f, q_weight=w, k_weight=w)
    assert all(torch.equal(got[n][:, FRONT:], ref[n]) for n in ("dq", "dk"))
