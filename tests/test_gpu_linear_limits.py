"""Linear attention with a decay per head on the GPU at the limits of its arguments, against the fp64 oracle. Tolerances
are those of test_gpu_linear.py, whose checks these tests use."""
import numpy as np
import pytest
import torch

from linear_attention_delta_gdn_b200 import binding
from linear_attention_delta_gdn_b200.inputs import to_f64
from oracle import linear as lin
from test_gpu_linear import built, check_dense, check_states, check_tokens, make, packed_case  # noqa: F401 (built: the module's fixture)

pytestmark = pytest.mark.gpu


def check_packed(x, d, cu, lengths, Tmax, dtype):
    args = (d["q"], d["k"], d["v"], d["g"])
    o, ST = binding.gdn2_linear_varlen_fwd(*args, cu, Tmax, d["S0"])
    g = binding.gdn2_linear_varlen_bwd(*args, d["do"], cu, Tmax, d["S0"], d["dST"])
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
@pytest.mark.parametrize("Tmax", [2 ** 31 - 128, 2 ** 31 - 127, 2 ** 31 - 1])
@pytest.mark.parametrize("lengths", [[300, 0, 41], [2600, 1]])
def test_a_bound_far_above_the_lengths(dtype, Tmax, lengths):
    x, d, cu = packed_case(lengths, 2, 64, 32, dtype, 70)
    check_packed(x, d, cu, lengths, Tmax, dtype)


def test_every_record_is_named():
    """A bad slot, a sequence cut at Tmax and a bad axis between two readings: each is in the detail."""
    x, d, cu = packed_case([70, 30], 2, 64, 64, "bf16", 71)
    binding.gdn2_device_status()
    args = (d["q"], d["k"], d["v"], d["g"])
    binding.gdn2_linear_decode_step(*(t[:2] for t in args[:3]), args[3], d["S0"].clone(), torch.tensor([1, 1], dtype=torch.int32).cuda())
    binding.gdn2_linear_varlen_fwd(*args, cu, 64)
    pos, f = torch.zeros(1, 100, dtype=torch.int32, device="cuda"), torch.ones(8, device="cuda")
    binding.gdn2_qk_norm_rope_fwd(args[0][None], args[1][None], pos, f, torch.full((8,), 3, dtype=torch.int32, device="cuda"))
    assert binding.gdn2_device_status() == binding.GDN2_ERR_INVALID
    assert all(s in binding.last_error() for s in ("slots", "Tmax", "axes")), binding.last_error()
    assert binding.gdn2_device_status() == binding.GDN2_OK


# one long sequence among many of 0 and 1 tokens (states by row), and sequences of one length (states by sequence), both with
# a workspace of just the size asked for
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lengths", [[1, 0, 900, 1, 1, 0, 65, 0, 64, 1, 63, 0], [64] * 5, [129, 128, 127]])
def test_packed_workspace_is_enough(dtype, lengths):
    N, H, Dk, Dv = len(lengths), 2, 32, 64
    x, d, cu = packed_case(lengths, H, Dk, Dv, dtype, 72, tail=3)
    code = {"f32": binding.GDN2_F32, "bf16": binding.GDN2_BF16}[dtype]
    args, Tmax, Ttot = (d["q"], d["k"], d["v"], d["g"]), max(lengths), sum(lengths) + 3
    sizes = [binding.gdn2_linear_varlen_workspace_size(op, N, Tmax, Ttot, H, Dk, Dv, code) for op in (binding.GDN2_OP_FWD, binding.GDN2_OP_BWD)]
    rooms = [torch.full((n + 4096,), 0x5a, dtype=torch.uint8, device="cuda") for n in sizes]
    o, ST = binding.gdn2_linear_varlen_fwd(*args, cu, Tmax, d["S0"], ws=rooms[0][:sizes[0]])
    g = binding.gdn2_linear_varlen_bwd(*args, d["do"], cu, Tmax, d["S0"], d["dST"], ws=rooms[1][:sizes[1]])
    assert binding.gdn2_device_status() == binding.GDN2_OK, binding.last_error()
    assert all(bool((r[n:] == 0x5a).all()) for r, n in zip(rooms, sizes))
    for i, n in enumerate(lengths):   # each sequence alone, bit for bit
        at = slice(sum(lengths[:i]), sum(lengths[:i + 1]))
        one = [d[m][at][None].contiguous() for m in ("q", "k", "v")] + [d["g"]]
        o1, ST1 = binding.gdn2_linear_fwd(*one, d["S0"][i:i + 1])
        g1 = binding.gdn2_linear_bwd(*one, d["do"][at][None].contiguous(), d["S0"][i:i + 1], d["dST"][i:i + 1])
        if dtype == "f32":
            assert torch.equal(o[at], o1[0]) and torch.equal(ST[i:i + 1], ST1), i
            assert all(torch.equal(g[m][at], g1[m][0]) for m in ("dq", "dk", "dv")) and torch.equal(g["dS0"][i:i + 1], g1["dS0"]), i
    check_packed(x, d, cu, lengths, Tmax, dtype)


# either side of a decay of 1/4 a token (-2 ln 2 = -1.38629436), where the pairs' weights change from products of a row's and a
# column's part, largest there, to one read by distance
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
def test_decays_around_a_quarter(dtype, D):
    x, d = make((1, 333), 1, 8, D, D, dtype, 73, [-1.0, -1.2, -1.386, -1.3862943, -1.3862944, -1.3863, -1.5, -2.5])
    check_dense(x, d, dtype)


# Large and small numbers: outputs are products of three inputs, 2^84 to 2^92 here (or their inverses), and 32 bits hold
# 2^127. What a weight's two parts add on the way (2^30 either way at the strongest decay that has them) must fit, too.
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [28, -28])
def test_large_and_small_numbers(dtype, scale):
    x, d = make((1, 333), 1, 5, 64, 64, dtype, 74, [-1.386, -1.2, -0.7, 0.0, -3.0])
    for n, times in (("q", 1), ("k", 1), ("v", 1), ("do", 1), ("S0", 2), ("dST", 2)):
        x[n] = x[n] * 2.0 ** (scale * times)   # a power of two: exact
        d[n] = x[n].cuda()
    check_dense(x, d, dtype)
