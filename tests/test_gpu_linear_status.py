"""The waits of the bf16 linear attention kernel are bounded, and its way out is sound: GDN2_TEST_SKIP_LINEAR_ROLE leaves out
one of the kernel's roles on the host's word, so that the barriers it would arrive at are never closed. The other roles give
up (after 5 ms instead of 2 s), the kernel returns, gdn2_device_status reports it, and the next call is right."""
import os

import pytest
import torch

from linear_attention_delta_gdn_b200 import binding
from test_gpu_linear import make

pytestmark = pytest.mark.gpu


def run(d):
    o, ST = binding.gdn2_linear_fwd(d["q"], d["k"], d["v"], d["g"], d["S0"])
    g = binding.gdn2_linear_bwd(d["q"], d["k"], d["v"], d["g"], d["do"], d["S0"], d["dST"])
    return [o, ST, g["dq"], g["dk"], g["dv"], g["dS0"]]


# one chunk, more chunks than the tiles have stages (the loads then wait for a role that never answers, too), and a sequence
# cut into segments, whose first launch makes states only; heads of 128 have two stages, of 64 four
@pytest.mark.parametrize("role", [1, 2, 3, 4, 5])
@pytest.mark.parametrize("T,D", [(100, 128), (1000, 128), (1000, 64), (5000, 64)])
def test_a_role_that_does_nothing_is_reported(role, T, D):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    _, d = make((1, T), 1, 2, D, D, "bf16", 80 + role)
    binding.gdn2_device_status()
    want = run(d)
    assert binding.gdn2_device_status() == binding.GDN2_OK, binding.last_error()
    os.environ["GDN2_TEST_SKIP_LINEAR_ROLE"] = str(role)
    try:
        run(d)
        status = binding.gdn2_device_status()
    finally:
        del os.environ["GDN2_TEST_SKIP_LINEAR_ROLE"]
    assert status == binding.GDN2_ERR_TIMEOUT and "linear_chunk_kernel" in binding.last_error(), binding.last_error()
    assert binding.gdn2_device_status() == binding.GDN2_OK
    got = run(d)
    assert binding.gdn2_device_status() == binding.GDN2_OK, binding.last_error()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
