"""The query/key norm with rotation on the GPU at the limits of its arguments, against the fp64 oracle.

Tolerance (relative L2) in float32: 1e-6 for the arithmetic, as test_gpu_rope.py derives it, and what the angle is off by: a
pair turned by an angle off by e is off by e of its length. The angle's error is |position| * 2^-63 turns (the turn per
position is a whole number of 2^-64 turns, each of its two parts off by one at most).
"""
import numpy as np
import pytest
import torch

from conftest import rel_l2
from linear_attention_delta_gdn_b200 import binding
from linear_attention_delta_gdn_b200.inputs import to_f64
from oracle import linear as lin
from test_gpu_rope import built  # noqa: F401 (the module's fixture)

pytestmark = pytest.mark.gpu


def allowed(pos):
    return 1e-6 + float(pos.abs().max()) * 2.0 ** -63 * 2 * np.pi


@pytest.mark.parametrize("sign", [1, -1, 0])
@pytest.mark.parametrize("far,pos64", [(n, b) for n in (0, 1 << 20, (1 << 31) - 10, 1 << 34, -(1 << 36), 1 << 40) for b in (True, False)
                                       if b or abs(n) < 1 << 31])
def test_far_positions_and_signs_of_the_frequencies(far, sign, pos64):
    """Frequencies of either sign (0: in turn), from 8 rad a position down to 1e-5."""
    g = torch.Generator().manual_seed(90)
    B, T, Hq, Hk, D, pairs = 1, 16, 2, 1, 64, 32
    q, k, dyq, dyk = (torch.randn(B, T, h, D, generator=g) for h in (Hq, Hk, Hq, Hk))
    pos = torch.randint(-5, 6, (B, T), generator=g) + far
    pos = pos.to(torch.int64 if pos64 else torch.int32)
    f = 8 * torch.exp(-13.6 * torch.arange(pairs) / pairs).float()
    f = f * (sign if sign else torch.tensor([1.0, -1.0]).repeat(pairs // 2))
    w = 1 + 0.2 * torch.randn(D, generator=g)
    a = (pos.cuda(), f.cuda(), None, w.cuda(), w.cuda())
    qo, ko = binding.gdn2_qk_norm_rope_fwd(q.cuda(), k.cuda(), *a)
    d = binding.gdn2_qk_norm_rope_bwd(q.cuda(), k.cuda(), dyq.cuda(), dyk.cuda(), *a)
    tol = allowed(pos)
    ref = (pos[None].numpy(), f.numpy(), np.zeros(pairs, int), to_f64(w))
    for x, y, out, dx in ((q, dyq, qo, d["dq"]), (k, dyk, ko, d["dk"])):
        assert rel_l2(to_f64(out), lin.rope_fwd(to_f64(x), *ref)) <= tol
        assert rel_l2(to_f64(dx), lin.rope_bwd(to_f64(x), to_f64(y), *ref)[0]) <= tol
