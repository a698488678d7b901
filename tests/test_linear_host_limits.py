"""Linear attention with a decay per head at the limits of its arguments, without a GPU: plans and refusals on the host."""
import os
import subprocess

import pytest

from conftest import ROOT

P = 1 << 20   # an address that passes the checks; every call here is refused before anything could read it
INT_MAX = 2 ** 31 - 1
CSRC = os.path.join(ROOT, "linear_attention_delta_gdn_b200", "csrc")


@pytest.fixture(scope="module")
def L():
    from linear_attention_delta_gdn_b200 import build, binding
    build.build()
    return binding.lib()


# ------------------------------------------------------------------ any bound on the lengths

@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    """choose_cut of the tensor-core path, compiled for the host: (nseg, cps, slots, items the workspace holds)."""
    d = tmp_path_factory.mktemp("cut")
    src, exe = str(d / "cut.cpp"), str(d / "cut")
    with open(src, "w") as f:
        f.write('#include <stdio.h>\n#include <stdlib.h>\n#include "linear_cut.h"\nusing namespace gdn2::linear;\n'
                'int main(int n, char** a) {\n'
                '    for (int i = 1; i + 5 < n; i += 6) {\n'
                '        const Cut c = choose_cut(atoi(a[i]), atoi(a[i + 1]), atoll(a[i + 2]), atoi(a[i + 3]), atoll(a[i + 4]), atoi(a[i + 5]));\n'
                '        printf("%d %d %lld %lld\\n", c.nseg, c.cps, c.slots, most_items(atoll(a[i + 4]), atoi(a[i + 5])));\n'
                '    }\n}\n')
    subprocess.run(["g++", "-O2", "-std=c++17", "-fsanitize=signed-integer-overflow", "-fno-sanitize-recover", "-I", CSRC, src, "-o", exe],
                   check=True)
    return lambda cases: [tuple(int(x) for x in line.split()) for line in
                          subprocess.run([exe] + [str(int(x)) for c in cases for x in c], check=True, capture_output=True,
                                         text=True).stdout.splitlines()]


def test_plans_cover_every_length(plan):
    cases = [(N, T, Ttot, packed, N * per, 148)
             for T in (0, 1, 127, 128, 129, 5000, 65536, 2 ** 30, 2 ** 31 - 129, 2 ** 31 - 128, 2 ** 31 - 127, INT_MAX)
             for N in (1, 3, 20) for per in (1, 2, 16, 64) for packed in (0, 1)
             for Ttot in ((N * T,) if not packed else (0, 300, 12557, INT_MAX)) if Ttot <= INT_MAX]
    got = plan(cases)
    assert len(got) == len(cases)
    for (N, T, Ttot, _, heads, _), (nseg, cps, slots, items) in zip(cases, got):
        chunks = -(-T // 128)
        assert nseg >= 1 and cps >= 1 and nseg * cps >= chunks, (N, T, Ttot, nseg, cps)
        if nseg > 1:   # a state for each segment that ends in front of its sequence's last one, and room for it
            assert slots >= Ttot // (cps * 128) + N and slots * (heads // N) <= items


@pytest.mark.parametrize("dt", [0, 1])
@pytest.mark.parametrize("Tmax", [2 ** 31 - 128, 2 ** 31 - 127, INT_MAX])
@pytest.mark.parametrize("H", [1, 200])
def test_a_loose_bound_counts_as_the_rows(L, dt, Tmax, H):
    """What a packed call needs goes by its tensor where the bound is looser (the calls stop at the missing workspace)."""
    N, Ttot = 3, 300
    for bwd in (False, True):
        said = []
        for bound in (Ttot, Tmax):
            tail = (H, 64, 64, dt, None, 0, None)
            if dt == 1 and H == 200:   # many heads are not cut: nothing is needed, and the missing o stops the call
                rc = L.gdn2_linear_varlen_fwd(P, P, P, P, P, N, bound, Ttot, None, None, None, *tail)
            elif bwd:
                rc = L.gdn2_linear_varlen_bwd(P, P, P, P, P, N, bound, Ttot, None, P, None, P, P, P, None, *tail)
            else:
                rc = L.gdn2_linear_varlen_fwd(P, P, P, P, P, N, bound, Ttot, None, P, None, *tail)
            said.append((rc, L.gdn2_last_error()))
        assert said[0] == said[1] and said[0][0] in (1, 3) and b"too large" not in said[0][1], said


# ------------------------------------------------------------------ workspace of packed calls

def _packed(L, bwd, N, Tmax, Ttot, H, Dk, Dv, dt, wsb):
    tail = (H, Dk, Dv, dt, P, wsb, None)
    if bwd:
        return L.gdn2_linear_varlen_bwd(P, P, P, P, P, N, Tmax, Ttot, None, P, None, P, P, P, None, *tail)
    return L.gdn2_linear_varlen_fwd(P, P, P, P, P, N, Tmax, Ttot, None, P, None, *tail)


@pytest.mark.parametrize("dt", [0, 1])
@pytest.mark.parametrize("op,bwd", [(0, False), (2, True)])
def test_packed_workspace_goes_by_the_rows(L, dt, op, bwd):
    size, dense = L.gdn2_linear_varlen_workspace_size, L.gdn2_linear_workspace_size
    sets = 2 if bwd else 1
    for N, Tmax, Ttot, H, Dk, Dv in ((24, 16384, 20000, 16, 128, 128), (3, INT_MAX, 300, 2, 64, 32), (1, 1, 1, 1, 16, 16),
                                     (500, 2000, 2499, 2, 64, 64), (8, 64, 512, 2, 64, 64), (4, 100, 4000, 2, 32, 64)):
        need = size(op, N, Tmax, Ttot, H, Dk, Dv, dt)
        assert need % 256 == 0 and need <= dense(op, N, min(Tmax, Ttot), H, Dk, Dv, dt)
        for looser in (Ttot, INT_MAX):
            assert size(op, N, max(Tmax, looser), Ttot, H, Dk, Dv, dt) >= need
        if dt == 0:
            states = min(Ttot // 64 + N, N * -(-min(Tmax, Ttot) // 64))
            assert need == -(-states * H * Dk * Dv * 4 * sets // 256) * 256, (N, Tmax, Ttot)
        # the call asks for just that
        if need:
            assert _packed(L, bwd, N, Tmax, Ttot, H, Dk, Dv, dt, need - 1) == 3
            assert b"needs %d workspace" % need in L.gdn2_last_error()
    # one long sequence among short ones, in 32 bits: a state for each 64 rows, not 24 sequences of the longest
    assert size(op, 24, 16384, 20000, 16, 128, 128, 0) == 336 * 16 * 65536 * sets
    for bad in ((1, 2, 8, 10, 1, 64, 64, dt), (op, 0, 8, 10, 1, 64, 64, dt), (op, 2, -1, 10, 1, 64, 64, dt),
                (op, 2, 8, -1, 1, 64, 64, dt), (op, 2, 8, 10, 1, 48, 64, dt), (op, 2, 8, 1 << 31, 1, 64, 64, dt),
                (op, 2, 8, 10, 1, 64, 64, 7)):
        assert size(*bad) == 0


# ------------------------------------------------------------------ what has no gradient

def test_frequencies_that_want_a_gradient_are_refused():
    import torch
    from linear_attention_delta_gdn_b200 import binding as b
    x, pos, f = torch.zeros(1, 4, 2, 16), torch.zeros(1, 4, dtype=torch.int32), torch.ones(8, requires_grad=True)
    with pytest.raises(ValueError, match="inv_freq has no gradient"):
        b.qk_norm_rope(x, x, pos, f)
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):   # nothing is lost there: on to the next check
        b.qk_norm_rope(x, x, pos, f)
