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
    for op, bwd in ((0, False), (2, True)):
        need = L.gdn2_linear_workspace_size(op, N, Ttot, H, 64, 64, dt)
        tail = (H, 64, 64, dt, P, need - 256, None)
        if need == 0:   # many heads are not cut: nothing is needed, and nothing would stop the call
            assert dt == 1 and H == 200
            continue
        if bwd:
            rc = L.gdn2_linear_varlen_bwd(P, P, P, P, P, N, Tmax, Ttot, None, P, None, P, P, P, None, *tail)
        else:
            rc = L.gdn2_linear_varlen_fwd(P, P, P, P, P, N, Tmax, Ttot, None, P, None, *tail)
        assert rc == 3 and b"needs %d workspace" % need in L.gdn2_last_error(), L.gdn2_last_error()
