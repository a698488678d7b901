"""The debug build's index checks in the linear attention kernels: the small GPU suites of these operators pass on it in a child
process, and no check fires (conftest looks at the device status after every GPU test under GDN2_DEBUG). The tests that make
waits give up on purpose stay with the release build."""
import os
import subprocess
import sys

import pytest
import torch

from conftest import ROOT

pytestmark = pytest.mark.gpu


def test_linear_suites_pass_on_the_debug_build():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from linear_attention_delta_gdn_b200 import build
    assert build.build(debug=True).endswith("libgdn2_debug.so")
    files = ["tests/test_gpu_linear.py", "tests/test_gpu_linear_limits.py", "tests/test_gpu_linear_layer.py"]
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-m", "gpu", "-p", "no:cacheprovider", *files], cwd=ROOT,
                       env=dict(os.environ, GDN2_DEBUG="1"), capture_output=True, text=True, timeout=1200)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
