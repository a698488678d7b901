"""What gdn2_device_status makes of the kernels' error words, without a GPU: a wait that gave up is never hidden by what
happened beside it, and everything that was recorded is named."""
import itertools
import os
import subprocess

import pytest

from conftest import ROOT

INCLUDES = ["-I", os.path.join(ROOT, "linear_attention_delta_gdn_b200", "csrc"), "-I", os.path.join(ROOT, "include")]
DBG = 1 << 30
OK, INVALID, TIMEOUT = 0, 1, 5


@pytest.fixture(scope="module")
def describe(tmp_path_factory):
    """describe_records compiled for the host: (status, text) of words (fwd, bwd, varlen, linear, step, rope)."""
    d = tmp_path_factory.mktemp("records")
    src, exe = str(d / "r.cpp"), str(d / "r")
    with open(src, "w") as f:
        f.write('#include <stdlib.h>\n#include "device_records.h"\n'
                'int main(int, char** a) {\n'
                '    auto w = [&](int i) { return (unsigned int)strtoul(a[i], nullptr, 10); };\n'
                '    const gdn2::DeviceRecords r{w(1), w(2), w(3), w(4), w(5), w(6)};\n'
                '    const size_t cap = atoi(a[7]);\n'
                '    char* text = new char[cap + 1];\n'
                '    text[cap] = 0x7f;\n'
                '    const int s = gdn2::describe_records(r, text, cap);\n'
                '    printf("%d\\n%s", text[cap] == 0x7f ? s : -1, cap ? text : "");\n}\n')
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-Werror", *INCLUDES, src, "-o", exe], check=True)

    def run(words, cap=1024):
        r = subprocess.run([exe, *map(str, words), str(cap)], check=True, capture_output=True, text=True).stdout
        status, text = r.split("\n", 1)
        return int(status), text
    return run


WAITS = {"fwd": ((4, 0, 0, 0, 0, 0), "chunk_fwd_kernel bits 0x4"), "bwd": ((0, 9, 0, 0, 0, 0), "chunk_bwd_kernel bits 0x9"),
         "linear": ((0, 0, 0, 8, 0, 0), "linear_chunk_kernel")}
OTHERS = {"index": ((DBG, 0, 0, 0, 0, 0), "index check"), "cut": ((0, 0, 1, 0, 0, 0), "Tmax"),
          "outside": ((0, 0, 0, 2, 0, 0), "outside [0, Ttot)"), "slot": ((0, 0, 0, 0, 4, 0), "slots"),
          "axis": ((0, 0, 0, 0, 0, 1), "axes")}


def test_nothing_recorded(describe):
    assert describe((0,) * 6) == (OK, "")


@pytest.mark.parametrize("name", WAITS)
def test_a_wait_alone(describe, name):
    words, detail = WAITS[name]
    status, text = describe(words)
    assert status == TIMEOUT and "gave up" in text and detail in text


@pytest.mark.parametrize("name", OTHERS)
def test_another_record_alone(describe, name):
    words, detail = OTHERS[name]
    status, text = describe(words)
    assert status == INVALID and detail in text and "gave up" not in text


@pytest.mark.parametrize("wait,n", list(itertools.product(WAITS, (1, 2, 5))))
def test_a_wait_goes_first_and_hides_nothing(describe, wait, n):
    for others in itertools.combinations(OTHERS, n):
        words = list(WAITS[wait][0])
        for o in others:
            words = [a | b for a, b in zip(words, OTHERS[o][0])]
        status, text = describe(words)
        assert status == TIMEOUT and text.startswith("device wait gave up") and WAITS[wait][1] in text, text
        assert all(OTHERS[o][1] in text for o in others), text


def test_all_at_once_fit_and_a_short_buffer_is_kept(describe):
    words = (DBG | 31, DBG | 31, 3, 11, 4, 1)
    status, text = describe(words)
    assert status == TIMEOUT and len(text) < 1023 and all(d in text for _, d in OTHERS.values())
    for cap in (0, 1, 2, 40):
        assert describe(words, cap) == (TIMEOUT, text[:max(cap - 1, 0)])


def test_the_binding_asks_the_device_it_is_given(monkeypatch):
    """The error words belong to a device: the call runs with the named one current, and on its stream."""
    import torch
    from linear_attention_delta_gdn_b200 import binding
    current, asked = [0], []

    class device:
        def __init__(self, d):
            self.d = current[0] if d is None else torch.device(d).index

        def __enter__(self):
            self.before, current[0] = current[0], self.d

        def __exit__(self, *_):
            current[0] = self.before

    class Stream:
        def __init__(self, d):
            self.cuda_stream = 100 + (current[0] if d is None else torch.device(d).index)

    class Lib:
        def gdn2_device_status(self, stream):
            asked.append((current[0], int(getattr(stream, "value", stream))))
            return 0
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: Stream(d))
    monkeypatch.setattr(binding, "lib", Lib)
    assert binding.gdn2_device_status() == 0 and binding.gdn2_device_status("cuda:1") == 0
    assert asked == [(0, 100), (1, 101)] and current == [0]


def test_an_index_check_of_the_linear_kernels(describe):
    status, text = describe((0, 0, 0, DBG, 0, 0))
    assert status == INVALID and text.startswith("index check") and "linear attention" in text
    status, text = describe((0, 0, 0, DBG | 8 | 1, 0, 0))
    assert status == TIMEOUT and all(s in text for s in ("linear_chunk_kernel", "index check", "Tmax"))
