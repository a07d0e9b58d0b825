"""Arguments of the calls around the linear at the ends of their ranges, refused or accepted by
the C ABI with made-up addresses in a process that sees no CUDA device."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

import w4a4_mxfp4_quantize_b200 as mq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
hidden_device = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up device addresses: run with the device hidden")


@pytest.fixture(scope="module")
def L():
    mq.build()
    return mq.lib()


def test_run_with_the_device_hidden():
    if not torch.cuda.is_available():
        pytest.skip("no device visible: the tests run in this process")
    r = subprocess.run([sys.executable, "-m", "pytest", os.path.abspath(__file__), "-x", "-q", "-p", "no:cacheprovider",
                        "-k", "with_no_device"], cwd=ROOT, env=dict(os.environ, CUDA_VISIBLE_DEVICES=""),
                       capture_output=True, text=True, timeout=900)
    assert r.returncode == 0 and " passed" in r.stdout, r.stdout[-3000:] + r.stderr[-2000:]


def at(i, off=0):
    return ctypes.c_void_p((i << 36) + off)


@hidden_device
@pytest.mark.parametrize("per", [63, 64, 2 ** 31 - 1, 2 ** 31, 2 ** 63 - 64, 2 ** 63 - 1])
@pytest.mark.parametrize("M", [1, 63, 64])
def test_gate_rows_with_no_device(L, per, M):
    # one gate row serves the call (two where M is 64 and per 63): an output over its bytes is refused, behind it not
    def f(ho):
        return L.macaq_block_norm(at(1), 0, at(2), None, at(4), 0, per, at(5), 1.0, 1e-6, 0.0, ho, at(7), M, 1024, None)

    rows = -(-M // per)
    for row in range(rows):
        assert f(at(4, row * 2048)) == f(at(4, row * 2048 + 2032)) == -5
    assert f(at(4, rows * 2048)) == f(at(6)) == -8  # accepted: the missing device is the next refusal
