"""barrier.cluster with .aligned is undefined for a warp whose lanes are apart, and where the
compiler brings them together again is its choice.  So in the sources a barrier of the warp,
of the CTA or of the cluster stands directly before each of them, in the same block (what may
come between moves no lane away from the others)."""
import os
import re

import pytest

import w4a4_mxfp4_quantize_b200 as mq

CSRC = os.path.join(os.path.dirname(os.path.abspath(mq.__file__)), "csrc")
BARRIER = re.compile(r"__syncwarp\(\);|__syncthreads\(\);|cluster_sync_all\(\);|cluster_wait_acquire\(\);|"
                     r"cluster_arrive_release\(\);")
TOGETHER = re.compile(r"(if (constexpr )?\([^;{]*\) ?)?\{?$|pdl_trigger\(\);$|tc_fence_(before|after)\(\);$|"
                      r"const uint32_t tmem = \*tmem_holder;$")


def lines(name):
    text = open(os.path.join(CSRC, name)).read()
    return [re.sub(r"\s*//.*", "", line).strip() for line in text.splitlines()]


def unprotected(name, call):
    """Lines with `call` that no barrier of the warp precedes."""
    src, bad = lines(name), []
    for i, line in enumerate(src):
        if call not in line:
            continue
        j = i - 1
        while TOGETHER.match(src[j]):
            j -= 1
        if not BARRIER.search(src[j]):
            bad.append((name, i + 1, line))
    return bad


def test_the_full_barrier_brings_the_warp_together_itself():
    src = lines("ptx.cuh")
    at = src.index("__device__ __forceinline__ void cluster_sync_all() {")
    assert src[at + 1] == "__syncwarp();"


@pytest.mark.parametrize("name", ["moe.cuh", "macaq.cu"])
def test_arrivals_are_directly_behind_a_barrier_of_the_warp(name):
    assert "cluster_arrive_release();" in "".join(lines(name))
    assert unprotected(name, "cluster_arrive_release();") == []


def test_the_check_sees_a_missing_barrier(tmp_path, monkeypatch):
    (tmp_path / "k.cuh").write_text("if (threadIdx.x == 0) {\n  *flag = 0;\n}\nif (split) cluster_arrive_release();\n")
    monkeypatch.setattr("test_aligned_barriers.CSRC", str(tmp_path))
    assert len(unprotected("k.cuh", "cluster_arrive_release();")) == 1
