"""Refusals of the calls around the linear (norms, routing, mixture-of-experts layer):
by the binding, with CPU tensors (the device check comes last), and by the C ABI,
with made-up addresses in a process that sees no CUDA device."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

import w4a4_mxfp4_quantize_b200 as mq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF16, FP32 = 0, 1


@pytest.fixture(scope="module")
def L():
    mq.build()
    return mq.lib()


# ---------------------------------------------------------------- binding
M, C = 4, 32


def norm_args(**kw):
    a = dict(h=torch.zeros((M, C), dtype=torch.bfloat16), y=torch.zeros((M, C), dtype=torch.bfloat16),
             w_post=torch.ones(C), w_pre=torch.ones(C))
    a.update(kw)
    return a


@pytest.mark.parametrize("change,message", [
    (dict(h=torch.zeros((M, C), dtype=torch.float16)), "h must be torch.bfloat16 or torch.float32"),
    (dict(h=torch.zeros((M, 2, C), dtype=torch.bfloat16)), "h must have 2 dimensions"),
    (dict(y=torch.zeros((M, C))), "y must be torch.bfloat16"),
    (dict(y=torch.zeros((M + 1, C), dtype=torch.bfloat16)), "y must be"),
    (dict(w_post=torch.ones(C + 1)), "w_post must be"),
    (dict(w_pre=torch.ones(C, dtype=torch.bfloat16)), "w_pre must be torch.float32"),
    (dict(gate=torch.ones((M, C), dtype=torch.float16)), "gate must be torch.bfloat16 or torch.float32"),
    (dict(gate=torch.ones((M - 1, C))), "gate must be"),
    (dict(gate=torch.ones((M, C)), rows_per_gate=2), "gate must be"),
    (dict(gate=torch.ones((M, C)), rows_per_gate=0), "rows_per_gate must be at least 1"),
    (dict(gate=torch.ones(C), rows_per_gate=2), "rows_per_gate does not apply"),
    (dict(y=None), "go with y"),
    (dict(y=None, w_post=None, out_h=torch.zeros((M, C), dtype=torch.bfloat16)), "go with y"),
    (dict(w_pre=None, out_n=torch.zeros((M, C), dtype=torch.bfloat16)), "goes with w_pre"),
    (dict(out_h=torch.zeros((M, C))), "out_h must be torch.bfloat16"),
    (dict(out_n=torch.zeros((M, C))), "out_n must be torch.bfloat16"),
    (dict(), "contiguous CUDA tensors"),
])
def test_norm_refusals(L, change, message):
    with pytest.raises(ValueError, match=message):
        mq.block_norm(**norm_args(**change))


@pytest.mark.parametrize("logits,k,message", [
    (torch.zeros((3, 8), dtype=torch.float16), 2, "logits must be torch.bfloat16 or torch.float32"),
    (torch.zeros(8), 2, "logits must have 2 dimensions"),
    (torch.zeros((3, 8)), 0, "k must be between 1 and"),
    (torch.zeros((3, 8)), 9, "k must be between 1 and"),
    (torch.zeros((3, 100)), 33, "k must be between 1 and"),
    (torch.zeros((3, 8)), 2, "contiguous CUDA tensors"),
])
def test_route_refusals(L, logits, k, message):
    with pytest.raises(ValueError, match=message):
        mq.moe_route(logits, k)


E, H, I = 3, 256, 512


def moe_args(**kw):
    up, down = mq.weight_bytes(E, 2 * I, H), mq.weight_bytes(E, H, I)
    a = dict(x=torch.zeros((M, H), dtype=torch.bfloat16), logits=torch.zeros((M, E)), D_up=torch.ones((E, H)),
             Wq_up=torch.zeros(up[0], dtype=torch.uint8), Ws_up=torch.zeros(up[1], dtype=torch.uint8),
             D_down=torch.ones((E, I)), Wq_down=torch.zeros(down[0], dtype=torch.uint8),
             Ws_down=torch.zeros(down[1], dtype=torch.uint8), inner=I, k=2)
    a.update(kw)
    return a


@pytest.mark.parametrize("change,message", [
    (dict(x=torch.zeros((M, H))), "x must be torch.bfloat16"),
    (dict(logits=torch.zeros((M + 1, E))), "logits must be"),
    (dict(logits=torch.zeros((M, E), dtype=torch.int32)), "logits must be torch.bfloat16 or torch.float32"),
    (dict(D_up=torch.ones((E, H + 1))), "D_up must be"),
    (dict(D_up=torch.ones((E - 1, H))), "D_up must be"),
    (dict(D_down=torch.ones((E, I), dtype=torch.float64)), "D_down must be torch.float32"),
    (dict(inner=I + 256), "D_down must be"),
    (dict(Wq_up=torch.zeros(8, dtype=torch.uint8)), "Wq_up holds"),
    (dict(Ws_up=torch.zeros(8, dtype=torch.uint8)), "Ws_up holds"),
    (dict(Wq_down=torch.zeros(8, dtype=torch.uint8)), "Wq_down holds"),
    (dict(Ws_down=torch.zeros(8, dtype=torch.int8)), "Ws_down must be torch.uint8"),
    (dict(out=torch.zeros((M, H))), "out must be torch.bfloat16"),
    (dict(status=torch.zeros(1)), "status must be torch.int32"),
    (dict(), "contiguous CUDA tensors"),
])
def test_moe_refusals(L, change, message):
    with pytest.raises(ValueError, match=message):
        mq.moe_mm(**moe_args(**change))


def test_gate_up_refusals(L):
    with pytest.raises(ValueError, match="as many gate rows"):
        mq.prepare_gate_up(torch.zeros((E, 5, H)), torch.ones((E, H)))
    with pytest.raises(ValueError, match="D must be"):
        mq.prepare_gate_up(torch.zeros((E, 512, H)), torch.ones((E, H - 1)))
    with pytest.raises(ValueError, match="contiguous CUDA tensors"):
        mq.prepare_gate_up(torch.zeros((E, 512, H)), torch.ones((E, H)))


# ---------------------------------------------------------------- C ABI
def _device_visible() -> bool:
    return torch.cuda.is_available()


hidden_device = pytest.mark.skipif(_device_visible(), reason="made-up device addresses: run with the device hidden")


def test_c_refusals_run_with_the_device_hidden():
    if not _device_visible():
        pytest.skip("no device visible: the refusal tests run in this process")
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    r = subprocess.run([sys.executable, "-m", "pytest", os.path.abspath(__file__), "-x", "-q", "-p", "no:cacheprovider",
                        "-k", "by_name or named_cuda_error"], cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-2000:]
    assert " passed" in r.stdout and "skipped" not in r.stdout.splitlines()[-1], r.stdout[-2000:]


P = ctypes.c_void_p


def at(i, off=0):
    return P((i << 36) + off)


@hidden_device
def test_norm_refused_by_name(L):
    def f(h=at(1), ht=BF16, y=at(2), wp=at(3), g=at(4), gt=BF16, per=1, wn=at(5), scale=1.0, eps=1e-6, off=0.0, ho=at(6),
          no=at(7), M=64, C=1024):
        return L.macaq_block_norm(h, ht, y, wp, g, gt, per, wn, scale, eps, off, ho, no, M, C, None)

    assert f(M=-1) == f(M=2 ** 31) == f(C=8) == f(C=1000) == f(C=65552) == f(per=0) == -3
    assert f(ht=2) == f(gt=-1) == f(scale=float("nan")) == f(eps=-1.0) == f(eps=float("inf")) == f(off=float("inf")) == -14
    assert f(h=None) == f(y=None) == f(ho=None) == f(wn=None) == f(no=None) == -1
    assert f(y=None, ho=None, wp=None) == -1                                  # a gate without a branch
    assert f(y=None, ho=None, wp=None, g=None, wn=None, no=None) == -1        # nothing to do
    for name in ("h", "y", "wp", "g", "wn", "ho", "no"):
        assert f(**{name: at(9, 8)}) == -2, name
    size = 64 * 1024 * 2
    assert f(ho=at(1, 16)) == -5            # in place means the same rows
    assert f(ho=at(1)) == -8                # (accepted: the missing device is the next refusal)
    assert f(y=at(1), ho=at(1)) == -5       # in place, and the branch in the same memory
    assert f(ho=at(2)) == f(no=at(1)) == f(no=at(2)) == f(no=at(6, size - 16)) == f(ho=at(3)) == f(no=at(4)) == -5
    assert f(ho=at(4, size - 16)) == -5     # the gate of the last row
    assert f(g=at(4), per=64, ho=at(4, 2048)) != -5  # one gate row: behind it is free
    assert f(M=0, h=None) == 0


@hidden_device
def test_route_refused_by_name(L):
    def f(l=at(1), lt=FP32, T=1000, E=128, k=8, score=0, scale=1.0, ids=at(2), w=at(3), c=at(4), o=at(5), ws=at(6),
          wsb=1 << 20):
        return L.macaq_moe_route(l, lt, T, E, k, score, 1, scale, ids, w, c, o, ws, wsb, None)

    assert f(E=0) == f(E=1025) == -6
    assert f(k=0) == f(k=33) == f(E=4, k=5) == f(T=-1) == f(T=2 ** 31) == f(T=2 ** 30, k=4) == -3
    assert f(lt=2) == f(score=2) == f(scale=float("inf")) == -14
    assert f(l=None) == f(ids=None) == f(w=None) == f(c=None) == f(o=None) == -1
    for name in ("l", "ids", "w", "c", "o"):
        assert f(**{name: at(9, 4)}) == -2, name
    assert f(ids=at(1)) == f(w=at(2, 1000 * 32 - 16)) == f(c=at(3)) == f(o=at(2)) == f(ws=at(1)) == f(ws=at(5)) == -5
    assert f(ws=None) == f(wsb=1000) == f(ws=at(6, 8)) == -11
    assert f(T=0, c=None, o=None, l=None, ids=None, w=None) == 0
    assert L.macaq_route_workspace_bytes(64, 128) == 0 and L.macaq_route_workspace_bytes(65, 128) > 0


@hidden_device
def test_moe_refused_by_name(L):
    def f(x=at(1), l=at(2), lt=FP32, du=at(3), qu=at(4), su=at(5), dd=at(6), qd=at(7), sd=at(8), T=16, E=4, k=2, H=512,
          I=256, score=0, scale=1.0, act=5, y=at(9), ws=at(10), wsb=1 << 20):
        return L.macaq_moe_mm(x, l, lt, du, qu, su, dd, qd, sd, T, E, k, H, I, score, 1, scale, act, y, ws, wsb, None,
                              None)

    assert f(E=0) == f(E=513) == -6
    assert f(T=-1) == f(T=129) == f(k=0) == f(k=5) == f(E=100, k=17) == f(H=128) == f(H=300) == f(H=8448) == f(I=0) == f(I=8448) == -3
    assert f(lt=3) == f(score=-1) == f(scale=float("nan")) == -14
    for act in (0, 1, 3, 4, 6):
        assert f(act=act) == -13
    names = ("x", "l", "du", "qu", "su", "dd", "qd", "sd", "y")
    for name in names:
        assert f(**{name: None}) == -1, name
        assert f(**{name: at(11, 8)}) == -2, name
    assert f(ws=None) == f(wsb=16) == f(ws=at(10, 8)) == -11
    for i in range(1, 9):
        assert f(y=at(i)) == -5 and f(ws=at(i)) == -5, i
    assert f(ws=at(9)) == -5
    assert f(T=0, x=None) == 0
    assert L.macaq_moe_workspace_bytes(0, 2, 256) == L.macaq_moe_workspace_bytes(129, 2, 256) == 0
    assert L.macaq_moe_workspace_bytes(16, 17, 256) == L.macaq_moe_workspace_bytes(16, 2, 300) == 0


@hidden_device
def test_gate_up_refused_by_name(L):
    def f(w=at(1), d=at(2), E=4, I=256, K=512, q=at(3), s=at(4)):
        return L.macaq_prepare_gate_up(w, d, E, I, K, q, s, None)

    assert f(E=0) == -6
    assert f(I=0) == f(I=32769) == f(I=4) == f(K=500) == -3
    assert f(w=None) == f(s=None) == -1
    assert f(d=at(2, 4)) == -2
    assert f(q=at(1)) == f(s=at(3)) == -5


@hidden_device
def test_valid_calls_without_a_device_are_a_named_cuda_error(L):
    assert L.macaq_block_norm(at(1), BF16, None, None, None, 0, 1, at(5), 1.0, 1e-6, 0.0, None, at(7), 4, 64, None) == -8
    assert L.macaq_moe_route(at(1), FP32, 4, 8, 2, 0, 1, 1.0, at(2), at(3), None, None, None, 0, None) == -8
