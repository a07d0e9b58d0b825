"""The calls around the linear reach the library two ways: through the compiled module
(usual calls) and through ctypes (another stream, given outputs, no sorting, odd integer
types).  Both give the same bits, the same refusals, and work from any device and stream."""
import pytest
import torch

import w4a4_mxfp4_quantize_b200 as mq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    mq.build()
    mq.lib()
    torch.cuda.init()


@pytest.fixture
def slow(monkeypatch):
    """Calls f through ctypes alone."""
    def run(f):
        with monkeypatch.context() as m:
            m.setattr(mq, "_fast", None)
            return f()
    return run


def same(a, b):
    a, b = (a, b) if isinstance(a, tuple) else ((a,), (b,))
    for x, y in zip(a, b, strict=True):
        assert (x is None and y is None) or (x.dtype == y.dtype and x.shape == y.shape and torch.equal(x, y))


def randn(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def test_the_compiled_module_is_loaded():
    assert mq._fast is not None


@pytest.mark.parametrize("stream_type", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("gate", [None, "token", "channel", "sequence"])
@pytest.mark.parametrize("pre", [True, False])
def test_norm_both_ways(slow, stream_type, gate, pre):
    M, C = 37, 160
    h, y, w = randn(M, C).to(stream_type), randn(M, C, seed=1).bfloat16(), randn(C, seed=2)
    g, per = {None: (None, None), "token": (randn(M, C, seed=3), None), "channel": (randn(C, seed=3).bfloat16(), None),
              "sequence": (randn(4, C, seed=3).bfloat16(), 10)}[gate]

    def f():
        return mq.block_norm(h, y, w_post=w, gate=g, rows_per_gate=per, w_pre=w if pre else None, scale=0.5)

    assert mq._fast.block_norm(h, y, w, None if gate == "channel" else g, per, w, 0.5, 1e-6, 0.0) is not None
    same(f(), slow(f))


@pytest.mark.parametrize("T,E,k", [(1, 8, 2), (300, 128, 8)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_route_both_ways(slow, T, E, k, dtype):
    l = randn(T, E).to(dtype)
    for kw in ({}, {"score": mq.SCORE_SIGMOID, "renorm": False, "scale": 2.5}):
        assert mq._fast.moe_route(l, k, 0, True, 1.0) is not None
        same(mq.moe_route(l, k, **kw), slow(lambda: mq.moe_route(l, k, **kw)))


def layer(E=4, H=256, I=256):
    d1, d2 = randn(E, H, seed=4).abs() + 0.5, randn(E, I, seed=5).abs() + 0.5
    up = mq.prepare_gate_up(0.02 * randn(E, 2 * I, H, seed=6), d1)
    down = mq.prepare_weights(0.02 * randn(E, H, I, seed=7), d2)
    return (d1, *up, d2, *down)


@pytest.mark.parametrize("T", [1, 40])
def test_layer_both_ways(slow, T):
    args, x, l = layer(), randn(T, 256).bfloat16(), randn(T, 4, seed=1)

    def f():
        return mq.moe_mm(x, l, *args, inner=256, k=2)

    assert mq._fast.moe_mm(x, l, *args, 256, 2, 0, True, 1.0, 5) is not None
    same(f(), slow(f))
    out = torch.empty_like(x)
    assert mq.moe_mm(x, l, *args, inner=256, k=2, out=out) is out
    same(out, f())


def test_what_the_short_way_leaves_to_the_other():
    h, y, w = randn(8, 64).bfloat16(), randn(8, 64, seed=1).bfloat16(), randn(64, seed=2)
    for change in (dict(y=y.float()), dict(w=w[:32]), dict(h=h[:, :32]), dict(y=y.t().contiguous().t()), dict(y=None),
                   dict(y=y.cpu()), dict(h=h.half())):
        a = dict(h=h, y=y, w=w) | change
        assert mq._fast.block_norm(a["h"], a["y"], a["w"], None, None, w, 1.0, 1e-6, 0.0) is None, change
    for bad in (dict(y=y.float()), dict(w_post=w[:32]), dict(y=y.t().contiguous().t()), dict(y=y.cpu())):
        with pytest.raises(ValueError):
            mq.block_norm(**(dict(h=h, y=y, w_post=w, w_pre=w) | bad))
    l = randn(5, 6)
    assert mq._fast.moe_route(l, 7, 0, True, 1.0) is None and mq._fast.moe_route(l.t(), 2, 0, True, 1.0) is None
    same(mq.moe_route(l, 2, scale=1), mq.moe_route(l, 2))  # an int factor goes the other way
    args, x, l = layer(), randn(3, 256).bfloat16(), randn(3, 4)
    for i in range(6):
        short = [*args]
        short[i] = short[i].reshape(-1)[:-1]
        assert mq._fast.moe_mm(x, l, *short, 256, 2, 0, True, 1.0, 5) is None
        with pytest.raises(ValueError):
            mq.moe_mm(x, l, *short, inner=256, k=2)


def test_refusals_of_the_library_are_the_same(slow):
    h, y, w = randn(4, 24).bfloat16(), randn(4, 24).bfloat16(), randn(24)  # 24 columns: not a multiple of 16
    for call in (lambda: mq.block_norm(h, y, w_pre=w), lambda: slow(lambda: mq.block_norm(h, y, w_pre=w))):
        with pytest.raises(mq.MacaqError) as e:
            call()
        assert e.value.status == -3
    big = randn(4, 64).bfloat16()
    with pytest.raises(mq.MacaqError) as e:
        mq.block_norm(big, big.clone(), w_pre=randn(64), eps=float("nan"))
    assert e.value.status == -14
    args, x, l = layer(), randn(3, 256).bfloat16(), randn(3, 4)
    for act in (0, 1, 4):
        with pytest.raises(mq.MacaqError) as e:
            mq.moe_mm(x, l, *args, inner=256, k=2, act_type=act)
        assert e.value.status == -13
    wide = randn(129, 256).bfloat16()
    with pytest.raises(mq.MacaqError) as e:
        mq.moe_mm(wide, randn(129, 4), *args, inner=256, k=2)
    assert e.value.status == -3


def test_streams_of_both_ways():
    # work queued on a side stream right before the call is what the call reads
    s = torch.cuda.Stream()
    h, w = torch.zeros(2000, 1024, device="cuda"), torch.ones(1024, device="cuda")
    y = torch.zeros(2000, 1024, device="cuda", dtype=torch.bfloat16)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for _ in range(20):
            h.add_(1.0)
        got, _ = mq.block_norm(h, y, w_pre=w)
        h.zero_()
    s.synchronize()
    assert (got == 20).all()
    with torch.cuda.stream(s):
        for _ in range(20):
            h.add_(1.0)
    got, _ = mq.block_norm(h, y, w_pre=w, stream=s)
    s.synchronize()
    assert (got == 20).all()
