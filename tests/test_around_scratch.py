"""Scratch of the calls around the linear: each call has its own, so threads that share a
stream do not share it (their two-kernel calls may be queued interleaved)."""
import threading

import pytest
import torch

import w4a4_mxfp4_quantize_b200 as mq


def test_calls_at_once_never_share_scratch(monkeypatch):
    # two calls on one stream that are both between their allocation and their second launch
    empty = torch.empty

    def on_cpu(*a, device=None, **kw):
        return empty(*a, **kw)

    monkeypatch.setattr(torch, "empty", on_cpu)
    monkeypatch.setattr(torch, "zeros", lambda *a, device=None, **kw: empty(*a, **kw).zero_())
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(mq, "_raw_stream", lambda dev: 0)
    monkeypatch.setattr(mq, "_ws", {(0, 0): empty(1 << 20, dtype=torch.uint8)})  # what an earlier linear left
    a, b = mq._scratch(1000, 0, None), mq._scratch(1000, 0, None)
    assert a.numel() >= 1000 and a.data_ptr() != b.data_ptr()
    assert mq._scratch(0, 0, None) is None
    given = empty(1000, dtype=torch.uint8)
    assert mq._scratch(1000, 0, given) is given
    with pytest.raises(mq.MacaqError):
        mq._scratch(1001, 0, given)


@pytest.mark.gpu
def test_threads_on_one_stream():
    mq.build()
    mq.lib()
    E, H, I, k, g = 16, 512, 256, 4, torch.Generator(device="cuda").manual_seed(1)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    d_up, d_down = randn(E, H).abs() + 0.5, randn(E, I).abs() + 0.5
    args = (d_up, *mq.prepare_gate_up(0.02 * randn(E, 2 * I, H), d_up), d_down,
            *mq.prepare_weights(0.02 * randn(E, H, I), d_down))
    calls = [(randn(T, H).bfloat16(), randn(T, E)) for T in (20, 60, 100, 128)]  # the tables go through the scratch
    routed = [randn(T, E) for T in (100, 300, 700, 2000)]
    want = [mq.moe_mm(x, l, *args, inner=I, k=k).clone() for x, l in calls]
    orders = [mq.moe_route(l, k) for l in routed]
    torch.cuda.synchronize()
    stream, failed = torch.cuda.Stream(), []

    def work(i):
        try:
            x, l = calls[i]
            for _ in range(100):
                with torch.cuda.stream(stream):
                    y = mq.moe_mm(x, l, *args, inner=I, k=k, stream=stream)  # the ctypes way
                    r = mq.moe_route(routed[i], k, stream=stream)
                    if not torch.equal(y, want[i]) or not all(torch.equal(a, b) for a, b in zip(r, orders[i])):
                        failed.append(i)
        except Exception as e:
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
