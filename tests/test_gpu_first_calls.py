"""The first calls of a process may come from many threads at once: what the library asks once
per device (attributes, how many clusters fit) is asked by all of them."""
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

PROGRAM = """
import threading, torch
import w4a4_mxfp4_quantize_b200 as mq

g = torch.Generator(device="cuda").manual_seed(1)
randn = lambda *s: torch.randn(*s, generator=g, device="cuda")
E, H, I, k = 8, 512, 256, 2
d_up, d_down = randn(E, H).abs() + 0.5, randn(E, I).abs() + 0.5
w_up, w_down = 0.02 * randn(E, 2 * I, H), 0.02 * randn(E, H, I)
data = [(randn(T, H).bfloat16(), randn(T, E)) for T in (1, 5, 17, 33, 64, 90, 127, 128)]
mq.lib()
torch.cuda.synchronize()
ready, got, failed = threading.Barrier(8), [None] * 8, []

def work(i):
    try:
        s, (x, l) = torch.cuda.Stream(), data[i]
        with torch.cuda.stream(s):
            ready.wait()
            up, down = mq.prepare_gate_up(w_up, d_up), mq.prepare_weights(w_down, d_down)
            y = mq.moe_mm(x, l, d_up, *up, d_down, *down, inner=I, k=k, stream=s)
            z = mq.dense_mm(x, d_up[0], *mq.prepare_weights(w_up[0], d_up[0]), N=2 * I, stream=s)
            r = mq.moe_route(l, k, stream=s)
            n = mq.block_norm(x, y, w_pre=d_up[0], stream=s)
        s.synchronize()
        got[i] = (y, z, *r, *n)
    except Exception as e:
        failed.append((i, e))

threads = [threading.Thread(target=work, args=(i,)) for i in range(8)]
[t.start() for t in threads]
[t.join() for t in threads]
assert not failed, failed
up, down = mq.prepare_gate_up(w_up, d_up), mq.prepare_weights(w_down, d_down)
for (x, l), have in zip(data, got):
    y = mq.moe_mm(x, l, d_up, *up, d_down, *down, inner=I, k=k)
    want = (y, mq.dense_mm(x, d_up[0], *mq.prepare_weights(w_up[0], d_up[0]), N=2 * I), *mq.moe_route(l, k),
            *mq.block_norm(x, y, w_pre=d_up[0]))
    assert all(torch.equal(a, b) for a, b in zip(have, want))
print("all equal")
"""


def test_first_calls_from_many_threads():
    r = subprocess.run([sys.executable, "-c", PROGRAM], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "all equal" in r.stdout, r.stdout[-1000:] + r.stderr[-3000:]
