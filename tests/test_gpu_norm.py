"""block_norm against its formula in 64 bits.

Tolerances, counted before the first run.  A rounding to bf16 is off by at most
2^-8 of the value, one to fp32 by 2^-24.  In FP32 the mean of squares is a sum of
non-negative terms over at most 64 additions in a row (a thread's own elements,
then two trees of five), so it is within 64 x 2^-24 of itself and its inverse root
within 32 x 2^-24, the root's own 2 ulp (4 x 2^-24) and at most six products beside
it: 48 x 2^-24 bounds the branch and the normed row.
  h':  48 x 2^-24 |s gate p| + 2^-24 |h'| and one rounding to the stream's type
  n:   from the h' that the call returned, 48 x 2^-24 |n| and one rounding to bf16
The widest rows (wide: their threads add up to 64 elements each, read again) have
up to 140 additions: 96 x 2^-24 there.
"""
import pytest
import torch

import w4a4_mxfp4_quantize_b200 as mq

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _lib():
    mq.build()
    mq.lib()
    torch.cuda.init()


def inputs(M, C, seed=0, stream=torch.bfloat16, gate="none", post=True, gate_dtype=torch.bfloat16, per=1):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    a = dict(h=(4 * normal(M, C)).to(stream), y=(2 * normal(M, C)).bfloat16(),
             w_post=1 + 0.2 * normal(C) if post else None, w_pre=1 + 0.2 * normal(C), scale=0.22, eps=EPS)
    if gate == "token":
        a["gate"] = normal(M, C).to(gate_dtype)
    elif gate == "channel":
        a["gate"] = normal(C).to(gate_dtype)
    elif gate == "sequence":
        a["gate"], a["rows_per_gate"] = normal(-(-M // per), C).to(gate_dtype), per
    return a


def rms(v, w, eps, offset):
    return v / torch.sqrt(v.square().mean(1, keepdim=True) + eps) * (offset + w.double())


def branch_of(a, offset=0.0):
    b = a["y"].double()
    if a.get("w_post") is not None:
        b = rms(b, a["w_post"], a["eps"], offset)
    gate = a.get("gate")
    if gate is not None:
        rows = torch.arange(len(b), device=b.device) // a.get("rows_per_gate", 1)
        b = b * (gate.double()[None] if gate.dim() == 1 else gate.double()[rows])
    return a["scale"] * b


def check(a, h, n, offset=0.0, sums=48):
    half = torch.finfo(h.dtype).eps / 2
    b = branch_of(a, offset)
    want = a["h"].double() + b
    # the rounding to the stream's type is of a value that may itself be off
    off = sums * U * b.abs() + U * want.abs()
    assert ((h.double() - want).abs() <= off + half * (want.abs() + off)).all()
    want = rms(h.double(), a["w_pre"], a["eps"], offset)
    assert ((n.double() - want).abs() <= (2.0 ** -8 + 2 * sums * U) * want.abs()).all()


# widths: one warp, ragged last warp, the limits of each form (256, 512, 1024 with many rows; 8192; 16384), wide
@pytest.mark.parametrize("M,C", [(1, 16), (3, 48), (1, 2048), (7, 1040), (1300, 16), (1300, 256), (1201, 272),
                                 (1300, 512), (1200, 528), (1301, 1024), (1300, 1040), (5, 8192), (3, 8208),
                                 (4, 16384), (333, 5120)])
@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
def test_widths_and_rows(M, C, stream):
    a = inputs(M, C, seed=M + C, stream=stream)
    h, n = mq.block_norm(**a)
    assert h.dtype == stream and n.dtype == torch.bfloat16
    check(a, h, n)


@pytest.mark.parametrize("M,C", [(2, 16400), (301, 20480), (1, 65536)])
@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
def test_wide_rows(M, C, stream):
    a = inputs(M, C, seed=C, stream=stream, gate="channel")
    h, n = mq.block_norm(**a)
    check(a, h, n, sums=96)
    inplace = a["h"].clone()
    h2, n2 = mq.block_norm(**{**a, "h": inplace}, out_h=inplace)
    assert h2 is inplace and torch.equal(h2, h) and torch.equal(n2, n)


@pytest.mark.parametrize("gate,per", [("token", 1), ("channel", 1), ("sequence", 100), ("sequence", 257), ("sequence", 4000)])
@pytest.mark.parametrize("gate_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("M,C", [(257, 1152), (1500, 320)])
def test_gates(gate, per, gate_dtype, post, M, C):
    a = inputs(M, C, seed=per, gate=gate, gate_dtype=gate_dtype, post=post, per=per)
    check(a, *mq.block_norm(**a))


@pytest.mark.parametrize("M,C", [(9, 2048), (1500, 512), (2, 20480)])
def test_parts_alone_and_in_place(M, C):
    a = inputs(M, C, seed=5)
    whole_h, whole_n = mq.block_norm(**a)
    # no second norm; the first norm of a model (no branch); both together give what the whole call gives
    only_h, none = mq.block_norm(a["h"], a["y"], w_post=a["w_post"], scale=a["scale"], eps=EPS)
    assert none is None and torch.equal(only_h, whole_h)
    same, n = mq.block_norm(whole_h, w_pre=a["w_pre"], eps=EPS)
    assert same is whole_h and torch.equal(n, whole_n)
    h = a["h"].clone()
    out_n = torch.empty_like(whole_n)
    got_h, got_n = mq.block_norm(**{**a, "h": h}, out_h=h, out_n=out_n)
    assert got_h is h and got_n is out_n and torch.equal(h, whole_h) and torch.equal(out_n, whole_n)


def test_weight_offset_and_eps():
    a = inputs(40, 768, seed=6)
    a.update(w_post=a["w_post"] - 1, w_pre=a["w_pre"] - 1, eps=0.5)
    h, n = mq.block_norm(**a, weight_offset=1.0)
    check(a, h, n, offset=1.0)


def test_zero_rows_zero_values_and_infinities():
    a = inputs(4, 256, seed=7)
    a["h"][0] = 0
    a["y"][:2] = 0                 # 0 / sqrt(0 + eps) = 0
    a["y"][2, 5] = float("inf")    # inf / inf in its own place, 0 beside it
    h, n = mq.block_norm(**a)
    assert (h[0] == 0).all() and (n[0] == 0).all()
    assert torch.equal(h[1], a["h"][1])
    assert torch.isnan(h[2, 5]) and torch.isnan(n[2]).all()
    keep = torch.arange(256, device="cuda") != 5
    assert torch.equal(h[2, keep], a["h"][2, keep])
    b = {**a, "h": a["h"][3:], "y": a["y"][3:]}
    check(b, h[3:], n[3:])
    empty = mq.block_norm(a["h"][:0], a["y"][:0], w_pre=a["w_pre"])
    assert empty[0].shape == empty[1].shape == (0, 256)


def test_offsets_past_32_bits():
    # 2^31 + 64 K elements of bf16 (4.3 GB): the last rows lie past 32-bit element and byte offsets
    C = 8192
    M = 2 ** 31 // C + 8
    h = torch.zeros((M, C), dtype=torch.bfloat16, device="cuda")
    tail = inputs(16, C, seed=8)
    h[-16:] = tail["h"]
    _, n = mq.block_norm(h, w_pre=tail["w_pre"], eps=EPS)
    want = rms(tail["h"].double(), tail["w_pre"], EPS, 0.0)
    assert ((n[-16:].double() - want).abs() <= (2.0 ** -8 + 96 * U) * want.abs()).all()
    assert (n[:1000] == 0).all()


def test_streams_and_graphs():
    a, b = inputs(64, 1024, seed=9), inputs(64, 1024, seed=10)
    want = [t.clone() for t in mq.block_norm(**a)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = mq.block_norm(**a, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    live = {k: v.clone() if torch.is_tensor(v) else v for k, v in a.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h, n = mq.block_norm(**live)
        h2, n2 = mq.block_norm(h, n, w_post=live["w_post"], w_pre=live["w_pre"])  # a second block follows
    for src in (a, b):
        for k in ("h", "y", "w_post", "w_pre"):
            live[k].copy_(src[k])
        graph.replay()
        eager = mq.block_norm(**src)
        eager2 = mq.block_norm(eager[0], eager[1], w_post=src["w_post"], w_pre=src["w_pre"])
        for x, y in zip((h, n, h2, n2), (*eager, *eager2)):
            assert torch.equal(x, y)
