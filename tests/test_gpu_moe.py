"""moe_mm, the mixture-of-experts layer for a few tokens, against its formula in 64 bits.

The layer quantises twice, and a value on a border of a rounding may fall on either
side of it, so the two halves are checked one after the other; the quantised
activations between them are in the workspace.  The up linear's codes are bit-exact
(the oracle's).  The products of 32 four-bit codes add up exactly, so a linear rounds
K / 32 times, each within 2^-23 of the running sum of magnitudes S: d = K / 32 x 2^-23 S.
  a:  act(g) u moves by at most (1.13 |u| + |act(g)|) d (the slopes of SILU and GELU
      stay below 1.13), the exponential and the division add (4 + |z|) 2^-22 of it.
      Where the whole interval rounds to one bf16 value for each of a block's 32
      elements, the block's codes and scale must be the oracle's.  Elsewhere a value may
      move by a step of bf16, its scaled value by that and one more rounding, the rotated
      ones by the sum of these and a rounding; both encodings are within two units of
      their scale of what they encode (saturation at 6 of up to 8).
  y:  from the codes that the call left, d per expert weighted by |w|, k + 2 products
      and sums of the experts, (k + 2) 2^-23 sum |w y|, the weights' own error (2^-17,
      tests of routing) and one rounding to bf16 (2^-8).
"""
import numpy as np
import pytest
import torch

import oracle
import synth
import w4a4_mxfp4_quantize_b200 as mq

pytestmark = pytest.mark.gpu

INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    mq.build()
    mq.lib()
    torch.cuda.init()


class Layer:
    """Seeded weights of a layer, prepared, and their dequantised values per expert (by the oracle)."""

    def __init__(self, E, H, I, seed=0):
        rng = np.random.default_rng(seed)
        self.E, self.H, self.I = E, H, I
        self.w_up, self.w_down = synth.make_w(E, 2 * I, H, rng), synth.make_w(E, H, I, rng)
        self.d_up = np.exp2(rng.uniform(-2, 2, (E, H))).astype(np.float32)
        self.d_down = np.exp2(rng.uniform(-2, 2, (E, I))).astype(np.float32)
        self.d_up[:, 5] *= -1  # factors may be negative
        up = mq.prepare_gate_up(torch.from_numpy(self.w_up).cuda(), torch.from_numpy(self.d_up).cuda())
        down = mq.prepare_weights(torch.from_numpy(self.w_down).cuda(), torch.from_numpy(self.d_down).cuda())
        self.args = (torch.from_numpy(self.d_up).cuda(), *up, torch.from_numpy(self.d_down).cuda(), *down)

    def values(self, W, D, e):
        return oracle.dequantize(*oracle.quantize_weights(W[e], D[e]))

    def tokens(self, T, seed):
        rng = np.random.default_rng(seed)
        bits = synth.make_x(T, self.H, rng)
        return bits, torch.from_numpy(bits.view(np.int16)).view(torch.bfloat16).cuda()

    def logits(self, T, seed, scale=1.5):
        rng = np.random.default_rng(seed)
        return torch.from_numpy((scale * rng.standard_normal((T, self.E))).astype(np.float32)).cuda()


def product(a, values):
    """The exact products of dequantised activations [n, K] and weights [N, K], and what FP32 sums may be off."""
    return (a @ values.T) / 32, a.shape[1] / 32 * 2.0 ** -23 * (np.abs(a) @ np.abs(values).T) / 32


def activation(g, act):
    z = g if act == mq.ACT_SILU else 2 * np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)
    return g / (1 + np.exp(-z)), np.abs(z)


def bf16(v):
    return synth.bf16_bits_to_f32(oracle.f64_to_bf16(v)).astype(np.float64)


def check_activations(codes, scales, a, tol, D):
    """The stored operand [n, K] against the activations a +- tol; returns its values."""
    lo, mid, hi = bf16(a - tol), bf16(a), bf16(a + tol)
    want_codes, want_scales = oracle.quantize_act(oracle.f64_to_bf16(a), D)
    n, K = a.shape
    free = (lo != hi).reshape(n, K // 32, 32)
    same = ~free.any(-1)
    assert (scales == want_scales)[same].all()
    assert (codes.reshape(n, -1, 16) == want_codes.reshape(n, -1, 16)).all(-1)[same].all()
    got, want = oracle.dequantize(codes, scales), oracle.dequantize(want_codes, want_scales)
    r = np.abs(1 / D.astype(np.float64))
    moved = ((hi - lo) * r + 2.0 ** -7 * np.abs(mid) * r).reshape(n, K // 32, 32)
    moved = np.where(free, moved, 0).sum(-1)
    top = np.exp2(np.maximum(scales, want_scales).astype(np.float64) - 127)
    bound = moved + 2.0 ** -7 * 8 * top + 4 * top
    assert (np.abs(got - want).reshape(n, -1, 32).max(-1) <= bound)[~same].all()
    return got, same.mean()


def check(layer, bits, x, logits, k, act=mq.ACT_SILU, **route):
    T, H, I = len(bits), layer.H, layer.I
    ws = torch.full((max(16, mq.moe_workspace_bytes(T, k, I)),), 0xFF, dtype=torch.uint8, device="cuda")
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    y = mq.moe_mm(x, logits, *layer.args, inner=I, k=k, act_type=act, ws=ws, status=status, **route)
    torch.cuda.synchronize()
    assert status[0].item() == 0
    ids, w, _, _ = mq.moe_route(logits, k, sort=False, **route)
    ids, w = ids.cpu().numpy(), w.double().cpu().numpy()
    ws = ws.cpu().numpy()
    codes = ws[: T * k * I // 2].reshape(T, k, I // 2)
    scales = ws[T * k * I // 2 : T * k * I * 17 // 32].reshape(T, k, I // 32)
    want, off, size, exact = np.zeros((T, H)), np.zeros((T, H)), np.zeros((T, H)), []
    for e in range(layer.E):
        t, j = np.nonzero((ids == e) & (w != 0))
        if not len(t):
            continue
        up = oracle.dequantize(*oracle.quantize_act(np.ascontiguousarray(bits[t]), layer.d_up[e]))
        both, d = product(up, layer.values(layer.w_up, layer.d_up, e))
        g, u, dg, du = both[:, :I], both[:, I:], d[:, :I], d[:, I:]
        f, z = activation(g, act)
        tol = 1.13 * (np.abs(u) + du) * dg + np.abs(f) * du + (4 + z) * 2.0 ** -22 * np.abs(f * u) + 2.0 ** -130
        inner, share = check_activations(codes[t, j], scales[t, j], f * u, tol, layer.d_down[e])
        exact.append(share)
        part, d = product(inner, layer.values(layer.w_down, layer.d_down, e))
        we = w[t, j][:, None]
        want[t] += we * part
        off[t] += np.abs(we) * d
        size[t] += np.abs(we * part)
    off += ((k + 2) * 2.0 ** -23 + 2.0 ** -17) * size
    off += 2.0 ** -8 * (np.abs(want) + off)
    got = y.double().cpu().numpy()
    assert (np.abs(got - want) <= off).all(), np.max(np.abs(got - want) / np.maximum(off, 1e-300))
    # rows of weight zero are not written
    assert (codes[w == 0] == 0xFF).all() and (scales[w == 0] == 0xFF).all()
    return y


@pytest.fixture(scope="module")
def small():
    return Layer(8, 512, 256, seed=1)


# one token to the most; experts with none, one, exactly 16, 17 and all tokens (several groups of one expert)
@pytest.mark.parametrize("T,k", [(1, 1), (1, 8), (2, 3), (5, 2), (16, 1), (17, 8), (31, 3), (33, 2), (64, 4), (127, 1), (127, 2),
                                 (128, 8)])
@pytest.mark.parametrize("act", [mq.ACT_SILU, mq.ACT_GELU_TANH])
def test_tokens_and_choices(small, T, k, act):
    bits, x = small.tokens(T, T)
    check(small, bits, x, small.logits(T, k + T), k, act)


@pytest.mark.parametrize("score", [mq.SCORE_SOFTMAX, mq.SCORE_SIGMOID])
@pytest.mark.parametrize("renorm", [True, False])
def test_scores(small, score, renorm):
    bits, x = small.tokens(9, 2)
    check(small, bits, x, small.logits(9, 3), 3, score=score, renorm=renorm, scale=2.5)
    check(small, bits, x, small.logits(9, 3).bfloat16(), 3, score=score, renorm=renorm)


# widths: the least, more than a quantiser pass covers, more than the tokens' buffers hold twice; cluster sizes 8 to 1
@pytest.mark.parametrize("E,H,I,T,k", [(1, 256, 256, 3, 1), (3, 256, 1280, 20, 2), (4, 1280, 256, 7, 2), (2, 2048, 768, 40, 2),
                                       (5, 4096, 512, 9, 3), (2, 8192, 256, 18, 1), (2, 256, 8192, 18, 2),
                                       (70, 256, 256, 100, 4), (300, 256, 256, 30, 16), (512, 256, 256, 128, 16)])
def test_shapes(E, H, I, T, k):
    layer = Layer(E, H, I, seed=E + H)
    bits, x = layer.tokens(T, T)
    check(layer, bits, x, layer.logits(T, 4), k)


def test_skew(small):
    # all tokens choose the same experts: 8 groups of one expert, the others empty
    T = 128
    bits, x = small.tokens(T, 5)
    logits = small.logits(T, 6)
    logits[:, 2] += 50
    logits[:, 6] += 40
    check(small, bits, x, logits, 2)
    logits[:, 3] = -INF
    check(small, bits, x, logits, 5)


def test_masked_tokens_give_zeros(small):
    T, k = 20, 4
    bits, x = small.tokens(T, 7)
    logits = small.logits(T, 8)
    logits[3] = -INF            # padded rows
    logits[17:] = -INF
    logits[5, 2:] = -INF        # fewer experts than k
    x[18] = float("nan")        # what a padded row holds does not matter
    bits = x.view(torch.int16).cpu().numpy().view(np.uint16)
    y = check(small, bits, x, logits, k)
    assert (y[3] == 0).all() and (y[17:] == 0).all()
    logits[:] = -INF
    y = mq.moe_mm(x, logits, *small.args, inner=small.I, k=k)
    assert (y == 0).all()
    assert mq.moe_mm(x[:0], logits[:0], *small.args, inner=small.I, k=k).shape == (0, small.H)


def test_non_finite_tokens_stay_in_their_rows(small):
    T, k = 18, 2
    bits, x = small.tokens(T, 9)
    logits = small.logits(T, 10)
    want = mq.moe_mm(x, logits, *small.args, inner=small.I, k=k)
    bad, bad_logits = x.clone(), logits.clone()
    bad[4, 100] = float("nan")
    bad[11] = INF
    bad_logits[7, 3] = float("nan")
    bad_logits[7, :3] = -INF
    bad_logits[7, 4:] = -INF
    y = mq.moe_mm(bad, bad_logits, *small.args, inner=small.I, k=k)
    rows = [t for t in range(T) if t not in (4, 7, 11)]
    assert torch.equal(y[rows], want[rows])
    assert bool(torch.isnan(y[4]).all()) and bool(torch.isnan(y[11]).all())
    # row 7: all logits rank as -infinity, the lowest two are chosen, the NaN at 3 is neither chosen nor summed
    assert bool((y[7] == 0).all())
    bad_logits[7, 0] = float("nan")  # now it is chosen
    y = mq.moe_mm(bad, bad_logits, *small.args, inner=small.I, k=k)
    assert torch.equal(y[rows], want[rows]) and bool(torch.isnan(y[7]).all())


def test_same_as_the_grouped_path():
    # the layer against routing, two grouped linears and torch between them, at the 128-expert sizes
    E, H, I, T, k = 128, 2048, 768, 24, 8
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    w_up = 0.02 * torch.randn(E, 2 * I, H, generator=g, device="cuda")
    w_down = 0.02 * torch.randn(E, H, I, generator=g, device="cuda")
    d_up = torch.rand(E, H, generator=g, device="cuda") + 0.5
    d_down = torch.rand(E, I, generator=g, device="cuda") + 0.5
    logits = torch.randn(T, E, generator=g, device="cuda")
    y = mq.moe_mm(x, logits, d_up, *mq.prepare_gate_up(w_up, d_up), d_down, *mq.prepare_weights(w_down, d_down),
                  inner=I, k=k)
    ids, w, counts, order = mq.moe_route(logits, k)
    rows = x[order.long() // k].contiguous()
    both = mq.grouped_mm(rows, d_up, *mq.prepare_weights(w_up, d_up), counts, 1, 2 * I).float()
    inner = (torch.nn.functional.silu(both[:, :I]) * both[:, I:]).bfloat16()
    out = mq.grouped_mm(inner, d_down, *mq.prepare_weights(w_down, d_down), counts, 1, H).float()
    want = torch.zeros(T, H, device="cuda").index_add_(0, order.long() // k, out * w.reshape(-1)[order.long()][:, None])
    # The grouped path rounds g and u to bf16 too, which moves an activation by up to d = 2 x 2^-8 of itself.  A code
    # whose value moves by d crosses a border with probability d / s and then moves by s, the step of the four-bit
    # grid: a mean square of d s, with s at most half the value.  sqrt(2^-7 / 2) = 0.0625 of the output, and the
    # experts' outputs' own rounding, 2^-8.
    err = (y.float() - want).norm() / want.norm()
    assert err < 0.0625 + 2.0 ** -8, err


def test_repeated_calls_streams_graphs_and_devices(small):
    T, k = 31, 3
    _, xa = small.tokens(T, 11)
    _, xb = small.tokens(T, 12)
    la, lb = small.logits(T, 13), small.logits(T, 14)
    want = [mq.moe_mm(x, l, *small.args, inner=small.I, k=k).clone() for x, l in ((xa, la), (xb, lb))]
    for _ in range(30):  # back to back, the next call's first kernel overlapping the last one's second
        for (x, l), w in zip(((xa, la), (xb, lb)), want):
            assert torch.equal(mq.moe_mm(x, l, *small.args, inner=small.I, k=k), w)
    x, l = xa.clone(), la.clone()
    graphs, outs, streams = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(2):  # two graphs, replayed at the same time: each holds its own workspace
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(mq.moe_mm(x, l, *small.args, inner=small.I, k=k))
        graphs.append(g)
    for (xs, ls), w in zip(((xa, la), (xb, lb)), want):
        x.copy_(xs)
        l.copy_(ls)
        torch.cuda.synchronize()
        for _ in range(20):
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o in outs)
    side = streams[0]
    y = mq.moe_mm(xa, la, *small.args, inner=small.I, k=k, stream=side)
    side.synchronize()
    assert torch.equal(y, want[0])


def test_many_small_calls_at_once():
    # three CTAs of the second kernel share an SM here, of one call and of several: clusters of CTAs that wait for
    # one another, each with tensor memory of its own
    layer, T, k = Layer(8, 8192, 256, seed=21), 8, 2
    bits, x = layer.tokens(T, 22)
    logits = layer.logits(T, 23)
    check(layer, bits, x, logits, k)
    want = mq.moe_mm(x, logits, *layer.args, inner=256, k=k).clone()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    got = [mq.moe_mm(x, logits, *layer.args, inner=256, k=k, stream=s) for _ in range(25) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for y in got)


def test_a_block_as_it_is_used(small):
    # norm -> router logits -> layer -> norm with the residual, twice, captured and replayed
    T, k, H = 12, 2, small.H
    g = torch.Generator(device="cuda").manual_seed(15)
    h = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    router = 0.1 * torch.randn(small.E, H, generator=g, device="cuda").bfloat16()
    w1, w2 = (1 + 0.1 * torch.randn(H, generator=g, device="cuda") for _ in range(2))

    def block(h, n):
        y = mq.moe_mm(n, n @ router.t(), *small.args, inner=small.I, k=k)
        return mq.block_norm(h, y, w_post=w2, w_pre=w1, scale=0.5)

    def model():
        hh, n = mq.block_norm(h, w_pre=w1)
        for _ in range(2):
            hh, n = block(hh, n)
        return hh, n

    eager = [t.clone() for t in model()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = model()
    for _ in range(10):
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(out, eager))
    # and the layer inside it against the formula
    _, n = mq.block_norm(h, w_pre=w1)
    check(small, n.view(torch.int16).cpu().numpy().view(np.uint16), n, n @ router.t(), k)


def test_interleaved_images_hold_the_same_codes(small):
    # image row 2 c is gate row c, image row 2 c + 1 up row c
    E, I, H = small.E, small.I, small.H
    _, Wq, Ws = small.args[:3]
    codes, scales = mq.export_weights(Wq, Ws, E, 2 * I, H)
    for e in (0, E - 1):
        c, s = oracle.quantize_weights(small.w_up[e], small.d_up[e])
        order = np.arange(2 * I).reshape(2, I).T.reshape(-1)
        assert np.array_equal(codes[e].cpu().numpy(), c[order]) and np.array_equal(scales[e].cpu().numpy(), s[order])
