"""moe_route against its definition in 64 bits.

The choice compares the logits themselves, so ids, counts and order are exact.  A
weight is an exponential (the fast FP32 exponential of x is within (2 + |x|) x 2^-22
of itself: 2 ulp of the power of two and the rounding of its argument), a sum of up
to 1024 non-negative terms (at most 42 additions in a row) and a division (2 ulp):
    (2 (2 + span) + 12 + 4) x 2^-22 of the value, span the largest |l - max|, or |l|
for a sigmoid.
"""
import pytest
import torch

import w4a4_mxfp4_quantize_b200 as mq

pytestmark = pytest.mark.gpu

INF = float("inf")
SCORES = [mq.SCORE_SOFTMAX, mq.SCORE_SIGMOID]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    mq.build()
    mq.lib()
    torch.cuda.init()


def logits_of(T, E, seed, dtype=torch.float32, ties=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    l = 1.5 * torch.randn(T, E, generator=g, device="cuda")
    return (l * 2).round().div(2).to(dtype) if ties else l.to(dtype)


def definition(logits, k, score, renorm, scale):
    """ids (ties to the lowest index, NaN as -inf) and weights in 64 bits."""
    l = logits.double()
    rank = torch.nan_to_num(l, nan=-INF, posinf=INF, neginf=-INF)
    ids = torch.sort(rank, dim=1, descending=True, stable=True).indices[:, :k]
    top = l.gather(1, ids)
    if score == mq.SCORE_SIGMOID:
        w = torch.sigmoid(top)
        w = torch.where(w < 2.0 ** -126, 0.0, w)
        total = w.sum(1, keepdim=True) if renorm else torch.ones_like(w[:, :1])
    else:
        first = top[:, :1]
        zero = first == -INF
        w = torch.where(top == -INF, 0.0, torch.exp(top - first))
        if renorm:
            total = w.sum(1, keepdim=True)
        else:
            total = torch.where(l == -INF, 0.0, torch.exp(l - first)).sum(1, keepdim=True)
        total = torch.where(zero & (total == 0), 1.0, total)
    return ids, scale * w / torch.where(total == 0, 1.0, total)


def check(logits, k, score, renorm, scale=1.0, sort=True):
    ids, w, counts, order = mq.moe_route(logits, k, score=score, renorm=renorm, scale=scale, sort=sort)
    T, E = logits.shape
    want_ids, want = definition(logits, k, score, renorm, scale)
    assert ids.dtype == torch.int32 and torch.equal(ids.long(), want_ids)
    l = logits.double()
    # an exponential of less than -88 is below 2^-126: its relative error does not matter
    span = (l if score == mq.SCORE_SIGMOID else l.amax(1, keepdim=True) - l).abs()
    span = torch.nan_to_num(span, nan=0.0, posinf=0.0).clamp_max(88.0).amax(1, keepdim=True)
    tol = (2 * (2 + span) + 16) * 2.0 ** -22
    assert torch.equal(torch.isnan(want), torch.isnan(w))
    ok = (w.double() - want).abs() <= tol * want.abs() + 2.0 ** -126
    assert (ok | torch.isnan(want)).all(), (w.double() - want).abs().max()
    if not sort:
        assert counts is None and order is None
        return ids, w
    flat = want_ids.reshape(-1)
    assert torch.equal(counts, torch.bincount(flat, minlength=E))
    assert torch.equal(order.long(), torch.sort(flat, dim=0, stable=True).indices)
    return ids, w


# one CTA (one run of 64 tokens), several, more runs than CTAs (ragged last), every keys-per-lane form
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 128, 8), (2, 4, 4), (63, 60, 4), (64, 33, 5), (65, 128, 8), (129, 7, 7),
                                   (300, 200, 16), (1001, 60, 4), (777, 512, 32), (70, 1024, 32), (8192, 128, 8),
                                   (9473, 64, 2), (30001, 16, 3)])
@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("renorm", [True, False])
def test_sizes(T, E, k, score, renorm):
    check(logits_of(T, E, T + E), k, score, renorm, scale=2.5 if renorm else 1.0)


@pytest.mark.parametrize("ties", [True, False])
@pytest.mark.parametrize("E", [30, 128, 600])
def test_bf16_logits_and_ties(E, ties):
    check(logits_of(333, E, E, torch.bfloat16, ties), 6, mq.SCORE_SOFTMAX, True)
    check(torch.zeros((70, E), device="cuda"), 6, mq.SCORE_SIGMOID, True)  # all equal: experts 0..5
    signed = torch.zeros((2, E), device="cuda")
    signed[:, ::2] = -0.0                                                  # -0 ties with +0
    check(signed, 6, mq.SCORE_SOFTMAX, False)


@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("renorm", [True, False])
def test_masked_and_non_finite_logits(score, renorm):
    lowest = torch.finfo(torch.float32).min
    l = logits_of(12, 40, 3)
    l[0] = -INF                      # nothing left: the first k experts, weight zero
    l[1, 3:] = -INF                  # fewer than k left
    l[2] = lowest                    # a mask of the type's lowest value
    l[3, 5:] = lowest
    l[4, 7] = float("nan")           # not chosen
    l[5, :] = float("nan")           # every logit
    l[6, 8] = INF
    l[7, 4:] = float("nan")          # fewer than k numbers: NaNs are chosen, in order
    l[8, :20] = -INF
    l[9] = -100.0
    l[10] = 60.0
    ids, w = check(l, 6, score, renorm)
    assert ids[0].tolist() == [0, 1, 2, 3, 4, 5] and (w[0] == 0).all()
    assert (w[1, 3:] == 0).all() and (w[1, :3] > 0).all()


def test_without_sorting_and_no_tokens():
    check(logits_of(500, 96, 1), 8, mq.SCORE_SOFTMAX, True, sort=False)
    ids, w, counts, order = mq.moe_route(torch.empty((0, 12), device="cuda"), 3)
    assert ids.shape == (0, 3) and w.shape == (0, 3) and order.shape == (0,) and (counts == 0).all()


def test_streams_graphs_and_regrown_workspace():
    a, b = logits_of(2000, 64, 4), logits_of(2000, 64, 5)
    live = a.clone()
    graphs, outs = [], []
    for _ in range(2):  # two graphs of the same call, replayed on two streams at once
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(mq.moe_route(live, 4))
        graphs.append(g)
    mq.moe_route(logits_of(20000, 512, 6), 4)  # the kept workspace grows
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for src in (a, b):
        live.copy_(src)
        torch.cuda.synchronize()
        for _ in range(20):
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        want = mq.moe_route(src, 4)
        for o in outs:
            assert all(torch.equal(x, y) for x, y in zip(o, want))


def test_counts_and_order_drive_the_grouped_linear():
    # the sorted rows through grouped_mm are each expert's rows through dense_mm
    T, E, k, K, N = 200, 6, 2, 256, 64
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn(T, K, generator=g, device="cuda").bfloat16()
    W = 0.02 * torch.randn(E, N, K, generator=g, device="cuda")
    D = torch.rand(E, K, generator=g, device="cuda") + 0.5
    ids, w, counts, order = mq.moe_route(logits_of(T, E, 7), k)
    rows = x[order.long() // k].contiguous()
    y = mq.grouped_mm(rows, D, *mq.prepare_weights(W, D), counts, 1, N)
    for e in range(E):
        mine = ids.reshape(-1)[order.long()] == e
        alone = mq.dense_mm(rows[mine].contiguous(), D[e], *mq.prepare_weights(W[e], D[e]), N)
        assert torch.allclose(y[mine].float(), alone.float(), rtol=2.0 ** -7, atol=1e-3)
