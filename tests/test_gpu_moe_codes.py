"""The two halves of moe_mm on inputs whose first linear is exact in FP32 (layer_check.py): every
block of the stored activations is a rounding of act(g) u, and y follows from the stored codes.

y: the second linear's products add up exactly or are off by K / 32 roundings of 2^-23 of the
sum S of magnitudes, each expert's weight by 2^-17 of it (tests of routing), the k products and
sums by 2^-23 each, and y is rounded once (2^-8 of itself, half a step is 2^-9)."""
import numpy as np
import pytest
import torch

import oracle
import w4a4_mxfp4_quantize_b200 as mq
from layer_check import GELU, SILU, check_blocks, narrow_layer, narrow_tokens

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    mq.build()
    mq.lib()
    torch.cuda.init()


def cuda(a):
    return torch.from_numpy(a).cuda()


# one token to the most, groups of one expert from none to several; widths at and across a quantiser
# pass, one and many K tiles, clusters of 8 to 1, both ways of choosing (T k above and up to 32)
@pytest.mark.parametrize("E,H,I,T,k", [(4, 256, 256, 1, 1), (8, 512, 256, 3, 8), (8, 512, 768, 16, 2), (3, 1280, 512, 21, 2),
                                       (8, 512, 256, 128, 4), (6, 2048, 768, 37, 3), (2, 4096, 256, 5, 1),
                                       (2, 8192, 512, 17, 2), (64, 256, 1024, 100, 8), (2, 256, 8192, 33, 1)])
@pytest.mark.parametrize("act", [SILU, GELU])
def test_every_block(E, H, I, T, k, act):
    w_up, w_down, d_up, d_down = narrow_layer(E, H, I, seed=H + I + E)
    bits = narrow_tokens(T, H, seed=T)
    x = torch.from_numpy(bits.view(np.int16)).view(torch.bfloat16).cuda()
    logits = cuda(np.random.default_rng(k).standard_normal((T, E)).astype(np.float32))
    args = (cuda(d_up), *mq.prepare_gate_up(cuda(w_up), cuda(d_up)), cuda(d_down), *mq.prepare_weights(cuda(w_down), cuda(d_down)))
    ws = torch.zeros(mq.moe_workspace_bytes(T, k, I), dtype=torch.uint8, device="cuda")
    y = mq.moe_mm(x, logits, *args, inner=I, k=k, act_type=act, ws=ws).double().cpu().numpy()
    ids, w, _, _ = mq.moe_route(logits, k, sort=False)
    ids, w, ws = ids.cpu().numpy(), w.double().cpu().numpy(), ws.cpu().numpy()
    codes = ws[: T * k * I // 2].reshape(T, k, I // 2)
    scales = ws[T * k * I // 2 : T * k * I * 17 // 32].reshape(T, k, I // 32)
    want, off, size = np.zeros((T, H)), np.zeros((T, H)), np.zeros((T, H))
    for e in range(E):
        t, j = np.nonzero(ids == e)
        if not len(t):
            continue
        check_blocks(codes[t, j], scales[t, j], np.ascontiguousarray(bits[t]), d_up[e], w_up[e], d_down[e], act)
        a = oracle.dequantize(codes[t, j], scales[t, j])
        v = oracle.dequantize(*oracle.quantize_weights(w_down[e], d_down[e]))
        part, we = a @ v.T / 32, w[t, j][:, None]
        want[t] += we * part
        off[t] += we * (I / 32 * 2.0 ** -23) * (np.abs(a) @ np.abs(v).T) / 32
        size[t] += we * np.abs(part)
    off += ((k + 2) * 2.0 ** -23 + 2.0 ** -17) * size
    off += 2.0 ** -8 * (np.abs(want) + off)
    assert (np.abs(y - want) <= off).all()


def test_the_layer_of_128_experts():
    # the sizes of the 128-expert layer, its weights made on the device, the experts of 24 tokens checked
    E, H, I, T, k = 128, 2048, 768, 24, 8
    w_up, w_down, d_up, d_down = narrow_layer(4, H, I, seed=7)  # four experts' weights, each 32 times
    rep = lambda a: cuda(a).repeat(E // 4, *[1] * (a.ndim - 1)).contiguous()
    bits = narrow_tokens(T, H, seed=8)
    x = torch.from_numpy(bits.view(np.int16)).view(torch.bfloat16).cuda()
    logits = cuda(np.random.default_rng(9).standard_normal((T, E)).astype(np.float32))
    du, dd = rep(d_up), rep(d_down)
    up, down = mq.prepare_gate_up(rep(w_up), du), mq.prepare_weights(rep(w_down), dd)
    ids = mq.moe_route(logits, k, sort=False)[0].cpu().numpy()
    for act in (SILU, GELU):
        ws = torch.zeros(mq.moe_workspace_bytes(T, k, I), dtype=torch.uint8, device="cuda")
        mq.moe_mm(x, logits, du, *up, dd, *down, inner=I, k=k, act_type=act, ws=ws)
        out = ws.cpu().numpy()
        codes = out[: T * k * I // 2].reshape(T, k, I // 2)
        scales = out[T * k * I // 2 : T * k * I * 17 // 32].reshape(T, k, I // 32)
        for e in range(4):
            t, j = np.nonzero(ids % 4 == e)
            check_blocks(codes[t, j], scales[t, j], np.ascontiguousarray(bits[t]), d_up[e], w_up[e], d_down[e], act)


def test_grouped_calls_on_the_interleaved_images():
    # the images of prepare_gate_up serve grouped_mm too: its columns 2 c and 2 c + 1 are gate and up of channel c
    E, H, I, T, k = 8, 512, 256, 300, 2
    w_up, _, d_up, _ = narrow_layer(E, H, I, seed=3)
    bits = narrow_tokens(T, H, seed=4)
    x = torch.from_numpy(bits.view(np.int16)).view(torch.bfloat16).cuda()
    logits = cuda(np.random.default_rng(5).standard_normal((T, E)).astype(np.float32))
    _, _, counts, order = mq.moe_route(logits, k)
    rows, d = x[order.long() // k].contiguous(), cuda(d_up)
    pairs = mq.grouped_mm(rows, d, *mq.prepare_gate_up(cuda(w_up), d), counts, 1, 2 * I)
    halves = mq.grouped_mm(rows, d, *mq.prepare_weights(cuda(w_up), d), counts, 1, 2 * I)
    assert torch.equal(pairs[:, 0::2], halves[:, :I]) and torch.equal(pairs[:, 1::2], halves[:, I:])


def test_one_copy_of_the_weights_for_few_tokens_and_many():
    # the layer's call, and routing with two grouped calls on the same images as it is written for more tokens
    E, H, I, T, k = 16, 512, 512, 128, 4
    w_up, w_down, d_up, d_down = narrow_layer(E, H, I, seed=11)
    n = torch.from_numpy(narrow_tokens(T, H, seed=12).view(np.int16)).view(torch.bfloat16).cuda()
    logits = cuda(np.random.default_rng(13).standard_normal((T, E)).astype(np.float32))
    D_up, D_down = cuda(d_up), cuda(d_down)
    up, down = mq.prepare_gate_up(cuda(w_up), D_up), mq.prepare_weights(cuda(w_down), D_down)
    few = mq.moe_mm(n, logits, D_up, *up, D_down, *down, inner=I, k=k)
    ids, weights, counts, order = mq.moe_route(logits, k)
    token, order = order.long() // k, order.long()
    u = mq.grouped_mm(n[token], D_up, *up, counts, group_list_type=1, N=2 * I)
    a = (torch.nn.functional.silu(u[:, 0::2].float()) * u[:, 1::2].float()).bfloat16()
    v = mq.grouped_mm(a, D_down, *down, counts, group_list_type=1, N=H)
    many = torch.zeros_like(n, dtype=torch.float32).index_add_(0, token, v * weights.view(-1)[order][:, None])
    # the grouped calls round g and u to bf16, so an activation moves by up to d = 2^-7 of itself and its four-bit
    # code crosses a border with probability d / s, then moving by the grid's step s <= 1/2 of the value: a mean square
    # of d s <= 2^-8, 2^-4 of the output, and the experts' outputs' own rounding
    assert (few.float() - many).norm() / many.norm() < 2.0 ** -4 + 2.0 ** -8
