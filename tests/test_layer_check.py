"""The check of the layer's first half (layer_check.py) accepts what the formula gives, computed
in FP32, and refuses each planted mistake."""
import numpy as np
import pytest

import oracle
from layer_check import GELU, SILU, activation, check_blocks, exact_product, gate_and_up, narrow_layer, narrow_tokens, operand

SIZES = [(3, 256, 256), (9, 512, 512), (5, 2048, 768), (2, 8192, 256)]


def stored(bits, d_up, w_up, d_down, act, change=None):
    """What the layer stores for one expert, its activation computed in FP32, with a planted mistake."""
    if change == "one K tile dropped":
        K = bits.shape[1] - 256
        codes, scales = oracle.quantize_act(bits, d_up)
        wq, ws = oracle.quantize_weights(w_up, d_up)
        both = exact_product(operand(np.ascontiguousarray(codes[:, : K // 2]), np.ascontiguousarray(scales[:, : K // 32])),
                             operand(np.ascontiguousarray(wq[:, : K // 2]), np.ascontiguousarray(ws[:, : K // 32])))
        g, u = np.split(both, 2, 1)
    else:
        g, u = gate_and_up(bits, d_up, w_up)
    if change == "gate and up exchanged":
        g, u = u, g
    if change == "the other activation":
        act = SILU + GELU - act
    g, u = g.astype(np.float32), u.astype(np.float32)
    z = g if act == SILU else np.float32(2 * np.sqrt(2 / np.pi)) * (g + np.float32(0.044715) * g * g * g)
    a = g / (1 + np.exp(-z)) * u
    if change == "activations x 1.01":
        a = a * np.float32(1.01)
    if change == "one channel zero":
        a[:, 37] = 0
    if change == "one token's neighbour":
        a = np.roll(a, 1, 0)
    codes, scales = oracle.quantize_act(oracle.f64_to_bf16(a.astype(np.float64)), np.roll(d_down, 1) if change == "factors moved" else d_down)
    if change == "the low bit of the codes cleared":
        codes &= 0xEE
    if change == "one code":
        codes[0, 5] ^= 1
    if change == "one scale":
        scales[-1, -1] += 1
    return codes, scales


@pytest.mark.parametrize("T,H,I", SIZES)
@pytest.mark.parametrize("act", [SILU, GELU])
def test_accepts_the_formula_in_fp32(T, H, I, act):
    w_up, _, d_up, d_down = narrow_layer(1, H, I, seed=H + I)
    bits = narrow_tokens(T, H, seed=T)
    check_blocks(*stored(bits, d_up[0], w_up[0], d_down[0], act), bits, d_up[0], w_up[0], d_down[0], act)


@pytest.mark.parametrize("change", ["the other activation", "activations x 1.01", "one channel zero", "one K tile dropped",
                                    "the low bit of the codes cleared", "one code", "one scale", "gate and up exchanged",
                                    "one token's neighbour", "factors moved"])
@pytest.mark.parametrize("T,H,I", SIZES[1:])
@pytest.mark.parametrize("act", [SILU, GELU])
def test_refuses_mistakes(T, H, I, act, change):
    w_up, _, d_up, d_down = narrow_layer(1, H, I, seed=H + I)
    bits = narrow_tokens(T, H, seed=T)
    with pytest.raises(AssertionError, match="blocks are no rounding"):
        check_blocks(*stored(bits, d_up[0], w_up[0], d_down[0], act, change), bits, d_up[0], w_up[0], d_down[0], act)


def test_the_bound_covers_the_activation_in_fp32():
    g = np.linspace(-60, 60, 20001).astype(np.float32)
    for act in (SILU, GELU):
        a, tol = activation(g.astype(np.float64), np.float64(1.5), act)
        z = g if act == SILU else np.float32(2 * np.sqrt(2 / np.pi)) * (g + np.float32(0.044715) * g * g * g)
        with np.errstate(over="ignore"):
            got = g / (1 + np.exp(-z)) * np.float32(1.5)
        assert (np.abs(got - a) <= tol).all()
