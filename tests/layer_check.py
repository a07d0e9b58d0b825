"""What the first linear and the activation of moe_mm must leave in the workspace, block by block.

The inputs are narrow (no loud channels, factors within an octave of one), so that every
partial sum of a product is a whole number of its smallest terms and below 2^23 of them:
FP32 accumulation is then exact in any order, and g and u are known without error (this is
asserted from the operands, not assumed).  What is left is act(g) u in FP32, a rounding to
bf16 and the quantisation:
  the exponential is off by 2 + 1.16 |z| units of 2^-23 of itself, its argument z by
  1.25 |z| 2^-22 (GELU: five roundings of half a unit), the division by two units and the
  sum and product by half a unit each: (4 + 2 |z|) 2^-22 of act(g) u in all.  Below that, a
  quotient by more than 2^126 may be zero, which drops up to |g u| 2^-126 (z < -87), and a
  result below 2^-126 as well.
So almost every activation has one bf16 value, the others have two.  A block's 32 codes and
its scale must be the oracle's for one choice of these; no block is left out.
"""
import numpy as np

import oracle
import synth

SILU, GELU = 5, 2
MOST = 5  # activations of a block with two possible values: 32 choices


def narrow_layer(E, H, I, seed):
    """(w_up [E, 2 I, H], w_down [E, H, I], d_up [E, H], d_down [E, I])"""
    rng = np.random.default_rng(seed)
    w_up = (1.5 / np.sqrt(H) * rng.standard_normal((E, 2 * I, H))).astype(np.float32)
    w_down = (rng.standard_normal((E, H, I)) / np.sqrt(I)).astype(np.float32)
    d_up = np.exp2(rng.uniform(-0.5, 0.5, (E, H))).astype(np.float32)
    d_down = np.exp2(rng.uniform(-0.5, 0.5, (E, I))).astype(np.float32)
    return w_up, w_down, d_up, d_down


def narrow_tokens(T, H, seed):
    return synth.to_bf16_bits(np.random.default_rng(seed).standard_normal((T, H)).astype(np.float32))


def operand(codes, scales):
    """Values of an MXFP4 operand, and the exponent of its smallest step in each row."""
    return oracle.dequantize(codes, scales), scales.astype(int).min(-1) - 127 - 1


def exact_product(a, w):
    """a . w^T / 32 of two operands, after showing that FP32 sums of it are exact."""
    (va, ea), (vw, ew) = a, w
    terms = (np.abs(va) @ np.abs(vw).T) / np.exp2(ea[:, None] + ew[None, :])
    assert terms.max() < 2 ** 23, terms.max()
    return va @ vw.T / 32


def activation(g, u, act):
    z = g if act == SILU else 2 * np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)
    with np.errstate(over="ignore"):
        a = g / (1 + np.exp(-z)) * u
    return a, (4 + 2 * np.abs(z)) * 2.0 ** -22 * np.abs(a) + (1 + np.abs(g * u)) * 2.0 ** -126


def gate_and_up(bits, d_up, w_up):
    """g, u [T, I] of one expert, exactly."""
    both = exact_product(operand(*oracle.quantize_act(bits, d_up)), operand(*oracle.quantize_weights(w_up, d_up)))
    return both[:, : both.shape[1] // 2], both[:, both.shape[1] // 2 :]


def check_blocks(codes, scales, bits, d_up, w_up, d_down, act):
    """The stored rows [T, I / 2], [T, I / 32] of one expert's tokens `bits` [T, H]."""
    a, tol = activation(*gate_and_up(bits, d_up, w_up), act)
    n, I = a.shape
    lo, hi = oracle.f64_to_bf16(a - tol), oracle.f64_to_bf16(a + tol)
    free = (lo != hi).reshape(n, I // 32, 32)
    assert free.sum(-1).max() <= MOST, free.sum(-1).max()
    assert free.mean() < 2.0 ** -6, free.mean()
    nth = np.cumsum(free, -1) - 1  # which choice a free activation is
    matched = np.zeros((n, I // 32), bool)
    for choice in range(2 ** int(free.sum(-1).max())):
        up = (free & (choice >> np.where(free, nth, 0) & 1 == 1)).reshape(n, I)
        want_codes, want_scales = oracle.quantize_act(np.where(up, hi, lo), d_down)
        matched |= (scales == want_scales) & (codes.reshape(n, -1, 16) == want_codes.reshape(n, -1, 16)).all(-1)
    assert matched.all(), f"{(~matched).sum()} of {matched.size} blocks are no rounding of the activations"
