"""How far the attention kernel's and the rotation's results may be from
their 64-bit values, by counting roundings (half a step each: bf16 2^-8, fp16
2^-11, fp32 2^-24 of the value)."""

import numpy as np

BF16, FP16, FP32 = 2.0 ** -8, 2.0 ** -11, 2.0 ** -24


def attention(y, spread, reach, keys, D, fp8, vmax):
    """Per element of y.

    * Scores: D products summed in fp32, the key's scale, the product with
      scale log2(e) and the difference from the reference exponent: at most
      (D + 8) 2^-24 of scale sum |q k| (all intermediate values are below
      that sum, the reference exponent below it and the values' log2 scale,
      for which 64 2^-24 stand), in e^s a relative error of as much; 2^-21 for
      2^x itself.  It reaches y through the weights and through their sum:
      twice, times sum p |v| / sum p.
    * Weights: times the value's scale, and rounded to fp16 (E4M3 caches, 2^-11
      and at most 2^-24 of the largest weight for each key below fp16's normal
      range) or to the sum of two bf16 numbers (2^-16).
    * Sums in fp32 over the keys: 2^-24 a key, and the joining of partial
      results (32 steps).
    * y rounded once to bf16 (bf16's smallest step 2^-133 aside).
    """
    e = (D + 8) * FP32 * reach + 64 * FP32 + 2.0 ** -21
    weight = FP16 + FP32 if fp8 else BF16 ** 2
    rel = 2.0 * e + weight + 2.0 * (keys + 64) * FP32
    low = keys * 2.0 ** -24 * vmax if fp8 else 0.0 * keys
    inner = spread * rel[..., None] + low[..., None]
    return BF16 * np.abs(y) + (1.0 + BF16) * inner + 2.0 ** -133


def rotated(a, b, mscale):
    """Per value of a rotated pair (a, b), before it is rounded to its type:
    sine and cosine within four fp32 roundings of half of their largest value (the
    angle's half turn in fp32, the function, the scale's product), two products
    and a sum."""
    return (np.abs(a) + np.abs(b)) * abs(mscale) * 8.0 * FP32
