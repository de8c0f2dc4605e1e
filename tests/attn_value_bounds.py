"""How far paged_attn may be from its 64-bit values where every weight keeps
its precision whatever the others are, by counting roundings (half a step
each: bf16 2^-8, fp32 2^-24 of the value)."""

import numpy as np

BF16, FP32 = 2.0 ** -8, 2.0 ** -24


def attention(y, spread, reach, keys, D, vmax):
    """Per element of y; spread = sum p |v| / sum p of that element, so that
    an element to which the heaviest key adds nothing is held to the others'
    contributions.

    * Scores: D products summed in fp32, the key's scale, the product with
      scale log2(e) and the difference from the reference exponent: at most
      (D + 8) 2^-24 of scale sum |q k| (all intermediate values are below
      that sum, the reference exponent below it and the values' log2 scale,
      for which 64 2^-24 stand), in e^s a relative error of as much; 2^-21 for
      2^x itself.  It reaches y through the weights and through their sum:
      twice, times spread.
    * Weights: times the value's scale (2^-24) and rounded to the sum of two
      bf16 numbers (2^-16), each by itself.
    * Sums in fp32 over the keys: 2^-24 a key, and the joining of partial
      results (32 steps).
    * What is below 2^-126 is lost: a weight beside a largest one of at least 1
      (times its value, at most 448 of its scale's size, `vmax` at most), or
      its product with the scale (times a code of at most 448).
    * y rounded once to bf16 (bf16's smallest step 2^-133 aside).
    """
    e = (D + 8) * FP32 * reach + 64 * FP32 + 2.0 ** -21
    rel = 2.0 * e + BF16 ** 2 + FP32 + 2.0 * (keys + 64) * FP32
    inner = spread * rel[..., None] + (keys * 2.0 ** -126 * (vmax + 448.0))[..., None]
    return BF16 * np.abs(y) + (1.0 + BF16) * inner + 2.0 ** -133
