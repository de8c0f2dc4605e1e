"""The bound that paged_attn is held to sees weights that lose their
precision beside a heavier one: one row's arithmetic redone in numpy, with
weights as the sum of two bf16 numbers and, planted, as one fp16 number."""

import numpy as np
import pytest

import attn_value_bounds as bounds
from oracle import formats as F


def row(weights, gap, scale, keys, D=64, seed=0):
    """(y, exact y, bound) of one row: key 0 stands `gap` (log2) above the
    others and its value is 0, with the scale 1 that the codec gives it; the
    others' scales are about `scale`."""
    rng = np.random.default_rng(seed)
    s = rng.standard_normal(keys)
    s[0] = s[1:].max() + gap
    vs = scale * (0.3 + rng.random(keys))
    codes = F.e4m3_decode(F.e4m3_encode(rng.standard_normal((keys, D)) * 120.0)).astype(np.float64)
    vs[0], codes[0] = 1.0, 0.0
    p = np.exp2(s - s.max())
    exact = (p * vs) @ codes / p.sum()
    spread = (p * vs) @ np.abs(codes) / p.sum()
    w = (p * vs).astype(np.float32)
    y = weights(w) @ codes / p.sum()
    room = bounds.attention(exact[None], spread[None], np.zeros(1), np.full(1, float(keys)), D, 448.0)[0]
    return y, exact, room


def two_bf16(w):
    hi = F.bf16_round(w).astype(np.float32)
    return hi.astype(np.float64) + F.bf16_round(w - hi)


def one_fp16(w):
    """Times the power of two that takes the largest to 1, rounded to fp16."""
    top = w.max()
    return (w / top).astype(np.float16).astype(np.float64) * float(top)


CASES = [(10.0, 1.0, 300), (10.0, 0.1, 300), (8.0, 0.01, 300), (12.0, 1.0 / 448, 4096), (13.0, 1.0 / 448, 131072)]


@pytest.mark.parametrize("gap,size,keys", CASES)
def test_two_bf16_numbers_keep_every_weight(gap, size, keys):
    y, exact, room = row(two_bf16, gap, size / 448, keys)
    assert np.all(np.abs(y - exact) <= room)


# at 131072 keys the fp32 sums' own roundings are allowed 2^-6, as much as such weights lose there
@pytest.mark.parametrize("gap,size,keys", CASES[:-1])
def test_planted_fp16_weights_are_seen(gap, size, keys):
    y, exact, room = row(one_fp16, gap, size / 448, keys)
    assert np.any(np.abs(y - exact) > room)
