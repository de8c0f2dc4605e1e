"""The bounds for the MoE kernels tell their arithmetic from one that keeps
13 bits below the largest of eight products (the mistake is planted here, in
the oracle)."""

import numpy as np
import pytest

import moe_bounds as B
from block_scaled_precision_fp8_amd import synth
from oracle import formats as F
from oracle import layer as Y
from oracle import quant as Q
from oracle.gemm import dequant_act
from oracle.moe_mlp import silu


def dot(x, w, bits):
    """x (T, K) by w (N, K) with products in groups of eight neighbours, each
    cut below its group's largest times 2^-bits (None: exact)."""
    p = (x[:, None, :] * w[None]).reshape(len(x), len(w), -1, 8)
    if bits is not None:
        q = np.abs(p).max(3, keepdims=True)
        q = 2.0 ** (np.floor(np.log2(np.where(q == 0, 1.0, q))) - bits)
        p = np.trunc(p / q) * q
    return p.sum((2, 3))


@pytest.mark.parametrize("w4", [False, True])
@pytest.mark.parametrize("pair", [0, 6, 62, 126, 134, 190])
def test_cancelling_sums(pair, w4):
    x, w = B.cancelling(256, 128, pair, w4, 0)
    q, s = B.encode_weight(w, w4, 0)
    assert np.array_equal(B.weights64(q, s, 0, w4), w)
    assert np.array_equal(F.e4m3_decode(F.e4m3_encode(x)), x)
    g = dot(x[None], w[:1], None)[0, 0]
    assert g == 16.0 and dot(x[None], w[:1], 23)[0, 0] == 16.0
    if not w4:                              # MXFP4: the pair's group holds no small product
        assert dot(x[None], w[:1], 13)[0, 0] == 16.0 - 6 / 8


@pytest.mark.parametrize("fmt", [0, 1])
def test_codes_bound_tells_13_bits(fmt):
    """Codes of h from fp32 sums lie inside the bound, those of sums with 13
    bits and 50-fold outlier channels do not."""
    T, H, I = 24, 128, 128
    xb = synth.f32_to_bf16_bits(np.where(np.arange(H) % 40 == 7, 50.0, 1.0).astype(np.float32) *
                                np.random.default_rng(0).standard_normal((T, H), dtype=np.float32))
    xq, xs = Q.quant_act(xb, 128, fmt)
    w13, s13 = (a[None] for a in Q.quant_weight(synth.normal_bf16((2 * I, H), 0.05, "moe", "w", 0), 128, 128, fmt))
    ids = np.zeros((T, 1), np.int32)
    v, eps = B.gate_up(xq, xs, ids, w13, s13, fmt, False)
    x, w = F.e4m3_decode(xq), F.e4m3_decode(w13[0])
    scale = dequant_act(np.full_like(xq, 0x38), xs, 128, fmt)[:, :1] * \
        B.weights64(np.full_like(w13[0], 0x38), s13[0], fmt, False)[:, 0]

    def outside(bits):
        gu = dot(x, w, bits) * scale
        h = (silu(gu[:, :I]) * gu[:, I:]).astype(np.float32).astype(np.float64)
        q, s = Y.quant_rows(F.bf16_round(h).astype(np.float32), 128, fmt)
        return len(B.groups_outside(dequant_act(q, s, 128, fmt), v[:, 0], eps[:, 0], fmt))

    assert outside(None) == 0 and outside(24) == 0
    assert outside(13) > 0
