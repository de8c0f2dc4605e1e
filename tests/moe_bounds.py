"""Bounds of the MoE layer's kernels from their own arithmetic (host only).

Every E4M3 and E2M1 value is a bf16 value and the product of two is exact in
fp32.  A K block's 128 products are added by four bf16 MFMAs, which keep 24
bits below the largest addend: at most one unit of 2^-23 of the running sum
of |a b| for each of the 128 additions, 256 2^-24 in all.  A block's sum is
multiplied by its scales (two roundings) and added to those of the other KB
blocks (one each), and at most eight waves' pieces are joined: a row's sum
errs by at most (266 + KB) 2^-24 of its sum |a b|.  The down products are
then weighted and added over k choices, eight waves and the addend."""

import numpy as np

from oracle import formats as F
from oracle import layer as Y
from oracle import mxfp4 as X
from oracle.gemm import dequant_act, dequant_weight
from oracle.moe_mlp import silu

U = 2.0 ** -24


def sum_error(K):
    """Of a K-long product, in units of sum |a b|."""
    return (266 + -(-K // 128)) * U


def weights64(q, s, fmt, w4):
    return X.dequant_mxfp4(q, s) if w4 else dequant_weight(q, s, 128, 128, fmt)


def gate_up(xq, xs, ids, w13, s13, fmt, w4):
    """float64 silu(g) u before any rounding, and the bound on the kernel's
    fp32 value of it, (T, k, I)."""
    T, k = ids.shape
    I = w13.shape[1] // 2
    v, eps = np.zeros((T, k, I)), np.zeros((T, k, I))
    x = dequant_act(xq, xs, 128, fmt)
    gam = sum_error(x.shape[1])
    for e in range(w13.shape[0]):
        t, j = np.nonzero(ids == e)
        if not len(t):
            continue
        w = weights64(w13[e], s13[e], fmt, w4)
        gu, su = x[t] @ w.T, np.abs(x[t]) @ np.abs(w).T
        g, u, sg, su = gu[:, :I], gu[:, I:], su[:, :I], su[:, I:]
        sig = np.where(g == 0, 0.5, silu(g) / np.where(g == 0, 1.0, g))
        v[t, j] = silu(g) * u
        # the sums' errors through silu(g) u, whose slopes are sig (1 + g (1
        # - sig)) u and silu(g) (|silu''| <= 1/2); exponential, addition,
        # division and product of fp32: 2^-22 + 3 2^-24
        eps[t, j] = gam * (np.abs(sig * (1 + g * (1 - sig)) * u) * sg + np.abs(silu(g)) * su) + \
            gam * gam * sg * (su + 0.5 * sg * (np.abs(u) + gam * su)) + 7 * U * np.abs(v[t, j])
    return v, eps


def _quant(h, s):
    return F.e4m3_decode(F.e4m3_encode(np.clip((h.astype(np.float32) / np.float32(s)).astype(np.float64),
                                               -448, 448))) * float(s)


def groups_outside(h, v, eps, fmt):
    """Groups (n, 128) of dequantized h that no fp32 values within eps of v
    round to: bf16, then E4M3 by a scale that such values have (both
    roundings are monotone, so every element lies between those of v - eps
    and v + eps)."""
    lo, hi = F.bf16_round(v - eps), F.bf16_round(v + eps)
    bad = []
    for i in range(len(h)):
        a = Y.bf16_bits(F.bf16_round(np.maximum(np.abs(v[i]) - eps[i], 0)).max(keepdims=True))[0]
        b = Y.bf16_bits(F.bf16_round(np.abs(v[i]) + eps[i]).max(keepdims=True))[0]
        for bits in range(int(a), int(b) + 1):
            amax = F.bf16_decode(np.array([bits], np.uint16)).astype(np.float32)
            s = Y.quant_rows(amax[None], 128, fmt)[1][0, 0]
            s = np.float32(2.0 ** (int(s) - 127)) if fmt else s
            tiny = 1e-9 * (np.abs(h[i]) + float(s))
            if np.all(h[i] >= _quant(lo[i], s) - tiny) and np.all(h[i] <= _quant(hi[i], s) + tiny):
                break
        else:
            bad.append(i)
    return bad


def layer_error(h, ids, w, w2, s2, fmt, w4, add=None):
    """(float64 layer of the dequantized h, the bound on the kernel's bf16 y)."""
    T, k, I = h.shape
    ref = np.zeros((T, w2.shape[1])) if add is None else add.copy()
    mag = np.abs(ref)
    for e in range(w2.shape[0]):
        t, j = np.nonzero(ids == e)
        if len(t):
            d = weights64(w2[e], s2[e], fmt, w4)
            wt = w[t, j].astype(np.float64)[:, None]
            np.add.at(ref, t, wt * (h[t, j] @ d.T))
            np.add.at(mag, t, np.abs(wt) * (np.abs(h[t, j]) @ np.abs(d).T))
    return ref, 2.0 ** -8 * np.abs(ref) + (sum_error(I) + (k + 9) * U) * (1 + 2.0 ** -8) * mag + 2.0 ** -134


# ---------------------------------------------- sums that cancel, in closed form

def cancelling(H, I, pair, w4, fmt):
    """One token and one expert whose sums are +-448^2 (MXFP4: 448 384) and
    128 products of 1/8: 16 exactly, with any 21 bits kept below the
    largest.  Gate: g = 16 for every column, from the pair at columns
    (pair, pair + 1) of the token; up: 2^-(j % 3); so h_j = 16 2^-(j % 3).
    Returns the token's codes and the gate/up weight's codes and scales."""
    small = [c for c in range(H) if c not in (pair, pair + 1) and not (w4 and c // 32 == pair // 32)]
    small = sorted(small, key=lambda c: (c // 128 != pair // 128, c))[:128]
    x, g, u = np.zeros(H), np.zeros(H), np.zeros((I, H))
    x[small] = 1.0
    x[[pair, pair + 1]] = 448.0
    g[small] = 0.125
    g[[pair, pair + 1]] = (384.0, -384.0) if w4 else (448.0, -448.0)
    u[np.arange(I), small[0]] = 2.0 ** -(np.arange(I) % 3)
    return x, np.concatenate([np.tile(g, (I, 1)), u])


def encode_weight(w, w4, fmt):
    """Codes and scales of a (N, K) weight that they hold exactly."""
    if not w4:
        one = np.full((-(-w.shape[0] // 128), -(-w.shape[1] // 128)), 127 if fmt else 1.0,
                      np.uint8 if fmt else np.float32)
        return F.e4m3_encode(w), one
    N, K = w.shape
    groups = w.reshape(N, K // 32, 32)
    amax = np.abs(groups).max(2)
    e = np.where(amax == 0, 0, np.floor(np.log2(np.where(amax == 0, 1, amax)))).astype(int) - 2
    v = groups / 2.0 ** e[:, :, None]
    table = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
    code = np.abs(np.abs(v)[..., None] - table).argmin(-1)
    assert np.array_equal(table[code], np.abs(v)), "not an MXFP4 value"
    code = (code + 8 * (v < 0)).astype(np.uint8).reshape(N, K)
    return (code[:, ::2] | code[:, 1::2] << 4).astype(np.uint8), (e + 127).astype(np.uint8)
