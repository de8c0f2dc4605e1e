"""The operators between a layer's linears (test infrastructure): residual
RMS norm with FP8 output, a router's top-k, and a whole MoE layer over
unsorted (token, expert) slots.  Everything in float64, from the formulas.

Readings:
 25. h = bf16(x + residual); y = h * weight / sqrt(mean(h^2) + eps), rounded
     once to fp32 and quantized without a bf16 rounding in between, by the
     1 x 128 (or 1 x 32) activation quantizer or one static scale;
 26. router: scores softmax(l) or sigmoid(l); keys l (no bias, no groups) or
     s + bias; a group's score is the sum of its two largest keys; ties go
     to the lower index; NaN and -inf logits or keys are never chosen;
     weights s[ids] (/ their sum) * scale, without the bias;
 27. MoE layer: the slots' gate/up, SiLU product, bf16 rounding and
     requantization are readings 19-21; the down products are weighted and
     summed unrounded, with the addend, and rounded once to bf16.
"""

import numpy as np

from .formats import bf16_decode, bf16_round, e4m3_encode
from .gemm import dequant_act, dequant_weight
from .moe_mlp import silu
from .mxfp4 import dequant_mxfp4
from .quant import SCALE_FLOAT, _scale_and_codes


def bf16_bits(v):
    """bf16-representable float64 values -> bit patterns."""
    return (np.asarray(v, dtype=np.float32).view(np.uint32) >> 16).astype(np.uint16)


def add_rmsnorm(x_bits, w_bits, eps, res_bits=None):
    """(h float64 (M, K), y float32 (M, K)); eps as the fp32 it is passed as."""
    h = bf16_decode(x_bits)
    if res_bits is not None:
        h = bf16_round((h.astype(np.float32) + bf16_decode(res_bits).astype(np.float32))
                       .astype(np.float64))
    rs = 1.0 / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + float(np.float32(eps)))
    return h, (h * bf16_decode(w_bits) * rs).astype(np.float32)


def quant_rows(y, group_k=128, fmt=SCALE_FLOAT, static=None):
    """E4M3 codes and stored scales of fp32 rows (quant.quant_act's rules)."""
    M, K = y.shape
    G = -(-K // group_k)
    if static is not None:
        s = np.float32(static) if fmt == SCALE_FLOAT else np.float32(2.0 ** (int(static) - 127))
        q = np.clip((y / s).astype(np.float64), -448, 448)
        kind = np.float32 if fmt == SCALE_FLOAT else np.uint8
        return e4m3_encode(q), np.full((M, G), static, kind)
    pad = G * group_k - K
    yp = np.pad(y, ((0, 0), (0, pad))).reshape(M, G, group_k)
    vp = np.pad(np.ones((M, K), bool), ((0, 0), (0, pad))).reshape(M, G, group_k)
    q, s = _scale_and_codes(yp, vp, fmt)
    return q.reshape(M, -1)[:, :K].copy(), s


def route_topk(logits, k, bias=None, sigmoid=False, renorm=True, scale=1.0, n_group=1,
               topk_group=1):
    """ids int32 (T, k), weights float64 (T, k); plain loops over tokens."""
    logits = np.asarray(logits, dtype=np.float64)
    T, E = logits.shape
    ids = np.full((T, k), -1, np.int32)
    wts = np.zeros((T, k))
    for t in range(T):
        l = logits[t]
        ok = ~(np.isnan(l) | (l == -np.inf))
        s = np.zeros(E)
        if sigmoid:
            with np.errstate(over="ignore"):
                s[ok] = 1.0 / (1.0 + np.exp(-l[ok]))
        elif ok.any():
            m = l[ok].max()
            s[ok] = np.where(l[ok] == m, 1.0, np.exp(l[ok] - m if np.isfinite(m) else -np.inf))
            s /= s.sum()
        key = l if bias is None and n_group == 1 else s + (0.0 if bias is None else bias)
        ok = ok & ~np.isnan(key) & (key > -np.inf)
        if n_group > 1:
            gs = E // n_group
            score = []
            for g in range(n_group):
                mem = sorted((key[e] for e in range(g * gs, (g + 1) * gs) if ok[e]), reverse=True)
                score.append(sum(mem[:2]) if mem else -np.inf)
            best = sorted(range(n_group), key=lambda g: (-score[g], g))[:topk_group]
            ok = ok & np.isin(np.arange(E) // gs, best)
        pick = sorted((e for e in range(E) if ok[e]), key=lambda e: (-key[e], e))[:k]
        ids[t, :len(pick)] = pick
        w = s[pick]
        if renorm and len(pick):
            w = w / w.sum() if w.sum() > 0 else 0.0 * w
        wts[t, :len(pick)] = w * scale
    return ids, wts


def moe_layer(xq, x_scale, ids, weights, w13, s13, w2, s2, fmt=SCALE_FLOAT, w4=False,
              addend_bits=None):
    """y (T, H) float64, unrounded."""
    T, H = xq.shape
    E = w13.shape[0]
    x = dequant_act(xq, x_scale, 128, fmt)
    y = np.zeros((T, H)) if addend_bits is None else bf16_decode(addend_bits).copy()
    dense = dequant_mxfp4 if w4 else (lambda w, s: dequant_weight(w, s, 128, 128, fmt))
    for e in range(E):
        t, j = np.nonzero(np.asarray(ids) == e)
        if not len(t):
            continue
        gu = x[t] @ dense(w13[e], s13[e]).T
        I = gu.shape[1] // 2
        h = bf16_round(silu(gu[:, :I]) * gu[:, I:]).astype(np.float32)
        hq, hs = quant_rows(h, 128, fmt)
        d = dequant_act(hq, hs, 128, fmt) @ dense(w2[e], s2[e]).T
        np.add.at(y, t, d * np.asarray(weights, dtype=np.float64)[t, j][:, None])
    return y
