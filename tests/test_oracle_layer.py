"""Pins of the oracle's norm, router and MoE layer: torch's own functions,
closed forms and brute force (CPU)."""

import itertools

import numpy as np
import pytest

from oracle import formats as F
from oracle import gemm as G
from oracle import layer as Y
from oracle import moe_mlp as MM
from oracle import quant as Q


def bits(a):
    u = np.ascontiguousarray(a, np.float32).view(np.uint32).astype(np.uint64)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def test_norm_against_torch_and_closed_forms():
    import torch
    g = np.random.default_rng(0)
    x, r, w = (bits(g.standard_normal(s)) for s in ((5, 96), (5, 96), (96,)))
    h, y = Y.add_rmsnorm(x, w, 1e-5, r)
    xt, rt = (torch.from_numpy(F.bf16_decode(a)).to(torch.bfloat16) for a in (x, r))
    ht = xt + rt
    assert np.array_equal(h, ht.double().numpy())
    eps = float(np.float32(1e-5))
    ref = torch.nn.functional.rms_norm(ht.double(), (96,), torch.from_numpy(F.bf16_decode(w)), eps)
    assert np.allclose(y, ref.numpy(), rtol=2.0 ** -24, atol=0)
    one = bits(np.full((1, 32), 3.0))                       # constant rows: +-1 times the weight
    _, y = Y.add_rmsnorm(one, bits(np.arange(32.0)), 1e-30)
    assert np.array_equal(y[0], np.arange(32.0, dtype=np.float32))


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("group", [32, 128])
def test_quant_rows_is_the_pinned_quantizer_on_bf16_rows(group, fmt):
    x = bits(np.random.default_rng(1).standard_normal((4, 304)) * 7)
    q, s = Y.quant_rows(F.bf16_decode(x).astype(np.float32), group, fmt)
    rq, rs = Q.quant_act(x, group, fmt)
    assert np.array_equal(q, rq) and np.array_equal(s, rs)
    q, s = Y.quant_rows(np.array([[0.5, -700.0, 3.0, 0.0]], np.float32), 128, 0, 1.0)
    assert np.array_equal(F.e4m3_decode(q)[0], [0.5, -448.0, 3.0, 0.0]) and s[0, 0] == 1.0


@pytest.mark.parametrize("sigmoid", [False, True])
def test_route_against_torch_and_brute_force(sigmoid):
    import torch
    g = np.random.default_rng(2)
    l = g.standard_normal((20, 12))
    s = torch.sigmoid(torch.from_numpy(l)) if sigmoid else torch.softmax(torch.from_numpy(l), 1)
    ids, w = Y.route_topk(l, 3, sigmoid=sigmoid, renorm=False)
    v, i = torch.topk(s, 3, dim=1)
    assert np.array_equal(ids, i.numpy()) and np.allclose(w, v.numpy(), rtol=1e-14)
    _, w = Y.route_topk(l, 3, sigmoid=sigmoid, scale=2.0)
    assert np.allclose(w, 2 * (v / v.sum(1, keepdim=True)).numpy(), rtol=1e-14)
    # groups: the best of all pairs of groups by their top-two sums
    b = 0.1 * g.standard_normal(12)
    key = s.numpy() + b
    ids, _ = Y.route_topk(l, 4, b, sigmoid, n_group=4, topk_group=2)
    for t in range(20):
        two = np.sort(key[t].reshape(4, 3), 1)[:, 1:].sum(1)
        best = max(itertools.combinations(range(4), 2), key=lambda c: two[list(c)].sum())
        ok = [e for e in range(12) if e // 3 in best]
        assert list(ids[t]) == sorted(ok, key=lambda e: -key[t, e])[:4]


def test_route_masks():
    ids, w = Y.route_topk(np.array([[-np.inf, np.nan, 1.0, 1.0], [-np.inf] * 4]), 3)
    assert np.array_equal(ids, [[2, 3, -1], [-1, -1, -1]])
    assert np.array_equal(w, [[0.5, 0.5, 0], [0, 0, 0]])
    ids, w = Y.route_topk(np.array([[0.0, np.inf, 5.0, np.inf]]), 3)
    assert np.array_equal(ids, [[1, 3, 2]]) and np.array_equal(w, [[0.5, 0.5, 0]])


@pytest.mark.parametrize("fmt", [0, 1])
def test_moe_layer_against_the_grouped_oracle(fmt):
    """Slot by slot: the pinned gate/up, quantizer and GEMM oracles."""
    g = np.random.default_rng(3)
    T, k, H, I, E = 4, 2, 144, 128, 3
    xq, xs = Q.quant_act(bits(g.standard_normal((T, H))), 128, fmt)
    w13 = [Q.quant_weight(bits(g.standard_normal((2 * I, H)) * 0.1), 128, 128, fmt) for _ in range(E)]
    w2 = [Q.quant_weight(bits(g.standard_normal((H, I)) * 0.1), 128, 128, fmt) for _ in range(E)]
    a = [np.stack([x[i] for x in w]) for w in (w13, w2) for i in (0, 1)]
    ids = np.array([[0, 2], [1, 1], [-1, 0], [E, -7]], np.int32)
    wt = g.random((T, k)).astype(np.float32)
    add = bits(g.standard_normal((T, H)))
    y = Y.moe_layer(xq, xs, ids, wt, *a, fmt, False, add)
    for t in range(T):
        ref = F.bf16_decode(add[t]).copy()
        for j in range(k):
            e = ids[t, j]
            if 0 <= e < E:
                h = MM.gate_up_silu(xq[t:t + 1], xs[t:t + 1], a[0][e:e + 1], a[1][e:e + 1], [0, 1], fmt)
                hq, hs = Q.quant_act(bits(F.bf16_round(h)), 128, fmt)
                ref += wt[t, j] * G.block_gemm(hq, hs, a[2][e], a[3][e], fmt=fmt)[0]
        assert np.allclose(y[t], ref, rtol=1e-12, atol=1e-12)
