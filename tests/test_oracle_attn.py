"""Pins of the rotary, cache and attention oracle: closed forms and plain
loops (no GPU)."""

import math

import numpy as np
import pytest

from oracle import attn as A


def test_inv_freq_closed_forms():
    f = A.inv_freq(8, 10000.0)
    assert np.array_equal(f, np.array([1.0, 0.1, 0.01, 0.001], np.float32))
    assert np.array_equal(A.inv_freq(8, 10000.0, 1, factor=4.0), (np.array([1, .1, .01, .001]) / 4).astype(np.float32))
    # turns in 2 pi 100 positions: 100, 10, 1, 0.1; kept from 10 on, divided up to 1, in between by share
    g = A.inv_freq(8, 10000.0, 2, factor=4.0, low=1.0, high=10.0, orig_len=2 * math.pi * 100).astype(np.float64)
    assert np.allclose(g, [1.0, 0.1, 0.01 / 4, 0.001 / 4], rtol=1e-6)
    g = A.inv_freq(8, 10000.0, 2, factor=4.0, low=1.0, high=19.0, orig_len=2 * math.pi * 100).astype(np.float64)
    assert np.allclose(g[1], 0.1 * 0.5 + 0.1 / 4 * 0.5, rtol=1e-6)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation(interleaved):
    rng = np.random.default_rng(0)
    x = rng.standard_normal((3, 2, 12))
    freq = np.array([math.pi / 2, 0.0, math.pi], np.float32)        # a quarter turn, none, half a turn
    y = A.rotate(x, [0, 1, 2], freq, interleaved)
    ia, ib = ([0, 2, 4], [1, 3, 5]) if interleaved else ([0, 1, 2], [3, 4, 5])
    assert np.array_equal(y[0], x[0]) and np.array_equal(y[..., 6:], x[..., 6:])
    assert np.allclose(y[1][:, ia[0]], -x[1][:, ib[0]], atol=1e-6)
    assert np.allclose(y[1][:, ib[0]], x[1][:, ia[0]], atol=1e-6)
    assert np.array_equal(y[:, :, ia[1]], x[:, :, ia[1]])
    assert np.allclose(y[1][:, ia[2]], -x[1][:, ia[2]], atol=1e-6)
    assert np.allclose(y[2][:, ia[2]], x[2][:, ia[2]], atol=1e-6)
    # lengths stay, scaled by mscale, and scores depend on the distance alone
    z = A.rotate(x, [5, 6, 7], np.array([0.3, 0.7, 0.01], np.float32), interleaved, 2.0)
    assert np.allclose((z[..., :6] ** 2).sum(-1), 4 * (x[..., :6] ** 2).sum(-1))
    q, k = rng.standard_normal((2, 1, 1, 6))
    f = np.array([0.3, 0.7, 0.01], np.float32)
    dots = [(A.rotate(q, [p], f, interleaved) * A.rotate(k, [p - 3], f, interleaved)).sum() for p in (3, 10, 99)]
    assert np.allclose(dots, dots[0])


def test_attention_against_loops():
    rng = np.random.default_rng(1)
    P, Hkv, ps, D, Hq = 9, 2, 4, 6, 4
    k, v = rng.standard_normal((2, P, Hkv, ps, D))
    table = np.array([[3, 5, 1], [0, 7, 2]])
    ptable, prefix, lens, start, window = np.array([8, 6]), 7, [9, 3], [0, 2, 5], 6
    q = rng.standard_normal((6, Hq, D))
    y, spread, reach, keys = A.attention(q, k, v, lens, table, 0.5, start, ptable, prefix, window)
    assert np.isnan(y[5]).all()
    for b in range(2):
        n = start[b + 1] - start[b]
        for i in range(n):
            pos = prefix + lens[b] - n + i
            for h in range(Hq):
                num, den, low = np.zeros(D), 0.0, 0
                for j in range(max(0, pos - window + 1), pos + 1):
                    page, at = (ptable[j // ps], j % ps) if j < prefix else \
                        (table[b][(j - prefix) // ps], (j - prefix) % ps)
                    e = math.exp(0.5 * float(q[start[b] + i, h] @ k[page, h // 2, at]))
                    num, den, low = num + e * v[page, h // 2, at], den + e, low + 1
                assert np.allclose(y[start[b] + i, h], num / den) and keys[start[b] + i, h] == low
    assert (spread[:5] >= np.abs(y[:5]) - 1e-12).all() and (reach[:5] > 0).all()


def test_attention_of_nothing():
    k = np.ones((2, 1, 4, 3))
    q = np.ones((2, 1, 3))
    y = A.attention(q, k, k, [0, 3], np.array([[0], [-1]]), 1.0)[0]
    assert np.array_equal(y, np.zeros((2, 1, 3)))                     # no key; no page
    y = A.attention(q, k, k, [1], np.array([[0]]), 1.0, q_start=[0, 2])[0]
    assert np.array_equal(y[0], np.zeros((1, 3))) and np.allclose(y[1], 1.0)


def test_cache_values():
    codes = np.array([[[[0x38, 0xB8]]]], np.uint8)                    # 1, -1
    assert np.array_equal(A.cache_values(codes, np.float32([[[0.5]]]), 0)[0, 0, 0], [0.5, -0.5])
    assert np.array_equal(A.cache_values(codes, np.uint8([[[129]]]), 1)[0, 0, 0], [4.0, -4.0])
