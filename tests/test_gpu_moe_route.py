"""moe_route_topk against the float64 oracle: ids exactly, weights within the
fp32 bound derived in `check`."""

import numpy as np
import pytest

from block_scaled_precision_fp8_amd import synth
from oracle import formats as F
from oracle import layer as Y

from gpu_util import to_dev, to_dev_bf16, say

pytestmark = pytest.mark.gpu


def run(logits, k, bf16=False, bias=None, ldl=None, **kw):
    import torch
    from block_scaled_precision_fp8_amd import lib as L
    T, E = logits.shape
    ldl = ldl or E
    full = np.full((T, ldl), 99.0, np.float32)
    full[:, :E] = logits
    l = to_dev_bf16(synth.f32_to_bf16_bits(full)) if bf16 else to_dev(full)
    ids = torch.full((T + 1, k), -77, dtype=torch.int32, device="cuda")
    w = torch.full((T + 1, k), -77.0, device="cuda")
    b = None if bias is None else to_dev(np.asarray(bias, np.float32))
    L.moe_route_topk(l[:, :E], ids[:T], w[:T], bias=b, **kw)
    torch.cuda.synchronize()
    assert (ids[T:] == -77).all() and (w[T:] == -77.0).all(), "wrote past the last token"
    return ids[:T].cpu().numpy(), w[:T].cpu().numpy()


def check(logits, k, bf16=False, bias=None, ldl=None, score=0, renorm=True, scale=1.0, n_group=1,
          topk_group=1):
    logits = np.asarray(logits, np.float32)
    if bf16:
        with np.errstate(invalid="ignore"):
            bits = (logits.view(np.uint32) >> 16).astype(np.uint16)
        logits = (bits.astype(np.uint32) << 16).view(np.float32)
    ids, w = run(logits, k, bf16, bias, ldl, score=score, renorm=renorm, scale=scale,
                 n_group=n_group, topk_group=topk_group)
    b64 = None if bias is None else np.asarray(bias, np.float32).astype(np.float64)
    rid, rw = Y.route_topk(logits, k, b64, score == 1, renorm, float(np.float32(scale)), n_group,
                           topk_group)
    assert np.array_equal(ids, rid), np.argwhere(ids != rid)[:5]
    # a score is e^d (softmax, d = l - top) or 1 / (1 + e^-l) with fp32
    # exponentials at worst: d rounds by |d| 2^-24 (|d| <= 104 before e^d
    # leaves fp32), expf errs by two units, the sums and divisions by one
    # each; twice that for the quotient of two such numbers, and an absolute
    # 2^-126 where fp32 runs out
    tol = 2 * (104 + 2 + 4) * 2.0 ** -24
    assert np.all(np.abs(w - rw) <= tol * np.abs(rw) + abs(scale) * 2.0 ** -126), \
        np.max(np.abs(w - rw))


def logits(T, E, seed=0, sigma=2.0):
    return (sigma * np.random.default_rng(seed).standard_normal((T, E))).astype(np.float32)


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 256, 8), (3, 8, 2), (5, 64, 6), (7, 60, 4),
                                   (9, 65, 64), (33, 128, 8), (130, 160, 6), (2, 1024, 16),
                                   (4, 513, 5), (1, 2, 2), (6, 300, 1)])
def test_route_plain(T, E, k, bf16, score):
    say(f"route T={T} E={E} k={k} bf16={bf16} score={score}")
    l = logits(T, E, T + E)
    check(l, k, bf16, score=score)
    check(l, k, bf16, score=score, renorm=False, scale=2.5, ldl=E + 3)


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("T,E,k,ng,kg", [(1, 256, 8, 8, 4), (33, 256, 8, 8, 4), (5, 256, 8, 1, 1),
                                         (6, 160, 6, 8, 3), (4, 64, 64, 64, 5), (7, 60, 4, 3, 2),
                                         (3, 1024, 8, 32, 4), (9, 12, 12, 2, 1), (8, 70, 3, 7, 7)])
def test_route_bias_and_groups(T, E, k, ng, kg, score):
    say(f"route groups T={T} E={E} k={k} groups={ng}/{kg} score={score}")
    l = logits(T, E, T * E)
    b = 0.2 * np.random.default_rng(E).standard_normal(E)
    check(l, k, bias=b, score=score, n_group=ng, topk_group=kg)
    check(l, k, bias=None, score=score, n_group=ng, topk_group=kg, renorm=False)
    check(l, k, True, bias=b, score=score, n_group=ng, topk_group=kg, scale=-1.5)


@pytest.mark.parametrize("kw", [dict(), dict(bias=True), dict(bias=True, n_group=4, topk_group=2),
                                dict(n_group=4, topk_group=1)])
@pytest.mark.parametrize("score", [0, 1])
def test_route_ties_masks_and_limits(score, kw):
    """Equal logits (the lowest ids win, also over signed zeros), rows and
    groups masked off, NaN, infinities, the lowest finite value, a bias that
    masks."""
    E, k = 96, 6
    kw = dict(kw)
    g = np.random.default_rng(1)
    b = None
    if kw.pop("bias", False):
        b = np.zeros(E)
        b[10:20] = 0.25
        b[40] = -np.inf
        b[41] = np.nan
        b[42] = np.inf
    lo = np.finfo(np.float32).min
    rows = [np.zeros(E), np.where(np.arange(E) % 2 == 0, -0.0, 0.0), np.full(E, -np.inf),
            np.full(E, lo), np.full(E, np.nan), np.where(np.arange(E) < 93, -np.inf, 1.0),
            np.where(np.arange(E) % 3 == 0, lo, -np.inf), np.round(g.standard_normal(E)),
            np.where(np.arange(E) == 50, np.inf, g.standard_normal(E)),
            np.where(np.arange(E) % 40 == 7, np.inf, -3.0),
            np.where(g.random(E) < 0.3, np.nan, g.standard_normal(E)),
            np.where(np.arange(E) < 48, -np.inf, g.standard_normal(E)),
            g.standard_normal(E) * 60.0, np.full(E, -200.0), np.full(E, 60.0) + np.arange(E) % 2]
    say(f"route ties score={score} {kw}")
    check(np.array(rows), k, score=score, bias=b, **kw)
    check(np.array(rows), k, score=score, bias=b, renorm=False, **kw)


def test_route_large_and_close():
    """A prompt's worth of tokens with keys of bf16 logits (many exact ties)
    and with fp32 logits one unit apart under a bias."""
    say("route large")
    T, E = 1500, 256
    l = logits(T, E, 5)
    check(l, 8, True, bias=np.zeros(E), score=1, n_group=8, topk_group=4)
    near = np.float32(1.0) + np.random.default_rng(2).integers(-3, 4, (64, E)) * np.float32(2 ** -22)
    check(near, 8, score=1, bias=np.full(E, 0.125))


def test_route_streams_and_graph():
    import torch
    from block_scaled_precision_fp8_amd import lib as L
    T, E, k = 12, 256, 8
    l = to_dev(logits(T, E))
    ids = torch.empty((T, k), dtype=torch.int32, device="cuda")
    w = torch.empty((T, k), device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        L.moe_route_topk(l, ids, w, score=L.SCORE_SIGMOID, n_group=8, topk_group=4)
    for seed in range(1, 4):
        h = logits(T, E, seed)
        l.copy_(to_dev(h))
        g.replay()
        torch.cuda.synchronize()
        rid, rw = Y.route_topk(h, k, None, True, True, 1.0, 8, 4)
        assert np.array_equal(ids.cpu().numpy(), rid)
        assert np.allclose(w.cpu().numpy(), rw, rtol=2 * 110 * 2.0 ** -24, atol=0)


def test_route_more_tokens_than_one_grid_dimension():
    import torch
    from block_scaled_precision_fp8_amd import lib as L
    T, E, k = (4 << 20) + 777, 4, 2
    say(f"route T={T}")
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    l = torch.randn((T, E), generator=g, device="cuda")
    ids = torch.full((T + 1, k), -77, dtype=torch.int32, device="cuda")
    w = torch.full((T + 1, k), -77.0, device="cuda")
    L.moe_route_topk(l, ids[:T], w[:T])
    torch.cuda.synchronize()
    assert (ids[T] == -77).all() and (w[T] == -77.0).all()
    best = torch.topk(l, k, dim=1)                # distinct fp32 draws: no ties to order
    for lo in range(0, T, 1 << 20):
        v = torch.gather(l[lo:lo + (1 << 20)], 1, ids[lo:min(lo + (1 << 20), T)].long())
        assert torch.equal(v, best.values[lo:lo + (1 << 20)])
    rows = [0, (4 << 20) - 1, 4 << 20, T - 1]
    rid, rw = Y.route_topk(l[rows].cpu().numpy(), k)
    assert np.array_equal(ids[rows].cpu().numpy(), rid)
    assert np.allclose(w[rows].cpu().numpy(), rw, rtol=2 * 110 * 2.0 ** -24, atol=0)
