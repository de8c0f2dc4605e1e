"""moe_route_topk's weights within the rounding of their own type: scores,
sums and quotients are held in 64 bits, so a weight is off by half an fp32
step, 2^-24 of it (2^-149 below the smallest normal number), and a 2^-20th
of that for everything in 64 bits.

Only where softmax scores are not divided by their own sum and the logits
are the keys are the denominators sums of fp32 exponentials e^d, d = l -
top: d is rounded (|d| 2^-24 of the term) and the exponential errs by two
units (4 2^-24 of it); the terms are added in 64 bits."""

import numpy as np
import pytest

from oracle import layer as Y

from gpu_util import say
from test_gpu_moe_route import logits, run

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def check(l, k, bias=None, score=0, renorm=True, scale=1.0, n_group=1, topk_group=1):
    l = np.asarray(l, np.float32)
    ids, w = run(l, k, False, bias, None, score=score, renorm=renorm, scale=scale, n_group=n_group,
                 topk_group=topk_group)
    b = None if bias is None else np.asarray(bias, np.float32).astype(np.float64)
    rid, rw = Y.route_topk(l, k, b, score == 1, renorm, float(np.float32(scale)), n_group, topk_group)
    assert np.array_equal(ids, rid)
    tol = np.full(len(l), U)
    if score == 0 and not renorm and bias is None and n_group == 1:
        d = l.astype(np.float64)
        ok = d > -np.inf
        d = np.where(ok, d - np.where(ok, d, -np.inf).max(1, keepdims=True, initial=-1e30), 0.0)
        p = np.where(ok, np.exp(d), 0.0)
        tol = tol + U * (p * (np.abs(d) + 4)).sum(1) / np.maximum(p.sum(1), 1e-300)
    off = np.abs(w - rw)
    bound = tol[:, None] * (1 + 2.0 ** -20) * np.abs(rw) + 2.0 ** -149
    say(f"  weights at {np.max(off / bound):.3f} of their bound")
    assert np.all(off <= bound)


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("T,E,k,ng,kg", [(9, 1, 1, 1, 1), (400, 256, 8, 8, 4), (65, 60, 4, 1, 1), (30, 1024, 64, 1, 1),
                                         (33, 96, 6, 3, 2)])
def test_weights_round_once(T, E, k, ng, kg, score):
    for sigma in (0.1, 2.0, 20.0):
        say(f"route T={T} E={E} k={k} groups={ng}/{kg} score={score} sigma={sigma}")
        l = logits(T, E, T + E, sigma)
        l[T // 2, ::3] = -np.inf
        b = 0.2 * np.random.default_rng(E).standard_normal(E)
        for renorm in (True, False):
            check(l, k, None, score, renorm, 2.5, ng, kg)
            check(l, k, b, score, renorm, 1.0, ng, kg)


def test_weights_of_unrepresentable_scores():
    """Sigmoid scores below what 64 bits hold: ids by the logits, weights 0
    with and without their sum; just above, their quotients still hold."""
    E, k = 32, 4
    low = np.arange(E, dtype=np.float32)[None] / 4
    check(low - 800.0, k, score=1)
    check(low - 800.0, k, score=1, renorm=False)
    check(low - 650.0, k, score=1)
