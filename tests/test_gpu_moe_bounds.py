"""The MoE layer held to the bounds of its own arithmetic (moe_bounds): sums
that cancel, in closed form, and h's codes and the output element by element
with outlier channels and few K blocks, where the bounds are narrowest."""

import numpy as np
import pytest

import moe_bounds as B
from block_scaled_precision_fp8_amd import synth
from oracle import formats as F
from oracle import quant as Q

from gpu_util import to_dev, to_dev_bf16, bf16_bits, rel_fro, say
from test_gpu_moe_decode import case, codes_of, experts, layer, probe, routing

pytestmark = pytest.mark.gpu

PAIRS = [0, 6, 30, 62, 126, 134, 190, 254]


def unit_scales(T, H, fmt):
    return np.full((T, H // 128), 127 if fmt else 1.0, np.uint8 if fmt else np.float32)


@pytest.mark.parametrize("w4", [False, True])
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("T", [8, 40])
def test_cancelling_gate_up(T, fmt, w4):
    """h = 16 2^-(j % 3) exactly, whatever the place of the pair."""
    H, I = 256, 128
    say(f"cancelling gate/up T={T} fmt={fmt} w4={w4}")
    made = [B.cancelling(H, I, p, w4, fmt) for p in PAIRS]
    codes = [B.encode_weight(w, w4, fmt) for _, w in made]
    w13, s13 = (to_dev(np.stack([c[i] for c in codes])) for i in (0, 1))
    ids = (np.arange(T) % len(PAIRS)).astype(np.int32)[:, None]
    xq = np.stack([F.e4m3_encode(made[i][0]) for i in ids[:, 0]])
    w2, s2 = probe(len(PAIRS), H, I, 0, fmt, w4)
    y = layer(fmt, w4, to_dev(xq), to_dev(unit_scales(T, H, fmt)), to_dev(ids),
              to_dev(np.ones((T, 1), np.float32)), (w13, s13, w2, s2))
    want = np.zeros((T, H))
    want[:, :I] = 16.0 * 2.0 ** -(np.arange(I) % 3)
    assert np.array_equal(F.bf16_decode(bf16_bits(y)), want)


@pytest.mark.parametrize("w4", [False, True])
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("T,k", [(3, 2), (24, 8), (128, 2)])
def test_cancelling_down(T, k, fmt, w4):
    """h = 448 at the pair and 1 elsewhere, so y = sum_j w_j 16 exactly; h
    quantized in the down launch (few rows) and before it."""
    H, I, E = 256, 256, len(PAIRS)
    say(f"cancelling down T={T} k={k} fmt={fmt} w4={w4}")
    w13, w2 = np.zeros((E, 2 * I, H)), np.zeros((E, H, I))
    for e, p in enumerate(PAIRS):
        x, w = B.cancelling(I, 1, p, w4, fmt)               # the pattern along I
        w13[e, :I, 0] = 32.0                                # silu(32) = 32 in fp32
        w13[e, I:, 0] = np.where(x == 448.0, 0.0, 2.0 ** -5)
        w13[e, I:, 1] = np.where(x == 448.0, 8.0, 0.0)
        w2[e] = w[0] * np.where(np.arange(H) % 2, -1.0, 1.0)[:, None]
    codes = [B.encode_weight(w, w4, fmt) for w in (*w13, *w2)]
    dev = [to_dev(np.stack([c[i] for c in codes[n * E:(n + 1) * E]])) for n in (0, 1) for i in (0, 1)]
    xq = np.zeros((T, H), np.uint8)
    xq[:, 0], xq[:, 1] = 0x38, 0x3E                         # 1.0, 1.75
    ids, _ = routing(T, k, E, seed=T)
    wt = np.tile(np.array([1.0, 0.5, 0.25, 0.125] * 4, np.float32)[:k], (T, 1))
    y = layer(fmt, w4, to_dev(xq), to_dev(unit_scales(T, H, fmt)), to_dev(ids), to_dev(wt), dev)
    # MXFP4: no small product in the pair's group; their number stays 128.
    # h's second group has the scale 1 / 448 in fp32: 2^-24 of 128 products
    # of 1/8, far below half a bf16 step
    want = 16.0 * wt.sum(1)[:, None] * np.where(np.arange(H) % 2, -1.0, 1.0)
    assert np.array_equal(F.bf16_decode(bf16_bits(y)), F.bf16_round(want))


@pytest.mark.parametrize("w4", [False, True])
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("T,k,H,I,E", [(6, 2, 128, 256, 3), (40, 2, 256, 128, 2), (24, 3, 384, 384, 5),
                                       (9, 4, 2048, 256, 6)])
def test_layer_within_its_arithmetic(T, k, H, I, E, fmt, w4):
    import torch
    say(f"bounds T={T} k={k} H={H} I={I} E={E} fmt={fmt} w4={w4}")
    rng = np.random.default_rng(T + H)
    x = rng.standard_normal((T, H), dtype=np.float32)
    x[:, rng.permutation(H)[:max(1, H // 40)]] *= 50.0
    xq, xs = Q.quant_act(synth.f32_to_bf16_bits(x), 128, fmt)
    w13, s13, w2, s2 = experts(E, H, I, fmt, w4, seed=T)
    ids, w = routing(T, k, E, seed=T)
    w = w * np.where(rng.random((T, k)) < 0.5, np.float32(-1), np.float32(1))   # sums that cancel
    add = synth.normal_bf16((T, H), 1.0, "moe", "misc", seed=T)
    dx = [to_dev(a) for a in (xq, xs, ids)]
    dw = [to_dev(a) for a in (w13, s13, w2, s2)]
    y = F.bf16_decode(bf16_bits(layer(fmt, w4, *dx, to_dev(w), dw, to_dev_bf16(add))))
    # h, slot by slot, by a down weight of ones on a diagonal
    h = np.zeros((T, k, I))
    for c in range(-(-I // H)):
        wp, sp = probe(E, H, I, c, fmt, w4)
        n = min(I, (c + 1) * H) - c * H
        for j in range(k):
            one = torch.zeros((T, k), device="cuda")
            one[:, j] = 1.0
            p = F.bf16_decode(bf16_bits(layer(fmt, w4, *dx, one, (*dw[:2], wp, sp))))
            h[:, j, c * H:c * H + n] = p[:, :n]
    v, eps = B.gate_up(xq, xs, ids, w13, s13, fmt, w4)
    groups = h.reshape(-1, 128)
    if fmt == 0:
        groups = codes_of(groups, np.abs(v).reshape(-1, 128).max(1))
    assert B.groups_outside(groups, v.reshape(-1, 128), eps.reshape(-1, 128), fmt) == []
    ref, tol = B.layer_error(groups.reshape(T, k, I), ids, w, w2, s2, fmt, w4, F.bf16_decode(add))
    off = np.abs(y - ref)
    say(f"  y at {np.max(off / tol):.3f} of its bound, rel fro {rel_fro(y, ref):.2e}")
    assert np.all(off <= tol)


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("T,k,H,I,E", [(17, 1, 7168, 256, 3), (32, 1, 8192, 128, 2), (24, 2, 7184, 128, 4)])
def test_wide_rows_many_tokens(T, k, H, I, E, fmt):
    """More than 16 tokens whose h is quantized in the down launch, 28 or 32
    output features to a workgroup."""
    case(T, k, H, I, E, fmt, add=True, seed=T)
