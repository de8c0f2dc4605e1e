"""paged_attn's places in its workspace: no two workgroups share one, all lie
inside the size that is asked for, and the join reads what was written."""

import os
import random

import pytest

import attn_plan as model
from block_scaled_precision_fp8_amd import lib as L

pytestmark = pytest.mark.skipif(not os.path.exists(L.LIB_PATH), reason="libbsfp8.so not built")


def sizes(rng):
    Hkv = rng.choice((1, 2, 3, 8))
    Hq, D, page = Hkv * rng.choice((1, 2, 3, 4, 5, 7, 16)), rng.choice((64, 128, 256)), rng.choice((16, 32, 128))
    B = rng.choice((1, 2, 3, 7, 20, 70))
    most = rng.choice((0, 1, 3, 40, 300, 5000))
    new = rng.choice((1, 1, 4, 30, 200, 900))
    prefix = rng.choice((0, 0, 1, 333, 5000, 20000))
    return Hq, Hkv, D, page, B, most, new, prefix


def starts(rng, B, new):
    n = [rng.choice((0, 1, rng.randint(0, new), new)) for _ in range(B)]
    lead, tail = rng.choice((0, 0, 2)), rng.choice((0, 0, 5))
    start = [lead]
    for v in n:
        start.append(start[-1] + v)
    return start, start[-1] + tail


def check(p, w, T, Hq, Hkv):
    # every block number has its pair, every partial result rows of its own
    assert all(0 <= id < (p.own_blocks + p.pre_blocks) * Hkv for id in w.meta)
    assert (p.own_blocks + p.pre_blocks) * Hkv * 8 <= p.off_ml
    taken, spans = {}, []
    for id, place, rows in w.partials:
        spans.append((place * rows, place * rows + rows))
        taken.setdefault(id, []).append(place)
    spans.sort()
    assert all(a[1] <= b[0] for a, b in zip(spans, spans[1:]))
    if spans:
        assert not p.complete
        assert spans[0][0] >= 0 and spans[-1][1] <= p.partial_rows
        assert p.off_ml + spans[-1][1] * 8 <= p.off_part
    for id, (first, count) in w.meta.items():
        if count >= 0:
            assert sorted(taken.get(id, [])) == list(range(first, first + count))
        else:
            assert id in w.direct and id not in taken
    # a row's join finds the pairs and places of its own blocks
    for t in {0, 1, T // 3, T // 2, T - 2, T - 1}:
        if 0 <= t < T:
            for head in {0, Hq // 2, Hq - 1}:
                for id, row, rows in w.joined(t, head):
                    assert id in w.meta and 0 <= row < rows
                    assert all(r == rows for i, _, r in w.partials if i == id)


@pytest.mark.parametrize("seed", range(40))
def test_places(seed):
    rng = random.Random(seed)
    for _ in range(10):
        Hq, Hkv, D, page, B, most, new, prefix = sizes(rng)
        start, T = starts(rng, B, new)
        if T == 0:
            continue
        p = model.plan(T, B, Hq, Hkv, D, most * page, prefix)
        assert L.paged_attn_workspace_size(T, B, Hq, Hkv, D, most, page, prefix) == p.bytes
        for kind in range(3):
            room = most * page
            lens = [(0, room, rng.randint(0, room))[rng.randrange(3)] if kind else room for _ in range(B)]
            window = rng.choice((0, 0, 1, 100, 3000))
            w = model.Writes(p, T, Hq, Hkv, start, lens, window, prefix, D, rng.choice((256, 512, 768)))
            check(p, w, T, Hq, Hkv)


@pytest.mark.parametrize("T,B,Hq,Hkv,D,most,page,prefix", [
    (1, 1, 32, 8, 128, 44, 16, 0), (64, 64, 32, 8, 128, 10, 64, 16384), (4096, 2, 32, 8, 128, 94, 64, 0),
    (4096, 4096, 1, 1, 64, 2, 16, 0), (2048, 1, 64, 8, 128, 2048, 16, 700), (700, 2, 8, 2, 256, 600, 16, 333)])
def test_places_of_full_sequences(T, B, Hq, Hkv, D, most, page, prefix):
    p = model.plan(T, B, Hq, Hkv, D, most * page, prefix)
    assert L.paged_attn_workspace_size(T, B, Hq, Hkv, D, most, page, prefix) == p.bytes
    start = [T * b // B for b in range(B + 1)]
    w = model.Writes(p, T, Hq, Hkv, start, [most * page] * B, 0, prefix, D)
    check(p, w, T, Hq, Hkv)
    assert len(w.meta) >= T * (Hq // Hkv) // p.own_rows * Hkv


def test_a_planted_overlap_is_seen():
    """Places without the block's number: consecutive blocks of one workgroup share one."""
    p = model.plan(5, 5, 4, 1, 64, 160, 40)
    w = model.Writes(p, 5, 4, 1, list(range(6)), [160] * 5, 0, 40, 64, 2)
    w.partials = [(id, place - id, rows) for id, place, rows in w.partials]
    with pytest.raises(AssertionError):
        check(p, w, 5, 4, 1)
