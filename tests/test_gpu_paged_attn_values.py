"""paged_attn where values, scales and scores differ widely from key to key:
every weight keeps its precision whatever the others are."""

import numpy as np
import pytest
import torch

import attn_plan
import attn_value_bounds as bounds
import test_gpu_attn_layer as layers
import test_gpu_paged_attn as P
from block_scaled_precision_fp8_amd import lib as L
from gpu_util import bf16_bits, dev, say, to_dev
from oracle import attn as A, formats as F

pytestmark = pytest.mark.gpu

FLOAT, UE8M0, BF16 = L.KV_FP8_FLOAT, L.KV_FP8_UE8M0, L.KV_BF16
ROOM = P.ROOM


def held(y, k, v, q, cached, table, scale, **kw):
    """y (tensor) within its bound of the oracle's attention over the pages k, v."""
    want, spread, reach, keys = A.attention(q, k, v, cached, table, scale, **kw)
    live = ~np.isnan(want[:, 0, 0])
    got = F.bf16_decode(bf16_bits(y))[live]
    room = bounds.attention(want[live], spread[live], reach[live], keys[live], q.shape[2], np.abs(v).max())
    off = np.abs(got - want[live])
    assert np.all(np.isfinite(got))
    worst = float((off / room).max())
    say("  worst share of the bound", round(worst, 3))
    assert worst <= 1.0


def appended(k, v, fmt, page, spare=2, rng=None):
    """A cache that rope_kv_append wrote (keys n, heads, D on random pages):
    its tensors, its pages' float64 values and the table."""
    n, H, D = k.shape
    pages = -(-n // page) + spare
    order = rng.permutation(pages)[:-(-n // page)].astype(np.int32)
    slots = order[np.arange(n) // page].astype(np.int64) * page + np.arange(n) % page
    cdt = torch.bfloat16 if fmt == BF16 else torch.uint8
    c = lambda: torch.zeros(pages, H, page, D, dtype=cdt, device=dev())
    s = lambda: None if fmt == BF16 else torch.zeros(
        pages, H, page, dtype=torch.uint8 if fmt == UE8M0 else torch.float32, device=dev())
    t = dict(k_cache=c(), v_cache=c(), k_scale=s(), v_scale=s(), kv_fmt=fmt)
    L.rope_kv_append(None, None, k=P.on_dev(k), v=P.on_dev(v), slots=to_dev(slots), **t)
    host = lambda x: None if x is None else (F.bf16_decode(bf16_bits(x)) if x.dtype == torch.bfloat16 else
                                             x.cpu().numpy())
    values = [A.cache_values(host(t[m + "_cache"]), host(t[m + "_scale"]), fmt) for m in "kv"]
    return t, values, order


def attend(q, t, n, order, room, **kw):
    """The last tokens of a sequence of n keys; room: what its table has room for."""
    T = q.shape[0]
    table = np.full((1, len(order) + room), -1, np.int32)
    table[0, :len(order)] = order
    y = torch.empty(q.shape, dtype=torch.bfloat16, device=dev())
    L.paged_attn(P.on_dev(q), kv_len=to_dev(np.array([n], np.int32)), page_table=to_dev(table), y=y,
                 q_start=to_dev(np.array([0, T], np.int32)), **t, **kw)
    return y, table


def under_one_key(rng, n, T, Hq, Hkv, D, where, gap):
    """Queries near one direction, and keys of which `where` stands some `gap` above the others."""
    u = rng.standard_normal(D)
    q = F.bf16_round(u + 0.2 * rng.standard_normal((T, Hq, D)))
    k = 0.3 * rng.standard_normal((n, Hkv, D))
    k[where] = gap * D ** 0.5 / (u @ u) * u
    return q, F.bf16_round(k)


@pytest.mark.parametrize("fmt", [FLOAT, UE8M0, BF16])
@pytest.mark.parametrize("size", [1.0, 0.1, 0.03, 0.01])
@pytest.mark.parametrize("T,room", [(1, 2), (3, 2), (48, ROOM)])
def test_zero_value_under_the_top_score(fmt, size, T, room):
    """A key that takes most of the weight and has a value of zeros, which the
    codec gives the scale 1: what the others add is all of y."""
    for D, where in ((64, 0), (128, 200), (256, 250)):
        say("zero value", fmt, size, T, room, D, where)
        rng = np.random.default_rng(D + T)
        n = 300
        q, k = under_one_key(rng, n, T, 4, 1, D, where, 10.0)
        v = F.bf16_round(size * rng.standard_normal((n, 1, D)))
        v[where] = 0.0
        t, (kv, vv), order = appended(k, v, fmt, 16, rng=rng)
        y, table = attend(q, t, n, order, room)
        held(y, kv, vv, q, [n], table, D ** -0.5, q_start=[0, T])


@pytest.mark.parametrize("T,room,n,gap", [(1, 0, 4096, 12.0), (16, ROOM, 4096, 12.0), (16, ROOM, 40000, 12.0)])
def test_thousands_of_keys_under_a_zero_value(T, room, n, gap):
    """Each of them has little weight, all together much of it."""
    rng = np.random.default_rng(n + T)
    D = 64
    q, k = under_one_key(rng, n, T, 4, 1, D, 7, gap)
    v = F.bf16_round(1.0 + 0.3 * rng.standard_normal((n, 1, D)))
    v[7] = 0.0
    t, (kv, vv), order = appended(k, v, FLOAT, 64, rng=rng)
    y, table = attend(q, t, n, order, room)
    held(y, kv, vv, q, [n], table, D ** -0.5, q_start=[0, T])


@pytest.mark.parametrize("fmt", [FLOAT, UE8M0])
@pytest.mark.parametrize("T,room", [(1, 2), (30, ROOM)])
def test_elements_that_a_large_value_leaves_out(fmt, T, room):
    """A value of far larger scale whose codes are 0 in half of the elements:
    those are the other keys'."""
    rng = np.random.default_rng(31)
    for e in (20, 30, 40):
        cache, q, table, ptable, hidden = P.setup(rng, [T], [256], 4, 1, 64, fmt, 16, extra=room)
        codes, scale = cache.parts[1]
        p, at = table[0, 2], 5
        codes[p, :, at, ::2] = 0
        scale[p, :, at] = 127 + e if fmt == UE8M0 else 2.0 ** e
        cache.v = A.cache_values(codes, scale, fmt)
        y = P.run(cache, q, [T], [256], table, ptable, hidden)
        held(y, cache.k, cache.v, q, [256], table, 64 ** -0.5, q_start=[0, T])


@pytest.mark.parametrize("case", [0, 1, 3, 4, 6, 7, 9, 10, 12, 13, 16, 17, 18, 20, 21])
@pytest.mark.parametrize("room", [2, ROOM])
def test_ordinary_caches(case, room):
    """Sequences, prefixes and windows of FP8 caches within the same bound."""
    new, cached, Hq, Hkv, D, fmt, page, prefix, window = P.SHAPES[case]
    say("held", case, room, P.SHAPES[case])
    rng = np.random.default_rng(case + 301)
    cache, q, table, ptable, hidden = P.setup(rng, new, cached, Hq, Hkv, D, fmt, page, prefix, extra=room)
    y = P.run(cache, q, new, cached, table, ptable, hidden, prefix, window)
    held(y, cache.k, cache.v, q, cached, table, D ** -0.5, q_start=np.concatenate([[0], np.cumsum(new)]),
         prefix_table=ptable, prefix_len=prefix, window=window)


@pytest.mark.parametrize("fmt", [FLOAT, UE8M0])
@pytest.mark.parametrize("T,room", [(1, 2), (40, ROOM)])
@pytest.mark.parametrize("first,then", [(2.0 ** -85, 2.0 ** 75), (2.0 ** 75, 2.0 ** -85), (2.0 ** -60, 2.0 ** 70)])
def test_scales_of_both_ends_in_one_sequence(fmt, T, room, first, then):
    """Keys of equal scores and of value scales from both ends of their range: the
    weights' sum keeps the share of either half."""
    rng = np.random.default_rng(41)
    n = 1500
    cache, q, table, ptable, hidden = P.setup(rng, [T], [n], 4, 1, 64, fmt, 16, extra=room)
    cache.parts[0][0][:] = 0                                  # scores of 0
    cache.k = np.zeros_like(cache.k)
    codes, scale = cache.parts[1]
    for j in range(n):
        e = first if j < n // 2 else then
        scale[table[0, j // 16], :, j % 16] = 127 + int(np.log2(e)) if fmt == UE8M0 else e
    cache.v = A.cache_values(codes, scale, fmt)
    t = cache.tensors()
    P.poison(t, cache, hidden)
    y = torch.empty(T, 4, 64, dtype=torch.bfloat16, device=dev())
    L.paged_attn(P.on_dev(q), kv_len=to_dev(np.array([n], np.int32)), page_table=to_dev(table), y=y,
                 q_start=to_dev(np.array([0, T], np.int32)), **t)
    held(y, cache.k, cache.v, q, [n], table, 0.125, q_start=[0, T])


@pytest.mark.parametrize("T,room", [(1, 2), (2, 2), (40, ROOM)])
@pytest.mark.parametrize("D", [64, 256])
def test_value_scales_of_zero(T, room, D):
    """Keys whose value scales are 0 add nothing, alone in a tile or among
    others, whatever their codes."""
    for n, zeros in ((T, T), (T + 1, T + 1), (T + 32, T + 32), (T + 200, T), (T + 200, 60)):
        say("zero scales", T, room, D, n, zeros)
        rng = np.random.default_rng(n)
        cache, q, table, ptable, hidden = P.setup(rng, [T], [n], 4, 1, D, FLOAT, 16, extra=room)
        codes, scale = cache.parts[1]
        for j in range(zeros):
            scale[table[0, j // 16], :, j % 16] = 0.0
        cache.v = A.cache_values(codes, scale, FLOAT)
        y = P.run(cache, q, [T], [n], table, ptable, hidden)
        held(y, cache.k, cache.v, q, [n], table, D ** -0.5, q_start=[0, T])


@pytest.mark.parametrize("fmt", [FLOAT, UE8M0, BF16])
@pytest.mark.parametrize("T,room", [(1, 2), (40, ROOM)])
@pytest.mark.parametrize("scale", [1e5, 1e8, 1e11, 1e15, 1e30])
def test_scores_that_only_one_key_survives(fmt, T, room, scale):
    """Scores so large that their own rounding is whole exponents: the key
    with the largest has all the weight."""
    rng = np.random.default_rng(51)
    n, D = 700, 64
    for where in (0, 333, n - T):
        u = np.ones(D)
        u[::2] = -1.0
        q = F.bf16_round(u * (1.0 + rng.random((T, 4, 1))))
        k = rng.standard_normal((n, 1, D)) * 0.1
        k[where] = 1.5 * u                                    # by far the largest score of every row
        v = F.bf16_round(rng.standard_normal((n, 1, D)))
        t, (kv, vv), order = appended(F.bf16_round(k), v, fmt, 16, rng=rng)
        y, table = attend(q, t, n, order, room, scale=scale)
        at = vv[order[where // 16], 0, where % 16]
        got = F.bf16_decode(bf16_bits(y))
        assert np.all(np.isfinite(got))
        # the weight is 2^0 or, before a reference that rises, at most 2^10 of its own reference; the sums
        # are of one term: two roundings of 2^-16 and one to bf16
        assert np.all(np.abs(got - at) <= (bounds.BF16 * 1.01 + 2.0 ** -14) * np.abs(at))


@pytest.mark.parametrize("T,room", [(1, 2), (40, ROOM)])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_equal_scores_of_any_size(T, room, sign):
    """Equal keys have equal weights, however large their scores are."""
    n, D = 700, 64
    rng = np.random.default_rng(52)
    q = F.bf16_round(1.0 + rng.random((T, 4, D)))
    k = np.full((n, 1, D), sign * 1.234)
    v = F.bf16_round(rng.standard_normal((n, 1, D)))
    for fmt in (FLOAT, BF16):
        t, (kv, vv), order = appended(F.bf16_round(k), v, fmt, 16, rng=rng)
        at = vv[order[np.arange(n) // 16], 0, np.arange(n) % 16]
        for scale in (1.0, 1e4, 1e8, 1e11, 1e15, 1e30):
            y, table = attend(q, t, n, order, room, scale=scale)
            got = F.bf16_decode(bf16_bits(y))
            assert np.all(np.isfinite(got)), (fmt, scale)
            for i in range(T):
                see = at[:n - T + 1 + i]
                want, spread = see.mean(0), np.abs(see).mean(0)
                # equal products and sums: no error in the scores; weights 2^-16, fp32 sums 2^-24 a key
                room_ = bounds.BF16 * np.abs(want) + 1.01 * spread * (2.0 ** -15 + 2 * n * 2.0 ** -24)
                assert np.all(np.abs(got[i] - want) <= room_), (fmt, scale)


@pytest.mark.parametrize("D", [64, 256])
def test_rows_that_need_no_partial_sums(D):
    """Many short sequences, each row's keys in one piece: a workspace without
    partial sums, and nothing behind it is touched."""
    rng = np.random.default_rng(61)
    B, n, Hq, Hkv = 64, 9, 16, 4
    cached = [int(v) for v in rng.integers(0, 60, B)]
    cache, q, table, ptable, hidden = P.setup(rng, [n] * B, cached, Hq, Hkv, D, FLOAT, 16, extra=0)
    need = L.paged_attn_workspace_size(B * n, B, Hq, Hkv, D, table.shape[1], 16)
    assert need < B * n * Hq * D * 4                          # a partial sum per row would be more
    t = cache.tensors()
    P.poison(t, cache, hidden)
    ws = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device=dev())
    y = torch.empty(B * n, Hq, D, dtype=torch.bfloat16, device=dev())
    start = np.arange(B + 1) * n
    L.paged_attn(P.on_dev(q), kv_len=to_dev(np.array(cached, np.int32)), page_table=to_dev(table), y=y,
                 q_start=to_dev(start.astype(np.int32)), workspace=ws[:need], **t)
    torch.cuda.synchronize()
    assert torch.all(ws[need:] == 0xA5)
    held(y, cache.k, cache.v, q, cached, table, D ** -0.5, q_start=start)


@pytest.mark.parametrize("fmt", [FLOAT, UE8M0, BF16])
def test_a_layers_attention_within_its_roundings(fmt):
    """Norm to output linear: two prompts, then a token each, y within the
    attention's own roundings of what the cache holds."""
    rng = np.random.default_rng(70 + fmt)
    layer = layers.Layer(rng, fmt)
    table = rng.permutation(layers.PAGES)[:12].reshape(2, 6)
    td = layers.i32(table.tolist())
    slot = lambda b, j: int(table[b, j // layers.PAGE]) * layers.PAGE + j % layers.PAGE
    lens, new = [0, 0], [50, 21]
    for _ in range(3):
        at = [(b, lens[b] + j) for b in range(2) for j in range(new[b])]
        lens = [l + n for l, n in zip(lens, new)]
        start = np.concatenate([[0], np.cumsum(new)])
        x = P.on_dev(rng.standard_normal((len(at), layers.H)))
        q, y, _ = layer.step(x, layers.i32([j for _, j in at]),
                             torch.tensor([slot(b, j) for b, j in at], device=dev()), kv_len=layers.i32(lens),
                             page_table=td, q_start=layers.i32(start.tolist()))
        k, v = layer.values()
        held(y, k, v, F.bf16_decode(bf16_bits(q.contiguous())), lens, table, layers.D ** -0.5, q_start=start)
        new = [1, 1]


@pytest.mark.parametrize("B,n,keys", [(70, 6, 40), (70, 6, 300), (3, 13, 900), (3, 12, 900), (70, 12, 250)])
@pytest.mark.parametrize("fmt", [UE8M0, BF16])
def test_a_few_rows_of_each_sequence(fmt, B, n, keys):
    """24 to 52 rows of each, on either side of the borders between the launches."""
    rng = np.random.default_rng(B + n)
    new = [n] * B
    cached = [keys] + [int(v) for v in rng.integers(0, keys + 1, B - 1)]
    cache, q, table, ptable, hidden = P.setup(rng, new, cached, 8, 2, 64, fmt, 16, extra=0 if B > 3 else ROOM)
    y = P.run(cache, q, new, cached, table, ptable, hidden)
    held(y, cache.k, cache.v, q, cached, table, 0.125, q_start=np.arange(B + 1) * n)


@pytest.mark.parametrize("B,Hq,D,fmt,prefix,window", [
    # a prefix for the many-row launch: workgroups of four waves, of eight
    (64, 8, 64, FLOAT, 16600, 0), (33, 16, 256, BF16, 16000, 9000), (132, 16, 128, UE8M0, 4100, 0)])
def test_prefix_under_many_rows(B, Hq, D, fmt, prefix, window):
    rng = np.random.default_rng(D + prefix)
    cached = [1 + 3 * i % 50 for i in range(B)]
    cache, q, table, ptable, hidden = P.setup(rng, [1] * B, cached, Hq, 2, D, fmt, 64, prefix, extra=0)
    assert attn_plan.plan(B, B, Hq, 2, D, 64 * table.shape[1], prefix).pre_wide
    t = cache.tensors()
    P.poison(t, cache, hidden)
    y = torch.empty(B, Hq, D, dtype=torch.bfloat16, device=dev())
    L.paged_attn(P.on_dev(q), kv_len=to_dev(np.array(cached, np.int32)), page_table=to_dev(table), y=y,
                 prefix_table=to_dev(ptable), prefix_len=prefix, window=window, **t)
    held(y, cache.k, cache.v, q, cached, table, D ** -0.5, prefix_table=ptable, prefix_len=prefix, window=window)


@pytest.mark.parametrize("fmt", [FLOAT, UE8M0, BF16])
@pytest.mark.parametrize("T,room", [(1, 2), (40, ROOM)])
def test_largest_values(fmt, T, room):
    """Thousands of values of the largest size that is allowed, under scores
    that rise slowly: a reference that stays behind them."""
    rng = np.random.default_rng(81)
    n, D = 3000, 64
    u = rng.standard_normal(D)
    q = F.bf16_round(u + 0.01 * rng.standard_normal((T, 4, D)))
    k = (np.linspace(0.0, 6.0, n)[:, None] * u / (u @ u) * 8.0)[:, None]      # 0 to 6: under 2^10 of the first
    v = 2.0 ** 82 * rng.choice([-1.0, 1.0], (n, 1, D)) * rng.uniform(1.0, 2.0, (n, 1, D))
    t, (kv, vv), order = appended(F.bf16_round(k), F.bf16_round(v), fmt, 16, rng=rng)
    y, table = attend(q, t, n, order, room)
    held(y, kv, vv, q, [n], table, D ** -0.5, q_start=[0, T])
