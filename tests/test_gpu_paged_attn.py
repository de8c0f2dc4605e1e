"""paged_attn against the float64 oracle, within the bounds of its own roundings."""

import numpy as np
import pytest
import torch

import attn_bounds as bounds
from block_scaled_precision_fp8_amd import lib as L
from gpu_util import bf16_bits, dev, say, to_dev
from oracle import attn as A, formats as F

pytestmark = pytest.mark.gpu

FLOAT, UE8M0, BF16 = L.KV_FP8_FLOAT, L.KV_FP8_UE8M0, L.KV_BF16


def on_dev(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16).to(dev())


class Cache:
    """Random pages; .k and .v hold their float64 values."""

    def __init__(self, rng, pages, Hkv, page, D, fmt):
        self.fmt = fmt
        self.parts = []
        for _ in range(2):
            if fmt == BF16:
                codes, scale = F.bf16_round(rng.standard_normal((pages, Hkv, page, D))), None
            else:
                codes = F.e4m3_encode(np.clip(rng.standard_normal((pages, Hkv, page, D)) * 120.0, -448, 448))
                scale = (rng.integers(119, 122, (pages, Hkv, page)).astype(np.uint8) if fmt == UE8M0 else
                         ((0.3 + rng.random((pages, Hkv, page))) / 120.0).astype(np.float32))
            self.parts.append((codes, scale))
        self.k, self.v = (A.cache_values(c, s, fmt) for c, s in self.parts)

    def tensors(self):
        up = lambda c: on_dev(c) if self.fmt == BF16 else to_dev(c)
        (kc, ks), (vc, vs) = self.parts
        return dict(k_cache=up(kc), v_cache=up(vc), k_scale=None if ks is None else to_dev(ks),
                    v_scale=None if vs is None else to_dev(vs), kv_fmt=self.fmt)


def poison(t, cache, hidden):
    """NaN (or infinities) wherever `hidden` (pages, page) says."""
    at = to_dev(hidden)[:, None, :].expand(t["k_cache"].shape[:3])
    for name in ("k", "v"):
        if cache.fmt == BF16:
            t[name + "_cache"][at] = float("nan") if name == "k" else float("inf")
        else:
            t[name + "_cache"][at] = 0x7F
            t[name + "_scale"][at] = 255 if cache.fmt == UE8M0 else float("nan")


def setup(rng, new, cached, Hq, Hkv, D, fmt, page, prefix=0, spare=3, extra=2):
    own = [-(-l // page) for l in cached]
    pre = -(-prefix // page)
    pages = sum(own) + pre + spare
    order = rng.permutation(pages)
    ptable = order[:pre].astype(np.int32)
    most = max(own + [0]) + extra
    table = rng.choice(np.array([-1, -7, 1 << 30, pages], np.int32), (len(cached), most))   # nothing there
    at = pre
    hidden = np.ones((pages, page), bool)
    for j in range(pre):
        hidden[ptable[j], :min(page, prefix - j * page)] = False
    for b, m in enumerate(own):
        table[b, :m] = order[at:at + m]
        at += m
        for j in range(m):
            hidden[table[b, j], :min(page, cached[b] - j * page)] = False
    cache = Cache(rng, pages, Hkv, page, D, fmt)
    T = sum(new)
    q = F.bf16_round(1.5 * rng.standard_normal((T, Hq, D)))
    return cache, q, table.astype(np.int32), ptable, hidden


def check(y, cache, q, cached, table, scale, **kw):
    want, spread, reach, keys = A.attention(q, cache.k, cache.v, cached, table, scale, **kw)
    live = ~np.isnan(want[:, 0, 0])
    got = F.bf16_decode(bf16_bits(y))
    if cache.fmt == BF16:
        vmax = 0.0
    else:
        s = cache.parts[1][1]
        vmax = 448.0 * (2.0 ** (s.astype(np.float64) - 127) if cache.fmt == UE8M0 else s).max()
    room = bounds.attention(want[live], spread[live], reach[live], keys[live], q.shape[2],
                            cache.fmt != BF16, vmax)
    off = np.abs(got[live] - want[live])
    assert np.all(np.isfinite(got[live]))
    worst = float((off / room).max()) if off.size else 0.0
    say("  worst share of the bound", round(worst, 3), "rel",
        float(np.linalg.norm(off) / max(np.linalg.norm(want[live]), 1e-30)))
    assert worst <= 1.0
    return live


def run(cache, q, new, cached, table, ptable, hidden, prefix=0, window=0, scale=None, use_start=None, pad=0,
        tail=0):
    """One call with poisoned surroundings, checked; pad: wider query rows, tail: tokens of no sequence."""
    T, Hq, D = q.shape
    scale = D ** -0.5 if scale is None else scale
    t = cache.tensors()
    poison(t, cache, hidden)
    start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    use_start = any(n != 1 for n in new) or tail if use_start is None else use_start
    wide = torch.full((T + tail, Hq * D + pad), float("nan"), dtype=torch.bfloat16, device=dev())
    wide[:T, :Hq * D] = on_dev(q).view(T, -1)
    y = torch.full((T + tail, Hq, D), 7.0, dtype=torch.bfloat16, device=dev())
    L.paged_attn(wide[:, :Hq * D].unflatten(1, (Hq, D)), kv_len=to_dev(np.array(cached, np.int32)),
                 page_table=to_dev(table), y=y, q_start=to_dev(start) if use_start else None,
                 prefix_table=to_dev(ptable) if prefix else None, prefix_len=prefix, scale=scale,
                 window=window, **t)
    torch.cuda.synchronize()
    assert torch.all(y[T:] == 7.0)
    check(y[:T], cache, q, cached, table, scale, q_start=start, prefix_table=ptable, prefix_len=prefix,
          window=window)
    return y


SHAPES = [
    # new tokens, cached, Hq, Hkv, D, fmt, page, prefix, window
    ([1], [1], 1, 1, 64, FLOAT, 16, 0, 0),
    ([1], [700], 32, 8, 128, FLOAT, 16, 0, 0),
    ([1], [2049], 8, 1, 256, BF16, 64, 0, 0),
    ([1] * 5, [0, 1, 129, 31, 1000], 6, 2, 128, UE8M0, 32, 0, 0),
    ([1] * 5, [0, 3, 129, 31, 700], 20, 1, 64, FLOAT, 16, 0, 100),
    ([1] * 3, [513, 5, 2000], 4, 4, 64, BF16, 128, 0, 1),
    ([1] * 4, [300, 90, 16, 48], 3, 3, 256, UE8M0, 16, 0, 33),
    ([3, 1, 0, 4, 2], [700, 1, 50, 4, 333], 16, 2, 256, UE8M0, 16, 0, 0),
    ([3, 1, 0, 4, 2], [700, 1, 50, 4, 333], 4, 2, 64, BF16, 32, 0, 40),
    ([2, 5], [1, 3], 4, 2, 128, FLOAT, 16, 0, 0),            # more new tokens than cached ones
    ([70], [70], 4, 1, 128, FLOAT, 64, 0, 0),
    ([70, 200, 33], [170, 200, 901], 6, 2, 64, BF16, 16, 0, 0),
    ([129, 1, 0, 260], [400, 77, 3, 261], 4, 2, 128, UE8M0, 32, 0, 130),
    ([97], [350], 10, 2, 256, FLOAT, 16, 0, 0),
    ([64, 40], [64, 500], 8, 8, 256, BF16, 128, 0, 17),
    ([1] * 3, [5, 0, 60], 10, 2, 128, BF16, 16, 237, 0),
    ([1] * 3, [5, 40, 60], 2, 2, 256, FLOAT, 16, 1, 0),
    ([1] * 20, list(range(20)), 4, 2, 128, FLOAT, 32, 777, 0),
    ([1] * 20, list(range(1, 400, 20)), 8, 2, 64, UE8M0, 16, 555, 200),
    ([2, 7, 0, 3], [9, 7, 0, 100], 8, 2, 128, BF16, 64, 130, 0),
    ([2, 7, 0, 3], [9, 7, 0, 100], 16, 2, 64, FLOAT, 16, 130, 60),
    ([50, 90], [50, 130], 4, 2, 256, UE8M0, 16, 333, 0),
    ([50, 90], [50, 130], 8, 2, 64, BF16, 16, 333, 41),
]


@pytest.mark.parametrize("case", range(len(SHAPES)))
def test_shapes(case):
    new, cached, Hq, Hkv, D, fmt, page, prefix, window = SHAPES[case]
    say("shape", case, SHAPES[case])
    rng = np.random.default_rng(case + 1)
    cache, q, table, ptable, hidden = setup(rng, new, cached, Hq, Hkv, D, fmt, page, prefix)
    run(cache, q, new, cached, table, ptable, hidden, prefix, window, pad=24)


ROOM = 1 << 14     # pages of a table that may be used: the many-row launch goes by what may come


@pytest.mark.parametrize("case", [i for i, c in enumerate(SHAPES) if sum(c[0]) * c[2] // c[3] > 16 * len(c[0])])
def test_shapes_with_room(case):
    """The same with tables so wide that blocks of many rows are launched."""
    new, cached, Hq, Hkv, D, fmt, page, prefix, window = SHAPES[case]
    say("room", case, SHAPES[case])
    rng = np.random.default_rng(case + 101)
    cache, q, table, ptable, hidden = setup(rng, new, cached, Hq, Hkv, D, fmt, page, prefix, extra=ROOM)
    run(cache, q, new, cached, table, ptable, hidden, prefix, window, pad=24)


MANY = [
    # rows by the thousand: workgroups of eight waves
    ([300], [300], 4, 1, 64, FLOAT, 16, 0, 0),
    ([270], [1111], 4, 1, 128, FLOAT, 64, 0, 0),
    ([150], [777], 8, 1, 256, UE8M0, 32, 0, 300),
    ([257], [600], 8, 2, 128, BF16, 16, 77, 0),
    ([260, 300], [700, 301], 8, 1, 64, BF16, 128, 200, 250),
    ([140], [140], 16, 2, 256, BF16, 16, 0, 0),
    ([600, 3, 0, 500], [650, 3, 9, 900], 8, 1, 64, UE8M0, 16, 0, 0),
    # single tokens, and a prefix for the many-row launch (four waves, eight)
    ([1] * 64, [1 + 3 * i % 50 for i in range(64)], 8, 2, 64, FLOAT, 64, 8400, 0),
    ([1] * 150, [1 + 7 * i % 60 for i in range(150)], 16, 2, 64, UE8M0, 64, 3500, 3000),
    ([1, 2, 0, 1] * 20, [2, 30, 4, 1] * 20, 8, 2, 128, BF16, 16, 6700, 0),
    ([1] * 40, [9] * 40, 16, 2, 256, FLOAT, 32, 7000, 0),
]


@pytest.mark.parametrize("case", range(len(MANY)))
def test_many_rows(case):
    new, cached, Hq, Hkv, D, fmt, page, prefix, window = MANY[case]
    say("many", case, new[:4], cached[:4], MANY[case][2:])
    rng = np.random.default_rng(case + 201)
    cache, q, table, ptable, hidden = setup(rng, new, cached, Hq, Hkv, D, fmt, page, prefix,
                                            extra=ROOM if max(new) > 2 else 2)
    run(cache, q, new, cached, table, ptable, hidden, prefix, window, pad=8)


@pytest.mark.parametrize("room", [2, ROOM])
@pytest.mark.parametrize("fmt", [FLOAT, UE8M0, BF16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new,cached,prefix", [([1], [300], 0), ([1, 1], [40, 700], 70), ([40], [90], 0),
                                               ([20, 30], [20, 45], 50)])
def test_types_and_heads(fmt, D, new, cached, prefix, room):
    say("types", fmt, D, new, cached, prefix, room)
    rng = np.random.default_rng(D + fmt)
    cache, q, table, ptable, hidden = setup(rng, new, cached, 4, 2, D, fmt, 16, prefix, extra=room)
    run(cache, q, new, cached, table, ptable, hidden, prefix)


def test_tokens_of_no_sequence_stay():
    rng = np.random.default_rng(3)
    for new, cached, room in (([2, 1], [20, 40], 2), ([80, 90], [80, 100], 2), ([80, 90], [80, 100], ROOM)):
        cache, q, table, ptable, hidden = setup(rng, new, cached, 4, 2, 128, FLOAT, 16, 30, extra=room)
        run(cache, q, new, cached, table, ptable, hidden, 30, tail=5)
        run(cache, q, new, cached, table, ptable, hidden, 0, tail=5)


@pytest.mark.parametrize("room,prefix", [(2, 0), (ROOM, 0), (2, 30), (ROOM, 30)])
def test_starts_out_of_order_or_range(room, prefix):
    rng = np.random.default_rng(4)
    new, cached = [30, 25, 40], [40, 25, 77]
    cache, q, table, ptable, hidden = setup(rng, new, cached, 4, 1, 64, FLOAT, 16, prefix, extra=room)
    t = cache.tensors()

    def call(starts):
        y = torch.full((95, 4, 64), 7.0, dtype=torch.bfloat16, device=dev())
        L.paged_attn(on_dev(q), kv_len=to_dev(np.array(cached, np.int32)), page_table=to_dev(table), y=y,
                     q_start=to_dev(np.array(starts, np.int32)), prefix_len=prefix,
                     prefix_table=to_dev(ptable) if prefix else None, **t)
        torch.cuda.synchronize()
        return y

    for starts in ([0, 60, 30, 95], [95, 50, 20, 0], [0, 95, 0, 95]):
        assert torch.all(call(starts) == 7.0)
    # ends beyond the tokens count as the last one's
    inside, outside = call([0, 30, 55, 95]), call([-5, 30, 55, 1000])
    assert torch.equal(inside, outside) and not torch.any(torch.all(inside.view(95, -1) == 7.0, 1))


@pytest.mark.parametrize("fmt", [FLOAT, BF16])
@pytest.mark.parametrize("new,cached,room", [([1, 1], [200, 90], 2), ([70, 3], [200, 90], 2),
                                             ([70, 3], [200, 90], ROOM)])
def test_bad_pages_are_hidden(fmt, new, cached, room):
    """Pages outside the cache in the middle of a sequence and of the prefix."""
    rng = np.random.default_rng(11)
    cache, q, table, ptable, hidden = setup(rng, new, cached, 4, 1, 64, fmt, 16, 100, extra=room)
    table[0, 2], table[1, 0], ptable[3] = -1, 1 << 29, -(1 << 31)
    run(cache, q, new, cached, table, ptable, hidden, 100)
    table[1, :] = -1                                          # nothing of its own left
    run(cache, q, new, cached, table, ptable, hidden, 100)
    if new[1] == 1:
        run(cache, q, new, cached, table, ptable, hidden, 0)


@pytest.mark.parametrize("fmt", [FLOAT, BF16])
@pytest.mark.parametrize("D", [64, 256])
def test_values_only_later_tokens_see(fmt, D):
    """NaN and infinities of a later token's value reach that token and the
    later ones, and no earlier one."""
    rng = np.random.default_rng(12)
    for n, length, room in ((4, 50, 2), (60, 170, 2), (60, 170, ROOM)):
        cache, q, table, ptable, hidden = setup(rng, [n], [length], 4, 2, D, fmt, 16, extra=room)
        t = cache.tensors()
        poison(t, cache, hidden)
        key = length - 2                                      # the last but one token's
        p, at = table[0, key // 16], key % 16
        first = F.bf16_decode(bf16_bits(t["v_cache"]))[p, 1, at, 3] if fmt == BF16 else None
        if fmt == BF16:
            t["v_cache"][p, 1, at, 3] = float("inf")
            t["v_cache"][p, 1, at, 5] = float("nan")
        else:
            t["v_cache"][p, 1, at, 3] = 0x7F
            t["v_cache"][p, 1, at, 5] = 0xFF
        assert first is None or np.isfinite(first)
        y = torch.empty(n, 4, D, dtype=torch.bfloat16, device=dev())
        L.paged_attn(on_dev(q), kv_len=to_dev(np.array([length], np.int32)), page_table=to_dev(table),
                     y=y, q_start=to_dev(np.array([0, n], np.int32)), **t)
        got = F.bf16_decode(bf16_bits(y))
        odd = np.zeros((n, 4, D), bool)
        odd[n - 2:, 2:, 3] = odd[n - 2:, 2:, 5] = True        # heads 2 and 3 read key head 1
        assert np.array_equal(~np.isfinite(got), odd)
        if fmt == BF16:
            assert np.all(got[n - 2:, 2:, 3] == np.inf) and np.all(np.isnan(got[n - 2:, 2:, 5]))
        want = A.attention(q, cache.k, cache.v, [length], table, D ** -0.5, q_start=[0, n])[0]
        assert np.abs(got - want)[~odd].max() < 0.05


def test_scores_of_all_sizes():
    """Large scores of both signs, and a reference that rises tile by tile."""
    rng = np.random.default_rng(13)
    for fmt in (FLOAT, BF16):
        new, cached = [1, 2], [900, 300]
        cache, q, table, ptable, hidden = setup(rng, new, cached, 4, 2, 128, fmt, 16)
        for scale in (3.0, 1e-4):
            run(cache, q, new, cached, table, ptable, hidden, scale=scale)
        # keys that grow along the sequence, along the query
        c = cache.parts[0]
        for j in range(900):
            p, at = table[0, j // 16], j % 16
            row = F.bf16_round(q[0, 0] * (j / 900.0) * 0.5)
            if fmt == BF16:
                c[0][p, :, at] = row
            else:
                c[0][p, :, at] = F.e4m3_encode(row)
                c[1][p, :, at] = 1.0
        cache.k = A.cache_values(c[0], c[1], fmt)
        run(cache, q, new, cached, table, ptable, hidden)


@pytest.mark.parametrize("fmt", [FLOAT, UE8M0])
def test_value_scales_of_all_sizes(fmt):
    """Value scales that differ by 2^40 from token to token and are all tiny
    or all large: the weights keep their precision."""
    rng = np.random.default_rng(14)
    for lo, hi, new, room in ((87, 127, [1, 3], 2), (30, 34, [1, 3], 2), (200, 204, [1, 3], 2),
                              (87, 127, [40, 9], ROOM), (200, 204, [40, 9], ROOM)):
        cached = [600, 200]
        cache, q, table, ptable, hidden = setup(rng, new, cached, 4, 2, 128, fmt, 16, extra=room)
        codes, _ = cache.parts[1]
        e = rng.integers(lo, hi, codes.shape[:3]).astype(np.uint8)
        cache.parts[1] = (codes, e if fmt == UE8M0 else (2.0 ** (e.astype(np.float64) - 127)).astype(np.float32))
        cache.v = A.cache_values(*cache.parts[1], fmt)
        run(cache, q, new, cached, table, ptable, hidden)


def test_one_dominant_value_scale():
    """The largest value belongs to a key of almost no weight: the others'
    weights are small beside it and must not be lost."""
    rng = np.random.default_rng(15)
    for new, room in (([1], 2), ([30], ROOM)):
        cache, q, table, ptable, hidden = setup(rng, new, [256], 4, 1, 64, FLOAT, 16, extra=room)
        codes, scale = cache.parts[1]
        scale[table[0, 0], :, 0] = 2.0 ** 20
        cache.parts[0][1][table[0, 0], :, 0] = 0.0           # its score is 0, the others' large
        cache.k, cache.v = (A.cache_values(c, s, FLOAT) for c, s in cache.parts)
        run(cache, q, new, [256], table, ptable, hidden)


def test_same_bits_again_and_on_another_stream():
    rng = np.random.default_rng(16)
    new, cached = [1] * 7, [3, 500, 77, 0, 1200, 16, 17]
    cache, q, table, ptable, hidden = setup(rng, new, cached, 8, 2, 128, FLOAT, 16, 200)
    t = cache.tensors()
    kw = dict(kv_len=to_dev(np.array(cached, np.int32)), page_table=to_dev(table),
              prefix_table=to_dev(ptable), prefix_len=200, **t)
    qd = on_dev(q)
    ys = [torch.empty(7, 8, 128, dtype=torch.bfloat16, device=dev()) for _ in range(3)]
    L.paged_attn(qd, y=ys[0], **kw)
    need = L.paged_attn_workspace_size(7, 7, 8, 2, 128, table.shape[1], 16, 200)
    ws = torch.full((need + 64,), 0xA5, dtype=torch.uint8, device=dev())
    L.paged_attn(qd, y=ys[1], workspace=ws[:need], **kw)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    L.paged_attn(qd, y=ys[2], stream=st.cuda_stream, **kw)
    torch.cuda.synchronize()
    assert torch.equal(ys[0], ys[1]) and torch.equal(ys[0], ys[2])
    assert torch.all(ws[need:] == 0xA5)
    with pytest.raises(L.BsFp8Error) as e:
        L.paged_attn(qd, y=ys[1], workspace=ws[:need - 1], **kw)
    assert e.value.status == L.ENOSPC


def test_captured_call_serves_other_lengths():
    rng = np.random.default_rng(17)
    most = [300, 900, 40]
    cache, q, table, ptable, hidden = setup(rng, [1] * 3, most, 4, 2, 128, FLOAT, 16, 50)
    t = cache.tensors()
    lens = to_dev(np.array(most, np.int32))
    qd, y = on_dev(q), torch.empty(3, 4, 128, dtype=torch.bfloat16, device=dev())
    ws = torch.empty(L.paged_attn_workspace_size(3, 3, 4, 2, 128, table.shape[1], 16, 50),
                     dtype=torch.uint8, device=dev())
    call = lambda: L.paged_attn(qd, kv_len=lens, page_table=td, y=y, prefix_table=pd, prefix_len=50,
                                workspace=ws, **t)
    td, pd = to_dev(table), to_dev(ptable)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for cached in (most, [1, 2, 3], [300, 0, 17], [33, 899, 40], most):
        lens.copy_(torch.tensor(cached, dtype=torch.int32))
        y.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        first = y.clone()
        check(first, cache, q, cached, table, 128 ** -0.5, prefix_table=ptable, prefix_len=50)
        call()
        torch.cuda.synchronize()
        assert torch.equal(first, y)


def test_far_page_of_a_large_cache():
    """Byte offsets of a page past 2^32."""
    rng = np.random.default_rng(18)
    Hkv, D, page = 8, 256, 128
    pages = (1 << 32) // (Hkv * D * page) + 3
    small, q, table, _, _ = setup(rng, [1], [300], 8, Hkv, D, FLOAT, page, spare=0, extra=0)
    t = small.tensors()
    far = pages - 1 - np.arange(3)
    for name in ("k_cache", "v_cache", "k_scale", "v_scale"):
        big = torch.zeros((pages,) + t[name].shape[1:], dtype=t[name].dtype, device=dev())
        big[to_dev(far[table[0]])] = t[name][to_dev(table[0].astype(np.int64))]
        t[name] = big
    y = torch.empty(1, 8, D, dtype=torch.bfloat16, device=dev())
    L.paged_attn(on_dev(q), kv_len=to_dev(np.array([300], np.int32)),
                 page_table=to_dev(far[table].astype(np.int32)), y=y, **t)
    check(y, small, q, [300], table, D ** -0.5)


def test_many_sequences():
    """More sequences than a workgroup has lanes, most of them short."""
    rng = np.random.default_rng(19)
    cached = [int(v) for v in rng.integers(0, 40, 700)]
    cache, q, table, ptable, hidden = setup(rng, [1] * 700, cached, 2, 1, 64, UE8M0, 16)
    run(cache, q, [1] * 700, cached, table, ptable, hidden)


def test_as_many_sequences_as_there_may_be():
    rng = np.random.default_rng(23)
    cached = [int(v) for v in rng.integers(0, 20, 4096)]
    cache, q, table, ptable, hidden = setup(rng, [1] * 4096, cached, 1, 1, 64, FLOAT, 16, extra=0)
    run(cache, q, [1] * 4096, cached, table, ptable, hidden)


def test_long_sequence():
    """Many partial results of one row."""
    rng = np.random.default_rng(20)
    cache, q, table, ptable, hidden = setup(rng, [1], [20011], 2, 1, 64, FLOAT, 64, extra=0)
    run(cache, q, [1], [20011], table, ptable, hidden)


def test_no_tokens_and_no_pages():
    z = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t, device=dev())
    c = dict(k_cache=z(1, 2, 16, 64), v_cache=z(1, 2, 16, 64), kv_fmt=BF16)
    i32 = torch.int32
    L.paged_attn(z(0, 4, 64), kv_len=z(0, t=i32), page_table=z(0, 3, t=i32), y=z(0, 4, 64), **c)
    y = torch.full((2, 4, 64), 5.0, dtype=torch.bfloat16, device=dev())
    L.paged_attn(z(2, 4, 64), kv_len=torch.full((2,), 9, dtype=i32, device=dev()), page_table=z(2, 0, t=i32),
                 y=y, **c)
    assert torch.all(y == 0)
