"""rope_inv_freq and rope_kv_append against the float64 oracle."""

import numpy as np
import pytest
import torch

import attn_bounds as bounds
from block_scaled_precision_fp8_amd import lib as L
from gpu_util import bf16_bits, dev, say, to_dev, u8
from oracle import attn as A, formats as F, layer

pytestmark = pytest.mark.gpu

E4M3_HALF = 2.0 ** -4          # of the value, and 2^-10 of the scale below its normal range


def rand_bf16(rng, *shape):
    x = rng.standard_normal(shape) * np.exp(rng.standard_normal(shape[:-1] + (1,)))
    return F.bf16_round(x)


def on_dev(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16).to(dev())


def make_cache(rng, pages, Hkv, page, D, fmt):
    if fmt == L.KV_BF16:
        return on_dev(rng.standard_normal((pages, Hkv, page, D))), None
    codes = to_dev(rng.integers(0, 0x7F, (pages, Hkv, page, D), dtype=np.uint8))
    sc = rng.integers(100, 140, (pages, Hkv, page)).astype(np.uint8) if fmt else \
        rng.random((pages, Hkv, page)).astype(np.float32)
    return codes, to_dev(sc)


def values_of(t):
    return F.bf16_decode(bf16_bits(t)) if t.dtype == torch.bfloat16 else t.cpu().numpy()


def check_rows(name, got_codes, got_scale, want, slack, fmt):
    """Cached rows (n, H, D) against float64 ones, each within `slack` before rounding."""
    if fmt == L.KV_BF16:
        assert np.all(np.abs(got_codes - want) <= slack + bounds.BF16 * (np.abs(want) + slack)), name
        return
    amax = np.abs(want).max(-1)
    off = slack.max(-1)
    if fmt == L.KV_FP8_FLOAT:
        s = got_scale.astype(np.float64)
        zero = amax + off == 0
        assert np.all(np.where(zero, s == 1.0, np.abs(s * 448.0 - amax) <= off + 2 * bounds.FP32 * amax)), name
    else:
        e = got_scale.astype(np.int64) - 127
        lo = np.where(amax - off > 0, np.ceil(np.log2(np.maximum(amax - off, 1e-300) / 448.0) - 1e-12), -127)
        hi = np.where(amax + off > 0, np.ceil(np.log2(np.maximum(amax + off, 1e-300) / 448.0) + 1e-12), 0)
        assert np.all((e >= lo) & (e <= hi)), name
        s = 2.0 ** e
    got = F.e4m3_decode(got_codes).astype(np.float64) * s[..., None]
    room = slack + E4M3_HALF * (np.abs(want) + slack) + 2.0 ** -10 * s[..., None]
    assert np.all(np.abs(got - want) <= room * (1 + 1e-6)), name


CASES = [
    # T, Hq, Hkv, D, rot, interleaved, fmt, page, first, mscale
    (1, 32, 8, 128, 128, False, 0, 64, 700, 1.0),
    (1, 3, 1, 256, 64, True, 1, 16, 0, 1.0),
    (5, 7, 7, 64, 64, True, 0, 16, 12345, 1.25),
    (64, 16, 2, 128, 64, True, 1, 16, 4000, 1.0),
    (33, 4, 4, 64, 16, False, 2, 32, 1 << 20, 1.5),
    (17, 10, 5, 256, 256, False, 0, 128, 2 ** 31 - 400, 1.0),
    (1023, 5, 1, 64, 32, False, 1, 32, 7, 1.0),
    (1030, 9, 3, 128, 128, True, 2, 16, 99999, 0.75),
    (1025, 2, 1, 256, 128, False, 0, 16, 500000, 1.0),
    (9, 6, 2, 128, 0, False, 0, 16, 0, 1.0),
]


@pytest.mark.parametrize("T,Hq,Hkv,D,rot,inter,fmt,page,first,mscale", CASES)
def test_append(T, Hq, Hkv, D, rot, inter, fmt, page, first, mscale):
    say("append", T, Hq, Hkv, D, rot, inter, fmt, page, first)
    rng = np.random.default_rng(T * 1000 + D + rot)
    H = (Hq + 2 * Hkv) * D
    wide = np.zeros((T, H + 24))
    wide[:, :H] = rand_bf16(rng, T, Hq + 2 * Hkv, D).reshape(T, H)
    if T > 4:
        wide[2, Hq * D:] = 0.0                       # a key and a value of zeros: scale 1
    x = on_dev(wide)
    q, k, v = (t.unflatten(1, (-1, D)) for t in x[:, :H].split([Hq * D, Hkv * D, Hkv * D], 1))
    pos = (first + np.arange(T)).astype(np.int32)
    freq = A.inv_freq(rot, 500000.0)
    pages = -(-T // page) + 2
    slots = rng.permutation(pages * page)[:T].astype(np.int64)
    slots[rng.random(T) < 0.2] = -1
    if T > 8:
        slots[3], slots[5] = pages * page, 1 << 40   # outside: not cached
    kc, ks = make_cache(rng, pages, Hkv, page, D, fmt)
    vc, vs = make_cache(rng, pages, Hkv, page, D, fmt)
    before = [None if t is None else values_of(t).copy() for t in (kc, ks, vc, vs)]
    qo = torch.full((T, Hq * D + 16), 3.0, dtype=torch.bfloat16, device=dev())
    out = qo[:, :Hq * D].unflatten(1, (Hq, D))
    L.rope_kv_append(to_dev(pos), to_dev(freq) if rot else None, q=q, q_out=out, k=k, v=v,
                     slots=to_dev(slots), k_cache=kc, v_cache=vc, k_scale=ks, v_scale=vs, kv_fmt=fmt,
                     interleaved=inter, mscale=mscale)
    torch.cuda.synchronize()

    def slack(t):
        z = np.zeros_like(t)
        half = rot // 2
        ia = 2 * np.arange(half) if inter else np.arange(half)
        ib = ia + 1 if inter else ia + half
        z[..., ia] = z[..., ib] = bounds.rotated(t[..., ia], t[..., ib], mscale)
        return z

    xq, xk, xv = (t.reshape(T, -1, D) for t in np.split(wide[:, :H], [Hq * D, (Hq + Hkv) * D], 1))
    want = A.rotate(xq, pos, freq, inter, mscale)
    sl = slack(xq)
    got = values_of(out.contiguous())
    assert np.all(np.abs(got - want) <= sl + bounds.BF16 * (np.abs(want) + sl))
    assert np.array_equal(got[..., rot:], xq[..., rot:])
    assert torch.all(qo[:, Hq * D:] == 3.0)
    ok = (slots >= 0) & (slots < pages * page)
    p, at = slots[ok] // page, slots[ok] % page
    for name, c, s, c0, s0, w, slk in (
            ("k", kc, ks, before[0], before[1], A.rotate(xk, pos, freq, inter, mscale), slack(xk)),
            ("v", vc, vs, before[2], before[3], xv, np.zeros_like(xv))):
        got, gs = values_of(c), None if s is None else values_of(s)
        check_rows(name, got[p, :, at], None if gs is None else gs[p, :, at], w[ok], slk[ok], fmt)
        if name == "v" and fmt != L.KV_BF16 and ok.any():         # not rotated: the quantizer's own bits
            rq, rs = layer.quant_rows(w[ok].reshape(-1, D).astype(np.float32), D, fmt)
            assert np.array_equal(got[p, :, at].reshape(-1, D), rq)
            assert np.array_equal(gs[p, :, at].reshape(-1, 1), rs)
        rest = np.ones(got.shape[:3], bool)
        rest[p, :, at] = False
        assert np.array_equal(got[rest], c0[rest])
        assert gs is None or np.array_equal(gs[rest], s0[rest])


@pytest.mark.parametrize("T", [3, 1100])
def test_in_place_query_alone(T):
    rng = np.random.default_rng(T)
    x = rand_bf16(rng, T, 6, 128)
    q = on_dev(x)
    pos = np.arange(T, dtype=np.int32) * 7
    freq = A.inv_freq(128, 10000.0)
    L.rope_kv_append(to_dev(pos), to_dev(freq), q=q, q_out=q)
    want = A.rotate(x, pos, freq)
    sl = np.concatenate([bounds.rotated(x[..., :64], x[..., 64:], 1.0)] * 2, -1)
    assert np.all(np.abs(values_of(q) - want) <= sl + bounds.BF16 * (np.abs(want) + sl))


def test_keys_alone_and_other_stream():
    rng = np.random.default_rng(5)
    T, Hkv, D, page = 40, 2, 64, 16
    k, v = rand_bf16(rng, T, Hkv, D), rand_bf16(rng, T, Hkv, D)
    kc, _ = make_cache(rng, 3, Hkv, page, D, L.KV_BF16)
    vc, _ = make_cache(rng, 3, Hkv, page, D, L.KV_BF16)
    pos, freq = to_dev(np.zeros(T, np.int32)), to_dev(A.inv_freq(64, 10000.0))
    slots, kd, vd = to_dev(np.arange(T)), on_dev(k), on_dev(v)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    L.rope_kv_append(pos, freq, k=kd, v=vd, slots=slots, k_cache=kc, v_cache=vc, kv_fmt=L.KV_BF16,
                     stream=st.cuda_stream)
    st.synchronize()
    flat = lambda c: values_of(c).transpose(0, 2, 1, 3).reshape(-1, Hkv, D)[:T]
    assert np.array_equal(flat(kc), k) and np.array_equal(flat(vc), v)     # position 0 turns nothing


def test_far_page_of_a_large_cache():
    """Byte offsets of a page past 2^32."""
    rng = np.random.default_rng(6)
    Hkv, D, page = 8, 256, 128
    pages = (1 << 32) // (Hkv * D * page) + 3
    kc = torch.zeros(pages, Hkv, page, D, dtype=torch.uint8, device=dev())
    vc = torch.zeros_like(kc)
    ks = torch.zeros(pages, Hkv, page, device=dev())
    vs = torch.zeros_like(ks)
    k, v = rand_bf16(rng, 2, Hkv, D), rand_bf16(rng, 2, Hkv, D)
    slots = np.array([(pages - 1) * page + 127, 5], np.int64)
    L.rope_kv_append(None, None, k=on_dev(k), v=on_dev(v), slots=to_dev(slots), k_cache=kc, v_cache=vc,
                     k_scale=ks, v_scale=vs)
    for c, s, x in ((kc, ks, k), (vc, vs, v)):
        rq, rs = layer.quant_rows(x.reshape(-1, D).astype(np.float32), D, 0)
        got = torch.stack([c[pages - 1, :, 127], c[0, :, 5]])
        assert np.array_equal(u8(got).reshape(-1, D), rq)
        assert np.array_equal(torch.stack([s[pages - 1, :, 127], s[0, :, 5]]).cpu().numpy().reshape(-1, 1), rs)
        assert int((s != 0).sum()) == 2 * Hkv


@pytest.mark.parametrize("scaling,kw", [(0, {}), (1, dict(factor=4.0)),
                                        (2, dict(factor=8.0, low=1.0, high=32.0, orig_len=8192.0)),
                                        (2, dict(factor=32.0, low=0.0, high=0.5, orig_len=131072.0))])
@pytest.mark.parametrize("rot", [16, 64, 256])
def test_inv_freq(scaling, kw, rot):
    out = torch.empty(rot // 2, device=dev())
    L.rope_inv_freq(out, base=500000.0, scaling=scaling, **kw)
    want = A.inv_freq(rot, 500000.0, scaling, **kw).astype(np.float64)
    # both round a 64-bit value that pow() may have off by some 2^-50
    assert np.all(np.abs(out.cpu().numpy() - want) <= 2.0 ** -23 * want)


@pytest.mark.parametrize("scaling,kw", [
    (0, dict(factor=0.0)), (0, dict(factor=float("nan"))),
    (0, dict(factor=-1.0, low=float("nan"), high=float("nan"), orig_len=float("nan"))),
    (1, dict(factor=4.0, low=float("nan"), high=float("nan"), orig_len=float("nan"))),
    (2, dict(factor=5e-324, low=1.0, high=1.5, orig_len=1e30))])          # every angle keeps its own
def test_inv_freq_looks_at_what_its_scaling_uses(scaling, kw):
    out = torch.empty(64, device=dev())
    L.rope_inv_freq(out, base=500000.0, scaling=scaling, **kw)
    want = A.inv_freq(128, 500000.0, 1 if scaling == 1 else 0, factor=4.0).astype(np.float64)
    assert np.all(np.abs(out.cpu().numpy() - want) <= 2.0 ** -23 * want)
