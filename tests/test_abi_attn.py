"""Argument checks of the rotary table, the cache append and the attention:
every refusal is reached on the host, before any HIP call (no GPU needed)."""

import os

import pytest

from block_scaled_precision_fp8_amd import lib as L

pytestmark = pytest.mark.skipif(not os.path.exists(L.LIB_PATH), reason="libbsfp8.so not built")

FAKE = 0x100000       # 16-byte aligned, never dereferenced by the checks
MIS = 0x100008        # misaligned
NAN, INF = float("nan"), float("inf")


def _call(fn, order, base, kw):
    a = dict(base)
    a.update(kw)
    return getattr(L.load(), fn)(*[a[n] for n in order.split()])


def _freq(**kw):
    return _call("rope_inv_freq", "scaling rot base factor low high orig out stream",
                 dict(scaling=2, rot=128, base=10000.0, factor=8.0, low=1.0, high=32.0, orig=8192.0,
                      out=FAKE, stream=None), kw)


@pytest.mark.parametrize("kw,code", [
    (dict(scaling=3), L.EINVAL), (dict(scaling=-1), L.EINVAL), (dict(rot=-16), L.EINVAL),
    (dict(rot=24), L.EINVAL), (dict(rot=272), L.ENOTSUP), (dict(base=0.5), L.EINVAL),
    (dict(base=NAN), L.EINVAL), (dict(base=INF), L.EINVAL), (dict(factor=0.0), L.EINVAL),
    (dict(factor=-1.0), L.EINVAL), (dict(factor=NAN), L.EINVAL), (dict(scaling=1, factor=0.0), L.EINVAL),
    (dict(low=-1.0), L.EINVAL), (dict(low=32.0), L.EINVAL), (dict(high=NAN), L.EINVAL),
    (dict(high=INF), L.EINVAL), (dict(orig=0.0), L.EINVAL), (dict(orig=NAN), L.EINVAL),
    (dict(out=None), L.EINVAL), (dict(out=FAKE + 2), L.EINVAL), (dict(rot=0, out=None), L.OK),
])
def test_inv_freq_argument_checks(kw, code):
    assert _freq(**kw) == code


@pytest.mark.parametrize("kw", [dict(), dict(scaling=0, factor=NAN, low=NAN, high=NAN, orig=NAN),
                                dict(scaling=1, low=NAN, high=NAN, orig=NAN), dict(out=FAKE + 4),
                                dict(base=1.0)])
def test_inv_freq_accepts(kw):
    assert _freq(**kw) == L.EHIP                   # past the checks: no device here


def _append(**kw):
    return _call("rope_kv_append",
                 "q ldq qo ldqo k ldk v ldv pos freq rot inter m slots T Hq Hkv D fmt pages page kc vc "
                 "ks vs stream",
                 dict(q=FAKE, ldq=1024, qo=FAKE, ldqo=1024, k=FAKE, ldk=256, v=FAKE, ldv=256, pos=FAKE,
                      freq=FAKE, rot=128, inter=0, m=1.0, slots=FAKE, T=5, Hq=8, Hkv=2, D=128, fmt=0,
                      pages=3, page=16, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, stream=None), kw)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), L.EINVAL), (dict(T=2**31), L.EINVAL), (dict(inter=2), L.EINVAL),
    (dict(rot=-16), L.EINVAL), (dict(rot=24), L.EINVAL), (dict(rot=144), L.EINVAL),
    (dict(m=0.0), L.EINVAL), (dict(m=NAN), L.EINVAL), (dict(m=INF), L.EINVAL),
    (dict(D=0, rot=0), L.EINVAL), (dict(D=96), L.EINVAL), (dict(D=96, rot=96), L.ENOTSUP),
    (dict(D=512, ldq=4096, ldqo=4096, ldk=1024, ldv=1024), L.ENOTSUP), (dict(q=None), L.EINVAL),
    (dict(qo=None), L.EINVAL), (dict(k=None), L.EINVAL), (dict(v=None), L.EINVAL),
    (dict(q=None, qo=None, k=None, v=None), L.EINVAL), (dict(pos=None), L.EINVAL),
    (dict(freq=None), L.EINVAL), (dict(pos=FAKE + 2), L.EINVAL), (dict(freq=FAKE + 1), L.EINVAL),
    (dict(Hq=0), L.EINVAL), (dict(Hq=1025, ldq=2**18, ldqo=2**18), L.EINVAL), (dict(ldq=1016), L.EINVAL),
    (dict(ldq=1028), L.EINVAL), (dict(ldqo=1016), L.EINVAL), (dict(ldqo=1028), L.EINVAL),
    (dict(q=MIS), L.EINVAL), (dict(qo=MIS), L.EINVAL), (dict(Hkv=0), L.EINVAL),
    (dict(ldk=248), L.EINVAL), (dict(ldk=260), L.EINVAL), (dict(ldv=248), L.EINVAL),
    (dict(ldv=260), L.EINVAL), (dict(k=MIS), L.EINVAL), (dict(v=MIS), L.EINVAL),
    (dict(slots=None), L.EINVAL), (dict(slots=FAKE + 4), L.EINVAL), (dict(fmt=3), L.EINVAL),
    (dict(fmt=-1), L.EINVAL), (dict(pages=0), L.EINVAL), (dict(pages=2**31), L.EINVAL),
    (dict(page=0), L.EINVAL), (dict(page=-16), L.EINVAL), (dict(page=8), L.ENOTSUP),
    (dict(page=48), L.ENOTSUP), (dict(kc=None), L.EINVAL), (dict(vc=None), L.EINVAL),
    (dict(ks=None), L.EINVAL), (dict(vs=None), L.EINVAL), (dict(kc=MIS), L.EINVAL),
    (dict(vc=MIS), L.EINVAL), (dict(ks=MIS), L.EINVAL), (dict(vs=MIS), L.EINVAL),
    (dict(T=0), L.OK), (dict(T=0, q=None, qo=None, k=None, v=None), L.OK),
])
def test_append_argument_checks(kw, code):
    assert _append(**kw) == code


@pytest.mark.parametrize("kw", [
    dict(), dict(fmt=2, ks=None, vs=None), dict(fmt=1), dict(q=None, qo=None, Hq=0, ldq=0, ldqo=0),
    dict(k=None, v=None, slots=None, kc=None, vc=None, ks=None, vs=None, pages=0, page=0, fmt=7, Hkv=0),
    dict(rot=0, pos=None, freq=None), dict(inter=1, rot=64), dict(page=1 << 20, pages=2**31 - 1)])
def test_append_accepts(kw):
    assert _append(**kw) == L.EHIP


SIZES = dict(T=6, B=3, Hq=8, Hkv=2, D=128, most=4, page=16, pre=40)


def _need(**kw):
    a = dict(SIZES)
    a.update(kw)
    return L.load().paged_attn_workspace_size(*[a[n] for n in "T B Hq Hkv D most page pre".split()])


def _attn(**kw):
    base = dict(SIZES, q=FAKE, ldq=1024, qs=FAKE, kl=FAKE, pt=FAKE, ppt=FAKE, kc=FAKE, vc=FAKE, ks=FAKE,
                vs=FAKE, fmt=0, pages=9, scale=0.1, win=0, y=FAKE, ws=FAKE, wsb=_need(), stream=None)
    return _call("paged_attn",
                 "q ldq qs kl pt most ppt pre kc vc ks vs fmt pages page T B Hq Hkv D scale win y ws wsb "
                 "stream", base, kw)


REFUSED_SIZES = [
    (dict(T=-1), L.EINVAL), (dict(B=-1), L.EINVAL), (dict(T=2**31), L.EINVAL), (dict(Hkv=0), L.EINVAL),
    (dict(Hq=1), L.EINVAL), (dict(Hq=9), L.EINVAL), (dict(Hq=2048, Hkv=2048), L.EINVAL),
    (dict(D=0), L.EINVAL), (dict(D=96), L.ENOTSUP), (dict(D=512), L.ENOTSUP), (dict(page=0), L.EINVAL),
    (dict(page=8), L.ENOTSUP), (dict(page=24), L.ENOTSUP), (dict(most=-1), L.EINVAL),
    (dict(pre=-1), L.EINVAL), (dict(B=4097), L.ENOTSUP), (dict(most=2**26 + 1), L.ENOTSUP),
    (dict(pre=2**30 + 1), L.ENOTSUP), (dict(T=2**29), L.ENOTSUP),
    (dict(T=4096, B=4096, Hq=64, Hkv=64, most=2**16), L.ENOTSUP),      # work units past 32 bits
]


@pytest.mark.parametrize("kw,code", REFUSED_SIZES + [
    (dict(scale=0.0), L.EINVAL), (dict(scale=-1.0), L.EINVAL), (dict(scale=NAN), L.EINVAL),
    (dict(scale=INF), L.EINVAL), (dict(win=-1), L.EINVAL), (dict(win=2**31), L.EINVAL),
    (dict(ldq=1016), L.EINVAL), (dict(ldq=1028), L.EINVAL), (dict(qs=None), L.EINVAL),
    (dict(fmt=3), L.EINVAL), (dict(pages=0), L.EINVAL), (dict(pages=2**31), L.EINVAL),
    (dict(q=None), L.EINVAL), (dict(kl=None), L.EINVAL), (dict(pt=None), L.EINVAL),
    (dict(ppt=None), L.EINVAL), (dict(y=None), L.EINVAL), (dict(q=MIS), L.EINVAL),
    (dict(y=MIS), L.EINVAL), (dict(qs=FAKE + 2), L.EINVAL), (dict(kl=FAKE + 1), L.EINVAL),
    (dict(pt=FAKE + 2), L.EINVAL), (dict(ppt=FAKE + 2), L.EINVAL), (dict(kc=None), L.EINVAL),
    (dict(vc=MIS), L.EINVAL), (dict(ks=None), L.EINVAL), (dict(vs=MIS), L.EINVAL),
    (dict(ws=None), L.EINVAL), (dict(ws=MIS), L.EINVAL), (dict(wsb=_need() - 1 if
     os.path.exists(L.LIB_PATH) else 0), L.ENOSPC), (dict(wsb=0), L.ENOSPC),
    (dict(T=0, q=None, ws=None, wsb=0), L.OK), (dict(B=0, T=0, qs=None, ws=None, wsb=0), L.OK),
])
def test_attn_argument_checks(kw, code):
    assert _attn(**kw) == code


@pytest.mark.parametrize("kw", [
    dict(), dict(fmt=2, ks=None, vs=None), dict(pre=0, ppt=None), dict(T=3, qs=None),
    dict(most=0, pt=None), dict(win=2**31 - 1), dict(qs=FAKE + 4, kl=FAKE + 8)])
def test_attn_accepts(kw):
    assert _attn(wsb=1 << 40, **kw) == L.EHIP


@pytest.mark.parametrize("kw,code", REFUSED_SIZES)
def test_workspace_of_refused_sizes(kw, code):
    assert _need(**kw) == 2**64 - 1


def test_workspace_holds_what_the_kernels_write():
    """meta, statistics and sums of every block id and split that a launch of
    these sizes can reach (16 rows a block where workgroups share keys, 128 or
    64 elsewhere)."""
    for T, B in ((1, 1), (64, 64), (5, 3), (700, 2), (4096, 1), (4096, 4096)):
        for Hq, Hkv in ((1, 1), (8, 2), (32, 8)):
            for D in (64, 128, 256):
                for keys, pre in ((1, 0), (5, 0), (600, 333), (16, 16384)):
                    need = _need(T=T, B=B, Hq=Hq, Hkv=Hkv, D=D, most=keys, pre=pre)
                    rows = T * (Hq // Hkv)
                    # at least one partial result for every row of one source, with its head's copies
                    assert need < 2**63 and need >= rows * Hkv * 8
    assert _need(T=0) == 0 and _need(B=0, T=0) == 0


@pytest.mark.parametrize("kw", [
    dict(T=32768, B=8, Hq=64, Hkv=8, most=2048, page=16, pre=0), dict(T=8192, B=1, Hq=32, Hkv=8, most=512, pre=0),
    dict(T=576, B=64, Hq=16, Hkv=4, D=64, most=4, pre=0), dict(T=4096, B=2, Hq=16, Hkv=16, D=256, most=256, pre=0)])
def test_workspace_of_complete_rows(kw):
    """Where no row's keys are split and no prefix is there, y is written at
    once: a pair of numbers per block and per row (in blocks of up to 256) of
    each key head, no partial sums of D values."""
    a = dict(SIZES, **kw)
    rows = a["T"] * (a["Hq"] // a["Hkv"])
    assert 0 < _need(**kw) <= (rows + 256 * a["B"] + rows // 64 + a["B"]) * a["Hkv"] * 8 + 4096
    assert _need(**{**kw, "pre": 16}) > rows * a["Hkv"] * a["D"] * 4            # the prefix's and their own
