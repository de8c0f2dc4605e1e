"""Argument checks of the norm, router and MoE layer entry points: every
refusal is reached on the host, before any HIP call (no GPU needed)."""

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


def _norm(**kw):
    return _call("fp8_add_rmsnorm_quant",
                 "x ldx r ro ldr w eps M K gk sch fmt st y xq xs stream",
                 dict(x=FAKE, ldx=256, r=FAKE, ro=FAKE, ldr=256, w=FAKE, eps=1e-6, M=16, K=256,
                      gk=128, sch=0, fmt=0, st=None, y=FAKE, xq=FAKE, xs=FAKE, stream=None), kw)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), L.EINVAL), (dict(K=-16), L.EINVAL), (dict(K=0), L.EINVAL), (dict(K=200), L.EINVAL),
    (dict(M=2**31), L.EINVAL), (dict(ldx=128), L.EINVAL), (dict(ldx=260), L.EINVAL),
    (dict(ldr=128), L.EINVAL), (dict(ldr=260), L.EINVAL), (dict(eps=0.0), L.EINVAL),
    (dict(eps=-1e-6), L.EINVAL), (dict(eps=NAN), L.EINVAL), (dict(eps=INF), L.EINVAL),
    (dict(fmt=2), L.EINVAL), (dict(sch=2), L.EINVAL), (dict(gk=0), L.EINVAL),
    (dict(gk=64), L.ENOTSUP), (dict(gk=32, sch=1, st=FAKE), L.ENOTSUP),
    (dict(sch=1), L.EINVAL), (dict(sch=1, st=FAKE + 2), L.EINVAL),
    (dict(x=None), L.EINVAL), (dict(w=None), L.EINVAL), (dict(r=None), L.EINVAL),
    (dict(ro=None), L.EINVAL), (dict(xq=None), L.EINVAL), (dict(xs=None), L.EINVAL),
    (dict(y=None, xq=None, xs=None), L.EINVAL), (dict(x=MIS), L.EINVAL), (dict(r=MIS), L.EINVAL),
    (dict(ro=MIS), L.EINVAL), (dict(w=MIS), L.EINVAL), (dict(y=MIS), L.EINVAL),
    (dict(xq=MIS), L.EINVAL), (dict(xs=MIS), L.EINVAL), (dict(M=0), L.OK),
    (dict(M=0, x=None), L.OK), (dict(M=2**27, K=4096, ldx=4096, ldr=4096), L.EINVAL),
])
def test_norm_argument_checks(kw, code):
    assert _norm(**kw) == code


@pytest.mark.parametrize("kw", [dict(), dict(r=None, ro=None, ldr=0), dict(xq=None, xs=None),
                                dict(y=None), dict(sch=1, st=FAKE), dict(fmt=1, sch=1, st=FAKE + 1),
                                dict(sch=1, xq=None, xs=None)])
def test_norm_accepts(kw):
    assert _norm(**kw) == L.EHIP                   # past the checks: no device here


def _route(**kw):
    return _call("moe_route_topk", "l ldl bf b T E k score renorm scale ng kg ids w stream",
                 dict(l=FAKE, ldl=64, bf=0, b=None, T=4, E=64, k=8, score=0, renorm=1, scale=1.0,
                      ng=1, kg=1, ids=FAKE, w=FAKE, stream=None), kw)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), L.EINVAL), (dict(T=2**31), L.EINVAL), (dict(E=0), L.EINVAL),
    (dict(E=1025, ldl=1025), L.EINVAL), (dict(ldl=63), L.EINVAL), (dict(k=0), L.EINVAL),
    (dict(k=65), L.EINVAL), (dict(E=128, ldl=128, k=65), L.ENOTSUP), (dict(bf=2), L.EINVAL),
    (dict(renorm=2), L.EINVAL), (dict(score=2), L.EINVAL), (dict(ng=0), L.EINVAL),
    (dict(ng=3), L.EINVAL), (dict(ng=4, kg=0), L.EINVAL), (dict(ng=4, kg=5), L.EINVAL),
    (dict(E=128, ldl=128, ng=128), L.ENOTSUP), (dict(l=None), L.EINVAL), (dict(ids=None), L.EINVAL),
    (dict(w=None), L.EINVAL), (dict(l=FAKE + 2), L.EINVAL), (dict(l=FAKE + 1, bf=1), L.EINVAL),
    (dict(b=FAKE + 2), L.EINVAL), (dict(ids=FAKE + 2), L.EINVAL), (dict(w=FAKE + 1), L.EINVAL),
    (dict(T=0, l=None), L.OK),
])
def test_route_argument_checks(kw, code):
    assert _route(**kw) == code


@pytest.mark.parametrize("kw", [dict(), dict(l=FAKE + 2, bf=1, ldl=65), dict(b=FAKE + 4, ng=8, kg=8)])
def test_route_accepts(kw):
    assert _route(**kw) == L.EHIP


def _moe(fn="fp8_moe_decode", **kw):
    need = L.workspace_size(L.OP_MOE_DECODE, 32, 256, 256)
    return _call(fn, "xq xs ids wt w13 s13 w2 s2 add y T k H I E fmt ws wsb stream",
                 dict(xq=FAKE, xs=FAKE, ids=FAKE, wt=FAKE, w13=FAKE, s13=FAKE, w2=FAKE, s2=FAKE,
                      add=None, y=FAKE, T=16, k=2, H=256, I=256, E=8, fmt=0, ws=FAKE, wsb=need,
                      stream=None), kw)


@pytest.mark.parametrize("fn", ["fp8_moe_decode", "fp8_fp4_moe_decode"])
@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), L.EINVAL), (dict(k=0), L.EINVAL), (dict(E=0), L.EINVAL), (dict(E=1025), L.EINVAL),
    (dict(I=0), L.EINVAL), (dict(I=192), L.EINVAL), (dict(I=-128), L.EINVAL), (dict(H=0), L.EINVAL),
    (dict(H=264), L.EINVAL), (dict(H=-16), L.EINVAL), (dict(fmt=2), L.EINVAL),
    (dict(T=129), L.ENOTSUP), (dict(k=17), L.ENOTSUP), (dict(H=2**22 + 32), L.ENOTSUP),
    (dict(I=2**22 + 128), L.ENOTSUP), (dict(T=128, k=16, I=2**20), L.ENOTSUP),
    (dict(xq=None), L.EINVAL), (dict(xs=None), L.EINVAL), (dict(ids=None), L.EINVAL),
    (dict(wt=None), L.EINVAL), (dict(w13=None), L.EINVAL), (dict(s13=None), L.EINVAL),
    (dict(w2=None), L.EINVAL), (dict(s2=None), L.EINVAL), (dict(y=None), L.EINVAL),
    (dict(xq=MIS), L.EINVAL), (dict(xs=MIS), L.EINVAL), (dict(ids=FAKE + 2), L.EINVAL),
    (dict(wt=FAKE + 2), L.EINVAL), (dict(w13=MIS), L.EINVAL), (dict(s13=MIS), L.EINVAL),
    (dict(w2=MIS), L.EINVAL), (dict(s2=MIS), L.EINVAL), (dict(y=MIS), L.EINVAL),
    (dict(add=MIS), L.EINVAL), (dict(ws=None), L.EINVAL), (dict(ws=MIS), L.EINVAL),
    (dict(wsb=16), L.ENOSPC), (dict(T=17), L.ENOSPC), (dict(T=0, ids=None, ws=None, wsb=0), L.OK),
])
def test_moe_argument_checks(fn, kw, code):
    assert _moe(fn, **kw) == code


def test_moe_h_granularity():
    """FP8 weights take H in steps of 16, MXFP4 weights in steps of 32."""
    assert _moe(H=272, wsb=1 << 30) == L.EHIP
    assert _moe("fp8_fp4_moe_decode", H=272, wsb=1 << 30) == L.EINVAL
    assert _moe("fp8_fp4_moe_decode", H=288, wsb=1 << 30) == L.EHIP


def test_norm_binding_refuses_unlike_strides():
    import torch
    x = torch.zeros(2, 32, dtype=torch.bfloat16)
    wide = torch.zeros(2, 48, dtype=torch.bfloat16)[:, :32]
    with pytest.raises(ValueError):
        L.fp8_add_rmsnorm_quant(x, x[0], None, None, residual=x, residual_out=wide, y=x, stream=0)


def test_norm_binding_refuses_other_shapes_and_orders():
    import torch
    x = torch.zeros(32, 32, dtype=torch.bfloat16)
    for kw in (dict(residual=x[:16], residual_out=x), dict(residual=x, residual_out=x[:, :16]),
               dict(residual=x.t(), residual_out=x.t())):
        with pytest.raises(ValueError):
            L.fp8_add_rmsnorm_quant(x, x[0], None, None, y=x, stream=0, **kw)
    with pytest.raises(ValueError):
        L.fp8_add_rmsnorm_quant(x.t(), x[0], None, None, y=x, stream=0)


def test_route_binding_refuses_other_types_and_orders():
    import torch
    l, ids, w = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    for bad in ((l.half(), ids, w), (l.double(), ids, w), (l, ids.long(), w), (l, ids, w.double()),
                (l.t().contiguous().t(), ids, w), (l, ids.t().contiguous().t(), w),
                (l, ids, w.t().contiguous().t()), (l, ids[:3], w[:3]), (l, ids, w[:, :1])):
        with pytest.raises(ValueError):
            L.moe_route_topk(*bad, stream=0)


@pytest.mark.parametrize("w4", [False, True])
def test_moe_binding_refuses_other_types_and_shapes(w4):
    import torch
    T, k, H, I, E, per = 4, 2, 256, 128, 3, 2 if w4 else 1
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)
    good = dict(xq=u8(T, H), x_scale=torch.ones(T, 2), ids=torch.zeros(T, k, dtype=torch.int32),
                weights=torch.zeros(T, k), w13=u8(E, 2 * I, H // per), w13_scale=torch.ones(E, 2, 2),
                w2=u8(E, H, I // per), w2_scale=torch.ones(E, 2, 1),
                y=torch.zeros(T, H, dtype=torch.bfloat16), workspace=u8(16), stream=0)
    fn = L.fp8_fp4_moe_decode if w4 else L.fp8_moe_decode
    with pytest.raises(L.BsFp8Error):              # past the binding: a short workspace
        fn(**good)
    for kw in (dict(ids=good["ids"].long()), dict(weights=good["weights"].double()),
               dict(ids=good["ids"][:2]), dict(weights=good["weights"][:, :1]),
               dict(ids=good["ids"].t().contiguous().t()), dict(xq=good["xq"].t().contiguous().t()),
               dict(w13=good["w13"][:2]), dict(w13=good["w13"][:, :I]), dict(w2=good["w2"][:, :128]),
               dict(w13=u8(E, 2 * I, H // per // 2)), dict(y=good["y"][:2])):
        with pytest.raises(ValueError):
            fn(**dict(good, **kw))


def test_bindings_refuse_another_device(monkeypatch):
    """A tensor on GPU 1 while GPU 0 is the current one (stand-ins: no GPU)."""
    import torch

    class OnGpu1(torch.Tensor):
        def get_device(self):
            return 1
    L.load()
    monkeypatch.setattr(L, "_device", lambda: 0)
    t = torch.zeros(4, 256).as_subclass(OnGpu1)
    ids, w = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    with pytest.raises(ValueError, match="current device"):
        L.moe_route_topk(t, ids, w, stream=0)
    with pytest.raises(ValueError, match="current device"):
        L.fp8_add_rmsnorm_quant(t, t, None, None, y=t, stream=0)
    with pytest.raises(ValueError, match="current device"):
        L.fp8_moe_decode(t, t, ids, w, t, t, torch.zeros(1, 1, 1), t, t, stream=0)
