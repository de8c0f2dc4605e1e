"""The norm, router and MoE bindings refuse every tensor that the kernels
would read or write wrongly: type, shape, order of its elements, device.  No
GPU and no launch: tensors that say they are on GPU 0 or 1 stand in, and the
library's calls are recorded."""

import os

import pytest
import torch

from block_scaled_precision_fp8_amd import lib as L

pytestmark = pytest.mark.skipif(not os.path.exists(L.LIB_PATH), reason="libbsfp8.so not built")

BF16, F32, U8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


class Gpu0(torch.Tensor):
    def get_device(self):
        return 0


class Gpu1(torch.Tensor):
    def get_device(self):
        return 1


def on0(t):
    return None if t is None else t.as_subclass(Gpu0)


class Recorder:
    """The library with its entry points recorded, not called."""

    def __init__(self, lib):
        self.bsfp8_workspace_size = lib.bsfp8_workspace_size
        self.bsfp8_status_string = lib.bsfp8_status_string
        self.calls = []

    def __getattr__(self, name):
        return lambda *a: self.calls.append((name, a)) or L.OK


@pytest.fixture
def calls(monkeypatch):
    rec = Recorder(L.load())
    monkeypatch.setattr(L, "_lib", rec)
    monkeypatch.setattr(L, "_device", lambda: 0)
    monkeypatch.setattr(L, "_raw_stream", lambda device: 0)
    return rec.calls


def refuses(calls, f, **kw):
    with pytest.raises(ValueError):
        f(**kw)
    assert calls == []


def columns(t):
    """The same shape and values, with the elements in another order."""
    return t.t().contiguous().t() if t.dim() == 2 else t.transpose(-1, -2).contiguous().transpose(-1, -2)


def inside(t):
    """The same shape, a slice of wider rows."""
    wide = torch.zeros(*t.shape[:-1], t.shape[-1] + 16, dtype=t.dtype)
    return wide[..., :t.shape[-1]]


# ------------------------------------------------------------------ norm

def norm_args(fmt=0, group=128, static=False):
    M, K = 4, 272
    sdt = U8 if fmt else F32
    z = lambda *s, t=BF16: torch.zeros(s, dtype=t)
    return {k: on0(v) for k, v in dict(
        x=z(M, K), weight=z(K), xq=z(M, K, t=U8), x_scale=z(M, -(-K // group), t=sdt), residual=z(M, K),
        residual_out=z(M, K), y=z(M, K), act_scale=z(1, t=sdt) if static else None).items()} | dict(
        group_k=group, scale_fmt=fmt, act_scheme=L.ACT_STATIC if static else L.ACT_DYNAMIC)


@pytest.mark.parametrize("fmt,group,static", [(0, 128, False), (1, 32, False), (0, 128, True), (1, 128, True)])
def test_norm_operands(calls, fmt, group, static):
    f = L.fp8_add_rmsnorm_quant
    good = norm_args(fmt, group, static)
    f(**good)
    f(**dict(good, y=None))
    f(**dict(good, xq=None, x_scale=None))
    f(**dict(good, residual=None, residual_out=None))
    f(**dict(good, residual_out=good["residual"], x=on0(inside(good["x"]))))
    f(**dict(good, xq=on0(good["xq"].view(E4M3))))
    if fmt:
        f(**dict(good, x_scale=on0(good["x_scale"].view(E8M0))))
    assert len(calls) == 6 + fmt
    calls.clear()
    names = ["x", "weight", "xq", "x_scale", "residual", "residual_out", "y"] + ["act_scale"] * static
    for n in names:
        t = good[n]
        refuses(calls, f, **dict(good, **{n: t.as_subclass(torch.Tensor)}))     # on no GPU
        refuses(calls, f, **dict(good, **{n: t.as_subclass(Gpu1)}))
        refuses(calls, f, **dict(good, **{n: on0(t.to(torch.float16))}))
        refuses(calls, f, **dict(good, **{n: on0(t.to(U8 if t.dtype == F32 else F32))}))
        if t.dim() == 2:
            refuses(calls, f, **dict(good, **{n: on0(columns(t))}))
            refuses(calls, f, **dict(good, **{n: t[:3]}))
            if n != "x":
                refuses(calls, f, **dict(good, **{n: t[:, :-1]}))
    for n in ("xq", "x_scale", "y"):
        refuses(calls, f, **dict(good, **{n: on0(inside(good[n]))}))
    refuses(calls, f, **dict(good, weight=good["weight"][:-16]))
    refuses(calls, f, **dict(good, weight=on0(torch.zeros(544, dtype=BF16)[::2])))
    refuses(calls, f, **dict(good, x_scale=good["x_scale"].reshape(-1)))
    if static:
        refuses(calls, f, **dict(good, act_scale=good["act_scale"][:0]))


def test_norm_single_row_of_any_stride(calls):
    """One row has no next: a column vector's transpose is a dense row."""
    good = norm_args()
    one = {n: good[n][:1] for n in ("x", "xq", "x_scale", "residual", "residual_out", "y")}
    L.fp8_add_rmsnorm_quant(**dict(good, **one))
    turned = {n: on0(torch.zeros(272, 1, dtype=BF16).t()) for n in ("x", "residual", "residual_out")}
    assert turned["x"].stride() == (1, 1)
    L.fp8_add_rmsnorm_quant(**dict(good, **dict(one, **turned)))
    (_, a), (_, b) = calls
    assert a[1] == b[1] == a[4] == b[4] == 272      # ldx, ldr


# ----------------------------------------------------------------- router

def route_args(bf16=False):
    z = lambda *s, t=F32: torch.zeros(s, dtype=t)
    return {k: on0(v) for k, v in dict(logits=z(4, 24, t=BF16 if bf16 else F32), ids=z(4, 3, t=I32),
                                       weights=z(4, 3), bias=z(24)).items()}


@pytest.mark.parametrize("bf16", [False, True])
def test_route_operands(calls, bf16):
    f = L.moe_route_topk
    good = route_args(bf16)
    f(**good)
    f(**dict(good, bias=None))
    f(**dict(good, logits=on0(inside(good["logits"]))))
    assert len(calls) == 3
    calls.clear()
    for n, t in good.items():
        refuses(calls, f, **dict(good, **{n: t.as_subclass(torch.Tensor)}))
        refuses(calls, f, **dict(good, **{n: t.as_subclass(Gpu1)}))
        refuses(calls, f, **dict(good, **{n: on0(t.to(torch.float16))}))
        refuses(calls, f, **dict(good, **{n: on0(t.to(torch.float64))}))
        if t.dim() == 2:
            refuses(calls, f, **dict(good, **{n: on0(columns(t))}))
    for t in (good["bias"][:23], on0(torch.zeros(25)), on0(good["bias"].to(BF16)),
              on0(torch.zeros(48)[::2]), good["bias"].reshape(1, 24)):
        refuses(calls, f, **dict(good, bias=t))
    refuses(calls, f, **dict(good, ids=on0(inside(good["ids"]))))
    refuses(calls, f, **dict(good, weights=on0(inside(good["weights"]))))


def test_route_single_token_of_any_stride(calls):
    good = route_args()
    one = dict(good, ids=good["ids"][:1], weights=good["weights"][:1])
    L.moe_route_topk(**dict(one, logits=good["logits"][:1]))
    L.moe_route_topk(**dict(one, logits=on0(torch.zeros(24, 1).t())))
    (_, a), (_, b) = calls
    assert a[1] == b[1] == 24                       # ldl


# -------------------------------------------------------------- MoE layer

def moe_args(w4, fmt):
    T, k, H, I, E = 4, 2, 288, 256, 3
    z = lambda *s, t=U8: torch.zeros(s, dtype=t)
    sdt = U8 if fmt else F32
    if w4:
        w = dict(w13=z(E, 2 * I, H // 2), w13_scale=z(E, 2 * I, H // 32), w2=z(E, H, I // 2),
                 w2_scale=z(E, H, I // 32))
    else:
        w = dict(w13=z(E, 2 * I, H), w13_scale=z(E, 4, 3, t=sdt), w2=z(E, H, I), w2_scale=z(E, 3, 2, t=sdt))
    t = dict(w, xq=z(T, H), x_scale=z(T, 3, t=sdt), ids=z(T, k, t=I32), weights=z(T, k, t=F32),
             y=z(T, H, t=BF16), addend=z(T, H, t=BF16), workspace=z(1 << 20))
    return {n: on0(v) for n, v in t.items()} | dict(scale_fmt=fmt)


@pytest.mark.parametrize("w4", [False, True])
@pytest.mark.parametrize("fmt", [0, 1])
def test_moe_operands(calls, w4, fmt):
    f = L.fp8_fp4_moe_decode if w4 else L.fp8_moe_decode
    good = moe_args(w4, fmt)
    tensors = {n: t for n, t in good.items() if n != "scale_fmt"}
    f(**good)
    f(**dict(good, addend=None))
    f(**dict(good, addend=good["y"], xq=on0(good["xq"].view(E4M3))))
    f(**dict(good, **{n: on0(t.view(E8M0)) for n, t in tensors.items() if "scale" in n and t.dtype == U8}))
    if not w4:
        f(**dict(good, w13=on0(good["w13"].view(E4M3)), w2=on0(good["w2"].view(E4M3))))
    assert len(calls) == 4 + (not w4)
    calls.clear()
    for n, t in tensors.items():
        refuses(calls, f, **dict(good, **{n: t.as_subclass(torch.Tensor)}))     # on no GPU
        refuses(calls, f, **dict(good, **{n: t.as_subclass(Gpu1)}))
        if n == "workspace":
            refuses(calls, f, **dict(good, workspace=on0(torch.zeros(2 << 20, dtype=U8)[::2])))
            continue
        refuses(calls, f, **dict(good, **{n: on0(t.to(torch.float16))}))
        refuses(calls, f, **dict(good, **{n: on0(t.to(U8 if t.dtype == F32 else F32))}))
        refuses(calls, f, **dict(good, **{n: on0(columns(t))}))
        refuses(calls, f, **dict(good, **{n: on0(inside(t))}))
        refuses(calls, f, **dict(good, **{n: t[:1]}))
        refuses(calls, f, **dict(good, **{n: t[..., :-1]}))
    refuses(calls, f, **dict(good, scale_fmt=1 - fmt))
    refuses(calls, f, **dict(good, addend=good["addend"][0]))
