"""The attention bindings refuse every tensor that the kernels would read or
write wrongly: type, shape, order of its elements, device.  No GPU and no
launch: tensors that say they are on GPU 0 or 1 stand in, and the library's
calls are recorded."""

import os

import pytest
import torch

from block_scaled_precision_fp8_amd import lib as L
from test_bindings_layer import Gpu1, Recorder, on0, refuses

pytestmark = pytest.mark.skipif(not os.path.exists(L.LIB_PATH), reason="libbsfp8.so not built")

BF16, F32, U8, I32, I64 = torch.bfloat16, torch.float32, torch.uint8, torch.int32, torch.int64
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
FORMATS = [(L.KV_FP8_FLOAT, U8, F32), (L.KV_FP8_FLOAT, E4M3, F32), (L.KV_FP8_UE8M0, U8, U8),
           (L.KV_FP8_UE8M0, E4M3, E8M0), (L.KV_BF16, BF16, None)]


@pytest.fixture
def calls(monkeypatch):
    lib = L.load()
    rec = Recorder(lib)
    rec.paged_attn_workspace_size = lib.paged_attn_workspace_size
    monkeypatch.setattr(L, "_lib", rec)
    monkeypatch.setattr(L, "_device", lambda: 0)
    monkeypatch.setattr(L, "_raw_stream", lambda device: 0)
    return rec.calls


def z(*s, t=BF16):
    return on0(torch.zeros(s, dtype=t))


def cache(fmt, codes, scale):
    c = dict(k_cache=z(5, 2, 16, 64, t=codes), v_cache=z(5, 2, 16, 64, t=codes), kv_fmt=fmt)
    if scale is not None:
        c |= dict(k_scale=z(5, 2, 16, t=scale), v_scale=z(5, 2, 16, t=scale))
    return c


def spoiled(a, name, t):
    """The arguments with one of them as it must not be."""
    other = {BF16: torch.float16, F32: BF16, U8: torch.int8, I32: I64, I64: I32, E4M3: torch.float8_e5m2,
             E8M0: torch.int8}[t.dtype]
    plain = torch.zeros(t.shape, dtype=t.dtype)
    wider = torch.zeros(t.shape[:-1] + (t.shape[-1] + 16,), dtype=t.dtype)
    return {"type": on0(torch.zeros(t.shape, dtype=other)), "shape": on0(wider), "device": plain.as_subclass(Gpu1),
            "cpu": plain, "inside": on0(wider[..., :t.shape[-1]])}


# ---------------------------------------------------------------- append

def append_args(fmt=L.KV_FP8_FLOAT, codes=U8, scale=F32):
    wide = on0(torch.zeros(3, 8 * 64 + 24, dtype=BF16))
    q, k, v = (t.unflatten(1, (-1, 64)) for t in wide[:, :512].split([256, 128, 128], 1))
    return dict(positions=z(3, t=I32), inv_freq=z(16, t=F32), q=q, q_out=z(3, 4, 64), k=k, v=v,
                slots=z(3, t=I64)) | cache(fmt, codes, scale)


@pytest.mark.parametrize("fmt,codes,scale", FORMATS)
def test_append_operands(calls, fmt, codes, scale):
    a = append_args(fmt, codes, scale)
    for name, t in a.items():
        if not isinstance(t, torch.Tensor):
            continue
        for kind, bad in spoiled(a, name, t).items():
            if name in ("q", "q_out", "k", "v") and kind == "inside":
                bad = on0(torch.zeros(3, t.shape[1], 80, dtype=BF16))[..., :64]     # heads apart
            if name == "inv_freq" and kind == "shape":
                continue                               # another rot_dim
            if name in ("positions", "slots", "inv_freq") and kind == "inside":
                bad = on0(torch.zeros(2 * t.shape[0], dtype=t.dtype))[::2]
            refuses(calls, L.rope_kv_append, **{**a, name: bad})
    if scale is not None:
        refuses(calls, L.rope_kv_append, **{**a, "k_scale": None})
    for name in ("q_out", "v", "slots", "k_cache", "v_cache", "q", "k"):
        refuses(calls, L.rope_kv_append, **{**a, name: None})
    refuses(calls, L.rope_kv_append, **{**a, "kv_fmt": 3})
    refuses(calls, L.rope_kv_append, **{**a, "q": a["q"][:2]})
    refuses(calls, L.rope_kv_append, **{**a, "k_cache": z(5, 3, 16, 64, t=codes)})
    refuses(calls, L.rope_kv_append, **{**a, "k_cache": z(5, 2, 32, 64, t=codes)})
    L.rope_kv_append(**a)
    (name, got), = calls
    assert name == "rope_kv_append" and len(got) == 26
    assert got[1] == 536 and got[3] == 256 and got[5] == 536 and got[10] == 32
    assert got[14:21] == (3, 4, 2, 64, fmt, 5, 16)


def test_append_parts(calls):
    a = append_args()
    L.rope_kv_append(a["positions"], a["inv_freq"], q=a["q"], q_out=a["q_out"])
    keys = {n: a[n] for n in ("k", "v", "slots", "k_cache", "v_cache", "k_scale", "v_scale")}
    L.rope_kv_append(a["positions"], a["inv_freq"], **keys)
    L.rope_kv_append(None, None, **keys)
    assert [c[0] for c in calls] == ["rope_kv_append"] * 3
    assert calls[0][1][4] is None and calls[1][1][0] is None
    assert calls[2][1][8:11] == (None, None, 0)
    with pytest.raises(ValueError):
        L.rope_kv_append(a["positions"], a["inv_freq"])


def test_append_single_token_of_any_stride(calls):
    wide = on0(torch.zeros(4, 64, 7, dtype=BF16))
    q = on0(torch.zeros(1, 4, 64, dtype=BF16).as_strided((1, 4, 64), (3, 64, 1)))
    assert q.stride(0) == 3 and wide is not None
    L.rope_kv_append(z(1, t=I32), z(16, t=F32), q=q, q_out=z(1, 4, 64))
    assert calls[0][1][1] == 256


def test_inv_freq_operand(calls):
    for bad in (z(16, t=BF16), z(2, 8, t=F32), on0(torch.zeros(32)[::2]), torch.zeros(16),
                torch.zeros(16).as_subclass(Gpu1)):
        refuses(calls, L.rope_inv_freq, inv_freq=bad)
    L.rope_inv_freq(z(16, t=F32), base=500000.0, scaling=L.ROPE_LINEAR, factor=4.0)
    assert calls[0][1][:4] == (1, 32, 500000.0, 4.0)


# ------------------------------------------------------------- attention

def attn_args(fmt=L.KV_FP8_FLOAT, codes=U8, scale=F32):
    return dict(q=z(6, 4, 64), y=z(6, 4, 64), kv_len=z(3, t=I32), page_table=z(3, 7, t=I32),
                q_start=z(4, t=I32), prefix_table=z(3, t=I32), prefix_len=40,
                workspace=on0(torch.zeros(1 << 22, dtype=U8))) | cache(fmt, codes, scale)


@pytest.mark.parametrize("fmt,codes,scale", FORMATS)
def test_attn_operands(calls, fmt, codes, scale):
    a = attn_args(fmt, codes, scale)
    for name, t in a.items():
        if not isinstance(t, torch.Tensor) or name == "workspace":
            continue
        for kind, bad in spoiled(a, name, t).items():
            if name == "q" and kind == "inside":
                bad = on0(torch.zeros(6, 4, 80, dtype=BF16))[..., :64]
            if name == "prefix_table" and kind == "shape":
                continue                               # longer than needed
            if t.dim() == 1 and kind == "inside":
                bad = on0(torch.zeros(2 * t.shape[0], dtype=t.dtype))[::2]
            if name == "page_table" and kind == "shape":
                bad = z(4, 7, t=I32)
            refuses(calls, L.paged_attn, **{**a, name: bad})
    refuses(calls, L.paged_attn, **{**a, "prefix_table": z(2, t=I32)})           # 32 keys of 40
    refuses(calls, L.paged_attn, **{**a, "prefix_table": None})
    refuses(calls, L.paged_attn, **{**a, "q_start": None})                       # 6 tokens, 3 sequences
    refuses(calls, L.paged_attn, **{**a, "workspace": torch.zeros(1 << 22, dtype=U8)})
    refuses(calls, L.paged_attn, **{**a, "workspace": on0(torch.zeros(1 << 23, dtype=U8)[::2])})
    refuses(calls, L.paged_attn, **{**a, "kv_len": z(3, 1, t=I32)})
    refuses(calls, L.paged_attn, **{**a, "kv_fmt": 5})
    L.paged_attn(**a)
    (name, got), = calls
    assert name == "paged_attn" and len(got) == 26
    assert got[1] == 256 and got[5] == 7 and got[7] == 40
    assert got[12:20] == (fmt, 5, 16, 6, 3, 4, 2, 64) and got[20] == 64 ** -0.5 and got[24] == 1 << 22


def test_attn_without_prefix_or_starts(calls):
    a = attn_args()
    L.paged_attn(**{**a, "prefix_len": 0, "prefix_table": None, "q": z(3, 4, 64), "y": z(3, 4, 64),
                    "q_start": None, "scale": 0.25, "window": 9})
    got = calls[0][1]
    assert got[2] is None and got[6] is None and got[20:22] == (0.25, 9)
