"""Thin ctypes binding of libbsfp8.so (declared in include/bsfp8.h).

Argument marshalling only: every function here takes torch device tensors,
passes their data pointers, sizes and torch's current HIP stream to the
C entry point of the same name, and raises ``BsFp8Error`` on a non-OK
status.  The norm, router, MoE layer's and attention's functions check every
tensor's type, shape, order and device first (ValueError).  Nothing is computed in
Python.  The library is loaded from the package directory; if it is missing,
every call raises (there is no fallback path).
"""

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libbsfp8.so")

OK, EINVAL, ENOTSUP, ENOSPC, EHIP = 0, 1, 2, 3, 4
SCALE_FLOAT, SCALE_UE8M0 = 0, 1
ACT_DYNAMIC, ACT_STATIC = 0, 1
OP_BLOCK_GEMM, OP_LINEAR, OP_GROUPED_GEMM, OP_FP4_QUANT, OP_FP4_GEMM, OP_FP8_FP4_GEMM = \
    0, 1, 2, 3, 4, 5
OP_LINEAR_B32 = 6
OP_MOE_DECODE = 7
SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1
KV_FP8_FLOAT, KV_FP8_UE8M0, KV_BF16 = 0, 1, 2
ROPE_PLAIN, ROPE_LINEAR, ROPE_BY_PARTS = 0, 1, 2
GEMM_NONE, GEMM_TILE_128x256, GEMM_TILE_256x256, GEMM_DECODE = 0, 2, 3, 4

EXPORTS = ("bsfp8_version", "bsfp8_status_string", "bsfp8_workspace_size", "bsfp8_gemm_kernel",
           "fp8_quant_act", "fp8_quant_weight", "fp8_block_gemm", "fp8_linear",
           "fp8_grouped_gemm", "fp4_quant", "fp4_group_gemm", "fp8_dequant_weight",
           "fp8_scale_to_ue8m0", "mxfp4_quant_weight", "fp8_fp4_gemm",
           "fp8_grouped_gemm_silu_mul_quant", "fp8_linear_noalloc", "fp8_fp4_grouped_gemm",
           "fp8_add_rmsnorm_quant", "moe_route_topk", "fp8_moe_decode", "fp8_fp4_moe_decode",
           "rope_inv_freq", "rope_kv_append", "paged_attn", "paged_attn_workspace_size")
NOALLOC_SCRATCH_BYTES = 32 << 20     # BSFP8_NOALLOC_SCRATCH_BYTES


class BsFp8Error(RuntimeError):
    def __init__(self, fn, status, msg):
        super().__init__(f"{fn}: status {status} ({msg})")
        self.status = status


_lib = None

_P = ctypes.c_void_p
_F32 = ctypes.c_float
_F64 = ctypes.c_double
_I64 = ctypes.c_int64
_I32 = ctypes.c_int32
_SZ = ctypes.c_size_t
_REFUSED = ctypes.c_size_t(-1).value

_SIGS = {
    "bsfp8_version": (_I32, []),
    "bsfp8_status_string": (ctypes.c_char_p, [_I32]),
    "bsfp8_workspace_size": (_SZ, [_I32, _I64, _I64, _I64, _I32]),
    "bsfp8_gemm_kernel": (_I32, [_I64, _I64, _I64, _P]),
    "fp8_dequant_weight": (_I32, [_P, _I64, _I64, _I32, _I32, _I32, _P, _P, _P]),
    "fp8_scale_to_ue8m0": (_I32, [_P, _I64, _P, _P]),
    "mxfp4_quant_weight": (_I32, [_P, _I64, _I64, _I64, _P, _P, _P]),
    "fp8_fp4_gemm": (_I32, [_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I32, _P, _SZ, _P]),
    "fp8_grouped_gemm_silu_mul_quant": (_I32, [_P, _P, _P, _P, _P, _I32, _P, _P, _P, _I64, _I64,
                                               _I64, _I32, _P]),
    "fp8_quant_act": (_I32, [_P, _I64, _I64, _I64, _I32, _I32, _I32, _P, _P, _P]),
    "fp8_quant_weight": (_I32, [_P, _I64, _I64, _I64, _I32, _I32, _I32, _P, _P, _P]),
    "fp8_block_gemm": (_I32, [_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I32, _I32, _I32,
                              _P, _SZ, _P]),
    "fp8_linear": (_I32, [_P, _I64, _P, _P, _P, _P, _I64, _I64, _I64, _I32, _I32, _I32, _I32,
                          _P, _P, _SZ, _P]),
    "fp8_linear_noalloc": (_I32, [_P, _I64, _P, _P, _P, _P, _I64, _I64, _I64, _I32, _I32, _I32,
                                  _I32, _P, _P]),
    "fp8_fp4_grouped_gemm": (_I32, [_P, _P, _P, _P, _P, _I32, _P, _I64, _I64, _I64, _I32, _P]),
    "fp8_grouped_gemm": (_I32, [_P, _P, _P, _P, _P, _I32, _P, _I64, _I64, _I64, _I32, _I32,
                                _I32, _P, _SZ, _P]),
    "fp8_add_rmsnorm_quant": (_I32, [_P, _I64, _P, _P, _I64, _P, _F32, _I64, _I64, _I32, _I32,
                                     _I32, _P, _P, _P, _P, _P]),
    "moe_route_topk": (_I32, [_P, _I64, _I32, _P, _I64, _I32, _I32, _I32, _I32, _F32, _I32, _I32,
                              _P, _P, _P]),
    "fp8_moe_decode": (_I32, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I64, _I32, _I64, _I64,
                              _I32, _I32, _P, _SZ, _P]),
    "fp8_fp4_moe_decode": (_I32, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I64, _I32, _I64, _I64,
                                  _I32, _I32, _P, _SZ, _P]),
    "rope_inv_freq": (_I32, [_I32, _I64, _F64, _F64, _F64, _F64, _F64, _P, _P]),
    "rope_kv_append": (_I32, [_P, _I64, _P, _I64, _P, _I64, _P, _I64, _P, _P, _I64, _I32, _F32, _P,
                              _I64, _I32, _I32, _I32, _I32, _I64, _I32, _P, _P, _P, _P, _P]),
    "paged_attn": (_I32, [_P, _I64, _P, _P, _P, _I64, _P, _I64, _P, _P, _P, _P, _I32, _I64, _I32,
                          _I64, _I64, _I32, _I32, _I32, _F32, _I64, _P, _P, _SZ, _P]),
    "paged_attn_workspace_size": (_SZ, [_I64, _I64, _I32, _I32, _I32, _I64, _I32, _I64]),
    "fp4_quant": (_I32, [_P, _I64, _I64, _I32, _P, _P, _P, _P, _SZ, _P]),
    "fp4_group_gemm": (_I32, [_P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _P, _SZ, _P]),
}


def load(path=None):
    """Load (once) and return the ctypes handle; raises if the library is
    missing or lacks a declared symbol."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise BsFp8Error("load", -1, f"{p} not built; run "
                         "`python -m block_scaled_precision_fp8_amd.build`")
    # torch first: it brings its own HIP runtime under the same soname the
    # library links (libamdhip64.so.7), so the library then binds to that one
    # and kernels run on the runtime that owns torch's streams and memory.
    # Opened before torch, the library would load the system runtime and
    # torch a second one beside it.
    import torch
    global _device, _raw_stream
    _device = getattr(torch._C, "_cuda_getDevice", _device)
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _raw_stream)
    global _BF16, _FP32, _INT32, _BF16S, _FP32S, _BYTES, _CODES, _SCALES, _INT32S, _INT64S, _CACHES, _empty
    _BF16, _FP32, _INT32 = torch.bfloat16, torch.float32, torch.int32
    _INT32S, _INT64S, _empty = (_INT32,), (torch.int64,), torch.empty
    _BF16S, _FP32S, _BYTES = (_BF16,), (_FP32,), (torch.uint8,)
    _CODES = (torch.uint8, torch.float8_e4m3fn)
    _SCALES = (_FP32S, (torch.uint8, torch.float8_e8m0fnu))             # by scale_fmt
    _CACHES = (_CODES, _CODES, _BF16S)                                  # by kv_fmt
    lib = ctypes.CDLL(p)
    for name, (res, args) in _SIGS.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    if path is None:
        _lib = lib
    return lib


def status_string(s):
    return load().bsfp8_status_string(s).decode()


def _check(fn, s):
    if s != OK:
        raise BsFp8Error(fn, s, status_string(s))


def _ptr(t):
    return None if t is None else t.data_ptr()


# Replaced by load() with the functions below them, which make no objects (a
# call's stream: 0.2 against 3 us of host time).
def _device():
    import torch
    return torch.cuda.current_device()


def _raw_stream(device):
    import torch
    return torch.cuda.current_stream(device).cuda_stream


def _stream(stream):
    return _raw_stream(_device()) if stream is None else stream


def workspace_size(op, M, N, K, E=0):
    return int(load().bsfp8_workspace_size(op, M, N, K, E))


def gemm_kernel(M, N, K):
    """(GEMM_* kind, K splits) that fp8_block_gemm / fp8_linear use for M x N x K."""
    sp = ctypes.c_int32(0)
    kind = int(load().bsfp8_gemm_kernel(M, N, K, ctypes.byref(sp)))
    return kind, int(sp.value)


def _on_current_device(t):
    """Its device, -1 for none (refused later: shapes can be checked before)."""
    d = t.get_device()
    if d >= 0 and d != _device():
        raise ValueError("tensors must be on the current device")
    return d


def _operand(name, t, dtypes, shape, dev):
    """The address of a tensor that is as the kernels take it to be: dense, of
    one of the dtypes, the shape, on the device."""
    if t.dtype not in dtypes or t.shape != shape or not t.is_contiguous() or t.get_device() != dev:
        raise ValueError(f"{name} must be contiguous {tuple(shape)} of "
                         f"{' or '.join(str(d) for d in dtypes)} on device {dev}")
    return t.data_ptr()


def _heads(name, t, T, dev):
    """(address, row stride, heads, head size) of a bf16 (T, heads, size)
    tensor whose rows are dense; any row stride for a single row."""
    n, H, D = t.shape                      # ValueError for another number of dimensions
    ld, lh, one = t.stride()
    if t.dtype is not _BF16 or t.get_device() != dev:
        raise ValueError(f"{name} must be bf16 on device {dev}")
    if n != T or (one != 1 and D != 1) or (lh != D and H != 1):
        raise ValueError(f"rows of {name} must be contiguous, and {T} of them")
    return t.data_ptr(), (H * D if n <= 1 else ld), H, D


def _cache(k_cache, v_cache, k_scale, v_scale, kv_fmt, Hkv, D, dev):
    """(pages, page size, addresses of keys, values and their scales) of a
    paged cache, its tensors checked."""
    if kv_fmt not in (KV_FP8_FLOAT, KV_FP8_UE8M0, KV_BF16):
        raise ValueError("kv_fmt must be one of KV_FP8_FLOAT, KV_FP8_UE8M0, KV_BF16")
    pages, heads, page, size = shape = k_cache.shape
    if heads != Hkv or size != D:
        raise ValueError("caches must be (pages, key heads, page size, head size)")
    kinds = _CACHES[kv_fmt]
    pk = _operand("k_cache", k_cache, kinds, shape, dev)
    pv = _operand("v_cache", v_cache, kinds, shape, dev)
    if kv_fmt == KV_BF16:
        return pages, page, pk, pv, None, None
    if k_scale is None or v_scale is None:
        raise ValueError("FP8 caches need k_scale and v_scale")
    kinds, shape = _SCALES[kv_fmt], (pages, heads, page)
    return (pages, page, pk, pv, _operand("k_scale", k_scale, kinds, shape, dev),
            _operand("v_scale", v_scale, kinds, shape, dev))


def _launch_workspace(need, device, stream):
    """Workspace for one launch, from that launch's stream: memory of the
    current one may still be in use there, and is given out again while the
    launch runs."""
    if stream is None:
        return _empty(need, dtype=_BYTES[0], device=device)
    import torch
    st = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
    with torch.cuda.stream(st):
        return torch.empty(need, dtype=torch.uint8, device=device)


def _workspace(op, M, N, K, E, ws, device):
    need = workspace_size(op, M, N, K, E)
    if ws is None and need:
        import torch
        ws = torch.empty(need, dtype=torch.uint8, device=device)
    return ws, (ws.numel() * ws.element_size() if ws is not None else 0)


def fp8_quant_act(x, xq, x_scale, group_k=128, act_scheme=ACT_DYNAMIC, scale_fmt=SCALE_FLOAT,
                  stream=None):
    """x: bf16 (M, >=K) with row stride ldx; xq: uint8 (M, K); x_scale: (M, G)."""
    M, K = xq.shape
    ldx = x.stride(0) if x.dim() == 2 else K
    _check("fp8_quant_act", load().fp8_quant_act(_ptr(x), M, K, ldx, group_k, act_scheme,
                                                 scale_fmt, _ptr(xq), _ptr(x_scale),
                                                 _stream(stream)))


def fp8_dequant_weight(wq, w_scale_inv, w, block_n=128, block_k=128, scale_fmt=SCALE_FLOAT,
                       stream=None):
    """wq: uint8 (N, K) E4M3; w_scale_inv: (NB, KB); w: bf16 (N, K) out."""
    N, K = wq.shape
    _check("fp8_dequant_weight", load().fp8_dequant_weight(_ptr(wq), N, K, block_n, block_k,
                                                           scale_fmt, _ptr(w_scale_inv),
                                                           _ptr(w), _stream(stream)))


def fp8_scale_to_ue8m0(scale, out, stream=None):
    """scale: fp32 tensor; out: uint8 tensor of the same number of elements."""
    _check("fp8_scale_to_ue8m0", load().fp8_scale_to_ue8m0(_ptr(scale), scale.numel(),
                                                           _ptr(out), _stream(stream)))


def mxfp4_quant_weight(w, wq4, w_scale, stream=None):
    """w: bf16 (N, >=K); wq4: uint8 (N, K/2); w_scale: uint8 (N, K/32)."""
    N, K = wq4.shape[0], wq4.shape[1] * 2
    ldw = w.stride(0) if w.dim() == 2 else K
    _check("mxfp4_quant_weight", load().mxfp4_quant_weight(_ptr(w), N, K, ldw, _ptr(wq4),
                                                           _ptr(w_scale), _stream(stream)))


def fp8_fp4_gemm(xq, x_scale, wq4, w_scale, y, bias=None, scale_fmt=SCALE_FLOAT,
                 workspace=None, stream=None):
    """xq: uint8 (M, K) E4M3; x_scale (M, K/128); wq4 (N, K/2); w_scale (N, K/32)."""
    M, K = xq.shape
    N = wq4.shape[0]
    ws, wsb = _workspace(OP_FP8_FP4_GEMM, M, N, K, 0, workspace, xq.device)
    _check("fp8_fp4_gemm", load().fp8_fp4_gemm(_ptr(xq), _ptr(x_scale), _ptr(wq4), _ptr(w_scale),
                                               _ptr(bias), _ptr(y), M, N, K, scale_fmt, _ptr(ws), wsb,
                                               _stream(stream)))


def fp8_grouped_gemm_silu_mul_quant(xq, x_scale, wq, w_scale_inv, seg_offsets, hq, h_scale,
                                    h_bf16=None, scale_fmt=SCALE_FLOAT, stream=None):
    """xq (T, K); wq (E, 2I, K) gate rows then up rows; hq (T, I) uint8;
    h_scale (T, I/128); h_bf16 optional bf16 (T, I)."""
    T, K = xq.shape
    E, N2 = wq.shape[0], wq.shape[1]
    _check("fp8_grouped_gemm_silu_mul_quant", load().fp8_grouped_gemm_silu_mul_quant(
        _ptr(xq), _ptr(x_scale), _ptr(wq), _ptr(w_scale_inv), _ptr(seg_offsets), E, _ptr(hq),
        _ptr(h_scale), _ptr(h_bf16), T, N2 // 2, K, scale_fmt, _stream(stream)))


def fp8_quant_weight(w, wq, w_scale_inv, block_n=128, block_k=128, scale_fmt=SCALE_FLOAT,
                     stream=None):
    N, K = wq.shape
    ldw = w.stride(0) if w.dim() == 2 else K
    _check("fp8_quant_weight", load().fp8_quant_weight(_ptr(w), N, K, ldw, block_n, block_k,
                                                       scale_fmt, _ptr(wq), _ptr(w_scale_inv),
                                                       _stream(stream)))


def fp8_block_gemm(xq, x_scale, wq, w_scale_inv, y, bias=None, block_n=128, block_k=128,
                   scale_fmt=SCALE_FLOAT, workspace=None, stream=None):
    M, K = xq.shape
    N = wq.shape[0]
    ws, wsb = (None, 0) if block_n == 32 else _workspace(OP_BLOCK_GEMM, M, N, K, 0, workspace,
                                                          xq.device)
    _check("fp8_block_gemm", load().fp8_block_gemm(
        _ptr(xq), _ptr(x_scale), _ptr(wq), _ptr(w_scale_inv), _ptr(bias), _ptr(y), M, N, K,
        block_n, block_k, scale_fmt, _ptr(ws), wsb, _stream(stream)))


def fp8_linear(x, wq, w_scale_inv, y, bias=None, block_n=128, block_k=128,
               act_scheme=ACT_DYNAMIC, scale_fmt=SCALE_FLOAT, act_scale=None, workspace=None,
               stream=None):
    """act_scale: device tensor holding the static scheme's calibrated scale
    (fp32, or one E8M0 byte); None for the dynamic scheme."""
    M = x.shape[0]
    N, K = wq.shape
    ws, wsb = _workspace(OP_LINEAR_B32 if block_k == 32 else OP_LINEAR, M, N, K, 0, workspace,
                         x.device)
    _check("fp8_linear", load().fp8_linear(
        _ptr(x), x.stride(0), _ptr(wq), _ptr(w_scale_inv), _ptr(bias), _ptr(y), M, N, K,
        block_n, block_k, act_scheme, scale_fmt, _ptr(act_scale), _ptr(ws), wsb,
        _stream(stream)))


def fp8_grouped_gemm(xq, x_scale, wq, w_scale_inv, seg_offsets, y, block_n=128, block_k=128,
                     scale_fmt=SCALE_FLOAT, workspace=None, stream=None):
    T, K = xq.shape
    E, N, _ = wq.shape
    ws, wsb = _workspace(OP_GROUPED_GEMM, T, N, K, E, workspace, xq.device)
    _check("fp8_grouped_gemm", load().fp8_grouped_gemm(
        _ptr(xq), _ptr(x_scale), _ptr(wq), _ptr(w_scale_inv), _ptr(seg_offsets), E, _ptr(y),
        T, N, K, block_n, block_k, scale_fmt, _ptr(ws), wsb, _stream(stream)))


def fp8_fp4_grouped_gemm(xq, x_scale, wq4, w_scale, seg_offsets, y, scale_fmt=SCALE_FLOAT,
                         stream=None):
    """xq (T, K) E4M3; x_scale (T, K/128); wq4 uint8 (E, N, K/2); w_scale
    uint8 (E, N, K/32); seg_offsets int32 (E+1,) on the device; y bf16 (T, N)."""
    T, K = xq.shape
    E, N = wq4.shape[0], wq4.shape[1]
    _check("fp8_fp4_grouped_gemm", load().fp8_fp4_grouped_gemm(
        _ptr(xq), _ptr(x_scale), _ptr(wq4), _ptr(w_scale), _ptr(seg_offsets), E, _ptr(y), T, N, K,
        scale_fmt, _stream(stream)))


def fp4_quant(x, q4, gscale, tscale, dynamic_tscale=1, workspace=None, stream=None):
    R, K = x.shape
    ws, wsb = _workspace(OP_FP4_QUANT, R, 0, K, 0, workspace, x.device)
    _check("fp4_quant", load().fp4_quant(_ptr(x), R, K, dynamic_tscale, _ptr(q4), _ptr(gscale),
                                         _ptr(tscale), _ptr(ws), wsb, _stream(stream)))


def fp4_group_gemm(xq4, x_gscale, x_tscale, wq4, w_gscale, w_tscale, y, workspace=None,
                   stream=None):
    M = xq4.shape[0]
    N = wq4.shape[0]
    K = xq4.shape[1] * 2
    ws, wsb = _workspace(OP_FP4_GEMM, M, N, K, 0, workspace, xq4.device)
    _check("fp4_group_gemm", load().fp4_group_gemm(
        _ptr(xq4), _ptr(x_gscale), _ptr(x_tscale), _ptr(wq4), _ptr(w_gscale), _ptr(w_tscale),
        _ptr(y), M, N, K, _ptr(ws), wsb, _stream(stream)))


def fp8_add_rmsnorm_quant(x, weight, xq, x_scale, residual=None, residual_out=None, y=None,
                          eps=1e-6, group_k=128, act_scheme=ACT_DYNAMIC, scale_fmt=SCALE_FLOAT,
                          act_scale=None, stream=None):
    """x: bf16 (M, K) with row stride ldx; weight bf16 (K,); residual and
    residual_out bf16 (M, K) with one row stride; y bf16 (M, K) out or None;
    xq uint8 or float8_e4m3fn (M, K) and x_scale (M, G) out, fp32 or (UE8M0)
    uint8 or float8_e8m0fnu, or both None; act_scale as for fp8_linear, of
    x_scale's type."""
    lib = load()
    dev = _on_current_device(x)
    shape, (ldx, one), ldr = x.shape, x.stride(), 0
    M, K = shape
    res = residual is not None and residual_out is not None
    if res:
        if residual.shape != shape or residual_out.shape != shape:
            raise ValueError("residual and residual_out need the shape of x")
        ldr, inner = residual.stride()
        one = one if inner == 1 else 0
        if residual_out is not residual:
            ldo, inner = residual_out.stride()
            one = one if inner == 1 else 0
            if ldo != ldr and M > 1:
                raise ValueError("residual and residual_out need the same row stride")
    if one != 1:
        raise ValueError("rows must be contiguous")
    if M == 1:                             # any stride: there is no next row
        ldx = ldr = K
    if dev < 0:
        raise ValueError("tensors must be on a GPU")
    bf16 = _BF16
    if x.dtype is not bf16 or (res and (
            residual.dtype is not bf16 or residual.get_device() != dev or
            residual_out.dtype is not bf16 or residual_out.get_device() != dev)):
        raise ValueError("x, residual and residual_out must be bf16 on one device")
    pw = _operand("weight", weight, _BF16S, (K,), dev)
    py = None if y is None else _operand("y", y, _BF16S, shape, dev)
    if xq is None or x_scale is None or group_k <= 0:
        pq, ps = _ptr(xq), _ptr(x_scale)   # refused by the library, but for two None
    else:
        kinds = _SCALES[scale_fmt == SCALE_UE8M0]
        pq = _operand("xq", xq, _CODES, shape, dev)
        ps = _operand("x_scale", x_scale, kinds, (M, -(-K // group_k)), dev)
        if act_scheme == ACT_STATIC and act_scale is not None and (
                act_scale.dtype not in kinds or act_scale.numel() < 1 or
                act_scale.get_device() != dev):
            raise ValueError("act_scale must be a scale of x_scale's type on its device")
    _check("fp8_add_rmsnorm_quant", lib.fp8_add_rmsnorm_quant(
        x.data_ptr(), ldx, _ptr(residual), _ptr(residual_out), ldr, pw, eps, M, K, group_k,
        act_scheme, scale_fmt, _ptr(act_scale), py, pq, ps,
        _raw_stream(dev) if stream is None else stream))


def moe_route_topk(logits, ids, weights, bias=None, score=SCORE_SOFTMAX, renorm=True, scale=1.0,
                   n_group=1, topk_group=1, stream=None):
    """logits: fp32 or bf16 (T, E) with row stride ldl; bias fp32 (E,) or
    None; ids int32 (T, k) out; weights fp32 (T, k) out."""
    lib = load()
    dev = _on_current_device(logits)
    (T, E), (ldl, one), shape = logits.shape, logits.stride(), ids.shape
    bf16 = logits.dtype is _BF16
    if not (bf16 or logits.dtype is _FP32) or ids.dtype is not _INT32 or \
            weights.dtype is not _FP32:
        raise ValueError("logits must be fp32 or bf16, ids int32 and weights fp32")
    if one != 1 or not (ids.is_contiguous() and weights.is_contiguous()):
        raise ValueError("rows of logits, ids and weights must be contiguous")
    if weights.shape != shape or shape[0] != T:
        raise ValueError("ids and weights must be (T, k)")
    if T == 1:                             # any stride: there is no next row
        ldl = E
    if dev < 0 or ids.get_device() != dev or weights.get_device() != dev:
        raise ValueError("tensors must be on one GPU")
    pb = None if bias is None else _operand("bias", bias, _FP32S, (E,), dev)
    _check("moe_route_topk", lib.moe_route_topk(
        logits.data_ptr(), ldl, int(bf16), pb, T, E, shape[1], score, int(renorm), scale, n_group,
        topk_group, ids.data_ptr(), weights.data_ptr(),
        _raw_stream(dev) if stream is None else stream))


def _moe_decode(fn, xq, x_scale, ids, weights, w13, w13_scale, w2, w2_scale, y, I, addend,
                scale_fmt, workspace, stream):
    lib = load()
    dev = _on_current_device(xq)
    T, H = xq.shape
    k = ids.shape[1]
    if ids.dtype is not _INT32 or weights.dtype is not _FP32:
        raise ValueError("ids must be int32 and weights fp32")
    if not (xq.is_contiguous() and ids.is_contiguous() and weights.is_contiguous()):
        raise ValueError("xq, ids and weights must be contiguous")
    E, w4 = w13.shape[0], fn == "fp8_fp4_moe_decode"
    per = 2 if w4 else 1
    if ids.shape != weights.shape or ids.shape[0] != T or y.shape != xq.shape or \
            w13.shape != (E, 2 * I, H // per) or w2.shape != (E, H, I // per):
        raise ValueError("shapes of tokens, ids, weights and experts do not agree")
    need = lib.bsfp8_workspace_size(OP_MOE_DECODE, T * k, H, I, 0)
    wsb = need if workspace is None else workspace.numel() * workspace.element_size()
    if wsb >= need:                        # one that is too small is the library's to refuse
        if dev < 0 or ids.get_device() != dev or weights.get_device() != dev:
            raise ValueError("tensors must be on one GPU")
        if xq.dtype not in _CODES:
            raise ValueError("xq must be E4M3 codes")
        if workspace is not None and not (workspace.get_device() == dev and workspace.is_contiguous()):
            raise ValueError("the workspace must be contiguous, on the device of xq")
        kinds, HB = _SCALES[scale_fmt == SCALE_UE8M0], -(-H // 128)
        _operand("x_scale", x_scale, kinds, (T, HB), dev)
        _operand("y", y, _BF16S, (T, H), dev)
        if addend is not None:
            _operand("addend", addend, _BF16S, (T, H), dev)
        if w4:
            codes, kinds, s13, s2 = _BYTES, _SCALES[1], (E, 2 * I, H // 32), (E, H, I // 32)
        else:
            codes, s13, s2 = _CODES, (E, -(-2 * I // 128), HB), (E, HB, -(-I // 128))
        if w13.dtype not in codes or not w13.is_contiguous() or w13.get_device() != dev or \
                w2.dtype not in codes or not w2.is_contiguous() or w2.get_device() != dev:
            raise ValueError("w13 and w2 must be contiguous codes on the device of xq")
        _operand("w13_scale", w13_scale, kinds, s13, dev)
        _operand("w2_scale", w2_scale, kinds, s2, dev)
    if workspace is None:
        workspace = _launch_workspace(need, xq.device, stream)
    _check(fn, getattr(lib, fn)(
        _ptr(xq), _ptr(x_scale), _ptr(ids), _ptr(weights), _ptr(w13), _ptr(w13_scale), _ptr(w2),
        _ptr(w2_scale), _ptr(addend), _ptr(y), T, k, H, I, E, scale_fmt, _ptr(workspace), wsb,
        _stream(stream)))


def fp8_moe_decode(xq, x_scale, ids, weights, w13, w13_scale, w2, w2_scale, y, addend=None,
                   scale_fmt=SCALE_FLOAT, workspace=None, stream=None):
    """xq (T, H), w13 (E, 2I, H) and w2 (E, H, I) E4M3 codes (uint8 or
    float8_e4m3fn); their scales fp32, or (UE8M0) uint8 or float8_e8m0fnu,
    x_scale (T, ceil(H/128)), w13_scale (E, 2I/128, ceil(H/128)), w2_scale
    (E, ceil(H/128), I/128); ids int32 (T, k); weights fp32 (T, k); addend
    bf16 (T, H) or None; y bf16 (T, H) out."""
    _moe_decode("fp8_moe_decode", xq, x_scale, ids, weights, w13, w13_scale, w2, w2_scale, y,
                w2.shape[2], addend, scale_fmt, workspace, stream)


def fp8_fp4_moe_decode(xq, x_scale, ids, weights, w13, w13_scale, w2, w2_scale, y, addend=None,
                       scale_fmt=SCALE_FLOAT, workspace=None, stream=None):
    """As fp8_moe_decode with MXFP4 experts: w13 uint8 (E, 2I, H/2), w13_scale
    uint8 (E, 2I, H/32); w2 uint8 (E, H, I/2), w2_scale uint8 (E, H, I/32)."""
    _moe_decode("fp8_fp4_moe_decode", xq, x_scale, ids, weights, w13, w13_scale, w2, w2_scale, y,
                2 * w2.shape[2], addend, scale_fmt, workspace, stream)


def rope_inv_freq(inv_freq, base=10000.0, scaling=ROPE_PLAIN, factor=1.0, low=1.0, high=32.0,
                  orig_len=0.0, stream=None):
    """inv_freq: fp32 (rot_dim / 2,) out, the rotary angles per position."""
    lib = load()
    dev = _on_current_device(inv_freq)
    if inv_freq.dim() != 1 or dev < 0:
        raise ValueError("inv_freq must be (rot_dim / 2,) on a GPU")
    p = _operand("inv_freq", inv_freq, _FP32S, inv_freq.shape, dev)
    _check("rope_inv_freq", lib.rope_inv_freq(
        scaling, 2 * inv_freq.shape[0], base, factor, low, high, orig_len, p,
        _raw_stream(dev) if stream is None else stream))


def rope_kv_append(positions, inv_freq, q=None, q_out=None, k=None, v=None, slots=None,
                   k_cache=None, v_cache=None, k_scale=None, v_scale=None, kv_fmt=KV_FP8_FLOAT,
                   interleaved=False, mscale=1.0, stream=None):
    """positions: int32 (T,); inv_freq: fp32 (rot_dim / 2,) or None (nothing
    is rotated); q and q_out bf16 (T, Hq, D), k and v bf16 (T, Hkv, D), each
    with a row stride; slots int64 (T,); caches (pages, Hkv, page size, D),
    uint8 or float8_e4m3fn or (KV_BF16) bf16; scales (pages, Hkv, page size),
    fp32 or (KV_FP8_UE8M0) uint8 or float8_e8m0fnu."""
    lib = load()
    lead = q if q is not None else k
    if lead is None or (q is None) != (q_out is None) or (k is None) != (v is None):
        raise ValueError("q and q_out, or k and v, or both pairs are needed")
    dev = _on_current_device(lead)
    if dev < 0:
        raise ValueError("tensors must be on a GPU")
    T = lead.shape[0]
    rot, pp, pf = 0, None, None
    if inv_freq is not None and inv_freq.shape[0]:
        rot = 2 * inv_freq.shape[0]
        pf = _operand("inv_freq", inv_freq, _FP32S, (rot // 2,), dev)
        pp = _operand("positions", positions, _INT32S, (T,), dev)
    pq = po = pk = pv = psl = pkc = pvc = pks = pvs = None
    ldq = ldo = ldk = ldv = Hq = Hkv = pages = 0
    page = 16
    if q is not None:
        pq, ldq, Hq, D = _heads("q", q, T, dev)
        po, ldo, Ho, Do = _heads("q_out", q_out, T, dev)
        if (Ho, Do) != (Hq, D):
            raise ValueError("q and q_out need the same shape")
    if k is not None:
        pk, ldk, Hkv, Dk = _heads("k", k, T, dev)
        pv, ldv, Hv, Dv = _heads("v", v, T, dev)
        if q is None:
            D = Dk
        if Hv != Hkv or Dk != D or Dv != D:
            raise ValueError("k and v need the same shape, and the head size of q")
        if slots is None or k_cache is None or v_cache is None:
            raise ValueError("k and v need slots, k_cache and v_cache")
        psl = _operand("slots", slots, _INT64S, (T,), dev)
        pages, page, pkc, pvc, pks, pvs = _cache(k_cache, v_cache, k_scale, v_scale, kv_fmt, Hkv, D,
                                                 dev)
    _check("rope_kv_append", lib.rope_kv_append(
        pq, ldq, po, ldo, pk, ldk, pv, ldv, pp, pf, rot, int(interleaved), mscale, psl, T, Hq, Hkv,
        D, kv_fmt, pages, page, pkc, pvc, pks, pvs,
        _raw_stream(dev) if stream is None else stream))


def paged_attn_workspace_size(T, B, Hq, Hkv, D, max_pages, page_size, prefix_len=0):
    return int(load().paged_attn_workspace_size(T, B, Hq, Hkv, D, max_pages, page_size, prefix_len))


def paged_attn(q, k_cache, v_cache, kv_len, page_table, y, k_scale=None, v_scale=None,
               kv_fmt=KV_FP8_FLOAT, q_start=None, prefix_table=None, prefix_len=0, scale=None,
               window=0, workspace=None, stream=None):
    """q: bf16 (T, Hq, D) with a row stride; caches and scales as for
    rope_kv_append; kv_len int32 (B,); page_table int32 (B, max_pages);
    q_start int32 (B + 1,) or None (T == B); prefix_table int32
    (>= ceil(prefix_len / page size),) or None; scale 1 / sqrt(D) unless
    given; y bf16 (T, Hq, D) out."""
    lib = load()
    dev = _on_current_device(q)
    if dev < 0:
        raise ValueError("tensors must be on a GPU")
    T = q.shape[0]
    pq, ldq, Hq, D = _heads("q", q, T, dev)
    py = _operand("y", y, _BF16S, (T, Hq, D), dev)
    _, Hkv, _, _ = k_cache.shape
    pages, page, pkc, pvc, pks, pvs = _cache(k_cache, v_cache, k_scale, v_scale, kv_fmt, Hkv, D, dev)
    B, most = shape = page_table.shape
    pl = _operand("kv_len", kv_len, _INT32S, (B,), dev)
    pt = _operand("page_table", page_table, _INT32S, shape, dev)
    if q_start is None and T != B:
        raise ValueError("q_start is needed where sequences have other than one token")
    ps = None if q_start is None else _operand("q_start", q_start, _INT32S, (B + 1,), dev)
    pp = None
    if prefix_len > 0:
        if prefix_table is None or prefix_table.dim() != 1 or \
                prefix_table.shape[0] * page < prefix_len:
            raise ValueError("prefix_table must be (>= ceil(prefix_len / page size),)")
        pp = _operand("prefix_table", prefix_table, _INT32S, prefix_table.shape, dev)
    need = lib.paged_attn_workspace_size(T, B, Hq, Hkv, D, most, page, prefix_len)
    if need == _REFUSED:                   # sizes that the library refuses by a status
        need = 0
    if workspace is None:
        workspace = _launch_workspace(need, q.device, stream) if need else None
        wsb = need
    else:
        wsb = workspace.numel() * workspace.element_size()
        if wsb >= need and not (workspace.get_device() == dev and workspace.is_contiguous()):
            raise ValueError("the workspace must be contiguous, on the device of q")
    _check("paged_attn", lib.paged_attn(
        pq, ldq, ps, pl, pt, most, pp, prefix_len, pkc, pvc, pks, pvs,
        kv_fmt, pages, page, T, B, Hq, Hkv, D, D ** -0.5 if scale is None else scale, window, py,
        _ptr(workspace), wsb, _raw_stream(dev) if stream is None else stream))
