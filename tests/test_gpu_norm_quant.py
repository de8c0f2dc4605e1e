"""fp8_add_rmsnorm_quant against the float64 oracle: h bit-exact, the bf16 y,
codes and scales bit-exact (the kernel's row statistics are 64-bit and y is
the correctly rounded product, so nothing depends on the summation order)."""

import numpy as np
import pytest

from block_scaled_precision_fp8_amd import synth
from oracle import formats as F
from oracle import layer as Y

from gpu_util import to_dev, to_dev_bf16, bf16_bits, u8, say

pytestmark = pytest.mark.gpu


def run(x, w, r=None, fmt=0, group=128, static=None, with_y=True, with_q=True, in_place=False,
        eps=1e-6, pad=0, rpad=0, stream=None):
    """Device call on host bit patterns; returns host arrays."""
    import torch
    from block_scaled_precision_fp8_amd import lib as L
    M, K = x.shape

    def strided(a, p):
        full = np.full((M, K + p), 0x7FC0, np.uint16)         # NaN in the padding
        full[:, :K] = a
        return to_dev_bf16(full)[:, :K]

    xd, wd = strided(x, pad), to_dev_bf16(w)
    rd = strided(r, rpad) if r is not None else None
    ro = None
    if r is not None:
        ro = rd if in_place else strided(np.zeros_like(r), rpad)
    sdt = torch.uint8 if fmt else torch.float32
    G = -(-K // group)
    q_full = torch.full((M * K + 256,), 0xA5, dtype=torch.uint8, device="cuda")
    s_full = torch.full((M * G + 64,), 7, dtype=sdt, device="cuda")
    y_full = torch.full((M * K + 64,), float("nan"), dtype=torch.bfloat16, device="cuda")
    sc = None
    if static is not None:
        sc = torch.tensor([static], dtype=sdt, device="cuda")
    L.fp8_add_rmsnorm_quant(
        xd, wd, q_full[:M * K].view(M, K) if with_q else None,
        s_full[:M * G].view(M, G) if with_q else None, residual=rd, residual_out=ro,
        y=y_full[:M * K].view(M, K) if with_y else None, eps=eps, group_k=group,
        act_scheme=L.ACT_DYNAMIC if static is None else L.ACT_STATIC, scale_fmt=fmt,
        act_scale=sc, stream=stream)
    torch.cuda.synchronize()
    assert (q_full[M * K:] == 0xA5).all() and (s_full[M * G:] == 7).all()
    assert torch.isnan(y_full[M * K:].float()).all()
    if pad:
        assert (xd.as_strided((M, pad), (K + pad, 1), K).view(torch.int16) == 0x7FC0).all()
    if rpad:
        assert (ro.as_strided((M, rpad), (K + rpad, 1), K).view(torch.int16) == 0x7FC0).all()
    if not with_q:
        assert (q_full == 0xA5).all() and (s_full == 7).all()
    return (u8(q_full[:M * K].view(M, K)), s_full[:M * G].view(M, G).cpu().numpy(),
            None if ro is None else bf16_bits(ro.contiguous()),
            bf16_bits(y_full[:M * K].view(M, K)))


def check(x, w, r=None, fmt=0, group=128, static=None, eps=1e-6, **kw):
    q, s, h, y = run(x, w, r, fmt, group, static, eps=eps, **kw)
    rh, ry = Y.add_rmsnorm(x, w, eps, r)
    rq, rs = Y.quant_rows(ry, group, fmt, static)
    if r is not None:
        assert np.array_equal(F.bf16_decode(h), rh), "h differs"
    if kw.get("with_y", True):
        assert np.array_equal(F.bf16_decode(y), F.bf16_round(ry.astype(np.float64))), "y differs"
    if kw.get("with_q", True):
        assert np.array_equal(s, rs), f"{np.count_nonzero(s != rs)} scales differ"
        assert np.array_equal(q, rq), f"{np.count_nonzero(q != rq)} codes differ"


def inputs(M, K, seed=0):
    x = synth.llama_acts(M, K, seed=seed)
    r = synth.normal_bf16((M, K), 3.0, "single", "misc", seed=seed)
    w = synth.f32_to_bf16_bits(1.0 + 0.3 * synth.rng("single", "w", 0, seed).standard_normal(
        K, dtype=np.float32))
    return x, w, r


# row lengths below, at and past the chunk, wave, group and register limits
KS = [16, 32, 112, 128, 144, 496, 528, 1040, 2064, 4096, 4112, 7168, 8192, 8208, 16384, 20000,
      33024]


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("group", [128, 32])
@pytest.mark.parametrize("K", KS)
def test_norm_row_lengths(K, group, fmt):
    for M in (1, 5):
        say(f"norm M={M} K={K} group={group} fmt={fmt}")
        x, w, r = inputs(M, K, seed=K + M)
        check(x, w, r, fmt, group, pad=8, rpad=16)


@pytest.mark.parametrize("M,K", [(2, 4096), (64, 4096), (257, 1024), (1031, 528), (2500, 2048),
                                 (4100, 512), (300, 7168)])
def test_norm_many_rows(M, K):
    say(f"norm M={M} K={K}")
    x, w, r = inputs(M, K, seed=M)
    check(x, w, r, fmt=M % 2)
    check(x, w, None, fmt=1 - M % 2, group=32)


@pytest.mark.parametrize("K", [256, 4096, 20000])
def test_norm_in_place_and_parts(K):
    x, w, r = inputs(3, K, seed=2)
    say(f"norm parts K={K}")
    check(x, w, r, in_place=True)
    check(x, w, r, in_place=True, rpad=24, fmt=1)
    check(x, w, r, with_y=False)
    check(x, w, r, with_q=False)
    check(x, w, None, with_q=False)


@pytest.mark.parametrize("fmt,scale", [(0, 0.0437), (0, 3e-3), (0, 1e-41), (1, 123), (1, 110)])
def test_norm_static(fmt, scale):
    """Down to a scale that saturates nearly every code."""
    say(f"norm static fmt={fmt} scale={scale}")
    x, w, r = inputs(7, 1040, seed=9)
    check(x, w, r, fmt, 128, static=scale)


@pytest.mark.parametrize("fmt", [0, 1])
def test_norm_extremes(fmt):
    """Zero rows, signed zeros, rows far above and far below eps, one large
    element, constant rows whose maxima sit on a power-of-two border."""
    say(f"norm extremes fmt={fmt}")
    g = np.random.default_rng(4)
    K = 640
    rows = [np.zeros(K), np.full(K, -0.0), np.full(K, 1.0), np.full(K, 448.0),
            g.standard_normal(K) * 1e-20, g.standard_normal(K) * 1e-3,
            g.standard_normal(K) * 1e15, np.where(np.arange(K) == 77, 1e6, 0.0),
            np.where(np.arange(K) % 2 == 0, 0.0, -0.0), np.exp2(g.integers(-20, 20, K))]
    x = synth.f32_to_bf16_bits(np.array(rows, np.float32))
    w = synth.f32_to_bf16_bits(np.where(np.arange(K) % 5 == 0, -1.0, 0.5).astype(np.float32))
    w[3] = 0
    check(x, w, None, fmt, eps=1e-6)
    check(x, w, None, fmt, eps=1e-30, group=32)
    check(x, w, x[::-1].copy(), fmt, eps=2.5)


def test_norm_equals_quantizer_on_unit_rows():
    """Where y is a bf16 value (weights 1, mean square 1, eps lost), codes
    and scales are fp8_quant_act's of that y."""
    import torch
    from block_scaled_precision_fp8_amd import lib as L
    M, K = 9, 512
    x = synth.f32_to_bf16_bits(np.where(synth.rng("single", "x").random((M, K)) < 0.5, -1.0, 1.0)
                               .astype(np.float32))
    w = synth.f32_to_bf16_bits(synth.rng("single", "w").uniform(0.1, 4.0, K).astype(np.float32))
    q, s, _, y = run(x, w, eps=1e-30)
    xq = torch.empty((M, K), dtype=torch.uint8, device="cuda")
    xs = torch.empty((M, K // 128), dtype=torch.float32, device="cuda")
    L.fp8_quant_act(to_dev_bf16(y), xq, xs)
    assert np.array_equal(q, u8(xq)) and np.array_equal(s, xs.cpu().numpy())


def test_norm_other_stream_and_graph():
    """On a side stream, then captured with new inputs for every replay."""
    import torch
    from block_scaled_precision_fp8_amd import lib as L
    x, w, r = inputs(17, 2048, seed=3)
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        check(x, w, r)
    xd, wd, rd = to_dev_bf16(x), to_dev_bf16(w), to_dev_bf16(r)
    ro, y = torch.empty_like(rd), torch.empty_like(rd)
    q = torch.empty((17, 2048), dtype=torch.uint8, device="cuda")
    s = torch.empty((17, 16), dtype=torch.float32, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        L.fp8_add_rmsnorm_quant(xd, wd, q, s, residual=rd, residual_out=ro, y=y)
    for seed in range(4, 8):
        x, _, r = inputs(17, 2048, seed=seed)
        xd.copy_(to_dev_bf16(x))
        rd.copy_(to_dev_bf16(r))
        q.zero_()
        g.replay()
        torch.cuda.synchronize()
        rh, ry = Y.add_rmsnorm(x, w, 1e-6, r)
        rq, rs = Y.quant_rows(ry)
        assert np.array_equal(u8(q), rq) and np.array_equal(s.cpu().numpy(), rs)
        assert np.array_equal(F.bf16_decode(bf16_bits(ro)), rh)


def test_norm_feeds_block_gemm():
    """norm -> FP8 linear: the codes and scales go in unchanged."""
    import torch
    from block_scaled_precision_fp8_amd import lib as L
    from oracle import gemm as G, quant as Q
    from gpu_util import rel_fro
    M, K, N = 33, 1040, 264
    x, w, r = inputs(M, K, seed=6)
    q, s, _, _ = run(x, w, r, fmt=1)
    wq, ws = Q.quant_weight(synth.normal_bf16((N, K), 0.02, "single", "w"), 128, 128, 1)
    y = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    L.fp8_block_gemm(to_dev(q), to_dev(s), to_dev(wq), to_dev(ws), y, scale_fmt=1)
    torch.cuda.synchronize()
    assert rel_fro(F.bf16_decode(bf16_bits(y)), G.block_gemm(q, s, wq, ws, fmt=1)) <= 2e-3


def test_norm_more_rows_than_one_grid_dimension():
    """More workgroups than the grid's first dimension: every row as in a
    short call, and one past the last left alone."""
    import torch
    from block_scaled_precision_fp8_amd import lib as L
    M, K = (4 << 20) + 1001, 16
    say(f"norm M={M}")
    x = synth.device_normal_bf16((M, K), 1.0, "single", "x")
    w = synth.device_normal_bf16((K,), 1.0, "single", "w")

    def call(rows):
        n = rows.shape[0]
        q = torch.full((n + 1, K), 0xA5, dtype=torch.uint8, device="cuda")
        s = torch.full((n + 1, 1), 7.0, device="cuda")
        L.fp8_add_rmsnorm_quant(rows, w, q[:n], s[:n])
        torch.cuda.synchronize()
        assert (q[n] == 0xA5).all() and s[n] == 7.0
        return q[:n], s[:n]

    q, s = call(x)
    for lo, hi in ((0, 100), (M // 2, M // 2 + 100), ((4 << 20) - 50, (4 << 20) + 50), (M - 100, M)):
        a, b = call(x[lo:hi])
        assert torch.equal(a, q[lo:hi]) and torch.equal(b, s[lo:hi])
    rq, rs = Y.quant_rows(Y.add_rmsnorm(bf16_bits(x[M - 100:]), bf16_bits(w), 1e-6)[1])
    assert np.array_equal(u8(q[M - 100:]), rq) and np.array_equal(s[M - 100:].cpu().numpy(), rs)
