"""A decoder layer's attention half, run as a user runs it: norm and
quantization, QKV linear, rotary append, attention, output linear; prompts,
then single tokens, then a captured step."""

import numpy as np
import pytest
import torch

import attn_bounds as bounds
from block_scaled_precision_fp8_amd import lib as L
from gpu_util import bf16_bits, dev, rel_fro, say
from oracle import attn as A, formats as F, gemm as G, quant as Q

pytestmark = pytest.mark.gpu

HQ, HKV, D, H, PAGE, PAGES = 8, 2, 64, 256, 16, 40
QKV = (HQ + 2 * HKV) * D


class Layer:
    def __init__(self, rng, fmt):
        bf = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(torch.bfloat16).to(dev())
        self.fmt = fmt
        self.norm = 1.0 + 0.1 * bf(H)
        self.weights = []
        for n, k in ((QKV, H), (H, HQ * D)):
            w = bf(n, k) / k ** 0.5
            q = torch.empty(n, k, dtype=torch.uint8, device=dev())
            s = torch.empty(-(-n // 128), -(-k // 128), device=dev())
            L.fp8_quant_weight(w, q, s)
            self.weights.append((q, s))
        self.freq = torch.empty(D // 2, device=dev())
        L.rope_inv_freq(self.freq, base=10000.0, scaling=L.ROPE_BY_PARTS, factor=4.0, orig_len=64.0)
        cdt = torch.bfloat16 if fmt == L.KV_BF16 else torch.uint8
        c = lambda: torch.zeros(PAGES, HKV, PAGE, D, dtype=cdt, device=dev())
        sc = lambda: None if fmt == L.KV_BF16 else torch.zeros(
            PAGES, HKV, PAGE, dtype=torch.uint8 if fmt == L.KV_FP8_UE8M0 else torch.float32, device=dev())
        self.cache = dict(k_cache=c(), v_cache=c(), k_scale=sc(), v_scale=sc(), kv_fmt=fmt)

    def step(self, x, positions, slots, **kw):
        """(rotated queries, attention's y, the layer's output) of T tokens."""
        T = x.shape[0]
        e = lambda *s, t=torch.bfloat16: torch.empty(s, dtype=t, device=dev())
        xq, xs = e(T, H, t=torch.uint8), e(T, H // 128, t=torch.float32)
        L.fp8_add_rmsnorm_quant(x, self.norm, xq, xs)
        qkv = e(T, QKV)
        L.fp8_block_gemm(xq, xs, *self.weights[0], qkv)
        q, k, v = (t.unflatten(1, (-1, D)) for t in qkv.split([HQ * D, HKV * D, HKV * D], 1))
        L.rope_kv_append(positions, self.freq, q=q, q_out=q, k=k, v=v, slots=slots, **self.cache)
        y, out = e(T, HQ, D), e(T, H)
        L.paged_attn(q, y=y, **self.cache, **kw)
        L.fp8_linear(y.view(T, HQ * D), *self.weights[1], out)
        return q, y, out

    def values(self):
        host = lambda t: None if t is None else (F.bf16_decode(bf16_bits(t)) if t.dtype == torch.bfloat16 else
                                                 t.cpu().numpy())
        c = self.cache
        return [A.cache_values(host(c[n + "_cache"]), host(c[n + "_scale"]), self.fmt) for n in "kv"]


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=dev())


@pytest.mark.parametrize("fmt", [L.KV_FP8_FLOAT, L.KV_FP8_UE8M0, L.KV_BF16])
def test_prompts_then_tokens(fmt):
    rng = np.random.default_rng(40 + fmt)
    layer = Layer(rng, fmt)
    prompts, steps, prefix = [37, 5, 70], 3, 21
    order = rng.permutation(PAGES)
    ptable, table = order[:2], order[2:32].reshape(3, 10)
    td, pd = i32(table.tolist()), i32(ptable.tolist())
    slot = lambda t, j: int(t[j // PAGE]) * PAGE + j % PAGE
    new = lambda n: torch.from_numpy(rng.standard_normal((n, H)).astype(np.float32)).to(torch.bfloat16).to(dev())

    def check(q, y, out, lens, start):
        """y against the oracle's attention over what the cache holds, out against the oracle's linear."""
        k, v = layer.values()
        qv = F.bf16_decode(bf16_bits(q.contiguous()))
        want, spread, reach, keys = A.attention(qv, k, v, lens, table, D ** -0.5, q_start=start,
                                                prefix_table=ptable, prefix_len=prefix)
        got = F.bf16_decode(bf16_bits(y))
        room = bounds.attention(want, spread, reach, keys, D, fmt != L.KV_BF16, np.abs(v).max() * 448.0)
        assert np.all(np.abs(got - want) <= room)
        cq, cs = Q.quant_act(bf16_bits(y).reshape(-1, HQ * D))
        wq, ws = (t.cpu().numpy() for t in layer.weights[1])
        assert rel_fro(F.bf16_decode(bf16_bits(out)), G.block_gemm(cq, cs, wq, ws)) <= 2e-3

    # the shared prefix, as a sequence of its own whose table it becomes
    x = new(prefix)
    layer.step(x, i32(list(range(prefix))), torch.tensor([slot(ptable, j) for j in range(prefix)], device=dev()),
               kv_len=i32([prefix]), page_table=i32([ptable.tolist()]), q_start=i32([0, prefix]))
    # the prompts
    start = np.concatenate([[0], np.cumsum(prompts)])
    pos = [prefix + j for n in prompts for j in range(n)]
    slots = [slot(table[b], j) for b, n in enumerate(prompts) for j in range(n)]
    q, y, out = layer.step(new(sum(prompts)), i32(pos), torch.tensor(slots, device=dev()), kv_len=i32(prompts),
                           page_table=td, q_start=i32(start.tolist()), prefix_table=pd, prefix_len=prefix)
    check(q, y, out, prompts, start)
    # single tokens, the second sequence padded from the second step on
    lens = list(prompts)
    for s in range(steps):
        here = [b != 1 or s == 0 for b in range(3)]
        lens = [n + h for n, h in zip(lens, here)]
        slots = [slot(table[b], lens[b] - 1) if here[b] else -1 for b in range(3)]
        q, y, out = layer.step(new(3), i32([prefix + n - 1 for n in lens]), torch.tensor(slots, device=dev()),
                               kv_len=i32(lens), page_table=td, prefix_table=pd, prefix_len=prefix)
        check(q, y, out, lens, np.arange(4))


def test_tokens_one_by_one_or_at_once():
    """A prompt in one call, in two chunks and token by token: the same cache
    (the linears' rows do not depend on each other) and outputs within their bounds."""
    rng = np.random.default_rng(50)
    n = 33
    x = torch.from_numpy(rng.standard_normal((n, H)).astype(np.float32)).to(torch.bfloat16).to(dev())
    table = np.arange(5, 15)[None]
    results = []
    for chunks in ([n], [20, 13], [1] * n):
        layer = Layer(np.random.default_rng(51), L.KV_FP8_FLOAT)
        ys, at = [], 0
        for c in chunks:
            j = np.arange(at, at + c)
            slots = torch.from_numpy(table[0][j // PAGE] * PAGE + j % PAGE).to(dev())
            kw = dict(kv_len=i32([at + c]), page_table=i32(table.tolist()), q_start=i32([0, c]))
            _, y, _ = layer.step(x[at:at + c], i32(j.tolist()), slots, **kw)
            ys.append(y)
            at += c
        results.append((torch.cat(ys).float(), layer.values()))
    for y, (k, v) in results[1:]:
        # the QKV linears of 1, 13, 20 and 33 rows sum in other orders: bf16 steps, hence codes, may differ
        assert np.abs(k - results[0][1][0]).max() < 0.3 and rel_fro(k, results[0][1][0]) < 0.02
        assert rel_fro(y.cpu().numpy(), results[0][0].cpu().numpy()) < 0.02


def test_captured_step():
    """One step captured with its own buffers, replayed for step after step
    with eager work between, against the same steps without a graph."""
    rng = np.random.default_rng(60)
    table = np.arange(20).reshape(2, 10)
    xs = [torch.from_numpy(rng.standard_normal((2, H)).astype(np.float32)).to(torch.bfloat16).to(dev())
          for _ in range(6)]
    plans = [([s, 40 + s], [int(table[0, s // PAGE]) * PAGE + s % PAGE,
                            int(table[1, (40 + s) // PAGE]) * PAGE + (40 + s) % PAGE],
              [s + 1, 41 + s]) for s in range(6)]
    eager, graphed = (Layer(np.random.default_rng(61), L.KV_FP8_FLOAT) for _ in range(2))
    td = i32(table.tolist())
    x, pos, slots, lens = xs[0].clone(), i32([0, 0]), torch.full((2,), -1, device=dev()), i32([0, 0])
    ws = torch.empty(L.paged_attn_workspace_size(2, 2, HQ, HKV, D, 10, PAGE), dtype=torch.uint8, device=dev())
    graphed.step(x, pos, slots, kv_len=lens, page_table=td, workspace=ws)         # nothing is cached
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _, y, out = graphed.step(x, pos, slots, kv_len=lens, page_table=td, workspace=ws)
    for xv, (p, sl, ln) in zip(xs, plans):
        x.copy_(xv)
        pos.copy_(torch.tensor(p, dtype=torch.int32))
        slots.copy_(torch.tensor(sl))
        lens.copy_(torch.tensor(ln, dtype=torch.int32))
        graph.replay()
        _, ye, oe = eager.step(xv, i32(p), torch.tensor(sl, device=dev()), kv_len=i32(ln), page_table=td)
        torch.cuda.synchronize()
        assert torch.equal(y, ye) and torch.equal(out, oe)
    for a, b in zip(graphed.values(), eager.values()):
        assert np.array_equal(a, b)
    say("replayed", len(plans))
