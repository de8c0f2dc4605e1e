"""Cases, plain forms and 64-bit values of the operators between the QKV and the output linear:

* ``append``  rope_kv_append: rotary positions, keys and values into a paged FP8 or bf16 cache
* ``attn``    paged_attn: attention of new tokens over that cache, with a prefix that the batch shares

``own`` selects the library's calls; without it ``run`` computes the same in
elementary torch operations.
"""

import math

import torch

own = False

E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
FP8, UE8M0, BF16 = 0, 1, 2            # cache formats: E4M3 with fp32 or E8M0 scales, bf16


# ------------------------------------------------------------------ cases

def _append(name, T, seqs, Hq, Hkv, D, fmt, page, rot, interleaved=False, pad=0, first=0, factor=1.0,
            skip=0):
    """T new tokens of `seqs` sequences from about position `first` on; every `skip`-th is padding."""
    return {"name": name, "op": "append", "T": T, "seqs": seqs, "Hq": Hq, "Hkv": Hkv, "D": D,
            "fmt": fmt, "page": page, "rot": rot, "interleaved": interleaved, "pad": pad,
            "first": first, "factor": factor, "skip": skip}


def _attn(name, B, n, ctx, Hq, Hkv, D, fmt, page, even=False, window=0, prefix=0):
    """B sequences of up to n new tokens and up to ctx cached ones (all so many where `even`)."""
    return {"name": name, "op": "attn", "B": B, "n": n, "ctx": ctx, "Hq": Hq, "Hkv": Hkv, "D": D,
            "fmt": fmt, "page": page, "even": even, "window": window, "prefix": prefix}


def listed():
    return [
        # one decoded token
        _append("append 1", 1, 1, 32, 8, 128, FP8, 64, 128, first=700),
        # a decode batch, power-of-two scales, half of each head rotated in pairs, padded rows
        _append("append 64 ue8m0 half", 64, 64, 16, 2, 128, UE8M0, 16, 64, True, first=4000, skip=9),
        # prompts of a batch
        _append("append 8192", 8192, 5, 32, 8, 128, FP8, 64, 128),
        # bf16 cache, odd head counts, far positions with scaled angles, rows inside a wider tensor
        _append("append 1031 bf16 far", 1031, 3, 9, 3, 64, BF16, 32, 64, pad=24, first=1000000, factor=8.0),
        # one short sequence, one new token: latency
        _attn("attn 1x700", 1, 1, 700, 32, 8, 128, FP8, 16),
        # a decode batch of ragged lengths
        _attn("attn 64x8192 ragged", 64, 1, 8192, 32, 8, 128, FP8, 64),
        # one long sequence
        _attn("attn 1x131072", 1, 1, 131072, 32, 8, 128, FP8, 128),
        # as many key heads as query heads, small heads, bf16 cache, sliding window
        _attn("attn 24x5000 window bf16", 24, 1, 5000, 12, 12, 64, BF16, 32, window=1000),
        # a few drafted tokens per sequence, wide heads, power-of-two scales
        _attn("attn 9x4x2500 d256 ue8m0", 9, 4, 2500, 16, 2, 256, UE8M0, 16),
        # a chunk of two prompts behind what is cached of them
        _attn("attn 2x2048x6000", 2, 2048, 6000, 32, 8, 128, FP8, 64, even=True),
        # a batch behind a long common prompt
        _attn("attn 64x600 prefix 16384", 64, 1, 600, 32, 8, 128, FP8, 64, prefix=16384),
        # a small batch, a prefix that ends inside a page
        _attn("attn 7x333 prefix 1237", 7, 1, 333, 10, 2, 128, BF16, 16, prefix=1237),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    Hkv, D = rng.choice((1, 2, 3, 4, 8)), rng.choice((64, 128, 128, 256))
    Hq = Hkv * rng.choice((1, 2, 3, 4, 5, 7, 8, 16))
    fmt, page = rng.choice((FP8, FP8, UE8M0, BF16)), rng.choice((16, 32, 64, 128))
    if rng.random() < 0.3:
        T = _log_int(rng, 1, 8192)
        while T * (Hq + 2 * Hkv) * D > 8192 * 48 * 128:
            T = max(1, T // 2)
        seqs = _log_int(rng, 1, T)
        while seqs * 2 * page * Hkv * D > 1 << 26:                    # pages of their own
            seqs = max(1, seqs // 2)
        c = _append("", T, seqs, Hq, Hkv, D, fmt, page,
                    rng.choice((D, D, D // 2, D // 4)), rng.random() < 0.4, 8 * rng.randrange(4),
                    _log_int(rng, 1, 1000000), rng.choice((1.0, 1.0, 4.0, 32.0)),
                    rng.choice((0, 0, 3, 9)))
    else:
        while True:
            B, ctx = _log_int(rng, 1, 128), _log_int(rng, 1, 65536)
            n = rng.choice((1, 1, 1, rng.randint(2, 8), _log_int(rng, 16, 2048)))
            n = min(n, ctx)
            prefix = 0 if rng.random() < 0.6 else _log_int(rng, 1, 16384)
            if B * n * Hq * (ctx + prefix) <= 2 * 2048 * 32 * 6000 // 2 and \
                    (B * ctx + prefix) * Hkv * D * (2 if fmt == BF16 else 1) <= 64 * 8192 * 8 * 128 // 2:
                break
        window = 0 if rng.random() < 0.7 else _log_int(rng, 1, ctx + prefix)
        c = _attn("", B, n, ctx, Hq, Hkv, D, fmt, page, rng.random() < 0.3, window, prefix)
    del c["name"]
    return c


def _spread(count, lo, hi, step):
    """`count` whole numbers spread evenly over lo..hi, the first of them hi."""
    return [hi - int((hi - lo + 1) * ((i * step) % 1.0)) for i in range(count)]


def _lengths(c):
    """New tokens and cached ones (these included) of each sequence, in the cases' own order."""
    if c["even"]:
        return [c["n"]] * c["B"], [c["ctx"]] * c["B"]
    new = _spread(c["B"], 1, c["n"], 0.6180339887498949)
    return new, [max(n, l) for n, l in zip(new, _spread(c["B"], 1, c["ctx"], 0.7548776662466927))]


# ----------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(0xA77E + 7919 * int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _inv_freq(rot, factor):
    """Angles per position; scaled ones by how often they turn within 8192 positions (1 to 32 times)."""
    f = 500000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    if factor != 1.0:
        keep = ((8192.0 * f / (2.0 * math.pi) - 1.0) / 31.0).clamp(0.0, 1.0)
        f = f * (keep + (1.0 - keep) / factor)
    return f.float()


def _cache(g, pages, Hkv, page, D, fmt, part=1 << 25):
    """A cache of `pages` pages (keys or values) and its scales: normal values whose size varies by token."""
    codes = torch.empty(pages, Hkv, page, D, device="cuda", dtype=torch.bfloat16 if fmt == BF16 else torch.uint8)
    scales = None if fmt == BF16 else torch.empty(
        pages, Hkv, page, device="cuda", dtype=torch.uint8 if fmt == UE8M0 else torch.float32)
    step = max(1, part // (Hkv * page * D))
    for p in range(0, pages, step):
        m = min(step, pages - p)
        v = _randn(g, m, Hkv, page, D) * (0.3 + torch.rand((m, Hkv, page, 1), generator=g, device="cuda"))
        if fmt == BF16:
            codes[p:p + m] = v.to(torch.bfloat16)
        else:
            q, s = _codes(v, fmt)
            codes[p:p + m], scales[p:p + m] = q.view(torch.uint8), s
    return codes, scales


def _prepare_append(c, g):
    T, Hq, Hkv, D, page = c["T"], c["Hq"], c["Hkv"], c["D"], c["page"]
    H = (Hq + 2 * Hkv) * D
    wide = _randn(g, T, H + c["pad"])
    wide[:, torch.randperm(H, generator=g, device="cuda")[:max(1, H // 1000)]] *= 20.0
    wide = wide.to(torch.bfloat16)
    c["q"], c["k"], c["v"] = (t.unflatten(1, (-1, D)) for t in wide[:, :H].split([Hq * D, Hkv * D, Hkv * D], 1))
    # the sequences' new tokens stand in a row, each sequence's behind what it has cached
    seq = torch.arange(T, device="cuda") * c["seqs"] // T
    start = torch.searchsorted(seq, torch.arange(c["seqs"], device="cuda"))
    first = (c["first"] * (0.5 + torch.rand(c["seqs"], generator=g, device="cuda"))).long()
    pos = first[seq] + torch.arange(T, device="cuda") - start[seq]
    c["positions"] = pos.to(torch.int32)
    c["inv_freq"], c["mscale"] = _inv_freq(c["rot"], c["factor"]), 0.1 * math.log(c["factor"]) + 1.0
    # every sequence's part of the cache begins on a page of its own; the last page is nobody's
    per = -(-(-(-T // c["seqs"]) + page) // page)
    c["pages"] = per * c["seqs"]
    order = torch.randperm(c["pages"], generator=g, device="cuda")
    at = first[seq] % page + torch.arange(T, device="cuda") - start[seq]
    slots = order[seq * per + at // page] * page + at % page
    if c["skip"]:
        slots[c["skip"] - 1::c["skip"]] = -1
    c["slots"] = slots
    c["kc"], c["ks"] = _cache(g, c["pages"] + 1, Hkv, page, D, c["fmt"])
    c["vc"], c["vs"] = _cache(g, c["pages"] + 1, Hkv, page, D, c["fmt"])
    c["qo"] = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda")
    return c


def _prepare_attn(c, g):
    page, D = c["page"], c["D"]
    new, cached = _lengths(c)
    turn = torch.randperm(c["B"], generator=g, device="cuda").tolist()
    new, cached = [new[i] for i in turn], [cached[i] for i in turn]
    T = sum(new)
    own_pages = [-(-l // page) for l in cached]
    pre = -(-c["prefix"] // page)
    pages = sum(own_pages) + pre
    c["kc"], c["ks"] = _cache(g, pages, c["Hkv"], page, D, c["fmt"])
    c["vc"], c["vs"] = _cache(g, pages, c["Hkv"], page, D, c["fmt"])
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    c["prefix_table"] = order[:pre].contiguous() if pre else None
    table = torch.full((c["B"], -(-c["ctx"] // page)), -1, dtype=torch.int32)
    at, order_h = pre, order.cpu()
    for b, m in enumerate(own_pages):
        table[b, :m] = order_h[at:at + m]
        at += m
    c["table"] = table.cuda()
    c["kv_len"] = torch.tensor(cached, dtype=torch.int32, device="cuda")
    c["new"] = torch.tensor(new, device="cuda")
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    c["q_start"] = None if c["n"] == 1 else torch.tensor(starts, dtype=torch.int32, device="cuda")
    c["first"] = torch.tensor(starts[:-1], device="cuda")
    c["q"] = (1.5 * _randn(g, T, c["Hq"], D)).to(torch.bfloat16)
    c["y"] = torch.empty(T, c["Hq"], D, dtype=torch.bfloat16, device="cuda")
    return c


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    return _prepare_append(c, g) if c["op"] == "append" else _prepare_attn(c, g)


# ------------------------------------------------------------ plain forms

def _scale_values(s):
    """Stored scales (fp32, or E8M0 bytes) as fp32 multipliers."""
    return s if s.dtype == torch.float32 else torch.exp2(s.float() - 127.0)


def _codes(y, fmt):
    """E4M3 codes and stored scales of fp32 rows, a scale per row."""
    amax = y.abs().amax(-1)
    if fmt == UE8M0:
        e = torch.ceil(torch.log2(amax.double() / 448.0)).clamp(-127, 127)
        stored = torch.where(amax == 0, 127.0, e + 127.0).to(torch.uint8)
    else:
        # a tensor divides; a number would multiply by its rounded reciprocal
        stored = torch.where(amax == 0, 1.0, amax / torch.full_like(amax, 448.0))
    return (y / _scale_values(stored)[..., None]).clamp(-448.0, 448.0).to(E4M3), stored


def _rotate(x, cos, sin, rot, interleaved):
    cos, sin = cos[:, None], sin[:, None]
    r = x[..., :rot]
    a, b = (r[..., ::2], r[..., 1::2]) if interleaved else (r[..., :rot // 2], r[..., rot // 2:])
    a, b = a * cos - b * sin, b * cos + a * sin
    r = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((r, x[..., rot:]), -1)


def _append_plain(c):
    # 64 bits: far positions' angles, group maxima next to a power of two
    angle = c["positions"].double()[:, None] * c["inv_freq"].double()
    cos, sin = torch.cos(angle) * c["mscale"], torch.sin(angle) * c["mscale"]
    turn = (c["rot"], c["interleaved"])
    out = {"q": _rotate(c["q"].float(), cos.float(), sin.float(), *turn).to(torch.bfloat16)}
    k = _rotate(c["k"].double(), cos, sin, *turn).float()
    slots = torch.where(c["slots"] < 0, c["pages"] * c["page"], c["slots"])
    page, at = slots // c["page"], slots % c["page"]
    for name, x in (("k", k), ("v", c["v"].float())):
        cache, scales = c[name + "c"], c[name + "s"]
        if c["fmt"] == BF16:
            cache[page, :, at] = x.to(torch.bfloat16)
        else:
            q, s = _codes(x, c["fmt"])
            cache[page, :, at], scales[page, :, at] = q.view(torch.uint8), s
    return out | _written(c)


def _written(c):
    """The caches but for the last page, which no sequence has."""
    n, out = c["pages"], {}
    for name in ("k", "v"):
        cache, scales = c[name + "c"][:n], c[name + "s"]
        out[name] = cache if c["fmt"] == BF16 else cache.view(E4M3)
        if scales is not None:
            out[name + " scales"] = scales[:n].view(E8M0) if c["fmt"] == UE8M0 else scales[:n]
    return out


def _rows(c, cache, scales, table, length):
    """(.., Hkv, keys, D) fp32 of the pages of a table, zeros behind `length` keys."""
    at = table.clamp_min(0).long()
    x = cache[at] if c["fmt"] == BF16 else cache[at].view(E4M3)
    x = x.float()
    if scales is not None:
        x = x * _scale_values(scales[at])[..., None]
    x = x.transpose(-4, -3).flatten(-3, -2)
    there = torch.arange(x.shape[-2], device="cuda") < length[..., None]
    return torch.where(there[..., None, :, None], x, 0.0), there


def _attn_plain(c):
    B, n, Hq, Hkv, D = c["B"], c["n"], c["Hq"], c["Hkv"], c["D"]
    G, P, T = Hq // Hkv, c["prefix"], c["q"].shape[0]
    # rows of a sequence's tokens, as many for each; those that it lacks repeat its last one
    i = torch.minimum(torch.arange(n, device="cuda"), c["new"][:, None] - 1)
    token = c["first"][:, None] + i                                            # (B, n)
    pos = (P + c["kv_len"] - c["new"])[:, None] + i                            # (B, n)
    low = pos - c["window"] if c["window"] else torch.full_like(pos, -1)
    q = c["q"][token].float().view(B, n, Hkv, G, D).permute(0, 2, 1, 3, 4)     # (B, Hkv, n, G, D)
    q = q.reshape(B, Hkv, n * G, D) * D ** -0.5
    k, there = _rows(c, c["kc"], c["ks"], c["table"], c["kv_len"])
    v, _ = _rows(c, c["vc"], c["vs"], c["table"], c["kv_len"])

    def seen(s, key, there):
        ok = there[:, None] & (key <= pos[..., None]) & (key > low[..., None])  # (B, n, keys)
        s = s.view(B, Hkv, n, G, -1)
        return s.masked_fill_(~ok[:, None, :, None], float("-inf")).view(B, Hkv, n * G, -1)

    s = seen(q @ k.transpose(2, 3).contiguous(), P + torch.arange(k.shape[2], device="cuda"), there)
    top = s.amax(-1, keepdim=True)
    if P:
        whole = torch.tensor(P, device="cuda")
        pk, pthere = _rows(c, c["kc"], c["ks"], c["prefix_table"], whole)
        pv, _ = _rows(c, c["vc"], c["vs"], c["prefix_table"], whole)
        flat = q.transpose(0, 1).reshape(Hkv, B * n * G, D)
        ps = (flat @ pk.transpose(1, 2).contiguous()).view(Hkv, B, n * G, -1).transpose(0, 1).contiguous()
        ps = seen(ps, torch.arange(pk.shape[1], device="cuda"), pthere.expand(B, -1))
        top = torch.maximum(top, ps.amax(-1, keepdim=True))
    top = torch.where(top == float("-inf"), 0.0, top)
    e = s.sub_(top).exp_()
    total, y = e.sum(-1, keepdim=True), e @ v
    if P:
        e = ps.sub_(top).exp_()
        total = total + e.sum(-1, keepdim=True)
        flat = e.transpose(0, 1).reshape(Hkv, B * n * G, -1) @ pv
        y = y + flat.view(Hkv, B, n * G, D).transpose(0, 1)
    y = torch.where(total == 0, 0.0, y / torch.where(total == 0, 1.0, total))
    y = y.view(B, Hkv, n, G, D).permute(0, 2, 1, 3, 4).reshape(B * n, Hq, D).to(torch.bfloat16)
    out = c["y"]
    out[token.view(-1)] = y
    return out


def _own(c):
    from block_scaled_precision_fp8_amd import lib as L
    if c["op"] == "append":
        L.rope_kv_append(c["positions"], c["inv_freq"], q=c["q"], q_out=c["qo"], k=c["k"], v=c["v"],
                         slots=c["slots"], k_cache=c["kc"], v_cache=c["vc"], k_scale=c["ks"],
                         v_scale=c["vs"], kv_fmt=c["fmt"], interleaved=c["interleaved"],
                         mscale=c["mscale"])
        return {"q": c["qo"]} | _written(c)
    L.paged_attn(c["q"], c["kc"], c["vc"], c["kv_len"], c["table"], c["y"], k_scale=c["ks"],
                 v_scale=c["vs"], kv_fmt=c["fmt"], q_start=c["q_start"],
                 prefix_table=c["prefix_table"], prefix_len=c["prefix"], window=c["window"])
    return c["y"]


def run(state):
    if own:
        return _own(state)
    return _append_plain(state) if state["op"] == "append" else _attn_plain(state)


# ------------------------------------------------------------------- work

def work(case):
    c = case
    Hq, Hkv, D, fmt = c["Hq"], c["Hkv"], c["D"], c["fmt"]
    row = 2 * D if fmt == BF16 else D + (4 if fmt == FP8 else 1)      # a cached key or value
    if c["op"] == "append":
        T = c["T"]
        kept = T - T // c["skip"] if c["skip"] else T
        return {"bytes": T * Hq * D * 4 + kept * Hkv * 2 * (2 * D + row) + T * 12 + 2 * c["rot"],
                "flops": 3 * T * (Hq + Hkv) * c["rot"]}
    new, cached = _lengths(c)
    read, pairs, P, W = 0, 0, c["prefix"], c["window"]
    for n, l in zip(new, cached):
        first = P + l - n                                             # the first new token's position
        low = max(0, first - W + 1) if W else 0
        read += P + l - max(P, low)
        last = first + n
        if W and last > W:
            full = max(0, W - 1 - first)                              # tokens that see all before them
            full = min(full, n)
            pairs += full * first + full * (full + 1) // 2 + (n - full) * W
        else:
            pairs += n * first + n * (n + 1) // 2
    if P:
        low = min(max(0, P + l - n - W + 1) if W else 0 for n, l in zip(new, cached))
        read += max(0, P - low)
    return {"bytes": read * Hkv * 2 * row + sum(new) * Hq * D * 4, "flops": 4 * pairs * Hq * D}


# ------------------------------------------------- 64-bit values, by itself

def _exact_scale(stored):
    return stored.double() if stored.dtype == torch.float32 else 2.0 ** (stored.double() - 127.0)


def _exact_round(v, bits, low):
    """Round to `bits` significant bits, half to even; quantum at least 2^low."""
    e = torch.frexp(v)[1].double() - 1.0
    q = torch.exp2(torch.clamp(e - (bits - 1), min=low))
    return torch.where(v == 0, v, torch.round(v / q) * q)


def _exact_append(c):
    r, out = c["rot"], {}
    turns = c["positions"].double()[:, None] * c["inv_freq"].double()[None, :]
    z = torch.polar(torch.full_like(turns, c["mscale"]), turns)[:, None, :]

    def rotated(x):
        x = x.double().clone()
        if c["interleaved"]:
            w = torch.complex(x[..., 0:r:2], x[..., 1:r:2]) * z
            x[..., 0:r:2], x[..., 1:r:2] = w.real, w.imag
        else:
            h = r // 2
            w = torch.complex(x[..., :h], x[..., h:r]) * z
            x[..., :h], x[..., h:r] = w.real, w.imag
        return x

    out["q"] = rotated(c["q"])
    keep = torch.nonzero(c["slots"] >= 0)[:, 0]
    for name, x in (("k", rotated(c["k"])), ("v", c["v"].double())):
        cache, scales = c[name + "c"], c[name + "s"]
        if c["fmt"] == BF16:
            old, news, olds = cache.double(), None, None
        else:
            old, olds = cache.view(E4M3).double(), _exact_scale(scales)
            a = x.abs().max(dim=2)[0]
            if c["fmt"] == UE8M0:
                m, e = torch.frexp(a / 448.0)              # m in [1/2, 1): exact powers give 1/2
                news = torch.exp2(torch.where(m == 0.5, e - 1, e).double().clamp(-127, 127))
            else:
                news = a / 448.0
            news = torch.where(a == 0, torch.ones_like(a), news)
            x = _exact_round(x / news[:, :, None], 4, -9).clamp(-448.0, 448.0)
        old = old.transpose(1, 2).reshape(-1, c["Hkv"], c["D"])
        old[c["slots"][keep]] = x[keep]
        old = old.view(-1, c["page"], c["Hkv"], c["D"]).transpose(1, 2)
        out[name] = old[:c["pages"]]
        if news is not None:
            olds = olds.transpose(1, 2).reshape(-1, c["Hkv"])
            olds[c["slots"][keep]] = news[keep]
            out[name + " scales"] = olds.view(-1, c["page"], c["Hkv"]).transpose(1, 2)[:c["pages"]]
    return out


def _exact_attn(c):
    Hq, Hkv, D, P, W, page = c["Hq"], c["Hkv"], c["D"], c["prefix"], c["window"], c["page"]
    G = Hq // Hkv
    y = torch.zeros(c["q"].shape, dtype=torch.float64, device="cuda")

    def values(cache, scales, at, h):
        x = cache[at, h]
        x = x.double() if c["fmt"] == BF16 else x.view(E4M3).double() * _exact_scale(scales[at, h])[..., None]
        return x.reshape(-1, D)

    first, new, cached = c["first"].tolist(), c["new"].tolist(), c["kv_len"].tolist()
    for h in range(Hkv):
        if P:
            at = c["prefix_table"].long()
            pk, pv = values(c["kc"], c["ks"], at, h)[:P], values(c["vc"], c["vs"], at, h)[:P]
        for f, n, l, row in zip(first, new, cached, c["table"]):
            at = row[:-(-l // page)].long()
            k, v = values(c["kc"], c["ks"], at, h)[:l], values(c["vc"], c["vs"], at, h)[:l]
            if P:
                k, v = torch.cat([pk, k]), torch.cat([pv, v])
            q = c["q"][f:f + n, h * G:(h + 1) * G].double().reshape(n * G, D)
            s = q @ k.t() / math.sqrt(D)
            back = (P + l - n) + torch.arange(n, device="cuda")[:, None] - torch.arange(P + l, device="cuda")
            hidden = back < 0
            if W:
                hidden |= back >= W
            s.view(n, G, -1).masked_fill_(hidden[:, None], float("-inf"))
            y[f:f + n, h * G:(h + 1) * G] = (torch.softmax(s, 1) @ v).view(n, G, D)
    return y


def exact(case, seed):
    c = prepare(case, seed)
    return _exact_append(c) if c["op"] == "append" else _exact_attn(c)
