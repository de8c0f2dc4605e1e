"""Cases, plain forms and 64-bit values of the operators around the linears:

* ``norm``   fp8_add_rmsnorm_quant: residual addition, RMS norm, E4M3 codes with group scales
* ``route``  moe_route_topk: router scores to the top-k experts and their weights
* ``moe``    fp8_moe_decode / fp8_fp4_moe_decode: a whole MoE layer for a few tokens

``own`` selects the library's calls; without it ``run`` computes the same in
elementary torch operations.
"""

import torch

own = False

E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases

def _norm(name, M, K, fmt, group, residual=True, y=False, pad=0, static=False):
    return {"name": name, "op": "norm", "M": M, "K": K, "fmt": fmt, "group": group,
            "residual": residual, "y": y, "pad": pad, "static": static}


def _route(name, T, E, k, score, bias, groups, kept, bf16, masked=False):
    return {"name": name, "op": "route", "T": T, "E": E, "k": k, "score": score, "bias": bias,
            "groups": groups, "kept": kept, "bf16": bf16, "masked": masked}


def _moe(name, T, k, H, I, E, routed, fmt, w4, addend):
    return {"name": name, "op": "moe", "T": T, "k": k, "H": H, "I": I, "E": E, "routed": routed,
            "fmt": fmt, "w4": w4, "addend": addend}


def listed():
    return [
        # one token before its router and experts: the bf16 row feeds the router
        _norm("norm 1x7168", 1, 7168, 0, 128, y=True),
        # a decode batch, power-of-two scales
        _norm("norm 64x4096 ue8m0", 64, 4096, 1, 128),
        # a prompt
        _norm("norm 8192x4096", 8192, 4096, 0, 128),
        # (32, 32) weight blocks, ragged sizes, rows inside a wider tensor, first layer (no residual)
        _norm("norm 1031x5136 g32", 1031, 5136, 0, 32, residual=False, pad=24),
        # one token over 256 experts, sigmoid scores, correction bias, 4 of 8 expert groups
        _route("route 1x256 groups", 1, 256, 8, 1, True, 8, 4, False),
        # a prompt through the same router
        _route("route 4096x256 groups", 4096, 256, 8, 1, True, 8, 4, False),
        # softmax router in bf16, odd counts, some experts masked off
        _route("route 333x60 softmax", 333, 60, 4, 0, False, 1, 1, True, masked=True),
        # a single decoded token, 256 experts of 7168 -> 2 x 2048 -> 7168, top 8
        _moe("moe 1 of 256", 1, 8, 7168, 2048, 256, 256, 0, False, False),
        # a small decode batch through all 256 experts, power-of-two scales
        _moe("moe 16 of 256 ue8m0", 16, 8, 7168, 2048, 256, 256, 1, False, False),
        # one of 8 ranks: 32 of the 256 experts are here, the other slots skipped, shared expert added
        _moe("moe 64 rank of 8", 64, 8, 7168, 2048, 32, 256, 1, False, True),
        # few large experts in MXFP4, odd token count
        _moe("moe 33 of 8 fp4", 33, 2, 4096, 14336, 8, 8, 1, True, False),
        # many small experts, odd sizes
        _moe("moe 5 of 64 small", 5, 6, 2064, 1408, 64, 64, 0, False, True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(("norm", "route", "moe"))
    if op == "norm":
        while True:
            M, K = _log_int(rng, 1, 8192), 16 * _log_int(rng, 1, 1024)
            if M * K <= 8192 * 4096:
                break
        static = rng.random() < 0.2
        group = 128 if static or rng.random() < 0.6 else 32
        c = _norm("", M, K, rng.randrange(2), group, rng.random() < 0.7, rng.random() < 0.4,
                  8 * rng.randrange(4), static)
    elif op == "route":
        groups = rng.choice((1, 1, 2, 4, 8))
        E = groups * _log_int(rng, 4, 512 // groups)
        k = rng.randint(2, min(8, E))
        T = _log_int(rng, 1, 4096)
        if T * E > 4096 * 256:
            T = max(1, 4096 * 256 // E)
        score = rng.randrange(2)
        c = _route("", T, E, k, score, rng.random() < 0.5, groups,
                   rng.randint(1, groups), rng.random() < 0.5, rng.random() < 0.3)
    else:
        w4 = rng.random() < 0.4
        step = 32 if w4 else 16
        while True:
            H, I = step * _log_int(rng, 8, 7168 // step), 128 * _log_int(rng, 1, 64)
            E, T = _log_int(rng, 2, 128), _log_int(rng, 1, 128)
            if E * 3 * H * I <= 1 << 31:
                break
        routed = E * rng.choice((1, 1, 1, 2, 4))
        k = rng.randint(1, min(8, routed))
        c = _moe("", T, k, H, I, E, routed, rng.randrange(2), w4, rng.random() < 0.5)
    del c["name"]
    return c


# ----------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(0x5EED + 7919 * int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _acts(g, M, K):
    """N(0, 1) rows with 0.1% of the channels 50 times as large."""
    x = _randn(g, M, K)
    n = max(1, round(0.001 * K))
    x[:, torch.randperm(K, generator=g, device="cuda")[:n]] *= 50.0
    return x


def _fp8_weight(g, E, N, K, fmt):
    w = torch.empty(E, N, K, dtype=torch.uint8, device="cuda")
    for e in range(E):
        w[e] = (_randn(g, N, K) * 112.0).clamp_(-448.0, 448.0).to(E4M3).view(torch.uint8)
    s = torch.rand((E, -(-N // 128), -(-K // 128)), generator=g, device="cuda")
    if fmt:
        return w, (114 + 2 * s).to(torch.uint8)
    return w, (0.8 + 0.4 * s) * (0.08 / 448.0)


def _fp4_weight(g, E, N, K):
    w = torch.empty(E, N, K // 2, dtype=torch.uint8, device="cuda")
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    for e in range(E):
        v = _randn(g, N, K) * 2.0
        c = torch.bucketize(v.abs(), edges).to(torch.uint8) + 8 * (v < 0).to(torch.uint8)
        w[e] = c[:, ::2] + 16 * c[:, 1::2]
    s = torch.rand((E, N, K // 32), generator=g, device="cuda")
    return w, (119 + 2 * s).to(torch.uint8)


def _topk_in(g, T, k, E, routed):
    """Distinct random experts of `routed` for each token; those of the
    first `E` are here (one of them at least), the others are marked -1."""
    z = _randn(g, T, routed)
    z[0, torch.randint(E, (1,), generator=g, device="cuda")] = 9.0
    v, ids = torch.topk(z, k, dim=1)
    wt = torch.softmax(v, 1)
    return torch.where(ids < E, ids, -1).to(torch.int32), wt.contiguous()


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    if c["op"] == "norm":
        M, K, ld = c["M"], c["K"], c["K"] + c["pad"]
        wide = torch.zeros(M, ld, dtype=torch.bfloat16, device="cuda")
        wide[:, :K] = _acts(g, M, K).to(torch.bfloat16)
        c["x"] = wide[:, :K]
        c["r"] = (3.0 * _randn(g, M, K)).to(torch.bfloat16) if c["residual"] else None
        c["w"] = (1.0 + 0.2 * _randn(g, K)).to(torch.bfloat16)
        c["eps"] = 1e-6
        sdt = torch.uint8 if c["fmt"] else torch.float32
        c["scale"] = None
        if c["static"]:
            c["scale"] = torch.tensor([123], dtype=sdt, device="cuda") if c["fmt"] else \
                torch.tensor([0.0437], dtype=sdt, device="cuda")
        c["xq"] = torch.empty(M, K, dtype=torch.uint8, device="cuda")
        c["xs"] = torch.empty(M, -(-K // c["group"]), dtype=sdt, device="cuda")
        c["h"] = torch.empty(M, K, dtype=torch.bfloat16, device="cuda") if c["residual"] else None
        c["yb"] = torch.empty(M, K, dtype=torch.bfloat16, device="cuda") if c["y"] else None
    elif c["op"] == "route":
        T, E = c["T"], c["E"]
        z = 1.5 * _randn(g, T, E)
        if c["masked"]:
            z[:, torch.randperm(E, generator=g, device="cuda")[:E // 4]] = float("-inf")
            if T > 2:
                z[T // 2] = float("-inf")
        c["logits"] = z.to(torch.bfloat16) if c["bf16"] else z
        c["b"] = 0.1 * _randn(g, E) if c["bias"] else None
        c["ids"] = torch.empty(T, c["k"], dtype=torch.int32, device="cuda")
        c["wt"] = torch.empty(T, c["k"], dtype=torch.float32, device="cuda")
    else:
        T, H, I, E = c["T"], c["H"], c["I"], c["E"]
        xq, xs = _codes(_acts(g, T, H), 128, c["fmt"], None)
        c["xq"], c["xs"] = xq.view(torch.uint8), xs
        if c["w4"]:
            c["w13"], c["s13"] = _fp4_weight(g, E, 2 * I, H)
            c["w2"], c["s2"] = _fp4_weight(g, E, H, I)
        else:
            c["w13"], c["s13"] = _fp8_weight(g, E, 2 * I, H, c["fmt"])
            c["w2"], c["s2"] = _fp8_weight(g, E, H, I, c["fmt"])
        c["ids"], c["wt"] = _topk_in(g, T, c["k"], E, c["routed"])
        c["add"] = _randn(g, T, H).to(torch.bfloat16) if c["addend"] else None
        c["yb"] = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
        if c["w4"]:
            c["table"] = _byte_table()
    return c


# ------------------------------------------------------------ plain forms

def _scale_values(s):
    """Stored scales (fp32, or E8M0 bytes) as fp32 multipliers."""
    return s if s.dtype == torch.float32 else torch.exp2(s.float() - 127.0)


def _codes(y, group, fmt, static):
    """E4M3 codes and stored scales of fp32 rows in groups of `group`."""
    M, K = y.shape
    G = -(-K // group)
    if static is None:
        yp = torch.nn.functional.pad(y, (0, G * group - K)).view(M, G, group)
        amax = yp.abs().amax(-1)
        if fmt:
            e = torch.ceil(torch.log2(amax.double() / 448.0)).clamp(-127, 127)
            stored = torch.where(amax == 0, 127.0, e + 127.0).to(torch.uint8)
        else:
            stored = torch.where(amax == 0, 1.0, amax / 448.0)
    else:
        stored = static.expand(M, G).contiguous()
    s = _scale_values(stored).repeat_interleave(group, 1)[:, :K]
    return (y / s).clamp(-448.0, 448.0).to(E4M3), stored


def _norm_plain(c):
    x = c["x"].float()
    out = {}
    if c["r"] is not None:
        h = (x + c["r"].float()).to(torch.bfloat16)
        out["residual"] = h
    else:
        h = c["x"]
    # 64 bits: group maxima next to a power of two decide a whole scale
    h = h.double()
    rs = 1.0 / torch.sqrt((h * h).mean(1, keepdim=True) + c["eps"])
    y = (h * c["w"].double() * rs).float()
    q, s = _codes(y, c["group"], c["fmt"], c["scale"])
    out["codes"], out["scales"] = q, s.view(E8M0) if c["fmt"] else s
    if c["y"]:
        out["y"] = y.to(torch.bfloat16)
    return out


def _route_plain(c):
    l = c["logits"].double()
    T, E, k = c["T"], c["E"], c["k"]
    off = torch.isnan(l) | (l == float("-inf"))
    l = torch.where(off, float("-inf"), l)
    if c["score"]:
        s = 1.0 / (1.0 + torch.exp(-l))
    else:
        top = l.amax(1, keepdim=True)
        p = torch.where(off, 0.0, torch.exp(l - torch.where(torch.isinf(top), 0.0, top)))
        s = p / p.sum(1, keepdim=True).clamp_min(1e-300)
    plain = c["b"] is None and c["groups"] == 1
    key = l if plain else s + (c["b"].double() if c["b"] is not None else 0.0)
    key = torch.where(off, float("-inf"), key)
    if c["groups"] > 1:
        kg = key.view(T, c["groups"], -1)
        two = torch.sort(kg, dim=2, descending=True)[0][:, :, :2]
        gs = torch.where(torch.isinf(two), 0.0, two).sum(2)
        gs = torch.where(torch.isinf(two[:, :, 0]), float("-inf"), gs)
        order = torch.sort(gs, dim=1, descending=True, stable=True)[1]
        keep = torch.zeros_like(gs).scatter_(1, order[:, :c["kept"]], 1.0) > 0
        key = torch.where(keep[:, :, None], kg, float("-inf")).view(T, E)
    best, ids = torch.sort(key, dim=1, descending=True, stable=True)
    best, ids = best[:, :k], ids[:, :k]
    none = best == float("-inf")
    w = torch.where(none, 0.0, torch.gather(s, 1, ids))
    total = w.sum(1, keepdim=True)
    w = torch.where(total == 0, 0.0, w / torch.where(total == 0, 1.0, total)) * 2.5
    return {"ids": torch.where(none, -1, ids).to(torch.int32), "weights": w.float()}


def _byte_table():
    """The two E2M1 values of every byte, the low nibble first."""
    v = torch.tensor(E2M1 + tuple(-x for x in E2M1), device="cuda")
    b = torch.arange(256, device="cuda")
    return torch.stack([v[b & 15], v[b >> 4]], 1)


def _dense_fp8(w, s):
    """(B, N, K) codes and 128 x 128 block scales to fp32."""
    N, K = w.shape[-2:]
    s = _scale_values(s).repeat_interleave(128, 1)[:, :N]
    w = w.view(E4M3).float()
    if K % 128 == 0:
        return w.view(-1, N, K // 128, 128).mul_(s[..., None]).view(-1, N, K)
    return w.mul_(s.repeat_interleave(128, 2)[:, :, :K])


def _dense_fp4(w, s, table):
    B, N, K = w.shape[0], w.shape[1], 2 * w.shape[2]
    v = table[w.reshape(-1).int()].view(B, N, K // 32, 32)
    return v.mul_(_scale_values(s)[..., None]).view(B, N, K)


def _moe_plain(c):
    T, k, H, I, E = c["T"], c["k"], c["H"], c["I"], c["E"]
    xs = _scale_values(c["xs"]).repeat_interleave(128, 1)[:, :H]
    x = c["xq"].view(E4M3).float() * xs
    here = c["ids"] >= 0
    wt = torch.where(here, c["wt"], 0.0)
    dense = (lambda w, s: _dense_fp4(w, s, c["table"])) if c["w4"] else _dense_fp8
    # the slots' own experts, or all experts where that is fewer
    few = T * k <= E
    pick = (lambda w: w[c["ids"].clamp_min(0).reshape(-1)]) if few else (lambda w: w)
    w13 = dense(pick(c["w13"]), pick(c["s13"]))
    if few:
        gu = torch.bmm(w13, x.repeat_interleave(k, 0)[:, :, None])[:, :, 0]
    else:
        gu = (x @ w13.view(E * 2 * I, H).t()).view(T, E, 2 * I).transpose(0, 1).reshape(E * T, 2 * I)
    del w13
    g, u = gu[:, :I], gu[:, I:]
    h = (g / (1.0 + torch.exp(-g)) * u).to(torch.bfloat16).float()
    hq, hs = _codes(h, 128, c["fmt"], None)
    h = hq.float() * _scale_values(hs).repeat_interleave(128, 1)
    w2 = dense(pick(c["w2"]), pick(c["s2"]))
    if few:
        y = (torch.bmm(w2, h[:, :, None]).view(T, k, H) * wt[:, :, None]).sum(1)
    else:
        slot = (c["ids"][:, :, None] == torch.arange(E, device="cuda")).float()
        mix = (slot * wt[:, :, None]).sum(1)                            # (T, E)
        d = torch.bmm(h.view(E, T, I), w2.transpose(1, 2))
        y = (d * mix.t()[:, :, None]).sum(0)
    if c["add"] is not None:
        y = y + c["add"].float()
    return y.to(torch.bfloat16)


def _own(c):
    from block_scaled_precision_fp8_amd import lib as L
    if c["op"] == "norm":
        L.fp8_add_rmsnorm_quant(
            c["x"], c["w"], c["xq"], c["xs"], residual=c["r"], residual_out=c["h"], y=c["yb"],
            eps=c["eps"], group_k=c["group"],
            act_scheme=L.ACT_STATIC if c["static"] else L.ACT_DYNAMIC, scale_fmt=c["fmt"],
            act_scale=c["scale"])
        out = {"codes": c["xq"].view(E4M3), "scales": c["xs"].view(E8M0) if c["fmt"] else c["xs"]}
        if c["residual"]:
            out["residual"] = c["h"]
        if c["y"]:
            out["y"] = c["yb"]
        return out
    if c["op"] == "route":
        L.moe_route_topk(c["logits"], c["ids"], c["wt"], bias=c["b"],
                         score=L.SCORE_SIGMOID if c["score"] else L.SCORE_SOFTMAX,
                         renorm=True, scale=2.5, n_group=c["groups"], topk_group=c["kept"])
        return {"ids": c["ids"], "weights": c["wt"]}
    layer = L.fp8_fp4_moe_decode if c["w4"] else L.fp8_moe_decode
    layer(c["xq"], c["xs"], c["ids"], c["wt"], c["w13"], c["s13"], c["w2"], c["s2"], c["yb"],
          addend=c["add"], scale_fmt=c["fmt"])
    return c["yb"]


def run(state):
    if own:
        return _own(state)
    return {"norm": _norm_plain, "route": _route_plain, "moe": _moe_plain}[state["op"]](state)


# ------------------------------------------------------------------- work

def work(case):
    c = case
    if c["op"] == "norm":
        M, K = c["M"], c["K"]
        G = -(-K // c["group"])
        per = 2 + (4 if c["residual"] else 0) + (2 if c["y"] else 0) + 1
        return {"bytes": M * K * per + 2 * K + M * G * (1 if c["fmt"] else 4), "flops": 8 * M * K}
    if c["op"] == "route":
        T, E = c["T"], c["E"]
        return {"bytes": T * E * (2 if c["bf16"] else 4) + 8 * T * c["k"] + (4 * E if c["bias"] else 0),
                "flops": 8 * T * E}
    T, k, H, I, E = c["T"], c["k"], c["H"], c["I"], c["E"]
    used = E * (1.0 - (1.0 - k / c["routed"]) ** T)       # distinct experts here, expected
    rows = T * k * E / c["routed"]
    if c["w4"]:
        weight = 3 * H * I * (0.5 + 1 / 32)
    else:
        weight = 3 * H * I * (1 + (1 if c["fmt"] else 4) / 16384)
    return {"bytes": used * weight + T * H * (3 + (2 if c["addend"] else 0)) + 8 * T * k,
            "flops": 6 * rows * H * I}


# ------------------------------------------------- 64-bit values, by itself

def _exact_scale(stored):
    return stored.double() if stored.dtype == torch.float32 else 2.0 ** (stored.double() - 127.0)


def _exact_round(v, bits, low):
    """Round to `bits` significant bits, half to even; quantum at least 2^low."""
    e = torch.frexp(v)[1].double() - 1.0
    q = torch.exp2(torch.clamp(e - (bits - 1), min=low))
    return torch.where(v == 0, v, torch.round(v / q) * q)


def _exact_quant(y, group, fmt, static):
    M, K = y.shape
    codes, scales = torch.empty_like(y), []
    for k0 in range(0, K, group):
        v = y[:, k0:k0 + group]
        if static is not None:
            s = _exact_scale(static).expand(M)
        else:
            a = v.abs().max(dim=1)[0]
            if fmt:
                m, e = torch.frexp(a / 448.0)             # m in [1/2, 1): exact powers give 1/2
                s = torch.exp2(torch.where(m == 0.5, e - 1, e).double().clamp(-127, 127))
            else:
                s = a / 448.0
            s = torch.where(a == 0, torch.ones_like(a), s)
        codes[:, k0:k0 + group] = _exact_round(v / s[:, None], 4, -9).clamp(-448.0, 448.0)
        scales.append(s)
    return codes, torch.stack(scales, 1)


def _exact_norm(c):
    h = c["x"].double()
    out = {}
    if c["residual"]:
        h = _exact_round(h + c["r"].double(), 8, -133)
        out["residual"] = h
    rs = (h.square().sum(1) / c["K"] + c["eps"]) ** -0.5
    y = h * c["w"].double()[None] * rs[:, None]
    out["codes"], out["scales"] = _exact_quant(y, c["group"], c["fmt"], c["scale"])
    if c["y"]:
        out["y"] = y
    return out


def _exact_route(c):
    T, E, k, n = c["T"], c["E"], c["k"], c["groups"]
    l = c["logits"].double()
    w = torch.zeros(T, k, dtype=torch.float64, device=l.device)
    dead = ~(l > float("-inf"))
    if c["score"]:
        s = torch.sigmoid(l)
    else:
        s = torch.softmax(torch.where(dead, -1e300, l), 1)
    s = torch.where(dead, 0.0, s)
    key = l if c["b"] is None and n == 1 else s if c["b"] is None else s + c["b"].double()
    key = torch.where(dead, -torch.inf, key)
    if n > 1:
        v = key.view(T, n, E // n).topk(2, dim=2)[0]
        v = v[..., 0] + torch.where(v[..., 1] == -torch.inf, 0.0, v[..., 1])
        cut = v.topk(c["kept"], dim=1)[0][:, -1:]
        key = torch.where((v >= cut).repeat_interleave(E // n, 1), key, -torch.inf)
    for j in range(k):
        top, at = key.max(dim=1)
        w[:, j] = torch.where(top == -torch.inf, 0.0, s.gather(1, at[:, None])[:, 0])
        key.scatter_(1, at[:, None], -torch.inf)
    return {"ids": None, "weights": 2.5 * w / w.sum(1, keepdim=True).clamp_min(1e-300)}


def _exact_weight(w, s, w4):
    N, K = w.shape[0], w.shape[1] * (2 if w4 else 1)
    if w4:
        n = torch.stack([w & 15, w >> 4], 2).view(N, K)
        m = (n & 7).double()
        e = torch.clamp(torch.floor(m / 2), min=1.0)      # exponent field, 1 for the subnormals
        v = torch.where(m < 2, m / 2, (1 + (m % 2) / 2) * torch.exp2(e - 1))
        v = torch.where(n > 7, -v, v)
        return v * _exact_scale(s)[:, torch.arange(K, device=w.device) // 32]
    at = torch.arange(max(N, K), device=w.device) // 128
    return w.view(E4M3).double() * _exact_scale(s)[at[:N]][:, at[:K]]


def _exact_moe(c):
    T, H, I = c["T"], c["H"], c["I"]
    at = torch.arange(H, device="cuda") // 128
    x = c["xq"].view(E4M3).double() * _exact_scale(c["xs"])[:, at]
    y = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    if c["add"] is not None:
        y += c["add"].double()
    ids = c["ids"]
    for e in sorted(set(ids.flatten().tolist()) - {-1}):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        gu = x[t] @ _exact_weight(c["w13"][e], c["s13"][e], c["w4"]).t()
        h = _exact_round(gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:], 8, -133)
        q, s = _exact_quant(h, 128, c["fmt"], None)
        h = q * s.repeat_interleave(128, 1)
        d = h @ _exact_weight(c["w2"][e], c["s2"][e], c["w4"]).t()
        y.index_add_(0, t, d * c["wt"][t, j].double()[:, None])
    return y


def exact(case, seed):
    c = prepare(case, seed)
    return {"norm": _exact_norm, "route": _exact_route, "moe": _exact_moe}[c["op"]](c)
