"""Cases of the operators over a 4-bit paged cache and of sliding-window attention.

``run`` computes one pass of one operator on a state made by ``prepare``: with
``own`` false as elementary torch operations, with ``own`` true through the
library's binding.  The operators:

* write4:  per-head RMS norm and position rotation of a step's new queries and
           keys, K and V stored into the paged 4-bit cache
* read4:   cached tokens of a batch gathered back into dense fp16 K / V rows
* paged4:  tails of a batch over the 4-bit cache, all of it or a sliding window
           and the first tokens ("sinks")
* paged8w: the same tails with a window over the E4M3 cache
* prefillw: dense causal prefill with a window and sinks, fp16 or E4M3 K / V

A 4-bit row of one token and head holds D / 2 bytes of E2M1 codes (value 2i in
the low nibble of byte i) and D / 16 E4M3 scales, one for each 16 values; the
cache is [pages, Hkv, page, 9 D / 16], with one fp32 scale for all of K and one
for all of V.
"""

import math
import random

import torch

own = False

E4M3_MAX = 448.0
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # One decoding step of eight sequences: latency counts.
        {"name": "write4_decode_8", "op": "write4", "dtype": "f16", "tokens": 8, "batch": 8,
         "pad": 0, "ragged": False, "ctx": 1000, "page": 16, "Hq": 6, "Hkv": 1, "D": 256,
         "rot": 64, "interleaved": False, "norm": True},
        # The prefill workload's chunk: 8000 rows at the end of 40000 tokens.
        {"name": "write4_prefill_8000", "op": "write4", "dtype": "f16", "tokens": 8000,
         "batch": 1, "pad": 0, "ragged": False, "ctx": 40000, "page": 16, "Hq": 6, "Hkv": 1,
         "D": 256, "rot": 256, "interleaved": False, "norm": True},
        # Short ragged prefixes brought back for a continuation, padded rows behind them.
        {"name": "read4_ragged_1111", "op": "read4", "tokens": 1111, "batch": 5, "pad": 11,
         "ragged": True, "ctx": 700, "page": 32, "Hkv": 2, "D": 128},
        # The whole long context of the verifier tails.
        {"name": "read4_full_261888", "op": "read4", "tokens": 261888, "batch": 1, "pad": 0,
         "ragged": False, "ctx": 261888, "page": 16, "Hkv": 1, "D": 256},
        # One decoding row over the long context.
        {"name": "paged4_1x1_261888", "op": "paged4", "batch": 1, "rows": 1, "ctx": 261888,
         "page": 16, "Hq": 6, "Hkv": 1, "D": 256, "window": 0, "sinks": 0},
        # The verifier's eight rows at the end of the sweep's longest context.
        {"name": "paged4_1x8_128000", "op": "paged4", "batch": 1, "rows": 8, "ctx": 128000,
         "page": 16, "Hq": 6, "Hkv": 1, "D": 256, "window": 0, "sinks": 0},
        # A serving batch of ragged contexts, four KV heads of 128.
        {"name": "paged4_64x1_8192", "op": "paged4", "batch": 64, "rows": 1, "ctx": 8192,
         "page": 32, "Hq": 16, "Hkv": 4, "D": 128, "window": 0, "sinks": 0},
        # A layer with a window in a batch of long contexts, two verified rows each.
        {"name": "paged4_16x2_window_2000", "op": "paged4", "batch": 16, "rows": 2, "ctx": 40000,
         "page": 16, "Hq": 6, "Hkv": 1, "D": 256, "window": 2000, "sinks": 4},
        # One decoding row with a window over the long E4M3 context: latency counts.
        {"name": "paged8w_1x1_261888", "op": "paged8w", "batch": 1, "rows": 1, "ctx": 261888,
         "page": 16, "Hq": 6, "Hkv": 1, "D": 256, "window": 4096, "sinks": 4},
        # A serving batch's layer with a window, two KV heads of 128.
        {"name": "paged8w_48x2_window_8192", "op": "paged8w", "batch": 48, "rows": 2,
         "ctx": 32768, "page": 16, "Hq": 16, "Hkv": 2, "D": 128, "window": 8192, "sinks": 16},
        # A short chunk over an E4M3 cache.
        {"name": "prefillw_333_of_5000_e4m3", "op": "prefillw", "cache": "e4m3", "Q": 333,
         "KV": 5000, "Hq": 8, "Hkv": 2, "D": 128, "window": 1024, "sinks": 20},
        # The prefill workload with a window.
        {"name": "prefillw_8000_of_40000", "op": "prefillw", "cache": "f16", "Q": 8000,
         "KV": 40000, "Hq": 6, "Hkv": 1, "D": 256, "window": 4096, "sinks": 4},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write4", "read4", "paged4", "paged4", "paged8w", "prefillw"])
    Hq, Hkv, D = rng.choice([(6, 1, 256), (6, 2, 256), (8, 1, 128), (16, 4, 128), (12, 4, 256),
                             (6, 1, 128), (4, 4, 128), (16, 2, 128)])
    page = rng.choice([8, 16, 16, 32, 64, 128, 256])
    if op == "prefillw":
        Q = _log_int(rng, 1, 8000)
        KV = _log_int(rng, max(Q, 2), max(Q, min(40000, 8000 * 40000 * 6 // (Q * Hq))))
        most = max(1, 8000 * 4096 * 6 * 256 // (Q * Hq * D))
        return {"op": op, "cache": rng.choice(["f16", "f16", "e4m3"]), "Q": Q, "KV": KV, "Hq": Hq,
                "Hkv": Hkv, "D": D, "window": _log_int(rng, 1, min(9000, most, KV + 100)),
                "sinks": rng.choice([0, 1, 4, 16, rng.randint(0, 300)])}
    if op in ("paged4", "paged8w"):
        rows = rng.choice([r for r in (1, 1, 2, 3, 4, 8) if r * (Hq // Hkv) <= 48])
        batch = _log_int(rng, 1, 64)
        ctx = _log_int(rng, 8, 261888 * 256 // (batch * Hkv * D))
        windowed = op == "paged8w" or rng.random() < 0.4
        return {"op": op, "batch": batch, "rows": rows, "ctx": ctx, "page": page, "Hq": Hq,
                "Hkv": Hkv, "D": D, "window": _log_int(rng, 1, 9000) if windowed else 0,
                "sinks": rng.choice([0, 4, 16, rng.randint(0, 300)]) if windowed else 0}
    size = (Hq + 2 * Hkv if op == "write4" else Hkv) * D
    tokens = _log_int(rng, 1, (8000 * 8 if op == "write4" else 261888) * 256 // size)
    batch = min(tokens, _log_int(rng, 1, 64))
    ragged = rng.random() < 0.6
    pad = rng.randint(0, min(40, tokens // 8)) if ragged else 0
    if not ragged:
        tokens -= tokens % batch
    ctx = tokens + rng.randint(0, 3000) if batch == 1 else -(-tokens // batch) * 3 + rng.randint(8, 900)
    case = {"op": op, "tokens": tokens, "batch": batch, "pad": pad, "ragged": ragged, "ctx": ctx,
            "page": page, "Hkv": Hkv, "D": D}
    if op == "write4":
        case.update({"dtype": rng.choice(["f16", "bf16"]), "Hq": Hq,
                     "rot": rng.choice([0, 32, 48, 64, 64, 96, 128, D]),
                     "interleaved": rng.random() < 0.4, "norm": rng.random() < 0.8})
    return case


# ---------------------------------------------------------------- the inputs

def _lengths(case):
    """Rows and context length of each sequence, from the case alone."""
    batch, top = case["batch"], case["ctx"]
    rnd = random.Random(batch * 1000003 + top * 7)
    if "rows" in case:  # tails: contexts of all lengths, an idle place among many
        n = [case["rows"]] * batch
        ctx = [top if b == 0 else rnd.randint(top // 8, top) for b in range(batch)]
        if batch >= 8:
            ctx[5] = 0
        return n, ctx
    rows = case["tokens"] - case["pad"]
    if case["ragged"] and batch > 1:
        most = max(-(-rows // batch), min(top, 3 * rows // batch + 1))
        n = [0] * batch
        left = rows
        for b in range(batch):  # what is left always fits into the sequences behind
            rest = (batch - b - 1) * most
            n[b] = rnd.randint(max(0, left - rest), min(most, left, 2 * max(1, left // (batch - b))))
            left -= n[b]
        rnd.shuffle(n)
    else:
        n = [rows // batch] * batch
    return n, [top if batch == 1 else rnd.randint(max(1, x), max(1, x, top)) for x in n]


def _pack4(u):
    """Rows of E2M1 codes and E4M3 scales of the values u [..., D], in units of the tensor's scale."""
    block = u.unflatten(-1, (-1, 16))
    scale = (block.abs().amax(-1) / 6).clamp(max=E4M3_MAX).to(torch.float8_e4m3fn)
    s = scale.float()[..., None]
    x = torch.where(s > 0, block / s, torch.zeros_like(block))
    a = x.abs().clamp(max=6.0)
    # The nearest of 0, 1/2, 1, 3/2, 2, 3, 4, 6, ties to the even code.
    fine = torch.round(a * 2)                       # up to 2: halves
    mid = torch.round(a) + 2                        # up to 4: whole
    wide = torch.where(a > 5, torch.full_like(a, 7.0), torch.full_like(a, 6.0))
    code = torch.where(a < 2, fine, torch.where(a < 4, mid, wide)).to(torch.uint8)
    code = code + (torch.signbit(x) & (s > 0)).to(torch.uint8) * 8
    code = code.flatten(-2)
    return torch.cat([code[..., 0::2] + code[..., 1::2] * 16, scale.view(torch.uint8)], -1)


def _split4(cache, D):
    """Code bytes and scales of a cache."""
    return cache[..., : D // 2], cache[..., D // 2:].view(torch.float8_e4m3fn)


def _unpack4(rows, D, table):
    """The values of rows, in units of the tensor's scale, 32 bits."""
    codes, scale = _split4(rows, D)
    value = table[torch.stack([codes & 15, codes >> 4], -1).int()].flatten(-2)
    return (value.unflatten(-1, (-1, 16)) * scale.float()[..., None]).flatten(-2)


def _addresses(s, gen):
    """Block tables over a permuted pool, context lengths and row starts, on the GPU."""
    case = s["case"]
    n, ctx = _lengths(case)
    page = case["page"]
    stride = -(-case["ctx"] // page)
    pages = case["batch"] * stride + 3
    tables = torch.randperm(pages, generator=gen, device="cuda")[: case["batch"] * stride]
    starts = [0]
    for x in n:
        starts.append(starts[-1] + x)
    dev = {"device": "cuda", "dtype": torch.int32}
    s.update({"tables": tables.to(torch.int32).view(case["batch"], stride).contiguous(),
              "pages": pages, "ctx_lens": torch.tensor(ctx, **dev),
              "starts": torch.tensor(starts, **dev), "used": starts[-1]})


def _cache4(s, gen):
    case = s["case"]
    shape = (s["pages"], case["Hkv"], case["page"], case["D"])
    for name in ("kcache", "vcache"):
        s[name] = _pack4(torch.randn(shape, generator=gen, device="cuda") * 64).contiguous()
    s["table"] = torch.tensor(E2M1 + tuple(-x for x in E2M1), device="cuda")
    # Both nibbles of a byte as E4M3 values: 16 bits for each of 256 bytes.
    b = torch.arange(256, device="cuda")
    pair = torch.stack([s["table"][b & 15], s["table"][b >> 4]], -1).to(torch.float8_e4m3fn)
    s["pairs"] = pair.view(torch.int16)[:, 0].contiguous()


def _cache8(s, shape, gen):
    for name in ("kcache", "vcache"):
        x = torch.randn(shape, generator=gen, device="cuda") * 64
        s[name] = x.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 1000003 + 17)
    s = {"case": case, "scale": 1.0 / math.sqrt(case["D"])}
    s["kscale"] = torch.tensor([1.0 / 64], device="cuda")
    s["vscale"] = torch.tensor([1.0 / 60], device="cuda")
    Hkv, D = case["Hkv"], case["D"]
    if case["op"] == "prefillw":
        s["q"] = torch.randn(case["Q"], case["Hq"], D, generator=gen, device="cuda").half()
        if case["cache"] == "e4m3":
            _cache8(s, (case["KV"], Hkv, D), gen)
        else:
            for name in ("kcache", "vcache"):
                s[name] = torch.randn(case["KV"], Hkv, D, generator=gen, device="cuda").half()
        return s
    _addresses(s, gen)
    if case["op"] == "paged8w":
        _cache8(s, (s["pages"], case["page"], Hkv, D), gen)
    else:
        _cache4(s, gen)
    if "rows" in case:
        s["q"] = torch.randn(case["batch"], case["rows"], case["Hq"], D, generator=gen,
                             device="cuda").half()
        return s
    T = case["tokens"]
    if case["op"] == "read4":
        s["k_out"] = torch.zeros(T, Hkv, D, device="cuda", dtype=torch.float16)
        s["v_out"] = torch.zeros(T, Hkv, D, device="cuda", dtype=torch.float16)
        return s
    Hq = case["Hq"]
    dt = torch.float16 if case["dtype"] == "f16" else torch.bfloat16
    # The fused projection's output; q, k and v are views of it.
    s["qkv"] = torch.randn(T, (Hq + 2 * Hkv) * D, generator=gen, device="cuda").to(dt)
    weight = lambda: (1 + 0.1 * torch.randn(D, generator=gen, device="cuda")).to(dt)  # noqa: E731
    s["q_weight"], s["k_weight"] = (weight(), weight()) if case["norm"] else (None, None)
    i = torch.arange(case["rot"] // 2, device="cuda", dtype=torch.float64)
    s["inv_freq"] = (1e6 ** (-2 * i / max(1, case["rot"]))).to(torch.float32)
    s["q_out"] = torch.zeros(T, Hq, D, device="cuda", dtype=torch.float16)
    return s


# ---------------------------------------------------------------- the plain forms

def _slots(s):
    """Position, page and place in the page of each row that belongs to a sequence."""
    row = torch.arange(s["used"], device="cuda")
    starts = s["starts"].long()
    seq = torch.searchsorted(starts, row, right=True) - 1
    pos = s["ctx_lens"].long()[seq] - starts[seq + 1] + row
    page = s["case"]["page"]
    return pos, s["tables"].long()[seq, pos // page], pos % page


def _norm_rotate(x, weight, cos, sin, case):
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * weight.to(x.dtype)
    rot = case["rot"]
    if rot == 0:
        return x
    if case["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _views(s):
    case = s["case"]
    x = s["qkv"].view(case["tokens"], -1, case["D"])
    return x[:, : case["Hq"]], x[:, case["Hq"]: -case["Hkv"]], x[:, -case["Hkv"]:]


def _write4(s):
    case, n = s["case"], s["used"]
    pos, page, place = _slots(s)
    # Far positions lose their angle in 32 bits.
    angle = pos.double()[:, None] * s["inv_freq"].double()
    cos, sin = (f(angle).float()[:, None, :] for f in (torch.cos, torch.sin))
    q, k, v = (x[:n].float() for x in _views(s))
    s["q_out"][:n] = _norm_rotate(q, s["q_weight"], cos, sin, case).half()
    k = _norm_rotate(k, s["k_weight"], cos, sin, case)
    s["kcache"][page, :, place] = _pack4(k * (1 / s["kscale"]))
    s["vcache"][page, :, place] = _pack4(v * (1 / s["vscale"]))


def _read4(s):
    D, n = s["case"]["D"], s["used"]
    _, page, place = _slots(s)
    for cache, scale, out in (("kcache", "kscale", "k_out"), ("vcache", "vscale", "v_out")):
        x = _unpack4(s[cache][page, :, place], D, s["table"]) * s[scale]
        s[out][:n] = x.half()


def _attend(q, k, v, pos, case, scale):
    """q [..., rows, D], k and v [..., keys, D], the rows' positions [..., rows]."""
    score = q @ k.transpose(-1, -2) * scale
    key = torch.arange(k.shape[-2], device=q.device)
    seen = key <= pos[..., None]
    if case["window"]:
        seen = seen & ((key > pos[..., None] - case["window"]) | (key < case["sinks"]))
    score = torch.where(seen, score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top > -math.inf, top, torch.zeros_like(top)))
    total = p.sum(-1, keepdim=True)
    return p @ v / torch.where(total > 0, total, torch.ones_like(total))


def _paged(s):
    case = s["case"]
    B, R, Hq, Hkv, D = (case[x] for x in ("batch", "rows", "Hq", "Hkv", "D"))
    tables = s["tables"].long()
    kv = []
    for cache, scale in (("kcache", "kscale"), ("vcache", "vscale")):
        x = s[cache][tables]                       # [B, pages, ...]
        if case["op"] == "paged4":
            x = _unpack4(x, D, s["table"]).transpose(2, 3)
        else:
            x = x.view(torch.float8_e4m3fn).float()
        kv.append((x * s[scale]).flatten(1, 2).transpose(1, 2))   # [B, Hkv, keys, D]
    G = Hq // Hkv
    q = s["q"].float().view(B, R, Hkv, G, D).permute(0, 2, 3, 1, 4).flatten(2, 3)
    pos = s["ctx_lens"].long()[:, None] - R + torch.arange(R, device=q.device)
    out = _attend(q, *kv, pos[:, None, None, :].expand(B, 1, G, R).flatten(2), case, s["scale"])
    return out.view(B, Hkv, G, R, D).permute(0, 3, 1, 2, 4).reshape(B, R, Hq, D).half()


def _prefillw(s):
    case = s["case"]
    Q, KV, Hq, Hkv, D = (case[x] for x in ("Q", "KV", "Hq", "Hkv", "D"))
    G = Hq // Hkv
    q = s["q"].float().view(Q, Hkv, G, D).permute(1, 2, 0, 3).flatten(1, 2)
    k, v = s["kcache"], s["vcache"]
    if case["cache"] == "e4m3":
        k = k.view(torch.float8_e4m3fn).float() * s["kscale"]
        v = v.view(torch.float8_e4m3fn).float() * s["vscale"]
    k, v = k.float().transpose(0, 1), v.float().transpose(0, 1)
    pos = (KV - Q + torch.arange(Q, device=q.device)).repeat(G)
    out = _attend(q, k, v, pos, case, s["scale"])
    return out.view(Hkv, G, Q, D).permute(2, 0, 1, 3).reshape(Q, Hq, D).half()


# ---------------------------------------------------------------- the library's calls

def _own(s):
    from long_context_causal_gqa_gb300 import binding

    case = s["case"]
    op = case["op"]
    if op == "prefillw":
        how = {"scale": s["scale"], "window": case["window"], "sinks": case["sinks"]}
        if case["cache"] == "e4m3":
            return binding.prefill_e4m3_window(s["q"], s["kcache"], s["vcache"], s["kscale"],
                                               s["vscale"], **how)
        return binding.prefill_window(s["q"], s["kcache"], s["vcache"], **how)
    where = (s["tables"], s["ctx_lens"], case["ctx"])
    cache = (s["kcache"], s["vcache"], s["kscale"], s["vscale"])
    if op == "paged4":
        return binding.paged_fp4(s["q"], *cache, *where, scale=s["scale"], window=case["window"],
                                 sinks=case["sinks"])
    if op == "paged8w":
        return binding.paged_e4m3_window(s["q"], *cache, *where, scale=s["scale"],
                                         window=case["window"], sinks=case["sinks"])
    starts = s["starts"] if case["ragged"] else None
    if op == "read4":
        return binding.cache_read_fp4(*cache, *where, case["tokens"], row_starts=starts,
                                      k_out=s["k_out"], v_out=s["v_out"])
    return binding.cache_write_fp4(*_views(s), *cache, *where, q_weight=s["q_weight"],
                                   k_weight=s["k_weight"], eps=1e-6,
                                   inv_freq=s["inv_freq"] if case["rot"] else None,
                                   interleaved=case["interleaved"], row_starts=starts,
                                   q_out=s["q_out"])


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        got = _own(s)
    else:
        got = {"write4": _write4, "read4": _read4, "paged4": _paged, "paged8w": _paged,
               "prefillw": _prefillw}[op](s)
    if op == "write4":
        # The codes as the values they stand for, two for each byte.
        out = {"q": s["q_out"]}
        for name in ("kcache", "vcache"):
            codes, scale = _split4(s[name], case["D"])
            pair = s["pairs"].index_select(0, codes.int().view(-1))
            out[name + "_codes"] = pair.view(torch.float8_e4m3fn)
            out[name + "_scales"] = scale
        return out
    if op == "read4":
        return {"k": s["k_out"], "v": s["v_out"]}
    return {"out": got}


# ---------------------------------------------------------------- what a pass needs

def _seen(p, case):
    """Keys that the row at position p sees."""
    if p < 0:
        return 0
    W, S = case["window"], case["sinks"]
    if not W or W > p:
        return p + 1
    return W + min(S, p + 1 - W)


def work(case):
    D, Hkv = case["D"], case["Hkv"]
    if case["op"] == "prefillw":
        Q, KV, Hq = case["Q"], case["KV"], case["Hq"]
        pairs = sum(_seen(KV - Q + i, case) for i in range(Q))
        keys = min(KV, Q + case["window"] - 1 + case["sinks"])
        size = 1 if case["cache"] == "e4m3" else 2
        return {"bytes": 4 * Q * Hq * D + 2 * keys * Hkv * D * size, "flops": 4 * pairs * Hq * D}
    n, ctx = _lengths(case)
    row = 9 * D // 16 if case["op"] != "paged8w" else D
    if "rows" in case:
        R, Hq = case["rows"], case["Hq"]
        pairs = sum(_seen(c - R + r, case) for c in ctx for r in range(R))
        keys = 0
        for c in ctx:
            first = max(0, c - R - case["window"] + 1) if case["window"] else 0
            keys += c - first + min(first, case["sinks"] if case["window"] else 0)
        return {"bytes": 4 * case["batch"] * R * Hq * D + 2 * keys * Hkv * row
                + -(-keys // case["page"]) * 4 + 4 * case["batch"], "flops": 4 * pairs * Hq * D}
    T = sum(n)
    table = -(-T // case["page"]) * 4 + case["batch"] * 8
    if case["op"] == "read4":
        return {"bytes": table + T * 2 * Hkv * (row + 2 * D), "flops": 2 * T * 2 * Hkv * D}
    Hq = case["Hq"]
    return {"bytes": table + T * (2 * (Hq + 2 * Hkv) * D + 2 * Hq * D + 2 * Hkv * row)
            + 2 * case["rot"] + 4 * D, "flops": T * (Hq + 2 * Hkv) * D * 10}


# ---------------------------------------------------------------- the definition in 64 bits

def _decoded(rows, D):
    """Values of 4-bit rows in 64 bits, by the definition of the formats."""
    b = rows[..., : D // 2].long()
    nib = torch.stack([b % 16, b // 16], -1).flatten(-2)
    e, m = nib % 8 // 2, nib % 2
    mag = torch.where(e > 0, (2.0 + m) * 2.0 ** (e.double() - 2), m * 0.5)
    val = torch.where(nib >= 8, -mag, mag)
    sc = rows[..., D // 2:].long()
    es, ms = sc % 128 // 8, sc % 8
    scale = torch.where(es > 0, (8.0 + ms) * 2.0 ** (es.double() - 10), ms * 2.0 ** -9)
    return val * scale.repeat_interleave(16, -1)


def _rows_of(q, k, v, pos, case, scale):
    """Attention of rows [n, D] at positions pos [n] over keys and values [keys, D], by blocks of rows."""
    out = torch.zeros_like(q)
    for at in range(0, len(pos), 512):
        p = pos[at: at + 512]
        lo, hi = int(p.min()), int(p.max())
        if hi < 0:
            continue
        W = case["window"]
        begin = max(0, lo - W + 1) if W else 0
        keys = torch.arange(begin, hi + 1, device=q.device)
        if W:
            keys = torch.cat([torch.arange(min(begin, case["sinks"]), device=q.device), keys])
        x = (q[at: at + 512] * scale).matmul(k[keys].t())
        far = p[:, None] - keys
        hidden = (far < 0) | ((far >= W) & (keys >= case["sinks"])) if W else far < 0
        x = x.masked_fill(hidden, -math.inf)
        x = x - x.max(1, keepdim=True)[0].clamp(min=-1e300)
        w = x.exp()
        out[at: at + 512] = w.matmul(v[keys]) / w.sum(1, keepdim=True).clamp(min=1e-300)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    D, Hkv = case["D"], case["Hkv"]
    ks, vs = s["kscale"].double(), s["vscale"].double()
    if case["op"] == "prefillw":
        k, v = s["kcache"], s["vcache"]
        if case["cache"] == "e4m3":
            k, v = (x.view(torch.float8_e4m3fn).double() * f for x, f in ((k, ks), (v, vs)))
        Q, G = case["Q"], case["Hq"] // Hkv
        pos = torch.arange(case["KV"] - Q, case["KV"], device="cuda")
        out = torch.empty(Q, case["Hq"], D, device="cuda", dtype=torch.float64)
        for h in range(case["Hq"]):
            out[:, h] = _rows_of(s["q"][:, h].double(), k[:, h // G].double(), v[:, h // G].double(),
                                 pos, case, s["scale"])
        return {"out": out}
    page, ctx = case["page"], s["ctx_lens"].tolist()
    if "rows" in case:
        R, G = case["rows"], case["Hq"] // Hkv
        out = torch.zeros(case["batch"], R, case["Hq"], D, device="cuda", dtype=torch.float64)
        for b, c in enumerate(ctx):
            if c == 0:
                continue
            ids = s["tables"][b, : -(-c // page)].long()
            for g in range(Hkv):
                if case["op"] == "paged4":
                    k, v = (_decoded(x[ids, g], D).flatten(0, 1)[:c] for x in (s["kcache"], s["vcache"]))
                else:
                    k, v = (x[ids, :, g].view(torch.float8_e4m3fn).double().flatten(0, 1)[:c]
                            for x in (s["kcache"], s["vcache"]))
                pos = torch.arange(c - R, c, device="cuda").repeat_interleave(G)
                q = s["q"][b, :, g * G: (g + 1) * G].double().reshape(R * G, D)
                got = _rows_of(q, k * ks, v * vs, pos, case, s["scale"])
                out[b, :, g * G: (g + 1) * G] = got.view(R, G, D)
        return {"out": out}
    # Row by row on the host: position, page, place.
    starts, tables, n = s["starts"].tolist(), s["tables"].tolist(), s["used"]
    at = []
    for b in range(case["batch"]):
        for r in range(starts[b], starts[b + 1]):
            p = ctx[b] - (starts[b + 1] - r)
            at.append((p, tables[b][p // page], p % page))
    at = torch.tensor(at, device="cuda", dtype=torch.int64).view(-1, 3)
    if case["op"] == "read4":
        got = {}
        for name, cache, f in (("k", s["kcache"], ks), ("v", s["vcache"], vs)):
            x = torch.zeros(case["tokens"], Hkv, D, device="cuda", dtype=torch.float64)
            x[:n] = _decoded(cache[at[:, 1], :, at[:, 2]], D) * f
            got[name] = x
        return got
    rot = case["rot"]
    angle = at[:, :1].double() * s["inv_freq"].double()
    turn = torch.polar(torch.ones_like(angle), angle)[:, None, :]

    def formula(x, w):
        x = x[:n].double()
        if w is not None:
            x = x / (x.pow(2).sum(-1, keepdim=True) / D + 1e-6).sqrt() * w.double()
        if rot:
            pair = (x[..., :rot].unflatten(-1, (rot // 2, 2)) if case["interleaved"]
                    else x[..., :rot].unflatten(-1, (2, rot // 2)).transpose(-1, -2))
            z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
            z = z if case["interleaved"] else z.transpose(-1, -2)
            x = torch.cat([z.flatten(-2), x[..., rot:]], -1)
        return x

    Hq = case["Hq"]
    x = s["qkv"].view(case["tokens"], -1, D)
    q = torch.zeros(case["tokens"], Hq, D, device="cuda", dtype=torch.float64)
    q[:n] = formula(x[:, :Hq], s["q_weight"])
    got = {"q": q}
    for name, u in (("kcache", formula(x[:, Hq: Hq + Hkv], s["k_weight"]) / ks),
                    ("vcache", x[:n, Hq + Hkv:].double() / vs)):
        # What the scales and, with the rounded scales, the codes round.
        scales = s[name][..., D // 2:].view(torch.float8_e4m3fn).double()
        codes = _decoded(torch.cat([s[name][..., : D // 2],
                                    torch.full_like(s[name][..., D // 2:], 0x38)], -1), D)
        most = u.unflatten(-1, (-1, 16)).abs().amax(-1) / 6
        scales[at[:, 1], :, at[:, 2]] = most.clamp(max=E4M3_MAX)
        stored = most.float().clamp(max=E4M3_MAX).to(torch.float8_e4m3fn).double()
        part = (u.unflatten(-1, (-1, 16)) / stored.clamp(min=1e-30)[..., None]).clamp(-6, 6)
        codes[at[:, 1], :, at[:, 2]] = (part * (stored > 0)[..., None]).flatten(-2)
        got[name + "_codes"] = codes.flatten()
        got[name + "_scales"] = scales
    return got
