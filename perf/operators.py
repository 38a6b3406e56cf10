"""Cases of the operators that fill, read back and search the paged cache.

``run`` computes one pass of one operator on a state made by ``prepare``: with
``own`` false as elementary torch operations, with ``own`` true through the
library's binding.  The operators:

* write:  per-head RMS norm and position rotation of a step's new queries and
          keys, K and V stored into the paged cache (E4M3 codes or fp16)
* read:   cached tokens of a batch gathered back into dense K / V rows
* index:  an int8 summary and a scale for every 4-token block a step completes
* select: the blocks each query row attends, by the summaries' scores
"""

import math
import random

import torch

own = False

E4M3_MAX = 448.0


def listed():
    return [
        # One decoding step of eight sequences, E4M3 cache: latency counts.
        {"name": "write_decode_8", "op": "write", "cache": "e4m3", "dtype": "f16", "tokens": 8,
         "batch": 8, "pad": 0, "ragged": False, "ctx": 4096, "page": 16, "Hq": 6, "Hkv": 1,
         "D": 256, "rot": 64, "interleaved": False, "norm": True},
        # Verifier rows of a ragged batch inside a padded launch, bf16 model, fp16 cache.
        {"name": "write_ragged_509", "op": "write", "cache": "f16", "dtype": "bf16",
         "tokens": 509, "batch": 64, "pad": 13, "ragged": True, "ctx": 1777, "page": 32,
         "Hq": 16, "Hkv": 4, "D": 128, "rot": 128, "interleaved": True, "norm": True},
        # The prefill workload's chunk: 8000 rows at the end of 40000 tokens.
        {"name": "write_prefill_8000", "op": "write", "cache": "e4m3", "dtype": "f16",
         "tokens": 8000, "batch": 1, "pad": 0, "ragged": False, "ctx": 40000, "page": 16,
         "Hq": 6, "Hkv": 1, "D": 256, "rot": 256, "interleaved": False, "norm": True},
        # A short prefix brought back for a prefill continuation.
        {"name": "read_prefix_333", "op": "read", "cache": "e4m3", "tokens": 333, "batch": 1,
         "pad": 0, "ragged": False, "ctx": 333, "page": 16, "Hkv": 1, "D": 256},
        # A ragged batch of fp16 prefixes, padded rows behind it.
        {"name": "read_ragged_f16_20011", "op": "read", "cache": "f16", "tokens": 20011,
         "batch": 16, "pad": 100, "ragged": True, "ctx": 20000, "page": 64, "Hkv": 2, "D": 128},
        # The whole long context of the verifier tails.
        {"name": "read_full_261888", "op": "read", "cache": "e4m3", "tokens": 261888, "batch": 1,
         "pad": 0, "ragged": False, "ctx": 261888, "page": 16, "Hkv": 1, "D": 256},
        # Four verified tokens for each of sixteen sequences: about one block each.
        {"name": "index_verify_64", "op": "index", "cache": "e4m3", "tokens": 64, "batch": 16,
         "pad": 0, "ragged": False, "ctx": 4099, "page": 16, "Hkv": 1, "D": 256},
        # A prefill chunk's blocks, fp16 cache, two KV heads.
        {"name": "index_chunk_f16_8000", "op": "index", "cache": "f16", "tokens": 8000,
         "batch": 3, "pad": 5, "ragged": True, "ctx": 9001, "page": 32, "Hkv": 2, "D": 128},
        # The index of a whole long cache, built at once.
        {"name": "index_full_261888", "op": "index", "cache": "e4m3", "tokens": 261888,
         "batch": 1, "pad": 0, "ragged": False, "ctx": 261888, "page": 16, "Hkv": 1, "D": 256},
        # One decoding row over the long context, 512 tokens kept.
        {"name": "select_decode_261888", "op": "select", "rows": 1, "ctx": 261888, "page": 16,
         "Hq": 6, "Hkv": 1, "D": 256, "max_sel": 128, "first": 1, "last": 2},
        # The sparse prefill workload: 4096 rows at the end of 32768 tokens.
        {"name": "select_4096_32768", "op": "select", "rows": 4096, "ctx": 32768, "page": 16,
         "Hq": 6, "Hkv": 1, "D": 256, "max_sel": 128, "first": 0, "last": 1},
        # The same rows at the end of the prefill sweep's longest context.
        {"name": "select_4096_128000", "op": "select", "rows": 4096, "ctx": 128000, "page": 16,
         "Hq": 6, "Hkv": 1, "D": 256, "max_sel": 128, "first": 4, "last": 8},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "read", "index", "select"])
    Hq, Hkv, D = rng.choice([(6, 1, 256), (6, 2, 256), (8, 1, 128), (16, 4, 128), (12, 4, 256),
                             (6, 1, 128), (4, 4, 128), (16, 2, 128)])
    page = rng.choice([8, 16, 16, 32, 64, 128, 256])
    if op == "select":
        rows = _log_int(rng, 1, 4096)
        most = min(262144, 4096 * 128000 * 256 // (rows * Hkv * D))
        ctx = _log_int(rng, max(rows, 16), max(rows, min(most, 128000 if rows > 64 else most)))
        max_sel = rng.choice([8, 16, 33, 64, 128, 128, 200, 512])
        first = rng.randint(0, min(4, max_sel // 4))
        return {"op": op, "rows": rows, "ctx": ctx, "page": page, "Hq": Hq, "Hkv": Hkv, "D": D,
                "max_sel": max_sel, "first": first, "last": rng.randint(1, max_sel // 4)}
    cache = rng.choice(["e4m3", "e4m3", "f16"])
    size = 2 if cache == "f16" else 1
    if op == "write":
        most = 8000 * 8 * 256 // ((Hq + 2 * Hkv) * D * size)
    else:
        most = 261888 * 256 // (Hkv * D * (4 if cache == "f16" else 1))
    tokens = _log_int(rng, 1, most)
    batch = min(tokens, _log_int(rng, 1, 64))
    ragged = rng.random() < 0.6
    pad = rng.randint(0, min(40, tokens // 8)) if ragged else 0
    if not ragged:
        tokens -= tokens % batch
    ctx = tokens + rng.randint(0, 3000) if batch == 1 else -(-tokens // batch) * 3 + rng.randint(8, 900)
    case = {"op": op, "cache": cache, "tokens": tokens, "batch": batch, "pad": pad,
            "ragged": ragged, "ctx": ctx, "page": page, "Hkv": Hkv, "D": D}
    if op == "write":
        rot = rng.choice([0, 32, 64, 64, 96, 128, D])
        case.update({"dtype": rng.choice(["f16", "bf16"]), "Hq": Hq, "rot": rot,
                     "interleaved": rng.random() < 0.4, "norm": rng.random() < 0.8})
    return case


# ---------------------------------------------------------------- the inputs

def _lengths(case, rnd):
    """Rows and context length of each sequence (the rows sum to tokens - pad)."""
    batch, rows = case["batch"], case["tokens"] - case["pad"]
    if case["ragged"] and batch > 1:
        top = max(-(-rows // batch), min(case["ctx"], 3 * rows // batch + 1))
        n = [0] * batch
        left = rows
        for b in range(batch):  # what is left always fits into the sequences behind
            rest = (batch - b - 1) * top
            n[b] = rnd.randint(max(0, left - rest), min(top, left, 2 * max(1, left // (batch - b))))
            left -= n[b]
        rnd.shuffle(n)
    else:
        n = [rows // batch] * batch
    ctx = [case["ctx"] if batch == 1 else rnd.randint(max(1, x), max(1, x, case["ctx"])) for x in n]
    return n, ctx


def _addresses(case, seed, gen):
    """Block tables over a permuted pool, context lengths and row starts, on the GPU."""
    rnd = random.Random(seed * 7 + 1)
    n, ctx = _lengths(case, rnd)
    page = case["page"]
    stride = -(-case["ctx"] // page)
    pages = case["batch"] * stride + 3
    tables = torch.randperm(pages, generator=gen, device="cuda")[: case["batch"] * stride]
    starts = [0]
    for x in n:
        starts.append(starts[-1] + x)
    dev = {"device": "cuda", "dtype": torch.int32}
    return {"tables": tables.to(torch.int32).view(case["batch"], stride).contiguous(),
            "pages": pages, "ctx_lens": torch.tensor(ctx, **dev),
            "starts": torch.tensor(starts, **dev), "max_ctx": case["ctx"],
            "completed": sum(c // 4 - (c - x) // 4 for x, c in zip(n, ctx)),
            "rows": case["tokens"] - case["pad"]}


def _cache(case, pages, gen):
    """A cache with every token filled: codes of N(0, 1) values times 64, or fp16 N(0, 1)."""
    shape = (pages, case["page"], case["Hkv"], case["D"])
    got = []
    for _ in range(2):
        x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
        if case["cache"] == "e4m3":
            got.append((x * 64).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8))
        else:
            got.append(x.to(torch.float16))
    return got


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 1000003 + 17)
    s = {"case": case}
    if case["op"] == "select":
        rows, Hq, Hkv, D, page = case["rows"], case["Hq"], case["Hkv"], case["D"], case["page"]
        used = -(-case["ctx"] // page)
        pages = used + 2
        # Queries with a shared direction per stretch of rows, as neighbours have.
        drift = torch.randn(rows // 64 + 1, 1, Hq, D, generator=gen, device="cuda")
        q = torch.randn(rows, Hq, D, generator=gen, device="cuda")
        q = q + drift.expand(-1, 64, -1, -1).reshape(-1, Hq, D)[:rows]
        s["q"] = q.to(torch.float16)
        keys = torch.randn(pages, page // 4, Hkv, D, generator=gen, device="cuda") * 0.5
        s["index"], s["index_scale"] = _summaries_of(keys * 4, torch.tensor(1.0, device="cuda"))
        s["table"] = torch.randperm(pages, generator=gen, device="cuda")[:used].to(torch.int32)
        return s
    s.update(_addresses(case, seed, gen))
    s["kcache"], s["vcache"] = _cache(case, s["pages"], gen)
    s["kscale"] = torch.tensor([1.0 / 64], device="cuda")
    s["vscale"] = torch.tensor([1.0 / 60], device="cuda")
    T, Hkv, D = case["tokens"], case["Hkv"], case["D"]
    if case["op"] == "write":
        Hq = case["Hq"]
        dt = torch.float16 if case["dtype"] == "f16" else torch.bfloat16
        # The fused projection's output; q, k and v are views of it.
        s["qkv"] = torch.randn(T, (Hq + 2 * Hkv) * D, generator=gen, device="cuda").to(dt)
        weight = lambda: (1 + 0.1 * torch.randn(D, generator=gen, device="cuda")).to(dt)  # noqa: E731
        s["q_weight"], s["k_weight"] = (weight(), weight()) if case["norm"] else (None, None)
        i = torch.arange(case["rot"] // 2, device="cuda", dtype=torch.float64)
        s["inv_freq"] = (1e6 ** (-2 * i / max(1, case["rot"]))).to(torch.float32)
        s["q_out"] = torch.zeros(T, Hq, D, device="cuda", dtype=torch.float16)
    elif case["op"] == "read":
        s["k_out"] = torch.zeros(T, Hkv, D, device="cuda", dtype=torch.float16)
        s["v_out"] = torch.zeros(T, Hkv, D, device="cuda", dtype=torch.float16)
    else:
        blocks = (s["pages"], case["page"] // 4)
        s["index"] = torch.zeros(*blocks, Hkv, D, device="cuda", dtype=torch.int8)
        s["index_scale"] = torch.zeros(blocks, device="cuda")
    return s


# ---------------------------------------------------------------- the plain forms

def _positions(s):
    """Position and physical token of each row that belongs to a sequence."""
    row = torch.arange(s["rows"], device="cuda")
    starts = s["starts"].long()
    seq = torch.searchsorted(starts, row, right=True) - 1
    pos = s["ctx_lens"].long()[seq] - starts[seq + 1] + row
    page = s["case"]["page"]
    return pos, s["tables"].long()[seq, pos // page] * page + pos % page


def _encode(x, scale):
    return (x / scale).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)


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


def _split(s):
    case = s["case"]
    x = s["qkv"].view(case["tokens"], -1, case["D"])
    return x[:, : case["Hq"]], x[:, case["Hq"]: -case["Hkv"]], x[:, -case["Hkv"]:]


def _write(s):
    case, n = s["case"], s["rows"]
    pos, slot = _positions(s)
    # Far positions lose their angle in 32 bits.
    angle = pos.double()[:, None] * s["inv_freq"].double()
    cos, sin = (f(angle).float()[:, None, :] for f in (torch.cos, torch.sin))
    q, k, v = (x[:n].float() for x in _split(s))
    s["q_out"][:n] = _norm_rotate(q, s["q_weight"], cos, sin, case).to(torch.float16)
    k = _norm_rotate(k, s["k_weight"], cos, sin, case)
    shape = (-1, case["Hkv"], case["D"])
    if case["cache"] == "e4m3":
        s["kcache"].view(shape)[slot] = _encode(k, s["kscale"])
        s["vcache"].view(shape)[slot] = _encode(v, s["vscale"])
    else:
        s["kcache"].view(shape)[slot] = k.to(torch.float16)
        s["vcache"].view(shape)[slot] = v.to(torch.float16)


def _read(s):
    case, n = s["case"], s["rows"]
    _, slot = _positions(s)
    shape = (-1, case["Hkv"], case["D"])
    for cache, scale, out in (("kcache", "kscale", "k_out"), ("vcache", "vscale", "v_out")):
        x = s[cache].view(shape)[slot]
        if case["cache"] == "e4m3":
            x = (x.view(torch.float8_e4m3fn).float() * s[scale]).to(torch.float16)
        s[out][:n] = x


def _summaries_of(total, scale):
    """Codes and scales of blocks, from the sums of their four keys [..., Hkv, D]."""
    most = total.abs().amax((-2, -1))
    fine = torch.isfinite(most) & (most > 0)
    inverse = torch.where(fine, torch.full_like(most, 127.0) / most, torch.zeros_like(most))
    codes = torch.round(torch.where(fine[..., None, None], total, torch.zeros_like(total))
                        * inverse[..., None, None]).to(torch.int8)
    unit = (scale.double() / 508).float()
    return codes, torch.where(fine, most * unit, torch.zeros_like(most))


def _index(s):
    case, n = s["case"], s["rows"]
    pos, slot = _positions(s)
    # A row at the last place of its block completes it; how many do, the host knows.
    done = torch.nonzero_static(pos % 4 == 3, size=s["completed"])[:, 0]
    block = slot[done] // 4
    k = s["kcache"].view(-1, 4, case["Hkv"], case["D"])[block]
    k = (k.view(torch.float8_e4m3fn) if case["cache"] == "e4m3" else k).float()
    scale = s["kscale"] if case["cache"] == "e4m3" else torch.ones_like(s["kscale"])
    codes, unit = _summaries_of((k[:, 0] + k[:, 1]) + (k[:, 2] + k[:, 3]), scale)
    s["index"].view(-1, case["Hkv"], case["D"])[block] = codes
    s["index_scale"].view(-1)[block] = unit


def _select(s):
    case = s["case"]
    rows, Hkv, D, ctx = case["rows"], case["Hkv"], case["D"], case["ctx"]
    dev = s["q"].device
    # Sums of fp16 values are exact in 64 bits, dots of the codes in 32 (whole numbers).
    total = s["q"].double().view(rows, Hkv, -1, D).sum(2).flatten(1).float()
    most = total.abs().amax(1, keepdim=True)
    inverse = torch.where(most > 0, torch.full_like(most, 127.0) / most, torch.zeros_like(most))
    q = torch.round(total * inverse)
    blocks = -(-ctx // 4)
    index = s["index"][s["table"].long()].flatten(0, 1)[:blocks].flatten(1).float()
    scale = s["index_scale"][s["table"].long()].flatten()[:blocks]
    score = (q @ index.t()) * scale + 0.0
    own_block = (torch.arange(rows, device=dev) + (ctx - rows))[:, None] // 4
    b = torch.arange(blocks, device=dev)
    score = torch.where((b < case["first"]) | (b > own_block - case["last"]), math.inf, score)
    score = torch.where(b > own_block, -math.inf, score)
    keep = min(case["max_sel"], blocks)
    best = torch.sort(score, dim=1, descending=True, stable=True)[1][:, :keep]
    best = torch.where(best <= own_block, best, blocks)
    best = torch.sort(best, dim=1)[0]
    sel = torch.full((rows, case["max_sel"]), -1, device=dev, dtype=torch.int32)
    sel[:, :keep] = torch.where(best < blocks, best, -1).to(torch.int32)
    return sel, (own_block[:, 0] + 1).clamp(max=case["max_sel"]).to(torch.int32)


# ---------------------------------------------------------------- the library's calls

def _own(s):
    from long_context_causal_gqa_gb300 import binding

    case = s["case"]
    if case["op"] == "select":
        return binding.select_blocks(s["q"], s["index"], s["index_scale"], s["table"],
                                     case["ctx"], case["max_sel"], n_first=case["first"],
                                     n_last=case["last"])
    starts = s["starts"] if case["ragged"] else None
    e4m3 = case["cache"] == "e4m3"
    where = (s["tables"], s["ctx_lens"], s["max_ctx"])
    if case["op"] == "write":
        how = {"q_weight": s["q_weight"], "k_weight": s["k_weight"], "eps": 1e-6,
               "inv_freq": s["inv_freq"] if case["rot"] else None,
               "interleaved": case["interleaved"], "row_starts": starts, "q_out": s["q_out"]}
        q, k, v = _split(s)
        if e4m3:
            binding.cache_write_e4m3(q, k, v, s["kcache"], s["vcache"], s["kscale"], s["vscale"],
                                     *where, **how)
        else:
            binding.cache_write(q, k, v, s["kcache"], s["vcache"], *where, **how)
    elif case["op"] == "read":
        how = {"row_starts": starts, "k_out": s["k_out"], "v_out": s["v_out"]}
        if e4m3:
            binding.cache_read_e4m3(s["kcache"], s["vcache"], s["kscale"], s["vscale"], *where,
                                    case["tokens"], **how)
        else:
            binding.cache_read(s["kcache"], s["vcache"], *where, case["tokens"], **how)
    elif e4m3:
        binding.block_index_e4m3(s["kcache"], s["kscale"], *where, case["tokens"], s["index"],
                                 s["index_scale"], row_starts=starts)
    else:
        binding.block_index(s["kcache"], *where, case["tokens"], s["index"], s["index_scale"],
                            row_starts=starts)


def run(s):
    op = s["case"]["op"]
    got = None
    if own:
        got = _own(s)
    elif op == "select":
        got = _select(s)
    else:
        {"write": _write, "read": _read, "index": _index}[op](s)
    if op == "select":
        return {"sel_idx": got[0], "sel_cnt": got[1]}
    if op == "write":
        e4m3 = s["case"]["cache"] == "e4m3"
        view = (lambda x: x.view(torch.float8_e4m3fn)) if e4m3 else (lambda x: x)
        return {"q": s["q_out"], "k": view(s["kcache"]), "v": view(s["vcache"])}
    if op == "read":
        return {"k": s["k_out"], "v": s["v_out"]}
    return {"codes": s["index"], "scale": s["index_scale"]}


# ---------------------------------------------------------------- what a pass needs

def work(case):
    if case["op"] == "select":
        rows, K, ctx = case["rows"], case["Hkv"] * case["D"], case["ctx"]
        blocks = -(-ctx // 4)
        seen = sum((ctx - rows + i) // 4 for i in range(rows))
        return {"bytes": rows * case["Hq"] * case["D"] * 2 + blocks * (K + 4)
                + -(-ctx // case["page"]) * 4 + rows * (case["max_sel"] + 1) * 4,
                "flops": 2 * seen * K}
    T, kv = case["tokens"] - case["pad"], case["Hkv"] * case["D"]
    size = 1 if case["cache"] == "e4m3" else 2
    table = -(-T // case["page"]) * 4 + case["batch"] * 8
    if case["op"] == "write":
        q = case["Hq"] * case["D"]
        return {"bytes": table + T * (2 * (q + 2 * kv) + 2 * q + 2 * kv * size) + 2 * case["rot"]
                + 4 * case["D"], "flops": T * (q + kv) * 10}
    if case["op"] == "read":
        return {"bytes": table + T * 2 * kv * (size + 2), "flops": T * 2 * kv}
    blocks = T // 4
    return {"bytes": table + blocks * (4 * kv * size + kv + 4), "flops": blocks * kv * 6}


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    if case["op"] == "select":
        return None  # ids and counts only
    s = prepare(case, seed)
    n, page, D, Hkv = s["rows"], case["page"], case["D"], case["Hkv"]
    # Row by row on the host: sequence, position, physical token.
    starts, lens = s["starts"].tolist(), s["ctx_lens"].tolist()
    tables = s["tables"].tolist()
    at, where = [], []
    for b in range(case["batch"]):
        for r in range(starts[b], starts[b + 1]):
            p = lens[b] - (starts[b + 1] - r)
            at.append(p)
            where.append(tables[b][p // page] * page + p % page)
    where_t = torch.tensor(where, device="cuda", dtype=torch.int64)
    decoded = lambda c: (c.view(torch.float8_e4m3fn) if c.dtype == torch.uint8 else c).double()  # noqa: E731
    e4m3 = case["cache"] == "e4m3"
    ks, vs = (s["kscale"].double(), s["vscale"].double()) if e4m3 else (1.0, 1.0)
    if case["op"] == "read":
        out = []
        for cache, scale in ((s["kcache"], ks), (s["vcache"], vs)):
            x = torch.zeros(case["tokens"], Hkv, D, device="cuda", dtype=torch.float64)
            x[:n] = decoded(cache.view(-1, Hkv, D)[where_t]) * scale
            out.append(x)
        return {"k": out[0], "v": out[1]}
    if case["op"] == "index":
        last = torch.tensor([w for p, w in zip(at, where) if p % 4 == 3], device="cuda",
                            dtype=torch.int64)
        scale = torch.zeros(s["index_scale"].numel(), device="cuda", dtype=torch.float64)
        for part in last.split(16384):
            k = sum(decoded(s["kcache"].view(-1, Hkv, D)[part - j]) for j in range(4))
            scale[part // 4] = k.abs().flatten(1).amax(1) * ks / 4 / 127
        return {"codes": None, "scale": scale.view(s["index_scale"].shape)}
    rot = case["rot"]
    angle = torch.tensor(at, device="cuda", dtype=torch.float64)[:, None] * s["inv_freq"].double()
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

    x = s["qkv"].view(case["tokens"], -1, D)
    q = torch.zeros(case["tokens"], case["Hq"], D, device="cuda", dtype=torch.float64)
    q[:n] = formula(x[:, : case["Hq"]], s["q_weight"])
    k = formula(x[:, case["Hq"]: case["Hq"] + Hkv], s["k_weight"])
    kc, vc = decoded(s["kcache"]), decoded(s["vcache"])
    most = E4M3_MAX if e4m3 else 65504.0
    kc.view(-1, Hkv, D)[where_t] = (k / ks).clamp(-most, most)
    vc.view(-1, Hkv, D)[where_t] = (x[:n, case["Hq"] + Hkv:].double() / vs).clamp(-most, most)
    return {"q": q, "k": kc, "v": vc}
