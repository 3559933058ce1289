"""Workloads of the operators around an 8-bit paged KV cache.

Four operators:

* rope: rotary positions of a step's queries and keys (``attn_rope``).
* store: a step's new keys and values quantised into an 8-bit paged cache, with
  one scale for each block of tokens and kv head (``kv_quant_store``); with the
  rotary positions in the same call (``kv_quant_store_rope``), after which the
  sequences are read back as a prefill reads them.
* load: sequences read back from the 8-bit cache as bf16 rows (``kv_quant_load``).
* decode: one query token per sequence over the 8-bit cache (``attn_decode_quant``).

``run`` computes a case in its plain form (elementary torch operations, fp32,
rotary angles in 64 bits) or, with ``own`` set, through the library's calls.
``exact`` has the same results in 64 bits, from the definitions.
"""
import math

import torch

own = False

BF16, I32, F32, F64 = torch.bfloat16, torch.int32, torch.float32, torch.float64
DEV = "cuda"
LIMIT = {"e4m3": 448.0, "int8": 127.0}  # the largest code
DTYPE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
LEAST_SCALE = 2.0 ** -64


# --------------------------------------------------------------------- cases

def _rotary(rotary, interleaved=False, scaling="none", factor=1.0, base=1000000.0, first=0):
    """Positions begin at `first`; the first `rotary` numbers of a head are rotated."""
    return {"rotary": rotary, "interleaved": interleaved, "scaling": scaling, "factor": factor, "base": base,
            "original_len": 4096, "first": first}


def _rope(name, heads, tokens, step, **rotary):
    case = {"op": "rope", "heads": heads, "tokens": tokens, "step": step, **_rotary(**rotary)}
    return case if name is None else {"name": name, **case}


def _store(name, heads, block_size, scale_tokens, form, seqs, cached, new, **rotary):
    case = {"op": "store", "heads": heads, "block_size": block_size, "scale_tokens": scale_tokens, "form": form,
            "seqs": seqs, "cached_lo": cached[0], "cached_hi": cached[1], "new_lo": new[0], "new_hi": new[1],
            **_rotary(**{"rotary": 0, **rotary})}
    return case if name is None else {"name": name, **case}


def _load(name, heads, block_size, scale_tokens, form, seqs, lo, hi, align=1):
    case = {"op": "load", "heads": heads, "block_size": block_size, "scale_tokens": scale_tokens, "form": form,
            "seqs": seqs, "lo": lo, "hi": hi, "align": align}
    return case if name is None else {"name": name, **case}


def _decode(name, heads, block_size, scale_tokens, form, seqs, lo, hi, padding=0):
    case = {"op": "decode", "heads": heads, "block_size": block_size, "scale_tokens": scale_tokens, "form": form,
            "seqs": seqs, "lo": lo, "hi": hi, "padding": padding}
    return case if name is None else {"name": name, **case}


def listed():
    return [
        # the next token of one chat: latency alone
        _rope("rope_one_token", "16/8/128", 1, "decode", rotary=128, first=2049),
        # an odd prefill chunk: a part of each head, neighbouring pairs, frequencies scaled by their wavelength
        _rope("rope_chunk_partial", "16/4/128", 777, "prefill", rotary=64, interleaved=True, scaling="wavelength",
              factor=8.0, first=12345),
        # the largest prefill step, far into a document, positions stretched to 16 times the trained length
        _rope("rope_prefill_16k", "32/8/128", 16384, "prefill", rotary=128, scaling="yarn", factor=16.0,
              first=49152),
        # the benchmark's decode batch: each sequence's new token into a block that is partly filled
        _store("store_decode_64", "16/8/128", 256, 16, "e4m3", 64, (511, 4095), (1, 1)),
        # the benchmark's prefill batch, blocks of 64 tokens in whole numbers
        _store("store_prefill_8", "32/8/128", 256, 64, "int8", 8, (0, 0), (256, 2048)),
        # ragged chunks behind cached prefixes: rotate, store, and read all of it back for the prefill
        _store("rope_store_chunks", "16/8/128", 16, 16, "e4m3", 5, (32, 700), (17, 900), rotary=128, first=0),
        # cached prefixes of a prefill batch, laid out on pages of 16 rows
        _load("load_prefixes_8", "16/8/128", 256, 16, "e4m3", 8, 100, 2048, align=16),
        # one long document, a scale for each token
        _load("load_long", "32/8/128", 256, 1, "int8", 1, 131072, 131072),
        # three short requests on a tiny model: latency alone
        _decode("decode_tiny", "2/1/64", 16, 16, "e4m3", 3, 1, 50),
        # the benchmark's decode batch, padded to a graph's bucket
        _decode("decode_b64", "16/8/128", 256, 16, "e4m3", 62, 512, 4096, padding=2),
        # eight query heads per kv head over one long document
        _decode("decode_long", "64/8/128", 256, 64, "int8", 1, 131071, 131071),
        # the largest serving batch
        _decode("decode_b512", "32/8/128", 256, 16, "e4m3", 512, 1000, 8000),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


_HEADS = ["2/1/64", "4/2/64", "16/8/64", "8/8/128", "16/8/128", "32/8/128", "64/8/128", "8/1/128", "16/4/128"]


def _draw_rotary(rng, d):
    scaling = rng.choice(["none", "linear", "ntk", "yarn", "wavelength"])
    return {"rotary": rng.choice([d, d, d // 2, d // 4, 2 * rng.randint(2, d // 2)]), "interleaved": rng.random() < 0.4,
            "scaling": scaling, "factor": 1.0 if scaling == "none" else rng.choice([2.0, 4.0, 7.5, 32.0]),
            "base": rng.choice([10000.0, 500000.0, 1000000.0]), "first": _log_int(rng, 1, 1000000) - 1}


def draw(rng):
    """One more case of the ranges that the listed ones stand for."""
    op = rng.choice(["rope", "store", "store", "load", "decode", "decode", "decode"])
    heads = rng.choice(_HEADS)
    hq, hkv, d = (int(x) for x in heads.split("/"))
    if op == "rope":
        most = 16384 * 40 * 128 // ((hq + hkv) * d)
        return _rope(None, heads, _log_int(rng, 1, min(most, 40000)), rng.choice(["decode", "prefill"]),
                     **_draw_rotary(rng, d))
    block_size = rng.choice([16, 32, 64, 128, 256])
    scale_tokens = min(block_size, rng.choice([1, 4, 16, 16, 32, 64, 256]))
    form = rng.choice(["e4m3", "e4m3", "int8"])
    if op == "store":
        seqs = _log_int(rng, 1, 200)
        hi = 1 if rng.random() < 0.4 else _log_int(rng, 1, max(2, 6000 // seqs))
        cached = rng.choice([0, _log_int(rng, 1, max(2, 40000 // seqs))])
        rotary = _draw_rotary(rng, d) if rng.random() < 0.4 else {}
        return _store(None, heads, block_size, scale_tokens, form, seqs, (rng.randint(0, cached), cached),
                      (rng.randint(1, hi), hi), **rotary)
    if op == "load":
        seqs = _log_int(rng, 1, 100)
        hi = _log_int(rng, 1, max(2, 120000 // seqs))
        return _load(None, heads, block_size, scale_tokens, form, seqs, rng.randint(min(seqs, 2) % 2, hi), hi,
                     rng.choice([1, 16]))
    seqs = _log_int(rng, 1, 400)
    hi = _log_int(rng, 2, 100000)
    while seqs * hi > 2_000_000:
        hi //= 2
    return _decode(None, heads, block_size, scale_tokens, form, seqs, rng.randint(1, hi), hi,
                   padding=rng.choice([0, 0, 5]))


def _heads(case):
    hq, hkv, d = (int(x) for x in case["heads"].split("/"))
    return hq, hkv, d


def _spread(n, lo, hi):
    """n whole numbers spread evenly over lo..hi, both ends among them."""
    return [lo + (hi - lo) * i // max(1, n - 1) for i in range(n)]


def _ceil(a, b):
    return -(-a // b)


# -------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _shuffled(values, g):
    return [values[i] for i in torch.randperm(len(values), generator=g, device=DEV).tolist()]


def _frequencies(case):
    """Angle per position of each pair, in radians, and what cosine and sine are multiplied by."""
    r, base, factor, trained = case["rotary"], case["base"], case["factor"], case["original_len"]
    pairs = torch.arange(r // 2, dtype=F64)
    if case["scaling"] == "ntk":
        base = base * factor ** (r / (r - 2)) if r > 2 else base
    inv = base ** (-2.0 * pairs / r)
    if case["scaling"] == "linear":
        return inv / factor, 1.0
    if case["scaling"] == "yarn":
        turn = lambda turns: r * math.log(trained / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        low, high = max(0, math.floor(turn(32.0))), min(r - 1, math.ceil(turn(1.0)))
        slow = ((pairs - low) / max(high - low, 0.001)).clamp(0, 1)
        return inv * (1 - slow) + inv / factor * slow, 0.1 * math.log(factor) + 1.0
    if case["scaling"] == "wavelength":
        keep = ((trained * inv / (2 * math.pi) - 1.0) / (4.0 - 1.0)).clamp(0, 1)
        return inv * keep + inv / factor * (1 - keep), 1.0
    return inv, 1.0


def _prepare_rotary(case):
    """The frequencies that a program keeps for a model."""
    inv, magnitude = _frequencies(case)
    if own:
        import paged_kv_cache_125_gb300 as kvp
        freqs, magnitude = kvp.attn_rope_freqs(case["rotary"], base=case["base"], scaling=case["scaling"],
                                               factor=case["factor"], original_len=case["original_len"],
                                               device=DEV)
        return {"freqs": freqs, "magnitude": magnitude, "interleaved": case["interleaved"]}
    return {"inv": inv.to(DEV), "magnitude": magnitude, "interleaved": case["interleaved"]}


def _projected(n, hq, hkv, d, g):
    """q, k and v as parts of the rows that one projection writes."""
    rows = torch.empty((n, hq + 2 * hkv, d), dtype=BF16, device=DEV).normal_(generator=g)
    return rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:]


def _prepare_rope(case, g):
    hq, hkv, d = _heads(case)
    n = case["tokens"]
    q, k, _ = _projected(n, hq, hkv, d, g)
    if case["step"] == "decode":  # a row for each sequence, all at places of their own
        positions = torch.randint(0, case["first"] + 1, (n,), generator=g, device=DEV)
    else:
        positions = torch.arange(case["first"], case["first"] + n, device=DEV)
    return {"q": q, "k": k, "positions": positions, **_prepare_rotary(case)}


def _codes(shape, form, g):
    """Codes as quantising normal numbers leaves them."""
    out = torch.empty(shape, dtype=DTYPE[form], device=DEV)
    flat, step = out.view(torch.uint8).view(-1), 1 << 27
    for at in range(0, flat.numel(), step):
        x = torch.empty((min(step, flat.numel() - at),), dtype=F32, device=DEV).normal_(generator=g)
        x.mul_(LIMIT[form] / 4).clamp_(-LIMIT[form], LIMIT[form])
        flat[at:at + step] = (x.round_() if form == "int8" else x).to(DTYPE[form]).view(torch.uint8)
    return out


def _prepare_cache(case, lens, spare, g):
    """An 8-bit cache whose sequences have room for lens tokens, its block tables, and `spare` more pages."""
    bs, t = case["block_size"], case["scale_tokens"]
    _, hkv, d = _heads(case)
    pages = [_ceil(n, bs) for n in lens]
    blocks, width = sum(pages) + spare, max(1, max(pages))
    ids = torch.randperm(blocks, generator=g, device=DEV)
    inside = torch.arange(width, device=DEV) < torch.tensor(pages, device=DEV)[:, None]
    tables = torch.full((len(lens), width), -1, dtype=I32, device=DEV)
    tables[inside] = ids[:sum(pages)].to(I32)
    cache, size = {}, LIMIT[case["form"]] / 448.0
    for name in ("k", "v"):
        cache[name + "_cache"] = _codes((blocks, bs, hkv, d), case["form"], g)
        grow = torch.randint(-8, -5, (blocks, bs // t, hkv), generator=g, device=DEV)
        cache[name + "_scales"] = torch.exp2(grow.to(F32) + (0 if size == 1.0 else 2))
    return {**cache, "tables": tables}


def _prepare_store(case, g):
    bs, n = case["block_size"], case["seqs"]
    hq, hkv, d = _heads(case)
    cached = _shuffled(_spread(n, case["cached_lo"], case["cached_hi"]), g)
    new = _shuffled(_spread(n, case["new_lo"], case["new_hi"]), g)
    lens = [a + b for a, b in zip(cached, new)]
    s = _prepare_cache(case, lens, 3, g)
    rows = sum(new)
    q, s["k"], s["v"] = _projected(rows, hq, hkv, d, g)
    seq = torch.repeat_interleave(torch.arange(n, device=DEV), torch.tensor(new, device=DEV))
    before = torch.tensor([c - sum(new[:i]) for i, c in enumerate(cached)], device=DEV)
    at = torch.arange(rows, device=DEV) + before[seq]
    s["slots"] = (s["tables"][seq, at // bs].long() * bs + at % bs).to(I32)
    if case["rotary"]:
        s.update(_prepare_rotary(case), q=q, positions=at + case["first"], **_prepare_rows(case, lens))
    return s


def _prepare_rows(case, lens):
    """Where the sequences are read back to: bf16 rows, each sequence's from a multiple of `align` on."""
    _, hkv, d = _heads(case)
    align = case.get("align", 1)
    starts, at = [], 0
    for n in lens:
        starts.append(at)
        at += _ceil(n, align) * align
    rows = lambda: torch.zeros((max(at, 1), hkv, d), dtype=BF16, device=DEV)  # noqa: E731
    return {"contexts": torch.tensor(lens, dtype=I32, device=DEV), "starts": torch.tensor(starts, dtype=I32, device=DEV),
            "total": sum(lens), "longest": max(lens), "k_rows": rows(), "v_rows": rows()}


def _prepare_load(case, g):
    lens = _shuffled(_spread(case["seqs"], case["lo"], case["hi"]), g)
    return {**_prepare_cache(case, lens, 2, g), **_prepare_rows(case, lens)}


def _prepare_decode(case, g):
    hq, hkv, d = _heads(case)
    lens = _shuffled(_spread(case["seqs"], case["lo"], case["hi"]), g) + [0] * case["padding"]
    s = _prepare_cache(case, lens, 2, g)
    s["q"] = torch.empty((len(lens), hq, d), dtype=BF16, device=DEV).normal_(generator=g)
    s["contexts"] = torch.tensor(lens, dtype=I32, device=DEV)
    s["longest"] = max(lens)
    if own:
        import paged_kv_cache_125_gb300 as kvp
        # scratch that a serving loop keeps
        size = kvp.attn_decode_quant_workspace_size(len(lens), hq, hkv, d, s["longest"])
        s["workspace"] = torch.empty((size,), dtype=torch.uint8, device=DEV)
    return s


def prepare(case, seed):
    make = {"rope": _prepare_rope, "store": _prepare_store, "load": _prepare_load, "decode": _prepare_decode}
    return {"op": case["op"], "form": case.get("form"), **make[case["op"]](case, _gen(seed))}


# ---------------------------------------------------------------- plain forms

def _turned(x, s):
    """Rows [tokens, heads, d] with their first numbers rotated by their positions' angles, fp32."""
    angle = s["positions"].to(F64)[:, None] * s["inv"]
    cos, sin = ((f(angle) * s["magnitude"]).to(F32)[:, None] for f in (torch.cos, torch.sin))
    x, n = x.to(F32), 2 * s["inv"].numel()
    a, b = (x[..., 0:n:2], x[..., 1:n:2]) if s["interleaved"] else (x[..., :n // 2], x[..., n // 2:n])
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((a, b), -1).flatten(-2) if s["interleaved"] else torch.cat((a, b), -1)
    return torch.cat((turned, x[..., n:]), -1)


def _plain_rope(s):
    return {"q": _turned(s["q"], s).to(BF16), "k": _turned(s["k"], s).to(BF16)}


def _encoded(x, form):
    x = x.clamp(-LIMIT[form], LIMIT[form])
    return (x.round() if form == "int8" else x).to(DTYPE[form]).view(torch.uint8)


def _power_above(top, form):
    """The least power of two p with top <= p * (the largest code), at least LEAST_SCALE."""
    part, power = torch.frexp(top)  # top = part * 2^power, part in [1/2, 1)
    part_limit, power_limit = math.frexp(LIMIT[form])
    power = power - power_limit + (part > part_limit)
    return torch.where(top > 0, torch.exp2(power.to(F32)), 0.0).clamp(min=LEAST_SCALE)


def _plain_quantise(rows, slots, cache, scales, form):
    """fp32 rows into their slots; every block of tokens that they touch gets a scale that holds them too."""
    (blocks, bs, hkv, d), t = cache.shape, cache.shape[1] // scales.shape[1]
    codes, per_group = cache.view(torch.uint8).view(-1, t, hkv, d), scales.view(-1, hkv)
    groups, place = torch.unique(slots // t, return_inverse=True)
    top = torch.zeros((groups.numel(), hkv), device=DEV).index_reduce_(0, place, rows.abs().amax(-1), "amax")
    fresh = torch.zeros((groups.numel(),), device=DEV).index_reduce_(0, place, (slots % t == 0).to(F32), "amax")
    fresh = fresh[:, None] > 0
    old, need = per_group[groups], _power_above(top, form)
    new = torch.where(fresh, need, torch.maximum(old, need))
    before = codes[groups]
    values = before.view(DTYPE[form]).to(F32) * torch.where(fresh, 1.0, old / new)[:, None, :, None]
    codes[groups] = _encoded(values, form)
    codes.view(-1, hkv, d)[slots] = _encoded(rows / new[place][..., None], form)
    per_group[groups] = new


def _plain_read(s):
    """The sequences' tokens as bf16 rows at the places that their starts say."""
    ctx, bs = s["contexts"].long(), s["k_cache"].shape[1]
    seq = torch.repeat_interleave(torch.arange(ctx.numel(), device=DEV), ctx, output_size=s["total"])
    first = torch.cumsum(ctx, 0) - ctx
    at = torch.arange(s["total"], device=DEV) - first[seq]
    slot = s["tables"].long()[seq, at // bs] * bs + at % bs
    for name in ("k", "v"):
        s[name + "_rows"][s["starts"].long()[seq] + at] = _read_slots(s, name, slot).to(BF16)
    return {"k": s["k_rows"], "v": s["v_rows"]}


def _read_slots(s, name, slot):
    """fp32 values of cache slots (any shape): [..., kv heads, head_dim]."""
    cache, scales = s[name + "_cache"], s[name + "_scales"]
    _, bs, hkv, d = cache.shape
    codes = cache.view(torch.uint8).view(-1, hkv, d)[slot].view(cache.dtype).to(F32)
    return codes.mul_(scales.view(-1, hkv)[slot // (bs // scales.shape[1])][..., None])


def _plain_store(s):
    slots = s["slots"].long()
    k = _turned(s["k"], s) if "positions" in s else s["k"].to(F32)
    _plain_quantise(k, slots, s["k_cache"], s["k_scales"], s["form"])
    _plain_quantise(s["v"].to(F32), slots, s["v_cache"], s["v_scales"], s["form"])
    if "positions" in s:
        return {"q": _turned(s["q"], s).to(BF16), **_plain_read(s)}
    return {name: s[name] for name in ("k_cache", "v_cache", "k_scales", "v_scales")}


def _plain_decode(s):
    ctx, q = s["contexts"], s["q"]
    _, bs, hkv, d = s["k_cache"].shape
    batch, hq, _ = q.shape
    pos = torch.arange(s["tables"].shape[1] * bs, device=DEV)
    seen = pos < ctx[:, None]
    slot = torch.where(seen, s["tables"].long()[:, pos // bs] * bs + pos % bs, 0)
    keys = _read_slots(s, "k", slot).permute(0, 2, 3, 1)
    scores = torch.matmul(q.to(F32).view(batch, hkv, hq // hkv, d), keys) * d ** -0.5
    del keys
    scores = scores.masked_fill(~seen[:, None, None, :], -math.inf)
    top = scores.amax(-1, keepdim=True)
    weights = torch.exp(scores - torch.where(top == -math.inf, 0.0, top))
    total = weights.sum(-1, keepdim=True)
    del scores
    values = _read_slots(s, "v", slot).permute(0, 2, 1, 3)
    out = torch.matmul(weights, values) / torch.where(total == 0, 1.0, total)
    return {"out": out.view(batch, hq, d).to(BF16)}


# --------------------------------------------------------- the library's calls

def _own_rope(s, kvp):
    q, k = kvp.attn_rope(s["q"], s["k"], s["positions"], s["freqs"], s["magnitude"], s["interleaved"])
    return {"q": q, "k": k}


def _own_store(s, kvp):
    cache = (s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"])
    if "positions" not in s:
        kvp.kv_quant_store(s["k"], s["v"], s["slots"], *cache)
        return {name: s[name] for name in ("k_cache", "v_cache", "k_scales", "v_scales")}
    q = kvp.kv_quant_store_rope(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["freqs"], *cache,
                                s["magnitude"], s["interleaved"])
    return {"q": q, **_own_load(s, kvp)}


def _own_load(s, kvp):
    k, v = kvp.kv_quant_load(s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"], s["tables"], s["contexts"],
                             s["starts"], s["longest"], out=(s["k_rows"], s["v_rows"]))
    return {"k": k, "v": v}


def _own_decode(s, kvp):
    return {"out": kvp.attn_decode_quant(s["q"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"],
                                         s["tables"], s["contexts"], s["longest"], workspace=s["workspace"])}


def run(state):
    if own:
        import paged_kv_cache_125_gb300 as kvp
        return {"rope": _own_rope, "store": _own_store, "load": _own_load,
                "decode": _own_decode}[state["op"]](state, kvp)
    return {"rope": _plain_rope, "store": _plain_store, "load": _plain_read,
            "decode": _plain_decode}[state["op"]](state)


# ------------------------------------------------------------- least work

def _groups(lens, t):
    return sum(_ceil(n, t) for n in lens)


def work(case):
    hq, hkv, d = _heads(case)
    if case["op"] == "rope":
        n = case["tokens"]
        # every row once in and out, a position; three operations a rotated number
        return {"bytes": n * ((hq + hkv) * d * 4 + 8) + case["rotary"] * 4, "flops": n * (hq + hkv) * case["rotary"] * 3}
    row, t = hkv * d, case["scale_tokens"]
    if case["op"] == "store":
        new, cached = (_spread(case["seqs"], case[a + "_lo"], case[a + "_hi"]) for a in ("new", "cached"))
        n, total = sum(new), sum(new) + sum(cached)
        # rows in (bf16), codes out, the touched blocks' scales in and out, a slot; an operation for the
        # largest number and one for the code
        got = {"bytes": n * (2 * row * 3 + 4) + 2 * 2 * 4 * hkv * _groups(new, t), "flops": n * 2 * row * 2}
        if case["rotary"]:
            got["bytes"] += n * (hq * d * 4 + 8) + total * 2 * row * 2 + sum(cached) * 2 * row
            got["flops"] += n * (hq + hkv) * case["rotary"] * 3 + total * 2 * row
        return got
    lens = _spread(case["seqs"], case["lo"], case["hi"])
    n, entries = sum(lens), _groups(lens, case["block_size"])
    read = 2 * n * row + 2 * 4 * hkv * _groups(lens, t) + 4 * entries + 8 * len(lens)
    if case["op"] == "load":
        return {"bytes": read + 2 * n * row * 2, "flops": 2 * n * row}
    batch = case["seqs"] + case["padding"]
    return {"bytes": read + batch * hq * d * 4, "flops": 4 * hq * d * n}


# ------------------------------------------------------------ 64-bit definitions

def _exact_turned(x, case, positions):
    """Rotation of the pairs as complex numbers."""
    inv, magnitude = _frequencies(case)
    r = case["rotary"]
    turn = torch.polar(torch.full((1, 1), magnitude, dtype=F64, device=DEV),
                       positions.to(F64)[:, None] * inv.to(DEV))[:, None]
    out = x.to(F64).clone()
    first, second = (slice(0, r, 2), slice(1, r, 2)) if case["interleaved"] else (slice(0, r // 2), slice(r // 2, r))
    z = torch.complex(out[..., first], out[..., second]) * turn
    out[..., first], out[..., second] = z.real, z.imag
    return out


def _exact_codes(x, form):
    """Nearest code values, ties to the even one."""
    if form == "int8":
        return torch.round(x).clamp(-127, 127)
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _exact_quantise(rows, slots, cache, scales, form):
    """The cache's code values and scales after the rows were stored, block by block."""
    t = cache.shape[1] // scales.shape[1]
    values = cache.to(F64).view(-1, *cache.shape[2:])
    scales = scales.to(F64).clone().view(-1, cache.shape[2])
    slots, at = slots.tolist(), 0
    while at < len(slots):
        group, end = slots[at] // t, at
        while end < len(slots) and slots[end] // t == group:
            end += 1
        top = rows[at:end].abs().amax(-1).amax(0)
        need = torch.exp2(torch.ceil(torch.log2(top / LIMIT[form]))).clamp(min=LEAST_SCALE)
        if slots[at] % t:
            old, need = scales[group], torch.maximum(need, scales[group])
            whole = values[group * t:(group + 1) * t]
            whole.copy_(_exact_codes(whole * (old / need)[:, None], form))
        scales[group] = need
        values[slots[at]:slots[at] + end - at] = _exact_codes(rows[at:end] / need[:, None], form)
        at = end
    return values.view(cache.shape), scales.view(cache.shape[0], -1, cache.shape[2])


def _exact_read(s, case, k, v):
    out = []
    for (codes, scales), name in ((k, "k"), (v, "v")):
        rows = torch.zeros(s[name + "_rows"].shape, dtype=F64, device=DEV)
        values = codes * torch.repeat_interleave(scales, case["scale_tokens"], 1)[..., None]
        for b, (n, start) in enumerate(zip(s["contexts"].tolist(), s["starts"].tolist())):
            pages = s["tables"][b, :_ceil(n, case["block_size"])].long()
            rows[start:start + n] = values[pages].reshape(-1, *rows.shape[1:])[:n]
        out.append(rows)
    return {"k": out[0], "v": out[1]}


def _exact_store(s, case):
    turn = case["rotary"] > 0
    k = _exact_turned(s["k"], case, s["positions"]) if turn else s["k"].to(F64)
    k = _exact_quantise(k, s["slots"], s["k_cache"], s["k_scales"], case["form"])
    v = _exact_quantise(s["v"].to(F64), s["slots"], s["v_cache"], s["v_scales"], case["form"])
    if turn:
        return {"q": _exact_turned(s["q"], case, s["positions"]), **_exact_read(s, case, k, v)}
    whole = case["form"] == "int8"
    return {"k_cache": None if whole else k[0], "v_cache": None if whole else v[0], "k_scales": k[1],
            "v_scales": v[1]}


def _exact_decode(s, case):
    hq, hkv, d = _heads(case)
    bs, t = case["block_size"], case["scale_tokens"]
    out = torch.zeros(s["q"].shape, dtype=F64, device=DEV)
    for b, n in enumerate(s["contexts"].tolist()):
        if n == 0:
            continue
        pages = s["tables"][b, :_ceil(n, bs)].long()
        k, v = ((s[name + "_cache"][pages].to(F64) * torch.repeat_interleave(s[name + "_scales"][pages], t, 1)[..., None])
                .reshape(-1, hkv, d)[:n].transpose(0, 1) for name in ("k", "v"))
        q = s["q"][b].to(F64).view(hkv, hq // hkv, d)
        out[b] = (torch.softmax(q @ k.transpose(1, 2) / math.sqrt(d), dim=-1) @ v).view(hq, d)
    return {"out": out}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return {name: _exact_turned(s[name], case, s["positions"]) for name in ("q", "k")}
    if case["op"] == "load":
        k, v = ((s[name + "_cache"].to(F64), s[name + "_scales"].to(F64)) for name in ("k", "v"))
        return _exact_read(s, case, k, v)
    return (_exact_store if case["op"] == "store" else _exact_decode)(s, case)
