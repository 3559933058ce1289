"""Workloads of the operators around shared pages of the paged KV cache.

Four operators:

* decode: one query token per sequence over its paged history, in a batch
  whose sequences share long prefixes (``attn_shared_plan`` followed by one
  ``attn_decode_shared`` or ``attn_decode_shared_append`` per layer).
* fork: new rows of a block table from old ones (parallel sampling, beam
  search), with reference counts and copy on write (``kv_pages_fork``).
* extend: pages and slots for each row's new tokens (``kv_pages_extend``).
* compact: live pages moved to the front of the pool (``kv_pages_compact``).

``run`` computes a case in its plain form (elementary torch operations, fp32)
or, with ``own`` set, through the library's calls.  ``exact`` has the same
results in 64 bits, from the definitions.
"""
import math

import torch

own = False

BF16, I32, F32, F64 = torch.bfloat16, torch.int32, torch.float32, torch.float64
DEV = "cuda"


# --------------------------------------------------------------------- cases

def _decode(name, heads, block_size, groups, per_group, prefix, lo, hi, layers=1, append=False, singles=0,
            padding=0):
    case = {"op": "decode", "heads": heads, "block_size": block_size, "groups": groups, "per_group": per_group,
            "prefix": prefix, "suffix_lo": lo, "suffix_hi": hi, "layers": layers, "append": append,
            "singles": singles, "padding": padding}
    return case if name is None else {"name": name, **case}


def _fork(name, heads, block_size, prompts, beams, survivors, lo, hi, layers):
    case = {"op": "fork", "heads": heads, "block_size": block_size, "prompts": prompts, "beams": beams,
            "survivors": survivors, "len_lo": lo, "len_hi": hi, "layers": layers}
    return case if name is None else {"name": name, **case}


def _extend(name, block_size, rows, len_lo, len_hi, new_lo, new_hi):
    case = {"op": "extend", "block_size": block_size, "rows": rows, "len_lo": len_lo, "len_hi": len_hi,
            "new_lo": new_lo, "new_hi": new_hi}
    return case if name is None else {"name": name, **case}


def _compact(name, heads, block_size, pages, live, layers):
    case = {"op": "compact", "heads": heads, "block_size": block_size, "pages": pages, "live": live,
            "layers": layers}
    return case if name is None else {"name": name, **case}


def listed():
    return [
        # a few samples of one short prompt on a tiny model: latency alone
        _decode("decode_tiny", "2/1/64", 16, 1, 3, 32, 1, 20),
        # a small interactive batch behind one system prompt, four layers under one plan
        _decode("decode_chat_8", "16/8/128", 256, 1, 8, 1024, 1, 300, layers=4, append=True),
        # the benchmark's decode batch, all requests behind one 2048-token prompt, padded to a graph's bucket
        _decode("decode_b64", "16/8/128", 256, 1, 62, 2048, 100, 1500, append=True, padding=2),
        # parallel sampling: 16 prompts with 8 samples each, and a few requests that share nothing
        _decode("decode_samples_16x8", "32/8/128", 16, 16, 8, 1200, 17, 700, append=True, singles=5),
        # eight query heads per kv head: best-of-16 on one long document
        _decode("decode_long_document", "64/8/128", 256, 1, 16, 32768, 1, 64),
        # the largest serving batch behind one long prompt
        _decode("decode_b512", "32/8/128", 256, 1, 512, 8192, 64, 1000, append=True),
        # a beam step of one prompt on a tiny model: latency alone
        _fork("fork_tiny", "2/1/64", 16, 1, 4, 2, 37, 37, 2),
        # a beam step of 32 prompts with 8 beams over 8 layers
        _fork("fork_beams_32x8", "16/8/128", 256, 32, 8, 3, 300, 1900, 8),
        # a decode step's new token for the largest batch, small pages
        _extend("extend_decode_512", 16, 512, 128, 8000, 1, 1),
        # admission of a step's prompts, ragged
        _extend("extend_prompts_24", 256, 24, 0, 0, 1, 1400),
        # a small pool after a few requests left
        _compact("compact_small", "2/1/64", 16, 48, 0.4, 2),
        # half of a pool of 8 layers is free, in holes
        _compact("compact_half", "16/8/128", 256, 1024, 0.5, 8),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


_HEADS = ["2/1/64", "4/2/64", "16/8/64", "8/8/128", "16/8/128", "32/8/128", "64/8/128", "8/1/128", "16/4/128"]


def draw(rng):
    """One more case of the ranges that the listed ones stand for."""
    op = rng.choice(["decode", "decode", "decode", "fork", "extend", "compact"])
    block_size = rng.choice([16, 32, 64, 128, 256])
    heads = rng.choice(_HEADS)
    if op == "decode":
        groups = _log_int(rng, 1, 24)
        per_group = _log_int(rng, 2, max(2, 400 // groups))
        prefix = _log_int(rng, block_size, 24000)
        hi = _log_int(rng, 2, 2500)
        # at most the largest listed case's keys over all sequences
        while groups * per_group * (prefix + hi) > 4_000_000:
            prefix, hi = max(block_size, prefix // 2), max(2, hi // 2)
        return _decode(None, heads, block_size, groups, per_group, prefix, rng.randint(1, hi), hi,
                       layers=rng.choice([1, 1, 2]), append=rng.random() < 0.5, singles=rng.choice([0, 0, 1, 7]),
                       padding=rng.choice([0, 0, 3]))
    if op == "fork":
        beams = rng.randint(2, 12)
        hi = _log_int(rng, 2, 3000)
        return _fork(None, heads, block_size, _log_int(rng, 1, 24), beams, rng.randint(1, beams),
                     rng.randint(1, hi), hi, rng.choice([1, 2, 4, 6]))
    if op == "extend":
        hi = _log_int(rng, 1, 6000)
        new = _log_int(rng, 1, 500)
        return _extend(None, block_size, _log_int(rng, 1, 600), rng.randint(0, hi), hi, rng.randint(0, new), new)
    return _compact(None, heads, block_size, _log_int(rng, 8, 900), round(rng.uniform(0.05, 0.95), 3),
                    rng.choice([1, 2, 4, 6]))


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


def _prefix_pages(case):
    """Whole pages of the shared prefix (the engine shares full pages only)."""
    return case["prefix"] // case["block_size"]


def _suffixes(case):
    n = case["groups"] * case["per_group"] + case["singles"]
    return _spread(n, case["suffix_lo"], case["suffix_hi"])


def _prepare_decode(case, g):
    bs, pp = case["block_size"], _prefix_pages(case)
    hq, hkv, d = _heads(case)
    lens = _shuffled(_suffixes(case), g)
    in_groups = case["groups"] * case["per_group"]
    own_pages = [_ceil(n, bs) for n in lens]
    blocks = case["groups"] * pp + sum(own_pages) + 3
    ids = torch.randperm(blocks, generator=g, device=DEV).tolist()
    at = 0
    tables, contexts, slots = [], [], []
    shared = []
    for i, (n, pages) in enumerate(zip(lens, own_pages)):
        if i < in_groups and i % case["per_group"] == 0:
            shared, at = ids[at:at + pp], at + pp
        row = (shared if i < in_groups else []) + ids[at:at + pages]
        at += pages
        tables.append(row)
        contexts.append((pp * bs if i < in_groups else 0) + n)
        slots.append(row[-1] * bs + (n - 1) % bs)
    # padding rows of a graph's bucket
    tables += [[]] * case["padding"]
    contexts += [0] * case["padding"]
    slots += [-1] * case["padding"]
    width = max(len(r) for r in tables)
    tables = torch.tensor([r + [-1] * (width - len(r)) for r in tables], dtype=I32, device=DEV)
    batch, layers = len(contexts), case["layers"]
    cache = torch.empty((2, layers, blocks, bs, hkv, d), dtype=BF16, device=DEV).normal_(generator=g)
    q = torch.empty((layers, batch, hq, d), dtype=BF16, device=DEV).normal_(generator=g)
    k = torch.empty((layers, batch, hkv, d), dtype=BF16, device=DEV).normal_(generator=g)
    v = torch.empty((layers, batch, hkv, d), dtype=BF16, device=DEV).normal_(generator=g)
    state = {"cache": cache, "q": q, "k": k, "v": v, "tables": tables,
             "contexts": torch.tensor(contexts, dtype=I32, device=DEV),
             "slots": torch.tensor(slots, dtype=I32, device=DEV)}
    if own:
        import paged_kv_cache_125_gb300 as kvp
        # scratch that a serving loop keeps: the plan's buffer and the attention's workspace
        state["plan"] = torch.empty((kvp.attn_shared_plan_size(batch, hq, hkv),), dtype=torch.uint8, device=DEV)
        state["workspace"] = torch.empty((kvp.attn_decode_shared_workspace_size(batch, hq, hkv, d),),
                                         dtype=torch.uint8, device=DEV)
    return state


def _prepare_fork(case, g):
    bs, beams = case["block_size"], case["beams"]
    _, hkv, d = _heads(case)
    lens = _shuffled(_spread(case["prompts"], case["len_lo"], case["len_hi"]), g)
    full = [n // bs for n in lens]
    tails = [1 if n % bs else 0 for n in lens]
    rows = case["prompts"] * beams
    blocks = sum(full) + beams * sum(tails) + rows + 2
    ids = torch.randperm(blocks, generator=g, device=DEV).tolist()
    at = 0
    tables, contexts, parents = [], [], []
    counts = [0] * blocks
    for p in range(case["prompts"]):
        shared, at = ids[at:at + full[p]], at + full[p]
        for page in shared:
            counts[page] = beams
        for _ in range(beams):
            tail, at = ids[at:at + tails[p]], at + tails[p]
            for page in tail:
                counts[page] = 1
            tables.append(shared + tail)
            contexts.append(lens[p])
        chosen = torch.randperm(beams, generator=g, device=DEV).tolist()[:case["survivors"]]
        parents += [p * beams + chosen[b] for b in _shuffled([b % case["survivors"] for b in range(beams)], g)]
    width = max(1, max(len(r) for r in tables))
    return {"cache": torch.empty((2, case["layers"], blocks, bs, hkv, d), dtype=BF16, device=DEV).normal_(generator=g),
            "tables": torch.tensor([r + [-1] * (width - len(r)) for r in tables], dtype=I32, device=DEV),
            "contexts": torch.tensor(contexts, dtype=I32, device=DEV),
            "counts": torch.tensor(counts, dtype=I32, device=DEV),
            "parents": torch.tensor(parents, dtype=I32, device=DEV)}


def _others(pages):
    """Pages of the pool that other requests hold (waiting ones, or a kept prefix)."""
    return 8 + pages // 8


def _prepare_extend(case, g):
    bs, n = case["block_size"], case["rows"]
    lens = _shuffled(_spread(n, case["len_lo"], case["len_hi"]), g)
    new = _shuffled(_spread(n, case["new_lo"], case["new_hi"]), g)
    pages = [_ceil(x, bs) for x in lens]
    width = max(1, _ceil(case["len_hi"] + case["new_hi"], bs))
    added = sum(_ceil(a + b, bs) - _ceil(a, bs) for a, b in zip(lens, new))
    held, others = sum(pages), _others(sum(pages) + added)
    blocks = held + added + others + 5
    ids = torch.randperm(blocks, generator=g, device=DEV)
    used = ids[:held].to(I32)
    per_row = torch.tensor(pages, device=DEV)
    column = torch.arange(width, device=DEV)
    inside = column < per_row[:, None]
    tables = torch.full((n, width), -1, dtype=I32, device=DEV)
    tables[inside] = used
    counts = torch.zeros(blocks, dtype=I32, device=DEV)
    counts[ids[:held + others]] = 1
    return {"tables": tables, "contexts": torch.tensor(lens, dtype=I32, device=DEV), "counts": counts,
            "new": torch.tensor(new, dtype=I32, device=DEV), "total": sum(new), "block_size": bs}


def _prepare_compact(case, g):
    bs, blocks = case["block_size"], case["pages"]
    _, hkv, d = _heads(case)
    live = _live(case)
    ids = torch.randperm(blocks, generator=g, device=DEV).tolist()[:live]
    # rows of 1, 2, 3, ... 8 pages; the first two rows of a pool share their first page
    tables, at, n = [], 0, 1
    counts = [0] * blocks
    while at < live:
        tables.append(ids[at:at + n])
        at, n = at + n, n % 8 + 1
    for row in tables:
        for page in row:
            counts[page] += 1
    if len(tables) > 1:
        tables[1] = tables[0][:1] + tables[1]
        counts[tables[0][0]] += 1
    fill = _shuffled(_spread(len(tables), 1, bs), g)
    contexts = [(len(r) - 1) * bs + f for r, f in zip(tables, fill)]
    return {"cache": torch.empty((2, case["layers"], blocks, bs, hkv, d), dtype=BF16, device=DEV).normal_(generator=g),
            "tables": torch.tensor([r + [-1] * (9 - len(r)) for r in tables], dtype=I32, device=DEV),
            "contexts": torch.tensor(contexts, dtype=I32, device=DEV),
            "counts": torch.tensor(counts, dtype=I32, device=DEV)}


def _live(case):
    return max(1, round(case["pages"] * case["live"]))


def prepare(case, seed):
    g = _gen(seed)
    make = {"decode": _prepare_decode, "fork": _prepare_fork, "extend": _prepare_extend,
            "compact": _prepare_compact}[case["op"]]
    return {"op": case["op"], "append": case.get("append", False), **make(case, g)}


# ---------------------------------------------------------------- plain forms

def _plain_attention(s, layer):
    """softmax(q K^T / sqrt(d)) V of every sequence over its own gathered keys."""
    kc, vc, q, ctx = s["cache"][0, layer], s["cache"][1, layer], s["q"][layer], s["contexts"]
    _, bs, hkv, d = kc.shape
    batch, hq, _ = q.shape
    if s["append"]:
        real = s["slots"] >= 0
        slots = s["slots"][real].long()
        kc.view(-1, hkv, d)[slots] = s["k"][layer][real]
        vc.view(-1, hkv, d)[slots] = s["v"][layer][real]
    pos = torch.arange(s["tables"].shape[1] * bs, device=DEV)
    seen = pos < ctx[:, None]
    slot = torch.where(seen, s["tables"].long()[:, pos // bs] * bs + pos % bs, 0)
    keys = kc.view(-1, hkv, d)[slot].permute(0, 2, 3, 1).to(F32)
    scores = torch.matmul(q.to(F32).view(batch, hkv, hq // hkv, d), keys) * d ** -0.5
    del keys
    scores = scores.masked_fill(~seen[:, None, None, :], -math.inf)
    top = scores.amax(-1, keepdim=True)
    weights = torch.exp(scores - torch.where(top == -math.inf, 0.0, top))
    total = weights.sum(-1, keepdim=True)
    del scores
    values = vc.view(-1, hkv, d)[slot].permute(0, 2, 1, 3).to(F32)
    out = torch.matmul(weights, values) / torch.where(total == 0, 1.0, total)
    return out.view(batch, hq, d).to(BF16)


def _plain_decode(s):
    out = torch.stack([_plain_attention(s, layer) for layer in range(s["q"].shape[0])])
    return {"out": out, "cache": s["cache"]} if s["append"] else {"out": out}


def _count_pages(counts, tables, inside, by):
    """counts + by for every table entry inside its row."""
    pages = torch.where(inside, tables, 0).long().view(-1)
    return counts.index_add(0, pages, (inside.to(I32) * by).view(-1))


def _free_pages(counts, n):
    """The lowest free pages, ascending (the first min(n, pages) entries of free-then-used order)."""
    return torch.argsort((counts != 0).to(I32), stable=True)[:n]


def _plain_fork(s):
    cache, tables, ctx, parents = s["cache"], s["tables"], s["contexts"], s["parents"].long()
    _, layers, blocks, bs, hkv, d = cache.shape
    rows, width = tables.shape
    column, row = torch.arange(width, device=DEV), torch.arange(rows, device=DEV)
    some, parent = parents >= 0, parents.clamp(min=0)
    new_ctx = torch.where(some, ctx[parent], 0).to(I32)
    pages = (new_ctx + bs - 1) // bs
    inside = column < pages[:, None]
    new = torch.where(inside, tables[parent], -1)
    counts = _count_pages(s["counts"], tables, column < ((ctx + bs - 1) // bs)[:, None], -1)
    counts = _count_pages(counts, new, inside, 1)
    fill = new_ctx % bs
    last = (pages - 1).clamp(min=0).long()
    tail = new.gather(1, last[:, None])[:, 0].clamp(min=0).long()
    first = torch.full((blocks,), rows, device=DEV).scatter_reduce(0, tail, torch.where(fill > 0, row, rows), "amin")
    copied = (fill > 0) & (first[tail] != row)
    counts = counts.index_add(0, tail, -copied.to(I32))
    target = _free_pages(counts, rows)[(torch.cumsum(copied, 0) - 1).clamp(min=0)]
    new.scatter_(1, last[:, None], torch.where(copied, target, new.gather(1, last[:, None])[:, 0].long()).to(I32)[:, None])
    counts[target[copied]] = 1
    token = torch.arange(bs, device=DEV)
    moved = copied[:, None] & (token < fill[:, None])
    flat = cache.view(2 * layers, blocks * bs, hkv * d)
    flat[:, (target[:, None] * bs + token)[moved]] = flat[:, (tail[:, None] * bs + token)[moved]]
    return {"tables": new, "contexts": new_ctx, "counts": counts, "cache": cache}


def _plain_extend(s):
    tables, ctx, new, bs = s["tables"], s["contexts"], s["new"], s["block_size"]
    rows, width = tables.shape
    new_ctx = ctx + new
    before, after = (ctx + bs - 1) // bs, (new_ctx + bs - 1) // bs
    need = after - before
    start = torch.cumsum(need, 0) - need
    column = torch.arange(width, device=DEV)
    added = (column >= before[:, None]) & (column < after[:, None])
    free = _free_pages(s["counts"], s["counts"].shape[0])
    rank = torch.where(added, start[:, None] + column - before[:, None], 0)
    new_tables = torch.where(added, free[rank].to(I32), torch.where(column < before[:, None], tables, -1))
    counts = _count_pages(s["counts"], new_tables, added, 1)
    row = torch.repeat_interleave(torch.arange(rows, device=DEV), new.long(), output_size=s["total"])
    pos = ctx[row] + torch.arange(s["total"], device=DEV) - (torch.cumsum(new, 0) - new)[row]
    slots = new_tables[row, (pos // bs)] * bs + pos % bs
    return {"tables": new_tables, "contexts": new_ctx, "counts": counts, "slots": slots.to(I32)}


def _plain_compact(s):
    cache, tables, counts = s["cache"], s["tables"], s["counts"]
    bs = cache.shape[3]
    live = counts > 0
    page = torch.arange(counts.shape[0], device=DEV)
    above = page >= live.sum()
    src, dst = (live & above).nonzero()[:, 0], (~live & ~above).nonzero()[:, 0]
    flat = cache.view(-1, *cache.shape[2:])
    flat[:, dst] = flat[:, src]
    places = torch.where(live, page, -1).to(I32)
    places[src] = dst.to(I32)
    new_counts = torch.where(live & ~above, counts, 0)
    new_counts[dst] = counts[src]
    inside = torch.arange(tables.shape[1], device=DEV) < ((s["contexts"] + bs - 1) // bs)[:, None]
    new = torch.where(inside, places[tables.clamp(min=0).long()], -1)
    return {"tables": new, "counts": new_counts, "places": places, "cache": cache}


# ------------------------------------------------------------ the library's calls

def _own_decode(s):
    import paged_kv_cache_125_gb300 as kvp
    cache, q, tables = s["cache"], s["q"], s["tables"]
    _, layers, blocks, bs, hkv, _ = cache.shape
    plan = kvp.attn_shared_plan(tables, s["contexts"], bs, q.shape[2], hkv, blocks, plan=s["plan"])
    out = torch.empty_like(q)
    if s["append"]:
        [kvp.attn_decode_shared_append(q[i], s["k"][i], s["v"][i], s["slots"], cache[0, i], cache[1, i], tables, plan,
                                       workspace=s["workspace"], out=out[i]) for i in range(layers)]
        return {"out": out, "cache": cache}
    [kvp.attn_decode_shared(q[i], cache[0, i], cache[1, i], tables, plan, workspace=s["workspace"], out=out[i])
     for i in range(layers)]
    return {"out": out}


def _own_fork(s):
    import paged_kv_cache_125_gb300 as kvp
    tables, contexts, counts = kvp.kv_pages_fork(s["cache"], s["tables"], s["contexts"], s["counts"], s["parents"])
    return {"tables": tables, "contexts": contexts, "counts": counts, "cache": s["cache"]}


def _own_extend(s):
    import paged_kv_cache_125_gb300 as kvp
    tables, contexts, counts, slots = kvp.kv_pages_extend(s["tables"], s["contexts"], s["counts"], s["new"],
                                                          s["block_size"], s["total"])
    return {"tables": tables, "contexts": contexts, "counts": counts, "slots": slots}


def _own_compact(s):
    import paged_kv_cache_125_gb300 as kvp
    tables, counts, places = kvp.kv_pages_compact(s["cache"], s["tables"], s["contexts"], s["counts"])
    return {"tables": tables, "counts": counts, "places": places, "cache": s["cache"]}


def run(state):
    if own:
        return {"decode": _own_decode, "fork": _own_fork, "extend": _own_extend, "compact": _own_compact}[state["op"]](state)
    return {"decode": _plain_decode, "fork": _plain_fork, "extend": _plain_extend,
            "compact": _plain_compact}[state["op"]](state)


# ---------------------------------------------------------------------- floors

def work(case):
    bs = case["block_size"]
    if case["op"] == "extend":
        rows, lens = case["rows"], _spread(case["rows"], case["len_lo"], case["len_hi"])
        new = _spread(rows, case["new_lo"], case["new_hi"])
        held = sum(_ceil(n, bs) for n in lens)
        # lengths may meet in any order: the pages that are added are counted as if they met as listed
        added = sum(_ceil(a + b, bs) - _ceil(a, bs) for a, b in zip(lens, new))
        width = max(1, _ceil(case["len_hi"] + case["new_hi"], bs))
        pool = held + added + _others(held + added) + 5
        return {"bytes": 4 * (held + rows * width + 3 * rows + 2 * pool + sum(new)), "flops": 0}
    hq, hkv, d = _heads(case)
    row = hkv * d * 2
    if case["op"] == "fork":
        lens = _spread(case["prompts"], case["len_lo"], case["len_hi"])
        rows = case["prompts"] * case["beams"]
        copied = sum(n % bs for n in lens) * (case["beams"] - case["survivors"])
        width = max(1, max(_ceil(n, bs) for n in lens))
        held = sum(n // bs for n in lens) + case["beams"] * sum(1 for n in lens if n % bs) + rows + 2
        entries = sum(_ceil(n, bs) for n in lens) * case["beams"]
        return {"bytes": 2 * copied * row * 2 * case["layers"] + 4 * (entries + rows * width + 3 * rows + 2 * held),
                "flops": 0}
    if case["op"] == "compact":
        live, pages = _live(case), case["pages"]
        moved = live * (pages - live) / pages  # live pages above the live count, on average
        return {"bytes": 2 * moved * bs * row * 2 * case["layers"] + 4 * (2 * pages + pages + 10 * live / 4), "flops": 0}
    lens = _suffixes(case)
    shared = _prefix_pages(case) * bs
    in_groups = case["groups"] * case["per_group"]
    batch = len(lens) + case["padding"]
    keys = case["groups"] * shared + sum(lens)  # keys read once
    seen = in_groups * shared + sum(lens)       # keys seen by a query head, over the batch
    entries = in_groups * _prefix_pages(case) + sum(_ceil(n, bs) for n in lens)
    per_layer = 2 * keys * row + 2 * batch * hq * d * 2
    if case["append"]:
        per_layer += 2 * len(lens) * row  # the new rows' stores (their reads stand among the keys)
    return {"bytes": case["layers"] * per_layer + 4 * (entries + batch * 2),
            "flops": case["layers"] * 4 * hq * d * seen}


# ------------------------------------------------------------ 64-bit definitions

def _exact_decode(s):
    cache = s["cache"]
    layers, bs, hkv = cache.shape[1], cache.shape[3], cache.shape[4]
    batch, hq, d = s["q"].shape[1:]
    tables, contexts, slots = s["tables"].tolist(), s["contexts"].tolist(), s["slots"].tolist()
    out = torch.zeros((layers, batch, hq, d), dtype=F64, device=DEV)
    for layer in range(layers):
        if s["append"]:
            for b, slot in enumerate(slots):
                if slot >= 0:
                    cache[0, layer, slot // bs, slot % bs] = s["k"][layer, b]
                    cache[1, layer, slot // bs, slot % bs] = s["v"][layer, b]
        for b, n in enumerate(contexts):
            if n == 0:
                continue
            pages = torch.tensor(tables[b][:_ceil(n, bs)], device=DEV)
            k = cache[0, layer, pages].reshape(-1, hkv, d)[:n].to(F64)
            v = cache[1, layer, pages].reshape(-1, hkv, d)[:n].to(F64)
            for g in range(hkv):
                heads = slice(g * (hq // hkv), (g + 1) * (hq // hkv))
                p = torch.softmax(s["q"][layer, b, heads].to(F64) @ k[:, g].T / math.sqrt(d), dim=-1)
                out[layer, b, heads] = p @ v[:, g]
    return {"out": out, "cache": cache} if s["append"] else {"out": out}


def _exact_fork(s):
    cache, bs = s["cache"], s["cache"].shape[3]
    tables, contexts = s["tables"].tolist(), s["contexts"].tolist()
    counts = s["counts"].tolist()
    for row, n in zip(tables, contexts):
        for page in row[:_ceil(n, bs)]:
            counts[page] -= 1
    new, kept, copies = [], set(), []
    for r, p in enumerate(s["parents"].tolist()):
        pages = tables[p][:_ceil(contexts[p], bs)] if p >= 0 else []
        fill = contexts[p] % bs if p >= 0 else 0
        if fill and pages[-1] in kept:
            copies.append((r, pages[-1], fill))
        elif fill:
            kept.add(pages[-1])
        for page in pages[:-1] if copies and copies[-1][0] == r else pages:
            counts[page] += 1
        new.append(list(pages))
    free = (page for page, c in enumerate(list(counts)) if c == 0)
    for r, src, fill in copies:
        dst = next(free)
        new[r][-1], counts[dst] = dst, 1
        cache[:, :, dst, :fill] = cache[:, :, src, :fill].clone()
    return {"tables": None, "contexts": None, "counts": None, "cache": cache}


def _exact_compact(s):
    cache, counts = s["cache"], s["counts"].tolist()
    live = [p for p, c in enumerate(counts) if c > 0]
    holes = iter([p for p in range(len(live)) if counts[p] == 0])
    for p in live:
        if p >= len(live):
            cache[:, :, next(holes)] = cache[:, :, p].clone()
    return {"tables": None, "counts": None, "places": None, "cache": cache}


def exact(case, seed):
    if case["op"] == "extend":
        return None  # whole numbers only
    s = prepare(case, seed)
    return {"decode": _exact_decode, "fork": _exact_fork, "compact": _exact_compact}[case["op"]](s)
