"""The 8-bit cache where its numbers lie far apart, on the GPU against 64-bit
definitions.

Tolerances of decode: bf16 output 2^-8 |out|; weights p * scale rounded to fp16, by
2^-11 of each, so 2^-11 sum p |v|; and the same again for the scores' own error (below
2^-13 here) and for weights beyond 2^-25 of the largest, which a gap of 26 has some of:
2^-36 of it, 2^-9 of themselves, in either direction.  Nothing in them grows with the
context.
"""
import math

import pytest
import torch

import paged_kv_cache_125_gb300 as kvp
import quant_reference as ref
from test_gpu_quant import (DEV, E4M3, INT8, assert_decode, bf16, bits, cache_arrays, clean_status,  # noqa: F401
                            decode_case, f32, f64, gen, i32, randn, run_decode, to_dev)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------- decode: one dominant key

def dominated(hq, hkv, d, t, dtype, n, at, gap, seed, v_scale=None):
    """One sequence whose key `at` counts about 2^gap times as much as any other; its values are zero in the first
    half of the columns, the others' have a mean of a half.  -> q of three rows, arrays, tables, softmax scale."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    bs = 256
    blocks = -(-n // bs)
    size = 1.0 if dtype == E4M3 else 0.25
    k_scale, v_scale = 2.0 ** -5 / size, v_scale or 2.0 ** -6 / size

    def codes(mean, spread):
        x = torch.empty((blocks * bs, hkv, d), device=DEV).normal_(mean, spread, generator=g)
        return x.clamp_(-ref.LIMIT[dtype], ref.LIMIT[dtype])

    # scores (natural): 2 * k[0] and a spread of a half
    k, v = codes(0.0, 8.0 * size), codes(32.0 * size, 64.0 * size)
    k[at], k[at, :, 0] = 0.0, gap * math.log(2) / 2 / k_scale
    v[at, :, :d // 2] = 0.0
    arrays = [(x.round() if dtype == INT8 else x).to(dtype).view(blocks, bs, hkv, d) for x in (k, v)]
    scales = [torch.full((blocks, bs // t, hkv), s, device=DEV) for s in (k_scale, v_scale)]
    q = torch.empty((3, hq, d), device=DEV).normal_(generator=g)
    q[:, :, 0] = 16.0
    tables = torch.randperm(blocks, generator=g, device=DEV).to(i32)[None]
    for x in arrays + scales:  # pages in the table's order
        x.view(torch.uint8)[tables[0].long()] = x.view(torch.uint8).clone()
    return q.to(bf16), arrays, scales, tables, 0.125


def check_dominated(q, arrays, scales, tables, scale, n):
    """One sequence shared by many CTAs, and as many sequences as CTAs, none of them cut."""
    want, size, _ = ref.decode(q, *((c.to(f32), s) for c, s in zip(arrays, scales)), tables.expand(3, -1), [n] * 3, scale)
    tol = 2.0 ** -8 * want.abs() + 2 * 2.0 ** -11 * size
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    for rows in (1, sms):
        out = kvp.attn_decode_quant(q[torch.arange(rows, device=DEV) % 3], *arrays, *scales,
                                    tables.expand(rows, -1).contiguous(),
                                    torch.full((rows,), n, dtype=i32, device=DEV), n, softmax_scale=scale)
        for b in {0, rows // 2, rows - 1}:
            off = (out[b].cpu().to(f64) - want[b % 3]).abs()
            assert bool((off <= tol[b % 3]).all()), (rows, b, (off / size[b % 3]).max().item())
    assert kvp.device_status() == 0


@pytest.mark.parametrize("gap", [8, 18, 22, 24, 26])
@pytest.mark.parametrize("hq,hkv,d,t,dtype,n,at", [
    (8, 8, 64, 16, E4M3, 131072, 0), (16, 8, 128, 4, INT8, 65536, 0), (8, 1, 128, 16, E4M3, 131072, 0),
    (32, 8, 128, 16, E4M3, 40000, 20000), (64, 8, 64, 32, INT8, 30001, 30000), (4, 4, 128, 1, E4M3, 32768, 100)])
def test_decode_one_key_outweighs_a_long_context(hq, hkv, d, t, dtype, n, at, gap):
    """What lies behind a key that takes nearly all of the weight: each of the other weights keeps its bits, however
    many they are."""
    q, arrays, scales, tables, scale = dominated(hq, hkv, d, t, dtype, n, at, gap, n + gap)
    check_dominated(q, arrays, scales, tables, scale, n)


@pytest.mark.parametrize("dtype,power", [(E4M3, 60), (E4M3, 100), (E4M3, 119), (INT8, 100), (INT8, 120), (E4M3, -64), (INT8, -60)])
@pytest.mark.parametrize("gap", [7, 20])
def test_decode_values_of_any_size(dtype, power, gap):
    """V's scales from the least to the largest that bf16 rows give."""
    for hq, hkv, d, t in ((16, 8, 128, 16), (2, 2, 64, 4)):
        q, arrays, scales, tables, scale = dominated(hq, hkv, d, t, dtype, 20000, 0, gap, power, v_scale=2.0 ** power)
        check_dominated(q, arrays, scales, tables, scale, 20000)


# ------------------------------------------------------------- decode: workspace

@pytest.mark.parametrize("heads", [(16, 8, 128), (8, 1, 128), (2, 1, 64), (64, 8, 64)])
def test_decode_workspace_of_a_larger_batch_serves(heads):
    """No smaller batch, and none of shorter contexts, needs more."""
    bounds = [0, 1, 16, 64, 96, 97, 192, 256, 257, 512, 1024, 2048, 4096, 100000]
    below = [0] * len(bounds)
    for n in range(0, 400):
        need = [kvp.attn_decode_quant_workspace_size(n, *heads, bound) for bound in bounds]
        assert need == sorted(need), n
        assert all(a <= b for a, b in zip(below, need)), n
        below = need


def test_decode_batches_in_one_workspace():
    ws = torch.empty((kvp.attn_decode_quant_workspace_size(64, 16, 8, 128, 256),), dtype=torch.uint8, device=DEV)
    for n in (64, 48, 47, 32, 1):
        lens = [256 - 3 * i for i in range(n)]
        q, host, dev, tables = decode_case(16, 8, 128, 64, 16, E4M3, lens, n, poison=False)
        out = run_decode(q[:, :16], dev, tables, lens, longest=256, workspace=ws)
        assert_decode(out, q[:, :16], host, tables, lens, 128 ** -0.5)
    assert kvp.device_status() == 0


# -------------------------------------------------- store: scales that mean nothing

@pytest.mark.parametrize("dtype", [E4M3, INT8])
@pytest.mark.parametrize("t", [2, 8, 64])
def test_store_over_scales_that_mean_nothing(t, dtype):
    """A block that is continued over a scale of NaN, zero, below zero or infinity: the new rows' own scale, and zeros
    in the place of every other code, those that are NaN among them."""
    present = torch.tensor([math.nan, 0.0, -1.0, math.inf, -math.inf, -0.0, -math.nan])
    b, bs = len(present), 64
    codes = torch.randint(0, 256, (b, bs, 2, 64), generator=gen(t), dtype=torch.uint8)
    codes[:, 0], codes[:, bs - 1] = 0x7F, 0xFF
    scales = present[:, None, None].expand(b, bs // t, 2).contiguous()
    dev = [to_dev(codes.view(dtype), scales) for _ in range(2)]
    x = randn((b, 4, 64), gen(t + 1)).to(DEV)
    place = t - 1
    slots = torch.arange(b, dtype=i32) * bs + place
    kvp.kv_quant_store(x[:, :2], x[:, 2:], slots.to(DEV), dev[0][0], dev[1][0], dev[0][1], dev[1][1])
    for (c, s), rows in zip(dev, (x[:, :2], x[:, 2:])):
        rows = rows.cpu().to(f64)
        need = torch.tensor([[ref.scale_for(r.abs().max().item(), dtype) for r in head] for head in rows], dtype=f64)
        assert torch.equal(s[:, 0].cpu().to(f64), need)
        got = c.cpu()[:, :t].to(f32).to(f64)
        assert torch.equal(got[:, place], ref.encode(rows / need[..., None], dtype))
        assert not got[:, :place].any() and not torch.isnan(got).any()
        if t < bs:
            assert torch.equal(bits(c)[:, t:], codes[:, t:])
    assert kvp.device_status() == 0


# -------------------------------------------------------- decode: keys that are NaN

def test_decode_keys_that_are_nan():
    """A NaN key makes its kv head's outputs NaN, also where it fills the parts of many CTAs and no other."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    n = sms * 64  # four units of 16 tokens for each CTA
    q, host, dev, tables = decode_case(16, 8, 128, 256, 16, E4M3, [n], 61, poison=False)
    want = run_decode(q[:, :16], dev, tables, [n])
    codes = dev[0][0].view(torch.uint8)
    for first, last in ((0, 64 * 64), (5, 6), (n - 1, n), (0, n)):
        held = codes.clone()
        for p in range(first, last):
            codes[int(tables[0, p // 256]), p % 256, 3] = 0x7F
        out = run_decode(q[:, :16], dev, tables, [n])
        assert bool(torch.isnan(out[0, 6:8]).all()), (first, last)
        assert torch.equal(out[0, :6], want[0, :6]) and torch.equal(out[0, 8:], want[0, 8:])
        codes.copy_(held)


# ----------------------------------------------------------------- pages of the cache

def stacked_cache(blocks, bs, t, hkv, d, dtype, g):
    """K and V as planes of one allocation: codes [2, blocks, ...], scales [2, blocks, ...]."""
    (kc, ks), (vc, vs) = (cache_arrays(blocks, bs, t, hkv, d, dtype, g) for _ in range(2))
    return torch.stack((kc.view(torch.uint8), vc.view(torch.uint8))).to(DEV), torch.stack((ks, vs)).to(DEV)


def decode_stacked(q, codes, scales, dtype, tables, lens):
    return kvp.attn_decode_quant(q, codes[0].view(dtype), codes[1].view(dtype), scales[0], scales[1], tables, lens, 100)


def copy_scales(scales, pairs):
    """kv_copy_blocks of the scales, as 16-bit numbers of planes [blocks, scale blocks, kv heads, 2]."""
    pairs = torch.tensor(pairs, dtype=i32, device=DEV).view(-1, 2)
    kvp.kv_copy_blocks(scales.view(bf16).view(*scales.shape, 2), pairs)


@pytest.mark.parametrize("dtype", [E4M3, INT8])
@pytest.mark.parametrize("hkv,d,bs,t", [(2, 64, 32, 8), (1, 128, 16, 16), (3, 64, 48, 1)])
def test_pages_forked_and_compacted(hkv, d, bs, t, dtype):
    """kv_pages_fork and kv_pages_compact move the codes; the caller copies the scales of the pages that moved."""
    g = gen(bs + t)
    hq = hkv if hkv == 3 else 2 * hkv
    blocks, lens = 16, [bs + 5, 3, 2 * bs, 0]
    codes, scales = stacked_cache(blocks, bs, t, hkv, d, dtype, g)
    tables = torch.tensor([[9, 4, -1], [11, -1, -1], [2, 13, -1], [-1, -1, -1]], dtype=i32)
    counts = torch.zeros((blocks,), dtype=i32)
    counts[[9, 4, 11, 2, 13]] = 1
    lens_dev = torch.tensor(lens, dtype=i32, device=DEV)
    x = randn((6, hq + 2 * hkv, d), g).to(DEV)
    parents = [0, 0, 1, 2, 1, 0]

    def attend(tab, ctx, q):  # (decode takes 1, 2, 4 or 8 kv heads: otherwise the rows themselves)
        if hkv != 3:
            return decode_stacked(q, codes, scales, dtype, tab, ctx)
        n = ctx.tolist()
        starts = torch.tensor([sum(n[:i]) for i in range(len(n))], dtype=i32, device=DEV)
        k, v = kvp.kv_quant_load(codes[0].view(dtype), codes[1].view(dtype), *scales, tab, ctx, starts, max(n), num_rows=sum(n))
        return [torch.cat((k[a:a + m], v[a:a + m])) for a, m in zip(starts.tolist(), n)]

    want = attend(tables.to(DEV), lens_dev, x[:4, :hq])
    pool = codes.view(bf16)
    tab, ctx, cnt = kvp.kv_pages_fork(pool, tables.to(DEV), lens_dev, counts.to(DEV),
                                      torch.tensor(parents, dtype=i32, device=DEV))
    # a forked row whose last page is another than its parent's has a copy of it
    pairs = []
    for r, (p, n) in enumerate(zip(parents, ctx.tolist())):
        last = (n - 1) // bs
        src, dst = int(tables[p, last]), int(tab[r, last])
        if src != dst:
            pairs.append((src, dst))
    assert len(pairs) == 3
    copy_scales(scales, pairs)
    got = attend(tab, ctx, x[parents, :hq])
    for r, p in enumerate(parents):
        assert torch.equal(got[r], want[p]), r
    # each goes on by itself
    slots = torch.tensor([int(tab[r, n // bs]) * bs + n % bs if n % bs else -1 for r, n in enumerate(ctx.tolist())],
                         dtype=i32, device=DEV)
    kvp.kv_quant_store(8 * x[:, hq:hq + hkv], 8 * x[:, hq + hkv:], slots, codes[0].view(dtype), codes[1].view(dtype), *scales)
    ctx = ctx + (slots >= 0).to(i32)
    want = attend(tab, ctx, x[:, :hq])
    assert not torch.equal(want[0], want[1])
    # compact: places has the new id of every page
    tab, cnt, places = kvp.kv_pages_compact(pool, tab, ctx, cnt)
    copy_scales(scales, [(p, q) for p, q in enumerate(places.tolist()) if q >= 0 and q != p])
    got = attend(tab, ctx, x[:, :hq])
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert kvp.device_status() == 0


# ---------------------------------------------------------- decode: none of them cut

@pytest.mark.parametrize("dtype", [E4M3, INT8])
@pytest.mark.parametrize("hq,hkv,d,bs,t", [(16, 8, 128, 256, 16), (8, 8, 128, 24, 8), (64, 8, 64, 64, 32), (16, 4, 128, 128, 128),
                                           (8, 1, 128, 256, 64), (2, 1, 64, 16, 1), (8, 2, 64, 512, 256)])
@pytest.mark.parametrize("seqs,stages", [(12, 6), (60, 16)])
def test_decode_short_contexts_in_one_launch(hq, hkv, d, bs, t, dtype, seqs, stages):
    """Up to six stages of a sequence (16, where sequences are many) no sequence is cut: a stage holds 8 pieces of 16
    tokens and a kv head of 128, or 16 of 64."""
    longest = stages * 16 * (8 if d == 128 else 16) // hkv
    lens = [(longest - 5 * i) % (longest + 1) for i in range(seqs - 2)] + [0, 1]
    q, host, dev, tables = decode_case(hq, hkv, d, bs, t, dtype, lens, seqs + d)
    host = [(torch.nan_to_num(h[0].to(f32)), torch.nan_to_num(h[1])) for h in host]
    for bound in (longest, longest + 1):  # the largest that is not cut, the least that is
        out = run_decode(q[:, :hq], dev, tables, lens, longest=bound)
        assert_decode(out, q[:, :hq], host, tables, lens, d ** -0.5)
    assert kvp.device_status() == 0


# ------------------------------------------------------------- the rotating store

def test_store_rope_without_queries():
    """num_heads 0 of the C call: only k and v; the same codes as with queries beside them."""
    g = gen(71)
    n, hkv, d, t, bs = 40, 2, 64, 8, 32
    x = randn((n, 3 * hkv, d), g).to(DEV)
    q, k, v = x[:, :hkv], x[:, hkv:2 * hkv], x[:, 2 * hkv:]
    pos, slots = torch.arange(n, device=DEV), torch.arange(n, dtype=i32, device=DEV)
    freqs, magnitude = kvp.attn_rope_freqs(d, device=DEV)
    host = [cache_arrays(3, bs, t, hkv, d, E4M3, g) for _ in range(2)]
    both, alone = ([to_dev(*h) for h in host] for _ in range(2))
    kvp.kv_quant_store_rope(q, k, v, pos, slots, freqs, both[0][0], both[1][0], both[0][1], both[1][1], magnitude)
    rc = kvp.library().kv_quant_store_rope(
        None, 0, k.data_ptr(), v.data_ptr(), k.stride(0), v.stride(0), pos.data_ptr(), slots.data_ptr(), n,
        freqs.data_ptr(), d, 0, magnitude, 0, None, 0, alone[0][0].data_ptr(), alone[1][0].data_ptr(),
        alone[0][1].data_ptr(), alone[1][1].data_ptr(), 0, 3, bs, t, hkv, d, torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    for a, b in zip(both, alone):
        assert torch.equal(bits(a[0]), bits(b[0])) and torch.equal(a[1], b[1])
    assert kvp.device_status() == 0
