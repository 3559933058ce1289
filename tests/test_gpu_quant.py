"""Rotary positions and the 8-bit cache on the GPU against 64-bit definitions.

Tolerances (eps / 2 is half a step, relative: bf16 2^-8, e4m3 2^-4, fp16 2^-11):

* rope: one rounding to bf16, and angles whose cosines and sines are off by 2^-20
  (2^-21 of the fast functions, 2^-22 of the fp32 angle, its 2^-32 of a turn).
* store, load: exact.  Scales are powers of two and a code is one rounding, so
  codes and scales are equal; code * scale has at most 7 significant bits.
* rotated store: a code is off by half a step of what was rotated, plus the
  rotation's error; scales are equal where the largest number is no border case.
* decode: bf16 output 2^-8 |out|; weights p * scale rounded to fp16, by 2^-11 of
  each, so 2^-11 sum p |v|, or, where they are below 2^-14 of the largest, by
  fp16's least half step 2^-25 of what the largest counts (at least 1): 2^-25 of
  `unit`; fp32 scores off by at most d * 2^-24 * sum |q k| * scale, and p by as
  much of itself (below 2^-12 for the inputs here: 128 * 2^-24 * 32).
"""
import math

import pytest
import torch

import paged_kv_cache_125_gb300 as kvp
import quant_reference as ref

pytestmark = pytest.mark.gpu
bf16, i32, f32, f64 = torch.bfloat16, torch.int32, torch.float32, torch.float64
E4M3, INT8 = torch.float8_e4m3fn, torch.int8
DEV = "cuda"


@pytest.fixture(autouse=True)
def clean_status():
    kvp.device_status()
    yield
    torch.cuda.synchronize()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(shape, g, dtype=bf16):
    return torch.randn(shape, generator=g).to(dtype)


# ------------------------------------------------------------------------ rope

def rope_case(n, hq, hkv, d, r, interleaved, scaling, seed, far=1 << 20, strided=True, fast=True):
    g = gen(seed)
    rows = randn((n, hq + hkv + 1, d), g).to(DEV)
    q, k = rows[:, :hq], rows[:, hq:hq + hkv]
    if not strided:
        q, k = q.contiguous(), k.contiguous()
    pos = torch.randint(0, far, (n,), generator=g)
    low, high = {"yarn": (1.0, 32.0), "wavelength": (1.0, 4.0)}.get(scaling, (0.0, 0.0))
    inv, mag = ref.inverse_frequencies(r, 10000.0, scaling, 4.0, 2048, low, high)
    freqs, magnitude = kvp.attn_rope_freqs(r, 10000.0, scaling, 4.0, 2048, device=DEV)
    assert abs(magnitude - mag) < 1e-6
    return q, k, pos, inv, mag, freqs, magnitude


def assert_rope(got, x, pos, inv, mag, interleaved):
    want = ref.rope(x.cpu(), pos, inv, mag, interleaved)
    r = 2 * len(inv)
    size = x.cpu().to(f64).abs()
    pair = torch.zeros_like(size)
    if interleaved:
        pair[..., 0:r:2] = pair[..., 1:r:2] = size[..., 0:r:2] + size[..., 1:r:2]
    else:
        pair[..., :r // 2] = pair[..., r // 2:r] = size[..., :r // 2] + size[..., r // 2:r]
    # the angle's own error: freqs hold it to 2^-53 per position
    tol = 2.0 ** -8 * want.abs() + 2.0 ** -20 * mag * pair * (1 + 2.0 ** -7)
    off = (got.cpu().to(f64) - want).abs()
    assert bool((off <= tol).all()), (off - tol).max().item()
    assert torch.equal(got[..., r:].cpu(), x[..., r:].cpu())


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n,hq,hkv,d,r,scaling", [
    (1, 16, 8, 128, 128, "none"), (33, 2, 1, 64, 64, "linear"), (257, 16, 4, 128, 64, "yarn"),
    (100, 5, 3, 128, 32, "ntk"), (19, 32, 8, 128, 128, "wavelength"),
    (7, 3, 2, 64, 36, "none"), (11, 2, 1, 64, 2, "yarn"), (5, 1, 1, 36, 20, "ntk"), (3, 2, 2, 96, 48, "none"),
])
def test_rope(n, hq, hkv, d, r, scaling, interleaved):
    q, k, pos, inv, mag, freqs, magnitude = rope_case(n, hq, hkv, d, r, interleaved, scaling, n + r)
    q0, k0 = q.clone(), k.clone()
    oq, ok = kvp.attn_rope(q, k, pos.to(DEV), freqs, magnitude, interleaved)
    assert_rope(oq, q, pos, inv, mag, interleaved)
    assert_rope(ok, k, pos, inv, mag, interleaved)
    assert torch.equal(q, q0) and torch.equal(k, k0)
    only, none = kvp.attn_rope(q, None, pos.to(DEV), freqs, magnitude, interleaved)
    assert none is None and torch.equal(only, oq)
    # in place, within the projection's rows
    got = kvp.attn_rope(q, k, pos.to(DEV), freqs, magnitude, interleaved, out=(q, k))
    assert got[0].data_ptr() == q.data_ptr() and torch.equal(q, oq) and torch.equal(k, ok)


def test_rope_far_and_negative_positions():
    q, k, _, inv, mag, freqs, magnitude = rope_case(6, 2, 1, 64, 64, False, "none", 3)
    pos = torch.tensor([0, 1, (1 << 31) - 1, 1 << 31, -1, -5])
    oq, _ = kvp.attn_rope(q, k, pos.to(DEV), freqs)
    assert torch.equal(oq[0], q[0])
    # fp64 angles of 2^31 are off by 2^-22 themselves: within the tolerance's 2^-20
    assert_rope(oq, q, pos, inv, mag, False)


def test_rope_misaligned_rows():
    g = gen(5)
    flat = randn((1 + 9 * 2 * 64,), g).to(DEV)
    q = flat[1:].view(9, 2, 64)
    freqs, _ = kvp.attn_rope_freqs(64, device=DEV)
    inv, _ = ref.inverse_frequencies(64, 10000.0, "none", 1.0, 0, 0, 0)
    pos = torch.arange(9)
    oq, _ = kvp.attn_rope(q, None, pos.to(DEV), freqs)
    assert_rope(oq, q, pos, inv, 1.0, False)


def test_rope_undone_by_negative_positions():
    q, k, pos, inv, mag, freqs, magnitude = rope_case(40, 4, 2, 128, 128, False, "linear", 9)
    x = kvp.attn_rope(q, k, pos.to(DEV), freqs)
    y = kvp.attn_rope(x[0], x[1], -pos.to(DEV), freqs)
    # two roundings and two angles' errors of both numbers of a pair
    assert (y[0].float() - q.float()).abs().max().item() < 2 * 2 ** -8 * 1.5 * q.abs().max().item()


# -------------------------------------------------------------- a cache and steps

def cache_arrays(blocks, bs, t, hkv, d, dtype, g, poison=False):
    """Codes and scales, on the host."""
    if poison:
        codes = torch.full((blocks, bs, hkv, d), 0x7F, dtype=torch.uint8).view(dtype)
        scales = torch.full((blocks, bs // t, hkv), math.nan)
        return codes, scales
    x = torch.randn((blocks, bs, hkv, d), generator=g) * (ref.LIMIT[dtype] / 4)
    codes = x.clamp(-ref.LIMIT[dtype], ref.LIMIT[dtype])
    codes = (codes.round() if dtype == INT8 else codes).to(dtype)
    shift = 0 if dtype == E4M3 else 2
    scales = torch.exp2(torch.randint(-9, -5, (blocks, bs // t, hkv), generator=g).float() + shift)
    return codes, scales


def to_dev(*tensors):
    return tuple(t.to(DEV) for t in tensors)


def bits(t):
    return t.cpu().view(torch.uint8)


def assert_store(arrays, wanted, dtype):
    """Device arrays against code values and scales in fp64."""
    codes, scales = arrays
    want, want_scales = wanted
    got = codes.cpu().to(f32).to(f64)
    same = (got == want) | (torch.isnan(got) & torch.isnan(want))
    assert bool(same.all()), f"{(~same).sum().item()} codes differ"
    s = scales.cpu().to(f64)
    assert bool(((s == want_scales) | (torch.isnan(s) & torch.isnan(want_scales))).all())


CACHES = [(8, 128, 256, 16), (1, 64, 16, 16), (2, 64, 32, 1), (4, 128, 64, 64), (8, 128, 256, 256), (3, 128, 48, 8),
          (8, 64, 64, 4), (2, 128, 128, 128), (1, 128, 32, 32), (5, 64, 512, 256), (1, 128, 6, 2)]


@pytest.mark.parametrize("dtype", [E4M3, INT8])
@pytest.mark.parametrize("hkv,d,bs,t", CACHES)
def test_store_steps(hkv, d, bs, t, dtype):
    """A prefill of ragged sequences, a second chunk that ends inside a block, then
    decode steps, some with numbers that make scales grow."""
    g = gen(hkv * 1000 + d + bs + t)
    lens = [1, bs, bs + 1, max(1, 2 * bs - 3), 37]
    blocks = sum(-(-(n + 40) // bs) for n in lens) + 2
    ids = torch.randperm(blocks, generator=g).tolist()
    tables = [[ids.pop() for _ in range(-(-(n + 40) // bs))] for n in lens]
    host = [cache_arrays(blocks, bs, t, hkv, d, dtype, g) for _ in range(2)]
    dev = [to_dev(*h) for h in host]
    want = [(h[0].to(f32).to(f64), h[1].to(f64)) for h in host]
    done = [0] * len(lens)
    for step in range(6):
        new = [(n if step == 0 else 1 + 5 * i if step == 1 else 1) for i, n in enumerate(lens)]
        slots, grow = [], []
        for i, n in enumerate(new):
            slots += [tables[i][p // bs] * bs + p % bs for p in range(done[i], done[i] + n)]
            grow += [4.0 ** ((step + i) % 3) if step >= 1 else 1.0] * n
            done[i] += n
        if step == 2:  # a padded bucket
            slots += [-1, -1]
            grow += [1.0, 1.0]
        slots = torch.tensor(slots, dtype=i32)
        rows = [(torch.randn((len(slots), hkv + 1, d), generator=g) * torch.tensor(grow)[:, None, None]).to(bf16)
                for _ in range(2)]
        if step == 3:
            rows[0][0] = 0
            rows[1][0, 0, :3] = torch.tensor([math.inf, -math.inf, math.nan])
        k, v = (r.to(DEV)[:, :hkv] for r in rows)
        kvp.kv_quant_store(k, v, slots.to(DEV), dev[0][0], dev[1][0], dev[0][1], dev[1][1])
        for r, (codes, scales) in zip(rows, want):
            ref.store(r[:, :hkv].to(f64), slots, codes, scales, dtype)
        for d_, w in zip(dev, want):
            assert_store(d_, w, dtype)
    assert kvp.device_status() == 0


def test_store_extreme_numbers():
    """Zeros, the smallest and largest bf16 numbers, and border cases of the scale."""
    for dtype in (E4M3, INT8):
        limit = ref.LIMIT[dtype]
        tops = [0.0, 2.0 ** -133, 2.0 ** -64 * limit, 2.0 ** -63 * limit, 1.0, limit, limit * 2, 3.38e38, 1e30,
                limit * 2.0 ** -70, limit * 1.0078125 if dtype == E4M3 else 128.0]
        n = len(tops)
        x = torch.zeros((n, 1, 64))
        for i, top in enumerate(tops):
            x[i, 0] = torch.linspace(-1, 1, 64) * top
        x = x.to(bf16)
        host = [cache_arrays(1, n + 5, 1, 1, 64, dtype, gen(1)) for _ in range(2)]
        dev = [to_dev(*h) for h in host]
        slots = torch.arange(n, dtype=i32)
        kvp.kv_quant_store(x.to(DEV), x.to(DEV), slots.to(DEV), dev[0][0], dev[1][0], dev[0][1], dev[1][1])
        for h, d_ in zip(host, dev):
            w = (h[0].to(f32).to(f64), h[1].to(f64))
            ref.store(x.to(f64), slots, *w, dtype)
            assert_store(d_, w, dtype)


def test_store_scales_that_mean_nothing():
    """A block that is continued over a scale of NaN, zero, below zero or infinity, and over one that is no
    power of two."""
    for dtype in (E4M3, INT8):
        codes, _ = cache_arrays(5, 8, 8, 1, 64, dtype, gen(2))
        scales = torch.tensor([math.nan, 0.0, -1.0, 0.3, 1e-3]).view(5, 1, 1)
        dev = [to_dev(codes.clone(), scales.clone()) for _ in range(2)]
        x = randn((5, 1, 64), gen(3))
        slots = torch.arange(5, dtype=i32) * 8 + 3
        kvp.kv_quant_store(x.to(DEV), x.to(DEV), slots.to(DEV), dev[0][0], dev[1][0], dev[0][1], dev[1][1])
        need = [ref.scale_for(row.abs().max().item(), dtype) for row in x.float()]
        got = dev[0][1].cpu().flatten().tolist()
        for i, (old, n) in enumerate(zip(scales.flatten().tolist(), need)):
            assert got[i] == pytest.approx(max(old, n) if old == old else n, rel=1e-7)
        back = ref.values(dev[0][0].cpu().to(f32), dev[0][1].cpu())[:, 3].double()
        step = {E4M3: 2.0 ** -4, INT8: 0.0}[dtype] * x.double().abs() + \
            dev[0][1].cpu().double() * {E4M3: 2.0 ** -10, INT8: 0.5}[dtype]
        assert bool(((back - x.double()).abs() <= step * (1 + 2.0 ** -20)).all())
        assert torch.equal(bits(dev[0][0][:3, :3]), torch.zeros_like(bits(dev[0][0][:3, :3]))) or dtype == E4M3


def test_store_slots_outside_the_pool():
    host = cache_arrays(2, 16, 16, 2, 64, INT8, gen(4))
    dev = [to_dev(*host) for _ in range(2)]
    x = randn((5, 2, 64), gen(5))
    slots = torch.tensor([32, 40, -1, 1 << 30, -7], dtype=i32)
    kvp.kv_quant_store(x.to(DEV), x.to(DEV), slots.to(DEV), dev[0][0], dev[1][0], dev[0][1], dev[1][1])
    assert kvp.device_status() == -6
    for codes, scales in dev:
        assert torch.equal(codes.cpu(), host[0]) and torch.equal(scales.cpu(), host[1])


@pytest.mark.parametrize("dtype", [E4M3, INT8])
@pytest.mark.parametrize("hkv,d,bs,t,r,interleaved", [
    (8, 128, 256, 16, 128, False), (1, 64, 16, 16, 64, True), (4, 128, 64, 64, 64, False), (2, 64, 32, 1, 20, False),
    (2, 128, 16, 4, 48, True), (8, 128, 256, 256, 36, False), (1, 64, 64, 32, 64, False)])
def test_store_rope(hkv, d, bs, t, r, interleaved, dtype):
    g = gen(d + r)
    n, hq = 75, 2 * hkv
    rows = randn((n, hq + 2 * hkv, d), g).to(DEV)
    q, k, v = rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:]
    blocks = -(-n // bs) + 3
    host = [cache_arrays(blocks, bs, t, hkv, d, dtype, g) for _ in range(2)]
    dev = [to_dev(*h) for h in host]
    ids = torch.randperm(blocks, generator=g)
    p = torch.arange(n)
    slots = (ids[p // bs] * bs + p % bs).to(i32)
    pos = p + 100003
    inv, mag = ref.inverse_frequencies(r, 10000.0, "yarn", 4.0, 2048, 1.0, 32.0)
    freqs, magnitude = kvp.attn_rope_freqs(r, 10000.0, "yarn", 4.0, 2048, device=DEV)
    oq = kvp.kv_quant_store_rope(q, k, v, pos.to(DEV), slots.to(DEV), freqs, dev[0][0], dev[1][0], dev[0][1],
                                 dev[1][1], magnitude, interleaved)
    assert_rope(oq, q, pos, inv, mag, interleaved)
    want = (host[1][0].to(f32).to(f64), host[1][1].to(f64))
    ref.store(v.cpu().to(f64), slots, *want, dtype)
    assert_store(dev[1], want, dtype)
    turned = ref.rope(k.cpu(), pos, inv, mag, interleaved)
    want = (host[0][0].to(f32).to(f64), host[0][1].to(f64))
    ref.store(turned, slots, *want, dtype)
    assert torch.equal(dev[0][1].cpu().to(f64), want[1])
    got = ref.values(dev[0][0].cpu().to(f32), dev[0][1].cpu()).view(-1, hkv, d)[slots.long()]
    step = dev[0][1].cpu().to(f64).view(-1, hkv)[slots.long() // t][..., None]
    tol = {E4M3: 2.0 ** -4, INT8: 0.0}[dtype] * turned.abs() + step * {E4M3: 2.0 ** -10, INT8: 0.5}[dtype]
    top = k.cpu().to(f64).abs().amax(-1, keepdim=True)
    assert bool(((got - turned).abs() <= tol * (1 + 2.0 ** -20) + 2.0 ** -18 * mag * top).all())
    # in place of q, and nothing to rotate but k
    again = kvp.kv_quant_store_rope(q, k, v, pos.to(DEV), slots.to(DEV), freqs, dev[0][0], dev[1][0], dev[0][1],
                                    dev[1][1], magnitude, interleaved, out=q)
    assert again.data_ptr() == q.data_ptr() and torch.equal(q, oq)


@pytest.mark.parametrize("dtype", [E4M3, INT8])
@pytest.mark.parametrize("hkv,d,bs,t,rotate", [
    (8, 128, 256, 64, False), (8, 128, 256, 256, False), (8, 128, 64, 1, False), (3, 64, 48, 2, False),
    (6, 128, 64, 16, False), (8, 128, 256, 16, True), (5, 64, 64, 1, True), (8, 128, 256, 256, True),
    (2, 128, 32, 32, True)])
def test_store_many_rows(hkv, d, bs, t, rotate, dtype):
    """More rows than the CTAs that run at once: sequences end to end, each from the start of a page, some rows
    without a slot; the same bits as calls of a sequence each, and the formula's numbers.  The rows without a slot cut
    a block's run in two, which leaves that block undefined, and only that one."""
    g = gen(t + d)
    lens = [3700, 1, 2049, 0, 1600, 1023, 255, 800]
    n, hq = sum(lens), hkv
    pages = [-(-x // bs) for x in lens]
    blocks = sum(pages) + 2
    ids = torch.randperm(blocks, generator=g)
    slots, first = [], 0
    for x, m in zip(lens, pages):
        p = torch.arange(x)
        slots.append(ids[first:first + m][p // bs] * bs + p % bs)
        first += m
    slots = torch.cat(slots).to(i32)
    slots[5000:5003] = -1
    x = randn((n, hq + 2 * hkv, d), g).to(DEV)
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    pos = torch.arange(n, device=DEV) + 77
    freqs, magnitude = kvp.attn_rope_freqs(d, device=DEV)
    host = [cache_arrays(blocks, bs, t, hkv, d, dtype, g) for _ in range(2)]
    dev, parts = ([to_dev(*h) for h in host] for _ in range(2))
    out = [torch.zeros((n, hq, d), dtype=bf16, device=DEV) for _ in range(2)]

    def store(a, b, arrays, to):
        cache = (arrays[0][0], arrays[1][0], arrays[0][1], arrays[1][1])
        if rotate:
            kvp.kv_quant_store_rope(q[a:b], k[a:b], v[a:b], pos[a:b], slots[a:b].to(DEV), freqs, *cache, magnitude,
                                    out=to[a:b])
        else:
            kvp.kv_quant_store(k[a:b], v[a:b], slots[a:b].to(DEV), *cache)

    store(0, n, dev, out[0])
    a = 0
    for m in lens:
        store(a, a + m, parts, out[1])
        a += m
    cut = slots[4999].item() // t
    if cut != slots[5003].item() // t:
        cut = None

    def without_cut(codes, scales):
        if cut is not None:
            codes.view(-1, t, hkv, d)[cut] = 0
            scales.view(-1, hkv)[cut] = 0
        return codes, scales

    for one, many in zip(dev, parts):
        for arrays in (one, many):
            without_cut(arrays[0].view(torch.uint8), arrays[1])
        assert torch.equal(bits(one[0]), bits(many[0])) and torch.equal(one[1], many[1])
    assert torch.equal(*out)
    for rows, h, arrays in ((k, host[0], dev[0]), (v, host[1], dev[1])):
        if rotate and rows is k:
            continue
        want = (h[0].to(f32).to(f64), h[1].to(f64))
        ref.store(rows.cpu().to(f64), slots, *want, dtype)
        without_cut(*want)
        assert_store(arrays, want, dtype)
    assert kvp.device_status() == 0


# ------------------------------------------------------------------------ load

def batch(lens, bs, spare, g, width=None):
    """Block tables with -1 behind each row's pages -> tables, blocks."""
    pages = [-(-n // bs) for n in lens]
    blocks = sum(pages) + spare
    ids = torch.randperm(blocks, generator=g).tolist()
    width = width or max(1, max(pages))
    tables = torch.full((len(lens), width), -1, dtype=i32)
    for i, p in enumerate(pages):
        tables[i, :p] = torch.tensor([ids.pop() for _ in range(p)], dtype=i32)
    return tables, blocks


def poison_behind(arrays, tables, lens, bs, t, dtype):
    """NaN codes and scales wherever no token of a context lies."""
    used = torch.zeros(arrays[0][0].shape[0] * bs, dtype=torch.bool)
    for row, n in zip(tables, lens):
        for p in range(n):
            used[int(row[p // bs]) * bs + p % bs] = True
    groups = used.view(-1, t).any(-1)
    for codes, scales in arrays:
        flat = codes.view(torch.uint8).view(used.numel(), -1)
        flat[~used] = 0x7F
        scales.view(groups.numel(), -1)[~groups] = math.nan


@pytest.mark.parametrize("dtype", [E4M3, INT8])
@pytest.mark.parametrize("hkv,d,bs,t", CACHES)
def test_load(hkv, d, bs, t, dtype):
    g = gen(bs + t)
    lens = [0, 1, bs - 1, bs, 3 * bs + 1, 77, 0]
    tables, blocks = batch(lens, bs, 2, g)
    host = [cache_arrays(blocks, bs, t, hkv, d, dtype, g) for _ in range(2)]
    poison_behind(host, tables, lens, bs, t, dtype)
    dev = [to_dev(*h) for h in host]
    starts, at = [], 3
    for n in lens:
        starts.append(at)
        at += -(-n // 16) * 16
    rows = [randn((at, hkv + 1, d), g).to(DEV)[:, :hkv] for _ in range(2)]
    before = [r.clone() for r in rows]
    st, ctx = (torch.tensor(x, dtype=i32) for x in (starts, lens))
    got = kvp.kv_quant_load(dev[0][0], dev[1][0], dev[0][1], dev[1][1], tables.to(DEV), ctx.to(DEV), st.to(DEV),
                            max(lens), out=(rows[0], rows[1]))
    for out, old, h in zip(got, before, host):
        vals = ref.values(h[0].to(f32), h[1])
        want = old.cpu().to(f64)
        for i, n in enumerate(lens):
            want[starts[i]:starts[i] + n] = ref.tokens(vals, tables[i].tolist(), n)
        assert torch.equal(out.cpu().to(f64), want)
    # a bound that is too small, and new tensors
    k2, v2 = kvp.kv_quant_load(dev[0][0], dev[1][0], dev[0][1], dev[1][1], tables.to(DEV), ctx.to(DEV), st.to(DEV), 1,
                               num_rows=at)
    for i, n in enumerate(lens):
        assert torch.equal(k2[starts[i]:starts[i] + n], got[0][starts[i]:starts[i] + n])
    assert kvp.device_status() == 0


def test_load_of_scales_that_are_no_powers():
    g = gen(8)
    tables, blocks = batch([50], 16, 0, g)
    codes, scales = cache_arrays(blocks, 16, 8, 2, 64, INT8, g)
    scales = torch.rand(scales.shape, generator=g) + 0.01
    dev = to_dev(codes, scales, tables)
    k, _ = kvp.kv_quant_load(dev[0], dev[0], dev[1], dev[1], dev[2], torch.tensor([50], dtype=i32, device=DEV),
                             torch.zeros(1, dtype=i32, device=DEV), 50, num_rows=50)
    want = ref.tokens(ref.values(codes.to(f32), scales), tables[0].tolist(), 50)
    assert bool(((k.cpu().to(f64) - want).abs() <= want.abs() * (2.0 ** -8 + 2.0 ** -23)).all())


def test_load_bad_pages_and_rows():
    g = gen(9)
    tables, blocks = batch([40, 40, 40], 16, 0, g)
    codes, scales = cache_arrays(blocks, 16, 16, 1, 64, E4M3, g)
    bad = tables.clone()
    bad[1, 1] = blocks
    bad[1, 2] = -1
    dev = to_dev(codes, scales)
    args = lambda tab, lens, starts: (dev[0], dev[0], dev[1], dev[1], tab.to(DEV),  # noqa: E731
                                      torch.tensor(lens, dtype=i32, device=DEV),
                                      torch.tensor(starts, dtype=i32, device=DEV), 40)
    out = [torch.zeros((120, 1, 64), dtype=bf16, device=DEV) for _ in range(2)]
    kvp.kv_quant_load(*args(bad, [40, 40, 40], [0, 40, 80]), out=tuple(out))
    assert kvp.device_status() == -6
    vals = ref.values(codes.to(f32), scales)
    want = torch.cat([ref.tokens(vals, tables[i].tolist(), 40) for i in range(3)])
    want[56:80] = 0
    assert torch.equal(out[0].cpu().to(f64), want) and torch.equal(out[1].cpu().to(f64), want)
    # rows before and behind the output, lengths that no table holds
    for lens, starts in (([40, 40, 40], [0, -20, 100]), ([40, -1, 40], [0, 0, 80]), ([1000, 1, 1], [0, 60, 61])):
        out = [torch.zeros((120, 1, 64), dtype=bf16, device=DEV) for _ in range(2)]
        kvp.kv_quant_load(*args(tables, lens, starts), out=tuple(out))
        assert kvp.device_status() == -6


# ---------------------------------------------------------------------- decode

def run_decode(q, dev, tables, lens, longest=None, **kw):
    return kvp.attn_decode_quant(q.to(DEV), dev[0][0], dev[1][0], dev[0][1], dev[1][1], tables.to(DEV),
                                 torch.tensor(lens, dtype=i32, device=DEV), max(lens) if longest is None else longest,
                                 **kw)


def assert_decode(out, q, host, tables, lens, scale, weight=2.0 ** -11 + 2.0 ** -12):
    want, size, unit = ref.decode(q.cpu(), *((c.to(f32), s) for c, s in host), tables, lens, scale)
    tol = 2.0 ** -8 * want.abs() + (weight * size + 2.0 ** -25 * unit) * (1 + 2.0 ** -8)
    off = (out.cpu().to(f64) - want).abs()
    assert bool((off <= tol).all()), ((off - tol).max().item(), off.max().item())


def decode_case(hq, hkv, d, bs, t, dtype, lens, seed, poison=True, grow=1.0):
    g = gen(seed)
    tables, blocks = batch(lens, bs, 3, g)
    host = [cache_arrays(blocks, bs, t, hkv, d, dtype, g) for _ in range(2)]
    if poison:
        poison_behind(host, tables, lens, bs, t, dtype)
        for h in host:  # the reference multiplies what it does not use
            h[1][torch.isnan(h[1])] = math.nan
    q = randn((len(lens), hq + 1, d), g) * grow
    return q.to(bf16), host, [to_dev(*h) for h in host], tables


@pytest.mark.parametrize("dtype", [E4M3, INT8])
@pytest.mark.parametrize("hq,hkv,d,bs,t", [
    (16, 8, 128, 256, 16), (2, 1, 64, 16, 16), (8, 8, 128, 64, 1), (32, 8, 128, 16, 16), (64, 8, 128, 256, 64),
    (8, 1, 128, 32, 4), (16, 4, 128, 128, 128), (4, 2, 64, 256, 256), (16, 2, 64, 48, 16), (16, 4, 64, 24, 8),
    (32, 8, 64, 256, 2), (64, 8, 64, 64, 32), (4, 4, 128, 6, 2), (1, 1, 128, 512, 256)])
def test_decode(hq, hkv, d, bs, t, dtype):
    lens = [1, 0, 15, 16, 17, 300, 2, 33, 64, 0, 129, 1000]
    q, host, dev, tables = decode_case(hq, hkv, d, bs, t, dtype, lens, hq + d + bs)
    host = [(torch.nan_to_num(h[0].to(f32)), torch.nan_to_num(h[1])) for h in host]
    for longest in (1000, 100000, 256):  # in shares, of few and of all CTAs; not cut
        out = run_decode(q[:, :hq], dev, tables, lens, longest=longest)
        assert_decode(out, q[:, :hq], host, tables, lens, d ** -0.5)
        assert not out[1].any() and not out[9].any()
    assert kvp.device_status() == 0


@pytest.mark.parametrize("hq,hkv,d", [(16, 8, 128), (1, 1, 64), (2, 1, 128), (64, 8, 128), (8, 4, 64), (4, 2, 128)])
@pytest.mark.parametrize("lens", [[1], [17], [0, 300, 0], [129, 128, 127], [2048] * 15, [1, 2047] * 7, [1024, 5, 600] * 11])
def test_decode_small_batches(hq, hkv, d, lens):
    """Fewer units than CTAs, empty sequences between, and the same result twice."""
    q, host, dev, tables = decode_case(hq, hkv, d, 64, 16, E4M3, lens, 29 + len(lens), poison=False)
    out = run_decode(q[:, :hq], dev, tables, lens, longest=max(max(lens), 257))
    assert_decode(out, q[:, :hq], host, tables, lens, d ** -0.5)
    again = run_decode(q[:, :hq], dev, tables, lens, longest=max(max(lens), 257))
    assert torch.equal(out, again)
    assert kvp.device_status() == 0


@pytest.mark.parametrize("lens", [[1], [16], [5000], [40000], [3] * 400, [1700] * 40 + [0] * 8, [9, 12000, 1, 1]])
@pytest.mark.parametrize("heads", [(16, 8, 128), (8, 1, 128), (2, 1, 64)])
def test_decode_splits(heads, lens):
    hq, hkv, d = heads
    q, host, dev, tables = decode_case(hq, hkv, d, 64, 16, E4M3, lens, sum(lens) % 97, poison=False)
    out = run_decode(q[:, :hq], dev, tables, lens)
    assert_decode(out, q[:, :hq], host, tables, lens, d ** -0.5)
    # a bound above the lengths changes nothing but the split
    out = run_decode(q[:, :hq], dev, tables, lens, longest=tables.shape[1] * 64)
    assert_decode(out, q[:, :hq], host, tables, lens, d ** -0.5)


def test_decode_one_key_rules():
    """Scores far apart: the largest takes all, wherever it lies."""
    lens = [700, 700, 700]
    q, host, dev, tables = decode_case(8, 2, 128, 16, 16, INT8, lens, 12, poison=False, grow=40.0)
    out = run_decode(q[:, :8], dev, tables, lens)
    assert_decode(out, q[:, :8], host, tables, lens, 128 ** -0.5)
    for scale in (0.0, -0.1, 3.0):
        out = run_decode(q[:, :8], dev, tables, lens, softmax_scale=scale)
        # scores off by 2^-17 of sum |q k| * scale, |k| of 3 and less on average
        x = q[:, :8].to(f64).abs().amax().item() * 128 * 3 * abs(scale) * 2.0 ** -17
        assert_decode(out, q[:, :8], host, tables, lens, scale, weight=2.0 ** -11 + x)


def test_decode_scales_far_apart():
    """Blocks of very small and very large values; a block of zeros whose scale is zero."""
    lens = [256, 250]
    for dtype in (E4M3, INT8):
        q, host, dev, tables = decode_case(4, 1, 64, 32, 8, dtype, lens, 13, poison=False)
        g = gen(14)
        for h in host[1:]:
            h[1].copy_(torch.exp2(torch.randint(-40, 30, h[1].shape, generator=g).float()))
        host[1][1][tables[0, 0]] = 0.0
        host[1][1][tables[1]] = 2.0 ** -50
        dev = [to_dev(*h) for h in host]
        out = run_decode(q[:, :4], dev, tables, lens)
        assert_decode(out, q[:, :4], host, tables, lens, 0.125)


def test_decode_q_of_any_size():
    """Queries whose numbers lie far apart or near the ends of bf16's range."""
    for grow in (1e-30, 1e-5, 300.0):
        q, host, dev, tables = decode_case(2, 2, 64, 16, 16, E4M3, [90], 15, poison=False, grow=grow)
        q[0, 0, 0] *= 64
        scale = 0.125 if grow < 1 else 1e-3
        out = run_decode(q[:, :2], dev, tables, [90], softmax_scale=scale)
        assert_decode(out, q[:, :2], host, tables, [90], scale)


@pytest.mark.parametrize("dtype", [E4M3, INT8])
@pytest.mark.parametrize("hq,hkv,d,t", [(16, 8, 128, 16), (8, 1, 64, 4)])
def test_decode_q_not_finite(hq, hkv, d, t, dtype):
    """An infinite score's softmax is NaN; the other heads keep their numbers, in a sequence that is one CTA's, in one
    that many share, and in one without a context."""
    lens = [40, 4000, 0]
    q, _, dev, tables = decode_case(hq, hkv, d, 64, t, dtype, lens, 16, poison=False)
    q = q[:, :hq].contiguous()
    want = run_decode(q, dev, tables, lens)
    heads = {0: math.inf, 3: -math.inf, hq - 1: math.nan}
    for h, x in heads.items():
        q[:, h, h % d] = x
    out = run_decode(q, dev, tables, lens)
    for h in range(hq):
        if h in heads:
            assert bool(torch.isnan(out[:2, h]).all()) and not out[2, h].any()
        else:
            assert torch.equal(out[:, h], want[:, h])


def test_bounds_far_above_the_lengths():
    """max_context_len may be any bound: work is sized by the tables where that is less."""
    lens, most = [70, 3], 2 ** 31 - 1
    q, host, dev, tables = decode_case(8, 8, 128, 16, 16, E4M3, lens, 17, poison=False)
    q = q[:, :8].contiguous()
    assert_decode(run_decode(q, dev, tables, lens, longest=most), q, host, tables, lens, 128 ** -0.5)
    rows = [[torch.zeros((80, 8, 128), dtype=bf16, device=DEV) for _ in range(2)] for _ in range(2)]
    for out, longest in zip(rows, (70, most)):
        kvp.kv_quant_load(dev[0][0], dev[1][0], dev[0][1], dev[1][1], tables.to(DEV),
                          torch.tensor(lens, dtype=i32, device=DEV), torch.tensor([0, 72], dtype=i32, device=DEV),
                          longest, out=tuple(out))
    assert all(torch.equal(a, b) for a, b in zip(*rows))


def test_decode_bad_pages_and_lengths():
    lens = [40, 40]
    q, host, dev, tables = decode_case(2, 1, 64, 16, 16, E4M3, lens, 16, poison=False)
    bad = tables.clone()
    bad[0, 1] = 1 << 20
    out = run_decode(q[:, :2], dev, bad, lens)
    assert kvp.device_status() == -6
    assert_decode(out[1:], q[1:, :2], host, tables[1:], lens[1:], 0.125)
    bad[0, 1] = -1
    run_decode(q[:, :2], dev, bad, lens)
    assert kvp.device_status() == -6
    run_decode(q[:, :2], dev, tables, [49, -3], longest=48)
    assert kvp.device_status() == -6


def test_decode_out_and_strides():
    lens = [100, 3]
    q, host, dev, tables = decode_case(4, 2, 128, 32, 16, E4M3, lens, 17)
    host = [(torch.nan_to_num(h[0].to(f32)), torch.nan_to_num(h[1])) for h in host]
    wide = torch.full((2, 6, 128), 7.0, dtype=bf16, device=DEV)
    need = kvp.attn_decode_quant_workspace_size(2, 4, 2, 128, 100)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=DEV)
    rows = q.to(DEV)
    got = kvp.attn_decode_quant(rows[:, :4], dev[0][0], dev[1][0], dev[0][1], dev[1][1], tables.to(DEV),
                                torch.tensor(lens, dtype=i32, device=DEV), 100, workspace=ws, out=wide[:, :4])
    assert got.data_ptr() == wide.data_ptr() and bool((wide[:, 4:] == 7).all())
    assert_decode(got, q[:, :4], host, tables, lens, 128 ** -0.5)
    # in place of q
    kvp.attn_decode_quant(rows[:, :4], dev[0][0], dev[1][0], dev[0][1], dev[1][1], tables.to(DEV),
                          torch.tensor(lens, dtype=i32, device=DEV), 100, out=rows[:, :4])
    assert torch.equal(rows[:, :4], got)
    with pytest.raises(kvp.KvpError, match="workspace"):
        run_decode(q[:, :4], dev, tables, lens, workspace=ws[:need - 16])


def test_caches_past_two_billion_numbers():
    """Code offsets past 2^31 and past 2^32."""
    nb, bs, hkv, d, t = 17000, 256, 8, 128, 16
    k, v = (torch.zeros((nb, bs, hkv, d), dtype=E4M3, device=DEV) for _ in range(2))
    ks, vs = (torch.zeros((nb, bs // t, hkv), device=DEV) for _ in range(2))
    assert k.numel() > 1 << 32
    g = gen(18)
    pages, n = [nb - 1, 9000, 3], 600
    tables = torch.tensor([pages], dtype=i32)
    p = torch.arange(n)
    slots = (tables[0].long()[p // bs] * bs + p % bs).to(i32)
    x, y = randn((n, hkv, d), g), randn((n, hkv, d), g)
    kvp.kv_quant_store(x.to(DEV), y.to(DEV), slots.to(DEV), k, v, ks, vs)
    small = [(torch.zeros((3, bs, hkv, d), dtype=f64), torch.zeros((3, bs // t, hkv), dtype=f64)) for _ in range(2)]
    for rows, (codes, scales) in zip((x, y), small):
        ref.store(rows.to(f64), p, codes, scales, E4M3)
    for a, s, (codes, scales) in ((k, ks, small[0]), (v, vs, small[1])):
        assert torch.equal(a[pages].cpu().to(f32).to(f64), codes) and torch.equal(s[pages].cpu().to(f64), scales)
    ctx = torch.tensor([n], dtype=i32, device=DEV)
    back, _ = kvp.kv_quant_load(k, v, ks, vs, tables.to(DEV), ctx, torch.zeros(1, dtype=i32, device=DEV), n, num_rows=n)
    assert torch.equal(back.cpu().to(f64), ref.values(*small[0]).view(-1, hkv, d)[:n])
    q = randn((1, 16, d), g)
    out = kvp.attn_decode_quant(q.to(DEV), k, v, ks, vs, tables.to(DEV), ctx, n)
    assert_decode(out, q, [(small[0][0].to(f32), small[0][1]), (small[1][0].to(f32), small[1][1])],
                  torch.tensor([[0, 1, 2]], dtype=i32), [n], d ** -0.5)


def test_more_sequences_than_threads():
    """Lengths in runs of several for a thread; empty rows in front, between and behind."""
    lens = [0] * 5 + [(i * 7) % 41 for i in range(1200)] + [0] * 9
    q, host, dev, tables = decode_case(2, 1, 64, 16, 16, INT8, lens, 22, poison=False)
    for longest in (40, 300):  # none cut; cut where shares end
        out = run_decode(q[:, :2], dev, tables, lens, longest=longest)
        assert_decode(out, q[:, :2], host, tables, lens, 0.125)
        assert not out[torch.tensor(lens) == 0].any()
    assert kvp.device_status() == 0


@pytest.mark.parametrize("hq,hkv,d,bs", [(8, 1, 128, 256), (8, 1, 128, 16), (4, 2, 64, 64), (2, 1, 64, 2048), (16, 8, 64, 32)])
def test_decode_many_short_segments(hq, hkv, d, bs):
    """More segments in a CTA than the producer tells ahead, in one launch and in two."""
    lens = [1 + (i * 13) % 50 for i in range(152 * 20)]
    q, host, dev, tables = decode_case(hq, hkv, d, bs, 16, E4M3, lens, 23, poison=False)
    for longest in (50, 1000):
        out = run_decode(q[:, :hq], dev, tables, lens, longest=longest)
        some = slice(0, None, 61)
        assert_decode(out[some], q[some, :hq], host, tables[some], lens[some], d ** -0.5)
        assert bool(torch.isfinite(out).all())
    assert kvp.device_status() == 0


def test_store_rows_of_other_calls_stay():
    """What a call does not name stays as it was: blocks behind the last run, and pages between."""
    for dtype in (E4M3, INT8):
        codes, scales = cache_arrays(9, 32, 8, 3, 128, dtype, gen(24))
        dev = [to_dev(codes.clone(), scales.clone()) for _ in range(2)]
        slots = torch.cat((torch.arange(70, 83), torch.arange(160, 161), torch.arange(200, 216))).to(i32)
        x = randn((len(slots), 3, 128), gen(25))
        kvp.kv_quant_store(x.to(DEV), x.to(DEV), slots.to(DEV), dev[0][0], dev[1][0], dev[0][1], dev[1][1])
        touched = torch.zeros(9 * 32 // 8, dtype=torch.bool)
        touched[slots.long() // 8] = True
        for got, old in ((dev[0][0], codes), (dev[1][0], codes)):
            assert torch.equal(bits(got).view(-1, 8 * 3 * 128)[~touched], bits(old).view(-1, 8 * 3 * 128)[~touched])
        for got in (dev[0][1], dev[1][1]):
            assert torch.equal(got.cpu().view(-1, 3)[~touched], scales.view(-1, 3)[~touched])


def test_calls_without_the_extension_module(monkeypatch):
    """The same results where the binding makes the calls itself."""
    lens = [33, 0, 70]
    q, host, dev, tables = decode_case(4, 2, 64, 32, 16, INT8, lens, 26, poison=False)
    rows = randn((3, 4 + 2 + 2, 64), gen(27)).to(DEV)
    freqs, _ = kvp.attn_rope_freqs(64, device=DEV)
    pos = torch.tensor([32, 5, 69], device=DEV)
    slots = torch.tensor([int(tables[0, 1]) * 32, -1, int(tables[2, 2]) * 32 + 5], dtype=i32, device=DEV)
    st, ctx = torch.tensor([0, 40, 50], dtype=i32, device=DEV), torch.tensor(lens, dtype=i32, device=DEV)

    def everything():
        cache = [t.clone() for t in (dev[0][0], dev[1][0], dev[0][1], dev[1][1])]
        got = list(kvp.attn_rope(rows[:, :4], rows[:, 4:6], pos, freqs, 1.25, True))
        kvp.kv_quant_store(rows[:, 4:6], rows[:, 6:], slots, *cache)
        got += [t.clone() for t in cache]
        got.append(kvp.kv_quant_store_rope(rows[:, :4], rows[:, 4:6], rows[:, 6:], pos, slots, freqs, *cache, 1.25, True))
        out = tuple(torch.zeros((120, 2, 64), dtype=bf16, device=DEV) for _ in range(2))
        got += list(kvp.kv_quant_load(*cache, tables.to(DEV), ctx, st, 70, out=out))
        got.append(kvp.attn_decode_quant(rows[:, :4], *cache, tables.to(DEV), ctx, 70))
        return got + cache

    want = everything()
    monkeypatch.setattr(kvp, "_CALLS", kvp._NoCalls())
    for a, b in zip(everything(), want):
        assert torch.equal(bits(a.contiguous()), bits(b.contiguous()))


def test_binding_refusals():
    """What the calls do not take, with device tensors."""
    _, _, dev, tables = decode_case(4, 2, 64, 32, 16, INT8, [33, 70], 28, poison=False)
    arrays = (dev[0][0], dev[1][0], dev[0][1], dev[1][1])
    x = torch.zeros((2, 2, 64), dtype=bf16, device=DEV)
    slots = torch.tensor([1, 2], dtype=i32, device=DEV)
    tab, ctx = tables.to(DEV), torch.tensor([33, 70], dtype=i32, device=DEV)
    freqs, _ = kvp.attn_rope_freqs(64, device=DEV)
    pos = torch.tensor([0, 1], device=DEV)
    with pytest.raises(ValueError, match="rows|row per"):
        kvp.kv_quant_store(x[:1], x, slots, *arrays)
    with pytest.raises(ValueError, match="head_dim|must be"):
        kvp.attn_decode_quant(torch.zeros((2, 4, 128), dtype=bf16, device=DEV), *arrays, tab, ctx, 70)
    with pytest.raises(ValueError, match="k_scales"):
        kvp.kv_quant_store(x, x, slots, arrays[0], arrays[1], arrays[2][:, :1, :1], arrays[3])
    with pytest.raises(TypeError, match="float32"):
        kvp.kv_quant_store(x, x, slots, arrays[0], arrays[1], arrays[2].half(), arrays[3])
    with pytest.raises(TypeError, match="int8"):
        kvp.kv_quant_store(x, x, slots, arrays[0], arrays[1].view(E4M3), *arrays[2:])
    with pytest.raises(ValueError, match="contiguous"):
        kvp.kv_quant_store(x, x, slots, arrays[0].transpose(1, 2), arrays[1], *arrays[2:])
    with pytest.raises(ValueError, match="num_rows"):
        kvp.kv_quant_load(*arrays, tab, ctx, slots, 70)
    with pytest.raises(ValueError, match="positions"):
        kvp.attn_rope(x, x, pos[:1], freqs)
    with pytest.raises(ValueError, match="head_dim"):
        kvp.attn_rope(x, torch.zeros((2, 2, 128), dtype=bf16, device=DEV), pos, freqs)
    with pytest.raises(kvp.KvpError, match="rotary_dim"):
        kvp.attn_rope(x[..., :32].contiguous(), None, pos, freqs)
    with pytest.raises(kvp.KvpError, match="bad shape"):  # the workspace that it would need
        kvp.attn_decode_quant(torch.zeros((2, 6, 64), dtype=bf16, device=DEV), *arrays, tab, ctx, 70)
    with pytest.raises(kvp.KvpError, match="scale_tokens"):
        kvp.kv_quant_store(x, x, slots, *(torch.zeros((2, 48, 2, 64), dtype=torch.int8, device=DEV) for _ in range(2)),
                           *(torch.zeros((2, 2, 2), device=DEV) for _ in range(2)))
    kvp.kv_quant_store(x[:0], x[:0], slots[:0], *arrays)  # no rows: nothing to do
    assert kvp.attn_decode_quant(torch.zeros((0, 4, 64), dtype=bf16, device=DEV), *arrays, tab[:0], ctx[:0], 70).shape[0] == 0
    kvp.attn_rope(x[:0], None, pos[:0], freqs)


# ------------------------------------------------------- streams, graphs, a whole run

def test_another_stream_and_a_graph():
    """The calls captured once, replayed on new contents of the same buffers; and two at once, each on its own
    stream with its own workspace."""
    lens = [200, 1, 90]
    q, host, dev, tables = decode_case(4, 2, 128, 32, 16, E4M3, lens, 19)
    g = gen(20)
    freqs, _ = kvp.attn_rope_freqs(128, device=DEV)
    rows = randn((3, 4 + 2 + 2, 128), g).to(DEV)
    slots = torch.tensor([int(tables[i, (n - 1) // 32]) * 32 + (n - 1) % 32 for i, n in enumerate(lens)],
                         dtype=i32, device=DEV)
    pos = torch.tensor([n - 1 for n in lens], device=DEV)
    ctx, tab = torch.tensor(lens, dtype=i32, device=DEV), tables.to(DEV)
    st = torch.tensor([0, 208, 224], dtype=i32, device=DEV)

    def step(cache, ws, read):
        arrays = (cache[0][0], cache[1][0], cache[0][1], cache[1][1])
        turned = kvp.kv_quant_store_rope(rows[:, :4], rows[:, 4:6], rows[:, 6:], pos, slots, freqs, *arrays)
        out = kvp.attn_decode_quant(turned, *arrays, tab, ctx, 224, workspace=ws)
        kvp.kv_quant_load(*arrays, tab, ctx, st, 224, out=read)
        return out

    caches = [[tuple(t.clone() for t in pair) for pair in dev] for _ in range(3)]
    spaces = [torch.empty(kvp.attn_decode_quant_workspace_size(3, 4, 2, 128, 224), dtype=torch.uint8, device=DEV)
              for _ in range(3)]
    reads = [tuple(torch.zeros((330, 2, 128), dtype=bf16, device=DEV) for _ in range(2)) for _ in range(3)]
    want = step(caches[0], spaces[0], reads[0])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for s, c, w, r in zip(streams, caches[1:], spaces[1:], reads[1:]):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            outs.append(step(c, w, r))
    torch.cuda.synchronize()
    for o, r in zip(outs, reads[1:]):
        assert torch.equal(o, want) and torch.equal(r[0], reads[0][0]) and torch.equal(r[1], reads[0][1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step(caches[1], spaces[1], reads[1])
    for n in range(3):
        rows.copy_(randn(tuple(rows.shape), gen(30 + n)))
        fresh = [tuple(t.to(DEV) for t in h) for h in host]
        for a, b in zip(caches[1], fresh):
            for x, y in zip(a, b):
                x.copy_(y)
        graph.replay()
        want = step(fresh, spaces[0], reads[0])
        torch.cuda.synchronize()
        assert torch.equal(held, want) and torch.equal(reads[1][0], reads[0][0])
    assert kvp.device_status() == 0


@pytest.mark.parametrize("dtype", [E4M3, INT8])
def test_a_serving_run(dtype):
    """Two prompts, the second a prefix hit on the first: rotate and store, read back, prefill the suffixes over
    the read rows, then decode three tokens; against attention in 64 bits over what was stored."""
    hq, hkv, d, bs, t = 4, 2, 128, 32, 16
    g = gen(40)
    freqs, _ = kvp.attn_rope_freqs(d, 1e6, device=DEV)
    shape = (24, bs, hkv, d)
    cache = [torch.zeros(shape, dtype=torch.uint8, device=DEV).view(dtype) for _ in range(2)]
    scales = [torch.zeros((24, bs // t, hkv), device=DEV) for _ in range(2)]
    arrays = (*cache, *scales)
    tables = torch.tensor([[5, 9, 2, 11], [5, 9, 7, 8]], dtype=i32)
    slot = lambda b, p: int(tables[b, p // bs]) * bs + p % bs  # noqa: E731
    lens, cached = [90, 101], [0, 64]

    def ints(x):
        return torch.tensor(x, dtype=i32, device=DEV)

    steps = [[(0, 0, 90)], [(1, 64, 101)]] + [[(0, 90 + i, 91 + i), (1, 101 + i, 102 + i)] for i in range(3)]
    for n, parts in enumerate(steps):
        rows = sum(b - a for _, a, b in parts)
        x = randn((rows, hq + 2 * hkv, d), g).to(DEV)
        pos = torch.tensor([p for _, a, b in parts for p in range(a, b)], device=DEV)
        slots = ints([slot(i, p) for i, a, b in parts for p in range(a, b)])
        q = kvp.kv_quant_store_rope(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], pos, slots, freqs, *arrays)
        held = [(c.cpu().to(f32), s.cpu()) for c, s in zip(cache, scales)]
        if n < 2:
            (i, a, b), = parts
            pages = -(-b // 16)
            k, v = kvp.kv_quant_load(*arrays, tables[i:i + 1].to(DEV), ints([b]), ints([0]), b, num_rows=pages * 16)
            k[b:], v[b:] = 0, 0
            out = kvp.attn_prefill_varlen(q, ints([0, b - a]), ints([0, b]), b - a, b, k_cache=k.view(pages, 16, hkv, d),
                                          v_cache=v.view(pages, 16, hkv, d),
                                          block_tables=torch.arange(pages, dtype=i32, device=DEV)[None])
            for row in range(b - a):  # (the prefill rounds its weights to bf16: 2^-8)
                assert_decode(out[row:row + 1], q[row:row + 1], held, tables[i:i + 1], [a + row + 1], d ** -0.5,
                              weight=2.0 ** -8 + 2.0 ** -10)
        else:
            now = [parts[0][2], parts[1][2]]
            out = kvp.attn_decode_quant(q, *arrays, tables.to(DEV), ints(now), 128)
            assert_decode(out, q, held, tables, now, d ** -0.5)
    assert kvp.device_status() == 0


def test_pages_of_an_8_bit_cache_are_copied():
    """kv_copy_blocks on the codes (as 16-bit numbers) and on the scales."""
    g = gen(50)
    codes, scales = cache_arrays(6, 16, 4, 2, 64, INT8, g)
    dev = to_dev(codes, scales)
    pairs = torch.tensor([[1, 4], [0, 5]], dtype=i32, device=DEV)
    kvp.kv_copy_blocks(dev[0].view(bf16), pairs)
    kvp.kv_copy_blocks(dev[1].view(bf16).view(6, 4, 2, 2), pairs)
    for new, old in zip(dev, (codes, scales)):
        want = old.clone()
        want[4], want[5] = old[1], old[0]
        assert torch.equal(new.cpu(), want)
