"""attn_shared_plan + attn_decode_shared (+ _append) against the fp64 oracle.

The oracle attends every sequence over its own table row; the calls must give
the same whatever pages the rows share.  Tolerance, element by element, with A
= sum_i p_i |v_i| / sum_i p_i (the oracle's decode of the caches with |V|):

  output rounded to bf16                      eps / 2 * |ref| = 2^-8 |ref|
  weights p rounded to bf16 before P V        2^-8 A
  scores in fp32: d = 128 products, each sum within (d + 2) 2^-24 * scale *
  sum |q k| of the exact one (< 10 here): 8e-5, on p and on the sum l; exp2
  within 2^-21; l and P V summed in fp32 over at most 2^13 keys a part, 2^13 *
  2^-24 = 2^-11 each: together below                 2^-9 A

so |out - ref| <= 2^-8 |ref| (1 + 2^-6) + (2^-8 + 2^-9) A."""
import math

import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_125_gb300 as kvp

from pages_reference import ceil, shared_prefixes
from parity import assert_status_ok, u16

pytestmark = pytest.mark.gpu
BF16, I32 = torch.bfloat16, torch.int32


class Batch:
    """groups: (prefix pages, [own tokens of each member]); a prefix of 0
    pages makes a sequence of its own; own tokens 0 with prefix 0: padding."""

    def __init__(self, heads, bs, groups, seed, poison=True, extra=3):
        self.hq, self.hkv, self.d = heads
        self.bs = bs
        rng = np.random.default_rng(seed)
        rows, need = [], 0
        for prefix, own in groups:
            shared = list(range(need, need + prefix))
            need += prefix
            for n in own:
                pages = ceil(n, bs)
                rows.append((shared + list(range(need, need + pages)), prefix * bs + n))
                need += pages
        self.nb = need + extra
        ids = rng.permutation(self.nb)
        self.b = len(rows)
        width = max([len(r) for r, _ in rows] + [1])
        self.tables = np.full((self.b, width), -1, np.int32)
        for i, (r, _) in enumerate(rows):
            self.tables[i, :len(r)] = ids[r]
        self.lens = np.array([n for _, n in rows], np.int32)
        self.slots = np.array([-1 if n == 0 else self.tables[i, (n - 1) // bs] * bs + (n - 1) % bs
                               for i, n in enumerate(self.lens)], np.int32)
        g = torch.Generator(device="cuda").manual_seed(seed)
        shape = (self.nb, bs, self.hkv, self.d)
        self.kc, self.vc = (torch.randn(shape, generator=g, device="cuda").to(BF16) for _ in range(2))
        if poison:  # everything no sequence may read
            used = np.zeros((self.nb, bs), bool)
            for i, n in enumerate(self.lens):
                for p in range(n):
                    used[self.tables[i, p // bs], p % bs] = True
            free = torch.from_numpy(~used).cuda()
            self.kc[free] = float("nan")
            self.vc[free] = float("nan")
            self.vc.view(-1, self.hkv, self.d)[(~torch.from_numpy(used).view(-1)).nonzero()[::2, 0].cuda()] = float("inf")
        self.q = torch.randn((self.b, self.hq, self.d), generator=g, device="cuda").to(BF16)
        self.k, self.v = (torch.randn((self.b, self.hkv, self.d), generator=g, device="cuda").to(BF16)
                          for _ in range(2))
        self.scale = 1.0 / math.sqrt(self.d)

    def dev(self, a):
        return torch.from_numpy(np.ascontiguousarray(a)).cuda()

    def plan(self, min_shared=0):
        return kvp.attn_shared_plan(self.dev(self.tables), self.dev(self.lens), self.bs, self.hq, self.hkv,
                                    self.nb, min_shared)

    def reference(self, kc=None, vc=None):
        """-> (ref, A) of the caches as they are."""
        k, v = u16(self.kc if kc is None else kc), u16(self.vc if vc is None else vc)
        args = (torch.from_numpy(self.tables), torch.from_numpy(self.lens), self.hq, self.hkv, self.scale)
        return oracle.decode(self.q.cpu(), k, v, *args), oracle.decode(self.q.cpu(), k, v & 0x7FFF, *args)

    def check(self, out, ref, what=""):
        ref, a = ref
        got = out.float().cpu().double().numpy()
        assert np.isfinite(got).all(), f"{what}: non-finite output"
        tol = 2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -6) + (2.0 ** -8 + 2.0 ** -9) * np.abs(a)
        worst = float((np.abs(got - ref) - tol).max(initial=-1.0))
        assert worst <= 0, f"{what}: {worst} past the tolerance"
        assert not got[self.lens == 0].any(), f"{what}: rows without context are not zero"


def plan_prefixes(plan, b):
    """The prefix lengths in a plan, at their place in its layout."""
    raw = plan.cpu().numpy().tobytes()
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    head = 80 + 32 * sms + 32 * 2 * sms  # and where each CTA starts
    return np.frombuffer(raw, np.int32, b, head + 16 * (b + 1) + 4 * b).tolist()


HEADS = [(2, 1, 64), (4, 2, 64), (16, 8, 64), (8, 1, 128), (4, 4, 128), (8, 8, 128), (16, 8, 128),
         (32, 8, 128), (64, 8, 128)]
SHAPES = {
    "two": [(16, [1, 7])],
    "one_token_each": [(8, [1, 1, 1])],
    "alone": [(0, [1]), (0, [300]), (0, [17])],
    "odd": [(9, [5, 40, 33]), (0, [129]), (11, [16, 17]), (0, [0]), (25, [3, 2, 1, 250])],
    "padding": [(0, [0]), (12, [20, 50]), (0, [0, 0])],
    "many": [(8 + i, [1 + (7 * i + 3 * j) % 90 for j in range(2 + i % 5)]) for i in range(14)],
    "tall": [(13, [1 + (5 * i) % 37 for i in range(150)])],
}


@pytest.mark.parametrize("heads", HEADS, ids=lambda h: "%d/%d/%d" % h)
@pytest.mark.parametrize("shape", SHAPES)
def test_matches_oracle(heads, shape):
    w = Batch(heads, 16, SHAPES[shape], seed=len(shape) + heads[0])
    out = kvp.attn_decode_shared(w.q, w.kc, w.vc, w.dev(w.tables), w.plan(), softmax_scale=w.scale)
    torch.cuda.synchronize()
    assert_status_ok()
    w.check(out, w.reference(), shape)


@pytest.mark.parametrize("bs", [16, 32, 64, 128, 256, 512])
def test_block_sizes(bs):
    groups = [(ceil(400, bs), [1, bs, bs + 1, 3]), (0, [2 * bs + 5]), (ceil(1000, bs), [7, 200])]
    for heads in ((16, 8, 128), (4, 2, 64)):
        w = Batch(heads, bs, groups, seed=bs)
        out = kvp.attn_decode_shared(w.q, w.kc, w.vc, w.dev(w.tables), w.plan(), softmax_scale=w.scale)
        torch.cuda.synchronize()
        assert_status_ok()
        w.check(out, w.reference(), f"bs {bs}")


@pytest.mark.parametrize("heads", [(16, 8, 128), (32, 8, 128), (4, 2, 64)], ids=lambda h: "%d/%d/%d" % h)
def test_long_prefix_and_long_own_parts(heads):
    w = Batch(heads, 256, [(24, [1000, 3, 700, 2000]), (3, [5000, 1])], seed=5)
    out = kvp.attn_decode_shared(w.q, w.kc, w.vc, w.dev(w.tables), w.plan(), softmax_scale=w.scale)
    torch.cuda.synchronize()
    assert_status_ok()
    w.check(out, w.reference(), "long")


@pytest.mark.parametrize("heads", [(2, 1, 64), (16, 8, 128), (32, 8, 128), (64, 8, 128), (8, 1, 128)],
                         ids=lambda h: "%d/%d/%d" % h)
@pytest.mark.parametrize("shape", ["odd", "padding", "one_token_each", "tall"])
def test_append_stores_and_attends(heads, shape):
    w = Batch(heads, 16, SHAPES[shape], seed=11 + heads[0])
    plan = w.plan()
    kc, vc = w.kc.clone(), w.vc.clone()
    out = kvp.attn_decode_shared_append(w.q, w.k, w.v, w.dev(w.slots), w.kc, w.vc, w.dev(w.tables), plan,
                                        softmax_scale=w.scale)
    torch.cuda.synchronize()
    assert_status_ok()
    kr, vr = u16(kc), u16(vc)
    oracle.kv_store(w.k.cpu(), w.v.cpu(), torch.from_numpy(w.slots), kr, vr)
    assert np.array_equal(u16(w.kc), kr) and np.array_equal(u16(w.vc), vr)
    w.check(out, w.reference(), shape)


@pytest.mark.parametrize("heads", [h for h in HEADS if h[0] <= 2 * h[1]], ids=lambda h: "%d/%d/%d" % h)
@pytest.mark.parametrize("shape", ["shared", "alone"])
def test_weights_are_held_to_15_bits(shape, heads):
    """Where attn_decode_paged has its weights in fp32 (one and two query heads
    per kv head), a weight is two bf16 numbers, off by 2^-15 at most.  Few keys,
    so that a rounding to one bf16 would show.  Against the tolerance above, with A as there:

      output                                      2^-8 |ref| (1 + 2^-6)
      weights                                     2^-15 A = 3.1e-5 A
      scores: d = 128 products, each sum within (d + 2) 2^-23 * scale * sum |q k|
      (< 10 here), if its additions cut off instead of rounding: 1.55e-4, on p and
      on the sum l                                3.1e-4 A
      exponents of at most 32 in fp32, exp2       5e-6 A, twice
      l and P V over at most 512 keys             512 (2^-24 + 2^-23) A = 9.2e-5 A

    together below 2^-11 A."""
    groups = {"shared": [(1 + i % 7, [1 + (3 * i + j) % 5 for j in range(2 + i % 4)]) for i in range(24)],
              "alone": [(0, [1 + (5 * i) % 60]) for i in range(70)]}[shape]
    w = Batch(heads, 16, groups, seed=31 + heads[0])
    plan = w.plan(16)
    assert any(plan_prefixes(plan, w.b)) == (shape == "shared")
    out = kvp.attn_decode_shared(w.q, w.kc, w.vc, w.dev(w.tables), plan, softmax_scale=w.scale)
    torch.cuda.synchronize()
    assert_status_ok()
    ref, a = w.reference()
    tol = 2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -6) + 2.0 ** -11 * np.abs(a)
    over = np.abs(out.float().cpu().double().numpy() - ref) - tol
    assert over.max() <= 0, f"{(over > 0).mean():.2%} past the tolerance"


@pytest.mark.parametrize("heads", HEADS, ids=lambda h: "%d/%d/%d" % h)
def test_infinite_values(heads):
    """An infinity in V at a key that is read is one in the output (weights are
    above 0), in the shared part, in a part of its own and in a single token's."""
    w = Batch(heads, 16, [(9, [20, 3, 1]), (0, [1]), (0, [40])], seed=17, poison=False)
    for b, pos, col, sign in ((0, 30, 2, 1), (0, 143, 5, -1), (1, 144, 7, 1), (3, 0, 9, -1), (4, 25, 11, 1)):
        w.vc[int(w.tables[b, pos // 16]), pos % 16, :, col] = sign * float("inf")
    out = kvp.attn_decode_shared(w.q, w.kc, w.vc, w.dev(w.tables), w.plan(), softmax_scale=w.scale)
    torch.cuda.synchronize()
    assert_status_ok()
    want = {2: [1, 1, 1, 0, 0], 5: [-1, -1, -1, 0, 0], 7: [0, 1, 0, 0, 0], 9: [0, 0, 0, -1, 0], 11: [0, 0, 0, 0, 1]}
    for col in range(w.d):
        for b, sign in enumerate(want.get(col, [0] * 5)):
            x = out[b, :, col].float()
            assert torch.all(x == sign * float("inf")) if sign else torch.isfinite(x).all(), (b, col)


def test_strided_rows():
    """q, k, v and out are views into wider rows; nothing beside them is written."""
    w = Batch((16, 8, 128), 32, [(6, [40, 9, 1]), (0, [77])], seed=3)
    qkv = torch.randn((w.b, 16 + 8 + 8 + 2, 128), device="cuda").to(BF16)
    qkv[:, :16], qkv[:, 16:24], qkv[:, 24:32] = w.q, w.k, w.v
    wide = torch.full((w.b, 20, 128), 7.0, dtype=BF16, device="cuda")
    kvp.attn_decode_shared_append(qkv[:, :16], qkv[:, 16:24], qkv[:, 24:32], w.dev(w.slots), w.kc, w.vc,
                                  w.dev(w.tables), w.plan(), softmax_scale=w.scale, out=wide[:, 2:18])
    torch.cuda.synchronize()
    assert_status_ok()
    w.check(wide[:, 2:18], w.reference(), "strided")
    assert torch.all(wide[:, :2] == 7) and torch.all(wide[:, 18:] == 7)


def test_large_and_masked_scores():
    """Scores that grow along the sequence (the running maximum moves all the
    time) and a key with -inf scores for every head."""
    w = Batch((16, 8, 128), 16, [(20, [33, 50, 1])], seed=9, poison=False)
    w.kc[int(w.tables[0, 3]), 5, :, :] = float("-inf")
    w.q.abs_()
    for i in range(w.tables.shape[1]):
        for page in set(w.tables[:, i].tolist()) - {-1}:
            w.kc[page] = (w.kc[page].float() * (0.2 + 0.35 * i)).to(BF16)
    w.kc[int(w.tables[0, 3]), 5, :, :] = float("-inf")
    out = kvp.attn_decode_shared(w.q, w.kc, w.vc, w.dev(w.tables), w.plan(), softmax_scale=w.scale)
    torch.cuda.synchronize()
    assert_status_ok()
    got = out.float().cpu().double().numpy()
    # fp64 from the definition (the scores reach some hundreds, so the fp32
    # sums' error is taken from the values: (d + 2) 2^-24 max sum |q k| scale)
    for b in range(w.b):
        n = int(w.lens[b])
        pages = torch.from_numpy(w.tables[b, :ceil(n, 16)].astype(np.int64)).cuda()
        k = w.kc[pages].reshape(-1, 8, 128)[:n].double()
        v = w.vc[pages].reshape(-1, 8, 128)[:n].double()
        for h in range(16):
            s = (k[:, h // 2] @ w.q[b, h].double()) * w.scale
            p = torch.softmax(s, 0)
            ref = (p @ v[:, h // 2]).cpu().numpy()
            a = (p @ v[:, h // 2].abs()).cpu().numpy()
            fin = torch.isfinite(s)
            size = ((k[fin][:, h // 2].abs() @ w.q[b, h].double().abs()) * w.scale).max().item()
            tol = 2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -6) + (2.0 ** -8 + 2.0 ** -9 + 4 * 130 * 2.0 ** -24 * size) * a
            assert (np.abs(got[b, h] - ref) <= tol).all(), (b, h)


@pytest.mark.parametrize("times", [-1.0, 0.0, 0.02, -1e-20, 1e-44])
def test_any_scale(times):
    """softmax_scale is any finite number, 0 (the values' mean) and negative
    ones too; prefixes that end inside a step of the prefix kernel."""
    w = Batch((16, 8, 128), 16, SHAPES["odd"], seed=22)
    w.scale *= times
    out = kvp.attn_decode_shared(w.q, w.kc, w.vc, w.dev(w.tables), w.plan(), softmax_scale=w.scale)
    torch.cuda.synchronize()
    assert_status_ok()
    w.check(out, w.reference(), str(times))


def test_plan_finds_the_groups():
    cases = [SHAPES[s] for s in ("odd", "many", "tall", "alone", "padding")]
    cases.append([(1, [3, 4]), (64, [5, 6, 7]), (8, [1, 2])])
    for i, groups in enumerate(cases):
        w = Batch((16, 8, 128), 16, groups, seed=i)
        # a page that every sequence has in common must not join the groups
        if i == 5:
            w.tables[:, 0] = w.tables[0, 0]
        for min_shared in (0, 16, 176):
            want = shared_prefixes(w.tables.tolist(), w.lens.tolist(), 16, min_shared or 128)
            assert plan_prefixes(w.plan(min_shared), w.b) == want, (i, min_shared)


def test_more_sequences_than_one_round_of_the_plan():
    """Over 1024 sequences, groups across the rounds' borders among them."""
    groups = [(9, [1 + i % 5 for i in range(700)])] + [(0, [3 + i % 40]) for i in range(200)]
    groups += [(8 + i % 7, [1 + (3 * j + i) % 30 for j in range(2 + i % 6)]) for i in range(120)]
    groups += [(20, [2] * 650), (0, [0] * 5)]
    w = Batch((4, 2, 64), 16, groups, seed=4)
    assert w.b > 1900
    plan = w.plan()
    assert plan_prefixes(plan, w.b) == shared_prefixes(w.tables.tolist(), w.lens.tolist(), 16)
    out = kvp.attn_decode_shared(w.q, w.kc, w.vc, w.dev(w.tables), plan, softmax_scale=w.scale)
    torch.cuda.synchronize()
    assert_status_ok()
    w.check(out, w.reference(), "many sequences")


@pytest.mark.parametrize("seed", range(24))
def test_random_tables(seed):
    """Any tables: pages shared by neighbours, by others, at other places, the
    same page twice in a row, and rows in any order."""
    rng = np.random.default_rng(1000 + seed)
    heads = HEADS[seed % len(HEADS)]
    bs = int(rng.choice([16, 32, 64, 256]))
    w = Batch(heads, bs, [(0, [1])], seed=seed, poison=False, extra=int(rng.integers(4, 60)))
    b, width = int(rng.integers(1, 90)), int(rng.integers(1, 40))
    tables = rng.integers(0, w.nb, (b, width))
    for i in range(1, b):  # leading pages of an earlier row, mostly of the one before
        if rng.random() < 0.7:
            j = i - 1 if rng.random() < 0.8 else int(rng.integers(0, i))
            n = int(rng.integers(0, width + 1)) if rng.random() < 0.5 else width
            tables[i, :n] = tables[j, :n]
    lens = rng.integers(0, width * bs + 1, b)
    lens[rng.random(b) < 0.5] = width * bs - int(rng.integers(0, bs))
    w.b, w.tables, w.lens = b, tables.astype(np.int32), lens.astype(np.int32)
    w.q = torch.randn((b, heads[0], heads[2]), device="cuda").to(BF16)
    min_shared = int(rng.choice([0, 1, 64, 300]))
    plan = w.plan(min_shared)
    assert plan_prefixes(plan, b) == shared_prefixes(w.tables.tolist(), lens.tolist(), bs, min_shared or 128)
    out = kvp.attn_decode_shared(w.q, w.kc, w.vc, w.dev(w.tables), plan, softmax_scale=w.scale)
    torch.cuda.synchronize()
    assert_status_ok()
    w.check(out, w.reference(), str(seed))


def test_same_sequence_twice_and_whole_rows_shared():
    """Forked rows before their first own token: identical tables and lengths."""
    for n in (129, 160, 161, 1):
        w = Batch((32, 8, 128), 16, [(0, [n])], seed=n)
        w.tables, w.lens, w.b = np.repeat(w.tables, 5, 0), np.repeat(w.lens, 5), 5
        w.q = torch.randn((5, 32, 128), device="cuda").to(BF16)
        out = kvp.attn_decode_shared(w.q, w.kc, w.vc, w.dev(w.tables), w.plan(), softmax_scale=w.scale)
        torch.cuda.synchronize()
        assert_status_ok()
        w.check(out, w.reference(), str(n))


def test_results_do_not_change_between_calls():
    w = Batch((32, 8, 128), 16, SHAPES["many"], seed=1)
    plan, bt = w.plan(), w.dev(w.tables)
    outs = [kvp.attn_decode_shared(w.q, w.kc, w.vc, bt, plan) for _ in range(6)]
    torch.cuda.synchronize()
    assert all(torch.equal(o.view(torch.int16), outs[0].view(torch.int16)) for o in outs)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(other):
        o = kvp.attn_decode_shared(w.q, w.kc, w.vc, bt, plan)
    other.synchronize()
    assert torch.equal(o.view(torch.int16), outs[0].view(torch.int16))


def test_two_streams_one_plan():
    """Calls that run side by side with workspaces of their own."""
    w = Batch((16, 8, 128), 16, SHAPES["many"], seed=2)
    plan, bt = w.plan(), w.dev(w.tables)
    want = kvp.attn_decode_shared(w.q, w.kc, w.vc, bt, plan)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [torch.empty(kvp.attn_decode_shared_workspace_size(w.b, 16, 8, 128), dtype=torch.uint8, device="cuda")
          for _ in streams]
    outs = [[torch.empty_like(want) for _ in range(20)] for _ in streams]
    for i in range(20):
        for s, st in enumerate(streams):
            with torch.cuda.stream(st):
                kvp.attn_decode_shared(w.q, w.kc, w.vc, bt, plan, workspace=ws[s], out=outs[s][i])
    torch.cuda.synchronize()
    assert_status_ok()
    assert all(torch.equal(o.view(torch.int16), want.view(torch.int16)) for group in outs for o in group)


def test_graph_replay_follows_the_tables():
    """plan + append captured once; the replays see other tables, lengths and
    slots, groups coming and going.  Two graphs share plan and workspace."""
    heads, bs = (16, 8, 128), 16
    w0 = Batch(heads, bs, [(10, [30, 31, 32, 33]), (0, [5, 6, 7, 8])], seed=0, extra=200)
    b, width, nb = w0.b, 60, w0.nb
    bt = torch.full((b, width), -1, dtype=I32, device="cuda")
    ctx, slots = torch.zeros(b, dtype=I32, device="cuda"), torch.full((b,), -1, dtype=I32, device="cuda")
    kc, vc = torch.zeros_like(w0.kc), torch.zeros_like(w0.vc)
    q, k, v = torch.zeros_like(w0.q), torch.zeros_like(w0.k), torch.zeros_like(w0.v)
    plan = torch.empty(kvp.attn_shared_plan_size(b, 16, 8), dtype=torch.uint8, device="cuda")
    ws = torch.empty(kvp.attn_decode_shared_workspace_size(b, 16, 8, 128), dtype=torch.uint8, device="cuda")
    outs = [torch.zeros_like(q) for _ in range(2)]

    def step(out):
        kvp.attn_shared_plan(bt, ctx, bs, 16, 8, nb, plan=plan)
        kvp.attn_decode_shared_append(q, k, v, slots, kc, vc, bt, plan, workspace=ws, out=out)

    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        step(outs[0])
    torch.cuda.synchronize()
    graphs = []
    for out in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            step(out)
        graphs.append(g)
    steps = [[(10, [30, 31, 32, 33]), (0, [5, 6, 7, 8])], [(0, [9] * 8)], [(9, [1, 2]), (30, [3, 4, 5, 6, 7, 8])],
             [(0, [0] * 8)], [(12, [100] * 8)]]
    for i, groups in enumerate(steps):
        w = Batch(heads, bs, groups, seed=50 + i, extra=0)
        assert w.nb <= nb
        kc[:w.nb], vc[:w.nb] = w.kc, w.vc
        bt.fill_(-1)
        bt[:, :w.tables.shape[1]] = w.dev(w.tables)
        ctx.copy_(w.dev(w.lens))
        slots.copy_(w.dev(w.slots))
        q.copy_(w.q), k.copy_(w.k), v.copy_(w.v)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert_status_ok()
        w.kc, w.vc = kc[:w.nb].clone(), vc[:w.nb].clone()
        ref = w.reference()
        for out in outs:
            w.check(out, ref, f"step {i}")


def test_pages_past_2_31_elements():
    """A cache of 3.1e9 elements, the batch's pages at its far end."""
    w = Batch((16, 8, 128), 256, [(3, [100, 300]), (0, [513])], seed=6)
    nb = 12000
    ids = np.arange(nb - w.nb, nb)
    kc, vc = (torch.empty((nb, 256, 8, 128), dtype=BF16, device="cuda") for _ in range(2))
    kc[nb - w.nb:], vc[nb - w.nb:] = w.kc, w.vc
    tables = np.where(w.tables >= 0, ids[w.tables], -1).astype(np.int32)
    slots = np.array([ids[s // 256] * 256 + s % 256 for s in w.slots], np.int32)
    plan = kvp.attn_shared_plan(w.dev(tables), w.dev(w.lens), 256, 16, 8, nb)
    out = kvp.attn_decode_shared_append(w.q, w.k, w.v, w.dev(slots), kc, vc, w.dev(tables), plan)
    torch.cuda.synchronize()
    assert_status_ok()
    kr, vr = u16(w.kc), u16(w.vc)
    oracle.kv_store(w.k.cpu(), w.v.cpu(), torch.from_numpy(w.slots), kr, vr)
    assert np.array_equal(u16(kc[nb - w.nb:]), kr) and np.array_equal(u16(vc[nb - w.nb:]), vr)
    w.check(out, w.reference(kc[nb - w.nb:], vc[nb - w.nb:]))


def test_out_may_be_q():
    w = Batch((32, 8, 128), 16, SHAPES["odd"], seed=21)
    ref = w.reference()
    out = kvp.attn_decode_shared(w.q, w.kc, w.vc, w.dev(w.tables), w.plan(), out=w.q)
    torch.cuda.synchronize()
    assert_status_ok()
    assert out.data_ptr() == w.q.data_ptr()
    w.check(out, ref, "in place")


def test_empty_batch():
    w = Batch((16, 8, 128), 16, [(0, [4])], seed=0)
    e = torch.zeros((0, 16, 128), dtype=BF16, device="cuda")
    bt = torch.zeros((0, 3), dtype=I32, device="cuda")
    plan = kvp.attn_shared_plan(bt, torch.zeros(0, dtype=I32, device="cuda"), 16, 16, 8, w.nb)
    assert kvp.attn_decode_shared(e, w.kc, w.vc, bt, plan).shape == (0, 16, 128)
    torch.cuda.synchronize()
    assert_status_ok()


def test_buffers_that_are_too_small_are_refused():
    w = Batch((16, 8, 128), 16, [(10, [3, 4])], seed=8)
    bt, plan = w.dev(w.tables), w.plan()
    need = kvp.attn_shared_plan_size(2, 16, 8)
    assert need < kvp.attn_shared_plan_size(512, 16, 8) and kvp.attn_shared_plan_size(0, 16, 8) > 0
    small = torch.empty(need - 1, dtype=torch.uint8, device="cuda")
    with pytest.raises(kvp.KvpError, match="plan needs %d bytes" % need):
        kvp.attn_shared_plan(bt, w.dev(w.lens), 16, 16, 8, w.nb, plan=small)
    with pytest.raises(kvp.KvpError, match="plan needs %d bytes" % need):
        kvp.attn_decode_shared(w.q, w.kc, w.vc, bt, small)
    need = kvp.attn_decode_shared_workspace_size(2, 16, 8, 128)
    small = torch.empty(need - 1, dtype=torch.uint8, device="cuda")
    with pytest.raises(kvp.KvpError, match="workspace needs %d bytes" % need):
        kvp.attn_decode_shared(w.q, w.kc, w.vc, bt, plan, workspace=small)


def test_arguments_of_the_wrong_kind_are_named():
    w = Batch((16, 8, 128), 16, [(10, [3, 4])], seed=8)
    bt, lens, slots, plan = w.dev(w.tables), w.dev(w.lens), w.dev(w.slots), w.plan()
    ok = dict(q=w.q, k=w.k, v=w.v, slot_mapping=slots, k_cache=w.kc, v_cache=w.vc, block_tables=bt, plan=plan)
    wide = torch.empty((2, 16, 130), dtype=BF16, device="cuda")
    cases = [(TypeError, "q must be", dict(q=w.q.float())), (ValueError, "head_dim", dict(q=w.q[..., :64])),
             (ValueError, "contiguous", dict(q=wide[..., :128])),
             (ValueError, "k must have one row", dict(k=w.k[:1])), (ValueError, "v must be a CUDA", dict(v=w.v.cpu())),
             (TypeError, "k must be", dict(k=None)), (TypeError, "v must be", dict(v=None)),
             (ValueError, "slot_mapping", dict(slot_mapping=slots[:1])),
             (TypeError, "slot_mapping", dict(slot_mapping=slots.long())),
             (ValueError, "block_tables", dict(block_tables=bt.t().contiguous().t())),
             (TypeError, "plan", dict(plan=None)), (TypeError, "plan", dict(plan=plan.float())),
             (ValueError, "out", dict(out=torch.empty((2, 16, 64), dtype=BF16, device="cuda"))),
             (ValueError, "v_cache|caches", dict(v_cache=w.vc[:-1])),
             (TypeError, "workspace", dict(workspace=torch.empty(9, device="cuda")))]
    for error, match, change in cases:
        with pytest.raises(error, match=match):
            kvp.attn_decode_shared_append(**{**ok, **change})
    for error, match, args in ((ValueError, "context_lens", (bt, lens[:1])), (TypeError, "context_lens", (bt, lens.long())),
                               (ValueError, "block_tables", (bt[0], lens)), (TypeError, "block_tables", (None, lens))):
        with pytest.raises(error, match=match):
            kvp.attn_shared_plan(*args, 16, 16, 8, w.nb)
    # numbers of other types are taken as they are elsewhere
    a = kvp.attn_decode_shared(w.q, w.kc, w.vc, bt, plan, softmax_scale=1)
    b = kvp.attn_decode_shared(w.q, w.kc, w.vc, bt, plan, softmax_scale=1.0)
    torch.cuda.synchronize()
    assert_status_ok()
    assert torch.equal(a, b)


def test_wrong_metadata_is_reported():
    """A plan of another shape writes nothing; a page outside the pool, a
    length past the table and a slot that is not the last token's are
    reported, and the other sequences are right."""
    w = Batch((16, 8, 128), 16, [(10, [3, 4, 40]), (0, [20])], seed=8, poison=False)
    bt, plan = w.dev(w.tables), w.plan()
    out = torch.full_like(w.q, 3.0)
    kvp.device_status()
    kvp.attn_decode_shared(w.q[:3], w.kc, w.vc, bt[:3], plan, out=out[:3])
    torch.cuda.synchronize()
    assert kvp.device_status() == -6 and torch.all(out == 3)
    ref = w.reference()
    good = w.tables.copy()
    for bad_id in (-1, w.nb, 1 << 30):
        bad = good.copy()
        bad[2, 11] = bad_id  # a page of sequence 2's own part
        out = kvp.attn_decode_shared(w.q, w.kc, w.vc, w.dev(bad), plan)
        torch.cuda.synchronize()
        assert kvp.device_status() == -6
        keep = [0, 1, 3]
        tol = 2.0 ** -8 * np.abs(ref[0]) * (1 + 2.0 ** -6) + (2.0 ** -8 + 2.0 ** -9) * ref[1]
        err = np.abs(out.float().cpu().double().numpy() - ref[0])
        assert (err[keep] <= tol[keep]).all()
        bad = good.copy()
        bad[:3, 4] = bad_id  # in the shared part
        w2 = kvp.attn_shared_plan(w.dev(bad), w.dev(w.lens), 16, 16, 8, w.nb)
        kvp.attn_decode_shared(w.q, w.kc, w.vc, w.dev(bad), w2)
        torch.cuda.synchronize()
        assert kvp.device_status() == -6
    lens = w.lens.copy()
    lens[3] = w.tables.shape[1] * 16 + 1
    p = kvp.attn_shared_plan(bt, w.dev(lens), 16, 16, 8, w.nb)
    torch.cuda.synchronize()
    assert kvp.device_status() == -6
    slots = w.slots.copy()
    slots[1] += 1 if slots[1] % 16 < 15 else -1
    kvp.attn_decode_shared_append(w.q, w.k, w.v, w.dev(slots), w.kc, w.vc, bt, plan)
    torch.cuda.synchronize()
    assert kvp.device_status() == -6
    slots[1] = w.nb * 16
    kvp.attn_decode_shared_append(w.q, w.k, w.v, w.dev(slots), w.kc, w.vc, bt, plan)
    torch.cuda.synchronize()
    assert kvp.device_status() == -6
