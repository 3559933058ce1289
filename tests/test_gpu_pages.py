"""kv_pages_fork / kv_pages_extend / kv_pages_compact against plain host
implementations (tests/pages_reference.py): tables, lengths, counts, slots and
every byte of the cache, bit for bit."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
import pages_reference as ref
import paged_kv_cache_125_gb300 as kvp

from parity import assert_attn_close, u16

pytestmark = pytest.mark.gpu
BF16, I32 = torch.bfloat16, torch.int32


def dev(x, shape=None):
    a = np.asarray(x, np.int32)
    return torch.from_numpy(a.reshape(shape) if shape else a).cuda()


def bits(shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randint(-(1 << 15), 1 << 15, shape, generator=g, device="cuda", dtype=torch.int32)
    return x.to(torch.int16).view(BF16)


def raw(t):
    return t.view(torch.int16).cpu().numpy()


class Pool:
    """Rows of random lengths; some share leading pages."""

    def __init__(self, nb, bs, rows, width, seed, share=0.4, fill=0.7, pins=3):
        rng = np.random.default_rng(seed)
        self.nb, self.bs, self.width = nb, bs, width
        free = list(rng.permutation(nb))
        self.counts = [0] * nb
        for p in [free.pop() for _ in range(min(pins, nb // 4))]:
            self.counts[p] = 1  # held by someone outside the tables
        self.tables, self.lens = [], []
        budget = int(nb * fill)
        for _ in range(rows):
            n = int(rng.integers(0, width * bs + 1))
            n = min(n, max(0, (budget - (nb - len(free))) * bs))
            row = []
            if self.tables and rng.random() < share:  # leading full pages of an earlier row
                p = int(rng.integers(len(self.tables)))
                row = self.tables[p][:min(self.lens[p], n) // bs]
            while len(row) < ref.ceil(n, bs):
                row = row + [int(free.pop())]
            self.tables.append(row)
            self.lens.append(n)
            for e in row:
                self.counts[e] += 1
        self.rng = rng
        self.tables = [list(map(int, r)) + [-1] * (width - len(r)) for r in self.tables]

    def args(self):
        return dev(self.tables, (len(self.tables), self.width)), dev(self.lens), dev(self.counts)


POOLS = [(12, 16, 3, 3), (40, 16, 7, 5), (200, 1, 9, 20), (300, 32, 40, 9), (700, 7, 90, 13), (5000, 16, 300, 40),
         (9000, 256, 1100, 8), (600001, 2, 70, 3001)]


def check_status(bad):
    torch.cuda.synchronize()
    assert kvp.device_status() == (-6 if bad else 0)


@pytest.mark.parametrize("pool", POOLS, ids=str)
@pytest.mark.parametrize("kind", ["identity", "random", "all_from_one", "none", "fewer", "more"])
def test_fork(pool, kind):
    p = Pool(*pool, seed=pool[0] + len(kind))
    n = len(p.tables)
    m = {"fewer": max(1, n // 3), "more": 2 * n + 1}.get(kind, n)
    parents = {"identity": list(range(n)), "all_from_one": [int(np.argmax(p.lens))] * n, "none": [-1] * n}.get(
        kind, p.rng.integers(-1, n, m).tolist())
    row, planes = (2, 64), 3
    cache = bits((planes, p.nb, p.bs, *row), 5)
    want = raw(cache).copy()
    t, l, c, copies, bad = ref.fork(p.tables, p.lens, p.counts, parents, p.bs)
    for s, d, k in copies:
        want[:, d, :k] = want[:, s, :k]
    kvp.device_status()
    ot, ol, oc = kvp.kv_pages_fork(cache, *p.args(), dev(parents))
    check_status(bad)
    assert ol.tolist() == l and oc.tolist() == c and ot.tolist() == t
    assert np.array_equal(raw(cache), want)


def test_fork_when_the_pool_runs_out():
    """Rows past the last free page become empty and let go of their pages."""
    bs, nb = 16, 9
    tables = [[0, 1, 2, -1], [3, 4, -1, -1]]
    lens, counts = [40, 20], [1, 1, 1, 1, 1, 0, 1, 1, 0]
    for parents in ([0, 0, 0, 0, 1, 1], [1, 1, 1, 0, 0, 1], [0] * 6, [1, -1, 1, 1, 1]):
        t, l, c, copies, bad = ref.fork(tables, lens, counts, parents, bs)
        cache = bits((4, nb, bs, 1, 64), 1)
        want = raw(cache).copy()
        for s, d, k in copies:
            want[:, d, :k] = want[:, s, :k]
        kvp.device_status()
        ot, ol, oc = kvp.kv_pages_fork(cache, dev(tables), dev(lens), dev(counts), dev(parents))
        check_status(bad)
        assert (ot.tolist(), ol.tolist(), oc.tolist()) == (t, l, c)
        assert np.array_equal(raw(cache), want)


def test_fork_wrong_metadata():
    """Parents, lengths and pages outside their ranges."""
    tables = [[0, 1, -1], [7, 99, 2], [3, -1, -1], [4, 5, 6]]
    lens, counts = [17, 40, 49, -5], [1] * 8 + [0] * 6
    for parents in ([0, 1, 1, 2], [4, -2, 3, 0], [1 << 30, 0, 0, 0]):
        t, l, c, copies, bad = ref.fork(tables, lens, counts, parents, 16)
        cache = bits((2, 14, 16, 1, 64), 1)
        kvp.device_status()
        ot, ol, oc = kvp.kv_pages_fork(cache, dev(tables), dev(lens), dev(counts), dev(parents))
        check_status(bad)
        assert bad and (ot.tolist(), ol.tolist(), oc.tolist()) == (t, l, c)


@pytest.mark.parametrize("row_elems,offset", [(12, 0), (64, 1), (8, 0)])
def test_copies_of_unaligned_rows(row_elems, offset):
    """Rows that are not whole 16-byte units, and a cache off a 16-byte boundary."""
    nb, bs, planes = 10, 16, 3
    tables, lens, counts, parents = [[4, 8], [1, -1]], [21, 9], [0, 1, 0, 0, 1, 0, 0, 0, 1, 0], [0, 0, 1, 1, 0]
    t, l, c, copies, _ = ref.fork(tables, lens, counts, parents, bs)
    flat = bits((planes * nb * bs * row_elems + 8,), 2)
    cache = flat[offset:offset + planes * nb * bs * row_elems]
    want = raw(flat).copy()
    w = want[offset:offset + cache.numel()].reshape(planes, nb, bs, row_elems)
    for s, d, k in copies:
        w[:, d, :k] = w[:, s, :k]
    lib = kvp.library()
    it, il, ic, ip = dev(tables), dev(lens), dev(counts), dev(parents)
    ot, ol, oc = dev([[0, 0]] * 5), dev([0] * 5), dev([0] * nb)
    ws = torch.empty(kvp.kv_pages_workspace_size(nb, 5), dtype=torch.uint8, device="cuda")
    rc = lib.kv_pages_fork(cache.data_ptr(), planes, nb * bs * row_elems, nb, bs, row_elems, it.data_ptr(), 2,
                           il.data_ptr(), 2, ic.data_ptr(), ip.data_ptr(), 5, ot.data_ptr(), ol.data_ptr(),
                           oc.data_ptr(), ws.data_ptr(), ws.numel(),
                           ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert rc == 0, lib.kvp_last_error()
    check_status(False)
    assert (ot.tolist(), ol.tolist(), oc.tolist()) == (t, l, c)
    assert np.array_equal(raw(flat), want)


@pytest.mark.parametrize("pool", POOLS, ids=str)
@pytest.mark.parametrize("kind", ["one", "ragged", "none", "too_many", "first"])
@pytest.mark.parametrize("in_place", [False, True])
def test_extend(pool, kind, in_place):
    p = Pool(*pool, seed=pool[0] + len(kind), share=0.4 if kind != "first" else 0.0)
    n, cap = len(p.tables), p.width * p.bs
    if kind == "first":
        p.lens = [0] * n
        p.counts = [1 if c and p.rng.random() < 0.3 else 0 for c in p.counts]
    room = [cap - x for x in p.lens]
    new = {"one": [min(1, r) for r in room], "none": [0] * n,
           "ragged": [int(p.rng.integers(0, min(r, 3 * p.bs) + 1)) for r in room],
           "first": [int(p.rng.integers(0, min(r, 2 * p.bs) + 1)) for r in room],
           "too_many": [int(p.rng.integers(-1, r + 3)) for r in room]}[kind]
    total = sum(x for x, r in zip(new, room) if 0 <= x <= r) + 5
    t, l, c, s, bad = ref.extend(p.tables, p.lens, p.counts, new, p.bs, total)
    a = p.args()
    kvp.device_status()
    if in_place:
        slots = torch.full((total,), 77, dtype=I32, device="cuda")
        kvp.kv_pages_extend(*a, dev(new), p.bs, total, out=(*a, slots))
        ot, ol, oc = a
    else:
        before = [x.clone() for x in a]
        ot, ol, oc, slots = kvp.kv_pages_extend(*a, dev(new), p.bs, total)
        assert all(torch.equal(x, y) for x, y in zip(a, before))
    check_status(bad)
    assert ol.tolist() == l and slots.tolist() == s and oc.tolist() == c and ot.tolist() == t


def test_extend_refuses_what_is_not_its_own():
    """An unfilled last page with another holder; fewer slots than tokens;
    lengths and pages outside; huge counts of new tokens."""
    tables, lens = [[0, 1, -1], [2, -1, -1], [9, -1, -1], [3, 4, 5]], [20, 9, 4, 99]
    counts = [1, 2, 1, 1, 1, 1, 0, 0]
    for new, slots in (([1, 1, 1, 1], 4), ([12, 30, 0, 0], 50), ([0, 8, 0, 0], 3),
                       ([1 << 30, 2, 1 << 30, 1 << 30], 9), ([-1, -1, -7, 1], 2)):
        t, l, c, s, bad = ref.extend(tables, lens, counts, new, 16, slots)
        kvp.device_status()
        ot, ol, oc, os_ = kvp.kv_pages_extend(dev(tables), dev(lens), dev(counts), dev(new), 16, slots)
        check_status(bad)
        assert bad and (ol.tolist(), os_.tolist(), oc.tolist(), ot.tolist()) == (l, s, c, t), new


@pytest.mark.parametrize("pool", POOLS, ids=str)
@pytest.mark.parametrize("fill", [0.0, 0.2, 0.95])
def test_compact(pool, fill):
    p = Pool(*pool, seed=pool[0], fill=fill)
    cache = bits((3, p.nb, p.bs, 1, 64), 5)
    want = raw(cache).copy()
    t, c, places, moves, bad = ref.compact(p.tables, p.lens, p.counts, p.bs)
    for s, d in moves:
        want[:, d] = want[:, s]
    kvp.device_status()
    ot, oc, op = kvp.kv_pages_compact(cache, *p.args())
    check_status(bad)
    assert not bad and oc.tolist() == c and op.tolist() == places and ot.tolist() == t
    assert np.array_equal(raw(cache), want)


def test_compact_all_live_all_free_and_wrong_pages():
    for counts in ([1] * 20, [0] * 20, [0] * 19 + [1], [1] + [0] * 19):
        tables, lens = [[19, 0, 50], [3, -1, -1]], [33, 60]
        cache = bits((2, 20, 16, 1, 64), 3)
        want = raw(cache).copy()
        t, c, places, moves, bad = ref.compact(tables, lens, counts, 16)
        for s, d in moves:
            want[:, d] = want[:, s]
        kvp.device_status()
        ot, oc, op = kvp.kv_pages_compact(cache, dev(tables), dev(lens), dev(counts))
        check_status(bad)
        assert (ot.tolist(), oc.tolist(), op.tolist()) == (t, c, places)
        assert np.array_equal(raw(cache), want)


def test_moves_across_2_32_bytes():
    """Copies from the end of a pool of 12.6 GB to its start, in both planes."""
    nb, bs = 12000, 256
    cache = torch.empty((2, nb, bs, 8, 128), dtype=BF16, device="cuda")
    tables = [[nb - 1, nb - 2, 5, nb // 2], [nb - 7, -1, -1, -1]]
    lens, counts = [4 * bs - 3, 100], [0] * nb
    for p in tables[0] + tables[1][:1]:
        counts[p] = 1
        cache[:, p] = bits((2, bs, 8, 128), p)
    t, c, places, moves, bad = ref.compact(tables, lens, counts, bs)
    want = {d: raw(cache[:, s]).copy() for s, d in moves}
    kvp.device_status()
    ot, oc, op = kvp.kv_pages_compact(cache, dev(tables), dev(lens), dev(counts))
    check_status(bad)
    assert (ot.tolist(), oc.tolist(), op.tolist()) == (t, c, places) and len(moves) == 5
    for d, w in want.items():
        assert np.array_equal(raw(cache[:, d]), w), d
    parents = [0, 0, 1, 1]
    t2, l2, c2, copies, bad = ref.fork(t, lens, c, parents, bs)
    ot2, ol2, oc2 = kvp.kv_pages_fork(cache, ot, dev(lens), oc, dev(parents))
    check_status(bad)
    assert (ot2.tolist(), ol2.tolist(), oc2.tolist()) == (t2, l2, c2) and len(copies) == 2
    for s, d, n in copies:
        assert torch.equal(cache[:, d, :n].view(torch.int16), cache[:, s, :n].view(torch.int16))


@pytest.mark.parametrize("kind", ["one", "ragged"])
def test_extend_beside_other_work(kind):
    """Rows with unfilled last pages in a table so large that CTAs beside the
    team keep it, into outputs that hold other pages' ids, while matrix
    products of a second stream have SMs: the slots of a page that the row had
    must not wait for its entry in the new table."""
    bs, rows, width = 16, 512, 500
    rng = np.random.default_rng(7)
    lens = [int(x) // bs * bs + int(rng.integers(1, bs)) for x in rng.integers(128, (width - 4) * bs, rows)]
    held = sum(ref.ceil(n, bs) for n in lens)
    nb = held + 3 * rows
    ids, at, tables, counts = rng.permutation(nb).tolist(), 0, [], [0] * nb
    for n in lens:
        row, at = ids[at:at + ref.ceil(n, bs)], at + ref.ceil(n, bs)
        tables.append(row + [-1] * (width - len(row)))
        for p in row:
            counts[p] = 1
    new = [1] * rows if kind == "one" else rng.integers(0, 2 * bs, rows).tolist()
    total = sum(new)
    t, l, c, s, bad = ref.extend(tables, lens, counts, new, bs, total)
    assert not bad
    args, new = (dev(tables), dev(lens), dev(counts)), dev(new)
    want = [dev(x) for x in (t, l, c, s)]
    outs = [[torch.empty_like(x) for x in want] for _ in range(8)]
    side, m = torch.cuda.Stream(), torch.randn((4096, 4096), device="cuda").to(BF16)
    kvp.device_status()
    for i in range(12):
        for out in outs:
            for x in out:
                x.fill_((i * 977 + 5) % nb)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for _ in range(6):
                torch.matmul(m, m)
        for out in outs:
            kvp.kv_pages_extend(*args, new, bs, total, out=out)
        check_status(False)
        for out in outs:
            assert all(torch.equal(x, y) for x, y in zip(out, want)), i


def test_more_rows_than_fit_in_shared_memory():
    """Over 2048 rows: the searches of kv_pages_extend go through the workspace."""
    p = Pool(9000, 16, 2600, 4, seed=3)
    new = [int(p.rng.integers(0, min(64 - x, 20) + 1)) for x in p.lens]
    total = sum(new)
    t, l, c, s, bad = ref.extend(p.tables, p.lens, p.counts, new, 16, total)
    kvp.device_status()
    ot, ol, oc, slots = kvp.kv_pages_extend(*p.args(), dev(new), 16, total)
    check_status(bad)
    assert ol.tolist() == l and slots.tolist() == s and oc.tolist() == c and ot.tolist() == t
    parents = p.rng.integers(-1, 2600, 3000).tolist()
    cache = bits((1, 9000, 16, 1, 64), 4)
    want = raw(cache).copy()
    t2, l2, c2, copies, bad = ref.fork(t, l, c, parents, 16)
    for a, b, n in copies:
        want[:, b, :n] = want[:, a, :n]
    ot, ol, oc = kvp.kv_pages_fork(cache, ot, ol, oc, dev(parents))
    check_status(bad)
    assert (ot.tolist(), ol.tolist(), oc.tolist()) == (t2, l2, c2)
    assert np.array_equal(raw(cache), want)


def test_empty_tables():
    cache = bits((2, 6, 16, 1, 64), 3)
    before = raw(cache).copy()
    none, counts = torch.zeros((0, 4), dtype=I32, device="cuda"), dev([0, 1, 0, 0, 0, 2])
    z = torch.zeros(0, dtype=I32, device="cuda")
    t, l, c = kvp.kv_pages_fork(cache, none, z, counts, z)
    assert t.shape == (0, 4) and torch.equal(c, counts) and np.array_equal(raw(cache), before)
    t, l, c = kvp.kv_pages_fork(cache, none, z, counts, dev([-1, -1]))
    assert t.tolist() == [[-1] * 4] * 2 and l.tolist() == [0, 0] and torch.equal(c, counts)
    t, l, c, s = kvp.kv_pages_extend(none, z, counts, z, 16, 3)
    assert s.tolist() == [-1] * 3 and torch.equal(c, counts)
    want = ref.compact([], [], counts.tolist(), 16)
    t, c, places = kvp.kv_pages_compact(cache, none, z, counts)
    assert c.tolist() == want[1] and places.tolist() == want[2]
    check_status(False)


def test_arguments_of_the_wrong_kind_are_named():
    p = Pool(60, 16, 5, 6, seed=3)
    bt, lens, counts = p.args()
    cache, par = bits((2, 60, 16, 1, 64), 3), dev([0, 1])
    i32 = dict(dtype=I32, device="cuda")
    for error, match, call in (
            (ValueError, "ref_counts", lambda: kvp.kv_pages_fork(cache, bt, lens, counts[:-1], par)),
            (TypeError, "parents", lambda: kvp.kv_pages_fork(cache, bt, lens, counts, par.long())),
            (TypeError, "parents", lambda: kvp.kv_pages_fork(cache, bt, lens, counts, [0, 1])),
            (ValueError, "kv_cache", lambda: kvp.kv_pages_fork(cache[0, 0], bt, lens, counts, par)),
            (ValueError, "kv_cache", lambda: kvp.kv_pages_fork(cache.transpose(0, 1), bt, lens, counts, par)),
            (ValueError, "3 tensors", lambda: kvp.kv_pages_fork(cache, bt, lens, counts, par, out=(bt, lens))),
            (ValueError, "out tables", lambda: kvp.kv_pages_fork(
                cache, bt, lens, counts, par, out=(bt.clone(), lens.clone(), counts.clone()))),
            (kvp.KvpError, "overlaps an input", lambda: kvp.kv_pages_fork(
                cache, bt, lens, counts, dev(range(5)), out=(bt, lens.clone(), counts.clone()))),
            (kvp.KvpError, "workspace needs", lambda: kvp.kv_pages_fork(
                cache, bt, lens, counts, par, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))),
            (ValueError, "context_lens", lambda: kvp.kv_pages_extend(bt, lens[:-1], counts, lens, 16, 4)),
            (ValueError, "new_tokens", lambda: kvp.kv_pages_extend(bt, lens, counts, lens.cpu(), 16, 4)),
            (ValueError, "slot_mapping", lambda: kvp.kv_pages_extend(
                bt, lens, counts, dev([0] * 5), 16, 4, out=[bt, lens, counts, torch.empty(3, **i32)])),
            (ValueError, "block_tables", lambda: kvp.kv_pages_compact(cache, bt.t().contiguous().t(), lens, counts)),
            (ValueError, "places", lambda: kvp.kv_pages_compact(
                cache, bt, lens, counts, out=(bt.clone(), counts.clone(), par)))):
        with pytest.raises(error, match=match):
            call()
    check_status(False)


def test_given_outputs_are_returned():
    p = Pool(60, 16, 5, 6, seed=4)
    bt, lens, counts = p.args()
    out = [torch.empty((2, 6), dtype=I32, device="cuda"), torch.empty(2, dtype=I32, device="cuda"), counts.clone()]
    got = kvp.kv_pages_fork(bits((2, 60, 16, 1, 64), 3), bt, lens, counts, dev([3, 3]), out=out)
    assert isinstance(got, tuple) and all(a is b for a, b in zip(got, out))
    out = [bt, lens, counts, torch.empty(9, dtype=I32, device="cuda")]
    got = kvp.kv_pages_extend(bt, lens, counts, dev([1] * 5), 16, 9, out=out)
    assert isinstance(got, tuple) and all(a is b for a, b in zip(got, out))
    torch.cuda.synchronize()
    kvp.device_status()  # (whether the rows fit is not this test's matter)


def test_work_of_another_stream_is_waited_for():
    """The inputs are written late on one stream; the calls run on another one
    that waits for it, behind a kernel of its own."""
    p = Pool(700, 16, 60, 9, seed=8)
    real, parents, new = p.args(), dev(p.rng.integers(-1, 60, 50)), dev(p.rng.integers(0, 3, 60))
    cache = bits((1, 700, 16, 1, 64), 5)
    image = raw(cache).copy()

    def ops(a):
        return (*kvp.kv_pages_fork(cache, *a, parents), *kvp.kv_pages_extend(*a, new, 16, 180),
                *kvp.kv_pages_compact(cache, *a), kvp.attn_shared_plan(a[0], a[1], 16, 2, 1, 700))

    want = [x.clone() for x in ops(real)]
    after = raw(cache).copy()
    kvp.device_status()  # (rows that cannot grow are not this test's matter)
    for _ in range(3):
        cache.copy_(torch.from_numpy(image).cuda().view(BF16))
        a = [torch.zeros_like(x) for x in real]
        torch.cuda.synchronize()
        writer, reader = torch.cuda.Stream(), torch.cuda.Stream()
        with torch.cuda.stream(writer):
            torch.cuda._sleep(4_000_000)
            for x, y in zip(a, real):
                x.copy_(y)
        with torch.cuda.stream(reader):
            torch.zeros(1000, device="cuda").add_(1)
            reader.wait_stream(writer)
            got = ops(a)
        torch.cuda.synchronize()
        kvp.device_status()
        assert all(torch.equal(x, y) for x, y in zip(got[:-1], want[:-1]))
        assert torch.equal(got[-1][:80], want[-1][:80])  # the plan's head, its totals among it
        assert np.array_equal(raw(cache), after)


def test_results_do_not_depend_on_order():
    p = Pool(5000, 16, 300, 40, seed=1)
    parents = dev(p.rng.integers(0, 300, 300))
    cache = bits((2, p.nb, 16, 1, 64), 5)
    a = p.args()
    first = kvp.kv_pages_fork(cache, *a, parents)
    image = raw(cache).copy()
    for _ in range(5):
        again = kvp.kv_pages_fork(cache, *a, parents)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(first, again))
        assert np.array_equal(raw(cache), image)


def test_beam_search_loop_in_one_graph():
    """extend -> plan + shared decode with the store -> fork, captured once and
    replayed: the arrays live on the device, every replay's state is checked
    against the host implementations and the oracle; compaction at the end."""
    hq, hkv, d, bs, layers, rows, width, nb = 4, 2, 64, 16, 2, 6, 20, 90
    g = torch.Generator(device="cuda").manual_seed(1)
    rng = np.random.default_rng(2)
    cache = torch.randn((2, layers, nb, bs, hkv, d), generator=g, device="cuda").to(BF16)
    prompt = [int(x) for x in rng.permutation(nb)[:12]]
    n0 = 12 * bs - 3
    # one prompt; the first fork spreads it over the beams
    tables, lens, counts = [prompt + [-1] * (width - 12)], [n0], [0] * nb
    for p in prompt:
        counts[p] = 1
    t, l, c = kvp.kv_pages_fork(cache, dev(tables), dev(lens), dev(counts), dev([0] * rows))
    tables, lens, counts, copies, bad = ref.fork(tables, lens, counts, [0] * rows, bs)
    assert not bad and (t.tolist(), l.tolist(), c.tolist()) == (tables, lens, counts) and len(copies) == rows - 1
    state = [t, l, c]
    ext = [torch.empty_like(x) for x in state] + [torch.empty(rows, dtype=I32, device="cuda")]
    new, parents = torch.ones(rows, dtype=I32, device="cuda"), torch.zeros(rows, dtype=I32, device="cuda")
    q = torch.zeros((layers, rows, hq, d), dtype=BF16, device="cuda")
    k, v = (torch.zeros((layers, rows, hkv, d), dtype=BF16, device="cuda") for _ in range(2))
    out = torch.zeros_like(q)
    plan = torch.empty(kvp.attn_shared_plan_size(rows, hq, hkv), dtype=torch.uint8, device="cuda")
    ws = torch.empty(kvp.attn_decode_shared_workspace_size(rows, hq, hkv, d), dtype=torch.uint8, device="cuda")
    pws = torch.empty(kvp.kv_pages_workspace_size(nb, rows), dtype=torch.uint8, device="cuda")

    def step():
        kvp.kv_pages_extend(*state, new, bs, rows, workspace=pws, out=ext)
        kvp.attn_shared_plan(ext[0], ext[1], bs, hq, hkv, nb, plan=plan)
        for i in range(layers):
            kvp.attn_decode_shared_append(q[i], k[i], v[i], ext[3], cache[0, i], cache[1, i], ext[0], plan,
                                          workspace=ws, out=out[i])
        kvp.kv_pages_fork(cache, *ext[:3], parents, workspace=pws, out=state)

    saved = [x.clone() for x in (*state, cache)]
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step()
    for x, y in zip((*state, cache), saved):
        x.copy_(y)
    kvp.device_status()
    for i in range(40):
        choice = rng.integers(0, rows, rows).tolist()
        parents.copy_(dev(choice))
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
        image = raw(cache).view(np.uint16).copy()
        graph.replay()
        check_status(False)
        tables, lens, counts, slots, bad = ref.extend(tables, lens, counts, [1] * rows, bs, rows)
        assert not bad and ext[3].tolist() == slots and ext[0].tolist() == tables
        for layer in range(layers):
            kc, vc = np.ascontiguousarray(image[0, layer]), np.ascontiguousarray(image[1, layer])
            oracle.kv_store(k[layer].cpu(), v[layer].cpu(), torch.tensor(slots, dtype=I32), kc, vc)
            want = oracle.decode(q[layer].cpu(), kc, vc, torch.tensor(tables, dtype=I32),
                                 torch.tensor(lens, dtype=I32), hq, hkv, d ** -0.5)
            assert_attn_close(out[layer], want, f"step {i} layer {layer}")
            image[0, layer], image[1, layer] = kc, vc
        tables, lens, counts, copies, bad = ref.fork(tables, lens, counts, choice, bs)
        assert not bad and (state[0].tolist(), state[1].tolist(), state[2].tolist()) == (tables, lens, counts)
        for s, dst, n in copies:
            image[:, :, dst, :n] = image[:, :, s, :n]
        assert np.array_equal(raw(cache).view(np.uint16), image), i
    # free every beam but one, compact, and read the survivor again
    parents.copy_(dev([3, -1, -1, -1, -1, -1]))
    t, l, c = kvp.kv_pages_fork(cache, *state, parents)
    t2, c2, places = kvp.kv_pages_compact(cache, t, l, c)
    check_status(False)
    n = int(l[0])
    used = ref.ceil(n, bs)
    assert sorted(t2[0, :used].tolist()) == list(range(used)) and int((c2 > 0).sum()) == used
    want = oracle.decode(q[0, 3:4].cpu(), image[0, 0], image[1, 0], torch.tensor([tables[3]], dtype=I32),
                         torch.tensor([n], dtype=I32), hq, hkv, d ** -0.5)
    got = kvp.attn_decode_paged(q[0, 3:4].contiguous(), cache[0, 0], cache[1, 0], t2[:1].contiguous(),
                                l[:1].contiguous(), n)
    torch.cuda.synchronize()
    assert_attn_close(got, want, "after compaction")
