"""The library needs neither torch nor its headers to be built, and the calls
that go through the extension module run without it, with the same results."""
import os
import sys

import pytest
import torch

import paged_kv_cache_125_gb300 as kvp
from paged_kv_cache_125_gb300 import _build


@pytest.fixture
def building(monkeypatch, tmp_path):
    """_build.build() into a folder of its own; -> the names of what it built."""
    built = []
    monkeypatch.setattr(_build, "OUT", str(tmp_path))
    monkeypatch.setattr(_build, "_build_library", lambda *args: built.append("library"))
    monkeypatch.setattr(_build, "_link_calls", lambda obj: built.append("calls"))
    return built


def test_library_is_built_without_torch(building, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)  # as if it were not installed
    _build.build()
    _build.build(force=True)
    assert building == ["library", "library"]


def test_library_is_built_where_the_extension_cannot_be(building, monkeypatch):
    def fails(*args):
        raise RuntimeError("no compiler")

    old = _build.calls_path()
    with open(old, "w"):
        pass
    os.utime(old, (0, 0))
    monkeypatch.setattr(_build, "_compile_calls", fails)
    with pytest.warns(UserWarning, match="ctypes: no compiler"):
        _build.build()
    assert building == ["library"]
    assert not os.path.exists(old)  # built from an older header


def test_extension_is_built_where_it_can_be(building, monkeypatch):
    monkeypatch.setattr(_build, "_compile_calls", lambda: "calls_py.o")
    _build.build()
    assert building == ["library", "calls"]


@pytest.mark.parametrize("there", ["none", "broken"])
def test_calls_without_the_extension(monkeypatch, tmp_path, recwarn, there):
    path = tmp_path / "_kvpaged_calls.so"
    if there == "broken":
        path.write_bytes(b"nothing to load")
    monkeypatch.setattr(_build, "calls_path", lambda: str(path))
    monkeypatch.setattr(kvp, "_CALLS", None)
    i32 = dict(dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        kvp.attn_shared_plan(torch.zeros((2, 3), **i32), torch.ones(2, **i32), 16, 4, 2, 4)
    with pytest.raises(ValueError, match="CUDA"):
        kvp.kv_pages_extend(torch.zeros((2, 3), **i32), torch.ones(2, **i32), torch.ones(9, **i32),
                            torch.ones(2, **i32), 16, 2)
    assert [w for w in recwarn if "does not load" in str(w.message)] or there == "none"


def test_extension_is_what_runs_here():
    assert kvp._calls().__name__ == "_kvpaged_calls"


@pytest.mark.gpu
def test_same_results_without_the_extension(monkeypatch):
    """extend, plan, decode with and without the store, fork and compact, with
    outputs and buffers of the caller's and without."""
    g = torch.Generator(device="cuda").manual_seed(3)
    rows, width, bs, nb, hq, hkv, d = 9, 12, 16, 140, 16, 8, 128
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    draw = lambda *shape: torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    ids = torch.randperm(nb, generator=g, device="cuda").tolist()
    lens = [130 + 3 * i for i in range(rows)]
    tables, at = [], 8  # rows behind one prefix of 8 pages
    for n in lens:
        own = -(-n // bs) - 8
        tables.append(ids[:8] + ids[at:at + own] + [-1] * (width - 8 - own))
        at += own
    counts = [0] * nb
    for row in tables:
        for p in row:
            if p >= 0:
                counts[p] += 1
    cache0, q, k, v = draw(2, nb, bs, hkv, d), draw(rows, hq, d), draw(rows, hkv, d), draw(rows, hkv, d)
    parents = ints([0, 0, 3, 3, 3, -1, 5, 1, 8, 0])

    def step(given):
        cache = cache0.clone()
        a = (ints(tables), ints(lens), ints(counts))
        new = ints([1] * rows)
        size = lambda n: torch.empty(n, dtype=torch.uint8, device="cuda")  # noqa: E731
        ws = dict(workspace=size(kvp.kv_pages_workspace_size(nb, 10))) if given else {}
        out = dict(out=[torch.empty_like(x) for x in (*a, new)]) if given else {}
        t, l, c, s = kvp.kv_pages_extend(*a, new, bs, rows, **ws, **out)
        plan = kvp.attn_shared_plan(t, l, bs, hq, hkv, nb, **(
            dict(plan=size(kvp.attn_shared_plan_size(rows, hq, hkv))) if given else {}))
        more = dict(workspace=size(kvp.attn_decode_shared_workspace_size(rows, hq, hkv, d)),
                    out=torch.empty_like(q)) if given else {}
        first = kvp.attn_decode_shared_append(q, k, v, s, cache[0], cache[1], t, plan, **more).clone()
        again = kvp.attn_decode_shared(q, cache[0], cache[1], t, plan, **more)
        f = kvp.kv_pages_fork(cache, t, l, c, parents, **ws)
        z = kvp.kv_pages_compact(cache, *f, **ws)
        return [t, l, c, s, first, again, *f, *z, cache]

    kvp.device_status()
    want = step(False)
    assert kvp._CALLS.__name__ == "_kvpaged_calls"
    monkeypatch.setattr(kvp, "_CALLS", kvp._NoCalls())
    for given in (False, True):
        got = step(given)
        torch.cuda.synchronize()
        assert kvp.device_status() == 0
        assert all(torch.equal(x, y) for x, y in zip(got, want))
