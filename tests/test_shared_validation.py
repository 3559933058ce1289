"""Host-side refusals of the shared-prefix decode and of the page operators
(no GPU): every case returns before the library's first CUDA call, so the
pointers are fake addresses that nothing dereferences.  And the binding's own
refusals, of host tensors and of wrong shapes."""
import pytest
import torch

import paged_kv_cache_125_gb300 as kvp

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, -1, -2, -3
A, MIS = 0x10000, 0x10002
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    return kvp.library()


def _err(lib):
    return lib.kvp_last_error().decode()


def _plan(lib, **kw):
    a = dict(bt=A, mb=16, ctx=A, b=4, nb=64, bs=256, hq=16, hkv=8, ms=0, plan=A, n=1 << 20)
    a.update(kw)
    return lib.attn_shared_plan(a["bt"], a["mb"], a["ctx"], a["b"], a["nb"], a["bs"], a["hq"], a["hkv"], a["ms"],
                                a["plan"], a["n"], None)


def test_plan_validation(lib):
    assert _plan(lib, b=0) == OK
    for kw in (dict(b=-1), dict(b=1 << 20), dict(nb=0), dict(mb=-1), dict(ms=-1)):
        assert _plan(lib, **kw) == INVALID and "attn_shared_plan: bad sizes" in _err(lib), kw
    for kw in (dict(hq=24), dict(hkv=3, hq=12), dict(bs=48), dict(bs=8), dict(bs=8192), dict(hkv=0)):
        assert _plan(lib, **kw) == UNSUPPORTED and "unsupported" in _err(lib), kw
    assert _plan(lib, mb=1 << 20, bs=4096) == UNSUPPORTED and "capacity" in _err(lib)
    for name in ("bt", "ctx", "plan"):
        assert _plan(lib, **{name: None}) == INVALID and "null" in _err(lib)
    assert _plan(lib, plan=MIS) == INVALID and "16-byte" in _err(lib)


def test_sizes(lib):
    assert kvp.kv_pages_workspace_size(1000, 10) > kvp.kv_pages_workspace_size(100, 10)
    for args in ((-1, 16, 8), (1 << 20, 16, 8), (4, 24, 8)):
        with pytest.raises(kvp.KvpError, match="bad shape"):
            kvp.attn_shared_plan_size(*args)
    for args in ((0, 4), (1 << 31, 4), (4, -1), (4, 1 << 20)):
        with pytest.raises(kvp.KvpError, match="bad shape"):
            kvp.kv_pages_workspace_size(*args)
    with pytest.raises(kvp.KvpError, match="bad shape"):
        kvp.attn_decode_shared_workspace_size(4, 16, 8, 96)


def _decode(lib, append, **kw):
    a = dict(q=A, qs=16 * 128, k=A, v=A, ks=8 * 128, vs=8 * 128, slots=A, kc=A, vc=A, nb=64, bs=256, bt=A, mb=16,
             plan=A, pn=1 << 20, b=4, hq=16, hkv=8, d=128, ws=A, wn=BIG, out=A, os=16 * 128)
    a.update(kw)
    tail = (a["kc"], a["vc"], a["nb"], a["bs"], a["bt"], a["mb"], a["plan"], a["pn"], a["b"], a["hq"], a["hkv"],
            a["d"], 0.088, a["ws"], a["wn"], a["out"], a["os"], None)
    if append:
        return lib.attn_decode_shared_append(a["q"], a["qs"], a["k"], a["v"], a["ks"], a["vs"], a["slots"], *tail)
    return lib.attn_decode_shared(a["q"], a["qs"], *tail)


@pytest.mark.parametrize("append", [False, True])
def test_decode_validation(lib, append):
    name = "attn_decode_shared_append" if append else "attn_decode_shared"
    assert _decode(lib, append, b=0) == OK
    for kw in (dict(b=-1), dict(b=1 << 20), dict(nb=0), dict(mb=-1)):
        assert _decode(lib, append, **kw) == INVALID and f"{name}: bad sizes" in _err(lib), kw
    for kw in (dict(hq=24), dict(hkv=3, hq=12), dict(d=96), dict(bs=48), dict(hkv=16, hq=16)):
        assert _decode(lib, append, **kw) == UNSUPPORTED and "unsupported" in _err(lib), kw
    for kw in (dict(qs=16 * 128 - 8), dict(os=16 * 128 - 8)) + ((dict(ks=1016), dict(vs=1016)) if append else ()):
        assert _decode(lib, append, **kw) == INVALID and "stride too small" in _err(lib), kw
    assert _decode(lib, append, mb=1 << 20, bs=4096) == UNSUPPORTED and "capacity" in _err(lib)
    assert _decode(lib, append, nb=1 << 23, bs=256) == UNSUPPORTED and "2^31" in _err(lib)
    names = ["q", "kc", "vc", "out", "plan"] + (["k", "v"] if append else [])
    for n in names + ["bt"] + (["slots"] if append else []):
        assert _decode(lib, append, **{n: None}) == INVALID and "null" in _err(lib), n
    for n in names:
        assert _decode(lib, append, **{n: MIS}) == INVALID and "16-byte" in _err(lib), n
    for n in ["qs", "os"] + (["ks", "vs"] if append else []):
        assert _decode(lib, append, **{n: 16 * 128 + 4}) == INVALID and "multiples" in _err(lib), n


def _pages(lib, op, **kw):
    a = dict(cache=0x1000000, planes=4, stride=64 * 16 * 128, nb=64, bs=16, row=128, bt=0x100000, mb=8, ctx=0x200000,
             n=5, ref=0x300000, par=0x400000, m=5, new=0x400000, slots=9, sm=0x800000, ot=0x500000, ol=0x600000,
             oc=0x700000, places=0x800000, ws=0x900000, wn=kvp.kv_pages_workspace_size(64, 5))
    a.update(kw)
    pool = (a["cache"], a["planes"], a["stride"], a["nb"], a["bs"], a["row"], a["bt"], a["mb"], a["ctx"], a["n"],
            a["ref"])
    if op == "fork":
        return lib.kv_pages_fork(*pool, a["par"], a["m"], a["ot"], a["ol"], a["oc"], a["ws"], a["wn"], None)
    if op == "compact":
        return lib.kv_pages_compact(*pool, a["ot"], a["oc"], a["places"], a["ws"], a["wn"], None)
    return lib.kv_pages_extend(a["bt"], a["mb"], a["ctx"], a["n"], a["ref"], a["nb"], a["bs"], a["new"], a["slots"],
                               a["ot"], a["ol"], a["oc"], a["sm"], a["ws"], a["wn"], None)


@pytest.mark.parametrize("op", ["fork", "extend", "compact"])
def test_pages_validation(lib, op):
    bad = [dict(n=-1), dict(n=1 << 20), dict(mb=-1), dict(nb=0), dict(bs=0)]
    bad += [dict(m=-1), dict(m=1 << 20)] if op == "fork" else []
    bad += [dict(slots=-1)] if op == "extend" else []
    for kw in bad:
        assert _pages(lib, op, **kw) == INVALID and f"kv_pages_{op}: bad sizes" in _err(lib), kw
    assert _pages(lib, op, nb=1 << 28, bs=16) == UNSUPPORTED and "2^31" in _err(lib)
    assert _pages(lib, op, mb=1 << 27) == UNSUPPORTED and "capacity" in _err(lib)
    if op == "extend":
        assert _pages(lib, op, slots=1 << 31) == UNSUPPORTED and "2^31" in _err(lib)
    else:
        for kw in (dict(planes=0), dict(row=0)):
            assert _pages(lib, op, **kw) == INVALID and "cache shape" in _err(lib)
        assert _pages(lib, op, stride=64 * 16 * 128 - 1) == INVALID and "plane_stride" in _err(lib)
        assert _pages(lib, op, row=(1 << 20) + 1, stride=BIG) == UNSUPPORTED and "row too long" in _err(lib)
    needed = {"fork": ["cache", "bt", "ctx", "ref", "par", "ot", "ol", "oc"],
              "extend": ["bt", "ctx", "ref", "new", "ot", "ol", "oc", "sm"],
              "compact": ["cache", "bt", "ctx", "ref", "ot", "oc", "places"]}[op]
    for n in needed:
        assert _pages(lib, op, **{n: None}) == INVALID and "null" in _err(lib), n
    assert _pages(lib, op, ws=None) == WORKSPACE
    assert _pages(lib, op, ws=0x900008) == WORKSPACE
    assert _pages(lib, op, wn=kvp.kv_pages_workspace_size(64, 5) - 1) == WORKSPACE and "workspace needs" in _err(lib)


@pytest.mark.parametrize("op", ["fork", "extend", "compact"])
def test_pages_refuse_overlapping_arrays(lib, op):
    outs = {"fork": ["ot", "ol", "oc"], "extend": ["ot", "ol", "oc", "sm"], "compact": ["ot", "oc", "places"]}[op]
    ins = {"fork": ["bt", "ctx", "ref", "par"], "extend": ["bt", "ctx", "ref", "new"],
           "compact": ["bt", "ctx", "ref"]}[op]
    at = dict(bt=0x100000, ctx=0x200000, ref=0x300000, par=0x400000, new=0x400000, ot=0x500000, ol=0x600000,
              oc=0x700000, sm=0x800000, places=0x800000)
    same = {("ot", "bt"), ("ol", "ctx"), ("oc", "ref")} if op == "extend" else set()
    for o in outs:
        for i in ins:
            if (o, i) not in same:
                assert _pages(lib, op, **{o: at[i]}) == INVALID and "overlaps an input" in _err(lib), (o, i)
            assert _pages(lib, op, **{o: at[i] + 4}) == INVALID and "overlaps an input" in _err(lib), (o, i)
        for p in outs:
            if p != o:
                assert _pages(lib, op, **{o: at[p] + 4}) == INVALID and "outputs overlap" in _err(lib), (o, p)
    assert _pages(lib, op, ws=at["bt"]) == INVALID and "overlaps" in _err(lib)


def test_binding_refuses_host_tensors_and_wrong_types():
    bf16, i32 = torch.bfloat16, torch.int32
    kc = torch.zeros((4, 16, 2, 64), dtype=bf16)
    q, bt, n = torch.zeros((2, 4, 64), dtype=bf16), torch.zeros((2, 3), dtype=i32), torch.ones(2, dtype=i32)
    plan, kv = torch.zeros(4096, dtype=torch.uint8), torch.zeros((2, 1, 4, 16, 2, 64), dtype=bf16)
    ref, row = torch.zeros(4, dtype=i32), torch.zeros((2, 2, 64), dtype=bf16)
    with pytest.raises(ValueError, match="CUDA"):
        kvp.attn_shared_plan(bt, n, 16, 4, 2, 4)
    with pytest.raises(TypeError, match="int32"):
        kvp.attn_shared_plan(bt.long(), n, 16, 4, 2, 4)
    with pytest.raises(ValueError, match="CUDA"):
        kvp.attn_decode_shared(q, kc, kc.clone(), bt, plan)
    with pytest.raises(ValueError, match="CUDA"):
        kvp.attn_decode_shared_append(q, row, row, n, kc, kc.clone(), bt, plan)
    with pytest.raises(TypeError):
        kvp.attn_decode_shared(q, kc.float(), kc, bt, plan)
    with pytest.raises(ValueError, match="CUDA"):
        kvp.kv_pages_fork(kv, bt, n, ref, n)
    with pytest.raises(ValueError, match="CUDA"):
        kvp.kv_pages_extend(bt, n, ref, n, 16, 2)
    with pytest.raises(ValueError, match="CUDA"):
        kvp.kv_pages_compact(kv, bt, n, ref)
    with pytest.raises(TypeError):
        kvp.kv_pages_compact(None, bt, n, ref)
