"""Host-side refusals of rotary positions and of the 8-bit cache (no GPU): every
case returns before the library's first CUDA call, so the pointers are fake
addresses that nothing dereferences.  The frequencies, which need no GPU.  And
the binding's own refusals."""
import ctypes
import math

import pytest
import torch

import paged_kv_cache_125_gb300 as kvp
import quant_reference as ref

OK, INVALID, UNSUPPORTED = 0, -1, -2
A, MIS = 0x10000, 0x10008


@pytest.fixture(scope="module")
def lib():
    return kvp.library()


def _err(lib):
    return lib.kvp_last_error().decode()


# ---------------------------------------------------------------- frequencies

@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "yarn", "wavelength"])
@pytest.mark.parametrize("r,base,factor,trained", [(128, 1e6, 4.0, 32768), (64, 1e4, 1.0, 2048), (2, 5e5, 8.0, 100),
                                                   (36, 1e4, 2.5, 7), (1024, 1e4, 32.0, 1)])
def test_frequencies(scaling, r, base, factor, trained):
    low, high = {"yarn": (1.0, 32.0), "wavelength": (1.0, 4.0)}.get(scaling, (0.0, 0.0))
    inv, magnitude = ref.inverse_frequencies(r, base, scaling, factor, trained, low, high)
    got, mag = kvp.attn_rope_freqs(r, base, scaling, factor, trained, device="cpu")
    assert got.shape == (r // 2,) and got.dtype == torch.int64 and int(got.min()) >= 0
    back = got.double() * 2.0 ** -64 * 2 * math.pi
    # 2^-53 of each operation, a handful of them; the fraction's own step is 2^-64 turns
    assert bool(((back - inv).abs() <= inv * 2.0 ** -47 + 2.0 ** -61).all())
    assert abs(mag - magnitude) <= magnitude * 2.0 ** -23


def _freqs(lib, **kw):
    a = dict(r=64, base=1e4, kind=0, factor=2.0, trained=100.0, low=1.0, high=4.0, null=False)
    a.update(kw)
    out, mag = (ctypes.c_uint64 * 512)(), ctypes.c_float()
    return lib.attn_rope_freqs(a["r"], a["base"], a["kind"], a["factor"], a["trained"], a["low"], a["high"],
                               None if a["null"] else out, ctypes.byref(mag))


def test_frequency_refusals(lib):
    assert _freqs(lib) == OK
    for kw in (dict(r=0), dict(r=63), dict(r=1026), dict(r=-2), dict(base=1.0), dict(base=math.inf),
               dict(base=math.nan), dict(kind=1, factor=0.5), dict(kind=2, factor=math.nan),
               dict(kind=3, trained=0.5), dict(kind=4, low=4.0), dict(kind=3, low=0.0), dict(null=True)):
        assert _freqs(lib, **kw) == INVALID and "attn_rope_freqs" in _err(lib), kw
    for kind in (-1, 5):
        assert _freqs(lib, kind=kind) == UNSUPPORTED
    with pytest.raises(ValueError, match="scaling"):
        kvp.attn_rope_freqs(64, scaling="dynamic")
    with pytest.raises(kvp.KvpError, match="rotary_dim"):
        kvp.attn_rope_freqs(65, device="cpu")


@pytest.mark.parametrize("r", [1026, 1 << 20, (1 << 32) + 64, -(1 << 32) + 64, 1 << 70, -5])
def test_frequencies_of_a_size_that_no_head_has(r):
    """Refused at once: no room is made for them, and no size wraps round to one that is taken."""
    with pytest.raises(kvp.KvpError, match="rotary_dim"):
        kvp.attn_rope_freqs(r, device="cpu")


# ---------------------------------------------------------------- C ABI

def _rope(lib, **kw):
    a = dict(q=A, qs=16 * 128, k=A, ks=8 * 128, pos=A, n=0, freqs=A, r=128, hq=16, hkv=8, d=128, qo=A, qos=16 * 128,
             ko=A, kos=8 * 128)
    a.update(kw)
    return lib.attn_rope(a["q"], a["qs"], a["k"], a["ks"], a["pos"], a["n"], a["freqs"], a["r"], 0, 1.0, a["hq"],
                         a["hkv"], a["d"], a["qo"], a["qos"], a["ko"], a["kos"], None)


def test_rope_refusals(lib):
    assert _rope(lib) == OK
    for kw in (dict(n=-1), dict(hq=-1), dict(hq=0, hkv=0), dict(d=0)):
        assert _rope(lib, **kw) == INVALID and "attn_rope: bad sizes" in _err(lib), kw
    for kw in (dict(d=2048, qs=1 << 20, ks=1 << 20, qos=1 << 20, kos=1 << 20), dict(n=1 << 31)):
        assert _rope(lib, **kw) == UNSUPPORTED, kw
    for r in (0, 3, 130, -2):
        assert _rope(lib, r=r) == INVALID and "rotary_dim" in _err(lib)
    for name in ("qs", "ks", "qos", "kos"):
        assert _rope(lib, **{name: 1000}) == INVALID and "stride" in _err(lib)
    for name in ("q", "k", "pos", "freqs", "qo", "ko"):
        assert _rope(lib, n=4, **{name: None}) == INVALID and "null" in _err(lib)
    assert _rope(lib, n=4, qos=16 * 128 + 8) == INVALID and "in place" in _err(lib)


def _cache(**kw):
    a = dict(k=A, v=A, ks=8 * 128, vs=8 * 128, slots=A, n=4, kc=A, vc=A, ksc=A, vsc=A, form=0, nb=64, bs=256, t=16,
             hkv=8, d=128)
    a.update(kw)
    return a


def _store(lib, **kw):
    a = _cache(**kw)
    return lib.kv_quant_store(a["k"], a["v"], a["ks"], a["vs"], a["slots"], a["n"], a["kc"], a["vc"], a["ksc"],
                              a["vsc"], a["form"], a["nb"], a["bs"], a["t"], a["hkv"], a["d"], None)


def _store_rope(lib, **kw):
    a = dict(_cache(), q=A, qs=16 * 128, pos=A, freqs=A, r=128, hq=16, qo=A + 64, qos=16 * 128)
    a.update(kw)
    return lib.kv_quant_store_rope(a["q"], a["qs"], a["k"], a["v"], a["ks"], a["vs"], a["pos"], a["slots"], a["n"],
                                   a["freqs"], a["r"], 0, 1.0, a["hq"], a["qo"], a["qos"], a["kc"], a["vc"],
                                   a["ksc"], a["vsc"], a["form"], a["nb"], a["bs"], a["t"], a["hkv"], a["d"], None)


def _load(lib, **kw):
    a = dict(_cache(), bt=A, mb=16, ctx=A, st=A, b=4, most=4096, rows=1000)
    a.update(kw)
    return lib.kv_quant_load(a["kc"], a["vc"], a["ksc"], a["vsc"], a["form"], a["nb"], a["bs"], a["t"], a["bt"],
                             a["mb"], a["ctx"], a["st"], a["b"], a["most"], a["hkv"], a["d"], a["rows"], a["k"],
                             a["ks"], a["v"], a["vs"], None)


def _decode(lib, **kw):
    a = dict(_cache(), q=A, qs=16 * 128, bt=A, mb=16, ctx=A, b=0, most=4096, hq=16, out=A, os=16 * 128)
    a.update(kw)
    return lib.attn_decode_quant(a["q"], a["qs"], a["kc"], a["vc"], a["ksc"], a["vsc"], a["form"], a["nb"], a["bs"],
                                 a["t"], a["bt"], a["mb"], a["ctx"], a["b"], a["most"], a["hq"], a["hkv"], a["d"],
                                 0.088, A, 1 << 30, a["out"], a["os"], None)


@pytest.mark.parametrize("call,name", [(_store, "kv_quant_store"), (_store_rope, "kv_quant_store_rope"),
                                       (_load, "kv_quant_load"), (_decode, "attn_decode_quant")])
def test_cache_refusals(lib, call, name):
    assert call(lib, n=0, b=0) == OK
    for kw in (dict(nb=0), dict(bs=0), dict(t=0), dict(hkv=0), dict(d=0)):
        assert call(lib, **kw) == INVALID and f"{name}: non-positive" in _err(lib), kw
    for kw in (dict(form=2), dict(form=-1), dict(d=96), dict(d=256), dict(t=3), dict(t=512, bs=512), dict(bs=24),
               dict(hkv=1 << 12), dict(nb=1 << 23)):
        assert call(lib, **kw) == UNSUPPORTED and name in _err(lib), kw
    if call is _decode:
        return
    for n in ("kc", "vc", "ksc", "vsc"):
        assert call(lib, **{n: None}) == INVALID and "null" in _err(lib), n
        assert call(lib, **{n: MIS}) == INVALID and "16-byte" in _err(lib), n
    for n in ("k", "v"):
        assert call(lib, **{n: None}) == INVALID and "null" in _err(lib), n
        assert call(lib, **{n: MIS}) == INVALID and "16-byte" in _err(lib), n
    for n in ("ks", "vs"):
        assert call(lib, **{n: 1020}) == INVALID and "stride" in _err(lib)
        assert call(lib, **{n: 1028}) == INVALID and "multiples of 8" in _err(lib)


def test_store_refusals(lib):
    for call in (_store, _store_rope):
        assert call(lib, n=-1) == INVALID
        assert call(lib, n=1 << 31) == UNSUPPORTED
        assert call(lib, slots=None) == INVALID and "null" in _err(lib)
    for n in ("q", "qo", "pos", "freqs"):
        assert _store_rope(lib, **{n: None}) == INVALID and "null" in _err(lib)
    assert _store_rope(lib, r=7) == INVALID and "rotary_dim" in _err(lib)
    assert _store_rope(lib, qs=100) == INVALID and "stride" in _err(lib)
    assert _store_rope(lib, qo=A, qos=16 * 128 + 8) == INVALID and "in place" in _err(lib)


def test_load_refusals(lib):
    for kw in (dict(b=-1), dict(mb=-1), dict(most=-1), dict(rows=-1)):
        assert _load(lib, **kw) == INVALID and "bad sizes" in _err(lib)
    assert _load(lib, b=65536) == UNSUPPORTED and "65535" in _err(lib)
    assert _load(lib, mb=1 << 23) == UNSUPPORTED and "capacity" in _err(lib)
    for n in ("bt", "ctx", "st"):
        assert _load(lib, **{n: None}) == INVALID and "null" in _err(lib)
    assert _load(lib, mb=0) == OK


def test_decode_refusals(lib):
    assert _decode(lib, b=-1) == INVALID and "attn_decode_quant: bad sizes" in _err(lib)
    for kw in (dict(hq=24), dict(hkv=16, hq=16), dict(hkv=3, hq=3), dict(hq=128)):
        assert _decode(lib, **kw) == UNSUPPORTED and "unsupported heads" in _err(lib), kw
    for n in ("q", "kc", "vc", "bt", "ctx", "out"):
        assert _decode(lib, b=1, **{n: None}) == INVALID and "null" in _err(lib), n
    for n in ("q", "kc", "out"):
        assert _decode(lib, b=1, **{n: MIS}) == INVALID and "16-byte" in _err(lib), n
    for n in ("ksc", "vsc"):
        assert _decode(lib, b=1, **{n: None}) == INVALID and "null" in _err(lib), n
    for kw in (dict(qs=2040), dict(os=2040)):
        assert _decode(lib, b=1, **kw) == INVALID and "stride" in _err(lib)
    assert _decode(lib, mb=1 << 23) == UNSUPPORTED and "capacity" in _err(lib)
    assert _decode(lib, b=1 << 11, bs=16, mb=1 << 20) == UNSUPPORTED and "2^31" in _err(lib)
    for args in ((-1, 16, 8, 128, 10), (1, 24, 8, 128, 10), (1, 16, 8, 96, 10), (1, 16, 8, 128, -1)):
        with pytest.raises(kvp.KvpError, match="bad shape"):
            kvp.attn_decode_quant_workspace_size(*args)


# ---------------------------------------------------------------- the binding

def _tensors(dtype=torch.int8):
    c = lambda: torch.zeros((4, 16, 2, 64)).to(dtype)  # noqa: E731
    s = lambda: torch.zeros((4, 4, 2))  # noqa: E731
    return c(), c(), s(), s()


def test_binding_refuses_host_tensors_and_wrong_types():
    x = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    slots, pos, freqs = torch.zeros(3, dtype=torch.int32), torch.zeros(3, dtype=torch.int64), torch.zeros(32, dtype=torch.int64)
    table, ctx = torch.zeros((3, 1), dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    for dtype in (torch.int8, torch.float8_e4m3fn):
        arrays = _tensors(dtype)
        for call in (lambda: kvp.kv_quant_store(x, x, slots, *arrays),
                     lambda: kvp.kv_quant_store_rope(x, x, x, pos, slots, freqs, *arrays),
                     lambda: kvp.kv_quant_load(*arrays, table, ctx, ctx, 16, num_rows=3),
                     lambda: kvp.attn_decode_quant(x, *arrays, table, ctx, 16)):
            with pytest.raises(ValueError, match="CUDA"):
                call()
    with pytest.raises(ValueError, match="CUDA"):
        kvp.attn_rope(x, x, pos, freqs)
    with pytest.raises(TypeError, match="bfloat16"):
        kvp.attn_rope(x.float(), x, pos, freqs)
    for dtype in (torch.float8_e5m2, torch.uint8, torch.bfloat16):
        with pytest.raises(TypeError, match="float8_e4m3fn or int8"):
            kvp.kv_quant_store(x, x, slots, *_tensors(dtype))
    with pytest.raises(TypeError, match="Tensor"):
        kvp.attn_decode_quant(x, None, *_tensors()[1:], table, ctx, 16)
