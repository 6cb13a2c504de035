"""Host-side checks of the 4-bit cache calls and of attn_rope_axes: every
refusal happens before any CUDA call, so they run without a GPU."""
import ctypes

import numpy as np
import pytest

import fp4_reference as ref

FAKE = 0x10000  # 16-byte aligned, never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    from exact_attention_40_gb300 import build
    build.build()
    from exact_attention_40_gb300 import exattn
    return exattn.lib


def i64(*x):
    return (ctypes.c_int64 * len(x))(*x)


def ints(*x):
    return (ctypes.c_int * len(x))(*x)


def rope(lib, q=FAKE, k=FAKE + 16, qo=FAKE + 32, ko=FAKE + 48, pos=FAKE + 64, strides="default", sections=(16, 24, 24),
         axes=None, B=2, Hq=8, Hkv=2, N=5, d=128, base=500000.0, per_axis=0, inverse=0, **change):
    if strides == "default":
        s = [Hq * N * d, N * d, d, Hkv * N * d, N * d, d, Hq * N * d, N * d, d, Hkv * N * d, N * d, d, B * N, N, 1]
        for at, v in change.items():
            s[int(at[1:])] = v
        strides = i64(*s)
    return lib.attn_rope_axes(q, k, qo, ko, pos, strides, ints(*sections) if sections else None,
                              len(sections) if axes is None else axes, B, Hq, Hkv, N, d, base, per_axis, inverse, None)


def test_rope_axes_rejections(lib):
    assert rope(lib, d=24) == 2
    assert rope(lib, d=272, sections=(136,)) == 2
    assert rope(lib, sections=(16, 24)) == 1          # does not cover the pairs
    assert rope(lib, sections=(70, -6)) == 1
    assert rope(lib, sections=(2 ** 31 - 1, 2 ** 31 - 1, 66)) == 1  # a sum that wraps
    assert rope(lib, sections=(16, 16, 16, 8, 8)) == 1
    assert rope(lib, axes=0) == 1
    assert rope(lib, sections=None, axes=3) == 1
    assert rope(lib, base=1.0) == 1
    assert rope(lib, base=float("inf")) == 1
    assert rope(lib, B=-1) == 1
    assert rope(lib, strides=None) == 1
    assert rope(lib, q=None) == 1
    assert rope(lib, pos=None) == 1
    assert rope(lib, qo=FAKE, ko=FAKE) == 1           # both outputs in one place
    assert rope(lib, q=FAKE + 8) == 3
    assert rope(lib, pos=FAKE + 2) == 3
    assert rope(lib, s2=132) == 3                     # rows off the 16-byte boundaries
    assert rope(lib, s8=64) == 1                      # output rows that overlap
    assert rope(lib, s7=0) == 1                       # every head into one row
    assert rope(lib, s6=0) == 1
    assert rope(lib, s2=-128) == 1
    assert rope(lib, s12=-1) == 1
    assert rope(lib, q=FAKE, qo=FAKE, s2=256) == 1    # in place with other strides
    assert rope(lib, B=70000, N=70000) == 2           # 2^31 tokens or more
    # nothing to do
    assert rope(lib, B=0, q=None, k=None, qo=None, ko=None, pos=None) == 0
    assert rope(lib, N=0, q=None, k=None, qo=None, ko=None, pos=None) == 0
    assert rope(lib, Hq=0, Hkv=0, q=None, k=None, qo=None, ko=None, pos=None) == 0


def test_outputs_over_another_tensors_place_are_refused(lib):
    assert rope(lib, qo=FAKE + 16) == 1               # queries over the keys
    assert rope(lib, ko=FAKE) == 1                    # keys over the queries
    assert append(lib, qo=FAKE + 16) == 1             # queries over the keys
    assert append(lib, qo=FAKE + 32) == 1             # ... the values


def append(lib, q=FAKE, k=FAKE + 16, v=FAKE + 32, qo=FAKE + 48, sid=FAKE + 64, slots=FAKE + 80, pos=FAKE + 96,
           bt=FAKE + 112, cache=FAKE + 128, strides="default", sections=(64,), T=4, Hq=8, Hkv=2, d=128, S=2, nb=10,
           mb=4, base=10000.0, per_axis=0, ks=1.0, vs=1.0, **change):
    if strides == "default":
        s = [Hq * d, d, Hkv * d, d, Hkv * d, d, Hq * d, d, T]
        for at, x in change.items():
            s[int(at[1:])] = x
        strides = i64(*s)
    return lib.attn_rope_cache_write_fp4(q, k, v, qo, sid, slots, pos, bt, cache, strides, ints(*sections),
                                         len(sections), T, Hq, Hkv, d, S, nb, mb, base, per_axis, ks, vs, None)


def test_append_rejections(lib):
    assert append(lib, d=96, sections=(48,)) == 2
    assert append(lib, T=-1) == 1
    assert append(lib, Hkv=0) == 1
    assert append(lib, S=0) == 1
    assert append(lib, nb=0) == 1
    assert append(lib, mb=0) == 1
    assert append(lib, mb=(1 << 26) + 1) == 2
    assert append(lib, ks=0.0) == 1
    assert append(lib, vs=float("nan")) == 1
    assert append(lib, ks=-1.0) == 1
    assert append(lib, vs=float("inf")) == 1
    assert append(lib, sections=(32,)) == 1
    assert append(lib, base=0.5) == 1
    assert append(lib, strides=None) == 1
    for name in ("q", "k", "v", "qo", "sid", "slots", "pos", "bt", "cache"):
        assert append(lib, **{name: None}) == 1, name
        assert append(lib, **{name: FAKE + 2}) == 3, name
    assert append(lib, s2=100) == 3
    assert append(lib, s7=0) == 1
    assert append(lib, qo=FAKE, s6=4096) == 1
    assert append(lib, T=0, q=None, k=None, v=None, qo=None, sid=None, slots=None, pos=None, bt=None, cache=None) == 0


def read(lib, cache=FAKE, sid=FAKE + 16, slots=FAKE + 32, bt=FAKE + 48, ko=FAKE + 64, vo=FAKE + 80, strides="default",
         T=4, Hkv=2, d=64, S=2, nb=10, mb=4, ks=1.0, vs=1.0, **change):
    if strides == "default":
        s = [Hkv * d, d, Hkv * d, d]
        for at, x in change.items():
            s[int(at[1:])] = x
        strides = i64(*s)
    return lib.attn_cache_read_fp4(cache, sid, slots, bt, ko, vo, strides, T, Hkv, d, S, nb, mb, ks, vs, None)


def test_read_rejections(lib):
    assert read(lib, d=32) == 2
    assert read(lib, T=-1) == 1
    assert read(lib, Hkv=0) == 1
    assert read(lib, ks=0.0) == 1
    assert read(lib, vs=float("inf")) == 1
    for name in ("cache", "sid", "slots", "bt", "ko", "vo"):
        assert read(lib, **{name: None}) == 1, name
        assert read(lib, **{name: FAKE + 2}) == 3, name
    assert read(lib, ko=FAKE + 80) == 1
    assert read(lib, strides=None) == 1
    assert read(lib, s0=8) == 1
    assert read(lib, s3=4) == 3
    assert read(lib, T=0, cache=None, sid=None, slots=None, bt=None, ko=None, vo=None) == 0


def dec(lib, ws_bytes=None, **kw):
    a = dict(q=FAKE, c=FAKE, bt=FAKE, cl=FAKE, out=FAKE, lse=None, S=2, Hq=8, Hkv=2, d=128, nb=10, mb=512, scale=0.1,
             ks=1.0, vs=1.0, ws=FAKE)
    a.update(kw)
    if ws_bytes is None:
        ws_bytes = lib.attn_decode_fp4_workspace_bytes(a["S"], a["Hq"], a["Hkv"], a["d"], a["mb"])
    return lib.attn_decode_paged_fp4(a["q"], a["c"], a["bt"], a["cl"], a["out"], a["lse"], a["S"], a["Hq"], a["Hkv"],
                                     a["d"], a["nb"], a["mb"], a["scale"], a["ks"], a["vs"], a["ws"], ws_bytes, None)


def test_decode_rejections(lib):
    assert dec(lib, d=80) == 2
    assert dec(lib, Hq=6, Hkv=4) == 1
    assert dec(lib, mb=0) == 1
    assert dec(lib, nb=0) == 1
    assert dec(lib, S=-1) == 1
    assert dec(lib, scale=0.0) == 1
    assert dec(lib, ks=float("nan")) == 1
    assert dec(lib, vs=0.0) == 1
    for name in ("q", "c", "bt", "cl", "out"):
        assert dec(lib, **{name: None}) == 1, name
        assert dec(lib, **{name: FAKE + 2}) == 3, name
    assert dec(lib, lse=FAKE + 2) == 3
    assert dec(lib, ws=None) == 4
    assert dec(lib, ws_bytes=16) == 4
    assert dec(lib, ws=FAKE + 4) == 3
    assert dec(lib, S=70000) == 2
    assert dec(lib, S=65535, Hq=65535, Hkv=65535) == 2               # more rows than 2^31
    assert dec(lib, S=65535, Hq=8, Hkv=8, mb=1 << 26, ws_bytes=1 << 30) == 2  # more work units than 2^31
    assert dec(lib, S=0, q=None) == 0


def test_decode_scale_products_out_of_range_are_refused(lib):
    assert dec(lib, scale=1e30, ks=1e30) == 1         # infinite: zeros times it would be NaN
    assert dec(lib, scale=1e-30, ks=1e-30) == 1       # zero: every weight the same


def test_workspace_of_refused_sizes_is_zero(lib):
    assert lib.attn_decode_fp4_workspace_bytes(2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1, 64, 2 ** 31 - 1) == 0
    assert lib.attn_decode_fp4_workspace_bytes(65536, 8, 8, 64, 64) == 0
    assert lib.attn_decode_fp4_workspace_bytes(1, 8, 8, 64, (1 << 26) + 1) == 0


def test_sizes(lib):
    assert lib.attn_fp4_cache_bytes(10, 8, 128) == 10 * 8 * 2304
    assert lib.attn_fp4_cache_bytes(1 << 20, 64, 128) == (1 << 26) * 2304  # past 32 bits
    assert lib.attn_fp4_cache_bytes(0, 8, 128) == 0
    assert lib.attn_fp4_cache_bytes(1, 1, 96) == 0
    assert lib.attn_decode_fp4_workspace_bytes(0, 8, 2, 64, 4) == 0
    assert lib.attn_decode_fp4_workspace_bytes(1, 8, 3, 64, 4) == 0
    assert lib.attn_decode_fp4_workspace_bytes(1, 8, 2, 96, 4) == 0
    assert lib.attn_decode_fp4_workspace_bytes(1, 1, 1, 64, 1) == 0     # one CTA a head: written directly
    assert lib.attn_decode_fp4_workspace_bytes(2, 8, 2, 128, 100) == 0  # few and short: merged in a cluster
    big = lib.attn_decode_fp4_workspace_bytes(64, 32, 8, 128, 512)
    assert 0 < big < 16 << 20  # two partial outputs for each of a wave of CTAs, however long the contexts
    assert lib.attn_decode_fp4_workspace_bytes(64, 32, 8, 128, 1 << 16) == big


def test_the_reference_of_the_format():
    # every code of both types back to itself, ties to even, saturation
    assert np.array_equal(ref.e4m3_round(ref.POSITIVE), np.arange(127))
    assert ref.e4m3_round(1e9) == 126 and ref.e4m3_round(2.0 ** -10) == 0 and ref.e4m3_round(3 * 2.0 ** -10) == 2
    assert ref.e4m3_round(17.0) == ref.e4m3_round(16.0) and ref.e4m3_round(19.0) == ref.e4m3_round(20.0)
    assert np.array_equal(ref.e2m1_round(ref.VALUES), np.arange(8))
    assert np.array_equal(ref.e2m1_round(-ref.VALUES), np.arange(8, 16))
    assert np.array_equal(ref.e2m1_round(ref.TIES), [0, 2, 2, 4, 4, 6, 6])
    x = np.linspace(-3, 3, 64, dtype=np.float32)[None]
    codes, s8 = ref.quantise(x, 0.01)
    assert np.abs(ref.values(codes, s8, 0.01) - x).max() < 3 / 6 + 0.2  # a step of the largest codes
    assert np.array_equal(ref.unpack(ref.pack(codes)), codes)


def test_binding_rejections():
    """The binding's own checks, on CPU tensors (no call is made)."""
    torch = pytest.importorskip("torch")
    from exact_attention_40_gb300 import exattn as ex
    bf, i32 = torch.bfloat16, torch.int32
    q = torch.zeros(1, 4, 3, 64, dtype=bf)
    with pytest.raises(ValueError):
        ex.attn_rope_axes(q, q, torch.zeros(1, 3, dtype=i32), (32,))
    cache = torch.zeros(2, 1, 18 * 64, dtype=torch.uint8)
    t = torch.zeros(1, dtype=i32)
    with pytest.raises(ValueError):
        ex.attn_cache_read_fp4(cache, t, t, t.view(1, 1))
    with pytest.raises(TypeError):
        ex.attn_cache_read_fp4(cache.to(torch.int8), t, t, t.view(1, 1))
    with pytest.raises(ValueError):
        ex.attn_decode_paged_fp4(q[0], cache, t.view(1, 1), t)
    with pytest.raises(ValueError):
        ex.attn_fp4_cache(0, 1, 64)
    with pytest.raises(ValueError):
        ex.attn_fp4_cache(1, 1, 80)
