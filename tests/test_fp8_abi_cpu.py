"""Host-side checks of the 8-bit cache calls: every refusal happens before any CUDA
call, so they run without a GPU.  And the plain implementation's format against a byte
by byte reading of it."""
import ctypes

import numpy as np
import pytest

import fp8_reference as ref
from fp4_reference import E4M3

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


def test_cache_bytes(lib):
    assert lib.attn_fp8_cache_bytes(10, 8, 128) == 10 * 8 * 4128
    assert lib.attn_fp8_cache_bytes(1, 1, 64) == 2080
    assert lib.attn_fp8_cache_bytes(2 ** 31 - 1, 65535, 128) == (2 ** 31 - 1) * 65535 * 4128
    for bad in ((0, 1, 64), (1, 0, 64), (1, 1, 96), (-1, 1, 64)):
        assert lib.attn_fp8_cache_bytes(*bad) == 0


def append(lib, q=FAKE, k=FAKE + 16, v=FAKE + 32, qo=FAKE + 48, st=FAKE + 64, cl=FAKE + 80, pos=FAKE + 96,
           bt=FAKE + 112, kv=FAKE + 128, strides="default", sections=(16, 24, 24), axes=None, T=5, Hq=8, Hkv=2, d=128,
           S=2, nb=10, mb=4, base=500000.0, per_axis=0, **change):
    if strides == "default":
        s = [Hq * d, d, Hkv * d, d, Hkv * d, d, Hq * d, d, T]
        for at, x in change.items():
            s[int(at[1:])] = x
        strides = i64(*s)
    return lib.attn_rope_cache_write_fp8(q, k, v, qo, st, cl, pos, bt, kv, strides, ints(*sections) if sections else None,
                                         len(sections) if axes is None else axes, T, Hq, Hkv, d, S, nb, mb, base,
                                         per_axis, None)


def test_append_rejections(lib):
    assert append(lib, d=96, sections=(48,)) == 2
    assert append(lib, sections=(16, 24)) == 1
    assert append(lib, sections=None, axes=3) == 1
    assert append(lib, sections=(16, 16, 16, 8, 8)) == 1
    assert append(lib, base=1.0) == 1
    assert append(lib, base=float("nan")) == 1
    assert append(lib, T=-1) == 1
    assert append(lib, Hq=-1) == 1
    assert append(lib, Hkv=0) == 1
    assert append(lib, S=0) == 1
    assert append(lib, nb=0) == 1
    assert append(lib, mb=0) == 1
    assert append(lib, mb=(1 << 26) + 1) == 2
    assert append(lib, Hq=65536) == 2
    assert append(lib, Hkv=65536) == 2
    assert append(lib, S=65536) == 2
    assert append(lib, strides=None) == 1
    for x in ("q", "k", "v", "qo", "cl", "pos", "bt", "kv"):
        assert append(lib, **{x: None}) == 1, x
    for x in ("q", "k", "v", "qo", "kv"):
        assert append(lib, **{x: FAKE + 8}) == 3, x
    for x in ("st", "cl", "pos", "bt"):
        assert append(lib, **{x: FAKE + 2}) == 3, x
    assert append(lib, st=None) == 1                  # five tokens of two sequences, and no starts
    assert append(lib, k=FAKE + 48) == 1              # queries over the keys
    assert append(lib, s0=8 * 128 + 4) == 3           # rows off the 16-byte boundaries
    assert append(lib, s6=128) == 1                   # output rows that overlap
    assert append(lib, s2=-8) == 1
    assert append(lib, qo=FAKE, s6=8 * 128 + 128) == 1  # in place with other strides
    assert append(lib, s8=-1) == 1
    # no tokens: success without touching the (null) pointers
    assert append(lib, T=0, q=None, k=None, v=None, qo=None, cl=None, pos=None, bt=None, kv=None) == 0


def read(lib, kv=FAKE, sid=FAKE + 16, sl=FAKE + 32, bt=FAKE + 48, ko=FAKE + 64, vo=FAKE + 80, strides="default", T=5,
         Hkv=2, d=128, S=2, nb=10, mb=4):
    if strides == "default":
        strides = i64(Hkv * d, d, Hkv * d, d)
    return lib.attn_cache_read_fp8(kv, sid, sl, bt, ko, vo, strides, T, Hkv, d, S, nb, mb, None)


def test_read_rejections(lib):
    assert read(lib, d=80) == 2
    assert read(lib, Hkv=0) == 1
    assert read(lib, Hkv=65536) == 2
    assert read(lib, T=-1) == 1
    assert read(lib, strides=None) == 1
    assert read(lib, strides=i64(128, 128, 256, 128)) == 1
    assert read(lib, strides=i64(256, 132, 256, 128)) == 3
    for x in ("kv", "sid", "sl", "bt", "ko", "vo"):
        assert read(lib, **{x: None}) == 1, x
        assert read(lib, **{x: FAKE + 2}) == 3, x
    assert read(lib, vo=FAKE + 64) == 1
    assert read(lib, T=0, kv=None, sid=None, sl=None, bt=None, ko=None, vo=None) == 0


def dec(lib, ws_bytes=None, **kw):
    a = dict(q=FAKE, kv=FAKE, bt=FAKE, cl=FAKE, out=FAKE + 16, lse=None, S=64, N=1, Hq=32, Hkv=8, d=128, nb=10, mb=512,
             scale=0.1, ws=FAKE)
    a.update(kw)
    if ws_bytes is None:
        ws_bytes = lib.attn_decode_fp8_workspace_bytes(a["S"], a["N"], a["Hq"], a["Hkv"], a["d"], a["mb"])
    return lib.attn_decode_paged_fp8(a["q"], a["kv"], a["bt"], a["cl"], a["out"], a["lse"], a["S"], a["N"], a["Hq"],
                                     a["Hkv"], a["d"], a["nb"], a["mb"], a["scale"], a["ws"], ws_bytes, None)


def test_decode_rejections(lib):
    assert dec(lib, d=80) == 2
    assert dec(lib, Hq=6, Hkv=4) == 1
    assert dec(lib, Hq=0) == 1
    assert dec(lib, mb=0) == 1
    assert dec(lib, nb=0) == 1
    assert dec(lib, S=-1) == 1
    assert dec(lib, S=65536) == 2
    assert dec(lib, N=0) == 1
    assert dec(lib, N=17) == 2
    assert dec(lib, S=65535, N=16, Hq=65528) == 2     # more rows than 32 bits number
    for bad in (0.0, -1.0, float("nan"), float("inf"), 3e38):
        assert dec(lib, scale=bad) == 1
    for x in ("q", "kv", "bt", "cl", "out"):
        assert dec(lib, **{x: None}) == 1, x
    for x in ("q", "kv", "out"):
        assert dec(lib, **{x: FAKE + 8}) == 3, x
    for x in ("bt", "cl", "lse"):
        assert dec(lib, **{x: FAKE + 2}) == 3, x
    assert dec(lib, ws=None) == 4
    assert dec(lib, ws_bytes=16) == 4
    assert dec(lib, ws=FAKE + 4) == 3
    assert dec(lib, S=0, q=None) == 0


def test_decode_workspace(lib):
    ws = lib.attn_decode_fp8_workspace_bytes
    assert ws(1, 1, 1, 1, 64, 1) == 0        # one CTA a head: written directly
    assert ws(2, 1, 8, 2, 128, 100) == 0     # few and short: merged in a cluster
    big = ws(64, 1, 32, 8, 128, 512)
    assert 0 < big < 8 << 20
    assert ws(64, 1, 32, 8, 128, 1 << 16) == big  # bounded by the wave of CTAs, not by the contexts
    assert ws(64, 4, 32, 8, 128, 512) > 0
    for bad in ((0, 1, 8, 2, 64, 4), (1, 0, 8, 2, 64, 4), (1, 17, 8, 2, 64, 4), (1, 1, 8, 3, 64, 4), (1, 1, 8, 2, 96, 4),
                (65536, 1, 8, 8, 64, 64), (1, 1, 8, 8, 64, (1 << 26) + 1)):
        assert ws(*bad) == 0, bad


@pytest.mark.parametrize("d", [64, 128])
def test_the_reference_format(d):
    """Every byte of a block's codes stands for one token and column."""
    at = ref.place(d)
    assert sorted(at.ravel()) == list(range(16 * d))
    assert at[5, 17] == 5 * d + 16 * (1 ^ (5 if d == 128 else 2)) + 1
    cache = np.zeros((1, 2, 32 * d + 32), np.uint8)
    cache[0, 1, 16 * d + at[9, 3]] = 0x38 | 0x80  # -1 in the values of head 1
    cache[0, 1, 32 * d + 4:32 * d + 8] = np.frombuffer(np.float32(0.25).tobytes(), np.uint8)
    k, v = ref.values(cache, d)
    assert (k == 0).all() and v[0, 1, 9, 3] == -0.25 and np.count_nonzero(v) == 1


def test_the_reference_scale():
    for most, e in ((448.0, 0), (448.1, 1), (224.0, -1), (225.0, 0), (0.0, -117), (1e-40, -117), (3.3895314e38, 119),
                    (1.0, -8), (0.875 * 2.0 ** -100, -109)):
        assert ref.exponent(most) == e, most
    x = np.array([448.0, 460.0, 2.0 ** -10, 2.0 ** -10 * 1.01, -17.0, -0.0, np.inf, np.nan, 26.0, 27.0])
    assert np.array_equal(E4M3[ref.codes_of(x, 0)], [448, 448, 0, 2.0 ** -9, -16, 0, np.nan, np.nan, 26, 28], equal_nan=True)
