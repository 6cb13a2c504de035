"""Cosines and sines of csrc/rotary.cuh against 64 bits: the function as it stands,
compiled for the host with the device's rounded operations as IEEE ones.  (The bf16 and
4-bit results of the GPU show one fp32 unit once in 2^16 only.)"""
import ctypes
import os
import subprocess

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "exact_attention_40_gb300", "csrc")

SOURCE = """
#include <cuda_runtime.h>
#include <cmath>
static inline float __fmul_rn(float a, float b) { return a * b; }
static inline float __fadd_rn(float a, float b) { return a + b; }
static inline float __fsub_rn(float a, float b) { return a - b; }
static inline float __fmaf_rn(float a, float b, float c) { return std::fma(a, b, c); }
#include "rotary.cuh"
extern "C" void cos_sin(const unsigned long long* turn, float* c, float* s, long n) {
  for (long i = 0; i < n; ++i) {
    const float2 y = exattn::turn_cos_sin(turn[i]);
    c[i] = y.x;
    s[i] = y.y;
  }
}
"""


@pytest.fixture(scope="module")
def cos_sin(tmp_path_factory):
    at = tmp_path_factory.mktemp("rotary")
    (at / "host.cpp").write_text(SOURCE)
    cuda = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    subprocess.run(["g++", "-O2", "-std=c++17", "-ffp-contract=off", "-shared", "-fPIC", "-I" + CSRC, "-I" + cuda,
                    str(at / "host.cpp"), "-o", str(at / "host.so")], check=True)
    lib = ctypes.CDLL(str(at / "host.so"))

    def call(turn):
        turn = np.ascontiguousarray(turn, np.uint64)
        c, s = np.empty(turn.size, np.float32), np.empty(turn.size, np.float32)
        lib.cos_sin(*(x.ctypes.data_as(ctypes.c_void_p) for x in (turn, c, s)), ctypes.c_long(turn.size))
        return c, s
    return call


def exact(turn):
    """fp64 cosine and sine of turn / 2^64 turns, reduced to an eighth first."""
    turn = turn.astype(np.uint64)
    quadrant = ((turn + np.uint64(1 << 61)) >> np.uint64(62)).astype(np.int64) & 3
    rest = (turn - (quadrant.astype(np.uint64) << np.uint64(62))).view(np.int64)
    x = rest.astype(np.float64) * (2 * np.pi / 2.0 ** 64)
    c, s = np.cos(x), np.sin(x)
    return (np.choose(quadrant, [c, -s, -c, s]), np.choose(quadrant, [s, c, -s, -c]))


def wrong(got, want):
    """How many are not the nearest fp32 number; none may be more than its neighbour."""
    near = want.astype(np.float32)
    off = np.abs(got.view(np.int32).astype(np.int64) - near.view(np.int32))
    zero = want == 0
    assert (np.abs(got[zero]) == 0).all()
    assert off[~zero].max(initial=0) <= 1
    return int((off[~zero] != 0).sum())


def check(cos_sin, turn):
    got, want = cos_sin(turn), exact(turn)
    return sum(wrong(g, w) for g, w in zip(got, want)), 2 * turn.size


def test_positions_of_a_spectrum(cos_sin):
    """20,000 positions of 64 pairs, base 500,000."""
    theta = 500000.0 ** -(np.arange(64) / 64.0)
    u = np.rint(theta * (2.0 ** 64 / (2 * np.pi))).astype(np.uint64)
    n, of = check(cos_sin, (np.arange(20000, dtype=np.uint64)[:, None] * u).reshape(-1))
    assert n <= 5e-4 * of, "%d of %d are not the nearest" % (n, of)


def test_any_turn(cos_sin):
    rng = np.random.default_rng(7)
    n, of = check(cos_sin, rng.integers(0, 2 ** 64, 1_000_000, dtype=np.uint64, endpoint=False))
    assert n <= 5e-4 * of, "%d of %d are not the nearest" % (n, of)


def test_around_the_eighths_and_small_turns(cos_sin):
    eighths = (np.arange(8, dtype=np.uint64) << np.uint64(61))[:, None]
    steps = 1 << np.arange(42, 58, dtype=np.int64)
    n, of = check(cos_sin, (eighths + np.concatenate([steps, -steps]).view(np.uint64)).reshape(-1))
    assert n <= 0.02 * of  # few of them, and none more than one unit off
    c, s = cos_sin(np.arange(4, dtype=np.uint64) << np.uint64(62))
    assert c.tolist() == [1, 0, -1, 0] and s.tolist() == [0, 1, 0, -1]


def test_turns_next_to_a_quarter(cos_sin):
    """Closer than 2^-22 of a turn to a quarter one of the two is nearly zero, and what it
    has is an absolute error: the turn is cut to units of 2^-50 (one unit), held as
    r1 2^24 + r0, and r0 < 2^24 units times 2 pi is good to 2^-23 (the constant's rounding
    and the product's, 2 units) like its sum with the r1 term (1 unit).  Four units of
    2 pi 2^-50 are below 2^-45, which an element of the size of an fp32 unit of its
    neighbour's product would not show."""
    rng = np.random.default_rng(8)
    near = rng.integers(-2 ** 42, 2 ** 42, 100_000, dtype=np.int64)
    near[:60] = np.concatenate([1 << np.arange(30, dtype=np.int64), -(1 << np.arange(30, dtype=np.int64))])
    quarter = rng.integers(0, 4, near.size).astype(np.uint64) << np.uint64(62)
    turn = quarter + near.view(np.uint64)
    for got, want in zip(cos_sin(turn), exact(turn)):
        big = np.abs(want) > 0.5
        assert wrong(got[big], want[big]) <= 5e-4 * big.sum()
        assert (np.abs(got[~big] - want[~big]) <= 2.0 ** -45 + 2.0 ** -24 * np.abs(want[~big])).all()
