"""The 8-bit decode where scores are so large that fp32 holds them in steps of 2^-4 to 2^7
(2^20 to 2^30 and more).  What a softmax gives does not depend on the size of its scores where
these are equal, or so far apart that all but the largest count nothing; so neither does the
bar, which is that of test_fp8_gpu.py without its term for the rounding of scores:
|o - ref| <= 2^-8 |ref| + 2^-10 mean|v| + n 2^-23 part.

Queries have one column that is not 0, keys one value in it for all tokens of a block: a score
is one product, and tokens with one key have one score to the last bit."""
import numpy as np
import pytest

import fp8_reference as ref
from exact_attention_40_gb300 import synth
from helpers import to_dev
from test_fp8_gpu import env  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu

VALUE_EXPONENTS = np.array([-8, -7, 4, -12, 16, 0, -3, 9, -15, -6])


def large_case(seed, lens, columns, d, key_of_block=None, queries=None, low=20, high=31):
    """Scores of magnitudes 2^low to 2^high, of both signs, one for each column; value scales
    that differ from block to block.  key_of_block(b): the key's value in a sequence's block b."""
    lens = np.asarray(lens, np.int32)
    S = len(lens)
    table, nb = synth.paged_layout(lens, 16, seed)
    cache = ref.random_cache(seed, nb, 1, d)
    codes, scales = ref.split(cache, d)
    scales[:, 0, 1] = 2.0 ** VALUE_EXPONENTS[np.arange(nb) * 7 % 10]
    codes[:, :, 0] = 0
    scales[:, :, 0] = 1.0
    at = ref.place(d)[:, 5]
    for s in range(S):
        for b in range((int(lens[s]) + 15) // 16):
            value = 1.0 if key_of_block is None else key_of_block(b)
            codes[table[s, b], 0, 0, at] = ref.codes_of(np.full(16, value), 0)
    N = 1 if queries is None else queries
    u = synth.uniform01(seed + 3, 3 * S * N * columns).reshape(3, S, N, columns)
    size = 2.0 ** np.floor(low + u[0] * (high - low)) * (1 + np.floor(u[1] * 128) / 128)  # bf16 numbers
    q = np.zeros((S, N, columns, d), np.float32)
    q[..., 5] = np.where(u[2] < 0.5, -size, size)
    q = synth.f32_to_bf16_bits(q)
    return q if queries is not None else q[:, 0], cache, table, lens


def check(env, case, d, label=""):
    torch, ex, dev = env
    q, cache, table, lens = case
    out, lse = ex.attn_decode_paged_fp8(*(to_dev(x, dev) for x in case), scale=1.0)
    torch.cuda.synchronize()
    assert ex.attn_get_device_status() == 0
    q4 = q if q.ndim == 4 else q[:, None]
    want, wl, big, mean, part = ref.decode(q4, cache, table, lens, d, 1.0)
    got, gl = out.double().cpu().numpy().reshape(want.shape), lse.double().cpu().numpy().reshape(wl.shape)
    assert np.isfinite(got).all(), label
    n = np.asarray(lens, np.float64)[:, None, None, None]
    bar = 2.0 ** -8 * np.abs(want) + 2.0 ** -10 * mean + n * 2.0 ** -23 * part[..., None]
    err = np.abs(got - want)
    assert (err <= bar).all(), "%s: out off by %.3e over the bar" % (label, (err - bar).max())
    seen = np.isfinite(wl)
    assert np.array_equal(np.isneginf(gl), ~seen) and (got[~seen] == 0).all(), label
    bar = 2.0 ** -16 * big[seen] + 2.0 ** -19 * (1 + np.abs(wl[seen]))
    assert (np.abs(gl[seen] - wl[seen]) <= bar).all(), label


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("S,columns", [(5, 3), (600, 2), (300, 12)])
def test_one_token_is_its_value(env, d, S, columns):
    """Whatever the score and the value's scale."""
    check(env, large_case(930, np.ones(S, np.int32), columns, d), d)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("S,columns,queries", [(3, 4, None), (500, 2, None), (200, 16, None), (40, 4, 4)])
def test_equal_scores_give_the_mean_of_the_values(env, d, S, columns, queries):
    """Contexts of one unit of work, whose blocks have scales of their own."""
    lens = 1 + np.arange(S) * 11 % (64 if d == 128 else 128)
    check(env, large_case(931, lens, columns, d, queries=queries), d)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("columns", [3, 14])
@pytest.mark.parametrize("key", ["rising", "falling", "mixed"])
def test_scores_far_apart_give_the_largest_ones_values(env, d, columns, key):
    """Blocks whose scores differ by a 32nd of their size and more."""
    key_of_block = {"rising": lambda b: 1.0 + b % 8 / 8 + 8.0 * (b // 8), "falling": lambda b: 2.0 ** -(b % 9),
                    "mixed": lambda b: 1.0 + b * 5 % 8 / 8}[key]
    check(env, large_case(932, [60, 100, 1, 250, 33, 1000], columns, d, key_of_block), d)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,columns,queries", [([1000, 77, 300], 4, None), ([1500, 90], 10, None), ([20000, 130], 4, None),
                                                  ([9000, 2, 4500], 12, None), ([3000] * 30, 3, 2), ([400, 700, 33] * 200, 2, None)],
                         ids=["cluster", "cluster 10", "two long", "long 12", "queries", "many"])
def test_equal_scores_in_several_ctas_give_the_mean_of_the_values(env, d, lens, columns, queries):
    """Their parts merge in a cluster, in a grid that finds the segments and in one that reads
    the list of shared ones."""
    check(env, large_case(933, lens, columns, d, queries=queries), d)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,queries", [(2, None), (12, None), (2, 3)])
@pytest.mark.parametrize("n", [40, 300, 9000])
def test_factors_past_what_fp32_holds(env, d, Hq, queries, n):
    """The largest element of a query meets keys of 0, the second is 2^-20 of it: the query's
    size, the key's scale and the scale together are 2^136 to 2^140, the scores 2^110 and 2^111.
    The first block has the larger scale and the smaller codes, and the larger scores."""
    shape = (1, Hq, d) if queries is None else (1, queries, Hq, d)
    table, nb = synth.paged_layout(np.array([n], np.int32), 16, 934)
    cache = ref.random_cache(934, nb, 1, d)
    codes, scales = ref.split(cache, d)
    codes[:, :, 0] = 0
    scales[:, 0, 0] = 2.0 ** 36
    codes[:, 0, 0, ref.place(d)[:, 9]] = 0x08  # 2^-6
    first = table[0, 0]
    scales[first, 0, 0] = 2.0 ** 40
    codes[first, 0, 0, ref.place(d)[:, 9]] = 0x01  # 2^-9
    q = np.zeros(shape, np.float32)
    q[..., 3], q[..., 9] = 2.0 ** 100, 2.0 ** 80
    case = synth.f32_to_bf16_bits(q), cache, table, np.array([n], np.int32)
    check(env, case, d)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [40, 300, 9000])
def test_scores_past_fp32_are_nan_in_their_head_alone(env, d, n):
    torch, ex, dev = env
    q, cache, table, lens = large_case(935, [n], 3, d, low=20, high=24)
    huge = synth.bf16_bits_to_f32(q)
    huge[0, 1, 5] = 2.0 ** 100
    scales = ref.split(cache, d)[1]
    scales[table[0, 0], 0, 0] = 2.0 ** 40  # the first block's score: 2^140
    args = [to_dev(x, dev) for x in (cache, table, lens)]
    want, want_lse = ex.attn_decode_paged_fp8(to_dev(q, dev), *args, scale=1.0)
    out, lse = ex.attn_decode_paged_fp8(to_dev(synth.f32_to_bf16_bits(huge), dev), *args, scale=1.0)
    assert torch.isnan(out[0, 1]).all() and torch.isnan(lse[0, 1])
    for h in (0, 2):
        assert torch.equal(out[0, h], want[0, h]) and torch.equal(lse[0, h], want_lse[0, h])
    assert torch.isfinite(want[0, [0, 2]]).all() and ex.attn_get_device_status() == 0
