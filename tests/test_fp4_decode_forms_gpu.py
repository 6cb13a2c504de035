"""4-bit decode: the forms that large batches, large groups and long tails take, against
the plain implementation in 64 bits.

Bar, from the arithmetic: scores are fp32 sums of exact products and the exponentials good
to 2^-21, so a weight is off by 2^-17 max|s| + 2^-21 relative at the most, and enters the
product with V rounded to fp16, by 2^-11 relative or by half of fp16's smallest
subnormal, 2^-25, where the reference weight is 2^7: by 2^-32 of the largest weight.
The sum of the weights takes them unrounded.  The output rounds to bf16 (2^-8; partial
outputs are fp32).  With W = sum of weights over the largest of them,
|o - ref| <= 2^-8 |ref| + (2^-10 + 2^-17 max|s|) mean|v| + n 2^-32 max|v| / W,
|lse - ref| <= 2^-20 (1 + max|s| + |ref|)."""
import numpy as np
import pytest

import fp4_reference as ref
from exact_attention_40_gb300 import synth
from helpers import to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from exact_attention_40_gb300 import build
    build.build()
    from exact_attention_40_gb300 import exattn
    return torch, exattn, torch.device("cuda:0")


def check(got, lse, want, lens):
    """got, lse against ref.decode's results."""
    out, wl, big, mean, most = want
    n = np.asarray(lens, np.float64)[:, None, None]
    # (the largest score is at most max|s|: W is no smaller than this)
    total = np.where(np.isfinite(wl), np.exp(wl - big), 1.0)[..., None]
    bar = 2.0 ** -8 * np.abs(out) + (2.0 ** -10 + 2.0 ** -17 * big[..., None]) * mean + n * 2.0 ** -32 * most / total
    assert np.isfinite(got).all()
    err = np.abs(got - out)
    assert (err <= bar).all(), "off by %.3e over the bar" % (err - bar).max()
    empty = np.isneginf(wl)
    assert np.array_equal(np.isneginf(lse), empty) and (got[empty] == 0).all()
    assert (np.abs(lse[~empty] - wl[~empty]) <= 2.0 ** -20 * (1 + big + np.abs(wl))[~empty]).all()


def run(env, q, cache, table, lens, d, scale, k_scale=1.0, v_scale=1.0, rows=None):
    """Decodes the whole batch; compares the sequences `rows` (all by default)."""
    torch, ex, dev = env
    out, lse = ex.attn_decode_paged_fp4(to_dev(q, dev), to_dev(cache, dev), to_dev(table, dev), to_dev(lens, dev),
                                        scale=scale, k_scale=k_scale, v_scale=v_scale)
    torch.cuda.synchronize()
    assert ex.attn_get_device_status() == 0
    rows = np.arange(len(lens)) if rows is None else rows
    want = ref.decode(q[rows], cache, table[rows], lens[rows], d, scale, k_scale, v_scale)
    check(out.double().cpu().numpy()[rows], lse.double().cpu().numpy()[rows], want, lens[rows])
    return out, lse


def shared_pages(lens, pages):
    """A block table over few pages that the sequences share, each in an order of its own."""
    most = int((lens.max() + 15) // 16)
    s, b = np.meshgrid(np.arange(len(lens)), np.arange(most), indexing="ij")
    table = ((s * 37 + b * (2 * (s % 13) + 1)) % pages).astype(np.int32)
    return np.where(b * 16 < lens[:, None], table, -1).astype(np.int32)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("S,Hq,Hkv,hi", [
    (64, 32, 8, 2500),    # 512 segments of up to 8 rows
    (64, 64, 8, 900),     # all 8 of them used
    (40, 96, 8, 1500),    # 320 segments of 12 rows, 304 CTAs
    (30, 160, 8, 700),    # 20 rows a KV head: two chunks of 16, the second of 4
    (120, 40, 1, 1000),   # one KV head, three chunks
    (160, 17, 1, 1200),   # a second chunk of one row
    (460, 2, 1, 1300),    # just above one wave of segments
])
def test_more_segments_than_ctas(env, d, S, Hq, Hkv, hi):
    """Segments that go on in further CTAs are then found in the list that the split
    kernel writes.  Lengths from 0 to hi, most of them short."""
    group = Hq // Hkv
    rows = 8 if group <= 8 else 16
    assert S * Hkv * -(-group // rows) > 152 * (3 if rows == 8 else 2)
    lens = np.floor(synth.uniform01(630 + S, S) ** 2 * (hi + 1)).astype(np.int32)
    lens[[0, S // 2, S - 1]] = 0
    lens[1] = hi
    cache = ref.random_cache(631, 150, Hkv, d, 0.01, 0.003)
    q = synth.normal_bf16(632, 0, (S, Hq, d))
    some = np.unique(np.concatenate([[0, 1, S // 2, S - 1], np.argsort(lens)[-4:], np.arange(2, S, max(1, S // 12))]))
    table = shared_pages(lens, 150)
    args = (q, cache, table, lens, d, d ** -0.5, 0.01, 0.003)
    out, lse = run(env, *args, rows=some)
    # every row, also those not compared above: a sequence alone gives nearly the same
    torch, ex, dev = env
    for s in range(0, S, max(1, S // 30)):
        one, one_lse = ex.attn_decode_paged_fp4(to_dev(q[s:s + 1], dev), to_dev(cache, dev), to_dev(table[s:s + 1], dev),
                                                to_dev(lens[s:s + 1], dev), scale=d ** -0.5, k_scale=0.01, v_scale=0.003)
        assert (one - out[s]).abs().max() <= 2.0 ** -6 * out[s].abs().max() + 1e-6
        assert torch.allclose(one_lse[0], lse[s], rtol=0, atol=1e-4)


@pytest.mark.parametrize("bits", [20, 27, 30])
@pytest.mark.parametrize("place", [0, 31])
@pytest.mark.parametrize("d,S,n,Hq", [(64, 1, 128, 1), (128, 3, 1000, 8), (64, 2, 20000, 12), (128, 500, 1500, 2)])
def test_weights_far_below_the_largest_are_not_lost(env, bits, place, d, S, n, Hq):
    """One token in 32 has nearly all the weight and a value of zero, the others 2^-bits of
    it each and a value of one: what they add up to is all that the output holds."""
    blocks = (n + 15) // 16
    cache = np.zeros((blocks, 1, 18 * d), np.uint8)
    ck, cv, sk, sv = ref.split(cache, d)
    sk[...] = sv[...] = 0x38           # 1.0
    cv[...] = 0x22                     # 1.0, 1.0
    tok = np.arange(blocks * 16)
    big = tok[tok % 32 == place]
    cv[big // 16, 0, big % 16] = 0
    ck[big // 16, 0, big % 16, 0] = 0x07  # 6 in column 0
    f = np.zeros((S, Hq, d), np.float32)
    f[..., 0] = 1.0
    table = np.tile(np.arange(blocks, dtype=np.int32), (S, 1))
    lens = np.full(S, n, np.int32)
    run(env, synth.f32_to_bf16_bits(f), cache, table, lens, d, bits * np.log(2.0) / 6, rows=np.arange(min(S, 3)))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bits", [20, 28, 34, 60])
@pytest.mark.parametrize("lens,Hq", [([900, 31, 1], 4), ([128, 100], 16), ([9000, 0, 300], 20)])
def test_scores_beyond_fp32_resolution(env, d, bits, lens, Hq):
    """Scores of about 2^bits and more: all the weight falls to the largest, and the output is its
    token's value.  (Where the largest two are closer than fp32's rounding of the sums of d
    products, 2^-18 of the largest, either may have it.)"""
    torch, ex, dev = env
    lens = np.asarray(lens, np.int32)
    table, nb = synth.paged_layout(lens, 16, 650)
    cache = ref.random_cache(650, nb, 1, d)
    q = synth.normal_bf16(651, 0, (len(lens), Hq, d))
    scale = 2.0 ** bits / d ** 0.5
    out, lse = ex.attn_decode_paged_fp4(to_dev(q, dev), to_dev(cache, dev), to_dev(table, dev), to_dev(lens, dev), scale=scale)
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    f = synth.bf16_bits_to_f32(q).astype(np.float64)
    for s, n in enumerate(lens):
        if n == 0:
            continue
        k, v = (x.transpose(0, 2, 1, 3).reshape(-1, d)[:n] for x in
                ref.cache_values(cache[table[s, :(n + 15) // 16]], d, 1.0, 1.0))
        x = f[s] @ k.T * scale
        for h in range(Hq):
            big = np.abs(x[h]).max()
            assert abs(lse[s, h] - x[h].max()) <= 2.0 ** -18 * big
            near = x[h] >= x[h].max() - 2.0 ** -18 * big - 25.0
            lo, hi = v[near].min(0), v[near].max(0)  # a mean of these
            assert (out[s, h] >= lo - 2.0 ** -8 * np.abs(lo) - 1e-9 * n).all()
            assert (out[s, h] <= hi + 2.0 ** -8 * np.abs(hi) + 1e-9 * n).all()
    assert ex.attn_get_device_status() == 0


@pytest.mark.parametrize("v_scale", [2e-38, 1e35])
@pytest.mark.parametrize("S,n,Hq", [(2, 3000, 4), (2, 100, 9), (1, 70000, 12), (460, 20000, 1)])
def test_value_scales_near_the_ends_of_fp32(env, v_scale, S, n, Hq):
    """Flat scores, so that the sum of the weights is as large as it gets beside them."""
    lens = np.full(S, n, np.int32)
    lens[S // 2] = n - 9
    cache = ref.random_cache(660, 300, 1, 64)
    ref.split(cache, 64)[3][...] |= 0x40  # scales of 2 and more
    q = np.zeros((S, Hq, 64), np.uint16)
    some = np.unique([0, S // 2, S - 1])
    run(env, q, cache, shared_pages(lens, 300), lens, 64, 0.125, v_scale=v_scale, rows=some)
