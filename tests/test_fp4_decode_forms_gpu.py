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
