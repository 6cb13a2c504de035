"""The 8-bit decode of several query tokens where a key or a value that only the later ones see is
NaN: every output against the definition in 64 bits, with the bar of test_fp8_gpu.py, while the
block that holds the NaN has most of the weight."""
import numpy as np
import pytest

import fp8_reference as ref
from exact_attention_40_gb300 import synth
from helpers import to_dev
from test_fp8_gpu import env  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


def nan_case(seed, n, back, Hq, d, queries, which, column):
    """Queries near one vector of signs; keys of the NaN's block near it too, so that their
    scores lie about sqrt(d) above the others'."""
    lens = np.array([n, 20], np.int32)
    table, nb = synth.paged_layout(lens, 16, seed)
    cache = ref.random_cache(seed, nb, 1, d)
    codes, scales = ref.split(cache, d)
    signs = np.where(synth.uniform01(seed + 1, d) < 0.5, -1.0, 1.0)
    tok = n - back
    block = table[0, tok // 16]
    noise = synth.bf16_bits_to_f32(synth.normal_bf16(seed, 3, (1, 16, d))).astype(np.float64) / 8
    ref.set_tokens(cache, d, block, 0, ref.codes_of(signs + noise, 0))
    scales[block, :, 0] = 1.0
    q = signs + synth.bf16_bits_to_f32(synth.normal_bf16(seed, 0, (2, queries, Hq, d))) / 4
    codes[block, 0, which, ref.place(d)[tok % 16, column]] = 0x7F
    return synth.f32_to_bf16_bits(q.astype(np.float32)), cache, table, lens


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,queries", [(1, 5), (3, 5), (2, 16)])
@pytest.mark.parametrize("n,back", [(37, 2), (64, 1), (129, 2), (9000, 2)])
@pytest.mark.parametrize("which", [0, 1], ids=["key", "value"])
def test_queries_on_both_sides_of_a_nan(env, d, Hq, queries, n, back, which):
    torch, ex, dev = env
    column = d - 7
    q, cache, table, lens = nan_case(940, n, back, Hq, d, queries, which, column)
    out, lse = ex.attn_decode_paged_fp8(*(to_dev(x, dev) for x in (q, cache, table, lens)))
    torch.cuda.synchronize()
    assert ex.attn_get_device_status() == 0
    with np.errstate(invalid="ignore"):
        want, wl, big, mean, part = ref.decode(q, cache, table, lens, d, d ** -0.5)
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    lost = np.zeros(want.shape, bool)  # where the definition has a NaN
    lost[0, queries - back:, :, slice(None) if which == 0 else column] = True
    assert np.array_equal(np.isnan(want), lost) and np.array_equal(np.isnan(got), lost)
    bar = (2.0 ** -8 * np.abs(want) + (2.0 ** -10 + 2.0 ** -15 * big[..., None]) * mean
           + lens[:, None, None, None] * 2.0 ** -23 * part[..., None])
    assert (np.abs(got - want)[~lost] <= bar[~lost]).all()
    # the outputs that the bar is held against are well above it
    assert np.abs(want[0])[~lost[0]].mean() > 20 * bar[0][~lost[0]].mean()
    seen = np.isfinite(wl)
    assert np.array_equal(np.isnan(gl), np.isnan(wl)) and np.array_equal(np.isneginf(gl), np.isneginf(wl))
    assert (np.abs(gl[seen] - wl[seen]) <= 2.0 ** -16 * big[seen] + 2.0 ** -19 * (1 + np.abs(wl[seen]))).all()
