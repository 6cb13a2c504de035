"""The 8-bit paged cache on the GPU: append, read and decode against the plain
implementations of fp8_reference.py.

Decode bar, from the arithmetic.  A score is an fp32 sum of d exact products, off by at
most d 2^-23 of the sum of their magnitudes, `big` (mma sums may truncate), which is
2^-16 for d = 128; a few roundings of the product with the scale and of its distance from
the reference come on top.  With both sums of the softmax a weight is off by 2^-15 big of
itself.  The exponentials are good to 2^-21.  Weights round to fp16 in the sum over the
values alone: by 2^-11 of themselves, or by half the smallest subnormal, 2^-25, where the
largest product of a weight and its block's value scale is at least 2^7: n tokens of
codes up to 2^9 add up to n 2^-23 of that product, `part`.  Merges add some 2^-20.  The
output rounds to bf16 (2^-8):
|o - ref| <= 2^-8 |ref| + (2^-10 + 2^-15 big) mean|v| + n 2^-23 part,
|lse - ref| <= 2^-16 big + 2^-19 (1 + |ref|)."""
import numpy as np
import pytest

import fp4_reference as ref4
import fp8_reference as ref
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


def bits(t):
    import torch
    return t.detach().cpu().contiguous().view(torch.int16).numpy().view(np.uint16)


# ------------------------------------------------------------------- decode
def decode_case(seed, lens, Hq, Hkv, d, queries=None, gain=1.0, k_exp=0, v_exp=0, extra_blocks=0, poison=True):
    """q, cache, table, lens; slots past a sequence's last token hold NaN codes."""
    lens = np.asarray(lens, np.int32)
    table, nb = synth.paged_layout(lens, 16, seed, extra_blocks)
    cache = ref.random_cache(seed, nb, Hkv, d, gain, k_exp, v_exp)
    if poison:
        codes = ref.split(cache, d)[0]
        for s, n in enumerate(lens):
            if n % 16:
                codes[table[s, n // 16]][..., ref.place(d)[n % 16:].ravel()] = 0x7F
    shape = (len(lens), Hq, d) if queries is None else (len(lens), queries, Hq, d)
    return synth.normal_bf16(seed, 0, shape), cache, table, lens


def check_decode(out, lse, q, cache, table, lens, d, scale, label=""):
    q4 = q.reshape(q.shape[0], -1, *q.shape[-2:]) if q.ndim == 4 else q[:, None]
    want, wl, big, mean, part = ref.decode(q4, cache, table, lens, d, scale)
    got, gl = out.double().cpu().numpy().reshape(want.shape), lse.double().cpu().numpy().reshape(wl.shape)
    n = np.asarray(lens, np.float64)[:, None, None, None]
    bar = 2.0 ** -8 * np.abs(want) + (2.0 ** -10 + 2.0 ** -15 * big[..., None]) * mean + n * 2.0 ** -23 * part[..., None]
    assert np.isfinite(got).all(), label
    err = np.abs(got - want)
    assert (err <= bar).all(), "%s: out off by %.3e over the bar" % (label, (err - bar).max())
    empty = np.isneginf(wl)
    assert np.array_equal(np.isneginf(gl), empty), label
    assert (got[empty] == 0).all(), label
    if (~empty).any():
        le = np.abs(gl[~empty] - wl[~empty])
        assert (le <= (2.0 ** -16 * big + 2.0 ** -19 * (1 + np.abs(wl)))[~empty]).all(), "%s: lse off by %.3e" % (label, le.max())


def run_decode(env, case, d, scale=None, status=0, label=""):
    torch, ex, dev = env
    q, cache, table, lens = case
    scale = d ** -0.5 if scale is None else scale
    out, lse = ex.attn_decode_paged_fp8(*(to_dev(x, dev) for x in (q, cache, table, lens)), scale=scale)
    torch.cuda.synchronize()
    assert ex.attn_get_device_status() == status
    assert out.shape == q.shape and lse.shape == q.shape[:-1]
    check_decode(out, lse, q, cache, table, lens, d, scale, label)
    return out, lse


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", [[0], [1], [15, 16, 17], [0, 33, 64, 65, 128, 129, 640, 1], [3000, 5], [70000, 0, 777]],
                         ids=lambda x: "-".join(map(str, x)))
def test_decode_lengths(env, d, lens):
    run_decode(env, decode_case(400, lens, 4, 1, d), d)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (8, 2), (7, 1), (16, 2), (9, 1), (16, 1), (34, 2), (40, 1)])
def test_decode_head_layouts(env, d, Hq, Hkv):
    run_decode(env, decode_case(401, [200, 1, 47], Hq, Hkv, d), d)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("queries", [1, 2, 3, 5, 16])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 2), (7, 1), (24, 2)])
def test_decode_several_queries(env, d, queries, Hq, Hkv):
    """Contexts that end around units, and ones with fewer tokens than queries."""
    run_decode(env, decode_case(402, [0, 1, 2, 15, 64, 66, 130, 300], Hq, Hkv, d, queries), d)


@pytest.mark.parametrize("lens", [[6000, 4100], [3, 20000], [8, 300, 7] * 60], ids=["long", "mixed", "many"])
def test_decode_several_queries_of_shared_segments(env, lens):
    """Shares that end inside sequences: partial outputs by the row of each query and head."""
    run_decode(env, decode_case(403, lens, 12, 2, 128, 3), 128)
    run_decode(env, decode_case(404, lens, 2, 1, 64, 4), 64)


def test_decode_queries_are_the_single_token_decodes(env):
    """Query i of n is the decode of the context that ends with it, to the roundings that
    other places of the units bring."""
    torch, ex, dev = env
    q, cache, table, lens = decode_case(405, [900, 64, 4], 4, 2, 128, 4)
    qd, cd, td, ld = (to_dev(x, dev) for x in (q, cache, table, lens))
    out, lse = ex.attn_decode_paged_fp8(qd, cd, td, ld)
    for i in range(4):
        one, one_lse = ex.attn_decode_paged_fp8(qd[:, i].contiguous(), cd, td, ld - (3 - i))
        # both are within 2^-8 |o| + 2^-10 mean|v| (and less) of the definition
        assert (out[:, i].float() - one.float()).abs().max() <= 2 * (2 ** -8 * 4 + 2 ** -10 * 4)
        assert (lse[:, i] - one_lse).abs().max() <= 1e-3
    assert ex.attn_get_device_status() == 0


@pytest.mark.parametrize("S,Hq,Hkv,hi", [(40, 4, 2, 5000), (160, 8, 4, 600), (700, 2, 1, 40), (130, 24, 2, 300),
                                         (129, 2, 1, 3000), (400, 3, 1, 1500), (1100, 4, 2, 280), (2100, 1, 1, 200)])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_many_sequences(env, S, Hq, Hkv, hi, d):
    """Ragged batches, empty sequences among them: shares that end inside sequences,
    shares of many sequences, more segments than CTAs, and no segment of two units."""
    lens = np.floor(synth.uniform01(70 + S, S) ** 2 * (hi + 1)).astype(np.int32)
    lens[[0, S // 2, S - 1]] = 0
    lens[1] = hi
    run_decode(env, decode_case(420, lens, Hq, Hkv, d), d)


@pytest.mark.parametrize("blocks", [4, 5, 8, 9, 64, 255, 256, 257, 264])
@pytest.mark.parametrize("Hq,Hkv", [(3, 1), (20, 2)])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_around_the_limits_of_a_small_call(env, blocks, Hq, Hkv, d):
    """Lengths at which a sequence gets a second unit, fills the cluster's shares and
    passes from the cluster to shares of the whole batch."""
    n = blocks * 16
    run_decode(env, decode_case(421, [n, n - 15, 1, 0, max(1, n - 128)], Hq, Hkv, d), d)


@pytest.mark.parametrize("queries", [None, 4])
def test_decode_serving_batch(env, queries):
    lens = synth.ctx_lengths(5, 24, 512, 8192)
    run_decode(env, decode_case(422, lens, 8, 2, 128, queries), 128)


@pytest.mark.parametrize("gain", [30.0, 1e-3])
def test_decode_peaked_and_flat_scores(env, gain):
    run_decode(env, decode_case(423, [900, 31], 4, 2, 128, gain=gain), 128)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("k_exp,v_exp", [(0, 100), (3, 60), (0, 20), (8, 0)])
def test_decode_blocks_of_very_different_scales(env, d, k_exp, v_exp):
    """Value scales up to 2^200 apart: a block with the weight but small values, beside one
    with large values and no weight."""
    run_decode(env, decode_case(424, [700, 90, 16, 4000], 6, 2, d, k_exp=k_exp, v_exp=v_exp), d,
               scale=d ** -0.5 if k_exp < 8 else 2.0 ** -9)


@pytest.mark.parametrize("d", [64, 128])
def test_decode_small_values_keep_their_part_beside_large_ones(env, d):
    """One block holds all the weight and values of 2^-30; the other blocks' values are
    normal and their weights some e^-90."""
    q, cache, table, lens = decode_case(425, [200], 2, 1, d, poison=False)
    codes, scales = ref.split(cache, d)
    one = np.ones((1, 16, d), np.float64)
    for b in table[0, :13]:
        ref.set_tokens(cache, d, b, 0, ref.codes_of(-one, 0))
        scales[b, :, 0] = 1.0
    ref.set_tokens(cache, d, table[0, 5], 0, ref.codes_of(one, 0))
    scales[table[0, 5], :, 1] = 2.0 ** -38
    q = synth.f32_to_bf16_bits(np.full(q.shape, 1.0, np.float32))
    case = (q, cache, table, lens)
    out, _ = run_decode(env, case, d, scale=45.0 / d)
    assert 0 < out.abs().max().item() < 2.0 ** -28


@pytest.mark.parametrize("d", [64, 128])
def test_decode_scores_that_keep_growing(env, d):
    """Keys whose scores rise by up to some thousands along the sequence: every
    block moves the running maximum."""
    q, cache, table, lens = decode_case(426, [400], 2, 1, d, poison=False)
    scales = ref.split(cache, d)[1]
    sign = np.where(synth.bf16_bits_to_f32(q[0, 0]) >= 0, 1.0, -1.0)
    for b in range(25):
        x = np.repeat(sign[None], 16, 0) * (16.0 + np.arange(16)[:, None])
        ref.set_tokens(cache, d, table[0, b], 0, ref.codes_of(x, 0)[None])
        scales[table[0, b], :, 0] = 2.0 ** (b // 5 - 4)
    run_decode(env, (q, cache, table, lens), d, scale=1.0)


def test_decode_queries_of_any_size(env):
    """Queries are scaled by powers of two on their way into fp16: tiny, huge and
    mixed rows lose nothing that the result could show; nor do products of huge queries
    and tiny keys."""
    q, cache, table, lens = decode_case(427, [100, 60], 8, 2, 128)
    f = synth.bf16_bits_to_f32(q)
    f[0, 0] *= 2.0 ** -100
    f[0, 1] *= 2.0 ** -130      # bf16 subnormals
    f[0, 2] = 0
    f[0, 3] *= 2.0 ** 12
    f[0, 4, ::2] *= 2.0 ** -20  # elements far below the row's largest
    f[0, 5, :] = 0
    f[0, 5, 7] = 1.0
    run_decode(env, (synth.f32_to_bf16_bits(f), cache, table, lens), 128, scale=2.0 ** -9)
    f[:] = synth.bf16_bits_to_f32(synth.normal_bf16(428, 0, f.shape)) * np.float32(2.0 ** 100)
    run_decode(env, (synth.f32_to_bf16_bits(f), cache, table, lens), 128, scale=2.0 ** -103)
    scales = ref.split(cache, 128)[1]
    scales[:, :, 0] *= np.float32(2.0 ** -104)
    run_decode(env, (synth.f32_to_bf16_bits(f), cache, table, lens), 128, scale=1.0)
    for up in (104, 100):
        scales[:, :, 0] *= np.float32(2.0 ** up)
        f *= np.float32(2.0 ** -up)
    run_decode(env, (synth.f32_to_bf16_bits(f), cache, table, lens), 128, scale=1.0)


def test_decode_of_an_empty_cache_that_is_taken_as_full(env):
    """Zeros: every weight alike, output 0."""
    torch, ex, dev = env
    cache = ex.attn_fp8_cache(4, 2, 64)
    table = torch.arange(4, device=dev, dtype=torch.int32)[None]
    out, lse = ex.attn_decode_paged_fp8(torch.randn(1, 4, 64, device=dev).bfloat16(), cache, table,
                                        torch.tensor([50], device=dev, dtype=torch.int32))
    assert (out == 0).all() and (lse - np.log(50)).abs().max() < 1e-5
    assert ex.attn_get_device_status() == 0


def test_decode_nan_stays_where_it_is_seen(env):
    torch, ex, dev = env
    d = 64
    q, cache, table, lens = decode_case(429, [50, 50], 4, 2, d)
    qd, cd, td, ld = (to_dev(x, dev) for x in (q, cache, table, lens))
    clean, clean_lse = ex.attn_decode_paged_fp8(qd, cd, td, ld)
    qd[0, 1, 3] = float("nan")
    got, lse = ex.attn_decode_paged_fp8(qd, cd, td, ld)
    assert torch.isnan(got[0, 1]).all() and torch.isnan(lse[0, 1])
    keep = torch.ones((2, 4), dtype=torch.bool, device=dev)
    keep[0, 1] = False
    assert torch.equal(got[keep], clean[keep]) and torch.equal(lse[keep], clean_lse[keep])
    qd = to_dev(q, dev)
    at = ref.place(d)
    ref.split(cache, d)[0][table[1, 2], 1, 1, at[4, 37]] = 0xFF  # column 37 of sequence 1's token 36, head 1
    got, lse = ex.attn_decode_paged_fp8(qd, to_dev(cache, dev), td, ld)
    assert torch.isnan(got[1, 2:, 37]).all()
    rest = torch.arange(d, device=dev) != 37
    assert torch.equal(got[1, 2:, rest], clean[1, 2:, rest])
    assert torch.equal(got[0], clean[0]) and torch.equal(got[1, :2], clean[1, :2])
    assert torch.equal(lse, clean_lse)
    assert ex.attn_get_device_status() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [37, 64, 129, 5000])
@pytest.mark.parametrize("which", [0, 1])
def test_decode_queries_before_a_nan_do_not_see_it(env, d, n, which):
    """The third-last token's key or value holds a NaN: the two queries from it on have it,
    those before it are as without it."""
    torch, ex, dev = env
    N = 5
    q, cache, table, lens = decode_case(430, [n, 20], 3, 1, d, N)
    qd, td, ld = (to_dev(x, dev) for x in (q, table, lens))
    clean, clean_lse = ex.attn_decode_paged_fp8(qd, to_dev(cache, dev), td, ld)
    tok = n - 3
    ref.split(cache, d)[0][table[0, tok // 16], 0, which, ref.place(d)[tok % 16, 9]] = 0x7F
    got, lse = ex.attn_decode_paged_fp8(qd, to_dev(cache, dev), td, ld)
    assert torch.equal(got[1], clean[1]) and torch.equal(lse[1], clean_lse[1])
    # (a value's NaN takes another order of sums in that unit)
    assert (got[0, :2].float() - clean[0, :2].float()).abs().max() <= 2 * (2 ** -8 * 4 + 2 ** -10 * 4)
    assert torch.equal(lse[0, :2], clean_lse[0, :2])
    if which == 0:
        assert torch.isnan(got[0, 2:]).all() and torch.isnan(lse[0, 2:]).all()
    else:
        assert torch.isnan(got[0, 2:, :, 9]).all()
        rest = torch.arange(d, device=dev) != 9
        assert torch.isfinite(got[0][..., rest]).all() and torch.equal(lse, clean_lse)
    assert ex.attn_get_device_status() == 0


def test_decode_bad_table_entries_and_lengths_are_flagged(env):
    torch, ex, dev = env
    q, cache, table, lens = decode_case(408, [300, 40, 16], 4, 1, 128)
    table = table.copy()
    table[0, 3] = -1
    table[0, 7] = cache.shape[0]
    table[2, 0] = 2 ** 31 - 1  # all that sequence 2 has
    run_decode(env, (q, cache, table, lens), 128, status=2, label="bad entries")
    out, lse = ex.attn_decode_paged_fp8(to_dev(q, dev), to_dev(cache, dev), to_dev(table, dev),
                                        torch.tensor([-5, 40, 10 ** 6], device=dev, dtype=torch.int32))
    torch.cuda.synchronize()
    assert ex.attn_get_device_status() == 2
    assert (out[0] == 0).all() and (lse[0] == -float("inf")).all()


def test_decode_entries_past_the_context_are_not_read(env):
    q, cache, table, lens = decode_case(409, [33, 500, 16], 4, 2, 64)
    wide = np.full((3, table.shape[1] + 70), 2 ** 31 - 1, np.int32)
    for s, n in enumerate(lens):
        wide[s, :(n + 15) // 16] = table[s, :(n + 15) // 16]
    run_decode(env, (q, cache, wide, lens), 64)


def test_decode_shared_pages(env):
    """Sequences that share physical blocks, one of them twice in one sequence."""
    q, cache, table, lens = decode_case(410, [64, 64, 64], 4, 2, 64)
    table = table.copy()
    table[1, :2] = table[0, :2]
    table[2, 1] = table[2, 0]
    run_decode(env, (q, cache, table, lens), 64)


def test_cache_past_32_bits(env):
    """A pool of more than 4 GiB whose used blocks lie at its end."""
    torch, ex, dev = env
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GiB")
    q, cache, table, lens = decode_case(411, [500, 130], 4, 1, 128)
    nb = 1_100_000  # x 4128 bytes = 4.5 GB
    big = torch.zeros((nb, 1, 4128), device=dev, dtype=torch.uint8)
    big[nb - cache.shape[0]:] = to_dev(cache, dev)
    moved = np.where(table >= 0, table + nb - cache.shape[0], -1).astype(np.int32)
    out, lse = ex.attn_decode_paged_fp8(to_dev(q, dev), big, to_dev(moved, dev), to_dev(lens, dev))
    torch.cuda.synchronize()
    assert ex.attn_get_device_status() == 0
    check_decode(out, lse, q, cache, table, lens, 128, 128 ** -0.5)
    # append to and read from the far end
    T, last = 3, nb - 1
    tbl = torch.tensor([[last]], device=dev, dtype=torch.int32)
    z = torch.zeros(T, device=dev, dtype=torch.int32)
    slots = torch.arange(T, device=dev, dtype=torch.int32)
    k = to_dev(synth.normal_bf16(411, 5, (T, 1, 128)), dev)
    first = big[0].clone()
    ends = torch.tensor([0, T], device=dev, dtype=torch.int32)
    ex.attn_rope_cache_write_fp8(k, k, k, ends, ends[1:], slots.view(1, T), tbl, big, (64,))
    _, v = ex.attn_cache_read_fp8(big, z, slots, tbl)
    assert (v - k).abs().max() <= 2 ** -4 * k.abs().max() and torch.equal(big[0], first)


def test_decode_outputs_given_no_lse_and_workspace(env):
    torch, ex, dev = env
    q, cache, table, lens = decode_case(412, [6000, 100], 8, 1, 128)
    args = [to_dev(x, dev) for x in (q, cache, table, lens)]
    want, want_lse = ex.attn_decode_paged_fp8(*args)
    need = ex.attn_decode_fp8_workspace_bytes(2, 1, 8, 1, 128, table.shape[1])
    assert need > 0
    guard = torch.full((need + 64,), 0xFF, device=dev, dtype=torch.uint8)  # NaNs where nothing is written
    out = torch.full_like(want, float("nan"))
    got, lse = ex.attn_decode_paged_fp8(*args, out=out, return_lse=False, workspace=guard[:need])
    assert got is out and lse is None and torch.equal(out, want)
    assert (guard[need:] == 0xFF).all()
    four = ex.attn_decode_paged_fp8(args[0][:, None], *args[1:])
    assert four[0].shape == (2, 1, 8, 128) and torch.equal(four[0][:, 0], want) and torch.equal(four[1][:, 0], want_lse)
    with pytest.raises(ex.ExattnError):
        ex.attn_decode_paged_fp8(*args, workspace=guard[:need - 16])
    with pytest.raises(ex.ExattnError):
        ex.attn_decode_paged_fp8(args[0][:, None].expand(2, 17, 8, 128).contiguous(), *args[1:])
    with pytest.raises(ex.ExattnError):
        ex.attn_decode_paged_fp8(args[0][:, None][:, :0], *args[1:])
    with pytest.raises(ValueError):
        ex.attn_decode_paged_fp8(*args, out=out[:1])
    with pytest.raises(ValueError):
        ex.attn_decode_paged_fp8(args[0], args[1], args[2][:1], args[3])
    with pytest.raises(TypeError):
        ex.attn_decode_paged_fp8(args[0], args[1], args[2].long(), args[3])
    with pytest.raises(ValueError):
        ex.attn_decode_paged_fp8(args[0][..., :64].contiguous(), *args[1:])
    with pytest.raises(ValueError):  # the 4-bit cache's spans
        ex.attn_decode_paged_fp8(args[0], ex.attn_fp4_cache(4, 1, 128), *args[2:])
    none = ex.attn_decode_paged_fp8(args[0][:0], args[1], args[2][:0], args[3][:0])
    assert none[0].shape == (0, 8, 128)
    assert torch.equal(ex.attn_decode_paged_fp8(*args)[0], want)


def test_decode_captured_replayed_and_sharing_a_workspace(env):
    """Two graphs over one workspace, replayed in turn with changed contents."""
    torch, ex, dev = env
    q, cache, table, lens = decode_case(413, [5000, 700, 1], 8, 2, 128)
    qd, cd, td, ld = (to_dev(x, dev) for x in (q, cache, table, lens))
    ws = torch.empty(ex.attn_decode_fp8_workspace_bytes(3, 1, 8, 2, 128, table.shape[1]), device=dev, dtype=torch.uint8)
    q2 = qd.flip(0).contiguous()
    want1 = [x.clone() for x in ex.attn_decode_paged_fp8(qd, cd, td, ld)]
    want2 = [x.clone() for x in ex.attn_decode_paged_fp8(q2, cd, td, ld)]
    graphs, results = [], []
    for x in (qd, q2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            results.append(ex.attn_decode_paged_fp8(x, cd, td, ld, workspace=ws))
        graphs.append(g)
    for _ in range(3):
        for g, got, want in zip(graphs, results, (want1, want2)):
            got[0].zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    shorter = np.array([900, 0, 1], np.int32)
    ld.copy_(to_dev(shorter, dev))
    graphs[0].replay()
    torch.cuda.synchronize()
    check_decode(*results[0], q, cache, table, shorter, 128, 128 ** -0.5)
    assert ex.attn_get_device_status() == 0


# ------------------------------------------------------------ append and read
def append_case(seed, held, new, Hq, Hkv, d, axes=1, gain=1.0, room=0):
    """New tokens after held ones: q, k, v, starts, ctx, positions, table, a cache whose
    blocks hold something (scales too)."""
    held, new = np.asarray(held, np.int32), np.asarray(new, np.int32)
    ctx = held + new
    table, nb = synth.paged_layout(np.maximum(ctx, 1) + room, 16, seed)
    starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    T = int(starts[-1])
    slots = np.concatenate([np.arange(h, h + n) for h, n in zip(held, new)]).astype(np.int32)
    if axes == 1:
        pos = slots[None]
    else:
        pos = np.floor(synth.uniform01(seed, axes * T).reshape(axes, T) * 40000 - 100).astype(np.int32)
    q, k, v = (synth.normal_bf16(seed, i, (T, h, d)) for i, h in ((3, Hq), (4, Hkv), (5, Hkv)))
    if gain != 1.0:  # tokens of very different sizes: blocks' scales grow with some of them
        f = gain ** (2 * synth.uniform01(seed + 1, T) - 1).astype(np.float32)
        k, v = (synth.f32_to_bf16_bits(synth.bf16_bits_to_f32(x) * f[:, None, None]) for x in (k, v))
    return dict(q=q, k=k, v=v, starts=starts, ctx=ctx, pos=np.ascontiguousarray(pos), table=table, slots=slots,
                seq=np.repeat(np.arange(len(ctx), dtype=np.int32), new), cache=ref.random_cache(seed, nb, Hkv, d))


def turned_keys(c, sections, base, per_axis):
    """The definition's fp32 operations with correctly rounded cosines and sines."""
    co, si = ref4.cos_sin(c["pos"], sections, base, per_axis)
    return ref4.turn(synth.bf16_bits_to_f32(c["k"]), co.astype(np.float32)[:, None], si.astype(np.float32)[:, None])


def check_cache(after, want, d, label=""):
    """Byte for byte, but for keys next to the border of two codes: a cosine that is one unit
    in the last place off (3 in 10,000 are) moves one of them once in some millions."""
    differ = after != want
    assert differ.sum() <= 2, "%s: %d bytes differ" % (label, differ.sum())
    if differ.any():
        assert not differ[..., 16 * d:].any(), label  # only key codes
        a, b = after[differ].astype(int), want[differ].astype(int)
        assert (np.abs(a - b) == 1).all(), label


def run_append(env, c, Hkv, d, sections, base=10000.0, per_axis=False, no_starts=False):
    torch, ex, dev = env
    cd = to_dev(c["cache"], dev)
    qd, kd, vd, st, ctx, pd, tbl = (to_dev(c[x], dev) for x in ("q", "k", "v", "starts", "ctx", "pos", "table"))
    q_out = ex.attn_rope_cache_write_fp8(qd, kd, vd, None if no_starts else st, ctx, pd, tbl, cd, sections, base=base,
                                         per_axis=per_axis)
    torch.cuda.synchronize()
    assert ex.attn_get_device_status() == 0
    if qd.shape[1] > 0:
        want_q, _ = ex.attn_rope_axes(qd.transpose(0, 1)[None], qd.transpose(0, 1)[None], pd[:, None], sections,
                                      base=base, per_axis=per_axis)
        assert torch.equal(q_out.view(torch.int16), want_q[0].transpose(0, 1).contiguous().view(torch.int16))
    want = c["cache"].copy()
    ref.append(want, d, c["table"], c["starts"], c["ctx"], turned_keys(c, sections, base, per_axis),
               synth.bf16_bits_to_f32(c["v"]))
    after = cd.cpu().numpy()
    check_cache(after, want, d)
    # read back: exactly what the bytes stand for, of all tokens of the sequences
    seq = np.repeat(np.arange(len(c["ctx"])), c["ctx"]).astype(np.int32)
    slots = np.concatenate([np.arange(n) for n in c["ctx"]]).astype(np.int32)
    kr, vr = ex.attn_cache_read_fp8(cd, to_dev(seq, dev), to_dev(slots, dev), tbl)
    held = ref.values(after, d)
    blk = c["table"][seq, slots // 16]
    for got, x in zip((kr, vr), held):
        x = x[blk, :, slots % 16]
        assert np.array_equal(got.double().cpu().numpy(), x, equal_nan=True)
    return cd


SECTIONS = {1: lambda h: (h,), 2: lambda h: (h // 2, h // 2), 3: lambda h: (h // 4, h // 4 + 4, h // 2 - 4),
            4: lambda h: (1, 2, h - 8, 5)}


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("held,new,Hq,Hkv,axes", [
    ([0], [1], 1, 1, 1), ([0, 15, 16, 299], [1, 1, 1, 1], 8, 2, 1), ([7, 0, 30, 5], [33, 3, 40, 28], 4, 4, 3),
    ([167], [333], 14, 2, 3), ([0] * 20, [64] * 20, 4, 1, 2), ([0, 1300], [700, 700], 3, 1, 4),
    ([0] * 3, [2500] * 3, 0, 1, 1), ([3, 100, 0, 9, 31], [0, 5, 0, 0, 2], 2, 3, 1)])
def test_append_bytes_and_read(env, d, held, new, Hq, Hkv, axes):
    c = append_case(500 + sum(new), held, new, Hq, Hkv, d, axes)
    run_append(env, c, Hkv, d, SECTIONS[axes](d // 2))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("gain", [4.0, 2.0 ** 12, 2.0 ** 40])
def test_append_blocks_whose_scale_grows(env, d, gain):
    """Token after token, each of its own size: scales grow by little or by more than fp16
    and e4m3 hold, the codes of the block's other tokens are rounded to them."""
    torch, ex, dev = env
    held, new = [0, 1, 5, 8, 14, 15], [1] * 6
    c = append_case(510, held, new, 2, 2, d, gain=gain, room=12)
    for step in range(12):
        c["cache"] = run_append(env, c, 2, d, (d // 2,), no_starts=step % 2 == 0).cpu().numpy()
        more = append_case(511 + step, c["ctx"], new, 2, 2, d, gain=gain)
        c = dict(more, table=c["table"], cache=c["cache"])


@pytest.mark.parametrize("d", [64, 128])
def test_append_grows_a_block_in_chunks(env, d):
    """The same block written by calls of 3, 1, 7 and 5 tokens, in a table of one block."""
    torch, ex, dev = env
    c = append_case(530, [0], [16], 1, 2, d, gain=2.0 ** 6)
    cache = c["cache"]
    at = 0
    for n in (3, 1, 7, 5):
        part = dict(c, q=c["q"][at:at + n], k=c["k"][at:at + n], v=c["v"][at:at + n], cache=cache,
                    pos=np.ascontiguousarray(c["pos"][:, at:at + n]), starts=np.array([0, n], np.int32),
                    ctx=np.array([at + n], np.int32))
        cache = run_append(env, part, 2, d, (d // 2,)).cpu().numpy()
        at += n


def test_append_a_block_given_to_another_sequence_starts_anew(env):
    """What an earlier owner left, a huge scale and NaN codes, has no part in it."""
    torch, ex, dev = env
    d = 64
    c = append_case(531, [0, 0], [5, 16], 1, 1, d)
    codes, scales = ref.split(c["cache"], d)
    codes[:] = 0x7F
    scales[:] = 2.0 ** 100
    cd = run_append(env, c, 1, d, (32,))
    assert ref.split(cd.cpu().numpy(), d)[1].max() < 2.0
    again = dict(c, cache=cd.cpu().numpy())  # and the same call twice leaves the same bytes
    assert np.array_equal(run_append(env, again, 1, d, (32,)).cpu().numpy(), again["cache"])


def test_append_many_heads_and_long_positions(env):
    run_append(env, append_case(511, [32760, 19992], [8, 8], 128, 16, 128), 16, 128, (64,), base=500000.0)


@pytest.mark.parametrize("S", [255, 256, 257, 700, 4097])
def test_append_many_sequences(env, S):
    """Ragged, most sequences with few tokens and many with none."""
    u = synth.uniform01(540 + S, 2 * S).reshape(2, S)
    new = np.where(u[0] < 0.4, 0, np.floor(u[0] ** 4 * 40)).astype(np.int32)
    new[[0, S // 2, S - 1]] = [0, 60, 3]
    held = np.floor(u[1] * 40).astype(np.int32)
    run_append(env, append_case(541, held, new, 2, 1, 64), 1, 64, (32,))


@pytest.mark.parametrize("held,new,Hq,Hkv,d", [([5, 0], [1100, 1100], 40, 4, 128), ([0] * 4, [1850] * 4, 3, 3, 128),
                                                ([3] * 4, [2600] * 4, 7, 2, 64)])
def test_append_large_calls(env, held, new, Hq, Hkv, d):
    """Ones that take a CTA an SM: with fewer runs than these, and with many."""
    run_append(env, append_case(548, held, new, Hq, Hkv, d), Hkv, d, (d // 2,))


@pytest.mark.parametrize("S", [1, 300, 3000])
def test_append_a_token_for_each_sequence(env, S):
    held = np.floor(synth.uniform01(545, S) * 50).astype(np.int32)
    c = append_case(546, held, np.ones(S, np.int32), 3, 2, 128)
    a = run_append(env, c, 2, 128, (64,))
    b = run_append(env, c, 2, 128, (64,), no_starts=True)
    assert bool((a == b).all())


@pytest.mark.parametrize("per_axis", [False, True])
def test_append_sections(env, per_axis):
    run_append(env, append_case(547, [30, 4], [130, 40], 4, 2, 64, 2), 2, 64, (16, 16), per_axis=per_axis)


def test_append_special_values(env):
    """NaN, infinities, zeros, subnormals and the type's largest value, at position
    0.  There a key is x 1 - y 0: unturned, but an infinity or a NaN makes its
    partner NaN as well.  What is not finite reads as NaN and leaves the others alone."""
    torch, ex, dev = env
    d = 64
    x = torch.randn(4, 1, d, device=dev).bfloat16()
    x[0, 0, 3] = float("nan")
    x[0, 0, 20] = float("inf")
    x[0, 0, 40] = -float("inf")
    x[1, 0, :16] = 0
    x[1, 0, 16:32] = -0.0
    x[3] = -x[3].abs()
    other = x.clone()
    other[2, 0, 5] = torch.finfo(torch.bfloat16).min
    other[2, 0, 6] = torch.finfo(torch.bfloat16).max
    tiny = x * 0 + 1e-39
    tiny[0, 0, 0] = 1e-36
    i = torch.arange(4, device=dev, dtype=torch.int32)
    z = torch.zeros(4, device=dev, dtype=torch.int32)
    ends = torch.tensor([0, 4], device=dev, dtype=torch.int32)
    for t in (x, other, tiny):
        cache = ex.attn_fp8_cache(1, 1, d)
        ex.attn_rope_cache_write_fp8(t, t, t, ends, ends[1:], z.view(1, 4), z[:1].view(1, 1), cache, (32,))
        k, v = ex.attn_cache_read_fp8(cache, z, i, z[:1].view(1, 1))
        f = synth.bf16_bits_to_f32(bits(t))
        with np.errstate(invalid="ignore"):
            turned = ref4.turn(f, np.float32(1.0), np.float32(0.0))
        want = np.zeros((1, 1, 32 * d + 32), np.uint8)
        ref.append(want, d, np.zeros((1, 1), int), [0, 4], [4], turned, f)
        assert np.array_equal(cache.cpu().numpy(), want)
        for got, w, x32 in zip((k, v), ref.values(want, d), (turned, f)):
            got = got.double().cpu().numpy()
            assert np.array_equal(got, w[0, :, :4].transpose(1, 0, 2), equal_nan=True)
            assert np.array_equal(np.isnan(got), ~np.isfinite(x32))
    assert ex.attn_get_device_status() == 0


def test_append_rows_of_no_sequence_are_left_alone(env):
    """A call with room: rows before the first sequence's and behind the last one's."""
    torch, ex, dev = env
    d, Hkv, Hq = 64, 2, 3
    c = append_case(550, [3, 20, 0], [20, 0, 9], Hq, Hkv, d)
    T, lead, room = 29, 4, 40
    wide = {}
    for x, h in (("q", Hq), ("k", Hkv), ("v", Hkv)):
        wide[x] = torch.full((room, h, d), float("nan"), device=dev, dtype=torch.bfloat16)
        wide[x][lead:lead + T] = to_dev(c[x], dev)
    pos = torch.full((1, room), 2 ** 30, device=dev, dtype=torch.int32)
    pos[:, lead:lead + T] = to_dev(c["pos"], dev)
    st, ctx, tbl = to_dev(c["starts"] + lead, dev), to_dev(c["ctx"], dev), to_dev(c["table"], dev)
    a, b = to_dev(c["cache"], dev), to_dev(c["cache"], dev)
    out = torch.full((room, Hq, d), 7.0, device=dev, dtype=torch.bfloat16)
    ex.attn_rope_cache_write_fp8(wide["q"], wide["k"], wide["v"], st, ctx, pos, tbl, a, (32,), q_out=out)
    want = ex.attn_rope_cache_write_fp8(*(to_dev(c[x], dev) for x in ("q", "k", "v", "starts", "ctx", "pos", "table")), b, (32,))
    torch.cuda.synchronize()
    assert ex.attn_get_device_status() == 0
    assert torch.equal(a, b) and torch.equal(out[lead:lead + T], want)
    assert (out[:lead] == 7).all() and (out[lead + T:] == 7).all()


def test_append_outside_the_table_is_flagged(env):
    torch, ex, dev = env
    d, Hkv = 64, 2
    c = append_case(551, [0, 4, 0, 10], [20, 8, 20, 5], 2, Hkv, d)
    table, ctx = c["table"].copy(), c["ctx"].copy()
    table[0, 1] = -1               # sequence 0's second block
    table[2, 0] = len(c["cache"])  # sequence 2's first
    ctx[1] = 3                     # sequence 1's first five of eight before its beginning
    ctx[3] = 16 * table.shape[1] + 2  # sequence 3's last two behind the table
    args = [to_dev(c[x], dev) for x in ("q", "k", "v", "starts")]
    cd = to_dev(c["cache"], dev)
    q = ex.attn_rope_cache_write_fp8(*args, to_dev(ctx, dev), to_dev(c["pos"], dev), to_dev(table, dev), cd, (32,))
    torch.cuda.synchronize()
    assert ex.attn_get_device_status() == 2
    want_q = ex.attn_rope_cache_write_fp8(*args, *(to_dev(c[x], dev) for x in ("ctx", "pos", "table")),
                                          to_dev(c["cache"], dev), (32,))
    assert torch.equal(q, want_q)  # rotated all the same
    want = c["cache"].copy()
    k32, v32 = turned_keys(c, (32,), 500000.0, False), synth.bf16_bits_to_f32(c["v"])

    def put(s, first, n, slot):  # the tokens of one run that has a place
        t = int(c["starts"][s]) + first
        b = slot // 16
        ref.append(want, d, table[s:s + 1, b:b + 1], [0, n], [slot % 16 + n], k32[t:t + n], v32[t:t + n])

    put(0, 0, 16, 0)
    put(1, 5, 3, 0)
    put(2, 16, 4, 16)
    # sequence 3: its first three tokens at the end of its last table entry, if that has a block
    last = table.shape[1] - 1
    if table[3, last] >= 0:
        put(3, 0, 3, 16 * last + 13)
    check_cache(cd.cpu().numpy(), want, d)
    sid = torch.tensor([0, 9, -1, 0, 0], device=dev, dtype=torch.int32)
    sl = torch.tensor([0, 0, 0, -1, 10 ** 6], device=dev, dtype=torch.int32)
    out = [torch.full((5, Hkv, d), 9.0, device=dev, dtype=torch.bfloat16) for _ in range(2)]
    k, v = ex.attn_cache_read_fp8(cd, sid, sl, to_dev(table, dev), k_out=out[0], v_out=out[1])
    torch.cuda.synchronize()
    assert ex.attn_get_device_status() == 2
    assert (k[1:] == 0).all() and (v[1:] == 0).all() and (v[0] != 0).any()


@pytest.mark.parametrize("starts", [[0, 9, 4, 12], [-1, 4, 8, 12], [0, 4, 8, 13], [0, 2 ** 31 - 1, -2 ** 31, 12],
                                    [12, 8, 4, 0]])
def test_append_of_starts_that_make_no_sequences_does_nothing(env, starts):
    torch, ex, dev = env
    d, Hkv = 64, 1
    c = append_case(552, [0, 5, 0], [4, 4, 4], 2, Hkv, d)
    cd = to_dev(c["cache"], dev)
    before = cd.clone()
    out = torch.full((12, 2, d), 7.0, device=dev, dtype=torch.bfloat16)
    args = [to_dev(c[x], dev) for x in ("q", "k", "v", "ctx", "pos", "table")]
    ex.attn_rope_cache_write_fp8(*args[:3], torch.tensor(starts, device=dev, dtype=torch.int64).int(), *args[3:], cd,
                                 (32,), q_out=out)
    torch.cuda.synchronize()
    assert ex.attn_get_device_status() == 2
    assert torch.equal(cd, before) and (out == 7).all()


def test_append_strided_in_place_and_read_into_views(env):
    torch, ex, dev = env
    Hq, Hkv, d = 6, 2, 64
    c = append_case(553, [13], [50], Hq, Hkv, d)
    T = 50
    qkv = torch.empty((T, Hq + 2 * Hkv, d), device=dev, dtype=torch.bfloat16)
    qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:] = (to_dev(c[x], dev) for x in ("q", "k", "v"))
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    st, ctx, pd, tbl = (to_dev(c[x], dev) for x in ("starts", "ctx", "pos", "table"))
    c1, c2 = to_dev(c["cache"], dev), to_dev(c["cache"], dev)
    want = ex.attn_rope_cache_write_fp8(*(to_dev(c[x], dev) for x in ("q", "k", "v")), st, ctx, pd, tbl, c1, (32,))
    kv = qkv[:, Hq:].clone()
    got = ex.attn_rope_cache_write_fp8(q, k, v, st, ctx, pd, tbl, c2, (32,), q_out=q)
    assert got is q and torch.equal(q, want) and torch.equal(c1, c2) and torch.equal(qkv[:, Hq:], kv)
    # the same key and value head for all (stride 0)
    wide_k, wide_v = k[:, :1].expand(-1, Hkv, -1), v[:, :1].expand(-1, Hkv, -1)
    c3, c4 = to_dev(c["cache"], dev), to_dev(c["cache"], dev)
    ex.attn_rope_cache_write_fp8(q, wide_k, wide_v, st, ctx, pd, tbl, c3, (32,))
    ex.attn_rope_cache_write_fp8(q, wide_k.contiguous(), wide_v.contiguous(), st, ctx, pd, tbl, c4, (32,))
    assert torch.equal(c3, c4)
    slots = torch.arange(13 + T, device=dev, dtype=torch.int32)
    idx = [torch.zeros_like(slots), slots]
    kr, vr = ex.attn_cache_read_fp8(c1, *idx, tbl)
    # one sequence into [Hkv, N, d] with room behind it
    n = 13 + T
    room = [torch.full((Hkv, n + 7, d), 5.0, device=dev, dtype=torch.bfloat16) for _ in range(2)]
    ex.attn_cache_read_fp8(c1, *idx, tbl, k_out=room[0][:, :n].transpose(0, 1), v_out=room[1][:, :n].transpose(0, 1))
    for x, w in zip(room, (kr, vr)):
        assert torch.equal(x[:, :n].transpose(0, 1), w) and (x[:, n:] == 5).all()
    with pytest.raises(ex.ExattnError):  # keys and values into the same rows
        ex.attn_cache_read_fp8(c1, *idx, tbl, k_out=kr, v_out=kr)
    with pytest.raises(ValueError):
        ex.attn_rope_cache_write_fp8(q, k[:-1], v, st, ctx, pd, tbl, c2, (32,))
    with pytest.raises(ValueError):
        ex.attn_rope_cache_write_fp8(q, k, v, st[:-1], ctx, pd, tbl, c2, (32,))
    with pytest.raises(ValueError):
        ex.attn_rope_cache_write_fp8(q, k, v, None, ctx, pd, tbl, c2, (32,))
    with pytest.raises(ValueError):
        ex.attn_rope_cache_write_fp8(q, k, v, st, ctx, pd[:, :-1].contiguous(), tbl, c2, (32,))
    with pytest.raises(ValueError):
        ex.attn_rope_cache_write_fp8(q, k, v, st, ctx, pd, tbl, c2, (16, 16))
    with pytest.raises(TypeError):
        ex.attn_rope_cache_write_fp8(q, k, v, st.long(), ctx, pd, tbl, c2, (32,))
    with pytest.raises(ValueError):
        ex.attn_rope_cache_write_fp8(q, k, v, st, ctx, pd, tbl, ex.attn_fp4_cache(4, Hkv, d), (32,))
    ex.attn_rope_cache_write_fp8(q[:0], k[:0], v[:0], st * 0, ctx, pd[:, :0].contiguous(), tbl, c2, (32,))
    assert ex.attn_cache_read_fp8(c2, *(x[:0] for x in idx), tbl)[0].shape == (0, Hkv, d)
    assert torch.equal(c1, c2)
    assert ex.attn_get_device_status() == 0


@pytest.mark.parametrize("d", [64, 128])
def test_read_onto_every_16_byte_boundary(env, d):
    """Rows on 16-byte boundaries that are not 32-byte ones, or on both kinds in turn, and
    nothing written between them."""
    torch, ex, dev = env
    T, Hkv = 37, 3
    cache = to_dev(ref.random_cache(554, 3, Hkv, d), dev)
    idx = [torch.zeros(T, device=dev, dtype=torch.int32), torch.arange(T, device=dev, dtype=torch.int32)]
    tbl = torch.tensor([[2, 0, 1]], device=dev, dtype=torch.int32)
    want = ex.attn_cache_read_fp8(cache, *idx, tbl)
    for gap, start in ((0, 8), (8, 0), (8, 8), (16, 8)):
        room = torch.full((2, T * Hkv * (d + gap) + 32), 5.0, device=dev, dtype=torch.bfloat16)
        outs = [x[start:start + T * Hkv * (d + gap)].view(T, Hkv, d + gap) for x in room]
        ex.attn_cache_read_fp8(cache, *idx, tbl, k_out=outs[0][..., :d], v_out=outs[1][..., :d])
        for x, w in zip(outs, want):
            assert torch.equal(x[..., :d], w) and (x[..., d:] == 5).all()
        assert (room[:, :start] == 5).all() and (room[:, start + T * Hkv * (d + gap):] == 5).all()


def test_read_any_order(env):
    """Tokens in any order, some of them several times."""
    torch, ex, dev = env
    cache = ref.random_cache(555, 40, 2, 128, v_exp=30)
    table = np.arange(40, dtype=np.int32)[::-1].reshape(2, 20).copy()
    u = synth.uniform01(556, 2 * 1000).reshape(2, 1000)
    seq, slots = np.floor(u[0] * 2).astype(np.int32), np.floor(u[1] * 320).astype(np.int32)
    got = ex.attn_cache_read_fp8(*(to_dev(x, dev) for x in (cache, seq, slots, table)))
    for g, x in zip(got, ref.values(cache, 128)):
        assert np.array_equal(g.double().cpu().numpy(), x[table[seq, slots // 16], :, slots % 16])


# ------------------------------------------------------------------- together
@pytest.mark.parametrize("d", [64, 128])
def test_serving_run(env, d):
    """Prompts are appended, then tokens one by one and drafts three by three, each
    attended to; the last step and a chunk's prefill over the read-back prefix agree with the
    64-bit attention over what the cache stands for."""
    torch, ex, dev = env
    S, Hq, Hkv, steps = 3, 8, 2, 4
    half = d // 2
    sections = (half // 2, half // 4, half // 4)
    lens = np.array([37, 16, 90], np.int32)
    table, nb = synth.paged_layout(lens + steps + 3, 16, 9)
    cache, td = ex.attn_fp8_cache(nb, Hkv, d), to_dev(table, dev)

    def step(new, seed, with_starts):
        nonlocal lens
        starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        slots = np.concatenate([np.arange(n, n + m) for n, m in zip(lens, new)]).astype(np.int32)
        lens = (lens + new).astype(np.int32)
        T = len(slots)
        q, k, v = (to_dev(synth.normal_bf16(seed, i, (T, h, d)), dev) for i, h in ((1, Hq), (2, Hkv), (3, Hkv)))
        pos = to_dev(np.stack([slots, slots // 7, slots % 7]), dev)
        ld = to_dev(lens, dev)
        return ex.attn_rope_cache_write_fp8(q, k, v, to_dev(starts, dev) if with_starts else None, ld, pos, td, cache,
                                            sections), ld

    first, lens = lens, np.zeros(S, np.int32)
    step(first, 600, True)
    for i in range(steps):
        qr, ld = step(np.ones(S, np.int32), 601 + i, False)
        out, lse = ex.attn_decode_paged_fp8(qr, cache, td, ld)
    check_decode(out, lse, bits(qr), cache.cpu().numpy(), table, lens, d, d ** -0.5)
    # the same token as a chunk of one over the prefix, through attn_fwd
    for s in range(S):
        n = int(lens[s])
        kk = torch.empty((1, Hkv, n, d), device=dev, dtype=torch.bfloat16)
        vv = torch.empty_like(kk)
        i = torch.arange(n, device=dev, dtype=torch.int32)
        ex.attn_cache_read_fp8(cache, torch.full_like(i, s), i, td, k_out=kk[0].transpose(0, 1), v_out=vv[0].transpose(0, 1))
        o, l2 = ex.attn_fwd(qr[s].view(1, Hq, 1, d), kk, vv, causal=True)
        # both within 2^-8 |o| (the prefill's weights round by 2^-9 as well)
        assert (o.view(Hq, d).float() - out[s].float()).abs().max() < 5e-2
        assert (l2.view(Hq) - lse[s]).abs().max() < 1e-3
    qr, ld = step(np.full(S, 3, np.int32), 650, True)
    qr = qr.view(S, 3, Hq, d)
    out, lse = ex.attn_decode_paged_fp8(qr, cache, td, ld)
    torch.cuda.synchronize()
    assert ex.attn_get_device_status() == 0
    check_decode(out, lse, bits(qr), cache.cpu().numpy(), table, lens, d, d ** -0.5)


def test_captured_step_follows_lengths_and_starts(env):
    """Append and decode in one graph, replayed as the contexts grow; then with other
    numbers of new tokens in the same room."""
    torch, ex, dev = env
    d, Hq, Hkv, S, room = 64, 4, 2, 3, 12
    lens = np.array([14, 40, 3], np.int32)
    table, nb = synth.paged_layout(lens + 30, 16, 11)
    td = to_dev(table, dev)
    start_cache = ref.random_cache(660, nb, Hkv, d)
    cache, twin = to_dev(start_cache, dev), to_dev(start_cache, dev)
    q, k, v = (torch.zeros((room, h, d), device=dev, dtype=torch.bfloat16) for h in (Hq, Hkv, Hkv))
    pos = torch.zeros((1, room), device=dev, dtype=torch.int32)
    starts = torch.zeros(S + 1, device=dev, dtype=torch.int32)
    ctx = to_dev(lens, dev)
    last = torch.zeros(S, device=dev, dtype=torch.int64)

    def once(cache):
        qr = ex.attn_rope_cache_write_fp8(q, k, v, starts, ctx, pos, td, cache, (32,), q_out=torch.empty_like(q))
        return ex.attn_decode_paged_fp8(qr[last], cache, td, ctx)

    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        once(to_dev(start_cache, dev))
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = once(cache)
    for i, new in enumerate(([1, 1, 1], [1, 1, 1], [5, 1, 6], [2, 0, 7], [0, 0, 0])):
        new = np.array(new, np.int32)
        lens = lens + new
        starts.copy_(to_dev(np.concatenate([[0], np.cumsum(new)]).astype(np.int32), dev))
        ctx.copy_(to_dev(lens.astype(np.int32), dev))
        last.copy_((starts[1:] - 1).clamp(min=0).long())
        for x, h, j in ((q, Hq, 0), (k, Hkv, 1), (v, Hkv, 2)):
            x.copy_(to_dev(synth.normal_bf16(661 + i, j, (room, h, d)), dev))
        pos.copy_(torch.arange(room, device=dev, dtype=torch.int32)[None] + i)
        graph.replay()
        want = once(twin)
        torch.cuda.synchronize()
        assert torch.equal(cache, twin)
        assert torch.equal(got[1], want[1]) or (new == 0).any()
        seen = torch.from_numpy(new > 0).to(dev)
        assert torch.equal(got[0][seen], want[0][seen])
    assert ex.attn_get_device_status() == 0


def test_threads_and_streams(env):
    """Four threads on streams of their own, each appending, reading and decoding
    on a cache of its own; every result equals the single thread's."""
    import threading
    torch, ex, dev = env
    d, Hq, Hkv = 64, 8, 2

    def work(i, stream):
        with torch.cuda.stream(stream):
            c = append_case(670 + i, [0, 3], [60 + 9 * i, 30], Hq, Hkv, d)
            t = [to_dev(c[x], dev) for x in ("q", "k", "v", "starts", "ctx", "pos", "table")]
            seq, slots = to_dev(c["seq"], dev), to_dev(c["slots"], dev)
            res = []
            for _ in range(10):
                cache = to_dev(c["cache"], dev)
                q = ex.attn_rope_cache_write_fp8(*t, cache, (32,), stream=stream)
                k, v = ex.attn_cache_read_fp8(cache, seq, slots, t[6], stream=stream)
                out, lse = ex.attn_decode_paged_fp8(q[[0, -1]].contiguous(), cache, t[6], t[4], stream=stream)
                res = [q, k, v, out, lse]
            stream.synchronize()
        return [x.clone() for x in res]

    want = [work(i, torch.cuda.current_stream()) for i in range(4)]
    got, errors = [None] * 4, []

    def body(i):
        try:
            torch.cuda.set_device(dev)
            got[i] = work(i, torch.cuda.Stream())
        except Exception as e:  # reported below
            errors.append(repr(e))

    threads = [threading.Thread(target=body, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    torch.cuda.synchronize()
    assert ex.attn_get_device_status() == 0
    for a, b in zip(got, want):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


# ------------------------------------- memory of calls on another stream
def decode_call(torch, ex, dev):
    q, cache, table, lens = decode_case(640, [20000, 3], 8, 1, 128)
    args = [to_dev(x, dev) for x in (q, cache, table, lens)]
    sizes = [ex.attn_decode_fp8_workspace_bytes(2, 1, 8, 1, 128, table.shape[1]), q.size * 2, 2 * 8 * 4]
    assert sizes[0] > 0
    return sizes, lambda stream: ex.attn_decode_paged_fp8(*args, stream=stream)


def append_call(torch, ex, dev):
    c = append_case(641, [0], [640], 2, 2, 64)
    args = [to_dev(c[x], dev) for x in ("q", "k", "v", "starts", "ctx", "pos", "table", "cache")]
    return [c["q"].size * 2], lambda stream: [ex.attn_rope_cache_write_fp8(*args, (32,), stream=stream)]


def read_call(torch, ex, dev):
    cache = to_dev(ref.random_cache(642, 40, 2, 64), dev)
    at = torch.arange(640, device=dev, dtype=torch.int32)
    seq, table = torch.zeros_like(at), torch.arange(40, device=dev, dtype=torch.int32)[None]
    return [640 * 2 * 64 * 2] * 2, lambda stream: ex.attn_cache_read_fp8(cache, seq, at, table, stream=stream)


@pytest.mark.parametrize("make", [decode_call, append_call, read_call])
def test_memory_of_calls_on_another_stream(env, make):
    """What a call on another stream allocates is not a block whose last use on the current
    stream is still to come, and is not handed out before the current stream has used it."""
    torch, ex, dev = env
    sizes, call = make(torch, ex, dev)
    main, side = torch.cuda.current_stream(), torch.cuda.Stream()
    want = [x.clone() for x in call(None)]
    side.wait_stream(main)
    call(side)
    torch.cuda.synchronize()
    for _ in range(3):
        held = [torch.full((n,), 7, device=dev, dtype=torch.uint8) for n in sizes]
        copies = [torch.zeros_like(t) for t in held]
        side.wait_stream(main)
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)  # some 10 ms
        for t, c in zip(held, copies):
            c.copy_(t)
        del held, t
        got = call(side)
        side.synchronize()
        torch.cuda.synchronize()
        assert all(bool((c == 7).all()) for c in copies)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    for _ in range(3):
        got = call(side)
        main.wait_stream(side)
        torch.cuda._sleep(20_000_000)
        copies = [x.clone() for x in got]
        del got
        for stream in (side, main):
            with torch.cuda.stream(stream):
                for n in sizes + sizes:
                    torch.full((n,), 0xFF, device=dev, dtype=torch.uint8)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(copies, want))
