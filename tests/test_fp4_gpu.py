"""The 4-bit paged cache on the GPU: append, read and decode against the plain
implementations of fp4_reference.py.

Decode bar, from the arithmetic: scores are fp32 sums of exact products, the
exponentials are good to 2^-21, each weight rounds to fp16, in numerator and
denominator: by 2^-11 relative, or by half the smallest subnormal, 2^-25, where
the largest weight is at least 1.  The latter does not shrink with the weight,
so n tokens add up to n 2^-25 max|v|, also in a column whose weighted mean is
tiny because the token that dominates is 0 there.  The output rounds to bf16
(2^-8):
|o - ref| <= 2^-8 |ref| + (2^-10 + 2^-17 max|s|) mean|v| + n 2^-24 max|v|,
|lse - ref| <= 2^-20 (1 + max|s|) + 2^-20 |ref|."""
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


# ------------------------------------------------------------------- decode
def decode_case(seed, lens, Hq, Hkv, d, k_scale=1.0, v_scale=1.0, gain=1.0, extra_blocks=0, poison=True):
    """q, cache, table, lens; slots past a sequence's last token hold NaN scales."""
    lens = np.asarray(lens, np.int32)
    table, nb = synth.paged_layout(lens, 16, seed, extra_blocks)
    cache = ref.random_cache(seed, nb, Hkv, d, k_scale, v_scale, gain)
    if poison:
        ck, cv, sk, sv = ref.split(cache, d)
        for s, n in enumerate(lens):
            if n % 16:
                b = table[s, n // 16]
                for view in (ck, cv, sk, sv):
                    view[b, :, n % 16:] = 0x7F
    q = synth.normal_bf16(seed, 0, (len(lens), Hq, d))
    return q, cache, table, lens


def check_decode(out, lse, q, cache, table, lens, d, scale, k_scale, v_scale, label=""):
    want, wl, big, mean, most = ref.decode(q, cache, table, lens, d, scale, k_scale, v_scale)
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    n = np.asarray(lens, np.float64)[:, None, None]
    bar = 2.0 ** -8 * np.abs(want) + (2.0 ** -10 + 2.0 ** -17 * big[..., None]) * mean + n * 2.0 ** -24 * most
    assert np.isfinite(got).all(), label
    err = np.abs(got - want)
    assert (err <= bar).all(), "%s: out off by %.3e over the bar" % (label, (err - bar).max())
    empty = np.isneginf(wl)
    assert np.array_equal(np.isneginf(gl), empty), label
    assert (got[empty] == 0).all(), label
    le = np.abs(gl[~empty] - wl[~empty])
    assert (le <= 2.0 ** -20 * (1 + big + np.abs(wl))[~empty]).all(), "%s: lse off by %.3e" % (label, le.max())


def run_decode(env, case, d, scale=None, k_scale=1.0, v_scale=1.0, status=0, label=""):
    torch, ex, dev = env
    q, cache, table, lens = case
    scale = d ** -0.5 if scale is None else scale
    out, lse = ex.attn_decode_paged_fp4(to_dev(q, dev), to_dev(cache, dev), to_dev(table, dev), to_dev(lens, dev),
                                        scale=scale, k_scale=k_scale, v_scale=v_scale)
    torch.cuda.synchronize()
    assert ex.attn_get_device_status() == status
    check_decode(out, lse, q, cache, table, lens, d, scale, k_scale, v_scale, label)
    return out, lse


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", [[0], [1], [15, 16, 17], [0, 33, 128, 129, 640, 1], [3000, 5], [70000, 0, 777]],
                         ids=lambda x: "-".join(map(str, x)))
def test_decode_lengths(env, d, lens):
    run_decode(env, decode_case(400, lens, 4, 1, d), d)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (8, 2), (7, 1), (16, 2), (9, 1), (16, 1), (34, 2), (40, 1)])
def test_decode_head_layouts(env, d, Hq, Hkv):
    run_decode(env, decode_case(401, [200, 1, 47], Hq, Hkv, d, k_scale=0.5, v_scale=0.01), d, k_scale=0.5, v_scale=0.01)


@pytest.mark.parametrize("S,Hq,Hkv,hi", [(40, 4, 2, 5000), (160, 8, 4, 600), (700, 2, 1, 40), (130, 24, 2, 300),
                                         (129, 2, 1, 3000), (400, 3, 1, 1500), (1100, 4, 2, 280), (2100, 1, 1, 200)])
def test_decode_many_sequences(env, S, Hq, Hkv, hi):
    """Ragged batches, empty sequences among them: shares that end inside sequences,
    shares of many sequences, more segments than CTAs, and no segment of two units."""
    lens = np.floor(synth.uniform01(70 + S, S) ** 2 * (hi + 1)).astype(np.int32)
    lens[[0, S // 2, S - 1]] = 0
    lens[1] = hi
    run_decode(env, decode_case(420, lens, Hq, Hkv, 64), 64)


@pytest.mark.parametrize("blocks", [8, 9, 64, 255, 256, 257, 264])
@pytest.mark.parametrize("Hq,Hkv", [(3, 1), (20, 2)])
def test_decode_around_the_limits_of_a_small_call(env, blocks, Hq, Hkv):
    """Lengths at which a sequence gets a second unit, fills the cluster's shares and
    passes from the cluster to shares of the whole batch."""
    n = blocks * 16
    run_decode(env, decode_case(421, [n, n - 15, 1, 0, max(1, n - 128)], Hq, Hkv, 128), 128)


def test_decode_serving_batch(env):
    lens = synth.ctx_lengths(5, 24, 512, 8192)
    run_decode(env, decode_case(402, lens, 8, 2, 128, k_scale=0.003, v_scale=0.002), 128, k_scale=0.003, v_scale=0.002)


@pytest.mark.parametrize("gain", [30.0, 1e-3])
def test_decode_peaked_and_flat_scores(env, gain):
    run_decode(env, decode_case(403, [900, 31], 4, 2, 128, k_scale=0.03 * gain, gain=gain), 128, k_scale=0.03 * gain)


@pytest.mark.parametrize("d", [64, 128])
def test_decode_scores_that_keep_growing(env, d):
    """Keys whose scores rise by up to some thousands along the sequence: every
    block moves the running maximum."""
    torch, ex, dev = env
    q, cache, table, lens = decode_case(404, [400], 2, 1, d, poison=False)
    ck, cv, sk, sv = ref.split(cache, d)
    for tok in range(400):
        b = table[0, tok // 16]
        ck[b, :, tok % 16] = ref.pack(np.where(synth.bf16_bits_to_f32(q[0, 0]) >= 0, 2, 10).astype(np.uint8))
        sk[b, :, tok % 16] = 8 + tok // 4
    run_decode(env, (q, cache, table, lens), d, scale=1.0)


def test_decode_queries_of_any_size(env):
    """Queries are scaled by powers of two on their way into fp16: tiny, huge and
    mixed rows lose nothing that the result could show."""
    q, cache, table, lens = decode_case(405, [100, 60], 8, 2, 128)
    f = synth.bf16_bits_to_f32(q)
    f[0, 0] *= 2.0 ** -100
    f[0, 1] *= 2.0 ** -130      # bf16 subnormals
    f[0, 2] = 0
    f[0, 3] *= 2.0 ** 12
    f[0, 4, ::2] *= 2.0 ** -20  # elements far below the row's largest
    f[0, 5, :] = 0
    f[0, 5, 7] = 1.0
    run_decode(env, (synth.f32_to_bf16_bits(f), cache, table, lens), 128, scale=2.0 ** -9)
    f[:] = synth.bf16_bits_to_f32(synth.normal_bf16(406, 0, f.shape)) * np.float32(2.0 ** 100)
    run_decode(env, (synth.f32_to_bf16_bits(f), cache, table, lens), 128, scale=2.0 ** -103)


def test_decode_infinite_queries_and_nan_scales_give_nan_in_their_rows_only(env):
    torch, ex, dev = env
    q, cache, table, lens = decode_case(407, [50, 50], 4, 2, 64)
    qd, cd, td, ld = (to_dev(x, dev) for x in (q, cache, table, lens))
    clean, clean_lse = ex.attn_decode_paged_fp4(qd, cd, td, ld)
    qd[0, 1, 3] = float("nan")
    got, lse = ex.attn_decode_paged_fp4(qd, cd, td, ld)
    assert torch.isnan(got[0, 1]).all() and torch.isnan(lse[0, 1])
    keep = torch.ones((2, 4), dtype=torch.bool, device=dev)
    keep[0, 1] = False
    assert torch.equal(got[keep], clean[keep]) and torch.equal(lse[keep], clean_lse[keep])
    qd = to_dev(q, dev)
    ref.split(cache, 64)[3][table[1, 2], 1, 4, 2] = 0x7F  # a value group of sequence 1's token 36, head 1
    got, lse = ex.attn_decode_paged_fp4(qd, to_dev(cache, dev), td, ld)
    assert torch.isnan(got[1, 2:, 32:48]).all()
    assert torch.equal(got[1, 2:, :32], clean[1, 2:, :32]) and torch.equal(got[1, 2:, 48:], clean[1, 2:, 48:])
    assert torch.equal(got[0], clean[0]) and torch.equal(got[1, :2], clean[1, :2])
    assert torch.equal(lse, clean_lse)
    ex.attn_get_device_status()


def test_decode_bad_table_entries_and_lengths_are_flagged(env):
    torch, ex, dev = env
    q, cache, table, lens = decode_case(408, [300, 40, 16], 4, 1, 128)
    table = table.copy()
    table[0, 3] = -1
    table[0, 7] = cache.shape[0]
    table[2, 0] = 2 ** 31 - 1  # all that sequence 2 has
    run_decode(env, (q, cache, table, lens), 128, status=2, label="bad entries")
    out, lse = ex.attn_decode_paged_fp4(to_dev(q, dev), to_dev(cache, dev), to_dev(table, dev),
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


def test_decode_cache_past_32_bits(env):
    """A pool of more than 4 GiB whose used blocks lie at its end."""
    torch, ex, dev = env
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GiB")
    q, cache, table, lens = decode_case(411, [500, 130], 4, 1, 128)
    nb = 2_000_000  # x 2304 bytes = 4.6 GB
    big = torch.zeros((nb, 1, 2304), device=dev, dtype=torch.uint8)
    big[nb - cache.shape[0]:] = to_dev(cache, dev)
    moved = np.where(table >= 0, table + nb - cache.shape[0], -1).astype(np.int32)
    out, lse = ex.attn_decode_paged_fp4(to_dev(q, dev), big, to_dev(moved, dev), to_dev(lens, dev))
    torch.cuda.synchronize()
    assert ex.attn_get_device_status() == 0
    check_decode(out, lse, q, cache, table, lens, 128, 128 ** -0.5, 1.0, 1.0)
    # append to and read from the far end
    T, last = 3, nb - 1
    tbl = torch.tensor([[last]], device=dev, dtype=torch.int32)
    z = torch.zeros(T, device=dev, dtype=torch.int32)
    slots = torch.arange(T, device=dev, dtype=torch.int32)
    k = to_dev(synth.normal_bf16(411, 5, (T, 1, 128)), dev)
    first = big[0].clone()
    ex.attn_rope_cache_write_fp4(k, k, k, z, slots, slots.view(1, T), tbl, big, (64,))
    _, v = ex.attn_cache_read_fp4(big, z, slots, tbl)
    assert (v - k).abs().max() < 1.0 and torch.equal(big[0], first)


def test_decode_outputs_given_no_lse_and_workspace(env):
    torch, ex, dev = env
    q, cache, table, lens = decode_case(412, [6000, 100], 8, 1, 128)
    args = [to_dev(x, dev) for x in (q, cache, table, lens)]
    want, want_lse = ex.attn_decode_paged_fp4(*args)
    need = ex.attn_decode_fp4_workspace_bytes(2, 8, 1, 128, table.shape[1])
    assert need > 0
    guard = torch.full((need + 64,), 0xFF, device=dev, dtype=torch.uint8)  # NaNs where nothing is written
    out = torch.full_like(want, float("nan"))
    got, lse = ex.attn_decode_paged_fp4(*args, out=out, return_lse=False, workspace=guard[:need])
    assert got is out and lse is None and torch.equal(out, want)
    assert (guard[need:] == 0xFF).all()
    with pytest.raises(ex.ExattnError):
        ex.attn_decode_paged_fp4(*args, workspace=guard[:need - 16])
    with pytest.raises(ValueError):
        ex.attn_decode_paged_fp4(*args, out=out[:1])
    with pytest.raises(ValueError):
        ex.attn_decode_paged_fp4(args[0], args[1], args[2][:1], args[3])
    with pytest.raises(TypeError):
        ex.attn_decode_paged_fp4(args[0], args[1], args[2].long(), args[3])
    with pytest.raises(ValueError):
        ex.attn_decode_paged_fp4(args[0][..., :64].contiguous(), *args[1:])
    none = ex.attn_decode_paged_fp4(args[0][:0], args[1], args[2][:0], args[3][:0])
    assert none[0].shape == (0, 8, 128)
    assert torch.equal(ex.attn_decode_paged_fp4(*args)[0], want)


def test_decode_captured_replayed_and_sharing_a_workspace(env):
    """Two graphs over one workspace, replayed in turn with changed contents."""
    torch, ex, dev = env
    q, cache, table, lens = decode_case(413, [5000, 700, 1], 8, 2, 128)
    qd, cd, td, ld = (to_dev(x, dev) for x in (q, cache, table, lens))
    ws = torch.empty(ex.attn_decode_fp4_workspace_bytes(3, 8, 2, 128, table.shape[1]), device=dev, dtype=torch.uint8)
    q2 = qd.flip(0).contiguous()
    want1 = [x.clone() for x in ex.attn_decode_paged_fp4(qd, cd, td, ld)]
    want2 = [x.clone() for x in ex.attn_decode_paged_fp4(q2, cd, td, ld)]
    graphs, results = [], []
    for x in (qd, q2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            results.append(ex.attn_decode_paged_fp4(x, cd, td, ld, workspace=ws))
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
    check_decode(*results[0], q, cache, table, shorter, 128, 128 ** -0.5, 1.0, 1.0)
    assert ex.attn_get_device_status() == 0


# ------------------------------------------------------------ append and read
def append_case(seed, lens, new, Hq, Hkv, d, axes=1):
    inp = synth.rope_inputs_lens(seed, lens, new, Hq, Hkv, d)
    T = inp["positions"].shape[0]
    slots = inp["positions"]
    if axes == 1:
        pos = slots[None]
    else:
        u = synth.uniform01(seed, axes * T).reshape(axes, T)
        pos = np.floor(u * 40000 - 100).astype(np.int32)
    return inp, slots, np.ascontiguousarray(pos)


def expected_bytes(inp, slots, pos, sections, base, per_axis, k_scale, v_scale, d):
    """Codes and scales of every token: the definition's fp32 operations with
    correctly rounded cosines and sines."""
    c, s = ref.cos_sin(pos, sections, base, per_axis)
    c, s = c.astype(np.float32)[:, None], s.astype(np.float32)[:, None]
    k = ref.turn(synth.bf16_bits_to_f32(inp["k"]), c, s)
    return k, ref.quantise(k, k_scale), ref.quantise(synth.bf16_bits_to_f32(inp["v"]), v_scale)


def run_append(env, seed, lens, new, Hq, Hkv, d, sections, base=10000.0, per_axis=False, k_scale=1.0, v_scale=1.0):
    torch, ex, dev = env
    inp, slots, pos = append_case(seed, lens, new, Hq, Hkv, d, len(sections))
    nb = inp["num_blocks"]
    before = synth.splitmix64(seed, nb * Hkv * 18 * d // 8).view(np.uint8).reshape(nb, Hkv, 18 * d).copy()
    cd = to_dev(before, dev)
    tensors = [to_dev(inp[x], dev) for x in ("q", "k", "v", "seq_ids")] + [to_dev(x, dev) for x in (slots, pos, inp["block_table"])]
    qd, kd, vd, sid, sl, pd, tbl = tensors
    q_out = ex.attn_rope_cache_write_fp4(qd, kd, vd, sid, sl, pd, tbl, cd, sections, base=base, per_axis=per_axis,
                                         k_scale=k_scale, v_scale=v_scale)
    torch.cuda.synchronize()
    assert ex.attn_get_device_status() == 0
    # q as attn_rope_axes turns it
    want_q, _ = ex.attn_rope_axes(qd.transpose(0, 1)[None], qd.transpose(0, 1)[None], pd[:, None], sections, base=base,
                                  per_axis=per_axis)
    assert torch.equal(q_out.view(torch.int16), want_q[0].transpose(0, 1).contiguous().view(torch.int16))
    after = cd.cpu().numpy()
    k32, (ck, sk), (cv, sv) = expected_bytes(inp, slots, pos, sections, base, per_axis, k_scale, v_scale, d)
    blk = inp["block_table"][inp["seq_ids"], slots // 16]
    off = slots % 16
    views = ref.split(after, d)
    got = [v[blk, :, off] for v in views]
    assert np.array_equal(got[1], ref.pack(cv)), "value codes"
    assert np.array_equal(got[3], sv), "value scales"
    # keys: a cosine that is one unit in the last place off (3 in 10,000 are) moves a
    # key across a border between two codes once in ten million; what moved lies on it
    bad_scale = got[2] != sk
    assert bad_scale.sum() <= 1
    diff = (ref.unpack(got[0]) != ck) & ~np.repeat(bad_scale, 16, -1)
    assert diff.sum() <= 1
    if diff.any():
        div = np.repeat(ref.E4M3[sk].astype(np.float32) * np.float32(k_scale), 16, -1)
        y = np.abs(k32[diff] / div[diff])
        assert (np.abs(y[:, None] - ref.TIES).min(-1) <= 1e-6 * np.maximum(y, 1)).all()
    # the other slots keep their bytes
    b2 = before.copy()
    for v, g in zip(ref.split(b2, d), got):
        v[blk, :, off] = g
    assert np.array_equal(after, b2), "a slot no token maps to changed"
    # read back: exactly what the bytes stand for
    kr, vr = ex.attn_cache_read_fp4(cd, sid, sl, tbl, k_scale=k_scale, v_scale=v_scale)
    for out, codes, s8, g in ((kr, got[0], got[2], k_scale), (vr, got[1], got[3], v_scale)):
        want = ref.values(ref.unpack(codes), s8, g)
        assert np.array_equal(out.float().cpu().numpy().view(np.uint32) & 0x7FFFFFFF,
                              torch.from_numpy(want).float().bfloat16().float().numpy().view(np.uint32) & 0x7FFFFFFF)
    return cd


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,new,Hq,Hkv,axes", [
    ([1], 1, 1, 1, 1), ([1, 16, 17, 300], 1, 8, 2, 1), ([40, 3, 70, 33], 40, 4, 4, 3), ([500], 333, 14, 2, 3),
    ([64] * 20, 64, 4, 1, 2), ([2000, 700], 700, 3, 1, 4),
    ([2500] * 3, 2500, 0, 1, 1)])
def test_append_bytes_and_read(env, d, lens, new, Hq, Hkv, axes):
    half = d // 2
    sections = {1: (half,), 2: (half // 2, half // 2), 3: (half // 4, half // 4 + 4, half // 2 - 4),
                4: (1, 2, half - 8, 5)}[axes]
    run_append(env, 500 + new, lens, new, Hq, Hkv, d, sections)


@pytest.mark.parametrize("k_scale,v_scale,per_axis", [(0.0089, 0.0023, True), (2.0 ** -7, 2.0 ** -9, False), (100.0, 3e-8, False)])
def test_append_scales(env, k_scale, v_scale, per_axis):
    """Scales of a calibration, and ones under which groups round to zero or saturate."""
    run_append(env, 510, [130, 40], 130, 4, 2, 64, (16, 16), per_axis=per_axis, k_scale=k_scale, v_scale=v_scale)


def test_append_many_heads_and_long_positions(env):
    run_append(env, 511, [32768, 20000], 8, 128, 16, 128, (64,), base=500000.0)


def test_append_rounds_products_before_their_difference(env):
    """Keys whose two products nearly cancel: what is left is 2^-9 of a product, so a
    product that was not rounded to fp32 (a fused multiply-add) shows up as
    2^-15 of the key.  With the oracle's own products fused that way 36 codes and
    scales of these move; a cosine one unit off does it to 3 in 10,000 of those."""
    torch, ex, dev = env
    T, Hkv, d = 2048, 4, 128
    half = d // 2
    pos = np.arange(1, T + 1, dtype=np.int32)[None]
    c, s = ref.cos_sin(pos, (half,), 10000.0, False)
    a = synth.bf16_bits_to_f32(synth.normal_bf16(570, 1, (T, Hkv, half)))
    b = np.where(np.abs(s[:, None]) > 0.01, a * c[:, None] / s[:, None], a)
    k = synth.f32_to_bf16_bits(np.concatenate([a, b], -1).astype(np.float32))
    k32 = ref.turn(synth.bf16_bits_to_f32(k), c.astype(np.float32)[:, None], s.astype(np.float32)[:, None])
    codes, s8 = ref.quantise(k32, 1e-4)
    kd = to_dev(k, dev)
    z = torch.zeros(T, device=dev, dtype=torch.int32)
    at = torch.arange(T, device=dev, dtype=torch.int32)
    tbl = torch.arange(T // 16, device=dev, dtype=torch.int32).view(1, -1)
    cache = ex.attn_fp4_cache(T // 16, Hkv, d)
    ex.attn_rope_cache_write_fp4(kd, kd, kd, z, at, to_dev(pos, dev), tbl, cache, (half,), base=10000.0, k_scale=1e-4)
    got = ref.split(cache.cpu().numpy(), d)
    got_codes = got[0].transpose(0, 2, 1, 3).reshape(T, Hkv, -1)
    got_s8 = got[2].transpose(0, 2, 1, 3).reshape(T, Hkv, -1)
    low = slice(0, half // 16)  # the low halves hold the differences
    wrong = (got_s8 != s8)[..., low].sum() + (ref.unpack(got_codes) != codes)[..., :half].sum()
    assert wrong <= 3, wrong


def test_append_special_values(env):
    """NaN, infinities, zeros, subnormals and the type's largest value, at position
    0.  There a key is x 1 - y 0: unturned, but an infinity or a NaN makes its
    partner NaN as well."""
    torch, ex, dev = env
    d = 64
    x = torch.randn(4, 1, d, device=dev).bfloat16()
    x[0, 0, 3] = float("nan")
    x[0, 0, 20] = float("inf")
    x[0, 0, 40] = -float("inf")
    x[1, 0, :16] = 0
    x[1, 0, 16:32] = 1e-40
    x[1, 0, 32:48] = torch.finfo(torch.bfloat16).max
    x[2, 0, 5] = torch.finfo(torch.bfloat16).min
    x[3] = -x[3].abs()
    i = torch.arange(4, device=dev, dtype=torch.int32)
    z = torch.zeros(4, device=dev, dtype=torch.int32)
    cache = ex.attn_fp4_cache(1, 1, d)
    ex.attn_rope_cache_write_fp4(x, x, x, z, i, z.view(1, 4), z[:1].view(1, 1), cache, (32,))
    k, v = ex.attn_cache_read_fp4(cache, z, i, z[:1].view(1, 1))
    bits = x.cpu().view(torch.int16).numpy().view(np.uint16)
    f = synth.bf16_bits_to_f32(bits)
    with np.errstate(invalid="ignore"):
        turned = ref.turn(f, np.float32(1.0), np.float32(0.0))
    for got, x32 in ((k, turned), (v, f)):
        codes, s8 = ref.quantise(x32, 1.0)
        want = ref.values(codes, s8, 1.0)
        g = got.double().cpu().numpy()
        assert (np.isnan(g) == np.isnan(want)).all()
        assert (np.nan_to_num(g) == np.nan_to_num(want)).all()
    assert np.isnan(want[0, 0, :48]).all() and np.isfinite(want[0, 0, 48:]).all()
    assert (want[1, 0, :32] == 0).all() and (want[1, 0, 32:48] == 448 * 6).all()


def test_append_and_read_outside_the_table_are_flagged(env):
    torch, ex, dev = env
    d, Hkv = 64, 2
    inp, slots, pos = append_case(520, [20, 20], 20, 2, Hkv, d)
    sid, sl, tbl = inp["seq_ids"].copy(), slots.copy(), inp["block_table"].copy()
    sid[3], sl[5], sl[6], sid[8] = 7, 10 ** 6, -1, -1
    tbl[1, 0], tbl[1, 1] = -1, inp["num_blocks"]
    good = np.ones(40, bool)
    good[[3, 5, 6, 8]] = False
    good[20:] = False
    cache = ex.attn_fp4_cache(inp["num_blocks"], Hkv, d)
    qd, kd, vd = (to_dev(inp[x], dev) for x in ("q", "k", "v"))
    sidd, sld, td = (to_dev(x, dev) for x in (sid, sl, tbl))
    q = ex.attn_rope_cache_write_fp4(qd, kd, vd, sidd, sld, to_dev(pos, dev), td, cache, (32,))
    torch.cuda.synchronize()
    assert ex.attn_get_device_status() == 2
    want_q = ex.attn_rope_cache_write_fp4(qd, kd, vd, *(to_dev(x, dev) for x in (inp["seq_ids"], slots, pos, inp["block_table"])),
                                          ex.attn_fp4_cache(inp["num_blocks"], Hkv, d), (32,))
    assert torch.equal(q, want_q)  # rotated all the same
    written = sum(int((x != 0).any(-1).sum()) for x in ref.split(cache.cpu().numpy(), d)[:1])
    assert written == good.sum() * Hkv
    k, v = ex.attn_cache_read_fp4(cache, sidd, sld, td, k_out=torch.full_like(kd, 9.0), v_out=torch.full_like(vd, 9.0))
    torch.cuda.synchronize()
    assert ex.attn_get_device_status() == 2
    assert (k[~good] == 0).all() and (v[~good] == 0).all() and (v[good] != 0).any(-1).all()


def test_same_slot_twice_touches_only_that_slot(env):
    torch, ex, dev = env
    d = 128
    x = torch.randn(6, 1, d, device=dev).bfloat16()
    z = torch.zeros(6, device=dev, dtype=torch.int32)
    slots = torch.tensor([0, 1, 1, 1, 2, 3], device=dev, dtype=torch.int32)
    cache = torch.full((1, 1, 18 * d), 0xA5, device=dev, dtype=torch.uint8)
    ex.attn_rope_cache_write_fp4(x, x, x, z, slots, slots.view(1, 6), z[:1].view(1, 1), cache, (64,))
    _, v = ex.attn_cache_read_fp4(cache, z, slots, z[:1].view(1, 1))
    assert (v[[0, 4, 5]] - x[[0, 4, 5]]).abs().max() < 1.0
    assert torch.isfinite(v).all()
    for view in ref.split(cache.cpu().numpy(), d):
        assert (view[0, 0, 4:] == 0xA5).all()


def test_append_strided_in_place_and_read_into_views(env):
    torch, ex, dev = env
    T, Hq, Hkv, d = 50, 6, 2, 64
    inp, slots, pos = append_case(530, [50], 50, Hq, Hkv, d)
    qkv = torch.empty((T, Hq + 2 * Hkv, d), device=dev, dtype=torch.bfloat16)
    qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:] = (to_dev(inp[x], dev) for x in ("q", "k", "v"))
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    idx = [to_dev(x, dev) for x in (inp["seq_ids"], slots)]
    pd, tbl = to_dev(pos, dev), to_dev(inp["block_table"], dev)
    c1, c2 = ex.attn_fp4_cache(inp["num_blocks"], Hkv, d), ex.attn_fp4_cache(inp["num_blocks"], Hkv, d)
    want = ex.attn_rope_cache_write_fp4(*(to_dev(inp[x], dev) for x in ("q", "k", "v")), *idx, pd, tbl, c1, (32,))
    kv = qkv[:, Hq:].clone()
    got = ex.attn_rope_cache_write_fp4(q, k, v, *idx, pd, tbl, c2, (32,), q_out=q)
    assert got is q and torch.equal(q, want) and torch.equal(c1, c2) and torch.equal(qkv[:, Hq:], kv)
    kr, vr = ex.attn_cache_read_fp4(c1, *idx, tbl)
    # one sequence into [Hkv, N, d] with room behind it
    room_k = torch.full((Hkv, T + 7, d), 5.0, device=dev, dtype=torch.bfloat16)
    room_v = torch.full((Hkv, T + 7, d), 5.0, device=dev, dtype=torch.bfloat16)
    ex.attn_cache_read_fp4(c1, *idx, tbl, k_out=room_k[:, :T].transpose(0, 1), v_out=room_v[:, :T].transpose(0, 1))
    assert torch.equal(room_k[:, :T].transpose(0, 1), kr) and torch.equal(room_v[:, :T].transpose(0, 1), vr)
    assert (room_k[:, T:] == 5).all() and (room_v[:, T:] == 5).all()
    with pytest.raises(ex.ExattnError):  # keys and values into the same rows
        ex.attn_cache_read_fp4(c1, *idx, tbl, k_out=kr, v_out=kr)
    with pytest.raises(ValueError):
        ex.attn_rope_cache_write_fp4(q, k[:-1], v, *idx, pd, tbl, c2, (32,))
    with pytest.raises(ValueError):
        ex.attn_rope_cache_write_fp4(q, k, v, *idx, pd[:, :-1].contiguous(), tbl, c2, (32,))
    with pytest.raises(ValueError):
        ex.attn_rope_cache_write_fp4(q, k, v, *idx, pd, tbl, c2, (16, 16))
    e = [x[:0] for x in idx]
    ex.attn_rope_cache_write_fp4(q[:0], k[:0], v[:0], *e, pd[:, :0].contiguous(), tbl, c2, (32,))
    assert ex.attn_cache_read_fp4(c2, *e, tbl)[0].shape == (0, Hkv, d)
    assert torch.equal(c1, c2)


@pytest.mark.parametrize("d", [64, 128])
def test_read_onto_every_16_byte_boundary(env, d):
    """Rows on 16-byte boundaries that are not 32-byte ones, or on both kinds in turn, and
    nothing written between them."""
    torch, ex, dev = env
    T, Hkv = 37, 3
    inp, slots, pos = append_case(531, [T], T, 1, Hkv, d)
    idx = [to_dev(x, dev) for x in (inp["seq_ids"], slots)]
    tbl = to_dev(inp["block_table"], dev)
    cache = ex.attn_fp4_cache(inp["num_blocks"], Hkv, d)
    t = [to_dev(inp[x], dev) for x in ("q", "k", "v")]
    ex.attn_rope_cache_write_fp4(*t, *idx, to_dev(pos, dev), tbl, cache, (d // 2,))
    want = ex.attn_cache_read_fp4(cache, *idx, tbl)
    for gap, start in ((0, 8), (8, 0), (8, 8), (16, 8)):
        room = torch.full((2, T * Hkv * (d + gap) + 32), 5.0, device=dev, dtype=torch.bfloat16)
        outs = [x[start:start + T * Hkv * (d + gap)].view(T, Hkv, d + gap) for x in room]
        ex.attn_cache_read_fp4(cache, *idx, tbl, k_out=outs[0][..., :d], v_out=outs[1][..., :d])
        for x, w in zip(outs, want):
            assert torch.equal(x[..., :d], w) and (x[..., d:] == 5).all()
        assert (room[:, :start] == 5).all() and (room[:, start + T * Hkv * (d + gap):] == 5).all()


# ------------------------------------------------------------------- together
@pytest.mark.parametrize("d", [64, 128])
def test_serving_run(env, d):
    """A prompt is appended, then token after token is appended and attended to;
    the last step and a chunk's prefill over the read-back prefix agree with the
    64-bit attention over what the cache stands for."""
    torch, ex, dev = env
    S, Hq, Hkv, first, steps = 3, 8, 2, [37, 16, 90], 5
    half = d // 2
    sections = (half // 2, half // 4, half // 4)
    lens = np.array(first, np.int32)
    table, nb = synth.paged_layout(lens + steps, 16, 9)
    cache, td = ex.attn_fp4_cache(nb, Hkv, d), to_dev(table, dev)
    ks, vs = 0.01, 0.003

    def new(T, seed):
        return (to_dev(synth.normal_bf16(seed, i, (T, h, d)), dev) for i, h in ((1, Hq), (2, Hkv), (3, Hkv)))

    def pos_of(slots):
        return torch.stack([slots, slots // 7, slots % 7]).contiguous()

    sid = torch.from_numpy(np.repeat(np.arange(S), first).astype(np.int32)).to(dev)
    slots = torch.from_numpy(np.concatenate([np.arange(n) for n in first]).astype(np.int32)).to(dev)
    q, k, v = new(len(slots), 600)
    ex.attn_rope_cache_write_fp4(q, k, v, sid, slots, pos_of(slots), td, cache, sections, k_scale=ks, v_scale=vs)
    one = torch.arange(S, device=dev, dtype=torch.int32)
    for step in range(steps):
        q, k, v = new(S, 601 + step)
        at = torch.from_numpy(lens).to(dev)
        qr = ex.attn_rope_cache_write_fp4(q, k, v, one, at, pos_of(at), td, cache, sections, k_scale=ks, v_scale=vs)
        lens = lens + 1
        out, lse = ex.attn_decode_paged_fp4(qr, cache, td, to_dev(lens, dev), k_scale=ks, v_scale=vs)
    torch.cuda.synchronize()
    assert ex.attn_get_device_status() == 0
    qb = qr.cpu().view(torch.int16).numpy().view(np.uint16)
    check_decode(out, lse, qb, cache.cpu().numpy(), table, lens, d, d ** -0.5, ks, vs)
    # the same token as a chunk of one over the prefix, through attn_fwd
    for s in range(S):
        n = int(lens[s])
        kk = torch.empty((1, Hkv, n, d), device=dev, dtype=torch.bfloat16)
        vv = torch.empty_like(kk)
        i = torch.arange(n, device=dev, dtype=torch.int32)
        ex.attn_cache_read_fp4(cache, torch.full_like(i, s), i, td, k_scale=ks, v_scale=vs,
                               k_out=kk[0].transpose(0, 1), v_out=vv[0].transpose(0, 1))
        o, l2 = ex.attn_fwd(qr[s].view(1, Hq, 1, d), kk, vv, causal=True)
        # keys and values rounded to bf16 (2^-8 each) on top of both outputs' own rounding
        assert (o.view(Hq, d).float() - out[s].float()).abs().max() < 5e-2
        assert (l2.view(Hq) - lse[s]).abs().max() < 2e-2


def test_threads_and_streams(env):
    """Four threads on streams of their own, each appending, reading and decoding
    on a cache of its own; every result equals the single thread's."""
    import threading
    torch, ex, dev = env
    d, Hq, Hkv = 64, 8, 2

    def work(i, stream):
        with torch.cuda.stream(stream):
            inp, slots, pos = append_case(540 + i, [60 + 9 * i, 30], 30, Hq, Hkv, d)
            t = [to_dev(inp[x], dev) for x in ("q", "k", "v", "seq_ids")] + [to_dev(slots, dev), to_dev(pos, dev)]
            tbl = to_dev(inp["block_table"], dev)
            lens = torch.tensor([60 + 9 * i, 30], device=dev, dtype=torch.int32)
            res = []
            for _ in range(10):
                cache = ex.attn_fp4_cache(inp["num_blocks"], Hkv, d)
                q = ex.attn_rope_cache_write_fp4(*t, tbl, cache, (32,), stream=stream)
                k, v = ex.attn_cache_read_fp4(cache, t[3], t[4], tbl, stream=stream)
                out, lse = ex.attn_decode_paged_fp4(q[[0, -1]].contiguous(), cache, tbl, lens, stream=stream)
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


def test_workspace_of_a_call_on_another_stream_is_not_reused_while_it_runs(env):
    """The call allocates its workspace, uses it on the given stream and drops it;
    what the current stream allocates next must not land there."""
    torch, ex, dev = env
    q, cache, table, lens = decode_case(560, [20000, 3], 8, 1, 128)
    args = [to_dev(x, dev) for x in (q, cache, table, lens)]
    want, want_lse = ex.attn_decode_paged_fp4(*args)
    n = ex.attn_decode_fp4_workspace_bytes(2, 8, 1, 128, table.shape[1])
    assert n > 0
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        out, lse = ex.attn_decode_paged_fp4(*args, stream=side)
        for _ in range(3):
            torch.full((n,), 0xFF, device=dev, dtype=torch.uint8)
        side.synchronize()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("S,ctx,Hq,Hkv", [(5, 3000, 8, 2), (40, 900, 8, 4), (2, 300, 4, 2)])
def test_calls_that_follow_each_other_wait_for_what_they_use(env, S, ctx, Hq, Hkv):
    """Each call may begin while the one before it ends, so each has to wait for what it
    reads (queries, lengths, the cache) and overwrites (the next step turns the same
    tensors in place): the same bits with and without a synchronisation after every
    call, and from a replayed graph."""
    torch, ex, dev = env
    d, steps = 128, 6
    blocks = (ctx + steps + 15) // 16
    table = torch.arange(S * blocks, device=dev, dtype=torch.int32).view(S, blocks)
    seq = torch.arange(S, device=dev, dtype=torch.int32)
    lens = [torch.tensor([ctx - 3 * i + step for i in range(S)], device=dev, dtype=torch.int32)
            for step in range(steps + 1)]
    start = ex.attn_fp4_cache(S * blocks, Hkv, d)
    kv = to_dev(synth.normal_bf16(576, 1, (S * ctx, Hkv, d)), dev)
    every = seq.repeat_interleave(ctx)
    place = torch.arange(ctx, device=dev, dtype=torch.int32).repeat(S)
    ex.attn_rope_cache_write_fp4(kv[:, :0], kv, kv, every, place, place[None], table, start, (64,))
    q0 = to_dev(synth.normal_bf16(576, 2, (S, Hq, d)), dev)
    q, x, cache = q0.clone(), q0.clone(), start.clone()
    seen = torch.empty(steps, S, Hq, d, device=dev, dtype=torch.bfloat16)
    back = torch.empty(steps, S, Hkv, d, device=dev, dtype=torch.bfloat16)

    def run(after):
        x.copy_(q0), cache.copy_(start), after()
        for i in range(steps):
            at = lens[i]
            ex.attn_rope_cache_write_fp4(x, x[:, :Hkv], x[:, Hq - Hkv:], seq, at, at[None], table, cache, (64,),
                                         q_out=q), after()
            ex.attn_decode_paged_fp4(q, cache, table, lens[i + 1], out=seen[i]), after()
            ex.attn_rope_axes(q[None].transpose(1, 2), q[None, :, :0].transpose(1, 2), at[None], (64,), inverse=True,
                              q_out=q[None].transpose(1, 2)), after()
            ex.attn_decode_paged_fp4(q, cache, table, lens[i + 1], out=x), after()
            ex.attn_cache_read_fp4(cache, seq, at, table, k_out=back[i]), after()

    run(torch.cuda.synchronize)
    want, want_back, want_cache = seen.clone(), back.clone(), cache.clone()
    assert torch.isfinite(want.float()).all() and want.float().abs().max() > 0
    for _ in range(10):
        seen.zero_(), back.zero_()
        run(lambda: None)
        assert torch.equal(seen, want) and torch.equal(back, want_back) and torch.equal(cache, want_cache)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(lambda: None)
    for _ in range(3):
        seen.zero_(), back.zero_()
        g.replay()
        assert torch.equal(seen, want) and torch.equal(back, want_back) and torch.equal(cache, want_cache)
    assert ex.attn_get_device_status() == 0


def test_calls_after_an_event_of_another_stream(env):
    """A call behind a kernel of its own stream and an event of another waits for both,
    and the other stream, behind an event after it, overwrites its inputs no sooner."""
    torch, ex, dev = env
    d, Hq, Hkv, S = 128, 8, 2, 6
    qs = [to_dev(synth.normal_bf16(590 + i, 1, (S, Hq, d)), dev) for i in range(12)]
    _, cache, table, lens = decode_case(589, [3000, 5, 700, 129, 0, 64], Hq, Hkv, d)
    cache, table, lens = (to_dev(x, dev) for x in (cache, table, lens))
    at = torch.arange(S, device=dev, dtype=torch.int32)[None]
    none = qs[0][:, :0]
    want = []
    for q in qs:
        turned, _ = ex.attn_rope_axes(q[None].transpose(1, 2), none[None].transpose(1, 2), at, (64,))
        torch.cuda.synchronize()
        want.append(ex.attn_decode_paged_fp4(turned[0].transpose(0, 1).contiguous(), cache, table, lens)[0])
        torch.cuda.synchronize()
    busy = torch.randn(4096, 4096, device=dev)
    side, main = torch.cuda.Stream(), torch.cuda.current_stream()
    x, y = torch.zeros_like(qs[0]), torch.zeros_like(qs[0])
    side.wait_stream(main)
    got = []
    for q in qs:
        with torch.cuda.stream(side):
            busy = (busy @ busy).clamp(-1, 1)  # the copy comes late
            x.copy_(q)
        ex.attn_rope_axes(y[None].transpose(1, 2), none[None].transpose(1, 2), at, (64,), q_out=y[None].transpose(1, 2))
        main.wait_stream(side)
        ex.attn_rope_axes(x[None].transpose(1, 2), none[None].transpose(1, 2), at, (64,), q_out=y[None].transpose(1, 2))
        side.wait_stream(main)
        got.append(ex.attn_decode_paged_fp4(y, cache, table, lens)[0])
        with torch.cuda.stream(side):
            x.fill_(float("nan"))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert ex.attn_get_device_status() == 0


def test_append_captured_and_replayed(env):
    torch, ex, dev = env
    d, Hkv = 128, 2
    inp, slots, pos = append_case(550, [40, 9], 9, 4, Hkv, d)
    t = [to_dev(inp[x], dev) for x in ("q", "k", "v", "seq_ids")] + [to_dev(slots, dev), to_dev(pos, dev)]
    tbl = to_dev(inp["block_table"], dev)
    cache, other = ex.attn_fp4_cache(inp["num_blocks"], Hkv, d), ex.attn_fp4_cache(inp["num_blocks"], Hkv, d)
    ex.attn_rope_cache_write_fp4(*t, tbl, other, (64,))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q = ex.attn_rope_cache_write_fp4(*t, tbl, cache, (64,))
        k, v = ex.attn_cache_read_fp4(cache, t[3], t[4], tbl)
        qa, ka = ex.attn_rope_axes(t[0].transpose(0, 1)[None], t[1].transpose(0, 1)[None], t[5][:, None], (64,))
    for _ in range(2):
        cache.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(cache, other)
        assert torch.equal(qa[0].transpose(0, 1), q)
    t[2].mul_(2)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(v, ex.attn_cache_read_fp4(other, t[3], t[4], tbl)[1] * 2)


def test_rows_and_blocks_past_32_bits(env):
    """Heads 2^31 elements apart, and blocks whose bytes pass 2^32."""
    torch, ex, dev = env
    T, H, d, far = 21, 2, 128, 1 << 31
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    x = to_dev(synth.normal_bf16(580, 1, (T, H, d)), dev)
    big = torch.zeros(far + T * d, device=dev, dtype=torch.bfloat16)
    wide = big.as_strided((T, H, d), (d, far, 1))
    wide.copy_(x)
    at = torch.arange(T, device=dev, dtype=torch.int32)
    want, _ = ex.attn_rope_axes(x[None].transpose(1, 2), x[None].transpose(1, 2), at[None], (64,))
    got, same = ex.attn_rope_axes(wide[None].transpose(1, 2), x[None].transpose(1, 2), at[None], (64,))
    assert torch.equal(got, want) and torch.equal(same, want)

    blocks = (1 << 32) // (H * 18 * d) + 4
    seq = torch.zeros(T, device=dev, dtype=torch.int32)
    near, ends = (torch.tensor([ids], device=dev, dtype=torch.int32) for ids in ([1, 0], [blocks - 1, blocks - 3]))
    small, cache = ex.attn_fp4_cache(2, H, d), ex.attn_fp4_cache(blocks, H, d)
    q = ex.attn_rope_cache_write_fp4(x, x, x, seq, at, at[None], near, small, (64,))
    ex.attn_rope_cache_write_fp4(x, wide, wide, seq, at, at[None], ends, cache, (64,))
    with pytest.raises(ex.ExattnError):  # queries over the keys that are yet to be read
        ex.attn_rope_cache_write_fp4(wide, wide, wide, seq, at, at[None], ends, cache, (64,), q_out=wide)
    qf = ex.attn_rope_cache_write_fp4(wide, x, x, seq, at, at[None], ends, cache, (64,), q_out=wide)
    assert qf is wide and torch.equal(wide, q) and torch.equal(q, want[0].transpose(0, 1))
    assert torch.equal(cache[-1], small[1]) and torch.equal(cache[-3], small[0])
    assert int(cache[:-3].view(-1)[:1 << 20].max()) == 0 and int(cache[-2].max()) == 0
    k, v = ex.attn_cache_read_fp4(small, seq, at, near)
    wide.zero_()
    kf, vf = ex.attn_cache_read_fp4(cache, seq, at, ends, k_out=wide)
    assert torch.equal(kf, k) and torch.equal(vf, v)
    lens = torch.tensor([T], device=dev, dtype=torch.int32)
    a, b = ex.attn_decode_paged_fp4(q[-1:], small, near, lens), ex.attn_decode_paged_fp4(q[-1:], cache, ends, lens)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert ex.attn_get_device_status() == 0


def test_first_calls_of_a_process_may_be_captured(env):
    """The kernels load and the device state is set up inside a capture, too."""
    import os
    import subprocess
    import sys
    code = """
import torch
from exact_attention_40_gb300 import exattn as ex
dev = torch.device("cuda:0")
T, Hq, Hkv, d, S = 40, 8, 2, 128, 2
g = torch.Generator(device=dev).manual_seed(1)
q, k, v = (torch.randn(T, h, d, device=dev, generator=g).bfloat16() for h in (Hq, Hkv, Hkv))
seq = torch.zeros(T, device=dev, dtype=torch.int32)
at = torch.arange(T, device=dev, dtype=torch.int32)
blocks = 700
table = torch.arange(S * blocks, device=dev, dtype=torch.int32).view(S, blocks)
lens = torch.tensor([T, 0], device=dev, dtype=torch.int32)
cache = ex.attn_fp4_cache(S * blocks, Hkv, d)

def run():
    a = ex.attn_rope_axes(q[None].transpose(1, 2), k[None].transpose(1, 2), at[None], (64,))
    b = ex.attn_rope_cache_write_fp4(q, k, v, seq, at, at[None], table, cache, (64,))
    c = ex.attn_cache_read_fp4(cache, seq, at, table)
    e = ex.attn_decode_paged_fp4(b[:S], cache, table, lens)          # split and merge
    f = ex.attn_decode_paged_fp4(b[:S], cache, table[:, :100].contiguous(), lens)  # a cluster for each segment
    return [*a, b, *c, *e, *f]

graph = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(graph):
    got = run()
graph.replay()
torch.cuda.synchronize()
for x, y in zip(got, run()):
    assert torch.equal(x, y)
assert ex.attn_get_device_status() == 0
print("captured")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stdout + r.stderr
