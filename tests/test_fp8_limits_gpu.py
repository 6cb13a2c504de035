"""The 8-bit cache at its largest and smallest sizes: as many sequences and columns as the
calls take, contexts of millions of tokens, the last place a table can name, no tokens at
all, layers of one tensor as caches.  The bars are those of test_fp8_gpu.py."""
import numpy as np
import pytest

import fp8_reference as ref
from exact_attention_40_gb300 import synth
from helpers import to_dev
from test_fp8_gpu import append_case, check_decode, decode_case, env, run_append, run_decode  # noqa: F401  (env: a fixture)

pytestmark = pytest.mark.gpu


def appended_values(x):
    """What x [S, H, d] reads back as from blocks that hold one token of it each."""
    x = synth.bf16_bits_to_f32(x).astype(np.float64)
    e = ref.exponent(ref.most_of(x, 2)).astype(np.float64)[..., None]
    return ref.E4M3[ref.codes_of(x, e)] * 2.0 ** e


@pytest.mark.parametrize("starts", [False, True])
def test_append_to_as_many_sequences_as_there_can_be(env, starts):
    """65535 sequences; with token_starts every second one has two tokens, of two blocks,
    and the others none."""
    torch, ex, dev = env
    S, d = 65535, 64
    k, v = (synth.normal_bf16(900, i, (S, 1, d)) for i in (1, 2))
    cache = ex.attn_fp8_cache(2 * S, 1, d, dev)
    table = np.arange(2 * S, dtype=np.int32).reshape(S, 2)[:, ::-1].copy()
    T = S if not starts else S // 2 * 2
    if starts:
        new = np.where(np.arange(S) % 2 == 1, 2, 0)
        ends = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        ctx = np.full(S, 17, np.int32)
        seq = np.repeat(np.arange(S, dtype=np.int32), new)
        slots = np.tile(np.array([15, 16], np.int32), T // 2)
    else:
        ctx, seq, slots = np.ones(S, np.int32), np.arange(S, dtype=np.int32), np.zeros(S, np.int32)
    k, v = k[:T], v[:T]
    q = np.zeros((T, 0, d), np.uint16)
    out = ex.attn_rope_cache_write_fp8(to_dev(q, dev), to_dev(k, dev), to_dev(v, dev), to_dev(ends, dev) if starts else None,
                                       to_dev(ctx, dev), torch.zeros((1, T), dtype=torch.int32, device=dev),
                                       to_dev(table, dev), cache, (d // 2,))
    assert out.shape == (T, 0, d)
    got = ex.attn_cache_read_fp8(cache, to_dev(seq, dev), to_dev(slots, dev), to_dev(table, dev))
    assert ex.attn_get_device_status() == 0
    for g, x in zip(got, (k, v)):
        assert np.array_equal(g.double().cpu().numpy(), appended_values(x))
    # no other byte of the cache is written
    at = ref.place(d)
    held = cache.cpu().numpy()
    used = table[seq, slots // 16]
    codes, scales = ref.split(held, d)
    assert (scales[used] != 0).all()
    mine = np.zeros((16, 16 * d), bool)
    for n in range(16):
        mine[n, at[n]] = True
    assert not codes[used][:, 0][np.repeat(~mine[slots % 16][:, None], 2, 1)].any()
    rest = np.ones(2 * S, bool)
    rest[used] = False
    assert not held[rest].any()


def test_decode_of_as_many_sequences_as_there_can_be(env):
    torch, ex, dev = env
    S, d = 65535, 64
    cache = ref.random_cache(901, 500, 1, d)
    u = synth.uniform01(902, 4 * S).reshape(4, S)
    table = np.floor(u[:3].T * 500).astype(np.int32)
    lens = np.floor(u[3] * 49).astype(np.int32)
    lens[[0, S - 1]] = [48, 47]
    q = synth.normal_bf16(903, 0, (S, 2, d))
    out, lse = ex.attn_decode_paged_fp8(*(to_dev(x, dev) for x in (q, cache, table, lens)))
    assert ex.attn_get_device_status() == 0
    some = np.concatenate([np.arange(100), np.arange(S // 2, S // 2 + 100), np.arange(S - 100, S)])
    pick = torch.from_numpy(some).to(dev)
    check_decode(out[pick], lse[pick], q[some], cache, table[some], lens[some], d, d ** -0.5)
    assert bool(torch.isfinite(out).all())
    assert np.array_equal(np.isneginf(lse.cpu().numpy()), np.repeat((lens == 0)[:, None], 2, 1))


def test_decode_of_as_many_heads_as_there_can_be(env):
    """65535 query heads of one KV head, of two tokens: 131070 columns, the last chunk ragged."""
    torch, ex, dev = env
    d, Hq = 64, 65535
    cache, table = ref.random_cache(904, 20, 1, d), np.arange(20, dtype=np.int32)[None]
    lens = np.array([300], np.int32)
    q = synth.normal_bf16(905, 0, (1, 2, Hq, d))
    out, lse = ex.attn_decode_paged_fp8(*(to_dev(x, dev) for x in (q, cache, table, lens)))
    assert ex.attn_get_device_status() == 0
    some = np.concatenate([np.arange(50), np.arange(30000, 30050), np.arange(Hq - 50, Hq)])
    pick = torch.from_numpy(some).to(dev)
    check_decode(out[:, :, pick], lse[:, :, pick], q[:, :, some], cache, table, lens, d, d ** -0.5)
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all())


@pytest.mark.parametrize("queries", [None, 3])
def test_decode_of_millions_of_tokens(env, queries):
    """A context that repeats the same 64 tokens 2^16 times: the output is that of the 64, the
    log-sum-exp larger by log 2^16.  (With several queries the last ones' unseen tokens are
    left out of the reference: their weight is below 2^-20.)  Added to the bar: fp32 sums
    of a lane's tokens, 2^22 / (2 x 456 x 4 x 8) < 2^8 of them at least, so off by at most 2^-16, in
    the weights' sum and in the values'."""
    torch, ex, dev = env
    d, times = 128, 1 << 16
    cache = ref.random_cache(906, 4, 1, d)
    table = np.tile(np.arange(4, dtype=np.int32), times)[None]
    shape = (1, 2, d) if queries is None else (1, queries, 2, d)
    q = synth.normal_bf16(907, 0, shape)
    lens = np.array([64 * times], np.int32)
    out, lse = ex.attn_decode_paged_fp8(*(to_dev(x, dev) for x in (q, cache, table, lens)))
    assert ex.attn_get_device_status() == 0
    once = np.arange(4, dtype=np.int32)[None]
    q1 = q.reshape(-1, 1, 2, d)  # each query as the only one
    n = len(q1)
    want, wl, big, mean, _ = ref.decode(q1, cache, np.repeat(once, n, 0), np.full(n, 64, np.int32), d, d ** -0.5)
    got, gl = out.double().cpu().numpy().reshape(want.shape), lse.double().cpu().numpy().reshape(wl.shape)
    slack = 2.0 ** -15 + 2.0 ** -19
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + (2.0 ** -10 + 2.0 ** -15 * big[..., None] + slack) * mean).all()
    assert (np.abs(gl - wl - np.log(times)) <= 2.0 ** -16 * big + 2.0 ** -19 * (1 + np.abs(wl) + np.log(times)) + slack).all()


def test_the_last_place_that_a_table_can_name(env):
    """max_blocks_per_seq 2^26: a token is appended at place 2^30 - 1 and read back; one past
    it is flagged."""
    torch, ex, dev = env
    if torch.cuda.mem_get_info()[0] < 8 << 30:
        pytest.skip("needs 8 GiB")
    d = 64
    cache = ex.attn_fp8_cache(3, 1, d, dev)
    table = torch.full((1, 1 << 26), -1, device=dev, dtype=torch.int32)
    table[0, -1] = 2
    k = synth.normal_bf16(908, 1, (1, 1, d))
    kd = to_dev(k, dev)
    one = lambda n: torch.tensor([n], device=dev, dtype=torch.int32)  # noqa: E731
    args = (torch.zeros((1, 1), device=dev, dtype=torch.int32), table, cache, (32,))
    ex.attn_rope_cache_write_fp8(kd, kd, kd, None, one(1 << 30), *args)
    got = ex.attn_cache_read_fp8(cache, one(0), one((1 << 30) - 1), table)
    assert ex.attn_get_device_status() == 0
    for g in got:
        assert np.array_equal(g.double().cpu().numpy(), appended_values(k))
    before = cache.clone()
    ex.attn_rope_cache_write_fp8(kd, kd, kd, None, one((1 << 30) + 1), *args)
    assert ex.attn_get_device_status() == 2 and torch.equal(cache, before)
    ex.attn_rope_cache_write_fp8(kd, kd, kd, torch.tensor([0, 1], device=dev, dtype=torch.int32), one(2 ** 31 - 1), *args)
    assert ex.attn_get_device_status() == 2 and torch.equal(cache, before)


def test_calls_without_tokens(env):
    torch, ex, dev = env
    cache = ex.attn_fp8_cache(2, 1, 64, dev)
    none = torch.zeros(0, device=dev, dtype=torch.int32)
    table = torch.zeros((3, 1), device=dev, dtype=torch.int32)
    x = torch.zeros((0, 1, 64), device=dev, dtype=torch.bfloat16)
    starts, lens = torch.zeros(4, device=dev, dtype=torch.int32), torch.full((3,), 5, device=dev, dtype=torch.int32)
    out = ex.attn_rope_cache_write_fp8(x, x, x, starts, lens, none.view(1, 0), table, cache, (32,))
    k, v = ex.attn_cache_read_fp8(cache, none, none, table)
    o, lse = ex.attn_decode_paged_fp8(x, cache, table[:0], none)
    assert out.shape == k.shape == v.shape == o.shape == (0, 1, 64) and lse.shape == (0, 1)
    o, lse = ex.attn_decode_paged_fp8(x.view(0, 4, 1, 64), cache, table[:0], none)
    assert o.shape == (0, 4, 1, 64) and lse.shape == (0, 4, 1)
    assert ex.attn_get_device_status() == 0 and not cache.any()


def test_append_without_queries(env):
    c = append_case(909, [3, 20], [40, 1], 0, 2, 128)
    run_append(env, c, 2, 128, (64,))


def test_layers_of_one_tensor(env):
    """Caches that are slices of one allocation: a call on one leaves the others as they are."""
    torch, ex, dev = env
    d, layers = 64, 3
    c = append_case(910, [5, 0, 31], [20, 3, 2], 4, 2, d)
    nb = c["cache"].shape[0]
    pool = torch.zeros((layers, nb, 2, 32 * d + 32), device=dev, dtype=torch.uint8)
    for layer in range(layers):
        pool[layer] = to_dev(c["cache"], dev)
    before = pool.clone()
    qd, kd, vd, st, ctx, pd, tbl = (to_dev(c[x], dev) for x in ("q", "k", "v", "starts", "ctx", "pos", "table"))
    ex.attn_rope_cache_write_fp8(qd, kd, vd, st, ctx, pd, tbl, pool[1], (32,))
    want = run_append(env, c, 2, d, (32,), base=500000.0)
    assert torch.equal(pool[1], want) and torch.equal(pool[0], before[0]) and torch.equal(pool[2], before[2])
    q = synth.normal_bf16(911, 0, (3, 4, d))
    out, lse = ex.attn_decode_paged_fp8(to_dev(q, dev), pool[1], tbl, ctx)
    check_decode(out, lse, q, want.cpu().numpy(), c["table"], c["ctx"], d, d ** -0.5)
    assert ex.attn_get_device_status() == 0


@pytest.mark.parametrize("d", [64, 128])
def test_drafted_tokens_taken_back(env, d):
    """Four drafted tokens, large ones among them, of which some are kept: the next step writes
    over the others, in the same block, in the one before and at a block's beginning."""
    torch, ex, dev = env
    first = append_case(912, [5, 30, 14, 16, 0], [4, 4, 4, 4, 4], 4, 2, d, gain=64.0, room=16)
    cache = run_append(env, first, 2, d, (d // 2,))
    step = append_case(913, [7, 31, 15, 16, 0], [4, 1, 4, 4, 2], 4, 2, d)
    step["table"], step["cache"] = first["table"], cache.cpu().numpy()
    after = run_append(env, step, 2, d, (d // 2,))
    q = synth.normal_bf16(914, 0, (5, 2, 4, d))
    out, lse = ex.attn_decode_paged_fp8(to_dev(q, dev), after, to_dev(step["table"], dev), to_dev(step["ctx"], dev))
    check_decode(out, lse, q, after.cpu().numpy(), step["table"], step["ctx"], d, d ** -0.5)
    assert ex.attn_get_device_status() == 0


@pytest.mark.parametrize("q_exp,k_exp,scale_exp", [(78, 60, -140), (-70, -56, 124), (75, 72, -149), (-110, 40, 68),
                                                    (120, -110, -12)])
def test_decode_factors_far_from_one(env, q_exp, k_exp, scale_exp):
    """Queries, keys and scale whose product is ordinary, though that of two of them may pass
    what a float's exponent holds."""
    d = 64
    q, cache, table, lens = decode_case(915, [70, 300], 4, 2, d, gain=2.0 ** k_exp)
    f = synth.bf16_bits_to_f32(q) * np.float32(2.0 ** q_exp)
    run_decode(env, (synth.f32_to_bf16_bits(f), cache, table, lens), d, scale=2.0 ** scale_exp)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("S,Hq,Hkv,queries", [(1, 8, 2, 1), (1, 12, 1, 1), (5, 16, 4, 1), (3, 6, 2, 5), (9, 16, 8, 1),
                                               (21, 10, 1, 2), (18, 16, 8, 2)])
def test_decode_merge_of_few_and_many_rows(env, S, Hq, Hkv, queries, d):
    """Contexts whose segments many CTAs share, of 8 to 640 rows that are merged."""
    lens = 4200 + np.arange(S) * 37 % 900
    lens[0] = 9001
    run_decode(env, decode_case(916, lens, Hq, Hkv, d, queries), d)
