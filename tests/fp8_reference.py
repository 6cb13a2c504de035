"""Plain implementations of the 8-bit cache in numpy: the definitions in 64 bits, token
by token and block by block."""
import numpy as np

from exact_attention_40_gb300 import synth
from fp4_reference import E4M3, e4m3_round

LOW, HIGH = -117, 119  # exponents of the scales


def place(d):
    """[16, d]: the byte of a block's codes that holds token n's column c."""
    out = np.empty((16, d), np.int64)
    for n in range(16):
        turn = n % 8 if d == 128 else n // 2 % 4
        for c in range(d):
            out[n, c] = n * d + 16 * (c // 16 ^ turn) + c % 16
    return out


def exponent(most):
    """Smallest e with most <= 448 * 2^e, within the range; most any shape >= 0."""
    most = np.asarray(most, np.float64)
    m, x = np.frexp(most)
    return np.where(most == 0, LOW, np.clip(np.where(m <= 0.875, x - 9, x - 8), LOW, HIGH))


def codes_of(x, e):
    """e4m3 codes of x / 2^e; what is not finite becomes NaN."""
    x = np.asarray(x, np.float64)
    ok = np.isfinite(x)
    c = e4m3_round(np.abs(np.where(ok, x, 0.0)) * 2.0 ** -np.asarray(e, np.float64))
    return np.where(ok, c, 0x7F).astype(np.uint8) | (np.signbit(x) & ok).astype(np.uint8) << 7


def most_of(x, axis):
    return np.where(np.isfinite(x), np.abs(x), 0.0).max(axis)


def split(cache, d):
    """Views: codes [nb, Hkv, 2, 16 d], scales [nb, Hkv, 2] (keys, values)."""
    nb, H = cache.shape[:2]
    return cache[..., :32 * d].reshape(nb, H, 2, 16 * d), cache.view(np.float32)[..., 8 * d:8 * d + 2]


def codes_by_token(cache, d):
    """[nb, Hkv, 2, 16, d], a copy."""
    return split(cache, d)[0][..., place(d)]


def values(cache, d):
    """(k, v) fp64 [nb, Hkv, 16, d]."""
    x = E4M3[codes_by_token(cache, d)] * split(cache, d)[1].astype(np.float64)[..., None, None]
    return x[:, :, 0], x[:, :, 1]


def set_tokens(cache, d, blk, which, codes):
    """Writes all 16 tokens' codes [Hkv, 16, d] of a block."""
    split(cache, d)[0][blk, :, which][:, place(d)] = codes


def random_cache(seed, nb, Hkv, d, gain=1.0, k_exp=0, v_exp=0):
    """A cache that holds quantised normal keys (times gain) and values; blocks' sizes
    spread over 2^-exp .. 2^exp."""
    k = synth.bf16_bits_to_f32(synth.normal_bf16(seed, 1, (nb, Hkv, 16, d))).astype(np.float64) * gain
    v = synth.bf16_bits_to_f32(synth.normal_bf16(seed, 2, (nb, Hkv, 16, d))).astype(np.float64)
    u = synth.uniform01(seed + 7, 2 * nb * Hkv).reshape(2, nb, Hkv, 1, 1)
    cache = np.zeros((nb, Hkv, 32 * d + 32), np.uint8)
    codes, scales = split(cache, d)
    at = place(d)
    for which, (x, spread) in enumerate(((k, k_exp), (v, v_exp))):
        x = x * 2.0 ** np.rint((2 * u[which] - 1) * spread)
        e = exponent(most_of(x, (2, 3)))
        codes[:, :, which, at] = codes_of(x, e[..., None, None])
        scales[:, :, which] = 2.0 ** e
    return cache


def append(cache, d, table, starts, ctx, k, v):
    """Appends k, v [T, Hkv, d] to the cache in place: each sequence's tokens in order,
    block by block."""
    codes, scales = split(cache, d)
    at = place(d)
    for s in range(len(ctx)):
        first = int(ctx[s]) - int(starts[s + 1] - starts[s])
        if first == ctx[s]:
            continue
        for b in range(first // 16, (int(ctx[s]) + 15) // 16):
            slots = np.arange(max(first, 16 * b), min(int(ctx[s]), 16 * b + 16))
            tok = int(starts[s]) + slots - first
            blk, off = table[s, b], slots - 16 * b
            for which, x in ((0, k), (1, v)):
                new = np.asarray(x[tok], np.float64).transpose(1, 0, 2)  # [Hkv, n, d]
                e = exponent(most_of(new, (1, 2)))
                if off[0] > 0:
                    held = scales[blk, :, which].astype(np.float64)
                    e_held = np.where(held > 0, np.log2(np.where(held > 0, held, 1.0)), -np.inf)
                    old = E4M3[codes[blk, :, which]] * held[:, None]
                    e = np.maximum(e, e_held)
                    moved = codes_of(old, e[:, None])
                    codes[blk, :, which] = np.where((e > e_held)[:, None], moved, codes[blk, :, which])
                scales[blk, :, which] = 2.0 ** e
                codes[blk, :, which][:, at[off]] = codes_of(new, e[:, None, None])


def decode(q, cache, table, lens, d, scale):
    """q [S, n, Hq, d] bf16 bits.  out [S,n,Hq,d], lse [S,n,Hq]; for the bars: the largest
    sum of |q k| of a score, and the mean of |v| by weight [S,n,Hq,d], and the largest
    product of a weight and its block's value scale [S,n,Hq]; fp64.  Blocks with a table
    entry out of range are left out."""
    S, N, Hq = q.shape[:3]
    nb, Hkv = cache.shape[:2]
    q = synth.bf16_bits_to_f32(q).astype(np.float64)
    out, lse = np.zeros((S, N, Hq, d)), np.full((S, N, Hq), -np.inf)
    big, mean, part = np.zeros((S, N, Hq)), np.zeros((S, N, Hq, d)), np.zeros((S, N, Hq))
    G = Hq // Hkv
    scales = split(cache, d)[1].astype(np.float64)
    for s in range(S):
        for i in range(N):
            n = int(lens[s]) - (N - 1 - i)
            if n <= 0:
                continue
            blk = table[s, :(n + 15) // 16]
            seen = np.repeat((blk >= 0) & (blk < nb), 16)[:n]
            if not seen.any():
                continue
            safe = np.clip(blk, 0, nb - 1)
            k, v = values(cache[safe], d)
            k, v = (x.transpose(1, 0, 2, 3).reshape(Hkv, -1, d)[:, :n][:, seen] for x in (k, v))
            unit = np.repeat(scales[safe, :, 1].T, 16, axis=1)[:, :n][:, seen]
            for h in range(Hq):
                x = k[h // G] @ q[s, i, h] * scale
                m = x.max()
                p = np.exp(x - m)
                total = p.sum()
                out[s, i, h] = p @ v[h // G] / total
                mean[s, i, h] = p @ np.abs(v[h // G]) / total
                lse[s, i, h] = m + np.log(total)
                big[s, i, h] = (np.abs(k[h // G]) @ np.abs(q[s, i, h])).max() * scale
                part[s, i, h] = (p * unit[h // G]).max() / total
    return out, lse, big, mean, part
