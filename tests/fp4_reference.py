"""Plain implementations of the 4-bit cache and of rotary positions with
several axes, in numpy: the definitions in 64 bits, and the append's fp32
operations one by one where its bytes are compared."""
import numpy as np

from exact_attention_40_gb300 import synth

VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
TIES = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])  # halfway between neighbours
TIE_UP = np.array([False, True, False, True, False, True, False])  # to the even code


def e4m3_table():
    out = np.empty(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        out[b] = (-x if b & 128 else x) if b & 127 != 127 else np.nan
    return out


E4M3 = e4m3_table()
POSITIVE = E4M3[:127]  # 0 .. 448, ascending


def e4m3_round(x):
    """Nearest e4m3 code of x >= 0, ties to even, saturating; x any shape, fp64."""
    x = np.minimum(np.asarray(x, np.float64), 448.0)
    hi = np.clip(np.searchsorted(POSITIVE, x), 0, 126)
    lo = np.maximum(hi - 1, 0)
    d_hi, d_lo = POSITIVE[hi] - x, x - POSITIVE[lo]
    return np.where((d_lo < d_hi) | ((d_lo == d_hi) & (lo % 2 == 0)), lo, hi).astype(np.uint8)


def e2m1_round(y):
    """e2m1 codes of y (nearest, ties to even, saturating), y fp32 or fp64."""
    m = np.abs(y)[..., None]
    up = (m > TIES) | ((m == TIES) & TIE_UP)
    code = up.sum(-1)
    code = np.where(np.isnan(y), 7, code)
    return (code + 8 * np.signbit(y)).astype(np.uint8)


def quantise(x, g):
    """Codes [..., d] and scale bytes [..., d/16] of x [..., d] (fp32), with the
    fp32 operations of the definition."""
    x = np.asarray(x, np.float32)
    g = np.float32(g)
    grp = x.reshape(x.shape[:-1] + (-1, 16))
    amax = np.abs(grp).max(-1)  # NaN if a value is
    ok = amax < np.inf
    with np.errstate(all="ignore"):
        t = (amax / (np.float32(6.0) * g)).astype(np.float32)
        s8 = np.where(ok, e4m3_round(np.where(ok, t, 0.0)), 0x7F).astype(np.uint8)
        div = (E4M3[s8].astype(np.float32) * g).astype(np.float32)[..., None]
        y = np.where(div == 0, np.float32(0.0), grp / div).astype(np.float32)
    return e2m1_round(y).reshape(x.shape), s8


def values(codes, s8, g):
    """What codes [..., d] and scales [..., d/16] stand for, fp64."""
    sign = np.where(codes & 8, -1.0, 1.0)
    v = sign * VALUES[codes & 7]
    return (v.reshape(v.shape[:-1] + (-1, 16)) * E4M3[s8][..., None]).reshape(v.shape) * float(np.float32(g))


def pack(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def unpack(b):
    return np.stack([b & 15, b >> 4], -1).reshape(b.shape[:-1] + (-1,))


def split(cache, d):
    """Views (key codes, value codes [nb,Hkv,16,d/2], key, value scales [nb,Hkv,16,d/16])."""
    nb, H = cache.shape[:2]
    return (cache[..., :8 * d].reshape(nb, H, 16, d // 2), cache[..., 8 * d:16 * d].reshape(nb, H, 16, d // 2),
            cache[..., 16 * d:17 * d].reshape(nb, H, 16, d // 16), cache[..., 17 * d:].reshape(nb, H, 16, d // 16))


def cache_values(cache, d, k_scale, v_scale):
    """(k, v) fp64 [nb, Hkv, 16, d]."""
    ck, cv, sk, sv = split(cache, d)
    return values(unpack(ck), sk, k_scale), values(unpack(cv), sv, v_scale)


def random_cache(seed, nb, Hkv, d, k_scale=1.0, v_scale=1.0, gain=1.0):
    """A cache that holds quantised normal keys (times gain) and values."""
    k = synth.bf16_bits_to_f32(synth.normal_bf16(seed, 1, (nb, Hkv, 16, d))) * np.float32(gain)
    v = synth.bf16_bits_to_f32(synth.normal_bf16(seed, 2, (nb, Hkv, 16, d)))
    cache = np.empty((nb, Hkv, 18 * d), np.uint8)
    (ck, sk), (cv, sv) = quantise(k, k_scale), quantise(v, v_scale)
    for view, x in zip(split(cache, d), (pack(ck), pack(cv), sk, sv)):
        view[...] = x
    return cache


def decode(q, cache, table, lens, d, scale, k_scale, v_scale):
    """out [S,Hq,d], lse [S,Hq], largest |score| [S,Hq], weighted mean and largest
    of |v| [S,Hq,d], fp64; blocks with a table entry out of range are left out."""
    S, Hq = q.shape[:2]
    nb, Hkv = cache.shape[:2]
    q = synth.bf16_bits_to_f32(q).astype(np.float64)
    out, lse = np.zeros((S, Hq, d)), np.full((S, Hq), -np.inf)
    big, mean, most = np.zeros((S, Hq)), np.zeros((S, Hq, d)), np.zeros((S, Hq, d))
    G = Hq // Hkv
    for s in range(S):
        n = int(lens[s])
        if n == 0:
            continue
        blk = table[s, :(n + 15) // 16]
        seen = np.repeat((blk >= 0) & (blk < nb), 16)[:n]
        k, v = cache_values(cache[np.clip(blk, 0, nb - 1)], d, k_scale, v_scale)
        k, v = (x.transpose(1, 0, 2, 3).reshape(Hkv, -1, d)[:, :n][:, seen] for x in (k, v))
        if not seen.any():
            continue
        for h in range(Hq):
            x = k[h // G] @ q[s, h] * scale
            m = x.max()
            p = np.exp(x - m)
            out[s, h] = p @ v[h // G] / p.sum()
            mean[s, h] = p @ np.abs(v[h // G]) / p.sum()
            most[s, h] = np.abs(v[h // G]).max(0)
            lse[s, h] = m + np.log(p.sum())
            big[s, h] = np.abs(x).max()
    return out, lse, big, mean, most


def cos_sin(positions, sections, base, per_axis):
    """fp64 cosines and sines [..., d/2] of positions int [axes, ...]."""
    half = sum(sections)
    cols, done = [], 0
    for a, n in enumerate(sections):
        for j in range(n):
            power = j / n if per_axis else (done + j) / half
            cols.append(np.asarray(positions[a], np.float64) * float(np.float32(base)) ** -power)
        done += n
    ang = np.stack(cols, -1)
    return np.cos(ang), np.sin(ang)


def turn(x, c, s):
    """x [..., d] turned (c, s broadcastable to [..., d/2]) in x's precision."""
    h = x.shape[-1] // 2
    a, b = x[..., :h], x[..., h:]
    return np.concatenate([a * c - b * s, b * c + a * s], -1)
