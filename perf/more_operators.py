"""Operators of the 8-bit paged KV cache: the cases they are measured on, with a
plain form of each.

  append  attn_rope_cache_write_fp8: new tokens rotated, quantised to 8 bits and
          stored into the paged cache; attn_cache_read_fp8 gives what the blocks that
          were written then hold
  read    attn_cache_read_fp8: cached tokens back as bf16, for attn_fwd to
          prefill a further chunk over them
  decode  attn_decode_paged_fp8: one query token of each sequence, or a few,
          against the cache

The cache is uint8 [num_blocks, Hkv, 32 d + 32].  The bytes of one block of 16 tokens
and one KV head are: key codes (16 d), value codes (16 d), the key scale and the value
scale (fp32), 24 unused.  A code is an e4m3 number, a scale a power of two; the value
is code * scale.  Token n's column c of a tensor's codes is byte
n d + 16 ((c / 16) ^ (n d / 128 % (d / 16))) + c % 16: its row's pieces of 16 bytes in
an order that changes with the row.

A block's scale is the smallest power of two (2^-117 to 2^119) with which its largest
finite magnitude is at most 448.  It grows with what a call adds, and the codes
already there are then rounded to the larger scale; a call that writes a block's
place 0 starts it anew.
"""
import math

import torch

own = False

BASE = 500000.0
LOW, HIGH = -117, 119  # exponents of the scales


# ------------------------------------------------------------------- cases
def _append(name, S, new, least, lo, hi, Hq, Hkv, d, sections, first=0):
    """Sequence i gets least .. new tokens after lo .. hi cached ones; with `first`, the
    first sequence gets that many after none instead."""
    return dict(name=name, op="append", S=S, new=new, least=least, lo=lo, hi=hi, Hq=Hq, Hkv=Hkv, d=d,
                sections=sections, first=first)


def _read(name, S, lo, hi, Hkv, d):
    return dict(name=name, op="read", S=S, lo=lo, hi=hi, Hkv=Hkv, d=d)


def _decode(name, S, lo, hi, Hq, Hkv, d, queries=1):
    return dict(name=name, op="decode", S=S, lo=lo, hi=hi, Hq=Hq, Hkv=Hkv, d=d, queries=queries)


def listed():
    return [
        # a serving step's new tokens, at the end of contexts of 512 to 8192 tokens
        _append("append step 64x1", 64, 1, 1, 511, 8191, 32, 8, 128, "64"),
        # 16384 prompt tokens of 64 sequences
        _append("append prompt 64x256", 64, 256, 256, 0, 0, 32, 8, 128, "64"),
        # a prompt's chunk in one batch with the single tokens of 63 sequences
        _append("append mixed 2048+63", 64, 1, 1, 511, 8191, 32, 8, 128, "64", first=2048),
        # ragged chunks of image and text tokens that start and end inside blocks, heads of 64
        _append("append chunk 5x1-333 d64", 5, 333, 1, 67, 1667, 14, 2, 64, "8,12,12"),
        # the prefix of one long conversation
        _read("read prefix 32768", 1, 32768, 32768, 8, 128),
        # short ragged prefixes, heads of 64
        _read("read ragged 3 d64", 3, 77, 999, 2, 64),
        # a serving batch: 64 sequences with contexts of 512 to 8192 tokens
        _decode("decode batch 64", 64, 512, 8192, 32, 8, 128),
        # all contexts full
        _decode("decode full 64x8192", 64, 8192, 8192, 32, 8, 128),
        # one sequence of 32768 tokens
        _decode("decode long 32768", 1, 32768, 32768, 32, 8, 128),
        # a few short contexts, one of them empty, heads of 64
        _decode("decode few short d64", 6, 0, 1500, 14, 2, 64),
        # four tokens of each sequence at once, three of them drafted
        _decode("decode drafts 32x4", 32, 512, 8192, 32, 8, 128, queries=4),
        # a ragged batch of a model without shared heads, heads of 64
        _decode("decode heads 128 d64", 128, 1, 2000, 8, 8, 64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _sections(rng, half, most=3):
    axes = rng.randint(1, most)
    cuts = sorted(rng.sample(range(1, half), axes - 1))
    return ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [half]))


def draw(rng):
    op = rng.choice(["append", "append", "read", "decode", "decode", "decode"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 7, 8, 12])
    if op == "append":
        S = _log(rng, 1, 64)
        new = 1 if rng.random() < 0.3 else _log(rng, 1, max(1, 16384 // S))
        lo = rng.choice([0, rng.randint(0, 4000)])
        c = _append("", S, new, rng.choice([new, rng.randint(1, new)]), lo, lo + rng.choice([0, rng.randint(0, 4000)]),
                    Hq, Hkv, d, _sections(rng, d // 2), first=_log(rng, 1, 4096) if rng.random() < 0.2 else 0)
    elif op == "read":
        S = _log(rng, 1, 64)
        hi = _log(rng, 1, 32768 // S)
        c = _read("", S, rng.randint(1, hi), hi, Hkv, d)
    else:
        S = _log(rng, 1, 128)
        hi = _log(rng, 1, min(65536, 64 * 8192 // S))
        c = _decode("", S, rng.randint(0 if S > 2 else 1, hi), hi, Hq, Hkv, d, rng.choice([1, 1, 1, 2, 3, 4, 6]))
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs
def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _keys(gen, tokens, Hkv, d):
    """Keys and values of a projection: normal, some key columns larger than others."""
    gain = torch.exp(0.7 * _normal(gen, 1, Hkv, d))
    return _normal(gen, tokens, Hkv, d) * gain, _normal(gen, tokens, Hkv, d)


def _range(n, lo, hi):
    """n numbers from lo to hi."""
    return [hi] if n == 1 else [lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _rows(case):
    """Cached and new tokens of each sequence of an append."""
    S = case["S"]
    rows = list(zip(_range(S, case["lo"], case["hi"]), _range(S, case["least"], case["new"])))
    if case["first"]:
        rows[0] = (0, case["first"])
    return rows


def _pages(gen, lens):
    """Block table of sequences of these lengths over a shuffled pool, unused entries -1."""
    need = (lens.long() + 15) // 16
    most, total = max(1, int(need.max())), max(1, int(need.sum()))
    order = torch.randperm(total, generator=gen, device="cuda").int()
    col = torch.arange(most, device="cuda")
    at = (need.cumsum(0) - need)[:, None] + col
    used = col < need[:, None]
    return torch.where(used, order[at.clamp(max=total - 1)], -1).int().contiguous(), total


def _image_positions(gen, axes, T):
    """Positions of a stream of text with images in it: the first axis counts on,
    the others run over rows and columns and start at the first one's value."""
    n = torch.arange(T, device="cuda", dtype=torch.int32)
    first = torch.randint(0, 20000, (1,), generator=gen, device="cuda", dtype=torch.int32)
    return torch.stack([first + n // 7, first + (n // 7) % 24, first + n % 37][:axes]).contiguous()


def _random_cache(gen, blocks, Hkv, d):
    """A cache as appends leave it: quantised keys and values."""
    cache = torch.zeros(blocks, Hkv, 32 * d + 32, device="cuda", dtype=torch.uint8)
    codes, scales = _parts(cache, d)
    place = _place(d, "cuda").flatten()
    for which, x in enumerate(_keys(gen, blocks * 16, Hkv, d)):
        x = x.bfloat16().float().reshape(blocks, 16, Hkv, d).transpose(1, 2)
        s = _scale_for(x.abs().amax((2, 3)))
        codes[:, :, which, place] = _code(x, s[..., None, None]).flatten(2)
        scales[:, :, which] = s
    return cache


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 2 + 1)
    s = dict(case)
    S, d, Hkv = case["S"], case["d"], case["Hkv"]
    shuffle = torch.randperm(S, generator=gen, device="cuda")
    if case["op"] != "append":
        lens = torch.tensor(_range(S, case["lo"], case["hi"]), device="cuda", dtype=torch.int32)[shuffle]
        s["block_table"], blocks = _pages(gen, lens)
        s["cache"] = _random_cache(gen, blocks, Hkv, d)
        if case["op"] == "read":
            s["seq_ids"], s["slots"] = _tokens(torch.zeros_like(lens), lens)
            return s
        s["ctx_lens"] = lens
        n = case["queries"]
        s["q"] = _normal(gen, S, n, case["Hq"], d).bfloat16()
        if n == 1:
            s["q"] = s["q"][:, 0].contiguous()
        return s
    cached, new = torch.tensor(_rows(case), device="cuda", dtype=torch.int32)[shuffle].unbind(1)
    s["ctx_lens"] = (cached + new).contiguous()
    s["block_table"], blocks = _pages(gen, s["ctx_lens"])
    s["cache"] = _random_cache(gen, blocks, Hkv, d)
    starts = torch.zeros(S + 1, device="cuda", dtype=torch.int32)
    starts[1:] = new.cumsum(0)
    T, Hq = int(starts[-1]), case["Hq"]
    s["token_starts"] = starts if T > S else None  # a token for each sequence needs none
    x = _normal(gen, T, Hq + 2 * Hkv, d)  # one fused projection, of which q, k and v are views
    x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:] = _keys(gen, T, Hkv, d)
    x = x.bfloat16()
    s["q"], s["k"], s["v"] = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    s["sections"] = tuple(int(n) for n in case["sections"].split(","))
    if len(s["sections"]) == 1:
        s["positions"] = _tokens(cached, s["ctx_lens"])[1][None].contiguous()
    else:
        s["positions"] = _image_positions(gen, len(s["sections"]), T)
    # what is read back: the blocks that get new tokens, from their first one on
    s["seq_ids"], s["slots"] = _tokens(cached // 16 * 16, s["ctx_lens"])
    return s


def _tokens(lo, hi):
    """Sequence and slot of the tokens lo .. hi - 1 of each sequence."""
    n = (hi - lo).long()
    first = (n.cumsum(0) - n - lo).repeat_interleave(n)
    seq = torch.arange(len(n), device="cuda", dtype=torch.int32).repeat_interleave(n)
    return seq.contiguous(), (torch.arange(int(n.sum()), device="cuda") - first).int().contiguous()


# -------------------------------------------------------------- plain forms
def _parts(cache, d):
    """Codes [blocks, Hkv, 2, 16 d] and scales [blocks, Hkv, 2] of the cache, as views."""
    codes = cache[..., :32 * d].unflatten(-1, (2, 16 * d))
    return codes, cache.view(torch.float32)[..., 8 * d:8 * d + 2]


def _place(d, device):
    """[16, d]: where a block's token n and column c lie."""
    n = torch.arange(16, device=device)[:, None]
    c = torch.arange(d, device=device)
    return n * d + 16 * ((c // 16) ^ (n * d // 128 % (d // 16))) + c % 16


def _power(e):
    """2^e in 32 bits, for the exponents of normal numbers."""
    return ((e + 127) << 23).view(torch.float32)


def _scale_for(most):
    """The power of two for a largest magnitude in 32 bits."""
    m, x = torch.frexp(most)  # most = m 2^x, m from 0.5 to below 1; 448 = 0.875 * 2^9
    e = torch.where(m <= 0.875, x - 9, x - 8)
    return _power(torch.where(most == 0, LOW, e.clamp(LOW, HIGH)).int())


def _code(x, scale):
    """e4m3 codes of x in 32 bits."""
    x = x / scale
    x = torch.where(x.abs() < torch.inf, x.clamp(-448.0, 448.0), torch.nan)
    return x.to(torch.float8_e4m3fn).view(torch.uint8)


def _value(codes, scale):
    return codes.view(torch.float8_e4m3fn).float() * scale


def _turned(x, s):
    """x [T, heads, d] turned by the tokens' positions; the angles in 64 bits, far positions need them."""
    half, n = s["d"] // 2, torch.tensor(s["sections"], device="cuda")
    axis = torch.arange(len(s["sections"]), device="cuda").repeat_interleave(n, output_size=half)
    i = torch.arange(half, device="cuda", dtype=torch.float64)
    theta = torch.tensor(BASE, dtype=torch.float64, device="cuda") ** -(i / half)
    angle = s["positions"].T[:, axis].double() * theta
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    a, b = x.float().chunk(2, dim=-1)
    return torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)


def _store(s, k, v):
    """k, v [T, Hkv, d] in 32 bits quantised and written into their slots."""
    T, d = k.shape[0], s["d"]
    starts = s["token_starts"]
    if starts is None:
        starts = torch.arange(T + 1, device="cuda", dtype=torch.int32)
    t = torch.arange(T, device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(starts, t, right=True) - 1
    slot = s["ctx_lens"][seq] - starts[seq + 1] + t
    off = (slot % 16).long()
    blk = s["block_table"][seq, (slot // 16).long()].long()
    codes, scales = _parts(s["cache"], d)
    blocks, Hkv = codes.shape[:2]
    anew = torch.zeros(blocks, device="cuda").index_reduce(0, blk, (off == 0).float(), "amax")[blk] > 0
    place = _place(d, "cuda")
    for which, x in enumerate((k, v)):
        size = torch.where(x.abs() < torch.inf, x.abs(), 0.0).amax(-1)
        most = torch.zeros(blocks, Hkv, device="cuda").index_reduce(0, blk, size, "amax")[blk]
        before = scales[blk, :, which]  # [T, Hkv]
        after = torch.where(anew[:, None], _scale_for(most), torch.maximum(before, _scale_for(most)))
        old = codes[blk, :, which]      # [T, Hkv, 16 d], each block once for each of its new tokens
        moved = _code(_value(old, before[..., None]), after[..., None])
        codes[blk, :, which] = torch.where((after > before)[..., None] & ~anew[:, None, None], moved, old)
        scales[blk, :, which] = after
        at = place[off][:, None].expand(-1, Hkv, -1)
        codes[blk[:, None, None], torch.arange(Hkv, device="cuda")[:, None], which, at] = _code(x, after[..., None])


def _load(s):
    d = s["d"]
    blk = s["block_table"][s["seq_ids"].long(), (s["slots"] // 16).long()].long()
    codes, scales = _parts(s["cache"], d)
    at = _place(d, "cuda")[(s["slots"] % 16).long()][:, None].expand(-1, codes.shape[1], -1)
    out = []
    for which in range(2):
        row = codes[blk[:, None, None], torch.arange(codes.shape[1], device="cuda")[:, None], which, at]
        out.append(_value(row, scales[blk, :, which, None]).bfloat16())
    return out


def _run_append(s):
    if own:
        from exact_attention_40_gb300 import exattn
        q = exattn.attn_rope_cache_write_fp8(s["q"], s["k"], s["v"], s["token_starts"], s["ctx_lens"], s["positions"],
                                             s["block_table"], s["cache"], s["sections"], base=BASE)
        k, v = exattn.attn_cache_read_fp8(s["cache"], s["seq_ids"], s["slots"], s["block_table"])
        return {"q": q, "k": k, "v": v}
    _store(s, _turned(s["k"], s), s["v"].float())
    k, v = _load(s)
    return {"q": _turned(s["q"], s).bfloat16(), "k": k, "v": v}


def _run_read(s):
    if own:
        from exact_attention_40_gb300 import exattn
        return exattn.attn_cache_read_fp8(s["cache"], s["seq_ids"], s["slots"], s["block_table"])
    return tuple(_load(s))


def _run_decode(s):
    if own:
        from exact_attention_40_gb300 import exattn
        return exattn.attn_decode_paged_fp8(s["q"], s["cache"], s["block_table"], s["ctx_lens"])
    d, Hkv, Hq, n = s["d"], s["Hkv"], s["Hq"], s["queries"]
    S, group = s["S"], s["Hq"] // s["Hkv"]
    codes, scales = _parts(s["cache"], d)
    pages = s["block_table"].clamp(min=0).long()  # [S, blocks]
    place = _place(d, "cuda").flatten()
    both = []
    for which in range(2):
        x = codes[pages, :, which][..., place].unflatten(-1, (16, d))  # [S, blocks, Hkv, 16, d]
        both.append(_value(x, scales[pages, :, which][..., None, None]).transpose(1, 2).flatten(2, 3))
    k, v = both
    q = s["q"].float().view(S, n, Hkv, group, d).permute(0, 2, 1, 3, 4).flatten(2, 3)  # [S, Hkv, n group, d]
    x = torch.matmul(q, k.transpose(-1, -2)) / math.sqrt(d)
    token = torch.arange(x.shape[-1], device="cuda")
    last = torch.arange(n, device="cuda") - n + 1  # the last query sees everything, each before it one less
    seen = token < (s["ctx_lens"][:, None] + last)[..., None]  # [S, n, tokens]
    x = torch.where(seen.repeat_interleave(group, 1)[:, None], x, -torch.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top == -torch.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    v = torch.where((token < s["ctx_lens"][:, None])[:, None, :, None], v, 0.0)
    out = torch.matmul(p, v) / torch.where(total == 0, 1.0, total)
    out = out.unflatten(2, (n, group)).permute(0, 2, 1, 3, 4).reshape(s["q"].shape).bfloat16()
    lse = (top + torch.log(total)).unflatten(2, (n, group)).permute(0, 2, 1, 3, 4)
    return out, lse.reshape(s["q"].shape[:-1])


def run(state):
    return {"append": _run_append, "read": _run_read, "decode": _run_decode}[state["op"]](state)


# ------------------------------------------------- the definition in 64 bits
def _exact_turn(x, s):
    """x [T, heads, d]: pair i as a complex number times exp(i angle)."""
    x = x.double()
    half = x.shape[-1] // 2
    angle = []
    for a, n in enumerate(s["sections"]):
        for j in range(n):
            angle.append(s["positions"][a].double() * BASE ** (-(sum(s["sections"][:a]) + j) / half))
    angle = torch.stack(angle, dim=-1)
    turn = torch.polar(torch.ones_like(angle), angle).unsqueeze(1)
    z = torch.complex(x[..., :half], x[..., half:]) * turn
    return torch.cat([z.real, z.imag], dim=-1)


def _exact_round(x):
    """x to the nearest e4m3 number, ties to the even one."""
    m = x.abs()
    step = torch.exp2(torch.floor(torch.log2(m.clamp(min=2.0 ** -6))) - 3)
    return torch.sign(x) * (torch.round(m / step) * step).clamp(max=448.0)


def _exact_exponent(x):
    """Exponents [blocks, Hkv] for values [blocks, 16, Hkv, d]; LOW where there is nothing."""
    most = x.abs().amax((1, 3))
    e = torch.ceil(torch.log2(torch.where(most == 0, 1.0, most) / 448.0)).clamp(LOW, HIGH)
    return torch.where(most == 0, float(LOW), e)


def _exact_blocks(s, pages):
    """Keys and values [blocks, 16, Hkv, d] and exponents [blocks, Hkv] that pages of the cache hold."""
    d = s["d"]
    e4m3 = []
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        e4m3.append(math.nan if b & 127 == 127 else -x if b & 128 else x)
    e4m3 = torch.tensor(e4m3, dtype=torch.float64, device="cuda")
    raw = s["cache"][pages.long()]  # [blocks, Hkv, 32 d + 32]
    swap = [[p ^ (n % 8 if d == 128 else n // 2 % 4) for p in range(d // 16)] for n in range(16)]
    swap = torch.tensor(swap, device="cuda")
    both = []
    for which in range(2):
        x = raw[..., which * 16 * d:(which + 1) * 16 * d].reshape(*raw.shape[:2], 16, d // 16, 16)
        x = torch.gather(x, 3, swap[None, None, :, :, None].expand_as(x))  # piece p lies where p ^ swap says
        word = raw[..., 32 * d + 4 * which:32 * d + 4 * which + 4].long()
        e = (word[..., 3] % 128 * 2 + word[..., 2] // 128 - 127).double()
        value = e4m3[x.flatten(-2).long()] * torch.exp2(e)[..., None, None]
        both.append((value.transpose(1, 2), e))
    return both


def _exact_append(s):
    d, Hkv, S = s["d"], s["Hkv"], s["S"]
    ctx = s["ctx_lens"].tolist()
    starts = list(range(S + 1)) if s["token_starts"] is None else s["token_starts"].tolist()
    ks, vs = [], []
    new = (_exact_turn(s["k"], s), s["v"].double())
    for i in range(S):
        n = starts[i + 1] - starts[i]
        first = ctx[i] - n
        b0, b1 = first // 16, (ctx[i] + 15) // 16
        held = _exact_blocks(s, s["block_table"][i, b0:b1])
        for which, out in ((0, ks), (1, vs)):
            old, e_old = held[which]
            added = torch.zeros_like(old).flatten(0, 1)
            added[first - b0 * 16:ctx[i] - b0 * 16] = new[which][starts[i]:starts[i + 1]]
            added = added.unflatten(0, (-1, 16))
            e = _exact_exponent(added)
            if first % 16:  # only the first block may hold tokens from before
                e[0] = torch.maximum(e[0], e_old[0])
            unit = torch.exp2(e)[:, None, :, None]
            row = (_exact_round(added / unit) * unit).flatten(0, 1)
            kept = (_exact_round(old / unit) * unit).flatten(0, 1)
            row[:first - b0 * 16] = kept[:first - b0 * 16]
            out.append(row[:ctx[i] - b0 * 16])
    return {"q": _exact_turn(s["q"], s), "k": torch.cat(ks), "v": torch.cat(vs)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(s)
    S = case["S"]
    if case["op"] == "read":
        rows = [_exact_blocks(s, s["block_table"][i][:(n + 15) // 16])
                for i, n in enumerate(torch.bincount(s["seq_ids"].long(), minlength=S).tolist())]
        lens = torch.bincount(s["seq_ids"].long(), minlength=S).tolist()
        return tuple(torch.cat([r[which][0].flatten(0, 1)[:n] for r, n in zip(rows, lens)]) for which in range(2))
    outs, lses = [], []
    n_q = case["queries"]
    q_all = s["q"].double().reshape(S, n_q, case["Hkv"], -1, case["d"])
    for i, ctx in enumerate(s["ctx_lens"].tolist()):
        (k, _), (v, _) = _exact_blocks(s, s["block_table"][i, :(ctx + 15) // 16])
        k, v = k.flatten(0, 1), v.flatten(0, 1)
        for j in range(n_q):
            n = max(0, ctx - (n_q - 1 - j))
            x = torch.einsum("hgd,nhd->hgn", q_all[i, j], k[:n]) / math.sqrt(case["d"])
            lse = torch.logsumexp(x, -1) if n else torch.full(x.shape[:2], -torch.inf, device="cuda", dtype=torch.float64)
            w = torch.exp(x - lse[..., None])
            outs.append(torch.einsum("hgn,nhd->hgd", w, v[:n]).flatten(0, 1))
            lses.append(lse.flatten())
    return torch.stack(outs).reshape(s["q"].shape), torch.stack(lses).reshape(s["q"].shape[:-1])


# -------------------------------------------------------------------- work
def work(case):
    d, Hkv, op = case["d"], case["Hkv"], case["op"]
    if op == "append":
        rows = _rows(case)
        T = sum(new for _, new in rows)
        back = sum(cached % 16 + new for cached, new in rows)
        # per token: queries in and out, keys and values in, their codes out, its position; then
        # what is read back, with the scales of a block spread over its tokens
        write = T * (case["Hq"] * d * 4 + Hkv * (d * 4 + 2 * d) + 4 * len(case["sections"].split(",")))
        return {"bytes": write + back * (Hkv * (2 * d + d * 4 + 0.5) + 8), "flops": 3.0 * T * (case["Hq"] + 2 * Hkv) * d}
    tokens = sum(_range(case["S"], case["lo"], case["hi"]))
    if op == "read":
        return {"bytes": tokens * (Hkv * (2 * d + d * 4 + 0.5) + 8), "flops": 2.0 * tokens * Hkv * d}
    rows = case["S"] * case["queries"] * case["Hq"]
    return {"bytes": tokens * (Hkv * (2 * d + 0.5) + 0.25) + rows * (d * 4 + 4),
            "flops": 4.0 * tokens * case["queries"] * case["Hq"] * d}
