"""Operators around the 4-bit paged KV cache and rotary positions with several
axes: the cases they are measured on, with a plain form of each.

  rope    attn_rope_axes: queries and keys turned by several position axes
          (time, height, width), and the transposed turn that their gradients take
  append  attn_rope_cache_write_fp4: new tokens rotated, quantised to 4 bits and
          stored into the paged cache; attn_cache_read_fp4 gives the stored values
  read    attn_cache_read_fp4: cached tokens back as bf16, for attn_fwd to
          prefill a further chunk over them
  decode  attn_decode_paged_fp4: one query token per sequence against the cache

The cache is uint8 [num_blocks, Hkv, 18 d].  The 18 d bytes of one block of 16
tokens and one KV head are: key codes [16][d/2], value codes [16][d/2], key
scales [16][d/16], value scales [16][d/16].  A code is an e2m1 number (two to a
byte, the even column in the low four bits), a scale an e4m3 number for 16
neighbouring columns; the value is code * scale * k_scale (or v_scale).
"""
import math

import torch

own = False

BASE = 500000.0
LUT = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------- cases
def _rope(name, B, N, Hq, Hkv, d, sections, per_axis=False, inverse=False, heads_first=False):
    return dict(name=name, op="rope", B=B, N=N, Hq=Hq, Hkv=Hkv, d=d, sections=sections,
                per_axis=per_axis, inverse=inverse, heads_first=heads_first)


def _append(name, S, new, lo, hi, Hq, Hkv, d, sections):
    return dict(name=name, op="append", S=S, new=new, lo=lo, hi=hi, Hq=Hq, Hkv=Hkv, d=d,
                sections=sections)


def _read(name, S, lo, hi, Hkv, d):
    return dict(name=name, op="read", S=S, lo=lo, hi=hi, Hkv=Hkv, d=d)


def _decode(name, S, lo, hi, Hq, Hkv, d):
    return dict(name=name, op="decode", S=S, lo=lo, hi=hi, Hq=Hq, Hkv=Hkv, d=d)


def listed():
    return [
        # one token for each of 64 sequences, as in a serving step
        _rope("rope step 64x1", 64, 1, 32, 8, 128, "16,24,24"),
        # the 2048-token prefill's heads, views of one fused projection
        _rope("rope prompt 2048", 1, 2048, 32, 8, 128, "16,24,24"),
        # gradients of a batched training step, a spectrum of its own for each axis
        _rope("rope gradient 8x4096", 8, 4096, 32, 32, 128, "22,21,21", per_axis=True, inverse=True,
              heads_first=True),
        # two axes (an image), odd length, heads of 64
        _rope("rope image 3x1001 d64", 3, 1001, 14, 2, 64, "16,16", per_axis=True),
        # a serving step's new tokens, at the end of contexts of 512 to 8192 tokens
        _append("append step 64x1", 64, 1, 512, 8192, 32, 8, 128, "64"),
        # 16384 prompt tokens of 64 sequences
        _append("append prompt 64x256", 64, 256, 256, 256, 32, 8, 128, "64"),
        # an odd chunk of image and text tokens, heads of 64
        _append("append chunk 5x333 d64", 5, 333, 400, 2000, 14, 2, 64, "8,12,12"),
        # the prefix of one long conversation
        _read("read prefix 32768", 1, 32768, 32768, 8, 128),
        # short ragged prefixes, heads of 64
        _read("read ragged 3 d64", 3, 77, 999, 2, 64),
        # a serving batch: 64 sequences with contexts of 512 to 8192 tokens
        _decode("decode batch 64", 64, 512, 8192, 32, 8, 128),
        # one sequence of 32768 tokens
        _decode("decode long 32768", 1, 32768, 32768, 32, 8, 128),
        # a few short contexts, one of them possibly empty, heads of 64
        _decode("decode few short d64", 6, 0, 1500, 14, 2, 64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _sections(rng, half, most=3):
    axes = rng.randint(1, most)
    cuts = sorted(rng.sample(range(1, half), axes - 1))
    return ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [half]))


def draw(rng):
    op = rng.choice(["rope", "append", "read", "decode", "decode"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 7, 8, 12])
    Hq = Hkv * group
    if op == "rope":
        most = 8 * 4096 * 64 // (Hq + Hkv)
        B = _log(rng, 1, 64)
        c = _rope("", B, _log(rng, 1, max(1, min(32768, most // B))), Hq, Hkv, d, _sections(rng, d // 2),
                  rng.random() < 0.5, rng.random() < 0.5, rng.random() < 0.5)
    elif op == "append":
        S = _log(rng, 1, 64)
        new = 1 if rng.random() < 0.3 else _log(rng, 1, max(1, 16384 // S))
        c = _append("", S, new, new, _log(rng, new, max(new, 8192)), Hq, Hkv, d, _sections(rng, d // 2))
    elif op == "read":
        S = _log(rng, 1, 64)
        hi = _log(rng, 1, 32768 // S)
        c = _read("", S, rng.randint(1, hi), hi, Hkv, d)
    else:
        S = _log(rng, 1, 128)
        hi = _log(rng, 1, min(65536, 64 * 8192 // S))
        c = _decode("", S, rng.randint(0 if S > 2 else 1, hi), hi, Hq, Hkv, d)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs
def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _keys(gen, tokens, Hkv, d):
    """Keys and values of a projection: normal, some key columns larger than others."""
    gain = torch.exp(0.7 * _normal(gen, 1, Hkv, d))
    return _normal(gen, tokens, Hkv, d) * gain, _normal(gen, tokens, Hkv, d)


def _spread(case):
    """S lengths from lo to hi."""
    S, lo, hi = case["S"], case["lo"], case["hi"]
    return [hi] if S == 1 else [lo + (hi - lo) * i // (S - 1) for i in range(S)]


def _lengths(gen, case):
    lens = torch.tensor(_spread(case), device="cuda", dtype=torch.int32)
    return lens[torch.randperm(case["S"], generator=gen, device="cuda")]


def _pages(gen, lens):
    """Block table of sequences of these lengths over a shuffled pool, unused entries -1."""
    need = (lens.long() + 15) // 16
    most, total = max(1, int(need.max())), max(1, int(need.sum()))
    order = torch.randperm(total, generator=gen, device="cuda").int()
    col = torch.arange(most, device="cuda")
    at = (need.cumsum(0) - need)[:, None] + col
    used = col < need[:, None]
    return torch.where(used, order[at.clamp(max=total - 1)], -1).int().contiguous(), total


def _image_positions(gen, axes, *shape):
    """Positions of a stream of text with images in it: the first axis counts on,
    the others run over rows and columns and start at the first one's value."""
    n = torch.arange(shape[-1], device="cuda", dtype=torch.int32).expand(*shape)
    first = torch.randint(0, 20000, shape[:-1] + (1,), generator=gen, device="cuda", dtype=torch.int32)
    rows = [first + n // 7, first + (n // 7) % 24, first + n % 37, first + n % 5]
    return (first + n).expand(1, *shape).contiguous() if axes == 1 else torch.stack(rows[:axes]).contiguous()


def _random_cache(gen, blocks, Hkv, d, k_scale, v_scale):
    """A cache as the append leaves it: quantised keys and values."""
    k, v = _keys(gen, blocks * 16, Hkv, d)
    ck, sk = _quantise(k.bfloat16().float(), k_scale)
    cv, sv = _quantise(v.bfloat16().float(), v_scale)
    return torch.cat([x.reshape(blocks, 16, Hkv, -1).transpose(1, 2).flatten(2) for x in (ck, cv, sk, sv)], dim=-1)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 2 + 1)
    s = dict(case)
    d, Hkv = case["d"], case["Hkv"]
    if "sections" in case:
        s["sections"] = tuple(int(x) for x in case["sections"].split(","))
    # as a calibration sets them: the largest group's e4m3 scale comes near 448
    s["k_scale"], s["v_scale"] = 0.0089, 0.0023
    if case["op"] == "rope":
        B, N, Hq = case["B"], case["N"], case["Hq"]
        if case["heads_first"]:
            s["q"] = _normal(gen, B, Hq, N, d).bfloat16()
            s["k"] = _normal(gen, B, Hkv, N, d).bfloat16()
        else:  # views of one fused projection [B, N, (Hq + 2 Hkv) d]
            x = _normal(gen, B, N, Hq + 2 * Hkv, d).bfloat16().transpose(1, 2)
            s["q"], s["k"] = x[:, :Hq], x[:, Hq:Hq + Hkv]
        s["positions"] = _image_positions(gen, len(s["sections"]), B, N)
        return s
    lens = _lengths(gen, case)
    s["block_table"], blocks = _pages(gen, lens)
    if case["op"] == "append":
        S, new = case["S"], case["new"]
        T = S * new
        x = _normal(gen, T, case["Hq"] + 2 * Hkv, d)
        k, v = _keys(gen, T, Hkv, d)
        x[:, case["Hq"]:case["Hq"] + Hkv], x[:, case["Hq"] + Hkv:] = k, v
        x = x.bfloat16()
        s["q"], s["k"], s["v"] = x[:, :case["Hq"]], x[:, case["Hq"]:case["Hq"] + Hkv], x[:, case["Hq"] + Hkv:]
        n = torch.arange(new, device="cuda", dtype=torch.int32)
        s["slots"] = (lens[:, None] - new + n).reshape(-1).contiguous()
        s["seq_ids"] = torch.arange(S, device="cuda", dtype=torch.int32).repeat_interleave(new).contiguous()
        axes = len(s["sections"])
        if axes == 1:
            s["positions"] = s["slots"].reshape(1, T)
        else:
            s["positions"] = _image_positions(gen, axes, S, new).reshape(axes, T).contiguous()
        s["cache"] = torch.zeros(blocks, Hkv, 18 * d, device="cuda", dtype=torch.uint8)
        return s
    s["cache"] = _random_cache(gen, blocks, Hkv, d, s["k_scale"], s["v_scale"])
    if case["op"] == "read":
        n = lens.long()
        first = (n.cumsum(0) - n).repeat_interleave(n)
        s["seq_ids"] = torch.arange(case["S"], device="cuda", dtype=torch.int32).repeat_interleave(n).contiguous()
        s["slots"] = (torch.arange(int(n.sum()), device="cuda") - first).int().contiguous()
        return s
    s["ctx_lens"] = lens
    s["q"] = _normal(gen, case["S"], case["Hq"], d).bfloat16()
    return s


# -------------------------------------------------------------- plain forms
def _frequencies(s):
    """Frequency and axis of each of the d/2 pairs."""
    half, n = s["d"] // 2, torch.tensor(s["sections"], device="cuda")
    axis = torch.arange(len(s["sections"]), device="cuda").repeat_interleave(n)
    i = torch.arange(half, device="cuda", dtype=torch.float64)
    if s.get("per_axis"):
        power = (i - (n.cumsum(0) - n)[axis]) / n[axis]
    else:
        power = i / half
    return torch.tensor(BASE, dtype=torch.float64, device="cuda") ** -power, axis


def _cos_sin(s):
    """[..., d/2] for positions [axes, ...]; the angles in 64 bits, far positions need them."""
    theta, axis = _frequencies(s)
    angle = s["positions"].movedim(0, -1)[..., axis].double() * theta
    return torch.cos(angle).float(), torch.sin(angle).float()


def _turn(x, cos, sin):
    a, b = x.float().chunk(2, dim=-1)
    return torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)


def _quantise(x, scale):
    """Codes (two to a byte) and e4m3 scales of x [..., d] in 32 bits, d innermost."""
    g = torch.tensor(scale, device=x.device, dtype=torch.float32)
    x = x.reshape(*x.shape[:-1], -1, 16)
    s8 = (x.abs().amax(-1) / (g * 6)).clamp(max=448.0).to(torch.float8_e4m3fn)
    y = x / (s8.float() * g)[..., None]
    y = torch.where((s8.float() == 0)[..., None], torch.zeros_like(y), y)
    m = y.abs()
    # nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6; ties to the even code
    code = ((m > 0.25).int() + (m >= 0.75).int() + (m > 1.25).int() + (m >= 1.75).int()
            + (m > 2.5).int() + (m >= 3.5).int() + (m > 5.0).int())
    code = (code + 8 * torch.signbit(y).int()).to(torch.uint8).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), s8.view(torch.uint8)


def _dequantise(codes, scales, scale):
    lut = torch.tensor(LUT + tuple(-x for x in LUT), device=codes.device)
    x = lut[torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2).long()]
    s8 = scales.view(torch.float8_e4m3fn).float()
    g = torch.tensor(scale, device=codes.device, dtype=torch.float32)
    return (x.unflatten(-1, (-1, 16)) * s8[..., None]).flatten(-2) * g


def _span(spans, d):
    """Key codes, value codes, key scales, value scales of spans [..., 18 d]."""
    c, e = 8 * d, d
    return (spans[..., :c].unflatten(-1, (16, d // 2)), spans[..., c:2 * c].unflatten(-1, (16, d // 2)),
            spans[..., 2 * c:2 * c + e].unflatten(-1, (16, d // 16)), spans[..., 2 * c + e:].unflatten(-1, (16, d // 16)))


def _store(s, k, v):
    """k, v [T, Hkv, d] quantised and written into their slots."""
    blk = s["block_table"][s["seq_ids"].long(), (s["slots"] // 16).long()].long()
    off = (s["slots"] % 16).long()
    parts = _span(s["cache"], s["d"])
    (ck, sk), (cv, sv) = _quantise(k, s["k_scale"]), _quantise(v, s["v_scale"])
    parts[0][blk, :, off] = ck
    parts[1][blk, :, off] = cv
    parts[2][blk, :, off] = sk.contiguous()
    parts[3][blk, :, off] = sv.contiguous()


def _load(s):
    blk = s["block_table"][s["seq_ids"].long(), (s["slots"] // 16).long()].long()
    off = (s["slots"] % 16).long()
    ck, cv, sk, sv = _span(s["cache"], s["d"])
    k = _dequantise(ck[blk, :, off], sk[blk, :, off].contiguous(), s["k_scale"])
    v = _dequantise(cv[blk, :, off], sv[blk, :, off].contiguous(), s["v_scale"])
    return k.bfloat16(), v.bfloat16()


def _run_rope(s):
    if own:
        from exact_attention_40_gb300 import exattn
        if not s["inverse"]:
            return exattn.attn_rope_axes(s["q"], s["k"], s["positions"], s["sections"], base=BASE,
                                         per_axis=s["per_axis"])
        # the gradients go back to the projection's layout, tokens before heads
        x = torch.empty(s["B"], s["N"], s["Hq"] + s["Hkv"], s["d"], device="cuda", dtype=torch.bfloat16).transpose(1, 2)
        return exattn.attn_rope_axes(s["q"], s["k"], s["positions"], s["sections"], base=BASE,
                                     per_axis=s["per_axis"], inverse=True, q_out=x[:, :s["Hq"]], k_out=x[:, s["Hq"]:])
    cos, sin = _cos_sin(s)
    cos, sin = cos[:, None], sin[:, None]
    if s["inverse"]:
        sin = -sin
    return _turn(s["q"], cos, sin).bfloat16(), _turn(s["k"], cos, sin).bfloat16()


def _run_append(s):
    if own:
        from exact_attention_40_gb300 import exattn
        q = exattn.attn_rope_cache_write_fp4(s["q"], s["k"], s["v"], s["seq_ids"], s["slots"], s["positions"],
                                             s["block_table"], s["cache"], s["sections"], base=BASE,
                                             k_scale=s["k_scale"], v_scale=s["v_scale"])
        k, v = exattn.attn_cache_read_fp4(s["cache"], s["seq_ids"], s["slots"], s["block_table"],
                                          k_scale=s["k_scale"], v_scale=s["v_scale"])
        return {"q": q, "k": k, "v": v}
    cos, sin = _cos_sin(s)
    cos, sin = cos[:, None], sin[:, None]
    _store(s, _turn(s["k"], cos, sin), s["v"].float())
    k, v = _load(s)
    return {"q": _turn(s["q"], cos, sin).bfloat16(), "k": k, "v": v}


def _run_read(s):
    if own:
        from exact_attention_40_gb300 import exattn
        return exattn.attn_cache_read_fp4(s["cache"], s["seq_ids"], s["slots"], s["block_table"],
                                          k_scale=s["k_scale"], v_scale=s["v_scale"])
    return _load(s)


def _run_decode(s):
    if own:
        from exact_attention_40_gb300 import exattn
        return exattn.attn_decode_paged_fp4(s["q"], s["cache"], s["block_table"], s["ctx_lens"],
                                            k_scale=s["k_scale"], v_scale=s["v_scale"])
    d, Hkv = s["d"], s["Hkv"]
    S, Hq = s["q"].shape[:2]
    ck, cv, sk, sv = _span(s["cache"][s["block_table"].clamp(min=0).long()], d)  # [S, blocks, Hkv, 16, ...]
    k = _dequantise(ck, sk.contiguous(), s["k_scale"]).transpose(1, 2).flatten(2, 3)
    v = _dequantise(cv, sv.contiguous(), s["v_scale"]).transpose(1, 2).flatten(2, 3)
    q = s["q"].float().view(S, Hkv, Hq // Hkv, d)
    x = torch.matmul(q, k.transpose(-1, -2)) / math.sqrt(d)
    seen = torch.arange(x.shape[-1], device="cuda") < s["ctx_lens"][:, None]
    x = torch.where(seen[:, None, None], x, -torch.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top == -torch.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    v = torch.where(seen[:, None, :, None], v, 0.0)
    out = torch.matmul(p, v) / torch.where(total == 0, 1.0, total)
    return out.reshape(S, Hq, d).bfloat16(), (top + torch.log(total)).reshape(S, Hq)


def run(state):
    return {"rope": _run_rope, "append": _run_append, "read": _run_read, "decode": _run_decode}[state["op"]](state)


# ------------------------------------------------- the definition in 64 bits
def _exact_turn(x, s, inverse=False):
    """x [..., d] with positions [axes, ...]: pair i as a complex number times exp(i angle)."""
    x = x.double()
    half = x.shape[-1] // 2
    angle = []
    for a, n in enumerate(s["sections"]):
        done = sum(s["sections"][:a])
        for j in range(n):
            power = j / n if s.get("per_axis") else (done + j) / half
            angle.append(s["positions"][a].double() * BASE ** -power)
    angle = torch.stack(angle, dim=-1)
    turn = torch.polar(torch.ones_like(angle), -angle if inverse else angle).unsqueeze(-3 if x.dim() == 4 else -2)
    z = torch.complex(x[..., :half], x[..., half:]) * turn
    return torch.cat([z.real, z.imag], dim=-1)


def _exact_stored(x, scale):
    """The value that 4 bits and an e4m3 scale for 16 columns keep of x."""
    g = float(torch.tensor(scale, dtype=torch.float32))
    x = x.unflatten(-1, (-1, 16))
    t = x.abs().amax(-1, keepdim=True) / (6 * g)
    step = torch.exp2(torch.floor(torch.log2(t.clamp(min=2.0 ** -6))) - 3)
    s8 = (torch.round(t / step) * step).clamp(max=448.0)
    y = x / torch.where(s8 == 0, 1.0, s8 * g)
    m = y.abs().clamp(max=6.0)
    step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0))
    return (torch.sign(y) * torch.round(m / step) * step * s8 * g).flatten(-2)


def _exact_token(s, seq, n):
    """Keys and values [n, Hkv, d] of a sequence's first n tokens."""
    d = s["d"]
    lut = [LUT[c & 7] * (-1 if c & 8 else 1) for c in range(16)]
    pair = torch.tensor([(lut[b & 15], lut[b >> 4]) for b in range(256)], dtype=torch.float64, device="cuda")
    e4m3 = []
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        e4m3.append(math.nan if b & 127 == 127 else -x if b & 128 else x)
    e4m3 = torch.tensor(e4m3, dtype=torch.float64, device="cuda")
    rows = s["cache"][s["block_table"][seq, :(n + 15) // 16].long()].long()  # [blocks, Hkv, 18 d]
    both = []
    for codes, scales, g in ((rows[..., :8 * d], rows[..., 16 * d:17 * d], s["k_scale"]),
                             (rows[..., 8 * d:16 * d], rows[..., 17 * d:], s["v_scale"])):
        x = pair[codes].reshape(*codes.shape[:2], 16, d // 16, 16)
        x = x * e4m3[scales].reshape(*codes.shape[:2], 16, d // 16, 1) * float(torch.tensor(g, dtype=torch.float32))
        both.append(x.flatten(-2).transpose(1, 2).flatten(0, 1)[:n])
    return both


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_turn(s["q"], s, s["inverse"]), _exact_turn(s["k"], s, s["inverse"])
    if case["op"] == "append":
        return {"q": _exact_turn(s["q"], s), "k": _exact_stored(_exact_turn(s["k"], s), s["k_scale"]),
                "v": _exact_stored(s["v"].double(), s["v_scale"])}
    S = case["S"]
    if case["op"] == "read":
        n = torch.bincount(s["seq_ids"].long(), minlength=S).tolist()
        rows = [_exact_token(s, i, n[i]) for i in range(S)]
        return torch.cat([r[0] for r in rows]), torch.cat([r[1] for r in rows])
    outs, lses = [], []
    for i, n in enumerate(s["ctx_lens"].tolist()):
        k, v = _exact_token(s, i, n)
        q = s["q"][i].double().unflatten(0, (case["Hkv"], -1))
        x = torch.einsum("hgd,nhd->hgn", q, k) / math.sqrt(case["d"])
        lse = torch.logsumexp(x, -1)
        w = torch.exp(x - lse[..., None])
        outs.append(torch.einsum("hgn,nhd->hgd", w, v).flatten(0, 1))
        lses.append(lse.flatten())
    return torch.stack(outs), torch.stack(lses)


# -------------------------------------------------------------------- work
def work(case):
    d, Hkv, op = case["d"], case["Hkv"], case["op"]
    tokens = 0 if op == "rope" else sum(_spread(case))
    pair = 2 * (d // 2 + d // 16)  # bytes of one token's key and value for one KV head
    if op == "rope":
        n = case["B"] * case["N"]
        rows = n * (case["Hq"] + Hkv)
        return {"bytes": rows * d * 4 + n * 4 * len(case["sections"].split(",")), "flops": 3.0 * rows * d}
    if op == "append":
        T = case["S"] * case["new"]
        write = T * (case["Hq"] * d * 4 + Hkv * (d * 4 + pair) + 16)
        return {"bytes": write + T * Hkv * (pair + d * 4), "flops": 3.0 * T * (case["Hq"] + 3 * Hkv) * d}
    if op == "read":
        T = tokens
        return {"bytes": T * (Hkv * (pair + d * 4) + 8), "flops": 4.0 * T * Hkv * d}
    q = case["S"] * case["Hq"] * (d * 4 + 4)
    return {"bytes": tokens * (Hkv * pair + 0.25) + q, "flops": 4.0 * tokens * case["Hq"] * d}
