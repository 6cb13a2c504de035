"""attn_rope_axes against the rotation in 64 bits.

Bar, from the arithmetic: cosine and sine are within 2^-24 of the exact ones
(a rounding of at most 2^-25 and 2^-29 before it, rounded up), the products
and their sum round once each (2^-24 relative to the products), and the result
rounds once to bf16 (2^-8): |y - ref| <= 2^-8 |ref| + 2^-21 (|x_i| + |x_(i+d/2)|),
eight times the fp32 part's sum."""
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


def f64(t):
    return t.double().cpu().numpy()


def positions(seed, axes, B, N, lo=-50, hi=5000):
    u = synth.uniform01(seed, axes * B * N).reshape(axes, B, N)
    return (lo + np.floor(u * (hi - lo))).astype(np.int32)


def check(got, x, pos, sections, base, per_axis, inverse, label):
    c, s = ref.cos_sin(pos, sections, base, per_axis)
    c, s = c[:, None], (-s if inverse else s)[:, None]
    x = f64(x)
    want = ref.turn(x, c, s)
    h = x.shape[-1] // 2
    pair = np.abs(x[..., :h]) + np.abs(x[..., h:])
    bar = 2.0 ** -8 * np.abs(want) + 2.0 ** -21 * np.concatenate([pair, pair], -1)
    err = np.abs(f64(got) - want)
    assert (err <= bar).all(), "%s: worst %.3e at %s" % (label, (err - bar).max(), np.unravel_index((err - bar).argmax(), err.shape))


def inputs(torch, dev, seed, B, N, Hq, Hkv, d):
    q = to_dev(synth.normal_bf16(seed, 1, (B, Hq, N, d)), dev)
    k = to_dev(synth.normal_bf16(seed, 2, (B, Hkv, N, d)), dev)
    return q, k


CASES = [  # B, N, Hq, Hkv, d, sections, per_axis
    (1, 1, 1, 1, 128, (64,), False),
    (1, 1, 40, 8, 128, (16, 24, 24), False),
    (64, 1, 32, 8, 128, (16, 24, 24), False),
    (1, 333, 4, 2, 64, (8, 12, 12), False),
    (3, 77, 7, 1, 64, (16, 16), True),
    (2, 1001, 3, 3, 128, (22, 21, 21), True),
    (1, 40, 2, 1, 256, (32, 32, 32, 32), True),
    (2, 19, 5, 3, 16, (1, 7), False),
    (1, 90, 3, 2, 48, (8, 8, 8), True),
    (1, 50, 2, 2, 96, (0, 48), False),
    (2, 3000, 2, 1, 112, (56,), True),
    (1, 5000, 1, 0, 256, (128,), False),  # one head and many tokens: the largest tiles
    (1, 60000, 0, 1, 16, (8,), True),
]


@pytest.mark.parametrize("case", CASES, ids=[str(c).replace(" ", "") for c in CASES])
@pytest.mark.parametrize("inverse", [False, True])
def test_against_64_bits(env, case, inverse):
    torch, ex, dev = env
    B, N, Hq, Hkv, d, sections, per_axis = case
    q, k = inputs(torch, dev, 300, B, N, Hq, Hkv, d)
    pos = positions(7, len(sections), B, N)
    qo, ko = ex.attn_rope_axes(q, k, to_dev(pos, dev), sections, base=10000.0, per_axis=per_axis, inverse=inverse)
    assert qo.is_contiguous() and ko.is_contiguous()
    check(qo, q, pos, sections, 10000.0, per_axis, inverse, "q")
    check(ko, k, pos, sections, 10000.0, per_axis, inverse, "k")


def test_far_and_negative_positions(env):
    torch, ex, dev = env
    pos = np.array([[[0, 1, -1, 2 ** 20, -2 ** 20, 2 ** 24 + 1, 123456789]]], np.int32)
    q, k = inputs(torch, dev, 301, 1, 7, 2, 1, 128)
    qo, ko = ex.attn_rope_axes(q, k, to_dev(pos, dev), (64,))
    # fp64 angles of 1.2e8 rad are themselves 1e-8 off; the bar covers that
    check(qo, q, pos, (64,), 500000.0, False, False, "q")
    # extreme positions: the turn of -2^31 is the reverse of the turn of 2^31
    ends = torch.tensor([[[2 ** 31 - 1, -2 ** 31 + 1]]], device=dev, dtype=torch.int32)
    x = q[:, :, :1].expand(1, 2, 2, 128)
    a, _ = ex.attn_rope_axes(x, x, ends, (64,))
    b, _ = ex.attn_rope_axes(x, x, ends.flip(-1), (64,), inverse=True)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_cosines_are_the_nearest_fp32(env):
    """A key pair (1, 0) comes out as (cos, sin); read through the 4-bit append the
    fp32 result is not visible, so the bf16 output is compared: it is the
    rounding of the exact value but for ties' neighbourhoods."""
    torch, ex, dev = env
    N = 20000
    x = torch.zeros((1, 1, N, 128), device=dev, dtype=torch.bfloat16)
    x[..., :64] = 1.0
    pos = torch.arange(N, device=dev, dtype=torch.int32).view(1, 1, N)
    y, _ = ex.attn_rope_axes(x, x, pos, (64,))
    c, s = ref.cos_sin(np.arange(N)[None], (64,), 500000.0, False)
    want = torch.from_numpy(np.concatenate([c, s], -1)).float().bfloat16().to(dev)
    assert (y[0, 0] != want).float().mean().item() < 2e-4


def test_strided_views_in_place_and_untouched_rest(env):
    torch, ex, dev = env
    B, N, Hq, Hkv, d, sections = 2, 65, 6, 2, 64, (10, 10, 12)
    qkv = to_dev(synth.normal_bf16(302, 0, (B, N, Hq + 2 * Hkv, d)), dev)
    x = qkv.transpose(1, 2)
    q, k = x[:, :Hq], x[:, Hq:Hq + Hkv]
    pos = positions(8, 3, B, N)
    pd = to_dev(pos, dev)
    qo, ko = ex.attn_rope_axes(q, k, pd, sections)
    check(qo, q, pos, sections, 500000.0, False, False, "q of a view")
    before = qkv.clone()
    q2, k2 = ex.attn_rope_axes(q, k, pd, sections, q_out=q, k_out=k)
    assert q2 is q and k2 is k
    assert torch.equal(q.contiguous().view(torch.int16), qo.view(torch.int16))
    assert torch.equal(k.contiguous().view(torch.int16), ko.view(torch.int16))
    assert torch.equal(qkv[:, :, Hq + Hkv:], before[:, :, Hq + Hkv:])  # the values
    # a new view object of the same rows is in place too; other strides on the same address are refused
    ex.attn_rope_axes(q, k, pd, sections, q_out=qkv.transpose(1, 2)[:, :Hq], k_out=k)
    with pytest.raises(ex.ExattnError):
        ex.attn_rope_axes(q, k, pd, sections, q_out=qkv.view(-1)[:B * Hq * N * d].view(B, Hq, N, d))


def test_broadcast_positions_and_inputs(env):
    torch, ex, dev = env
    B, N, H, d = 3, 33, 4, 64
    q, k = inputs(torch, dev, 303, B, N, H, 1, d)
    pos = positions(9, 2, 1, N)
    want = ex.attn_rope_axes(q, k.expand(B, H, N, d).contiguous(), to_dev(np.repeat(pos, B, 1), dev), (16, 16))
    got = ex.attn_rope_axes(q, k.expand(B, H, N, d), to_dev(pos[:, 0], dev), (16, 16))
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    # positions cut out of a larger, transposed tensor
    wide = torch.zeros((N, 5, B), device=dev, dtype=torch.int32)
    view = wide.permute(1, 2, 0)[1:3]
    view.copy_(to_dev(np.repeat(pos, B, 1), dev))
    got = ex.attn_rope_axes(q, k.expand(B, H, N, d), view, (16, 16))
    assert torch.equal(got[0].view(torch.int16), want[0].view(torch.int16))
    with pytest.raises(ex.ExattnError):  # an output that is one row many times over
        ex.attn_rope_axes(q, k, to_dev(pos[:, 0], dev), (16, 16), k_out=torch.empty_like(k[:, :, :1]).expand_as(k))


def test_gradient_against_differences(env):
    """The reverse turn is the gradient: for the scalar f = sum(w * turn(x)), it
    equals central differences of the 64-bit forward (exact, f is linear)."""
    torch, ex, dev = env
    sections, d, N = (3, 5), 16, 6
    x = synth.bf16_bits_to_f32(synth.normal_bf16(304, 1, (1, 1, N, d))).astype(np.float64)
    wb = synth.normal_bf16(304, 2, (1, 1, N, d))
    w = synth.bf16_bits_to_f32(wb).astype(np.float64)
    pos = positions(10, 2, 1, N)
    c, s = ref.cos_sin(pos, sections, 10000.0, True)

    def f(y):
        return float((w * ref.turn(y, c[:, None], s[:, None])).sum())

    grad = np.zeros_like(x)
    for at in np.ndindex(*x.shape):
        e = np.zeros_like(x)
        e[at] = 0.5
        grad[at] = f(x + e) - f(x - e)
    wd = to_dev(wb, dev)
    got, _ = ex.attn_rope_axes(wd, wd, to_dev(pos, dev), sections, base=10000.0, per_axis=True, inverse=True)
    assert (np.abs(f64(got) - grad) <= 2.0 ** -8 * np.abs(grad) + 1e-5).all()


def test_infinities_and_nan_stay_in_their_pair(env):
    torch, ex, dev = env
    q, k = inputs(torch, dev, 305, 1, 4, 2, 1, 64)
    pos = torch.arange(1, 5, device=dev, dtype=torch.int32).view(1, 1, 4)
    clean, _ = ex.attn_rope_axes(q, k, pos, (32,))
    q[0, 0, 2, 5] = float("nan")
    q[0, 1, 3, 40] = float("inf")
    got, _ = ex.attn_rope_axes(q, k, pos, (32,))
    bad = torch.zeros_like(got, dtype=torch.bool)
    bad[0, 0, 2, [5, 37]] = True
    bad[0, 1, 3, [8, 40]] = True
    assert not torch.isfinite(got[bad]).any()
    assert torch.equal(got[~bad], clean[~bad])


def test_empty_and_refused(env):
    torch, ex, dev = env
    e = torch.empty((0, 2, 5, 64), device=dev, dtype=torch.bfloat16)
    qo, ko = ex.attn_rope_axes(e, e, torch.empty((1, 0, 5), device=dev, dtype=torch.int32), (32,))
    assert qo.shape == e.shape
    q, k = inputs(torch, dev, 306, 2, 5, 2, 1, 64)
    pos = torch.zeros((1, 2, 5), device=dev, dtype=torch.int32)
    with pytest.raises(ex.ExattnError):
        ex.attn_rope_axes(q, k, pos, (31,))
    with pytest.raises(ValueError):
        ex.attn_rope_axes(q, k, pos[:, :, :4], (32,))
    with pytest.raises(ValueError):
        ex.attn_rope_axes(q, k[:1], pos, (32,))
    with pytest.raises(TypeError):
        ex.attn_rope_axes(q, k, pos.long(), (32,))
    with pytest.raises(TypeError):
        ex.attn_rope_axes(q.float(), k, pos, (32,))
    with pytest.raises(ValueError):
        ex.attn_rope_axes(q.transpose(2, 3), k, pos, (32,))
    odd = torch.zeros(2 * 2 * 5 * 64 + 8, device=dev, dtype=torch.bfloat16)[4:-4].view(2, 2, 5, 64)
    with pytest.raises(ex.ExattnError):
        ex.attn_rope_axes(odd, k, pos, (32,))


def test_training_step_over_rotated_heads(env):
    """rope -> attn_fwd -> attn_bwd -> reverse rope, against torch autograd of the
    same chain in fp64.  Each link rounds to bf16 and the attention's bars are
    relative RMS 5e-3 each way; three such links stay below 2e-2."""
    torch, ex, dev = env
    B, N, Hq, Hkv, d, sections = 2, 130, 4, 2, 64, (8, 12, 12)
    q, k = inputs(torch, dev, 307, B, N, Hq, Hkv, d)
    v = to_dev(synth.normal_bf16(307, 3, (B, Hkv, N, d)), dev)
    do = to_dev(synth.normal_bf16(307, 4, (B, Hq, N, d)), dev)
    pos = positions(11, 3, B, N)
    pd = to_dev(pos, dev)
    qr, kr = ex.attn_rope_axes(q, k, pd, sections)
    out, lse = ex.attn_fwd(qr, kr, v, causal=True)
    dqr, dkr, dv = ex.attn_bwd(qr, kr, v, out, do, lse, causal=True)
    dq, dk = ex.attn_rope_axes(dqr, dkr, pd, sections, inverse=True)
    c, s = (torch.from_numpy(x).to(dev)[:, None] for x in ref.cos_sin(pos, sections, 500000.0, False))
    leaves = [x.double().requires_grad_() for x in (q, k, v)]

    def turn(x):
        a, b = x.chunk(2, -1)
        return torch.cat([a * c - b * s, b * c + a * s], -1)

    kk, vv = (x.repeat_interleave(Hq // Hkv, 1) for x in (turn(leaves[1]), leaves[2]))
    x = turn(leaves[0]) @ kk.transpose(-1, -2) / d ** 0.5
    x = x.masked_fill(torch.ones(N, N, device=dev, dtype=torch.bool).triu(1), float("-inf"))
    (torch.softmax(x, -1) @ vv).backward(do.double())
    for name, got, leaf in zip(("dq", "dk", "dv"), (dq, dk, dv), leaves):
        rel = ((got.double() - leaf.grad).norm() / leaf.grad.norm()).item()
        assert rel <= 2e-2, "%s: %.3e" % (name, rel)


@pytest.mark.parametrize("Hq,Hkv,Nq,Nk", [(4, 4, 1500, 1500), (8, 2, 1000, 1000), (2, 2, 70, 4000), (2, 2, 3000, 100)])
def test_gradients_are_whole_when_they_are_turned_back(env, Hq, Hkv, Nq, Nk):
    """The turn may start while the backward's last kernel ends, whose own
    predecessor may still be running then: the same bits as with a synchronisation
    between the two."""
    torch, ex, dev = env
    q = to_dev(synth.normal_bf16(320, 1, (2, Hq, Nq, 128)), dev)
    k = to_dev(synth.normal_bf16(320, 2, (2, Hkv, Nk, 128)), dev)
    v = to_dev(synth.normal_bf16(320, 3, (2, Hkv, Nk, 128)), dev)
    do = to_dev(synth.normal_bf16(320, 4, (2, Hq, Nq, 128)), dev)
    pq = torch.arange(Nk - Nq, Nk, device=dev, dtype=torch.int32)[None]
    pk = torch.arange(Nk, device=dev, dtype=torch.int32)[None]
    out, lse = ex.attn_fwd(q, k, v, causal=True)
    none_q, none_k = q[:, :0], k[:, :0]

    def step(between):
        dq, dk, dv = ex.attn_bwd(q, k, v, out, do, lse, causal=True)
        between()
        ex.attn_rope_axes(dq, none_q, pq, (64,), inverse=True, q_out=dq)
        between()
        ex.attn_rope_axes(none_k, dk, pk, (64,), inverse=True, k_out=dk)
        between()
        return dq, dk, dv

    want = step(torch.cuda.synchronize)
    assert want[0].float().abs().max() > 0
    for _ in range(10):
        got = [step(lambda: None) for _ in range(3)]
        for g in got:
            for a, b in zip(g, want):
                assert torch.equal(a, b)
    assert ex.attn_get_device_status() == 0
