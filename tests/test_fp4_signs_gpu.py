"""Signs in the 4-bit cache: those of zeros on their way in, all of them on their way
out.  Stored bytes and read-back bits are compared whole."""
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


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("g,size", [(0.01, 1.0), (2.0 ** -6, 1.0), (1e-3, 1.0), (1e-30, 1e-30), (100.0, 1.0)])
def test_zeros_keep_their_sign(env, d, g, size):
    """Zeros of both signs among ordinary values: groups whose quotients come from the
    reciprocal, from the division (a saturated scale, a tensor scale near the end of
    fp32's range) and whose scale is zero.  At position 0 a key is x 1 - y 0, so its sign
    of zero is that of the definition's fp32 operations, too."""
    torch, ex, dev = env
    T, Hkv = 32, 2
    f = synth.bf16_bits_to_f32(synth.normal_bf16(620, 1, (T, Hkv, d))) * np.float32(size)
    f[:, :, 1::5] = 0.0
    f[:, :, 2::5] = -0.0
    f[3] = -0.0
    f[4] = 0.0
    bits = synth.f32_to_bf16_bits(f)
    f = synth.bf16_bits_to_f32(bits)
    assert (np.signbit(f) & (f == 0)).sum() >= T * Hkv * d // 5 - T * Hkv
    x = to_dev(bits, dev)
    z = torch.zeros(T, device=dev, dtype=torch.int32)
    slots = torch.arange(T, device=dev, dtype=torch.int32)
    table = torch.arange(2, device=dev, dtype=torch.int32).view(1, 2)
    cache = ex.attn_fp4_cache(2, Hkv, d)
    ex.attn_rope_cache_write_fp4(x, x, x, z, slots, z.view(1, T), table, cache, (d // 2,), k_scale=g, v_scale=g)
    got = [v.transpose(0, 2, 1, 3).reshape(T, Hkv, -1) for v in ref.split(cache.cpu().numpy(), d)]
    turned = ref.turn(f, np.float32(1.0), np.float32(0.0))
    for codes, scales, x32 in ((got[0], got[2], turned), (got[1], got[3], f)):
        want, s8 = ref.quantise(x32, g)
        assert np.array_equal(scales, s8)
        assert np.array_equal(ref.unpack(codes), want), "%d codes differ" % (ref.unpack(codes) != want).sum()
    assert ex.attn_get_device_status() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("k_scale,v_scale", [(1.0, 0.0023), (3e-8, 100.0)])
def test_every_code_reads_back_with_its_sign(env, d, k_scale, v_scale):
    """Spans of arbitrary codes and all finite scales, zero among them: the read-back equals
    code * scale * g, rounded once, in every bit."""
    torch, ex, dev = env
    nb, Hkv = 40, 3
    cache = synth.splitmix64(621, nb * Hkv * 18 * d // 8).view(np.uint8).reshape(nb, Hkv, 18 * d).copy()
    scales = cache[..., 16 * d:]
    scales &= 0x7F
    scales[scales == 0x7F] = 0x7E
    scales[..., ::7] = 0
    ck, cv, sk, sv = ref.split(cache, d)
    assert set(np.unique(ref.unpack(ck))) == set(range(16))
    order = np.argsort(synth.uniform01(622, nb)).astype(np.int32)
    slots = torch.arange(nb * 16, device=dev, dtype=torch.int32)
    out = ex.attn_cache_read_fp4(to_dev(cache, dev), torch.zeros_like(slots), slots, to_dev(order[None], dev),
                                 k_scale=k_scale, v_scale=v_scale)
    for got, codes, s8, g in zip(out, (ck, cv), (sk, sv), (k_scale, v_scale)):
        want = ref.values(ref.unpack(codes), s8, g)[order].transpose(0, 2, 1, 3).reshape(nb * 16, Hkv, d)
        want = torch.from_numpy(np.ascontiguousarray(want)).float().bfloat16()
        assert torch.equal(got.cpu().view(torch.int16), want.view(torch.int16))
    assert ex.attn_get_device_status() == 0
