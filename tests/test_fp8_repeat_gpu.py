"""The 8-bit decode gives the same bits each time, whatever its workspace held before and
whatever runs beside it."""
import pytest

from exact_attention_40_gb300 import synth
from helpers import to_dev
from test_fp8_gpu import decode_case, env  # noqa: F401  (env: a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,Hq,Hkv,queries", [([900, 31, 0], 8, 2, None), ([33000], 8, 2, None), ([3000, 700] * 20, 12, 4, 3),
                                                 ([300, 41, 900] * 150, 6, 2, None)], ids=["cluster", "long", "queries", "many"])
def test_decode_repeats_itself(env, d, lens, Hq, Hkv, queries):
    torch, ex, dev = env
    case = decode_case(960, lens, Hq, Hkv, d, queries)
    args = [to_dev(x, dev) for x in case]
    need = ex.attn_decode_fp8_workspace_bytes(len(lens), queries or 1, Hq, Hkv, d, case[2].shape[1])
    want, want_lse = ex.attn_decode_paged_fp8(*args)
    beside = torch.cuda.Stream()
    noise = to_dev(synth.normal_bf16(961, 0, (2048, 2048)), dev)
    for fill in (0, 0xFF, 0x7F, 0x3C):
        ws = torch.full((max(need, 16),), fill, device=dev, dtype=torch.uint8)
        torch.cuda.synchronize()
        with torch.cuda.stream(beside):
            for _ in range(3):
                noise @ noise
        out, lse = ex.attn_decode_paged_fp8(*args, workspace=ws)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
    torch.cuda.synchronize()
    assert ex.attn_get_device_status() == 0
