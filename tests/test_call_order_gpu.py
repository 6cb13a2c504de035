"""Calls that follow each other on a stream where one of them has little or nothing to
wait for: the same bits as with a synchronisation after every call."""
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


@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (8, 2)])
@pytest.mark.parametrize("S,ctx", [(6, 4090), (200, 128), (40, 3000)])
def test_backward_without_queries_after_a_decode(env, Hq, Hkv, S, ctx):
    """A backward without queries (dK = dV = 0) has no dQ pass in front of its dK/dV pass.
    Its outputs are given the memory of the decode's queries, as the allocator would once
    those are dropped, and the rotation after it turns the decode's output in place.  The
    decode as clusters, as CTAs of their own and with a merge behind it."""
    torch, ex, dev = env
    d = 128
    blocks = (ctx + 15) // 16
    pages = min(S, 8) * blocks  # sequences share pages
    table = (torch.arange(S * blocks, device=dev, dtype=torch.int32) % pages).view(S, blocks)
    lens = torch.tensor([ctx - 5 * (i % 16) for i in range(S)], device=dev, dtype=torch.int32)
    cache = to_dev(ref.random_cache(611, pages, Hkv, d), dev)
    q0 = to_dev(synth.normal_bf16(611, 0, (S, Hq, d)), dev)
    Nk = S * Hq // Hkv // 2
    k = to_dev(synth.normal_bf16(611, 3, (1, Hkv, Nk, d)), dev)
    none = k.new_empty((1, Hq, 0, d))
    no_lse = torch.empty((1, Hq, 0), device=dev, dtype=torch.float32)
    at = torch.arange(S, device=dev, dtype=torch.int32)[None]
    q, out = torch.empty_like(q0), torch.empty_like(q0)
    rows = q.view(-1)[:2 * Hkv * Nk * d].view(2, 1, Hkv, Nk, d)
    turned = out[None].transpose(1, 2)

    def run(after):
        q.copy_(q0), out.zero_(), after()
        _, lse = ex.attn_decode_paged_fp4(q, cache, table, lens, out=out)
        after()
        ex.attn_bwd(none, k, k, none, none, no_lse, dq=none, dk=rows[0], dv=rows[1]), after()
        ex.attn_rope_axes(turned, turned[:, :0], at, (64,), q_out=turned), after()
        return lse

    want_lse = run(torch.cuda.synchronize)
    want = out.clone()
    assert int((rows != 0).sum()) == 0 and torch.isfinite(want.float()).all() and want.float().abs().max() > 0
    for _ in range(20):
        lse = run(lambda: None)
        assert torch.equal(out, want) and torch.equal(lse, want_lse) and int((rows != 0).sum()) == 0
    assert ex.attn_get_device_status() == 0
