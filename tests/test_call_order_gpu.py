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


def test_captured_calls_between_two_streams(env):
    """A capture that forks to another stream and joins again: the calls have a kernel of
    their own stream and one of the other before them, and each graph node waits for both."""
    torch, ex, dev = env
    S, Hq, Hkv, d = 6, 8, 2, 128
    lens_list = [3000, 5, 700, 129, 0, 64]
    blocks = (max(lens_list) + 15) // 16
    table = (torch.arange(S * blocks, device=dev, dtype=torch.int32) % 400).view(S, blocks)
    lens = torch.tensor(lens_list, device=dev, dtype=torch.int32)
    cache = to_dev(ref.random_cache(612, 400, Hkv, d), dev)
    at = torch.arange(S, device=dev, dtype=torch.int32)[None]
    slots = torch.tensor([max(0, n - 1) for n in lens_list], device=dev, dtype=torch.int32)
    seq = torch.arange(S, device=dev, dtype=torch.int32)
    qs = to_dev(synth.normal_bf16(612, 1, (8, S, Hq, d)), dev)
    big = torch.randn(2048, 2048, device=dev)
    x, y = torch.zeros_like(qs[0]), torch.zeros_like(qs[0])
    out = torch.empty_like(qs)
    back = torch.empty((8, S, Hkv, d), device=dev, dtype=torch.bfloat16)
    side = torch.cuda.Stream()

    def heads(t):
        return t[None].transpose(1, 2)

    def run(apart):
        main = torch.cuda.current_stream()
        busy = big
        side.wait_stream(main)
        for i in range(8):
            with torch.cuda.stream(side):
                busy = (busy @ big).clamp(-1, 1)  # the copy comes late
                x.copy_(qs[i])
            apart()
            ex.attn_rope_axes(heads(y), heads(y)[:, :0], at, (64,), q_out=heads(y)), apart()
            main.wait_stream(side)
            ex.attn_rope_axes(heads(x), heads(x)[:, :0], at, (64,), q_out=heads(y)), apart()
            side.wait_stream(main)
            ex.attn_decode_paged_fp4(y, cache, table, lens, out=out[i]), apart()
            with torch.cuda.stream(side):
                x.fill_(float("nan"))
                ex.attn_cache_read_fp4(cache, seq, slots, table, k_out=back[i], v_out=x[:, Hkv:2 * Hkv])
            apart()
        main.wait_stream(side)
        return busy

    run(torch.cuda.synchronize)
    torch.cuda.synchronize()
    want, want_back = out.clone(), back.clone()
    assert torch.isfinite(want.float()).all() and want.float().abs().max() > 0
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(lambda: None)
    for _ in range(10):
        out.zero_(), back.zero_()
        g.replay()
        assert torch.equal(out, want) and torch.equal(back, want_back)
    assert ex.attn_get_device_status() == 0
