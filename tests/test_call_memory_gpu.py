"""Memory that a call allocates for itself when it runs on another stream than the
current one: it must not be a block whose last use on the current stream is still to
come, nor be handed out again while a stream uses it."""
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


def decode_fp4(torch, ex, dev):
    lens = torch.tensor([20000, 3], device=dev, dtype=torch.int32)
    cache = to_dev(ref.random_cache(640, 64, 1, 128), dev)
    table = (torch.arange(2 * 1250, device=dev, dtype=torch.int32) % 64).view(2, 1250)
    q = to_dev(synth.normal_bf16(640, 0, (2, 8, 128)), dev)
    sizes = [ex.attn_decode_fp4_workspace_bytes(2, 8, 1, 128, 1250), q.numel() * 2, 2 * 8 * 4]
    assert sizes[0] > 0
    return sizes, lambda stream: ex.attn_decode_paged_fp4(q, cache, table, lens, stream=stream)


def rope(torch, ex, dev):
    q = to_dev(synth.normal_bf16(641, 0, (2, 4, 300, 64)), dev)
    at = torch.arange(300, device=dev, dtype=torch.int32)[None]
    return [q.numel() * 2] * 2, lambda stream: ex.attn_rope_axes(q, q, at, (32,), stream=stream)


def append(torch, ex, dev):
    x = to_dev(synth.normal_bf16(642, 0, (640, 2, 64)), dev)
    at = torch.arange(640, device=dev, dtype=torch.int32)
    table = torch.arange(40, device=dev, dtype=torch.int32)[None]
    cache, seq = ex.attn_fp4_cache(40, 2, 64), torch.zeros_like(at)
    return [x.numel() * 2], lambda stream: [
        ex.attn_rope_cache_write_fp4(x, x, x, seq, at, at[None], table, cache, (32,), stream=stream)]


def read(torch, ex, dev):
    cache = to_dev(ref.random_cache(643, 40, 2, 64), dev)
    at = torch.arange(640, device=dev, dtype=torch.int32)
    seq = torch.zeros_like(at)
    table = torch.arange(40, device=dev, dtype=torch.int32)[None]
    return [640 * 2 * 64 * 2] * 2, lambda stream: ex.attn_cache_read_fp4(cache, seq, at, table, stream=stream)


def forward(torch, ex, dev):
    q = to_dev(synth.normal_bf16(644, 0, (1, 4, 300, 64)), dev)
    return [q.numel() * 2, 4 * 300 * 4], lambda stream: ex.attn_fwd(q, q, q, causal=True, stream=stream)


def backward(torch, ex, dev):
    q = to_dev(synth.normal_bf16(645, 0, (1, 4, 300, 64)), dev)
    k = q[:, :2].contiguous()
    out, lse = ex.attn_fwd(q, k, k)
    sizes = [q.numel() * 2, k.numel() * 2, k.numel() * 2, ex.lib.attn_bwd_workspace_bytes(1, 4, 2, 300, 300, 64)]
    return sizes, lambda stream: ex.attn_bwd(q, k, k, out, q, lse, stream=stream)


def decode(torch, ex, dev):
    lens = torch.tensor([20000, 3], device=dev, dtype=torch.int32)
    cache = to_dev(synth.normal_bf16(646, 0, (64, 1, 16, 128)), dev)
    table = (torch.arange(2 * 1250, device=dev, dtype=torch.int32) % 64).view(2, 1250)
    q = to_dev(synth.normal_bf16(646, 1, (2, 8, 128)), dev)
    sizes = [ex.attn_decode_workspace_bytes(2, 8, 128, 1250), q.numel() * 2, 2 * 8 * 4]
    return sizes, lambda stream: ex.attn_decode_paged(q, cache, cache, table, lens, stream=stream)


def norm(torch, ex, dev):
    x = to_dev(synth.normal_bf16(647, 0, (64, 512)), dev)
    return [x.numel() * 2] * 2, lambda stream: ex.attn_add_rms_norm(x, x, x[0], stream=stream)


CALLS = [decode_fp4, rope, append, read, forward, backward, decode, norm]


@pytest.mark.parametrize("make", CALLS)
def test_blocks_in_use_on_the_current_stream_stay_whole(env, make):
    """Tensors of the sizes that the call allocates, dropped while copies of them wait on
    the current stream behind a long kernel."""
    torch, ex, dev = env
    sizes, call = make(torch, ex, dev)
    main, side = torch.cuda.current_stream(), torch.cuda.Stream()
    want = [x.clone() for x in call(None)]
    side.wait_stream(main)
    call(side)
    torch.cuda.synchronize()
    for _ in range(3):
        held = [torch.full((n,), 7, device=dev, dtype=torch.uint8) for n in sizes]
        copies = [torch.zeros_like(t) for t in held]
        side.wait_stream(main)
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)  # some 10 ms
        for t, c in zip(held, copies):
            c.copy_(t)
        del held, t
        got = call(side)
        side.synchronize()
        torch.cuda.synchronize()
        assert all(bool((c == 7).all()) for c in copies)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("make", CALLS)
def test_outputs_dropped_on_the_current_stream_are_not_handed_out_before_their_use(env, make):
    torch, ex, dev = env
    sizes, call = make(torch, ex, dev)
    main, side = torch.cuda.current_stream(), torch.cuda.Stream()
    want = [x.clone() for x in call(None)]
    torch.cuda.synchronize()
    for _ in range(3):
        got = call(side)
        main.wait_stream(side)
        torch.cuda._sleep(20_000_000)
        copies = [x.clone() for x in got]
        del got
        for stream in (side, main):
            with torch.cuda.stream(stream):
                for n in sizes + sizes:
                    torch.full((n,), 0xFF, device=dev, dtype=torch.uint8)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(copies, want))


@pytest.mark.parametrize("make", CALLS)
def test_a_stream_is_any_object_with_its_handle(env, make):
    """The default stream among them, from a stream that is current instead."""
    from types import SimpleNamespace
    torch, ex, dev = env
    _, call = make(torch, ex, dev)
    want = [x.clone() for x in call(None)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = call(SimpleNamespace(cuda_stream=side.cuda_stream))
    with torch.cuda.stream(side):
        back = call(SimpleNamespace(cuda_stream=torch.cuda.default_stream().cuda_stream))
    torch.cuda.synchronize()
    for a, b, c in zip(got, back, want):
        assert torch.equal(a, c) and torch.equal(b, c)
