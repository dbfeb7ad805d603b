"""Calls on a given stream own the memory that they make: blocks that the
current stream has freed, with writes to them still queued there, are not used
by a call that another stream runs at once."""
import pytest
import torch

import block_causal_relu_b200 as lcla

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def calls():
    """(name, call(**kw) -> outputs) of every operator that makes outputs or a workspace."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    B, N, H, d = 1, 4000, 6, 32
    q, k, v, do = (r(B, N, H, d).to(BF) for _ in range(4))
    g, s0 = -0.05 * torch.rand(B, N, H, generator=gen, device="cuda"), r(B, H, d, d)
    w = 1 + 0.1 * r(d)
    c, s = lcla.rotary_tables(N, d)
    blocks = torch.tensor([0, 800, 2000, N], dtype=torch.int32, device="cuda")
    state = r(B, H, d + 1, d).abs()
    x, wt, bias = r(1, N, 192).to(BF), r(2, 192), r(192)
    one = [t[:, :9].contiguous() for t in (q, k, v, g)]
    return [
        ("rotary_tables", lambda **kw: lcla.rotary_tables(N, d, **kw)),
        ("qk_norm_rope", lambda **kw: lcla.qk_norm_rope(q, k, c, s, **kw)),
        ("qk_norm_rope_backward", lambda **kw: lcla.qk_norm_rope_backward(do, do, q, k, c, s, q_weight=w, k_weight=w, **kw)),
        ("gated_forward", lambda **kw: lcla.gated_forward(q, k, v, g, state_in=s0, **kw)),
        ("gated_step", lambda **kw: lcla.gated_step(*one, s0, False, **kw)),
        ("gated_backward", lambda **kw: lcla.gated_backward(do, q, k, v, g, state_in=s0, want_dstate_in=True, **kw)),
        ("forward", lambda **kw: lcla.forward(q, k, v, c, s, 800, **kw)),
        ("forward_blocks", lambda **kw: lcla.forward_blocks(q, k, v, c, s, blocks, **kw)),
        ("step", lambda **kw: lcla.step(q, k, v, c, s, state, False, **kw)),
        ("shard_begin", lambda **kw: lcla.shard_begin(k, v, c, s, 800, **kw)[0]),
        ("temporal_conv", lambda **kw: lcla.temporal_conv(x, 400, wt, bias, **kw)),
    ]


def flat(out):
    return [t for t in (out if isinstance(out, tuple) else (out,)) if t is not None]


@pytest.mark.parametrize("i", range(11))
def test_memory_freed_on_the_current_stream_is_left_alone(i):
    name, call = calls()[i]
    want = [t.clone() for t in flat(call())]
    sizes = [t.numel() * t.element_size() for t in want]
    side = torch.cuda.Stream()
    for handle in (side, side.cuda_stream):
        for _ in range(3):
            torch.cuda.synchronize()
            torch.cuda.empty_cache()
            # blocks of the outputs' sizes and larger ones, freed with a late write queued on the current stream
            junk = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes + [1 << 20, 1 << 22, 1 << 25]]
            torch.cuda._sleep(40_000_000)
            for t in junk:
                t.fill_(0xff)
            del junk, t
            got = call(stream=handle)
            side.synchronize()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(flat(got), want)), name


def test_results_outlive_their_use_on_the_current_stream():
    """A result that the current stream still reads when its last reference goes is not given out again before."""
    q = torch.randn(1, 4000, 6, 32, device="cuda").to(BF)
    c, s = lcla.rotary_tables(4000, 32)
    want, _ = lcla.qk_norm_rope(q, None, c, s)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got, _ = lcla.qk_norm_rope(q, None, c, s, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(40_000_000)
    kept = got.clone()
    del got
    with torch.cuda.stream(side):
        for _ in range(4):
            torch.full_like(q, float("nan"))
    torch.cuda.synchronize()
    assert torch.equal(kept, want)


def test_the_current_stream_and_captures_may_be_given():
    q = torch.randn(1, 300, 2, 32, device="cuda").to(BF)
    g = torch.zeros(1, 300, 2, device="cuda")
    want = lcla.gated_forward(q, q, q, g)
    got = lcla.gated_forward(q, q, q, g, stream=torch.cuda.current_stream())
    zero = lcla.gated_forward(q, q, q, g, stream=0)
    assert all(torch.equal(a, b) and torch.equal(a, e) for a, b, e in zip(want, got, zero))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = lcla.gated_forward(q, q, q, g, stream=torch.cuda.current_stream().cuda_stream)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, cap))
