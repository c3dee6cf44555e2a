"""Calls on an explicit stream: what they allocate must not be memory that work still queued on the caller's current
stream writes."""
from __future__ import annotations

import pytest
import torch

from gated_delta_rule_65_b200 import gdr2

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def randn(*shape):
    return torch.randn(*shape, device="cuda").bfloat16()


def attention_calls():
    """name -> (call(stream), tensors that it changes in place)"""
    torch.manual_seed(1)
    T, Hq, Hk, d, ps, R, P = 600, 8, 2, 64, 16, 3, 200
    num = R * P
    x, dy = randn(T, Hq + 2 * Hk, d), randn(T, Hq + Hk, d)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:]
    dq, dk = dy[:, :Hq].contiguous(), dy[:, Hq:].contiguous()
    gain = torch.rand(d, device="cuda")
    pos, seq = torch.arange(T, device="cuda").int(), torch.zeros(T, dtype=torch.int32, device="cuda")
    freqs, _ = gdr2.rope_freqs(d)
    pools = randn(num, Hk, ps, d), randn(num, Hk, ps, d)
    table = torch.randperm(num, device="cuda").view(R, P).int()
    lens, want, ref = ints([3100, 20, 901]), ints([3190, 60, 1000]), ints([1] * num)
    parent = ints([2, 1, 2])
    half, fewer = table.clone(), ref.clone()
    half[:, 100:] = -1
    fewer[table[:, 100:].flatten().long()] = 0
    a = (q, k, gain, gain, pos, freqs)
    return {
        "fwd": (lambda s: gdr2.attn_prologue_fwd(*a, stream=s), ()),
        "bwd": (lambda s: gdr2.attn_prologue_bwd(*a, dq, dk, stream=s), ()),
        "cache": (lambda s: gdr2.attn_prologue_cache(q, k, v, gain, gain, seq, pos, freqs, *pools, table, stream=s), pools),
        "decode": (lambda s: gdr2.attn_decode(dq[:R], *pools, table, lens, want_lse=True, stream=s), ()),
        "reserve": (lambda s: gdr2.kv_reserve(half, lens, want, fewer, page_size=ps, stream=s), ()),
        "fork": (lambda s: gdr2.kv_fork(half, lens, fewer, parent, *pools, stream=s), pools),
        "compact": (lambda s: gdr2.kv_compact(half, fewer, *pools, stream=s), pools),
    }


def mixer_calls():
    torch.manual_seed(2)
    B, T, H, d = 1, 256, 2, 128
    lens = ints([0, 100, 256])

    def inputs(H, Hv, T=T):
        shape, wide = (B, T, H, d) if T else (B, H, d), (B, T, Hv, d) if T else (B, Hv, d)
        q, k = (torch.nn.functional.normalize(torch.randn(*shape, device="cuda"), dim=-1).bfloat16() for _ in range(2))
        gate = lambda s: torch.rand(*s, device="cuda").bfloat16()  # noqa: E731
        return q, k, randn(*wide), -0.1 * torch.rand(*shape, device="cuda"), gate(shape), gate(wide)

    x, y, one = inputs(H, H), inputs(H, 2 * H), inputs(H, H, 0)
    f = tuple(t.float() for t in x)
    S = torch.randn(B, H, d, d, device="cuda")
    pre = tuple(randn(B, T, H, d) for _ in range(5)) + (torch.randn(H, d, device="cuda"), torch.randn(H, d, device="cuda"))
    grads = (*(randn(B, T, H, d) for _ in range(2)), torch.randn(B, T, H, d, device="cuda"), *(randn(B, T, H, d) for _ in range(2)))
    return {
        "chunk_fwd": (lambda s: gdr2.chunk_fwd(*x, stream=s), ()),
        "chunk_fwd f32": (lambda s: gdr2.chunk_fwd(*f, stream=s), ()),
        "chunk_fwd_noalloc": (lambda s: gdr2.chunk_fwd_noalloc(*x, stream=s), ()),
        "chunk_bwd": (lambda s: gdr2.chunk_bwd(*x, d_o=x[2], stream=s), ()),
        "chunk_fwd_gva": (lambda s: gdr2.chunk_fwd_gva(*y, stream=s), ()),
        "chunk_bwd_gva": (lambda s: gdr2.chunk_bwd_gva(*y, d_o=y[2], stream=s), ()),
        "chunk_fwd_varlen": (lambda s: gdr2.chunk_fwd_varlen(*x, lens, stream=s), ()),
        "chunk_bwd_varlen": (lambda s: gdr2.chunk_bwd_varlen(*x, lens, d_o=x[2], stream=s), ()),
        "gate_prologue_fwd": (lambda s: gdr2.gate_prologue_fwd(*pre, stream=s), ()),
        "gate_prologue_bwd": (lambda s: gdr2.gate_prologue_bwd(*pre, *grads, stream=s), ()),
        "decode_step": (lambda s: gdr2.decode_step(*one, S, stream=s), (S,)),
    }


def results(out):
    return [t for t in (out.values() if isinstance(out, dict) else out if isinstance(out, tuple) else (out,)) if t is not None]


def fresh_on_a_busy_stream(call, changed):
    """The caller's stream has 20 ms or more of copies queued, then writes to blocks of every size, which are let go on
    the host at once: a call on another stream, which has nothing to wait for, must not be given any of them."""
    before = [t.clone() for t in changed]
    want = [t.clone() for t in results(call(None))]
    after = [t.clone() for t in changed]
    for t, b in zip(changed, before):
        t.copy_(b)
    big = torch.empty(2, 1 << 29, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for how in (side, side.cuda_stream):
        for _ in range(100):
            big[0].copy_(big[1])
        for n in range(2, 27):
            for _ in range(6):
                torch.full((1 << n,), 0xff, dtype=torch.uint8, device="cuda")
        got = call(how)
        with torch.cuda.stream(side):
            changes = [t.clone() for t in changed]
            for t, b in zip(changed, before):
                t.copy_(b)
        torch.cuda.synchronize()
        for x, y in zip(results(got), want, strict=True):
            assert torch.equal(x, y)
        for x, y in zip(changes, after):
            assert torch.equal(x, y)
        del got


@pytest.mark.parametrize("name", ["fwd", "bwd", "cache", "decode", "reserve", "fork", "compact"])
def test_attention_half(name):
    fresh_on_a_busy_stream(*attention_calls()[name])


@pytest.mark.parametrize("name", ["chunk_fwd", "chunk_fwd f32", "chunk_fwd_noalloc", "chunk_bwd", "chunk_fwd_gva", "chunk_bwd_gva",
                                  "chunk_fwd_varlen", "chunk_bwd_varlen", "gate_prologue_fwd", "gate_prologue_bwd",
                                  "decode_step"])
def test_mixer(name):
    fresh_on_a_busy_stream(*mixer_calls()[name])


def test_current_and_default_streams_by_handle():
    """A handle of the current stream, 0 and 1 (the legacy stream's two names) are streams as any other."""
    call, _ = attention_calls()["decode"]
    want = results(call(None))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = [call(s) for s in (side, side.cuda_stream, 0, 1)]
    torch.cuda.synchronize()
    got += [call(s) for s in (torch.cuda.current_stream(), 0, 1, side.cuda_stream)]
    torch.cuda.synchronize()
    for out in got:
        for x, y in zip(results(out), want, strict=True):
            assert torch.equal(x, y)


def test_results_outlive_their_use_on_the_callers_stream():
    """A result that the caller's stream still reads when the host lets it go is not handed to the next call."""
    call, _ = attention_calls()["decode"]
    want = results(call(None))
    big = torch.empty(2, 1 << 29, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = call(side)
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(100):
        big[0].copy_(big[1])
    copies = [t.clone() for t in results(out)]
    shapes = [(t.shape, t.dtype) for t in results(out)]
    del out
    with torch.cuda.stream(side):
        for shape, dtype in shapes * 4:
            torch.empty(shape, dtype=dtype, device="cuda").fill_(7)
    torch.cuda.synchronize()
    for x, y in zip(copies, want, strict=True):
        assert torch.equal(x, y)


def test_the_threads_default_stream_by_handle():
    """2 is the runtime's handle of the calling thread's default stream."""
    call, _ = attention_calls()["decode"]
    want = results(call(None))
    torch.cuda.synchronize()
    for _ in range(2):
        got = call(2)
        torch.cuda.synchronize()
        for x, y in zip(results(got), want, strict=True):
            assert torch.equal(x, y)
        del got


@pytest.mark.parametrize("name", ["bwd", "decode", "fork", "chunk_bwd"])
def test_explicit_stream_inside_a_capture(name):
    """A capture that forks to another stream, makes the call there and joins: fresh outputs and workspaces are the
    graph's."""
    call, changed = {**attention_calls(), **mixer_calls()}[name]
    before = [t.clone() for t in changed]
    want = [t.clone() for t in results(call(None))]
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = results(call(side))
        torch.cuda.current_stream().wait_stream(side)
        twice = [t.clone() for t in got]
    for _ in range(2):
        for t, b in zip(changed, before):
            t.copy_(b)
        for t in got:
            t.zero_()
        trash = [torch.full((1 << n,), 0xff, dtype=torch.uint8, device="cuda") for n in range(2, 24) for _ in range(4)]
        graph.replay()
        torch.cuda.synchronize()
        for x, y, z in zip(got, twice, want, strict=True):
            assert torch.equal(x, z) and torch.equal(y, z)
        assert all((t == 0xff).all() for t in trash)
