"""Calls of the attention half at the edges of what its header allows, on the GPU: lengths beyond the page table, more
slots than sequences."""
from __future__ import annotations

import pytest
import torch

from gated_delta_rule_65_b200 import gdr2
from tests import attn_ref as ref

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def reserve_by_entries(table, lens, want, ref, ps):
    """The rule of the header entry by entry: j from lens / ps up to, but not with, ceil(want / ps); lowest pages first,
    past the table's end none to be had."""
    table, ref, missing = [list(row) for row in table], list(ref), 0
    for r, row in enumerate(table):
        for j in range(max(lens[r], 0) // ps, -(-max(want[r], 0) // ps)):
            if j < len(row) and 0 <= row[j] < len(ref):
                continue
            page = min((i for i, n in enumerate(ref) if n <= 0), default=-1) if j < len(row) else -1
            if page < 0:
                missing += 1
            else:
                row[j], ref[page] = page, 1
    return table, ref, missing


@pytest.mark.parametrize("P,ps,lens,want", [
    (2, 1, [5], [6]),              # one page asked for, past the table
    (2, 1, [5], [5]),              # none
    (4, 16, [100], [101]),         # entry 6 of 4
    (4, 16, [100], [80]),          # fewer than there are: none
    (4, 16, [64], [65]),           # the first entry past the table
    (4, 16, [63], [129]),          # the last entry of the table and five past it
    (4, 16, [-3], [200]),          # all of the table and nine past it
    (4, 16, [100, 0, 2**31 - 1, 40], [100, 17, 2**31 - 1, 90]),
    (3, 7, [21, 22, 2**31 - 1, 0], [22, 22, 0, -5]),
], ids=str)
@pytest.mark.parametrize("pages", [1, 9])
def test_missing_counts_what_was_asked_for(P, ps, lens, want, pages):
    R = len(lens)
    table, refs = [[-1] * P for _ in range(R)], [0] * pages
    et, er, em = reserve_by_entries(table, lens, want, refs, ps)
    t, r, m = gdr2.kv_reserve(ints(table), ints(lens), ints(want), ints(refs), page_size=ps)
    assert (t.tolist(), r.tolist(), m.tolist()) == (et, er, [em])


def test_missing_of_many_sequences_beyond_the_table():
    """A cluster of CTAs: only the sequences that ask for more count."""
    R, P, ps = 9000, 3, 4
    lens = [12 + r % 50 for r in range(R)]
    want = [x + r % 3 for r, x in enumerate(lens)]
    table = [[-1] * P for _ in range(R)]
    em = reserve_by_entries(table, lens, want, [0] * 5, ps)[2]
    t, r, m = gdr2.kv_reserve(ints(table), ints(lens), ints(want), ints([0] * 5), page_size=ps)
    assert m.tolist() == [em] and int((t >= 0).sum()) == 0 and r.tolist() == [0] * 5


@pytest.mark.parametrize("P", [4, 300])
def test_fork_takes_lengths_over_as_they_are(P):
    """A sequence that stays keeps its length, one that takes another's content gets that length, also where it lies
    outside the table; a released one ends at 0."""
    ps, R = 16, 7
    lens = [P * ps + 5, -4, P * ps, 2**31 - 1, 20, 7, -2**31]
    parent = [0, 1, 0, 3, 3, -1, 1]
    table = [[-1] * P for _ in range(R)]
    for r in (0, 3):
        table[r] = list(range(r * P, r * P + P))
    table[1][0], table[5][0] = 6 * P, 6 * P + 1
    num = 6 * P + 2
    refs = [0] * num
    for row in table:
        for e in row:
            if e >= 0:
                refs[e] += 1
    k = torch.randn(num, 1, ps, 64, device="cuda")
    v = torch.randn(num, 1, ps, 64, device="cuda")
    k0, v0 = k.clone(), v.clone()
    t, n, r, m = gdr2.kv_fork(ints(table), ints(lens), ints(refs), ints(parent), k, v)
    assert n.tolist() == [lens[p] if p >= 0 else 0 for p in parent] and m.tolist() == [0]
    # whole pages are shared, nothing is copied; a length below 0 shares none, and the one that stays keeps its page
    assert t.tolist() == [table[0], table[1], table[0], table[3], table[3], [-1] * P, [-1] * P]
    counts = [0] * num
    for e in (e for row in t.tolist() for e in row if e >= 0):
        counts[e] += 1
    assert r.tolist() == counts and torch.equal(k, k0) and torch.equal(v, v0)


def test_decode_of_more_slots_than_a_table_of_their_own_allows():
    """2,100 slots of one sequence with 2^20 table entries: N P is past the bound of a table, R P is not."""
    N, P, n = 2100, 1 << 20, 700
    torch.manual_seed(3)
    k, v = torch.randn(2, n + 3, 2, 1, 64, device="cuda").bfloat16()
    table = torch.full((1, P), -1, dtype=torch.int32, device="cuda")
    table[0, :n] = torch.randperm(n + 3, device="cuda")[:n].int()
    q, seq = torch.randn(N, 8, 64, device="cuda").bfloat16(), torch.zeros(N, dtype=torch.int32, device="cuda")
    o, lse = gdr2.attn_decode(q, k, v, table, ints([n]), seq, want_lse=True)
    for rows in ([0, 1, 1047], [1048, 2098, 2099]):
        ro, rl, to, tl, _ = ref.attention(q[rows], k, v, table, ints([n]), seq[rows])
        ref.check("o", o[rows], ro, to)
        ref.check("lse", lse[rows], rl, tl)


def serving_inputs():
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    R, Hk, d = 24, 2, 64
    x = torch.randn(40, R, 4 + 2 * Hk, d, generator=g, device="cuda").bfloat16()
    return x, torch.randint(0, R, (40, R), generator=g, device="cuda").int(), gdr2.rope_freqs(d)[0]


def serve(x, parents, freqs, chained):
    """Steps of a small server whose table, counts and pools change in place; `chained`, or the GPU waited for after each
    call. Every launch overlaps the end of the one before, which has just written what it reads."""
    R, P, ps, Hk, d, num = 24, 40, 8, 2, 64, 400
    pools = [torch.zeros(num, Hk, ps, d, device="cuda").bfloat16() for _ in range(2)]
    table, refs = torch.full((R, P), -1, dtype=torch.int32, device="cuda"), torch.zeros(num, dtype=torch.int32, device="cuda")
    seq, lens = torch.arange(R, device="cuda").int(), torch.arange(R, device="cuda").int()
    wait = (lambda: None) if chained else torch.cuda.synchronize
    wait()
    out = []
    for i in range(40):
        want = lens + 1
        wait()
        table, refs, _ = gdr2.kv_reserve(table, lens, want, refs, page_size=ps, window=100, out={"table": table, "ref": refs})
        wait()
        q = gdr2.attn_prologue_cache(x[i, :, :4], x[i, :, 4:4 + Hk], x[i, :, 4 + Hk:], None, None, seq, lens, freqs, *pools, table)
        wait()
        out.append(gdr2.attn_decode(q, *pools, table, want, window=100))
        wait()
        table, lens, refs, _ = gdr2.kv_fork(table, want, refs, parents[i], *pools)
        wait()
        table, refs, _ = gdr2.kv_compact(table, refs, *pools, out={"table": table, "ref": refs})
        wait()
        out.append(gdr2.attn_decode(q, *pools, table, lens, window=100))
        wait()
    return out + [table, lens, refs, *pools]


def test_calls_in_a_chain_see_what_the_call_before_wrote():
    x = serving_inputs()
    want = [t.clone() for t in serve(*x, False)]
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(serve(*x, True), want, strict=True))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = serve(*x, True)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want, strict=True))


@pytest.mark.parametrize("B,steps", [(5, 1), (1, 1), (5, 3), (40, 2)])
def test_prologue_of_a_batched_decode_step(B, steps):
    """[B, 1, H, d] views of a fused projection [B, 1, W], or of the last of several steps [B, steps, W]: forward, the
    cache form, and the gradients into a fused gradient of the same layout."""
    Hq, Hk, d, ps = 6, 2, 64, 16
    torch.manual_seed(6)
    W = (Hq + 2 * Hk) * d
    qkv = torch.randn(B, steps, W, device="cuda").bfloat16()[:, -1:]
    cut = lambda t, a, b: t[..., a * d:b * d].unflatten(-1, (b - a, d))  # noqa: E731
    xq, xk, xv = cut(qkv, 0, Hq), cut(qkv, Hq, Hq + Hk), cut(qkv, Hq + Hk, Hq + 2 * Hk)
    assert xq.shape == (B, 1, Hq, d) and (B == 1 or not xq.is_contiguous())
    gain, (freqs, mag) = 1 + 0.2 * torch.randn(d, device="cuda"), gdr2.rope_freqs(32)
    pos = torch.randint(0, 4096, (B, 1), device="cuda").int()
    out = gdr2.attn_prologue_fwd(xq, xk, gain, None, pos, freqs, mag=mag)
    flat = lambda t: t.reshape(B, -1, d)  # noqa: E731
    for n, x, g in (("q", xq, gain), ("k", xk, None)):
        y, tol = ref.prologue(flat(x), g, pos.view(-1), freqs, mag=mag)
        assert out[n].shape == x.shape and out[n].is_contiguous()
        ref.check(n, flat(out[n]), y, tol)
    dq, dk = torch.randn(B, 1, Hq, d, device="cuda").bfloat16(), torch.randn(B, 1, Hk, d, device="cuda").bfloat16()
    want = gdr2.attn_prologue_bwd(xq, xk, gain, None, pos, freqs, dq, dk, mag=mag)
    whole = torch.full((B, steps, W), 7.0, device="cuda").bfloat16()
    grad = whole[:, -1:]
    gdr2.attn_prologue_bwd(xq, xk, gain, None, pos, freqs, dq, dk, mag=mag,
                           out={"dxq": cut(grad, 0, Hq), "dxk": cut(grad, Hq, Hq + Hk)})
    for n, x, g, dy, at in (("dxq", xq, gain, dq, (0, Hq)), ("dxk", xk, None, dk, (Hq, Hq + Hk))):
        dx, _, tol, _ = ref.prologue_grad(flat(x), g, flat(dy), pos.view(-1), freqs, mag=mag)
        ref.check(n, flat(want[n]), dx, tol)
        assert torch.equal(cut(grad, *at), want[n])
    assert (whole[:, :-1] == 7).all() and (cut(grad, Hq + Hk, Hq + 2 * Hk) == 7).all()
    # into a cache, a page for each sequence
    k, v = torch.zeros(2, B, Hk, ps, d, device="cuda").bfloat16()
    table, seq, at = torch.randperm(B, device="cuda").int().view(B, 1), torch.arange(B, device="cuda").int(), pos.view(-1) % ps
    q = gdr2.attn_prologue_cache(xq, xk, xv, gain, None, seq, at, freqs, k, v, table, mag=mag)
    near = gdr2.attn_prologue_fwd(xq, xk, gain, None, at, freqs, mag=mag)
    page = table[:, 0].long()
    assert q.shape == xq.shape and torch.equal(q, near["q"])
    assert torch.equal(k[page, :, at.long()], flat(near["k"])) and torch.equal(v[page, :, at.long()], flat(xv))
    assert int((k != 0).any(-1).sum()) == B * Hk and int((v != 0).any(-1).sum()) == B * Hk


@pytest.mark.parametrize("Hk,ps", [(1, 8), (8, 64)])  # copies inside the cluster's kernel, and by one of their own
def test_fork_and_compaction_captured_and_not(Hk, ps):
    """A captured call copies its pages by another kernel than a small call that the host makes: the same bits."""
    R, P, d, num = 12, 4, 64, 80
    torch.manual_seed(8)
    pools = torch.randn(2, num, Hk, ps, d, device="cuda").bfloat16()
    table = torch.randperm(num, device="cuda")[:R * P].int().view(R, P)
    refs = torch.zeros(num, dtype=torch.int32, device="cuda")
    refs[table.flatten().long()] = 1
    lens, parent = torch.randint(0, P * ps, (R,), device="cuda").int(), torch.randint(-1, R, (R,), device="cuda").int()

    def both(k, v):
        t, n, r, m = gdr2.kv_fork(table, lens, refs, parent, k, v)
        return [t, n, r, m, *gdr2.kv_compact(t, r, k, v), k, v]

    want = both(*pools.clone())
    k, v = pools.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both(k, v)
    for _ in range(2):
        k.copy_(pools[0]), v.copy_(pools[1])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want, strict=True))
    assert not torch.equal(k, pools[0])
