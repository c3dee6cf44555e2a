"""Page bookkeeping of the key-value cache on the GPU against the same rules on Python lists (tests/attn_ref.py): whole
numbers and moved bits have to be equal. And a run of the attention half as it would be used."""
from __future__ import annotations

import random

import pytest
import torch

from gated_delta_rule_65_b200 import gdr2
from tests import attn_ref as ref

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def a_cache(rng, R, P, ps, num, share=True):
    """Lists table, lens, ref of a random state: scattered pages, shared prefixes, pages reserved past the length."""
    order = list(range(num))
    rng.shuffle(order)
    table, lens, refs = [[-1] * P for _ in range(R)], [0] * R, [0] * num
    for r in range(R):
        most = min(P, len(order))
        n = rng.randint(0, most)
        if rng.random() < 0.3:
            n = min(n, 2)
        first = 0
        if share and r and rng.random() < 0.4:
            p = rng.randrange(r)
            first = min(n, rng.randint(0, lens[p] // ps))
            for j in range(first):
                if table[p][j] < 0:
                    first = j
                    break
                table[r][j] = table[p][j]
                refs[table[r][j]] += 1
        for j in range(first, n):
            table[r][j] = order.pop()
            refs[table[r][j]] = 1
        lens[r] = max(first * ps, rng.randint(max(0, (n - 2) * ps), n * ps)) if n else 0
    return table, lens, refs


# R, P, page size, pages: one CTA, clusters of 2 to 8, a strip that ends inside a warp, pools that run out
SHAPES = [(1, 1, 1, 1), (3, 4, 16, 9), (7, 5, 3, 40), (40, 30, 16, 700), (100, 90, 8, 4000), (300, 40, 64, 6001),
          (257, 129, 16, 33000), (1, 9000, 16, 9001), (5000, 2, 16, 5003)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("seed", [1, 2])
def test_reserve(shape, seed):
    R, P, ps, num = shape
    rng = random.Random(seed)
    table, lens, refs = a_cache(rng, R, P, ps, num)
    want = [x + rng.choice([0, 1, 1, ps, 3 * ps, -5]) for x in lens]
    if R == 1:
        want = [P * ps + (2 * ps if seed == 2 else 0)]
    if seed == 2:
        table[0][0] = -9
        table[-1][-1] = num + 3
    for window in (0, 2 * ps + 1):
        t, r, m = gdr2.kv_reserve(ints(table), ints(lens), ints(want), ints(refs), page_size=ps, window=window)
        et, er, em = ref.reserve(table, lens, want, refs, ps, window)
        assert t.tolist() == et and r.tolist() == er and m.tolist() == [em]
        # in place
        tt, rr = ints(table), ints(refs)
        out = gdr2.kv_reserve(tt, ints(lens), ints(want), rr, page_size=ps, window=window, out={"table": tt, "ref": rr})
        assert out[0] is tt and tt.tolist() == et and rr.tolist() == er


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("how", ["mixed", "one parent", "all released", "rotated", "stay"])
def test_fork(shape, how):
    R, P, ps, num = shape
    rng = random.Random(R + P)
    table, lens, refs = a_cache(rng, R, P, ps, num)
    parent = {"mixed": [rng.choice([r, rng.randrange(R), -1, R, rng.randrange(R)]) for r in range(R)],
              "one parent": [R // 2] * R, "all released": [-1] * R, "rotated": [(r + 1) % R for r in range(R)],
              "stay": list(range(R))}[how]
    Hk, d = 2, 64
    k = torch.randn(num, Hk, ps, d, device="cuda").bfloat16()
    v = torch.randn(num, Hk, ps, d, device="cuda").bfloat16()
    ek, ev = k.clone(), v.clone()
    et, el, er, em, copies = ref.fork(table, lens, refs, parent, ps)
    for src, dst, n in copies:
        ek[dst, :, :n], ev[dst, :, :n] = k[src, :, :n], v[src, :, :n]
    t, n, r, m = gdr2.kv_fork(ints(table), ints(lens), ints(refs), ints(parent), k, v)
    assert t.tolist() == et and n.tolist() == el and r.tolist() == er and m.tolist() == [em]
    assert torch.equal(k, ek) and torch.equal(v, ev)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_compact(shape, dtype):
    R, P, ps, num = shape
    rng = random.Random(R * 3 + P)
    table, lens, refs = a_cache(rng, R, P, ps, num)
    refs[-1] += 1  # a pinned page
    if num > 4:
        refs[1] = -2  # free, whatever lies below zero
        table = [[-1 if e == 1 else e for e in row] for row in table]
    Hk, d = 3, 64
    k = torch.randn(num, Hk, ps, d, device="cuda").to(dtype)
    v = torch.randn(num, Hk, ps, d, device="cuda").to(dtype)
    et, er, el, moves = ref.compact(table, refs)
    ek, ev = k.clone(), v.clone()
    for a, b in moves:
        ek[b], ev[b] = k[a], v[a]
    t0, r0 = ints(table), ints(refs)
    for out in (None, {"table": t0, "ref": r0}):
        kk, vv = k.clone(), v.clone()
        t, r, live = gdr2.kv_compact(t0, r0, kk, vv, out=out)
        assert t.tolist() == et and r.tolist() == er and live.tolist() == [el]
        assert torch.equal(kk, ek) and torch.equal(vv, ev)


def test_empty_and_full_pools():
    k = torch.randn(5, 1, 4, 64, device="cuda")
    v = torch.randn(5, 1, 4, 64, device="cuda")
    t, r, live = gdr2.kv_compact(ints([[-1, -1]]), ints([0] * 5), k, v)
    assert live.tolist() == [0] and r.tolist() == [0] * 5 and t.tolist() == [[-1, -1]]
    t, r, live = gdr2.kv_compact(ints([[4, 2, 0, 1, 3]]), ints([1] * 5), k, v)
    assert live.tolist() == [5] and t.tolist() == [[4, 2, 0, 1, 3]]
    t, r, m = gdr2.kv_reserve(ints([[4, 2, 0, 1, 3, -1]]), ints([20]), ints([21]), ints([1] * 5), page_size=4)
    assert m.tolist() == [1] and t.tolist() == [[4, 2, 0, 1, 3, -1]]


def test_missing_pages_are_held_to_32_bits():
    table = [[-1, -1], [0, -1], [-1, -1]]
    for want in ([2**31 - 1, 5, 0], [2**31 - 1] * 3, [2**31 - 1, 3, 2], [2, 3, 4]):
        t, r, m = ref.reserve(table, [0, 1, 0], want, [1, 0, 0], 1)
        to, ro, mo = gdr2.kv_reserve(ints(table), ints([0, 1, 0]), ints(want), ints([1, 0, 0]), page_size=1)
        assert (to.tolist(), ro.tolist(), mo.tolist()) == (t, r, [min(m, 2**31 - 1)])


@pytest.mark.parametrize("num", [4, 40000])
def test_compact_largest_table(num):
    """The table of the largest allowed size, in place (8.6 GB): places up to its end and a step of the grid behind."""
    P = 0x7fff0000
    table = torch.full((1, P), -1, dtype=torch.int32, device="cuda")
    last = [num - 1, num - 2, 0]
    table[0, -3:] = ints(last)
    table[0, 5] = num - 2
    refs = torch.zeros(num, dtype=torch.int32, device="cuda")
    refs[num - 1], refs[num - 2], refs[0] = 1, 2, 1
    k = torch.randn(num, 1, 1, 64, device="cuda").bfloat16()
    v = torch.randn(num, 1, 1, 64, device="cuda").bfloat16()
    k0, v0 = k.clone(), v.clone()
    t, r, live = gdr2.kv_compact(table, refs, k, v, out={"table": table})
    assert t is table and live.tolist() == [3]
    moved = {0: 0, num - 2: 1 if num > 4 else 2, num - 1: 2 if num > 4 else 1}  # 4 pages: 3 moves to 1, 2 stays
    assert t[0, -3:].tolist() == [moved[x] for x in last] and t[0, 5].item() == moved[num - 2]
    assert int((t >= 0).sum()) == 4 and r[:3].sum().item() == 4 and int((r > 0).sum()) == 3
    for a, b in moved.items():
        assert torch.equal(k[b], k0[a]) and torch.equal(v[b], v0[a])
    del table, t
    torch.cuda.empty_cache()


def test_captured_bookkeeping():
    """reserve, fork and compact as one captured graph, replayed twice on the same inputs."""
    rng = random.Random(3)
    R, P, ps, num = 20, 12, 16, 400
    table, lens, refs = a_cache(rng, R, P, ps, num)
    parent = [rng.randrange(-1, R) for _ in range(R)]
    want = [x + 1 for x in lens]
    T, L, F, W, Q = ints(table), ints(lens), ints(refs), ints(want), ints(parent)
    k0 = torch.randn(num, 2, ps, 64, device="cuda")
    k, v = k0.clone(), k0.clone()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        a = gdr2.kv_reserve(T, L, W, F, page_size=ps)
        b = gdr2.kv_fork(a[0], W, a[1], Q, k, v)
        c = gdr2.kv_compact(b[0], b[2], k, v)
    t1, r1, m1 = ref.reserve(table, lens, want, refs, ps)
    t2, l2, r2, m2, copies = ref.fork(t1, want, r1, parent, ps)
    t3, r3, live, moves = ref.compact(t2, r2)
    e = k0.clone()
    for src, dst, n in copies:
        e[dst, :, :n] = k0[src, :, :n]
    f = e.clone()
    for s, d in moves:
        f[d] = e[s]
    for _ in range(2):
        k.copy_(k0), v.copy_(k0)
        gr.replay()
        torch.cuda.synchronize()
        assert (a[0].tolist(), a[1].tolist(), a[2].tolist()) == (t1, r1, [m1])
        assert (b[0].tolist(), b[1].tolist(), b[2].tolist(), b[3].tolist()) == (t2, l2, r2, [m2])
        assert (c[0].tolist(), c[1].tolist(), c[2].tolist()) == (t3, r3, [live])
        assert torch.equal(k, f) and torch.equal(v, f)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("window", [0, 40])
def test_serving_run(dtype, window):
    """Prompts, decode steps, a fork with a release, more steps, a compaction, more steps: at every step the attention
    of each sequence equals the definition over its own history of finished keys and values, kept on the side."""
    g = torch.Generator(device="cuda")
    g.manual_seed(31)
    R, P, ps, num, Hq, Hk, d = 5, 12, 16, 60, 6, 2, 64
    k = torch.full((num, Hk, ps, d), float("nan"), device="cuda").to(dtype)
    v = k.clone()
    table, refs, lens = torch.full((R, P), -1, dtype=torch.int32, device="cuda"), ints([0] * num), ints([0] * R)
    gq, gk = 1 + 0.1 * torch.randn(d, generator=g, device="cuda"), 1 + 0.1 * torch.randn(d, generator=g, device="cuda")
    fr, mag = gdr2.rope_freqs(32, scaling="parts", factor=4.0, orig_len=64, turns_high=8.0)
    hist = [([], []) for _ in range(R)]  # rows of xk, xv by sequence, with their positions

    def append(counts):
        nonlocal table, refs, lens
        seq = torch.repeat_interleave(torch.arange(R), torch.tensor(counts)).int().cuda()
        at = lens.tolist()
        pos = ints([at[r] + i for r in range(R) for i in range(counts[r])])
        want = lens + ints(counts)
        table, refs, missing = gdr2.kv_reserve(table, lens, want, refs, page_size=ps, window=window)
        assert missing.item() == 0
        T = sum(counts)
        x = torch.randn(T, Hq + 2 * Hk, d, generator=g, device="cuda").to(dtype)
        q = gdr2.attn_prologue_cache(x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:], gq, gk, seq, pos, fr, k, v, table, mag=mag)
        keys = gdr2.attn_prologue_fwd(x[:, :Hq], x[:, Hq:Hq + Hk], gq, gk, pos, fr, mag=mag)
        assert torch.equal(keys["q"], q)
        for t, r in enumerate(seq.tolist()):
            hist[r][0].append(keys["k"][t])
            hist[r][1].append(x[t, Hq + Hk:])
        lens = want
        return q, seq

    def step():
        q, seq = append([1] * R)
        o = gdr2.attn_decode(q, k, v, table, lens, seq, window=window)
        for r in range(R):
            n = len(hist[r][0])
            a = max(0, n - window) if window else 0
            kk, vv = torch.stack(hist[r][0][a:], 1), torch.stack(hist[r][1][a:], 1)  # [Hk, n, d]
            one = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
            ro, _, to, _, _ = ref.attention(q[r:r + 1], kk[None], vv[None], one, ints([n - a]))
            ref.check("o", o[r:r + 1], ro, to)
        assert torch.equal(refs.clamp(min=0), torch.bincount(table[table >= 0].long(), minlength=num).int())

    append([33, 1, 50, 16, 7])
    for _ in range(3):
        step()
    parent = [2, 1, 2, -1, 0]
    table, lens, refs, missing = gdr2.kv_fork(table, lens, refs, ints(parent), k, v)
    hist = [(list(hist[p][0]), list(hist[p][1])) if p >= 0 else ([], []) for p in parent]
    assert missing.item() == 0 and lens.tolist() == [len(h[0]) for h in hist]
    for _ in range(20):
        step()
    table, refs, live = gdr2.kv_compact(table, refs, k, v)
    assert live.item() == int((refs > 0).sum()) and int(table.max()) < live.item()
    for _ in range(3):
        step()
    assert gdr2.check() == gdr2.OK
