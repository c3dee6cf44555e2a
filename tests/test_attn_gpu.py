"""The attention half of the hybrid cell on the GPU against plain 64-bit forms (tests/attn_ref.py, which derives the
bounds): query / key prologue with its gradients, the prologue that writes the cache, attention of one new token."""
from __future__ import annotations

import math
import os
import subprocess
import sys

import pytest
import torch

from gated_delta_rule_65_b200 import gdr2
from tests import attn_ref as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def rows(g, T, H, d, dtype, extra=0):
    """[T, H, d], cut out of wider rows when extra > 0."""
    if not extra:
        return randn(g, T, H, d, dtype=dtype)
    wide = randn(g, T, (H + extra) * d, dtype=dtype)
    return wide[:, :H * d].view(T, H, d)


PROLOGUE = [
    # T, Hq, Hk, d, rot, interleaved, norm, dtype, extra heads of the fused row, first position
    (1, 1, 1, 64, 64, False, True, "f32", 0, 0),
    (1, 16, 2, 128, 128, True, True, "bf16", 3, 70001),
    (2, 3, 1, 128, 32, False, True, "f32", 2, 1 << 30),
    (17, 5, 5, 64, 16, True, True, "bf16", 0, 3),
    (63, 7, 1, 128, 48, False, True, "bf16", 1, 999),
    (300, 2, 1, 64, 32, True, False, "f32", 1, 65536),
    (130, 4, 4, 128, 128, False, False, "bf16", 0, 12),
    (77, 33, 11, 64, 48, False, True, "f32", 4, 0),
    (50, 2, 2, 128, 0, False, True, "bf16", 0, 0),
    (1500, 1, 1, 128, 64, True, True, "f32", 0, 0),
    (2500, 16, 8, 128, 128, False, True, "bf16", 8, 500000),
    # heads that do not fill a warp's rows, tokens enough that several share it, the last block not full
    (38003, 1, 1, 64, 64, False, True, "bf16", 0, 90000),
    (20003, 6, 2, 64, 48, True, True, "bf16", 1, 0),
    (19011, 3, 1, 128, 128, True, True, "bf16", 0, 17),
    (12001, 2, 2, 128, 32, False, False, "bf16", 0, 0),
    (19015, 1, 3, 64, 64, False, True, "f32", 0, 5),
    (9503, 5, 1, 128, 128, True, True, "f32", 2, 1 << 20),
]


def prologue_case(c):
    T, Hq, Hk, d, rot, inter, norm, dt, extra, p0 = c
    g = gen(7 * T + 3 * Hq + d + rot + len(dt))
    x = {"xq": rows(g, T, Hq, d, DT[dt], extra), "xk": rows(g, T, Hk, d, DT[dt], extra)}
    x["gq"], x["gk"] = (1 + 0.3 * randn(g, d), -1 + 0.3 * randn(g, d)) if norm else (None, None)
    x["pos"] = (p0 + torch.randperm(T, generator=g, device="cuda")).int() if rot else None
    x["freqs"], mag = gdr2.rope_freqs(rot, scaling="parts", factor=8.0, orig_len=4096) if rot else (None, 1.0)
    return x, dict(norm=norm, mag=mag, interleaved=inter, eps=1e-5), g


@pytest.mark.parametrize("c", PROLOGUE, ids=lambda c: "-".join(map(str, c)))
def test_prologue(c):
    x, kw, g = prologue_case(c)
    out = gdr2.attn_prologue_fwd(x["xq"], x["xk"], x["gq"], x["gk"], x["pos"], x["freqs"], **kw)
    for n in ("q", "k"):
        y, tol = ref.prologue(x["x" + n], x["g" + n], x["pos"], x["freqs"], **kw)
        ref.check(n, out[n], y, tol)
    T, Hq, Hk, d, dt = c[0], c[1], c[2], c[3], DT[c[7]]
    dq, dk = randn(g, T, Hq, d, dtype=dt), randn(g, T, Hk, d, dtype=dt)
    args = (x["xq"], x["xk"], x["gq"], x["gk"], x["pos"], x["freqs"], dq, dk)
    got = gdr2.attn_prologue_bwd(*args, **kw)
    assert ("dgq" in got) == kw["norm"]
    for n, dy in (("q", dq), ("k", dk)):
        dx, dg, tol, size = ref.prologue_grad(x["x" + n], x["g" + n], dy, x["pos"], x["freqs"], **kw)
        ref.check("dx" + n, got["dx" + n], dx, tol)
        if kw["norm"]:  # a lane adds up to T H / 148 terms, then 16 or 32 groups and 296 blocks: depth below this
            ref.check("dg" + n, got["dg" + n], dg, (64 + T * x["x" + n].shape[1] / 148 + 64) * ref.U * size)
    again = gdr2.attn_prologue_bwd(*args, **kw)
    for n in got:
        assert torch.equal(got[n], again[n]), n


def test_prologue_batched_views_and_fused_gradient():
    """[B, T, H, d] views of a fused q | k | v projection, their gradients written into one fused gradient."""
    B, T, Hq, Hk, d = 2, 37, 6, 2, 64
    g = gen(5)
    qkv = randn(g, B, T, (Hq + 2 * Hk) * d, dtype=torch.bfloat16)
    xq = qkv[..., :Hq * d].view(B, T, Hq, d)
    xk = qkv[..., Hq * d:(Hq + Hk) * d].view(B, T, Hk, d)
    pos = torch.arange(T, device="cuda", dtype=torch.int32).repeat(B, 1)
    fr, _ = gdr2.rope_freqs(d)
    out = gdr2.attn_prologue_fwd(xq, xk, None, None, pos, fr)
    assert out["q"].shape == xq.shape and out["k"].shape == xk.shape
    y, tol = ref.prologue(xq.reshape(-1, Hq, d), None, pos.view(-1), fr)
    ref.check("q", out["q"].view(-1, Hq, d), y, tol)
    dq, dk = randn(g, B, T, Hq, d, dtype=torch.bfloat16), randn(g, B, T, Hk, d, dtype=torch.bfloat16)
    grad = torch.full_like(qkv, 7.0)
    fused = {"dxq": grad[..., :Hq * d].view(B, T, Hq, d), "dxk": grad[..., Hq * d:(Hq + Hk) * d].view(B, T, Hk, d)}
    gdr2.attn_prologue_bwd(xq, xk, None, None, pos, fr, dq, dk, out=fused)
    dx, _, tol, _ = ref.prologue_grad(xk.reshape(-1, Hk, d), None, dk.view(-1, Hk, d), pos.view(-1), fr)
    ref.check("dxk", fused["dxk"].reshape(-1, Hk, d), dx, tol)
    assert (grad[..., (Hq + Hk) * d:] == 7).all()


def test_prologue_gradient_against_differences():
    """<dx, v> and <dg, v> against central differences of the kernel's own fp32 forward. h = 2^-7: the third-order term
    is below h^2 of the loss's scale (1e-4), rounding below 32 u / h (5e-4): 1e-3 of the sum of |y dy|."""
    T, H, d, h = 40, 3, 64, 2.0 ** -7
    g = gen(6)
    x, gain, dy = randn(g, T, H, d), 1 + 0.2 * randn(g, d), randn(g, T, H, d)
    pos = torch.arange(T, device="cuda", dtype=torch.int32) * 977
    fr, mag = gdr2.rope_freqs(32, scaling="linear", factor=4.0)
    kw = dict(mag=mag, interleaved=True)

    def loss(x, gain):
        y = gdr2.attn_prologue_fwd(x, x, gain, gain, pos, fr, **kw)["q"].double()
        return float((y * dy.double()).sum()), float((y * dy.double()).abs().sum())

    got = gdr2.attn_prologue_bwd(x, x, gain, gain, pos, fr, dy, dy, **kw)
    vx, vg = randn(g, T, H, d), randn(g, d)
    size = loss(x, gain)[1]
    for name, v, (a, b) in (("dxq", vx, ((x + h * vx, gain), (x - h * vx, gain))),
                            ("dgq", vg, ((x, gain + h * vg), (x, gain - h * vg)))):
        diff = (loss(*a)[0] - loss(*b)[0]) / (2 * h)
        assert abs(diff - float((got[name].double() * v.double()).sum())) <= 1e-3 * size, name


def test_prologue_zero_rows_and_infinities_outside_the_rotation():
    """A row of zeros stays zero with a finite gradient; an infinity in an unrotated channel stays in its channel."""
    x = torch.zeros(3, 2, 64, device="cuda")
    pos = torch.arange(3, device="cuda", dtype=torch.int32)
    fr, _ = gdr2.rope_freqs(32)
    out = gdr2.attn_prologue_fwd(x, x, None, None, pos, fr)
    assert (out["q"] == 0).all()
    got = gdr2.attn_prologue_bwd(x, x, None, None, pos, fr, torch.ones_like(x), torch.ones_like(x))
    assert torch.isfinite(got["dxq"]).all() and (got["dgq"] == 0).all()
    x[1, 1, 40] = math.inf
    for inter in (False, True):
        y = gdr2.attn_prologue_fwd(x, x, None, None, pos, fr, norm=False, interleaved=inter)["q"]
        assert y[1, 1, 40] == math.inf and int((y == 0).sum()) == y.numel() - 1


def test_prologue_on_another_stream_and_in_a_graph():
    x, kw, g = prologue_case(PROLOGUE[3])
    a = (x["xq"], x["xk"], x["gq"], x["gk"], x["pos"], x["freqs"])
    want = gdr2.attn_prologue_fwd(*a, **kw)
    dq, dk = torch.randn_like(want["q"]), torch.randn_like(want["k"])
    grads = gdr2.attn_prologue_bwd(*a, dq, dk, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = gdr2.attn_prologue_bwd(*a, dq, dk, **kw, stream=side)
    side.synchronize()
    for n in got:
        assert torch.equal(got[n], grads[n])
    out = {n: torch.zeros_like(t) for n, t in want.items()}
    gout = {n: torch.zeros_like(t) for n, t in grads.items()}
    ws = torch.empty(int(gdr2.lib().gdr2_attn_prologue_workspace_bytes(x["xq"].shape[-1])), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdr2.attn_prologue_fwd(*a, **kw, out=out)
        gdr2.attn_prologue_bwd(*a, dq, dk, **kw, out=gout, workspace=ws)
    for _ in range(2):
        for t in (*out.values(), *gout.values()):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for n in out:
            assert torch.equal(out[n], want[n])
        for n in gout:
            assert torch.equal(gout[n], grads[n])


def test_prologue_without_gradients_of_the_gains():
    """out without dgq and dgk: no workspace, the same dxq, dxk; out with one of them: only that one."""
    x, kw, g = prologue_case(PROLOGUE[3])
    a = (x["xq"], x["xk"], x["gq"], x["gk"], x["pos"], x["freqs"])
    dq, dk = torch.randn_like(x["xq"]), torch.randn_like(x["xk"])
    want = gdr2.attn_prologue_bwd(*a, dq, dk, **kw)
    for only in ((), ("dgk",)):
        out = {n: torch.empty_like(want[n]) for n in ("dxq", "dxk", *only)}
        assert gdr2.attn_prologue_bwd(*a, dq, dk, **kw, out=out) is out
        for n in out:
            assert torch.equal(out[n], want[n]), n


CAPTURE = """
import torch
from gated_delta_rule_65_b200 import gdr2
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
q = torch.randn(2, 8, 128, device="cuda").bfloat16()
kv = torch.randn(2, 4, 128, device="cuda").bfloat16()
k, v = torch.randn(2, 90, 2, 16, 128, device="cuda").bfloat16()
table = torch.arange(90, dtype=torch.int32, device="cuda").view(2, 45)
lens, seq, pos, ref, parent = i32([700, 33]), i32([0, 1]), i32([699, 32]), i32([1] * 90), i32([0, 1])
freqs, _ = gdr2.rope_freqs(128)
def step():
    t, r, _ = gdr2.kv_reserve(table, lens, lens, ref, page_size=16)
    y = gdr2.attn_prologue_cache(q, kv[:, :2], kv[:, 2:], None, None, seq, pos, freqs, k, v, t)
    o = gdr2.attn_decode(y, k, v, t, lens)
    g = gdr2.attn_prologue_bwd(q, kv, None, None, pos, freqs, q, kv)
    f = gdr2.attn_prologue_fwd(q, kv, None, None, pos, freqs)
    t, n, r, _ = gdr2.kv_fork(t, lens, r, parent, k, v)
    return (o, *g.values(), *f.values(), t, n, *gdr2.kv_compact(t, r, k, v))
graph = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(graph):
    got = step()
graph.replay()
torch.cuda.synchronize()
got = [x.clone() for x in got]
assert all(torch.equal(x, y) for x, y in zip(got, step()))
print("captured first")
"""


def test_first_call_of_a_process_inside_a_capture():
    """Nothing has to run before the first capture: a fresh process captures every kernel's first launch."""
    r = subprocess.run([sys.executable, "-c", CAPTURE], capture_output=True, text=True, timeout=240,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and "captured first" in r.stdout, r.stderr[-2000:]


# ---- the cache -----------------------------------------------------------------------------------------------


def cache(g, lens, ps, Hk, d, dtype, spare=3, P=None):
    """Pools, a table that holds `lens` tokens on scattered pages, counts."""
    P = P or max(1, max(-(-x // ps) for x in lens) + 1)
    held = [-(-x // ps) for x in lens]
    num = sum(held) + spare
    order = torch.randperm(num, generator=g, device="cuda").tolist()
    table, refs = [[-1] * P for _ in lens], [0] * num
    for r, n in enumerate(held):
        for j in range(n):
            table[r][j] = order.pop()
            refs[table[r][j]] = 1
    t = torch.tensor(table, dtype=torch.int32, device="cuda")
    return (randn(g, num, Hk, ps, d, dtype=dtype), randn(g, num, Hk, ps, d, dtype=dtype), t,
            torch.tensor(lens, dtype=torch.int32, device="cuda"), torch.tensor(refs, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("d,Hq,Hk,ps,inter", [(128, 8, 2, 16, False), (64, 3, 3, 7, True), (128, 5, 1, 1, True),
                                              (64, 17, 4, 40, False)])
def test_cache_prologue(dt, d, Hq, Hk, ps, inter):
    """Prompts, single tokens, padding, missing pages and places off the table in one call; everything that is not a
    new token's place keeps its bits."""
    g = gen(11 + d + ps)
    k0, v0, table, lens, _ = cache(g, [70, 9, 1, 130], ps, Hk, d, DT[dt])
    R, P = table.shape
    num = k0.shape[0]
    table[3, 0] = -1
    table[3, 1] = num  # not a page either
    tok = [(0, i) for i in range(70)] + [(1, 8), (-1, 0), (2, 0), (R, 3), (3, 0), (3, ps), (3, 129), (1, P * ps), (1, -1)]
    T = len(tok)
    seq = torch.tensor([a for a, _ in tok], dtype=torch.int32, device="cuda")
    pos = torch.tensor([b for _, b in tok], dtype=torch.int32, device="cuda")
    qkv = randn(g, T, (Hq + 2 * Hk) * d, dtype=DT[dt])
    xq, xk, xv = (qkv[:, a * d:b * d].view(T, b - a, d) for a, b in ((0, Hq), (Hq, Hq + Hk), (Hq + Hk, Hq + 2 * Hk)))
    gq, gk = 1 + 0.2 * randn(g, d), 1 + 0.2 * randn(g, d)
    fr, _ = gdr2.rope_freqs(32)
    k, v = k0.clone(), v0.clone()
    q = torch.full((T, Hq, d), 5.0, dtype=DT[dt], device="cuda")
    assert gdr2.attn_prologue_cache(xq, xk, xv, gq, gk, seq, pos, fr, k, v, table, interleaved=inter, q=q) is q
    kw = dict(interleaved=inter)
    y, tol = ref.prologue(xq, gq, pos, fr, **kw)
    z, tolk = ref.prologue(xk, gk, pos, fr, **kw)
    live = torch.tensor([0 <= a < R for a, _ in tok], device="cuda")
    ref.check("q", q[live], y[live], tol[live])
    assert (q[~live] == 5).all()
    kr, vr, tk = k0.double(), v0.clone(), torch.zeros_like(k0, dtype=torch.float64)
    tab = table.tolist()
    for t, (r, p) in enumerate(tok):
        if 0 <= r < R and 0 <= p < P * ps and 0 <= tab[r][p // ps] < num:
            at = (tab[r][p // ps], slice(None), p % ps)
            kr[at], vr[at], tk[at] = z[t], xv[t], tolk[t] + ref.HALF[DT[dt]] * z[t].abs()
    assert torch.equal(v, vr)
    err = (k.double() - kr).abs()
    assert (err <= tk).all() and int((tk > 0).sum()) > 0  # a bound of 0 where nothing was written


@pytest.mark.parametrize("d,Hq,Hk,dt", [(64, 1, 1, "bf16"), (128, 3, 1, "bf16"), (64, 2, 2, "f32")])
def test_cache_prologue_tokens_share_a_warp(d, Hq, Hk, dt):
    """Few heads and many tokens: several tokens of a warp, each with its own sequence, page, and none at times."""
    g = gen(5 + d + Hq)
    R, n, ps, num = 4, 10001, 16, 2600
    P = -(-n // ps)
    T = R * n + 3
    table = torch.randperm(num, generator=g, device="cuda")[:R * P].view(R, P).int()
    table[1, 5], table[2, 7] = -1, num
    seq = torch.cat([torch.arange(R, device="cuda").repeat_interleave(n), torch.tensor([0, -1, R], device="cuda")]).int()
    pos = torch.cat([torch.arange(n, device="cuda").repeat(R), torch.tensor([P * ps, 0, 0], device="cuda")]).int()
    seq[::97] = -1
    order = torch.randperm(T, generator=g, device="cuda")
    seq, pos = seq[order], pos[order]
    xq, xk, xv = (randn(g, T, h, d, dtype=DT[dt]) for h in (Hq, Hk, Hk))
    gq, gk = 1 + 0.2 * randn(g, d), 1 + 0.2 * randn(g, d)
    fr, _ = gdr2.rope_freqs(d)
    k0, v0 = randn(g, num, Hk, ps, d, dtype=DT[dt]), randn(g, num, Hk, ps, d, dtype=DT[dt])
    k, v = k0.clone(), v0.clone()
    q = torch.full((T, Hq, d), 5.0, dtype=DT[dt], device="cuda")
    gdr2.attn_prologue_cache(xq, xk, xv, gq, gk, seq, pos, fr, k, v, table, q=q)
    live = (seq >= 0) & (seq < R)
    y, tol = ref.prologue(xq, gq, pos, fr)
    ref.check("q", q[live], y[live], tol[live])
    assert (q[~live] == 5).all()
    put = live & (pos < P * ps)
    page = table[seq[put].long(), pos[put].long() // ps].long()
    ok = (page >= 0) & (page < num)
    page, at = page[ok], pos[put][ok].long() % ps
    z, tolk = ref.prologue(xk, gk, pos, fr)
    z, tolk = z[put][ok], tolk[put][ok]
    ref.check("k", k[page, :, at], z, tolk)
    vr = v0.clone()
    vr[page, :, at] = xv[put][ok]
    assert torch.equal(v, vr)
    k[page, :, at] = k0[page, :, at]
    assert torch.equal(k, k0)


DECODE = [
    # lens, Hq, Hk, d, ps, window, dtype
    ([1], 1, 1, 64, 16, 0, "bf16"),
    ([0], 4, 2, 128, 16, 0, "bf16"),
    ([0, 1, 15, 16, 17, 63, 64, 65, 128], 8, 2, 128, 16, 0, "bf16"),
    ([0, 1, 15, 16, 17, 63, 64, 65, 128], 6, 3, 64, 16, 0, "f32"),
    ([333], 16, 2, 64, 24, 0, "bf16"),
    ([5000, 3, 777], 7, 1, 128, 64, 0, "bf16"),
    ([5000, 3, 777], 7, 1, 128, 64, 0, "f32"),
    ([900, 100, 2000], 9, 1, 128, 1, 0, "bf16"),
    ([900, 100, 2000], 32, 2, 64, 7, 0, "bf16"),
    ([900, 100, 1100], 17, 1, 128, 300, 0, "bf16"),
    ([900, 100, 1100], 33, 1, 64, 32, 0, "f32"),
    ([900, 100, 1100], 16, 16, 128, 32, 0, "f32"),
    ([900, 100, 1100], 16, 4, 128, 8, 0, "f32"),
    ([400, 100, 130], 16, 16, 128, 16, 0, "bf16"),
    ([2000, 17, 513, 512, 1], 8, 2, 128, 16, 512, "bf16"),
    ([2000, 17, 513, 512, 1], 4, 4, 64, 48, 1, "f32"),
    ([37 * (i % 11) for i in range(300)], 4, 2, 64, 16, 100, "bf16"),
    ([20011], 8, 1, 128, 128, 0, "bf16"),
    ([30001, 2], 2, 1, 64, 16, 0, "f32"),
    # more rows than CTAs, some cut by their borders
    ([(i * 97) % 700 for i in range(150)], 8, 4, 64, 16, 0, "bf16"),
    ([(i * 97) % 400 for i in range(170)], 3, 3, 128, 16, 0, "f32"),
    # more sequences than a CTA has threads, most of them empty
    ([(i * 7919) % 23 if i % 3 == 0 else 0 for i in range(3000)], 2, 1, 64, 8, 0, "bf16"),
]


@pytest.mark.parametrize("c", DECODE, ids=lambda c: f"N{len(c[0])}-{max(c[0])}-{c[1]}x{c[2]}x{c[3]}-ps{c[4]}-w{c[5]}-{c[6]}")
def test_decode(c):
    lens, Hq, Hk, d, ps, window, dt = c
    g = gen(len(lens) + Hq * 7 + d + ps)
    k, v, table, ln, _ = cache(g, lens, ps, Hk, d, DT[dt])
    # nothing outside the attended tokens counts: NaN there
    seen = torch.zeros(k.shape[0], ps, dtype=torch.bool, device="cuda")
    tab = table.tolist()
    for r, x in enumerate(lens):
        i = torch.arange(max(0, x - window) if window else 0, x, device="cuda")
        seen[table[r].long()[i // ps], i % ps] = True
    for pool in (k, v):
        pool.masked_fill_(~seen[:, None, :, None], math.nan)
    q = (2 * randn(g, len(lens), Hq, d)).to(DT[dt])
    o, lse = gdr2.attn_decode(q, k, v, table, ln, window=window, want_lse=True)
    ro, rl, to, tl, _ = ref.attention(q, k, v, table, ln, window=window)
    ref.check("o", o, ro, to)
    ref.check("lse", lse, rl, tl)
    o2 = gdr2.attn_decode(q, k, v, table, ln, window=window)
    assert torch.equal(o, o2)
    assert gdr2.check() == gdr2.OK


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_decode_slots_missing_pages_and_lengths_off_the_table(dt):
    """seq in any order with padding and one sequence twice; pages that are not there; lengths past the table."""
    g = gen(21)
    k, v, table, lens, _ = cache(g, [200, 90, 0, 33, 400], 16, 2, 64, DT[dt], P=25)
    num = k.shape[0]
    table[0, 3] = -1
    table[1, :] = -1
    table[4, 0:20] = num + 5
    lens[4] = 1 << 30
    lens[2] = -7
    seq = torch.tensor([4, 0, -1, 0, 2, 5, 3, 1], dtype=torch.int32, device="cuda")
    q = randn(g, 8, 6, 64, dtype=DT[dt])
    o = torch.full((8, 6, 64), 3.0, dtype=DT[dt], device="cuda")
    lse = torch.full((8, 6), 4.0, device="cuda")
    gdr2.attn_decode(q, k, v, table, lens, seq, scale=0.2, o=o, lse=lse)
    ro, rl, to, tl, pad = ref.attention(q, k, v, table, lens, seq, scale=0.2)
    assert pad == [2, 5] and (o[pad] == 3).all() and (lse[pad] == 4).all()
    keep = [0, 1, 3, 4, 6, 7]
    ref.check("o", o[keep], ro[keep], to[keep])
    ref.check("lse", lse[keep], rl[keep], tl[keep])
    assert (o[[4, 7]] == 0).all() and (lse[[4, 7]] == -math.inf).all()


@pytest.mark.parametrize("dt,G", [("bf16", 4), ("bf16", 12), ("f32", 2), ("f32", 8)])
@pytest.mark.parametrize("scale", [-0.3, 0.0, 1.7])
def test_decode_scales(dt, G, scale):
    """A negative scale turns the order of the scores, a scale of zero weighs all tokens alike."""
    g = gen(26)
    k, v, table, lens, _ = cache(g, [700, 1, 90], 16, 2, 64, DT[dt])
    q = randn(g, 3, 2 * G, 64, dtype=DT[dt])
    o, lse = gdr2.attn_decode(q, k, v, table, lens, scale=scale, want_lse=True)
    ro, rl, to, tl, _ = ref.attention(q, k, v, table, lens, scale=scale)
    ref.check("o", o, ro, to)
    ref.check("lse", lse, rl, tl)


def test_captured_behind_memsets_and_other_streams():
    """Launches that follow a memset, a copy, and work of another stream inside one capture wait for all of them."""
    g = gen(27)
    k0, v0, table, lens, ref_ = cache(g, [600, 40], 16, 2, 64, torch.bfloat16)
    q0 = randn(g, 2, 8, 64, dtype=torch.bfloat16)
    k, v, q, n = torch.empty_like(k0), torch.empty_like(v0), torch.empty_like(q0), torch.empty_like(lens)
    want = gdr2.attn_decode(q0, k0, v0, table, lens)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        k.zero_(), n.zero_()
        k.copy_(k0)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            for _ in range(20):
                v.copy_(v0)
            q.zero_()
            q.copy_(q0)
        n.copy_(lens)
        main.wait_stream(side)
        o = gdr2.attn_decode(q, k, v, table, n)
        t, r, _ = gdr2.kv_reserve(table, n, n + 1, ref_, page_size=16)
        o2 = gdr2.attn_decode(q, k, v, t, n)
    for _ in range(3):
        for x in (k, v, q):
            x.fill_(math.nan)
        n.fill_(-1)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.equal(o2, want)


def test_decode_extreme_scores():
    """Scores of +-10^4 (one token takes all) and scores that are all equal."""
    g = gen(22)
    k, v, table, lens, _ = cache(g, [300, 300], 16, 1, 128, torch.bfloat16)
    q = randn(g, 2, 8, 128, dtype=torch.bfloat16)
    q[0] *= 1000
    q[1] = 0
    o, lse = gdr2.attn_decode(q, k, v, table, lens, want_lse=True)
    ro, rl, to, tl, _ = ref.attention(q, k, v, table, lens)
    # row 0: a score's own rounding (2 d u S) is far above 1 unless one token leads by more; compare row 1 by the bound
    ref.check("o", o[1], ro[1], to[1])
    ref.check("lse", lse[1], rl[1], tl[1])
    assert abs(float(lse[1, 0]) - math.log(300)) < 1e-5
    ref.check("lse", lse[0], rl[0], tl[0])
    assert torch.isfinite(o).all()


def test_decode_replayed_as_sequences_grow_and_two_graphs():
    """A captured step reads the lengths on the device: replayed with longer sequences it attends to them. Two graphs
    with workspaces of their own, replayed on two streams at once, give what they give alone."""
    g = gen(23)
    k, v, table, lens, _ = cache(g, [1000, 3000], 16, 2, 128, torch.bfloat16)
    qs = [randn(g, 2, 16, 128, dtype=torch.bfloat16) for _ in range(2)]
    ln = torch.tensor([5, 0], dtype=torch.int32, device="cuda")
    graphs, outs = [], []
    need = int(gdr2.lib().gdr2_attn_decode_workspace_bytes(2, 16, 2, 128, table.shape[1], 16, 0, gdr2.GDR2_BF16))
    assert need > 0
    for q in qs:
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        o, lse = torch.empty_like(q), torch.empty(2, 16, device="cuda")
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            gdr2.attn_decode(q, k, v, table, ln, o=o, lse=lse, workspace=ws)
        graphs.append((gr, ws))
        outs.append((o, lse))
    for a, b in ((5, 0), (1000, 3000), (17, 2047)):
        ln.copy_(torch.tensor([a, b], dtype=torch.int32))
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in qs]
        for s, (gr, _) in zip(streams, graphs):
            with torch.cuda.stream(s):
                gr.replay()
        torch.cuda.synchronize()
        for q, (o, lse) in zip(qs, outs):
            ro, rl, to, tl, _ = ref.attention(q, k, v, table, ln)
            ref.check("o", o, ro, to)
            ref.check("lse", lse, rl, tl)
            assert torch.equal(o, gdr2.attn_decode(q, k, v, table, ln))


def test_decode_on_another_stream():
    """stream= with fresh outputs and workspaces, the inputs made on the current stream, which then goes on at once."""
    g = gen(25)
    k, v, table, lens, _ = cache(g, [3000, 20, 900], 16, 2, 64, torch.bfloat16)
    q = randn(g, 3, 8, 64, dtype=torch.bfloat16)
    want = gdr2.attn_decode(q, k, v, table, lens)
    side = torch.cuda.Stream()
    got = []
    for _ in range(20):
        side.wait_stream(torch.cuda.current_stream())
        got.append(gdr2.attn_decode(q, k, v, table, lens, stream=side))
        torch.full((1 << 21,), math.nan, device="cuda")  # would reuse a workspace that was let go too early
    side.synchronize()
    assert all(torch.equal(x, want) for x in got)


def test_decode_offsets_past_32_bits():
    """A pool of more than 2^32 bytes and 2^31 elements: the last pages are read and written."""
    ps, Hk, d = 64, 8, 128
    num = (1 << 31) // (ps * Hk * d) + 3
    k = torch.zeros(num, Hk, ps, d, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    g = gen(24)
    table = torch.tensor([[num - 1, 0, num - 2]], dtype=torch.int32, device="cuda")
    T = 2 * ps + 5
    x = randn(g, T, 2 * Hk + Hk, d, dtype=torch.bfloat16)
    pos = torch.arange(T, device="cuda", dtype=torch.int32)
    fr, _ = gdr2.rope_freqs(d)
    q = gdr2.attn_prologue_cache(x[:, :Hk], x[:, Hk:2 * Hk], x[:, 2 * Hk:], None, None, torch.zeros_like(pos), pos, fr, k, v,
                                 table)
    lens = torch.tensor([T], dtype=torch.int32, device="cuda")
    y, tol = ref.prologue(x[:ps, Hk:2 * Hk], None, pos[:ps], fr)
    ref.check("k", k[num - 1].transpose(0, 1), y, tol)
    assert torch.equal(v[num - 2, :, :5], x[2 * ps:, 2 * Hk:].transpose(0, 1))
    o = gdr2.attn_decode(q[-1:], k, v, table, lens)
    ro, _, to, _, _ = ref.attention(q[-1:], k, v, table, lens)
    ref.check("o", o, ro, to)
