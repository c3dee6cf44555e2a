"""Plain 64-bit forms of the attention half of the hybrid cell, for the tests: query / key prologue and its gradients,
attention of one new token, and the page bookkeeping as ordinary Python on lists.

Error bounds. u = 2^-24 (half a step of fp32), e = half a step of the stored type (fp32 2^-24, bf16 2^-8).
  prologue   the norm's factor n: 12 adds deep and a reciprocal root of 2 steps, 10 u; u = x n g: 2 u; the angle: a
             rounding of at most half a turn, 2 pi 2^-26 < 2.6 u, sine and cosine 2 steps (4 u), times mag 1 u; the two
             products and their sum 3 u. Below 32 u of (|u_a| + |u_b|) mag in all, and e of the stored value.
  gradient   the same factors once more and a mean of 128 products: below 64 u of the sum of the terms' magnitudes.
  attention  a score: d / 16 accumulations of exact products, at most 16 u each relative to the sum of magnitudes S:
             below 2 d u S (fp32: d additions of rounded products, the same); p: twice that for score and maximum,
             (|s - m| + 4) 2 u for the exponential, 2^-17 for p as a pair of bf16; the sums over L tokens: L / 8 + 64
             additions deep, 2 u each. Relative to sum p |v| / l, and e of the stored value.
"""
from __future__ import annotations

import math

import torch

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def rotate(u, pos, freqs, mag, interleaved, back=False):
    """u [T, H, d] float64; pos [T]; freqs [rot / 2] float64."""
    if freqs is None or freqs.numel() == 0:
        return u.clone()
    r = freqs.numel()
    t = pos.double()[:, None, None] * freqs.double()[None, None, :]
    c, s = mag * torch.cos(t), mag * torch.sin(t) * (-1 if back else 1)
    y = u.clone()
    ia = torch.arange(r, device=u.device) * 2 if interleaved else torch.arange(r, device=u.device)
    ib = ia + 1 if interleaved else ia + r
    a, b = u[..., ia], u[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
    return y


def spread(u, freqs, mag, interleaved):
    """|u_a| + |u_b| (times mag) at both places of a rotated pair, |u| elsewhere."""
    u = u.abs()
    if freqs is None or freqs.numel() == 0:
        return u
    r = freqs.numel()
    y = u.clone()
    ia = torch.arange(r, device=u.device) * 2 if interleaved else torch.arange(r, device=u.device)
    ib = ia + 1 if interleaved else ia + r
    y[..., ia] = y[..., ib] = mag * (u[..., ia] + u[..., ib])
    return y


def prologue(x, g, pos, freqs, *, norm=True, eps=1e-6, mag=1.0, interleaved=False):
    """(y, bound on the computed error of y before it is stored)"""
    u = x.double()
    if norm:
        u = u / torch.sqrt(u.square().mean(-1, keepdim=True) + eps)
        if g is not None:
            u = u * g.double()
    return rotate(u, pos, freqs, mag, interleaved), 32 * U * spread(u, freqs, mag, interleaved)


def prologue_grad(x, g, dy, pos, freqs, *, norm=True, eps=1e-6, mag=1.0, interleaved=False):
    """(dx, dg or None, bound on dx's computed error, sum of the magnitudes of dg's terms)"""
    x, dy = x.double(), dy.double()
    dz = rotate(dy, pos, freqs, mag, interleaved, back=True)
    sz = spread(dy, freqs, mag, interleaved)
    if not norm:
        return dz, None, 64 * U * sz, None
    gg = torch.ones(x.shape[-1], dtype=torch.float64, device=x.device) if g is None else g.double()
    n = 1 / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    gz = gg * dz
    dx = n * (gz - x * n ** 2 * (x * gz).mean(-1, keepdim=True))
    size = n * (gg.abs() * sz + x.abs() * n ** 2 * (x.abs() * gg.abs() * sz).mean(-1, keepdim=True))
    return dx, (dz * x * n).sum((0, 1)), 64 * U * size, (sz * x.abs() * n).sum((0, 1))


def check(name, got, ref, tol):
    """|got - ref| within `tol` and half a step of got's type, everywhere; infinities have to be the same."""
    g, e = got.double(), HALF[got.dtype]
    fin = torch.isfinite(ref)
    assert torch.equal(fin, torch.isfinite(g)), f"{name}: not finite where the definition is, or the other way round"
    assert torch.equal(g[~fin], ref[~fin]), f"{name}: another infinity"
    err = (g - ref).abs() - e * ref.abs() - tol - 1e-37
    bad = fin & (err > 0)
    assert not bad.any(), (f"{name}: {int(bad.sum())} of {bad.numel()} values off, the worst by "
                           f"{float(((g - ref).abs() / (tol + e * ref.abs() + 1e-37))[fin].max()):.3g} times its bound")


def attention(q, k_pages, v_pages, table, lens, seq=None, *, scale=None, window=0):
    """(o, lse, bound of o, bound of lse, slots that are padding), float64, one slot and KV head at a time."""
    N, Hq, d = q.shape
    num, Hk, ps, _ = k_pages.shape
    R, P = table.shape
    G, scale = Hq // Hk, d ** -0.5 if scale is None else scale
    tab, ln = table.tolist(), lens.tolist()
    sq = list(range(N)) if seq is None else seq.tolist()
    o = torch.zeros(N, Hq, d, dtype=torch.float64, device=q.device)
    lse = torch.full((N, Hq), -math.inf, dtype=torch.float64, device=q.device)
    to, tl = torch.zeros_like(o), torch.zeros(N, Hq, dtype=torch.float64, device=q.device)
    padding = [n for n in range(N) if not 0 <= sq[n] < R]
    for n in range(N):
        if n in padding:
            continue
        x = min(max(ln[sq[n]], 0), P * ps)
        first = max(0, x - window) if window else 0
        at = [(tab[sq[n]][i // ps], i % ps) for i in range(first, x) if 0 <= tab[sq[n]][i // ps] < num]
        if not at:
            continue
        pg = torch.tensor([a for a, _ in at], device=q.device)
        of = torch.tensor([b for _, b in at], device=q.device)
        for h in range(Hk):
            k, v = k_pages[pg, h, of].double(), v_pages[pg, h, of].double()
            js = slice(h * G, (h + 1) * G)
            qq = q[n, js].double()
            s = scale * (qq @ k.T)
            m = s.max(-1, keepdim=True).values
            p = torch.exp(s - m)
            l = p.sum(-1, keepdim=True)
            o[n, js] = p @ v / l
            lse[n, js] = (m + torch.log(l))[:, 0]
            ds = abs(scale) * (qq.abs() @ k.abs().T) * 2 * d * U
            rel = (2 * ds + ((s - m).abs() + 4) * 2 * U).max(-1, keepdim=True).values + 2.0 ** -17 + \
                (len(at) / 8 + 64) * 2 * U
            to[n, js] = 2 * rel * (p @ v.abs() / l)
            tl[n, js] = (rel + 8 * U * (m.abs() + torch.log(l)))[:, 0]
    return o, lse, to, tl, padding


# ---- the bookkeeping, on Python lists ----------------------------------------------------------------------


def _valid(table, num):
    return [[e if 0 <= e < num else -1 for e in row] for row in table]


def reserve(table, lens, want, ref, ps, window=0):
    num, P = len(ref), len(table[0])
    table, ref = _valid(table, num), list(ref)
    lens = [max(x, 0) for x in lens]
    for r, row in enumerate(table):
        for j in range(P):
            if window and row[j] >= 0 and (j + 1) * ps <= lens[r] + 1 - window:
                ref[row[j]] -= 1
                row[j] = -1
    free = [i for i in range(num) if ref[i] <= 0]
    missing = 0
    for r, row in enumerate(table):
        last = -(-want[r] // ps) if want[r] > 0 else 0
        for j in range(lens[r] // ps, min(last, P)):
            if row[j] < 0:
                if free:
                    row[j] = free.pop(0)
                    ref[row[j]] = 1
                else:
                    missing += 1
        missing += max(0, last - P)
    return table, ref, missing


def fork(table, lens, ref, parent, ps):
    """(table, lens, ref, missing, copies [(source page, fresh page, token rows)])"""
    num, R, P = len(ref), len(table), len(table[0])
    old, ref = _valid(table, num), list(ref)
    lens = [min(max(x, 0), P * ps) for x in lens]
    keeper = {}
    for r, p in enumerate(parent):
        if 0 <= p < R and (p not in keeper or r == p):
            keeper[p] = r
    new, out_len, todo = [], [], []
    for r, p in enumerate(parent):
        if not 0 <= p < R:
            new.append([-1] * P)
            out_len.append(0)
            continue
        full = lens[p] // ps
        out_len.append(lens[p])
        if keeper[p] == r:
            new.append(list(old[p]))
        else:
            new.append([old[p][j] if j < full else -1 for j in range(P)])
            if lens[p] % ps and old[p][full] >= 0:
                todo.append((r, full, old[p][full], lens[p] % ps))
    for r in range(R):
        if parent[r] != r:
            for e in old[r]:
                if e >= 0:
                    ref[e] -= 1
            for e in new[r]:
                if e >= 0:
                    ref[e] += 1
    free = [i for i in range(num) if ref[i] <= 0]
    copies, missing = [], 0
    for r, j, src, rows in todo:
        if free:
            page = free.pop(0)
            new[r][j] = page
            ref[page] = 1
            copies.append((src, page, rows))
        else:
            missing += 1
            out_len[r] = j * ps
    return new, out_len, ref, missing, copies


def compact(table, ref):
    """(table, ref, live, moves [(from, to)])"""
    num = len(ref)
    live = sum(n > 0 for n in ref)
    low = [i for i in range(live) if ref[i] <= 0]
    high = [i for i in range(live, num) if ref[i] > 0]
    to = dict(zip(high, low))
    out = [n if n > 0 and i < live else 0 for i, n in enumerate(ref)]
    for a, b in to.items():
        out[b] = ref[a]
    return [[to.get(e, e) for e in row] for row in _valid(table, num)], out, live, list(to.items())
