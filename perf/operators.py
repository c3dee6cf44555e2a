"""Workloads of the attention half of the hybrid cell: the query / key prologue (per-head RMS norm and rotary
positions) in training and in serving, attention of one new token over a paged key-value cache, and the page
bookkeeping of that cache.

Every case is run either by the library's entry points (`own` true) or by the plain torch form of the same
formulas in 32 bits (angles in 64), from the same inputs.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ES = {"bf16": 2, "f32": 4}
EPS = 1e-6


def listed():
    return [
        # the 8 x 4096-token training batch of the 16-head, d = 128 layer: q and k of the attention layer, forward
        # and backward
        dict(name="train-8x4096", op="train", dtype="bf16", B=8, T=4096, Hq=16, Hk=16, d=128, rot=128,
             interleaved=False, scaling="none", factor=1.0, pos0=0, fused=False),
        # a short odd fp32 batch (fine-tuning on a few prompts): grouped heads cut out of a fused projection, a
        # rotation of half the head in interleaved layout, positions far out in a scaled context
        dict(name="train-odd-f32", op="train", dtype="f32", B=3, T=385, Hq=12, Hk=4, d=64, rot=32,
             interleaved=True, scaling="parts", factor=16.0, pos0=60001, fused=True),
        # one decode step of 256 sequences (six slots of the padded batch empty) before the attention
        dict(name="append-256", op="append", dtype="bf16", R=256, lo=1, hi=4096, new=1, pad=6, Hq=16, Hk=4, d=128,
             ps=16, window=2048, rot=128, interleaved=False, fused=True),
        # 16 packed prompts of mixed length, 32 K tokens in all, written into an empty cache
        dict(name="append-prompts-16", op="append", dtype="bf16", R=16, lo=0, hi=0, new=4040, pad=0, Hq=16, Hk=4,
             d=128, ps=64, window=0, rot=64, interleaved=True, fused=True),
        # a single chat turn: one sequence, a few hundred tokens, latency counts
        dict(name="decode-1-short", op="decode", dtype="bf16", N=1, lo=333, hi=333, Hq=16, Hk=2, d=64, ps=16,
             window=0),
        # the decode batch of 256 sequences in the hybrid cell's 2 K window
        dict(name="decode-256-window", op="decode", dtype="bf16", N=256, lo=100, hi=4096, Hq=16, Hk=4, d=128, ps=16,
             window=2048),
        # three sequences at the 65,536-token context: little batch, long axis
        dict(name="decode-3-long", op="decode", dtype="bf16", N=3, lo=50001, hi=65536, Hq=16, Hk=2, d=128, ps=64,
             window=0),
        # a ragged fp32 batch, empty sequences among it, small heads
        dict(name="decode-33-f32", op="decode", dtype="f32", N=33, lo=0, hi=2000, Hq=12, Hk=6, d=64, ps=32,
             window=0),
        # beam search: 8 prompts x 4 beams after one step
        dict(name="fork-beams-32", op="fork", dtype="bf16", R=32, lo=40, hi=700, Hk=4, d=128, ps=16, release=0.0),
        # parallel samples forked off shared prompts, finished rows released
        dict(name="fork-256", op="fork", dtype="bf16", R=256, lo=1, hi=4000, Hk=4, d=128, ps=64, release=0.2),
        # a small server's pool after most sequences have ended
        dict(name="compact-512", op="compact", dtype="bf16", R=16, hi=300, Hk=4, d=64, ps=16, pages=512),
        # a large pool, half of it live, scattered
        dict(name="compact-4096", op="compact", dtype="bf16", R=64, hi=4000, Hk=4, d=128, ps=64, pages=4096),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def _heads(rng, most=16):
    Hk = rng.choice([1, 2, 3, 4, 6, 8, 16])
    G = rng.choice([1, 2, 3, 4, 7, 8, 16])
    while Hk * G > most:
        G = max(1, G // 2)
        if G == 1 and Hk > most:
            Hk //= 2
    return Hk * G, Hk


def draw(rng):
    op = rng.choice(["train", "append", "decode", "decode", "fork", "compact"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    d = rng.choice([64, 128])
    Hq, Hk = _heads(rng)
    if op == "train":
        most = 8 * 4096 * 32 * 128 * 2 // ((Hq + Hk) * d * ES[dtype])
        n = _log(rng, 1, min(65536, most))
        B = rng.choice([1, 1, 2, 3, 8])
        return dict(op=op, dtype=dtype, B=B, T=max(1, n // B), Hq=Hq, Hk=Hk, d=d, rot=rng.choice([16, 32, d // 2, d]),
                    interleaved=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "parts"]),
                    factor=rng.choice([2.0, 4.0, 16.0]), pos0=rng.choice([0, 0, 4097, 500001]),
                    fused=rng.random() < 0.5)
    ps = rng.choice([8, 16, 24, 32, 64, 128])
    if op == "append":
        prompts = rng.random() < 0.4
        R = _log(rng, 1, 16) if prompts else _log(rng, 1, 256)
        hi = 0 if prompts else _log(rng, 1, 4096)
        most = 800_000_000 // (R * (2 * Hq + 4 * Hk) * d * ES[dtype])
        return dict(op=op, dtype=dtype, R=R, lo=0, hi=hi, new=_log(rng, 2, min(4000, most)) if prompts else 1,
                    pad=rng.choice([0, 0, 3]), Hq=Hq, Hk=Hk, d=d, ps=ps,
                    window=0 if prompts else rng.choice([0, 500, 2048]), rot=rng.choice([16, d // 2, d]),
                    interleaved=rng.random() < 0.5, fused=rng.random() < 0.5)
    if op == "decode":
        N = _log(rng, 1, 256)
        most = max(1, 256 * 2100 * 4 * 128 * 2 // (N * Hk * d * ES[dtype]))
        hi = _log(rng, 1, min(65536, most))
        return dict(op=op, dtype=dtype, N=N, lo=rng.choice([0, 1, hi // 2, hi]) if hi > 1 else 1, hi=hi, Hq=Hq,
                    Hk=Hk, d=d, ps=ps, window=rng.choice([0, 0, 0, 300, 2048]))
    if op == "fork":
        R = _log(rng, 2, 256)
        return dict(op=op, dtype=dtype, R=R, lo=1, hi=_log(rng, 2, 4000), Hk=min(Hk, 4), d=d, ps=ps,
                    release=rng.choice([0.0, 0.2, 0.6]))
    R, hi = _log(rng, 1, 64), _log(rng, 2, 4000)
    held = _held([_length(n, R, 1, hi) for n in range(R)], ps)
    return dict(op=op, dtype=dtype, R=R, hi=hi, Hk=min(Hk, 4), d=d, ps=ps,
                pages=held + _log(rng, 1, max(1, 4096 * 64 // ps - held) if held < 2048 else 64))


def _length(n, N, lo, hi):
    """Ragged lengths over [lo, hi], spread by the golden ratio; the largest is always there."""
    return hi if n == 0 else lo + int((hi - lo + 1) * ((n * 0.6180339887498949) % 1.0))


def _held(lens, ps):
    return sum(-(-x // ps) for x in lens)


def _perm(lens, g):
    p = torch.randperm(len(lens), generator=g, device="cuda")
    return torch.tensor(lens, dtype=torch.int32, device="cuda")[p]


def _tables(lens, ps, P, num_pages, g):
    """Rows of a page table that hold `lens` tokens, on pages scattered over the pool; and the counts of use."""
    R = lens.numel()
    held = (lens.long() + ps - 1) // ps
    used = torch.arange(P, device="cuda")[None, :] < held[:, None]
    order = torch.randperm(num_pages, generator=g, device="cuda").int()
    rank = used.flatten().long().cumsum(0).view(R, P) - 1
    table = torch.where(used, order[rank.clamp(min=0)], torch.full_like(rank, -1, dtype=torch.int32))
    return table.contiguous(), _counts(table, num_pages)


def _counts(table, num_pages):
    ref = torch.zeros(num_pages, dtype=torch.int32, device=table.device)
    on = table >= 0
    return ref.scatter_add_(0, table.clamp(min=0).flatten().long(), on.flatten().int())


def _freqs(rot, scaling, factor, base=10000.0, length=4096, low=1.0, high=32.0):
    """Radians per position of each rotated pair, in 64 bits, and the rotation's magnitude."""
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "parts":
        turns = length * f / (2 * math.pi)
        keep = ((turns - low) / (high - low)).clamp(0, 1)
        return f * (keep + (1 - keep) / factor), 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _pool_bytes(c):
    return c["Hk"] * c["ps"] * c["d"] * ES[c["dtype"]]


def _plan(c):
    """The sizes of a cache case that follow from the case alone."""
    if c["op"] == "append":
        if c["new"] > 1:
            new = [1 + _length(n, c["R"], c["new"] // 12, c["new"]) // 2 for n in range(c["R"])]
            lens = [0] * c["R"]
        else:
            new = [1] * c["R"]
            lens = [_length(n, c["R"], c["lo"], c["hi"]) for n in range(c["R"])]
        total = sum(-(-(x + y) // c["ps"]) for x, y in zip(lens, new))
        P = max(-(-(x + y) // c["ps"]) for x, y in zip(lens, new)) + 2
        return lens, new, P, total + max(3, total // 8)
    if c["op"] == "decode":
        lens = [_length(n, c["N"], c["lo"], c["hi"]) for n in range(c["N"])]
        total = _held(lens, c["ps"])
        return lens, None, max(1, -(-c["hi"] // c["ps"])), total + max(1, total // 16)
    if c["op"] == "fork":
        lens = [_length(n, c["R"], c["lo"], c["hi"]) for n in range(c["R"])]
        total = _held(lens, c["ps"])
        return lens, None, -(-c["hi"] // c["ps"]) + 1, total + c["R"]
    lens = [_length(n, c["R"], 1, c["hi"]) for n in range(c["R"])]
    return lens, None, -(-c["hi"] // c["ps"]), c["pages"]


def _randn(shape, dt, g):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dt) if math.prod(shape) < 1 << 26 \
        else torch.randn(*shape, generator=g, device="cuda", dtype=dt)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1009 + 17)
    dt = DTYPES[c["dtype"]]
    s = {"case": c}
    if c["op"] == "train":
        T, Hq, Hk, d = c["B"] * c["T"], c["Hq"], c["Hk"], c["d"]
        if c["fused"]:  # views of one fused q | k | v projection
            qkv = _randn((T, (Hq + 2 * Hk) * d), dt, g)
            s["xq"] = qkv[:, :Hq * d].view(T, Hq, d)
            s["xk"] = qkv[:, Hq * d:(Hq + Hk) * d].view(T, Hk, d)
        else:
            s["xq"], s["xk"] = _randn((T, Hq, d), dt, g), _randn((T, Hk, d), dt, g)
        s["dq"], s["dk"] = _randn((T, Hq, d), dt, g), _randn((T, Hk, d), dt, g)
        s["gq"] = 1 + 0.2 * torch.randn(d, generator=g, device="cuda")
        s["gk"] = 1 + 0.2 * torch.randn(d, generator=g, device="cuda")
        s["pos"] = (c["pos0"] + torch.arange(c["T"], device="cuda", dtype=torch.int32)).repeat(c["B"])
        s["freqs"], s["mag"] = _freqs(c["rot"], c["scaling"], c["factor"])
        return s
    lens, new, P, num_pages = _plan(c)
    Hk, d, ps = c["Hk"], c["d"], c["ps"]
    s["k_pages"] = _randn((num_pages, Hk, ps, d), dt, g)
    s["v_pages"] = _randn((num_pages, Hk, ps, d), dt, g)
    R = len(lens)
    if c["op"] == "append":
        perm = torch.randperm(R, generator=g, device="cuda")
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")[perm]
        nt = torch.tensor(new, dtype=torch.int32, device="cuda")[perm]
        s["want"] = s["lens"] + nt
        s["table"], s["ref"] = _tables(s["lens"], ps, P, num_pages, g)
        T, Hq = sum(new) + c["pad"], c["Hq"]
        seq = torch.repeat_interleave(torch.arange(R, device="cuda"), nt.long())
        first = (nt.long().cumsum(0) - nt.long())[seq]
        pos = s["lens"].long()[seq] + torch.arange(seq.numel(), device="cuda") - first
        s["seq"] = torch.cat([seq, torch.full((c["pad"],), -1, device="cuda")]).int()
        s["pos"] = torch.cat([pos, torch.zeros(c["pad"], dtype=pos.dtype, device="cuda")]).int()
        qkv = _randn((T, (Hq + 2 * Hk) * d), dt, g)
        parts = [qkv[:, a * d:b * d].view(T, b - a, d) for a, b in ((0, Hq), (Hq, Hq + Hk), (Hq + Hk, Hq + 2 * Hk))]
        s["xq"], s["xk"], s["xv"] = parts if c["fused"] else [x.contiguous() for x in parts]
        s["gq"] = 1 + 0.2 * torch.randn(d, generator=g, device="cuda")
        s["gk"] = 1 + 0.2 * torch.randn(d, generator=g, device="cuda")
        s["freqs"], s["mag"] = _freqs(c["rot"], "none", 1.0)
        s["q"] = torch.zeros((T, Hq, d), dtype=dt, device="cuda")
        return s
    s["lens"] = _perm(lens, g)
    s["table"], s["ref"] = _tables(s["lens"], ps, P, num_pages, g)
    if c["op"] == "decode":
        s["q"] = (1.5 * torch.randn(c["N"], c["Hq"], d, generator=g, device="cuda")).to(dt)
    elif c["op"] == "fork":
        parent = torch.randint(0, R, (R,), generator=g, device="cuda", dtype=torch.int32)
        stay = torch.rand(R, generator=g, device="cuda") < 0.4
        parent = torch.where(stay, torch.arange(R, device="cuda", dtype=torch.int32), parent)
        gone = torch.rand(R, generator=g, device="cuda") < c["release"]
        s["parent"] = torch.where(gone, torch.full_like(parent, -1), parent)
    return s


# ---- the plain forms --------------------------------------------------------------------------------------


def _turn(x, cos, sin, rot, interleaved):
    """Rotate the first `rot` channels of x [T, H, d]; cos, sin [T, rot / 2]."""
    r, rest = x[..., :rot], x[..., rot:]
    cos, sin = cos[:, None, :], sin[:, None, :]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1).flatten(-2)
    else:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat([a * cos - b * sin, a * sin + b * cos], dim=-1)
    return torch.cat([r, rest], dim=-1)


def _cos_sin(pos, freqs, mag):
    t = pos.double()[:, None] * freqs[None, :]
    return (mag * torch.cos(t)).float(), (mag * torch.sin(t)).float()


def _prologue(x, g, cos, sin, rot, interleaved):
    x = x.float()
    n = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    return _turn(x * n * g, cos, sin, rot, interleaved)


def _prologue_grad(x, g, dy, cos, sin, rot, interleaved):
    x = x.float()
    n = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    dz = _turn(dy.float(), cos, -sin, rot, interleaved)
    dg = (dz * x * n).sum((0, 1))
    gz = g * dz
    dx = n * (gz - x * (n * n) * (x * gz).mean(-1, keepdim=True))
    return dx, dg


def _train(s):
    c = s["case"]
    dt, rot, il = DTYPES[c["dtype"]], c["rot"], c["interleaved"]
    cos, sin = _cos_sin(s["pos"], s["freqs"], s["mag"])
    out = {"q": _prologue(s["xq"], s["gq"], cos, sin, rot, il).to(dt),
           "k": _prologue(s["xk"], s["gk"], cos, sin, rot, il).to(dt)}
    dxq, out["dgq"] = _prologue_grad(s["xq"], s["gq"], s["dq"], cos, sin, rot, il)
    dxk, out["dgk"] = _prologue_grad(s["xk"], s["gk"], s["dk"], cos, sin, rot, il)
    out["dxq"], out["dxk"] = dxq.to(dt), dxk.to(dt)
    return out


def _reserve(table, lens, want, ref, ps, window):
    R, P = table.shape
    num = ref.numel()
    j = torch.arange(P, device=table.device)[None, :]
    lens, want = lens.long()[:, None], want.long()[:, None]
    if window:
        dead = ((j + 1) * ps <= lens + 1 - window) & (table >= 0)
        ref = ref.scatter_add(0, table.clamp(min=0).flatten().long(), -dead.flatten().int())
        table = torch.where(dead, torch.full_like(table, -1), table)
    last = (want + ps - 1) // ps
    need = ((j >= lens // ps) & (j < last) & (table < 0)).flatten()
    rank = need.long().cumsum(0) - 1
    free = torch.argsort((ref > 0).int(), stable=True)
    got = need & (rank < (ref <= 0).sum())
    page = free[rank.clamp(0, num - 1)].int()
    table = torch.where(got, page, table.flatten()).view(R, P)
    ref = _set_taken(ref, page, got)
    missing = (need & ~got).sum() + (last - P).clamp(min=0).sum()
    return table, ref, missing.int().view(1)


def _set_taken(ref, page, got):
    """ref with 1 for every page that `got` took."""
    hit = torch.zeros_like(ref).scatter_add_(0, page.long(), got.int())
    return torch.where(hit > 0, torch.ones_like(ref), ref)


def _append(s):
    c = s["case"]
    dt, rot, il, ps = DTYPES[c["dtype"]], c["rot"], c["interleaved"], c["ps"]
    table, ref, missing = _reserve(s["table"], s["lens"], s["want"], s["ref"], ps, c["window"])
    cos, sin = _cos_sin(s["pos"], s["freqs"], s["mag"])
    on = s["seq"] >= 0
    q = _prologue(s["xq"], s["gq"], cos, sin, rot, il).to(dt)
    k = _prologue(s["xk"], s["gk"], cos, sin, rot, il).to(dt)
    q = torch.where(on[:, None, None], q, s["q"])
    seq, pos = s["seq"].long()[on], s["pos"].long()[on]
    page = table[seq, pos // ps].long()
    at = page >= 0
    page, off = page[at], (pos % ps)[at]
    s["k_pages"][page, :, off] = k[on][at]
    s["v_pages"][page, :, off] = s["xv"][on][at]
    return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"], "table": table, "ref": ref, "missing": missing}


def _decode(s):
    c = s["case"]
    N, Hq, Hk, d, ps = c["N"], c["Hq"], c["Hk"], c["d"], c["ps"]
    table, lens = s["table"], s["lens"].long()[:, None]
    P = table.shape[1]
    at = torch.arange(P * ps, device=table.device)[None, :]
    on = (at < lens) & (table >= 0).repeat_interleave(ps, 1)
    if c["window"]:
        on = on & (at >= lens - c["window"])
    idx = table.clamp(min=0).long()
    k = s["k_pages"][idx].permute(0, 2, 1, 3, 4).reshape(N, Hk, P * ps, d).float()
    v = s["v_pages"][idx].permute(0, 2, 1, 3, 4).reshape(N, Hk, P * ps, d).float()
    v = v.masked_fill(~on[:, None, :, None], 0.0)
    q = s["q"].view(N, Hk, Hq // Hk, d).float()
    sc = torch.matmul(q, k.transpose(-1, -2)) * (1.0 / math.sqrt(d))
    sc = sc.masked_fill(~on[:, None, None, :], -math.inf)
    m = sc.amax(-1, keepdim=True)
    p = torch.exp(sc - m.clamp(min=-3.0e38))
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(l > 0, l, torch.ones_like(l))
    return {"o": o.reshape(N, Hq, d).to(s["q"].dtype), "lse": (m + torch.log(l)).reshape(N, Hq)}


def _fork(s):
    c = s["case"]
    ps, table, lens, ref = c["ps"], s["table"], s["lens"].long(), s["ref"]
    R, P = table.shape
    r = torch.arange(R, device=table.device)
    on = (s["parent"] >= 0) & (s["parent"] < R)
    par = s["parent"].long().clamp(0, R - 1)
    key = torch.where(r == par, torch.full_like(r, -1), r)
    first = torch.full((R,), R, device=table.device).scatter_reduce(0, par, torch.where(on, key, R + 0 * key), "amin")
    owner = on & (key == first[par])
    plen = torch.where(on, lens[par], torch.zeros_like(lens))
    j = torch.arange(P, device=table.device)[None, :]
    old = torch.where(on[:, None], table[par], torch.full_like(table, -1))
    base = torch.where(owner[:, None] | (j < (plen // ps)[:, None]), old, torch.full_like(old, -1))
    jl = (plen // ps).clamp(max=P - 1)
    src = old[r, jl]
    need = on & ~owner & (plen % ps != 0) & (src >= 0)
    num = ref.numel()
    ref = ref - _counts(table, num) + _counts(base, num)
    rank = need.long().cumsum(0) - 1
    free = torch.argsort((ref > 0).int(), stable=True)
    got = need & (rank < (ref <= 0).sum())
    page = free[rank.clamp(0, num - 1)].int()
    ref = _set_taken(ref, page, got)
    base[r, jl] = torch.where(got, page, base[r, jl])
    out_len = torch.where(need & ~got, jl * ps, plen).int()
    rows = torch.where(got, plen % ps, torch.zeros_like(plen))[got]
    a, b = src[got].long(), page[got].long()
    keep = (torch.arange(ps, device=table.device)[None, :] < rows[:, None])[:, None, :, None]
    for pool in (s["k_pages"], s["v_pages"]):
        pool[b] = torch.where(keep, pool[a], pool[b])
    return {"table": base, "lens": out_len, "ref": ref, "missing": (need & ~got).sum().int().view(1),
            "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _compact(s):
    table, ref = s["table"], s["ref"]
    live = ref > 0
    L = live.sum()
    i = torch.arange(ref.numel(), device=ref.device)
    high = live & (i >= L)
    low = torch.argsort(live.int(), stable=True)
    new = torch.where(high, low[(high.long().cumsum(0) - 1).clamp(min=0)], i)
    out = torch.where(table >= 0, new[table.clamp(min=0).long()].int(), torch.full_like(table, -1))
    moved = torch.zeros_like(ref).scatter_add_(0, new, torch.where(live, ref, torch.zeros_like(ref)))
    a, b = i[high], new[high]
    for pool in (s["k_pages"], s["v_pages"]):
        pool[b] = pool[a]
    return {"table": out, "ref": moved, "live": L.int().view(1), "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


# ---- the library's calls ----------------------------------------------------------------------------------


def _own(s):
    from gated_delta_rule_65_b200 import gdr2
    c = s["case"]
    if c["op"] == "train":
        a = (s["xq"], s["xk"], s["gq"], s["gk"], s["pos"], s["freqs"])
        kw = dict(eps=EPS, mag=s["mag"], interleaved=c["interleaved"])
        out = gdr2.attn_prologue_fwd(*a, **kw)
        return {**out, **gdr2.attn_prologue_bwd(*a, s["dq"], s["dk"], **kw)}
    if c["op"] == "append":
        table, ref, missing = gdr2.kv_reserve(s["table"], s["lens"], s["want"], s["ref"], page_size=c["ps"],
                                              window=c["window"])
        q = gdr2.attn_prologue_cache(s["xq"], s["xk"], s["xv"], s["gq"], s["gk"], s["seq"], s["pos"], s["freqs"],
                                     s["k_pages"], s["v_pages"], table, eps=EPS, mag=s["mag"],
                                     interleaved=c["interleaved"], q=s["q"])
        return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"], "table": table, "ref": ref,
                "missing": missing}
    if c["op"] == "decode":
        o, lse = gdr2.attn_decode(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"], window=c["window"],
                                  want_lse=True)
        return {"o": o, "lse": lse}
    if c["op"] == "fork":
        table, lens, ref, missing = gdr2.kv_fork(s["table"], s["lens"], s["ref"], s["parent"], s["k_pages"],
                                                 s["v_pages"])
        return {"table": table, "lens": lens, "ref": ref, "missing": missing, "k_pages": s["k_pages"],
                "v_pages": s["v_pages"]}
    table, ref, live = gdr2.kv_compact(s["table"], s["ref"], s["k_pages"], s["v_pages"])
    return {"table": table, "ref": ref, "live": live, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


PLAIN = {"train": _train, "append": _append, "decode": _decode, "fork": _fork, "compact": _compact}


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# ---- what a pass cannot do without ------------------------------------------------------------------------


def work(case):
    c = case
    es, d = ES[c["dtype"]], c["d"]
    if c["op"] == "train":
        rows = c["B"] * c["T"] * (c["Hq"] + c["Hk"])
        # forward: x read, y written; backward: dy read, dx written (x, still in hand, is read once)
        return {"bytes": 4 * rows * d * es + 4 * c["B"] * c["T"], "flops": 25 * rows * d}
    lens, new, P, num_pages = _plan(c)
    if c["op"] == "append":
        T = sum(new)
        return {"bytes": T * (2 * c["Hq"] + 4 * c["Hk"]) * d * es + 8 * T + 8 * c["R"] * P + 8 * num_pages,
                "flops": 10 * T * (c["Hq"] + c["Hk"]) * d}
    if c["op"] == "decode":
        seen = sum(min(x, c["window"]) if c["window"] else x for x in lens)
        pages = _held([min(x, c["window"]) if c["window"] else x for x in lens], c["ps"])
        return {"bytes": 2 * seen * c["Hk"] * d * es + 2 * c["N"] * c["Hq"] * d * es + 4 * c["N"] * c["Hq"] + 4 * pages,
                "flops": 4 * seen * c["Hq"] * d}
    if c["op"] == "fork":
        copies = c["R"] * (1 - c["release"]) * 0.3
        moved = copies * 0.5 * c["ps"] * c["Hk"] * d * es * 2
    else:
        live = _held(lens, c["ps"])
        moved = live * (1 - live / num_pages) * _pool_bytes(c) * 2
    return {"bytes": int(2 * moved) + 8 * c["R"] * P + 8 * num_pages + 12 * c["R"], "flops": c["R"] * P + num_pages}


# ---- the definitions in 64 bits ---------------------------------------------------------------------------


def _exact_y(x, g, pos, freqs, mag, rot, interleaved):
    """RMS norm and rotation as products of complex numbers, in 64 bits; leaf gradients flow through it."""
    u = x * g / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS)
    w = torch.polar(torch.full_like(freqs, mag)[None, :].expand(pos.numel(), -1).contiguous(),
                    pos.double()[:, None] * freqs[None, :])[:, None, :]
    if interleaved:
        z = torch.view_as_complex(u[..., :rot].reshape(*u.shape[:-1], rot // 2, 2).contiguous()) * w
        return torch.cat([torch.view_as_real(z).flatten(-2), u[..., rot:]], -1)
    z = torch.complex(u[..., :rot // 2].contiguous(), u[..., rot // 2:rot].contiguous()) * w
    return torch.cat([z.real, z.imag, u[..., rot:]], -1)


def _exact_train(s):
    c, out = s["case"], {}
    for n in ("q", "k"):
        total, parts, grads = 0, [], []
        for a in range(0, s["x" + n].shape[0], 4096):  # a few tokens at a time: 64 bits and a graph take room
            sl = slice(a, a + 4096)
            x = s["x" + n][sl].double().requires_grad_(True)
            g = s["g" + n].double().requires_grad_(True)
            y = _exact_y(x, g, s["pos"][sl], s["freqs"], s["mag"], c["rot"], c["interleaved"])
            dx, dg = torch.autograd.grad(y, (x, g), s["d" + n][sl].double())
            parts.append(y.detach())
            grads.append(dx)
            total = total + dg
        out[n], out["dx" + n], out["dg" + n] = torch.cat(parts), torch.cat(grads), total
    return out


def _exact_append(s):
    c = s["case"]
    ps, rot, il, window = c["ps"], c["rot"], c["interleaved"], c["window"]
    table, ref = s["table"].tolist(), s["ref"].tolist()
    lens, want = s["lens"].tolist(), s["want"].tolist()
    P = len(table[0])
    if window:
        for r, row in enumerate(table):
            for j in range(P):
                if row[j] >= 0 and (j + 1) * ps <= lens[r] + 1 - window:
                    ref[row[j]] -= 1
                    row[j] = -1
    free = [p for p, n in enumerate(ref) if n <= 0][::-1]
    missing = 0
    for r, row in enumerate(table):
        for j in range(lens[r] // ps, -(-want[r] // ps)):
            if j >= P:
                missing += 1
            elif row[j] < 0:
                if free:
                    row[j] = free.pop()
                    ref[row[j]] = 1
                else:
                    missing += 1
    a = (s["pos"], s["freqs"], s["mag"], rot, il)
    q = _exact_y(s["xq"].double(), s["gq"].double(), *a)
    k = _exact_y(s["xk"].double(), s["gk"].double(), *a)
    kp, vp = s["k_pages"].double(), s["v_pages"].double()
    slots = [(t, table[r][p // ps], p % ps) for t, (r, p) in enumerate(zip(s["seq"].tolist(), s["pos"].tolist()))
             if r >= 0]
    q[[t for t, r in enumerate(s["seq"].tolist()) if r < 0]] = 0.0
    at = torch.tensor([x for x in slots if x[1] >= 0], device="cuda", dtype=torch.long).reshape(-1, 3)
    kp[at[:, 1], :, at[:, 2]] = k[at[:, 0]]
    vp[at[:, 1], :, at[:, 2]] = s["xv"].double()[at[:, 0]]
    return {"q": q, "k_pages": kp, "v_pages": vp, "table": None, "ref": None, "missing": None}


def _exact_decode(s):
    c = s["case"]
    Hq, Hk, d, ps = c["Hq"], c["Hk"], c["d"], c["ps"]
    o = torch.zeros(c["N"], Hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((c["N"], Hq), -math.inf, dtype=torch.float64, device="cuda")
    for n, x in enumerate(s["lens"].tolist()):
        first = max(0, x - c["window"]) if c["window"] else 0
        if x == 0:
            continue
        pages = s["table"][n, first // ps:-(-x // ps)].long()
        cut = slice(first % ps, first % ps + x - first)
        for h in range(Hk):
            k = s["k_pages"][pages, h].reshape(-1, d)[cut].double()
            v = s["v_pages"][pages, h].reshape(-1, d)[cut].double()
            js = slice(h * (Hq // Hk), (h + 1) * (Hq // Hk))
            sc = s["q"][n, js].double() @ k.T / math.sqrt(d)
            lse[n, js] = torch.logsumexp(sc, -1)
            o[n, js] = torch.exp(sc - lse[n, js, None]) @ v
    return {"o": o, "lse": lse}


def exact(case, seed):
    if case["op"] in ("fork", "compact"):
        return None  # these move whole numbers and copy values: nothing is computed
    s = prepare(case, seed)
    return {"train": _exact_train, "append": _exact_append, "decode": _exact_decode}[case["op"]](s)
