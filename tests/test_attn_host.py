"""Host-side checks of the attention half of the hybrid cell (no GPU: nothing here launches a kernel): statuses of the C
entry points, the binding's own refusals, and the rotary frequencies against their formulas."""
from __future__ import annotations

import ctypes
import math

import pytest
import torch

from gated_delta_rule_65_b200 import gdr2

FAKE = 0x10000       # aligned, never dereferenced: validation fails first
ODD = 0x10002        # not even 4-byte aligned
OFF8 = 0x10008
OK, ARG, UNS, WS = gdr2.OK, gdr2.ERR_INVALID_ARG, gdr2.ERR_UNSUPPORTED, gdr2.ERR_WORKSPACE


def call(name, defaults, **over):
    a = dict(defaults)
    a.update(over)
    return getattr(gdr2.lib(), name)(*a.values())


FWD = dict(xq=FAKE, xk=FAKE, gq=FAKE, gk=FAKE, norm=1, eps=1e-6, pos=FAKE, freqs=FAKE, mag=1.0, rot=64, inter=0, q=FAKE,
           k=FAKE, T=4, Hq=4, Hk=2, d=64, dtype=1, sq=256, sk=128, stream=None)
COMMON = [(dict(xq=None), ARG), (dict(xk=OFF8), ARG), (dict(T=0), ARG), (dict(Hq=0), ARG), (dict(Hk=-1), ARG),
          (dict(d=96), UNS), (dict(d=256), UNS), (dict(dtype=2), ARG), (dict(norm=2), ARG), (dict(norm=0), ARG),
          (dict(eps=-1.0), ARG), (dict(eps=math.nan), ARG), (dict(rot=8), UNS), (dict(rot=-16), ARG),
          (dict(rot=80), ARG), (dict(pos=None), ARG), (dict(pos=ODD), ARG), (dict(freqs=None), ARG),
          (dict(freqs=0x10004), ARG), (dict(gq=ODD), ARG), (dict(sq=255), ARG), (dict(sq=260), ARG), (dict(sk=64), ARG),
          (dict(Hq=70000), UNS)]


@pytest.mark.parametrize("over,status", COMMON + [(dict(q=None), ARG), (dict(k=OFF8), ARG)], ids=str)
def test_prologue_fwd_refusals(over, status):
    assert call("gdr2_attn_prologue_fwd", FWD, **over) == status


BWD = dict(xq=FAKE, xk=FAKE, gq=FAKE, gk=FAKE, norm=1, eps=1e-6, pos=FAKE, freqs=FAKE, mag=1.0, rot=64, inter=0, dq=FAKE,
           dk=FAKE, dxq=FAKE, dxk=FAKE, dgq=FAKE, dgk=FAKE, T=4, Hq=4, Hk=2, d=64, dtype=1, sq=256, sk=128, sdq=256,
           sdk=128, ws=FAKE, wsb=1 << 30, stream=None)


@pytest.mark.parametrize("over,status", COMMON + [
    (dict(dq=None), ARG), (dict(dxk=None), ARG), (dict(dgq=ODD), ARG), (dict(sdq=128), ARG), (dict(sdk=132), ARG),
    (dict(norm=0, gq=None, gk=None), ARG),  # no gains, no gradients of gains
    (dict(ws=None), WS), (dict(ws=OFF8), WS), (dict(wsb=16), WS)], ids=str)
def test_prologue_bwd_refusals(over, status):
    assert call("gdr2_attn_prologue_bwd", BWD, **over) == status


CACHE = dict(xq=FAKE, xk=FAKE, xv=FAKE, gq=FAKE, gk=FAKE, norm=1, eps=1e-6, seq=FAKE, pos=FAKE, freqs=FAKE, mag=1.0,
             rot=64, inter=0, q=FAKE, kp=FAKE, vp=FAKE, table=FAKE, T=4, Hq=4, Hk=2, d=64, R=3, P=5, ps=16, num=9,
             dtype=1, sq=256, sk=128, sv=128, stream=None)


@pytest.mark.parametrize("over,status", COMMON + [
    (dict(xv=None), ARG), (dict(seq=None), ARG), (dict(pos=None, rot=0), ARG), (dict(kp=OFF8), ARG), (dict(vp=None), ARG),
    (dict(table=ODD), ARG), (dict(R=0), ARG), (dict(P=0), ARG), (dict(ps=0), ARG), (dict(num=-1), ARG), (dict(sv=4), ARG),
    (dict(P=1 << 20, ps=1 << 12), UNS)], ids=str)
def test_prologue_cache_refusals(over, status):
    assert call("gdr2_attn_prologue_cache", CACHE, **over) == status


DECODE = dict(q=FAKE, kp=FAKE, vp=FAKE, table=FAKE, lens=FAKE, seq=None, scale=0.1, window=0, o=FAKE, lse=None, N=3, Hq=4,
              Hk=2, d=64, R=3, P=200, ps=16, num=9, dtype=1, ws=FAKE, wsb=1 << 30, stream=None)


@pytest.mark.parametrize("over,status", [
    (dict(q=None), ARG), (dict(kp=None), ARG), (dict(vp=OFF8), ARG), (dict(table=None), ARG), (dict(lens=ODD), ARG),
    (dict(seq=ODD), ARG), (dict(o=None), ARG), (dict(lse=ODD), ARG), (dict(window=-1), ARG), (dict(N=0), ARG),
    (dict(N=4), ARG), (dict(Hq=5), ARG), (dict(Hq=1), ARG), (dict(d=32), UNS), (dict(dtype=-1), ARG), (dict(R=0), ARG),
    (dict(ps=-4), ARG), (dict(P=1 << 30), UNS), (dict(N=1 << 30, seq=FAKE), UNS), (dict(ws=None), WS),
    (dict(wsb=1000), WS), (dict(num=1 << 30, ps=16, P=200), UNS), (dict(Hq=2050), UNS)], ids=str)
def test_decode_refusals(over, status):
    assert call("gdr2_attn_decode", DECODE, **over) == status


RESERVE = dict(table=FAKE, lens=FAKE, want=FAKE, ref=FAKE, t=FAKE, r=FAKE, m=FAKE, R=3, P=5, ps=16, num=9, window=0,
               ws=FAKE, wsb=1 << 30, stream=None)
FORK = dict(table=FAKE, lens=FAKE, ref=FAKE, parent=FAKE, t=FAKE + 16, n=FAKE + 16, r=FAKE, m=FAKE, kp=FAKE, vp=FAKE, R=3,
            P=5, Hk=2, ps=16, d=64, num=9, dtype=1, ws=FAKE, wsb=1 << 30, stream=None)
COMPACT = dict(table=FAKE, ref=FAKE, t=FAKE, r=FAKE, live=FAKE, kp=FAKE, vp=FAKE, R=3, P=5, Hk=2, ps=16, d=64, num=9,
               dtype=1, ws=FAKE, wsb=1 << 30, stream=None)
PAGES = [(dict(table=None), ARG), (dict(ref=ODD), ARG), (dict(t=None), ARG), (dict(r=None), ARG), (dict(R=0), ARG),
         (dict(P=-1), ARG), (dict(ps=0), ARG), (dict(num=0), ARG), (dict(P=1 << 30), UNS), (dict(ws=None), WS),
         (dict(ws=OFF8), WS), (dict(wsb=64), WS)]


@pytest.mark.parametrize("over,status", PAGES + [(dict(want=None), ARG), (dict(m=None), ARG), (dict(window=-1), ARG)], ids=str)
def test_reserve_refusals(over, status):
    assert call("gdr2_kv_reserve", RESERVE, **over) == status


@pytest.mark.parametrize("over,status", PAGES + [
    (dict(parent=None), ARG), (dict(lens=ODD), ARG), (dict(m=None), ARG), (dict(kp=OFF8), ARG), (dict(t=FAKE), ARG),
    (dict(n=FAKE), ARG), (dict(Hk=0), ARG), (dict(d=100), UNS), (dict(dtype=3), ARG)], ids=str)
def test_fork_refusals(over, status):
    assert call("gdr2_kv_fork", FORK, **over) == status


@pytest.mark.parametrize("over,status", PAGES + [(dict(live=None), ARG), (dict(vp=None), ARG), (dict(d=100), UNS)], ids=str)
def test_compact_refusals(over, status):
    assert call("gdr2_kv_compact", COMPACT, **over) == status


def test_workspace_sizes():
    L = gdr2.lib()
    f = L.gdr2_attn_prologue_workspace_bytes
    assert 0 < f(64) < f(128) < 1 << 24 and f(96) == 0
    f = L.gdr2_attn_decode_workspace_bytes  # N, Hq, Hk, d, P, page_size, window, dtype
    assert 0 < f(3, 8, 2, 64, 1000, 16, 0, 1) < f(3, 8, 2, 128, 1000, 16, 0, 1) < 1 << 24
    assert f(3, 8, 2, 64, 4, 16, 0, 1) == 0 and f(3, 8, 2, 64, 1000, 16, 64, 1) == 0  # short rows stay whole
    assert f(0, 8, 2, 64, 1000, 16, 0, 1) == 0 and f(3, 7, 2, 64, 1000, 16, 0, 1) == 0
    assert f(3, 8, 2, 96, 1000, 16, 0, 1) == 0 and f(3, 8, 2, 64, 1000, 16, -1, 1) == 0
    f = L.gdr2_kv_workspace_bytes  # R, P, num_pages
    assert 0 < f(3, 5, 100) < f(3, 500, 100)
    assert f(0, 5, 100) == 0 and f(3, 5, -1) == 0 and f(3, 0, 100) == 0 and f(1 << 20, 1 << 12, 100) == 0
    assert f(1 << 20, 5, 1 << 30) > 1 << 33  # more than 32 bits of bytes


# ---- the binding ---------------------------------------------------------------------------------------------


def bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def test_binding_refuses_wrong_shapes_before_it_looks_at_devices():
    x, y = bf(6, 4, 64), bf(6, 2, 64)
    fr, _ = gdr2.rope_freqs(64, device="cpu")
    pos = i32(6)
    bad = [
        lambda: gdr2.attn_prologue_fwd(x, bf(5, 2, 64), None, None, pos, fr),
        lambda: gdr2.attn_prologue_fwd(x, bf(6, 2, 128), None, None, pos, fr),
        lambda: gdr2.attn_prologue_fwd(x, y, torch.ones(63), None, pos, fr),
        lambda: gdr2.attn_prologue_fwd(x, y, torch.ones(64), None, pos, fr, norm=False),
        lambda: gdr2.attn_prologue_fwd(x, y, None, None, i32(7), fr),
        lambda: gdr2.attn_prologue_fwd(x, y, None, None, None, fr),
        lambda: gdr2.attn_prologue_fwd(x.transpose(0, 1), y, None, None, pos, fr),
        lambda: gdr2.attn_prologue_fwd(x[:, :, ::2], y[:, :, :32], None, None, pos, fr),
        lambda: gdr2.attn_prologue_fwd(bf(0, 4, 64), bf(0, 2, 64), None, None, i32(0), fr),
        lambda: gdr2.attn_prologue_bwd(x, y, None, None, pos, fr, y, y),
        lambda: gdr2.attn_prologue_cache(x, y, bf(6, 3, 64), None, None, i32(6), pos, fr, bf(9, 2, 16, 64),
                                         bf(9, 2, 16, 64), i32(3, 5)),
        lambda: gdr2.attn_prologue_cache(x, y, y, None, None, i32(6), pos, fr, bf(9, 3, 16, 64), bf(9, 3, 16, 64), i32(3, 5)),
        lambda: gdr2.attn_prologue_cache(x, y, y, None, None, i32(6), None, None, bf(9, 2, 16, 64), bf(9, 2, 16, 64),
                                         i32(3, 5)),
        lambda: gdr2.attn_prologue_cache(x, y, y, None, None, i32(5), pos, fr, bf(9, 2, 16, 64), bf(9, 2, 16, 64), i32(3, 5)),
        lambda: gdr2.attn_decode(bf(3, 4, 64), bf(9, 2, 16, 64), bf(9, 2, 8, 64), i32(3, 5), i32(3)),
        lambda: gdr2.attn_decode(bf(3, 4, 64), bf(9, 2, 16, 128), bf(9, 2, 16, 128), i32(3, 5), i32(3)),
        lambda: gdr2.attn_decode(bf(3, 4, 64), bf(9, 2, 16, 64), bf(9, 2, 16, 64), i32(3, 5), i32(2)),
        lambda: gdr2.attn_decode(bf(3, 4, 64), bf(9, 2, 16, 64), bf(9, 2, 16, 64), i32(15), i32(3)),
        lambda: gdr2.attn_decode(bf(3, 4, 64), bf(9, 2, 16, 64), bf(9, 2, 16, 64), i32(), i32(3)),
        lambda: gdr2.attn_decode(bf(3, 256), bf(9, 2, 16, 64), bf(9, 2, 16, 64), i32(3, 5), i32(3)),
        lambda: gdr2.attn_decode(bf(3, 4, 64), bf(9, 32, 64), bf(9, 32, 64), i32(3, 5), i32(3)),
        lambda: gdr2.attn_decode(bf(3, 4, 64), bf(9, 2, 16, 64), bf(9, 2, 16, 64), i32(3, 5), i32(3), i32(4)),
        lambda: gdr2.attn_decode(bf(3, 4, 64), bf(9, 2, 32, 64)[:, :, ::2], bf(9, 2, 16, 64), i32(3, 5), i32(3)),
        lambda: gdr2.kv_reserve(i32(15), i32(3), i32(3), i32(9), page_size=16),
        lambda: gdr2.kv_compact(i32(), i32(9), bf(9, 2, 16, 64), bf(9, 2, 16, 64)),
        lambda: gdr2.kv_fork(i32(3, 5), i32(3), i32(9), i32(3), bf(9, 2, 1024), bf(9, 2, 1024)),
        lambda: gdr2.attn_decode(bf(3, 4, 64), bf(9, 2, 16, 64), bf(9, 2, 16, 64), i32(5, 3).t(), i32(3)),
        lambda: gdr2.kv_reserve(i32(3, 5), i32(3), i32(4), i32(9), page_size=16),
        lambda: gdr2.kv_fork(i32(3, 5), i32(3), i32(9), i32(2), bf(9, 2, 16, 64), bf(9, 2, 16, 64)),
        lambda: gdr2.kv_fork(i32(3, 5), i32(3), i32(8), i32(3), bf(9, 2, 16, 64), bf(9, 2, 16, 64)),
        lambda: gdr2.kv_compact(i32(3, 5), i32(9, 1), bf(9, 2, 16, 64), bf(9, 2, 16, 64)),
        # right shapes, but not on a CUDA device
        lambda: gdr2.attn_prologue_fwd(x, y, None, None, pos, fr),
        lambda: gdr2.attn_decode(bf(3, 4, 64), bf(9, 2, 16, 64), bf(9, 2, 16, 64), i32(3, 5), i32(3)),
        lambda: gdr2.kv_reserve(i32(3, 5), i32(3), i32(3), i32(9), page_size=16),
    ]
    for n, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            print("accepted:", n)
    wrong_type = [
        lambda: gdr2.attn_prologue_fwd(x, y.float(), None, None, pos, fr),
        lambda: gdr2.attn_prologue_fwd(x.half(), y.half(), None, None, pos, fr),
        lambda: gdr2.attn_prologue_fwd(x, y, None, None, pos, fr.float()),
        lambda: gdr2.attn_prologue_fwd(x, y, torch.ones(64).double(), None, pos, fr),
        lambda: gdr2.attn_decode(bf(3, 4, 64), bf(9, 2, 16, 64), bf(9, 2, 16, 64), i32(3, 5).long(), i32(3)),
        lambda: gdr2.kv_reserve(i32(3, 5), i32(3).long(), i32(3), i32(9), page_size=16),
        lambda: gdr2.attn_decode(bf(3, 4, 64), bf(9, 2, 16, 64).float(), bf(9, 2, 16, 64).float(), i32(3, 5), i32(3)),
        lambda: gdr2.kv_compact(i32(3, 5), i32(9), bf(9, 2, 16, 64).half(), bf(9, 2, 16, 64).half()),
        lambda: gdr2.kv_fork(i32(3, 5), i32(3), i32(9), i32(3).long(), bf(9, 2, 16, 64), bf(9, 2, 16, 64)),
    ]
    for f in wrong_type:
        with pytest.raises(TypeError):
            f()


@pytest.mark.parametrize("name,base,cases", [
    ("gdr2_attn_prologue_fwd", FWD, COMMON + [(dict(q=None), ARG), (dict(k=OFF8), ARG)]),
    ("gdr2_attn_prologue_bwd", BWD, COMMON + [(dict(dxk=None), ARG), (dict(dgq=ODD), ARG), (dict(sdk=132), ARG), (dict(wsb=16), WS)]),
    ("gdr2_attn_prologue_cache", CACHE, COMMON + [(dict(table=ODD), ARG), (dict(num=-1), ARG), (dict(sv=4), ARG)]),
    ("gdr2_attn_decode", DECODE, [(dict(seq=ODD), ARG), (dict(lse=ODD), ARG), (dict(window=-1), ARG), (dict(Hq=5), ARG),
                                  (dict(dtype=-1), ARG), (dict(ps=-4), ARG), (dict(ws=None), WS), (dict(wsb=1000), WS)]),
    ("gdr2_kv_reserve", RESERVE, PAGES + [(dict(want=None), ARG), (dict(m=None), ARG), (dict(window=-1), ARG)]),
    ("gdr2_kv_fork", FORK, PAGES + [(dict(parent=None), ARG), (dict(n=FAKE), ARG), (dict(kp=OFF8), ARG), (dict(dtype=3), ARG)]),
    ("gdr2_kv_compact", COMPACT, PAGES + [(dict(live=None), ARG), (dict(vp=None), ARG), (dict(d=100), UNS)])],
    ids=lambda x: x if isinstance(x, str) else "")
def test_records(name, base, cases):
    """A call by its record refuses what the call itself refuses, and a record of another size."""
    number, record = gdr2._CALLS[name]
    for over, status in cases:
        packed = record.pack(*(0 if x is None else x for x in {**base, **over}.values()))
        assert gdr2.lib().gdr2_attn_call(number, packed, record.size) == status, over
    assert gdr2.lib().gdr2_attn_call(number, packed, record.size - 8) == ARG
    assert gdr2.lib().gdr2_attn_call(number, None, record.size) == ARG
    assert gdr2.lib().gdr2_attn_call(7, packed, record.size) == ARG


def test_binding_refuses_sizes_beyond_32_bits():
    pools = bf(9, 2, 16, 64), bf(9, 2, 16, 64)
    for f in (lambda: gdr2.attn_decode(bf(3, 4, 64), *pools, i32(3, 5), i32(3), window=2**32 + 5),
              lambda: gdr2.attn_decode(bf(3, 4, 64), *pools, i32(3, 5), i32(3), window=5 - 2**32),
              lambda: gdr2.kv_reserve(i32(3, 5), i32(3), i32(3), i32(9), page_size=2**32 + 16),
              lambda: gdr2.kv_reserve(i32(3, 5), i32(3), i32(3), i32(9), page_size=16, window=2**40)):
        with pytest.raises(ValueError, match="too large"):
            f()


# ---- rotary frequencies -----------------------------------------------------------------------------------------


def test_rope_freqs():
    rot, base = 64, 10000.0
    plain, mag = gdr2.rope_freqs(rot, base, device="cpu")
    want = torch.tensor([base ** (-2 * i / rot) for i in range(rot // 2)], dtype=torch.float64)
    assert plain.dtype == torch.float64 and mag == 1.0
    assert torch.allclose(plain, want, rtol=1e-14, atol=0)
    lin, mag = gdr2.rope_freqs(rot, base, scaling="linear", factor=4.0, device="cpu")
    assert mag == 1.0 and torch.allclose(lin, want / 4, rtol=1e-14, atol=0)
    b, mag = gdr2.rope_freqs(rot, base, scaling="base", factor=4.0, device="cpu")
    assert mag == 1.0 and b[0] == 1 and math.isclose(float(b[-1]), float(want[-1]) / 4, rel_tol=1e-13)
    parts, mag = gdr2.rope_freqs(rot, base, scaling="parts", factor=8.0, orig_len=4096, device="cpu")
    assert math.isclose(mag, 0.1 * math.log(8) + 1, rel_tol=1e-15)
    for i in range(rot // 2):
        turns = 4096 * float(want[i]) / (2 * math.pi)
        keep = min(1.0, max(0.0, (turns - 1) / 31))
        assert math.isclose(float(parts[i]), float(want[i]) * (keep + (1 - keep) / 8), rel_tol=1e-13)
    assert parts[0] == want[0] and math.isclose(float(parts[-1]), float(want[-1]) / 8, rel_tol=1e-13)


@pytest.mark.parametrize("kw", [dict(rot=0), dict(rot=7), dict(base=0.0), dict(base=math.inf), dict(scaling="linear", factor=0.5),
                                dict(scaling="base", factor=math.nan), dict(scaling="base", rot=2, factor=2.0),
                                dict(scaling="parts", factor=2.0), dict(scaling="parts", factor=2.0, orig_len=10, turns_low=3.0,
                                                                        turns_high=3.0)], ids=str)
def test_rope_freqs_refusals(kw):
    with pytest.raises(gdr2.GDR2Error):
        gdr2.rope_freqs(**{"rot": 16, "device": "cpu", **kw})
    assert gdr2.lib().gdr2_rope_freqs(None, None, 16, 1e4, 0, 1.0, 0.0, 0.0, 0.0) == ARG
    buf = (ctypes.c_double * 8)()
    assert gdr2.lib().gdr2_rope_freqs(buf, None, 16, 1e4, 4, 1.0, 0.0, 0.0, 0.0) == ARG


def test_rope_freqs_unknown_scaling():
    with pytest.raises(ValueError):
        gdr2.rope_freqs(16, scaling="other", device="cpu")
