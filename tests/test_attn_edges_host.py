"""Host-side edges of the attention half (no GPU: nothing here launches a kernel)."""
from __future__ import annotations

import os
import re

import pytest
import torch

from gated_delta_rule_65_b200 import build, gdr2


def test_decode_workspace_of_more_slots_than_sequences():
    """Slots may share sequences (seq), so that N P may pass the bound of a table, R P: the workspace, which depends on
    neither R nor the pool, is still asked for."""
    f = gdr2.lib().gdr2_attn_decode_workspace_bytes  # N, Hq, Hk, d, P, page_size, window, dtype
    P = 1 << 20
    few = f(3, 8, 2, 64, P, 16, 0, gdr2.GDR2_BF16)
    assert few > 0
    for n in (2047, 2048, 4096, 1 << 20):
        assert f(n, 8, 2, 64, P, 16, 0, gdr2.GDR2_BF16) == few
    assert f(1 << 28, 8, 2, 64, P, 16, 0, gdr2.GDR2_BF16) == 0  # N Hq past 32 bits: no such call
    assert f(3, 8, 2, 64, P, 2048, 0, gdr2.GDR2_BF16) == 0      # P page_size past 32 bits


def test_no_non_coherent_loads_where_launches_overlap():
    """The kernels of the attention half become resident while their predecessors still write what they will read; a
    non-coherent load asks that nobody does."""
    names = [p for p in build.sources() if os.path.basename(p).startswith(("attn_", "kv_"))]
    assert len(names) == 4
    for path in names + [os.path.join(build.CSRC, n) for n in ("attn.h", "attn_vec.cuh")]:
        with open(path) as f:
            code = re.sub(r"//[^\n]*", "", f.read())
        assert not re.search(r"__ldg\b|ld\.global\.nc|\bconst\b[^;,()]*\*\s*__restrict__", code), path


def test_workspace_sizes_are_kept_for_a_bounded_number_of_calls():
    """A process whose batches and tables keep changing does not grow by an entry for each of them."""
    like = torch.zeros(16)
    held = [n for n, x in vars(gdr2).items() if isinstance(x, (dict, list, set))]
    before = {n: len(getattr(gdr2, n)) for n in held}
    for n in range(1, 5000):
        ws, size = gdr2._scratch(like, None, "gdr2_kv_workspace_bytes", n, 3, 10)
        assert size == gdr2.lib().gdr2_kv_workspace_bytes(n, 3, 10) and ws.numel() * 4 >= size
    assert {n: len(getattr(gdr2, n)) for n in held} == before
    assert gdr2._need.cache_info().currsize <= 1024


FAKE = 0x10000  # aligned, never dereferenced: the missing workspace is found after the sizes and before any launch
TOP = 2**31 - 65536


def reserve(R, P, ps, num):
    return gdr2.lib().gdr2_kv_reserve(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, R, P, ps, num, 0, None, 0, None)


def compact(Hk, ps, d, num, dtype):
    return gdr2.lib().gdr2_kv_compact(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1, 1, Hk, ps, d, num, dtype, None, 0, None)


def fork(Hk, ps, d, num, dtype):
    return gdr2.lib().gdr2_kv_fork(FAKE, FAKE, FAKE, FAKE, FAKE + 64, FAKE + 64, FAKE, FAKE, FAKE, FAKE, 1, 1, Hk, ps, d, num,
                                   dtype, None, 0, None)


def decode(N, Hq, Hk, P, ps, num):
    return gdr2.lib().gdr2_attn_decode(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1.0, 0, FAKE, None, N, Hq, Hk, 64, 1, P, ps, num, 1,
                                       None, 0, None)


@pytest.mark.parametrize("call,held,beyond", [
    (reserve, (1, 1, TOP, 9), (1, 1, TOP + 1, 9)),
    (reserve, (1, TOP // 16, 16, 9), (1, TOP // 16 + 1, 16, 9)),
    (reserve, (TOP // 32, 32, 1, 9), (TOP // 32 + 1, 32, 1, 9)),
    (reserve, (3, 5, 16, TOP), (3, 5, 16, TOP + 1)),
    (compact, (65535, 16, 64, 9, 1), (65536, 16, 64, 9, 1)),
    (compact, (32767, 2**20, 64, 1, 1), (32768, 2**20, 64, 1, 1)),  # c = 2^31 at the second
    (fork, (2, 32, 64, 2**30 - 16385, 1), (2, 32, 64, 2**30 - 16384, 1)),  # c = 4
    (compact, (1, 8, 128, 2**31 - 65536, 0), (2, 8, 128, 2**31 - 65536, 0)),
    (decode, ((2**31 - 1) // 8, 8, 2, 1000, 16, 9), (2**28, 8, 2, 1000, 16, 9)),
    (decode, (3, 8, 2, 2, 2**30 - 32768, 1), (3, 8, 4, 2, 2**30 - 32768, 1)),
    (decode, (3, 8, 2, 1000, 16, 2**27 - 1), (3, 8, 2, 1000, 16, 2**27)),
    (decode, (3, 65520, 65520, 1000, 16, 9), (3, 65536, 65536, 1000, 16, 9)),
    (decode, (3, 1024, 1, 1000, 16, 9), (3, 1025, 1, 1000, 16, 9)),
], ids=lambda x: getattr(x, "__name__", str(x)))
def test_sizes_of_the_header_on_both_sides(call, held, beyond):
    assert call(*held) == gdr2.ERR_WORKSPACE and call(*beyond) == gdr2.ERR_UNSUPPORTED
