"""The attention half of the hybrid cell through the debug build (index checks that report GDR2_ERR_BOUNDS through
gdr2_check instead of trapping): the parity tests of tests/test_attn_gpu.py and tests/test_kv_gpu.py that end in a
check, and one call of each entry point at ragged sizes, in a child process with GDR2_DEBUG_BUILD=1."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CALLS = """
import random
import torch
from gated_delta_rule_65_b200 import build, gdr2
from tests import test_attn_gpu as A, test_kv_gpu as K
assert gdr2.lib()._name == build.DEBUG_LIB
gdr2.check()
def ok(name):
    assert gdr2.check() == gdr2.OK, name
    print(name, "ok", flush=True)
for c in A.PROLOGUE:
    A.test_prologue(c)
    ok("prologue")
A.test_cache_prologue("bf16", 64, 3, 3, 7, True)
A.test_cache_prologue("f32", 128, 5, 1, 1, True)
A.test_cache_prologue_tokens_share_a_warp(64, 1, 1, "bf16")
ok("cache")
for c in A.DECODE:
    A.test_decode(c)
ok("decode")
A.test_decode_slots_missing_pages_and_lengths_off_the_table("bf16")
ok("decode, pages missing")
for shape in K.SHAPES:
    K.test_reserve(shape, 2)
    for how in ("mixed", "one parent", "rotated"):
        K.test_fork(shape, how)
    K.test_compact(shape, torch.bfloat16)
    ok(f"pages {shape}")
K.test_serving_run(torch.bfloat16, 40)
ok("serving run")
print("all ok")
"""


def test_debug_build_attention():
    env = dict(os.environ, GDR2_DEBUG_BUILD="1")
    r = subprocess.run([sys.executable, "-c", CALLS], capture_output=True, text=True, timeout=280, cwd=ROOT, env=env)
    assert r.returncode == 0 and "all ok" in r.stdout, (r.stdout[-1000:], r.stderr[-2000:])
