"""ssu_prompts_workspace_bytes refuses, without a GPU, the sizes that ssu_update_prompts refuses.
Each query runs in a process of its own, as a library that divides by such a size ends it."""

from __future__ import annotations

import subprocess
import sys
from pathlib import Path

import pytest

ROOT = Path(__file__).resolve().parents[1]

# The handle is zeros, but for its second word, the number of SMs (struct ssu_handle_s).
QUERY = """
import ctypes, struct, sys
import selective_state_update_02_gb300 as ssu
handle = ctypes.create_string_buffer(struct.pack("ii", 0, 152), 4096)
*shape, tokens = (int(v) for v in sys.argv[1:])
n = ctypes.c_int64(-1)
status = ssu.lib().ssu_prompts_workspace_bytes(ctypes.addressof(handle),
                                               bytes(ssu.ssu_shape_t(*shape)), tokens,
                                               ctypes.byref(n))
print(status, n.value)
"""


def query(batch=2, heads=4, headdim=64, dstate=128, groups=1, pool=4, index=0, state=0,
          tokens=2000):
    from selective_state_update_02_gb300 import _build
    _build.build()
    r = subprocess.run([sys.executable, "-c", QUERY, *map(str, (
        batch, heads, headdim, dstate, groups, pool, index, state, tokens))], cwd=ROOT,
        capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, f"the query ended its process: {r.returncode} {r.stderr}"
    return tuple(map(int, r.stdout.split()))


@pytest.mark.parametrize("status,sizes", [
    (1, dict(groups=0)), (1, dict(groups=-1)), (1, dict(heads=4, groups=3)), (1, dict(heads=0)),
    (1, dict(batch=-1)), (1, dict(tokens=-1)), (1, dict(tokens=2 ** 31)), (1, dict(index=2)),
    (1, dict(state=7)), (2, dict(dstate=32)), (2, dict(heads=70000)), (2, dict(headdim=2 ** 21)),
    (2, dict(batch=2 ** 30, heads=4))], ids=str)
def test_refusals(status, sizes):
    assert query(**sizes) == (status, -1)


def test_sizes_that_are_accepted():
    status, n = query()
    assert status == 0 and n > 0 and n % 256 == 0
    assert query(dstate=256) == (0, 0) and query(headdim=24) == (0, 0) and query(batch=0)[0] == 0


@pytest.mark.parametrize("chunked,sizes", [
    (True, dict(batch=1, tokens=2 ** 31 - 1 - 512)),
    # token numbers past a chunk's end would not fit 32 bits: token by token
    (False, dict(batch=1, tokens=2 ** 31 - 512)), (False, dict(batch=1, tokens=2 ** 31 - 1)),
    # stretches times CTAs, where those are not shared: 4097 * 4864 and 32769 * 243200
    (True, dict(batch=4096, heads=1216, headdim=512, tokens=2 ** 31 - 600)),
    (False, dict(batch=32768, heads=60800, headdim=512, tokens=2 ** 31 - 600))], ids=str)
def test_calls_too_large_for_chunks_ask_for_no_workspace(chunked, sizes):
    status, n = query(**sizes)
    assert status == 0 and (n > 0) == chunked
