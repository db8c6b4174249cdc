"""Calls under torch.vmap, whose tensors have no storage of their own (and, from a fake mode, say that
they are on a GPU), end in an exception and leave the interpreter usable.  They run in a process of
their own, as an exception that passes the released interpreter lock ends it."""

from __future__ import annotations

import subprocess
import sys
from pathlib import Path

import pytest

ROOT = Path(__file__).resolve().parents[1]

CALLS = """
import sys
import torch
from torch._subclasses.fake_tensor import FakeTensorMode
import selective_state_update_02_gb300 as ssu

bf, i32, gpu = torch.bfloat16, torch.int32, "cuda"
with FakeTensorMode():
    if sys.argv[1] == "prompts":
        T, H, P, N = 20, 2, 64, 128
        f = lambda *s, d=torch.float32: torch.empty(*s, dtype=d, device=gpu)
        many = f(2, T, H, P, d=bf)
        run = lambda x: ssu.ssu_update_prompts(
            0, f(4, H, P, N), f(1, d=i32), f(2, d=i32), x, f(T, H, d=bf), f(H),
            f(H), f(T, 1, N, d=bf), f(T, 1, N, d=bf), f(H), f(T, H, P, d=bf), stream=0)
    else:
        f = lambda *s, d=bf: torch.empty(*s, dtype=d, device=gpu)
        many, kv, pages, at = f(2, 3, 2, 64), f(3, 1, 64), f(4, 16, 1, 64), f(3, d=i32)
        w = f(64, d=torch.float32)
        if sys.argv[1] == "rotate":
            run = lambda q: ssu.ssu_rotate_qk(0, q, kv, kv, w, w, f(8, 64, d=torch.float32),
                                              at, q, pages, pages, at, stream=0)
        else:
            run = lambda q: ssu.ssu_attend(0, q, pages, pages, f(3, 2, d=i32), at, q, stream=0)
    for _ in range(5):
        try:
            torch.vmap(run)(many)
        except RuntimeError as e:
            print("refused", e)
        else:
            print("accepted")
"""


@pytest.mark.parametrize("which", ["prompts", "rotate", "attend"])
def test_tensors_without_storage(which):
    from selective_state_update_02_gb300 import _build
    _build.build()
    r = subprocess.run([sys.executable, "-c", CALLS, which], cwd=ROOT, capture_output=True,
                       text=True, timeout=120)
    assert r.returncode == 0, (r.returncode, r.stderr[-2000:])
    assert r.stdout.count("refused") == 5 and "data pointer" in r.stdout, r.stdout
