"""Host logic of the attention kernel, checked without a GPU."""

from __future__ import annotations

import subprocess
from pathlib import Path

ROOT = Path(__file__).resolve().parents[1]


def test_empty_requests_are_looked_for_only_where_there_are_some(tmp_path):
    from selective_state_update_02_gb300 import _build
    exe = tmp_path / "empty_requests"
    subprocess.run([_build.nvcc_path(), *_build.ARCH, "-O1", "-std=c++17",
                    "-I", str(ROOT / "include"),
                    "-I", str(ROOT / "selective_state_update_02_gb300" / "csrc"),
                    str(ROOT / "tests" / "c" / "empty_requests.cu"), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr
