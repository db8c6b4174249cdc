"""A wait of the delta rule's passes that nothing ends: it gives up by itself."""

from __future__ import annotations

import subprocess
from pathlib import Path

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = Path(__file__).resolve().parents[1]


def test_a_wait_gives_up(tmp_path):
    """After a second and more, and less than the ten seconds that a wait for another CTA has."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from selective_state_update_02_gb300 import _build
    exe = tmp_path / "bounded_wait"
    subprocess.run([_build.nvcc_path(), *_build.ARCH, "-O3", "-std=c++17",
                    "-I", str(ROOT / "selective_state_update_02_gb300" / "csrc"),
                    str(ROOT / "tests" / "c" / "bounded_wait.cu"), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, (r.returncode, r.stderr)
    first, second = map(int, r.stdout.split())
    assert 5e8 < first < 1e10 and second < 1e6, (first, second)
