"""The prompt, rotation and attention entry points without a GPU: the declared argument structs
have the header's layout, and calls that must be refused are refused on the host."""

from __future__ import annotations

import ctypes
import re
import subprocess
from pathlib import Path

import pytest
import torch

ROOT = Path(__file__).resolve().parents[1]


@pytest.fixture(scope="module")
def ssu():
    from selective_state_update_02_gb300 import _build
    _build.build()
    import selective_state_update_02_gb300 as m
    m.lib()
    return m


def test_struct_layouts(ssu):
    for name, words, tail in (("ssu_rotate_shape_t", 8, 2), ("ssu_rotate_strides_t", 17, 0),
                              ("ssu_attend_shape_t", 7, 2), ("ssu_attend_strides_t", 13, 0)):
        assert ctypes.sizeof(getattr(ssu, name)) == 8 * words + 4 * tail


def prompts_operands(T=20, H=2, P=64, N=128):
    bf = torch.bfloat16
    return dict(pool=torch.zeros(4, H, P, N), slots=torch.zeros(1, dtype=torch.int32),
                cu=torch.tensor([0, T], dtype=torch.int32), x=torch.zeros(T, H, P, dtype=bf),
                dt=torch.zeros(T, H, dtype=bf), dt_bias=torch.zeros(H), A=torch.zeros(H),
                B=torch.zeros(T, 1, N, dtype=bf), C=torch.zeros(T, 1, N, dtype=bf),
                D=torch.zeros(H), out=torch.zeros(T, H, P, dtype=bf))


@pytest.mark.parametrize("error,change", [
    (TypeError, dict(x=torch.zeros(20, 2, 64))),
    (TypeError, dict(cu=torch.zeros(2, dtype=torch.int64))),
    (ValueError, dict(cu=torch.zeros(3, dtype=torch.int32))),
    (ValueError, dict(out=torch.zeros(19, 2, 64, dtype=torch.bfloat16))),
    (TypeError, dict(x=None)),
    (ValueError, {})])  # host tensors
def test_prompts_refusals(ssu, error, change):
    with pytest.raises(error):
        ssu.ssu_update_prompts(0, *{**prompts_operands(), **change}.values(), stream=0)


def test_rotate_and_attend_refuse_host_tensors_and_types(ssu):
    bf = torch.bfloat16
    q, kv, w = torch.zeros(3, 2, 64, dtype=bf), torch.zeros(3, 1, 64, dtype=bf), torch.ones(64)
    pages, at = torch.zeros(4, 16, 1, 64, dtype=bf), torch.zeros(3, dtype=torch.int32)
    table, rows = torch.zeros(8, 64), torch.zeros(3, 2, dtype=torch.int32)
    with pytest.raises(ValueError):
        ssu.ssu_rotate_qk(0, q, kv, kv, w, w, table, at, q, pages, pages, at)
    with pytest.raises(TypeError):
        ssu.ssu_rotate_qk(0, q.float(), kv, kv, w, w, table, at, q, pages, pages, at)
    with pytest.raises(ValueError):
        ssu.ssu_attend(0, q, pages, pages, rows, at, q.clone())
    with pytest.raises(TypeError):
        ssu.ssu_attend(0, q, pages, pages, rows.long(), at, q.clone())


def test_null_handles_are_refused(ssu):
    lib, n = ssu.lib(), ctypes.c_int64()
    shape = bytes(ssu.ssu_shape_t(1, 2, 64, 128, 1, 4, 0, 0))
    for status in (
            lib.ssu_prompts_workspace_bytes(None, shape, 20, ctypes.byref(n)),
            lib.ssu_update_prompts(None, *[None] * 12, shape, bytes(27 * 8), 20, None, 0, None),
            lib.ssu_rotate_qk(None, *[None] * 11, bytes(72), bytes(136), 1e-6, None),
            lib.ssu_attend_workspace_bytes(None, bytes(64), ctypes.byref(n)),
            lib.ssu_attend(None, *[None] * 6, bytes(64), bytes(104), 1.0, 0, 0, None, 0, None)):
        assert status == ssu.SSU_ERR_INVALID_ARG


# unit -> kernel -> (most registers, most spilled bytes).  Prompts: 352 threads, one CTA per SM, a
# row of 64 fp32 state values per thread; attention: one CTA of 8 warps per SM; rotation: 32 warps
# per SM.
BUDGETS = {
    "ssu_prompt.cu": {"ssu_prompt_mma_kernel": (168, 32), "ssu_prompt_seq_kernel": (128, 8)},
    "ssu_attend.cu": {"ssu_attend_kernelILi256E": (255, 256), "ssu_attend_kernelILi128E": (255, 0),
                      "ssu_attend_kernelILi64E": (255, 0)},
    "ssu_rotate.cu": {"ssu_rotate_kernel": (64, 32)},
}


@pytest.mark.parametrize("unit", sorted(BUDGETS))
def test_register_budgets(tmp_path, unit):
    from selective_state_update_02_gb300 import _build
    csrc = ROOT / "selective_state_update_02_gb300" / "csrc"
    out = subprocess.run(
        [_build.nvcc_path(), *_build.ARCH, "-O3", "-std=c++17", "-I", str(ROOT / "include"), "-I",
         str(csrc), "-Xptxas", "-v", "-cubin", "-c", str(csrc / unit), "-o",
         str(tmp_path / "unit.cubin")], capture_output=True, text=True, timeout=600,
        check=True).stderr
    seen = set()
    for block in out.split("ptxas info    : Compiling entry function '")[1:]:
        name = block.split("'")[0]
        used = int(re.search(r"Used (\d+) registers", block).group(1))
        spill = int(re.search(r"(\d+) bytes spill stores", block).group(1))
        for kernel, (most, spilled) in BUDGETS[unit].items():
            if kernel in name:
                seen.add(kernel)
                assert used <= most and spill <= spilled, (name, used, spill)
    assert seen == set(BUDGETS[unit])
