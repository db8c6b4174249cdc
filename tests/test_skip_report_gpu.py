"""What ssu_get_error says of a skipped token, request, page or prompt: its number in the call that
skipped it, and no word of a slot of the state pool where none was named."""

from __future__ import annotations

import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import selective_state_update_02_gb300 as ssu  # noqa: E402
import test_attend_gpu  # noqa: E402
import test_prompts_gpu  # noqa: E402
import test_rotate_gpu  # noqa: E402


@pytest.fixture(scope="module")
def op():
    handle = ssu.SelectiveStateUpdate(0)
    yield handle
    torch.cuda.synchronize()
    handle.close()


def report(op):
    n, first = ctypes.c_uint32(), ctypes.c_int64()
    status = ssu.lib().ssu_get_error(op.handle, None, ctypes.byref(n), ctypes.byref(first))
    assert status == ssu.SSU_ERR_INDEX_OOB
    return n.value, first.value, ssu.last_error()


def test_position_of_a_token(op):
    d = test_rotate_gpu.make(9, 4, 2, 64, 64)
    d["positions"][5] = d["table"].shape[0]
    op.rotate_qk(**d)
    n, first, text = report(op)
    assert (n, first) == (1, 5) and "position" in text and "number 5" in text
    assert "slot outside the pool" not in text


def test_length_and_page_of_a_request(op):
    d = test_attend_gpu.make([20, 30, 40])
    d["lengths"][2] = -1
    d["page_table"][1, 0] = -1
    op.attend(**d, workspace=test_attend_gpu.workspace(op, d))
    n, first, text = report(op)
    assert (n, first) == (2, 1) and "length" in text and "pages" in text
    assert "slot outside the pool" not in text


def test_offsets_of_a_prompt(op):
    d = test_prompts_gpu.make([20, 30], H=2)
    d["cu"][2] = 10 ** 6
    test_prompts_gpu.call(op, d)
    n, first, text = report(op)
    assert (n, first) == (1, 1) and "offset" in text and "number 1" in text
    assert "slot outside the pool" not in text
