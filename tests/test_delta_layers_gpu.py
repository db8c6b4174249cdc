"""The example's delta-rule layers: tokens that come one by one give what they give inside a prompt.

Tolerance, derived before the first run: the two ways differ by the roundings of each mixer's bf16
readout and of what its chunked form rounds, at most 2^-8 in the 2-norm each (both ways: 2^-7 per
layer), carried through norms and projections that keep relative size and, over two layers, added:
2^-6; the silu and norms between may stretch a difference by their slopes, less than 2: 2^-5.
"""

from __future__ import annotations

import importlib.util
from pathlib import Path

import pytest
import torch

pytestmark = pytest.mark.gpu

EXAMPLE = Path(__file__).resolve().parent.parent / "examples" / "delta_layers.py"


def load():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    spec = importlib.util.spec_from_file_location("delta_layers", EXAMPLE)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_tokens_continue_prompts():
    ex = load()
    more, lens = 3, [1, 40, 128, 261]
    g = torch.Generator(device="cuda").manual_seed(5)
    rows = [torch.randn(n + more, 512, generator=g, device="cuda").bfloat16() for n in lens]
    slots = torch.tensor([3, 1, 4, 0], dtype=torch.int32, device="cuda")
    whole = ex.DeltaLayers(6)
    want = whole.prompts(torch.cat(rows), [n + more for n in lens], slots)
    model = ex.DeltaLayers(6)
    model.prompts(torch.cat([r[:n] for r, n in zip(rows, lens)]), lens, slots)
    for k in range(more):
        got = model.step(torch.stack([r[n + k] for r, n in zip(rows, lens)]), slots)
    assert model.op.get_error() == (0, -1) and whole.op.get_error() == (0, -1)
    off = (got.double() - want.double()).norm(dim=1) / want.double().norm(dim=1)
    assert off.max() <= 2.0 ** -5, off


def test_example_runs(capsys):
    load().main()
    assert "; 0 skipped" in capsys.readouterr().out
