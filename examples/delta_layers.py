"""Layers of a model whose token mixer is the gated delta rule, served with a bf16 residual stream and
a norm in front of every mixer whose output may be 8 bits wide.

Each layer adds the last one's output to the residual and norms the sum in one call (``op.add_norm``:
bf16 for the first projections, or e4m3 with a scale per 128 columns where ``eight_bits`` is set),
projects it to queries, keys, values, decays and gates, and mixes: whole prompts through
``op.delta_prompts``, which leaves each conversation's state in its slot, new tokens through
``op.delta``, one per conversation.  Weights are random; projections are plain matrix products (of the
values that e4m3 and its scales stand for).

    python examples/delta_layers.py          # a few prompts and tokens on cuda:0
"""

from __future__ import annotations

import math
import sys
from pathlib import Path

import torch

sys.path.insert(0, str(Path(__file__).resolve().parent.parent))
import selective_state_update_02_gb300 as ssu  # noqa: E402


class DeltaLayers:
    """``layers`` delta-rule layers with room for ``conversations`` states each."""

    def __init__(self, conversations, layers=2, width=512, heads=8, key_heads=4, headdim=128,
                 dstate=128, eight_bits=False, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def weight(n, m):
            return (torch.randn(n, m, generator=g, device="cuda") * n ** -0.5).bfloat16()

        self.op = ssu.SelectiveStateUpdate(0)
        self.H, self.G, self.P, self.N, self.eight_bits = heads, key_heads, headdim, dstate, eight_bits
        edge = 2 * key_heads * dstate + heads * headdim
        self.layers = [dict(
            norm=torch.rand(width, generator=g, device="cuda") + 0.5,
            into=weight(width, edge + 2 * heads), back=weight(heads * headdim, width),
            dt_bias=torch.full((heads,), -2.0, device="cuda"),
            A=-torch.exp(torch.rand(heads, generator=g, device="cuda") * math.log(16.0)),
            pool=torch.zeros(conversations, heads, headdim, dstate, device="cuda"))
            for _ in range(layers)]
        self.last = torch.ones(width, device="cuda")

    def _normed(self, x, residual, weight, eight_bits):
        if not eight_bits:
            return self.op.add_norm(x, weight, torch.empty_like(x), residual=residual)
        out = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device="cuda")
        scales = torch.empty(x.shape[0], x.shape[1] // 128, device="cuda")
        self.op.add_norm(x, weight, out, residual=residual, scales=scales)
        return (out.float() * scales.repeat_interleave(128, 1)).bfloat16()

    def _operands(self, layer, x, residual):
        u = self._normed(x, residual, layer["norm"], self.eight_bits) @ layer["into"]
        T, keys, edge = len(u), self.G * self.N, 2 * self.G * self.N + self.H * self.P
        qkv = torch.nn.functional.silu(u[:, :edge])
        return (qkv[:, :keys].view(T, self.G, self.N),
                qkv[:, keys:2 * keys].view(T, self.G, self.N),
                qkv[:, 2 * keys:].view(T, self.H, self.P), u[:, edge:edge + self.H],
                u[:, edge + self.H:])

    def prompts(self, x, lens, slots):
        """New conversations in ``slots`` from packed prompts ``x`` ``[sum(lens), width]``; the
        layers' output at each prompt's last token."""
        counts = torch.tensor(lens, device="cuda")
        cu = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).int()
        residual = torch.zeros_like(x)
        for layer in self.layers:
            q, k, v, dt, b = self._operands(layer, x, residual)
            y = torch.empty(v.shape, dtype=torch.bfloat16, device="cuda")
            n = self.op.delta_workspace_bytes(layer["pool"], v, k, slots)
            self.op.delta_prompts(layer["pool"], slots, cu, q, k, v, dt, layer["dt_bias"],
                                  layer["A"], b, y,
                                  torch.empty(n, dtype=torch.uint8, device="cuda"),
                                  fresh=torch.ones_like(slots, dtype=torch.uint8))
            x = y.flatten(1) @ layer["back"]
        return self._normed(x, residual, self.last, False)[cu[1:].long() - 1]

    def step(self, x, slots):
        """One more token of each conversation in ``slots``, ``x`` ``[len(slots), width]``."""
        residual = torch.zeros_like(x)
        for layer in self.layers:
            q, k, v, dt, b = self._operands(layer, x, residual)
            y = torch.empty(v.shape, dtype=torch.bfloat16, device="cuda")
            self.op.delta(layer["pool"], slots, q, k, v, dt, layer["dt_bias"], layer["A"], b, y)
            x = y.flatten(1) @ layer["back"]
        return self._normed(x, residual, self.last, False)


def main():
    torch.manual_seed(0)
    lens = [37, 300, 5, 129]
    model = DeltaLayers(conversations=6, eight_bits=True)
    slots = torch.tensor([4, 0, 5, 2], dtype=torch.int32, device="cuda")
    out = model.prompts(torch.randn(sum(lens), 512, device="cuda").bfloat16(), lens, slots)
    for _ in range(8):
        out = model.step(out, slots)
    skipped, _ = model.op.get_error()  # waits for the work
    print(f"{len(lens)} conversations of {sum(lens)} prompt tokens, 8 more tokens each; "
          f"{skipped} skipped, last output's root mean square "
          f"{out.float().square().mean().sqrt().item():.3f}")


if __name__ == "__main__":
    main()
