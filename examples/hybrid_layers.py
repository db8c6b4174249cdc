"""A state-space layer and an attention layer of a hybrid model, served side by side.

Prompts come in packed: the state-space layer runs them through ``op.prompts``, which leaves each
conversation's state in its slot; the attention layer norms and rotates their queries and keys
into the paged cache (``op.rotate_qk``) and attends from every prompt's last token
(``op.attend``).  New tokens then go through both layers one per conversation: the decode-step
update (``op(...)``) continues the slots, and the cache grows by a key.  Weights are random;
projections are plain matrix products.

    python examples/hybrid_layers.py          # a few prompts and tokens on cuda:0
"""

from __future__ import annotations

import math
import sys
from pathlib import Path

import torch

sys.path.insert(0, str(Path(__file__).resolve().parent.parent))
import selective_state_update_02_gb300 as ssu  # noqa: E402


class HybridPair:
    """One state-space and one attention layer with room for ``conversations`` caches."""

    def __init__(self, conversations, max_tokens, width=512, H=16, P=64, N=128, G=1, q_heads=8,
                 kv_heads=2, dim=128, page=16, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def weight(n, m):
            return (torch.randn(n, m, generator=g, device="cuda") * n ** -0.5).bfloat16()

        self.H, self.P, self.N, self.G = H, P, N, G
        self.q_heads, self.kv_heads, self.dim, self.page = q_heads, kv_heads, dim, page
        self.op = ssu.SelectiveStateUpdate(0)
        self.to_xbc, self.to_dt = weight(width, H * P + 2 * G * N), weight(width, H)
        self.from_y, self.from_heads = weight(H * P, width), weight(q_heads * dim, width)
        self.to_qkv = weight(width, (q_heads + 2 * kv_heads) * dim)
        self.A = -torch.exp(torch.rand(H, generator=g, device="cuda") * math.log(16.0))
        self.D, self.dt_bias = torch.ones(H, device="cuda"), torch.full((H,), -2.0, device="cuda")
        self.q_weight, self.k_weight = (torch.ones(dim, device="cuda") for _ in range(2))
        angle = torch.arange(max_tokens, dtype=torch.float64)[:, None] * \
            10000.0 ** (-torch.arange(0, dim, 2, dtype=torch.float64) / dim)
        self.table = torch.cat([angle.cos(), angle.sin()], 1).float().cuda()
        # what a conversation keeps: a slot of states and its pages of keys and values
        self.pool = torch.zeros(conversations, H, P, N, device="cuda")
        per = -(-max_tokens // page)
        pages = torch.randperm(conversations * per, generator=g, device="cuda")
        self.page_table = pages.int().view(conversations, per)
        self.k_pages, self.v_pages = (
            torch.zeros(conversations * per, page, kv_heads, dim, dtype=torch.bfloat16,
                        device="cuda") for _ in range(2))
        self.lengths = torch.zeros(conversations, dtype=torch.int32, device="cuda")
        most = torch.empty(conversations, q_heads, dim, dtype=torch.bfloat16, device="cuda")
        n = self.op.attend_workspace_bytes(most, self.k_pages)  # zeros once; calls leave it so
        self.attend_workspace = torch.zeros(n, dtype=torch.uint8, device="cuda")

    def _state_space_operands(self, hidden):
        xbc, edge = _norm(hidden) @ self.to_xbc, self.H * self.P
        T, step = hidden.shape[0], self.G * self.N
        return (xbc[:, :edge].view(T, self.H, self.P), _norm(hidden) @ self.to_dt,
                xbc[:, edge:edge + step].view(T, self.G, self.N),
                xbc[:, edge + step:].view(T, self.G, self.N))

    def _into_cache(self, hidden, who, positions):
        """Queries of ``hidden``, whose keys and values are now in the cache."""
        T, hq, hk = hidden.shape[0], self.q_heads, self.kv_heads
        qkv = (_norm(hidden) @ self.to_qkv).view(T, hq + 2 * hk, self.dim)
        q = qkv[:, :hq]
        slots = self.page_table[who, positions // self.page] * self.page + positions % self.page
        self.op.rotate_qk(q, qkv[:, hq:hq + hk], qkv[:, hq + hk:], self.q_weight, self.k_weight,
                          self.table, positions.int(), q, self.k_pages, self.v_pages, slots.int())
        return q

    def _attend(self, q, who):
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
        self.op.attend(q, self.k_pages, self.v_pages, self.page_table[who], self.lengths[who],
                       out, self.attend_workspace)
        return out.flatten(1) @ self.from_heads

    def prompts(self, hidden, lens, who):
        """New conversations ``who`` from packed prompts ``hidden`` ``[sum(lens), width]``;
        the layers' output at each prompt's last token."""
        counts = torch.tensor(lens, device="cuda")
        cu = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).int()
        x, dt, B, C = self._state_space_operands(hidden)
        y = torch.empty(x.shape, dtype=torch.bfloat16, device="cuda")
        n = self.op.prompts_workspace_bytes(self.pool, x, B, who)
        self.op.prompts(self.pool, who, cu, x, dt, self.dt_bias, self.A, B, C, self.D, y,
                        torch.empty(n, dtype=torch.uint8, device="cuda"),
                        fresh=torch.ones_like(who, dtype=torch.uint8))
        hidden = hidden + y.flatten(1) @ self.from_y
        of = torch.repeat_interleave(who.long(), counts)
        positions = torch.arange(len(hidden), device="cuda") - \
            torch.repeat_interleave(cu[:-1].long(), counts)
        q = self._into_cache(hidden, of, positions)
        self.lengths[who.long()] = counts.int()
        last = cu[1:].long() - 1
        return hidden[last] + self._attend(q[last], who.long())

    def step(self, hidden, who):
        """One more token of each conversation in ``who``, ``hidden`` ``[len(who), width]``."""
        x, dt, B, C = self._state_space_operands(hidden)
        y = torch.empty(x.shape, dtype=torch.bfloat16, device="cuda")
        self.op(self.pool, who, x, dt, self.dt_bias, self.A, B, C, self.D, y)
        hidden = hidden + y.flatten(1) @ self.from_y
        at = who.long()
        q = self._into_cache(hidden, at, self.lengths[at].long())
        self.lengths[at] += 1
        return hidden + self._attend(q, at)


def _norm(t):
    t = t.float()
    return (t * torch.rsqrt(t.square().mean(-1, keepdim=True) + 1e-6)).bfloat16()


def main():
    torch.manual_seed(0)
    lens = [37, 300, 5, 129]
    pair = HybridPair(conversations=6, max_tokens=512)
    who = torch.tensor([4, 0, 5, 2], dtype=torch.int32, device="cuda")
    out = pair.prompts(torch.randn(sum(lens), 512, device="cuda").bfloat16(), lens, who)
    for _ in range(8):
        out = pair.step(out, who)
    skipped, _ = pair.op.get_error()  # waits for the work
    print(f"{len(lens)} conversations of {sum(lens)} prompt tokens, 8 more tokens each; "
          f"{skipped} skipped, last output's root mean square "
          f"{out.float().square().mean().sqrt().item():.3f}")


if __name__ == "__main__":
    main()
