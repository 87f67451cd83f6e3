"""Serving a small hybrid stack: Kimi Delta Attention, linear attention with a decay per head, and
softmax attention over a paged key-value cache, one layer of each.

Prompts of different lengths run packed in one call per layer (kda_chunk_fwd_qknorm,
kda_lin_chunk_fwd; kda_paged_append, then attention among the prompt's own tokens); each sequence
then continues token by token from what the layers keep for it -- two state pools and the pages of its
cache -- with kda_recurrent_step_qknorm, kda_lin_recurrent_step, kda_paged_append and
kda_paged_attention.  Weights are random; the projections are plain matrix products.

    python examples/hybrid_serving.py [--rows 8] [--prompt 700] [--steps 32]
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from linear_attention_fwd_gb300 import kda  # noqa: E402

HEADS, KV_HEADS, D, PAGE = 4, 2, 128, 16
WIDTH = HEADS * D


def _norm(x):
    return x * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6).to(x.dtype)


class HybridStack:
    """Three layers and what they keep for `rows` sequences of at most `longest` tokens."""

    def __init__(self, rows: int, longest: int, seed: int = 0, device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)
        w = lambda n: (torch.randn(WIDTH, n, generator=gen, device=device) / WIDTH ** 0.5).to(torch.bfloat16)  # noqa: E731
        kv = KV_HEADS * D
        self.w_kda, self.w_lin, self.w_att = w(4 * WIDTH + HEADS), w(2 * kv + WIDTH + HEADS), w(WIDTH + 2 * kv)
        self.w_out = [w(WIDTH) for _ in range(3)]
        self.rows, self.longest, self.device = rows, longest, device
        self.kda_state = torch.zeros(rows, HEADS, D, D, device=device)
        self.lin_state = torch.zeros(rows, HEADS, D, D, device=device)
        self.lin_head_g = -torch.exp2(-torch.arange(1.0, HEADS + 1, device=device))   # each head's own decay
        width = -(-longest // PAGE)
        order = torch.randperm(rows * width, generator=gen, device=device)             # pages as a server hands them out
        self.table = order.view(rows, width).to(torch.int32)
        self.k_cache, self.v_cache = (torch.zeros(rows * width, PAGE, KV_HEADS, D, dtype=torch.bfloat16, device=device) for _ in range(2))
        self.lens = torch.zeros(rows, dtype=torch.int32, device=device)

    # what a layer's input projects to: x [tokens, WIDTH]
    def _kda_in(self, x):
        q, k, v, g, beta = (_norm(x) @ self.w_kda).split([WIDTH] * 4 + [HEADS], -1)
        heads = [t.reshape(-1, HEADS, D).contiguous() for t in (q, k, v)]
        g = (-5 * torch.sigmoid(g.float() - 3)).to(x.dtype).reshape(-1, HEADS, D)
        return (*heads, g, torch.sigmoid(beta).contiguous())

    def _lin_in(self, x):
        q, k, v, g = (_norm(x) @ self.w_lin).split([KV_HEADS * D, KV_HEADS * D, WIDTH, HEADS], -1)
        unit = lambda t: torch.nn.functional.normalize(t.reshape(-1, KV_HEADS, D).float(), dim=-1).to(x.dtype)  # noqa: E731
        return unit(q), unit(k), v.reshape(-1, HEADS, D).contiguous(), -torch.nn.functional.softplus(g.float() - 3)

    def _att_in(self, x):
        q, k, v = (_norm(x) @ self.w_att).split([WIDTH, KV_HEADS * D, KV_HEADS * D], -1)
        return q.reshape(-1, HEADS, D).contiguous(), *(t.reshape(-1, KV_HEADS, D).contiguous() for t in (k, v))

    def _add(self, x, o, layer):
        return x + o.reshape(x.shape) @ self.w_out[layer]

    def prefill(self, x, cu):
        """Prompts packed as x [tokens, WIDTH], int32 cu [rows + 1]; returns the stack's outputs."""
        pack = lambda ts: [t[None] for t in ts]  # noqa: E731
        o, _ = kda.kda_chunk_fwd(*pack(self._kda_in(x)), None, cu, final_state=self.kda_state, qk_eps=1e-6)
        x = self._add(x, o, 0)
        q, k, v, g = pack(self._lin_in(x))
        o, _ = kda.kda_lin_chunk_fwd(q, k, v, g, self.lin_head_g, None, cu, final_state=self.lin_state)
        x = self._add(x, o, 1)
        q, k, v = self._att_in(x)
        kda.kda_paged_append(k, v, self.k_cache, self.v_cache, self.table, torch.zeros_like(self.lens), cu)
        # A prompt's token t attends to positions 0 .. t of its row.  The cache's attention takes one new token per
        # row, so each token of the pack becomes a row with a block table of its own: it reads its row's keys and
        # values anew, some tokens^2 / 2 of them a prompt, which is fit for an example's short prompts only.  A
        # server would attend among a prompt's tokens with a kernel for prompts and fill the cache beside it.
        n = cu.long()
        row = torch.repeat_interleave(torch.arange(self.rows, device=x.device), n[1:] - n[:-1])
        seen = (torch.arange(x.shape[0], device=x.device) - n[row] + 1).to(torch.int32)
        o, _ = kda.kda_paged_attention(q, self.k_cache, self.v_cache, self.table[row], seen, D ** -0.5, output_lse=False)
        self.lens.copy_(n[1:] - n[:-1])
        return self._add(x, o, 2)

    def decode(self, x):
        """One token per row, x [rows, WIDTH]; returns the stack's outputs."""
        x = self._add(x, kda.kda_recurrent_step(*self._kda_in(x), self.kda_state, qk_eps=1e-6), 0)
        q, k, v, g = self._lin_in(x)
        x = self._add(x, kda.kda_lin_recurrent_step(q, k, v, g, self.lin_head_g, self.lin_state), 1)
        q, k, v = self._att_in(x)
        kda.kda_paged_append(k, v, self.k_cache, self.v_cache, self.table, self.lens)
        self.lens += 1
        o, _ = kda.kda_paged_attention(q, self.k_cache, self.v_cache, self.table, self.lens, D ** -0.5, output_lse=False)
        return self._add(x, o, 2)


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--rows", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=700)
    ap.add_argument("--steps", type=int, default=32)
    a = ap.parse_args()
    lens = [max(1, a.prompt * (i + 1) // a.rows) for i in range(a.rows)]
    stack = HybridStack(a.rows, max(lens) + a.steps)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    x = torch.randn(sum(lens), WIDTH, device="cuda").to(torch.bfloat16)
    y = stack.prefill(x, cu)
    x = y[cu[1:].long() - 1]
    torch.cuda.synchronize()
    start = time.perf_counter()
    for _ in range(a.steps):
        x = _norm(stack.decode(x))
    torch.cuda.synchronize()
    ms = (time.perf_counter() - start) * 1e3 / a.steps
    print(f"{a.rows} prompts of {lens[0]} .. {lens[-1]} tokens, then {a.steps} tokens each: {ms:.2f} ms per step, "
          f"last outputs' RMS {float(x.float().square().mean().sqrt()):.3f}")


if __name__ == "__main__":
    main()
