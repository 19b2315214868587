"""One attention block of a served model on the library: W4A16 projections around a
paged key/value cache, for a batch of requests behind a shared prefix.

A step takes any mix of prompts, chunks of prompts and single tokens:

    slots    hq_kv_slots   pages for the new tokens, their slots and positions
    qkv      hq_gemm       W4A16 projection of the hidden states
    rotate   hq_rope_kv    rotary positions; keys and values into the cache
    attend   hq_attn       the shared prefix and each request's own pages
    output   hq_gemm       W4A16 projection back

Run it for a prompt step and a few decode steps with random weights:

    python3 examples/served_block.py
"""
from __future__ import annotations

import os
import sys

import numpy as np
import torch

if __package__ in (None, ""):
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from bit_quantized_gemm_w4a16_amd import hq  # noqa: E402


class Linear:
    """A W4A16 layer (symmetric INT4, group 128) of random weights, bf16."""

    def __init__(self, N, K, rng):
        self.N, self.K = N, K
        self.desc = hq.desc_w4a16(N, K, 128, bf16=True)
        codes = rng.integers(0, 1 << 32, (K // 8, N), dtype=np.uint32)
        scale = torch.full((K // 128, N), 0.25 / K ** 0.5, dtype=torch.bfloat16).view(torch.int16).numpy()
        w, s, _ = hq.hq_repack(self.desc, codes, scale)
        self.w, self.s = torch.from_numpy(w).cuda(), torch.from_numpy(s).cuda()

    def __call__(self, x, out, workspace):
        hq.hq_gemm(self.desc, x.shape[0], x, None, self.w, self.s, None, out, workspace, workspace.numel())
        return out


class ServedBlock:
    def __init__(self, hidden=1024, q_heads=16, kv_heads=2, head_dim=64, block=16, num_blocks=512, max_requests=64, max_tokens=2048,
                 max_context=4096, fp8_cache=False, seed=0):
        rng = np.random.default_rng(seed)
        self.q_heads, self.kv_heads, self.head_dim, self.block = q_heads, kv_heads, head_dim, block
        self.q_row, self.row = q_heads * head_dim, (q_heads + 2 * kv_heads) * head_dim
        self.qkv, self.proj = Linear(self.row, hidden, rng), Linear(hidden, self.q_row, rng)
        self.kv = hq.kv_desc(hq.HQ_DT_FP8_E4M3 if fp8_cache else hq.HQ_DT_BF16, num_blocks, block, kv_heads, head_dim)
        cache = torch.float8_e4m3fn if fp8_cache else torch.bfloat16
        self.k_cache, self.v_cache = (torch.zeros(num_blocks, block, kv_heads, head_dim, device="cuda").to(cache) for _ in range(2))
        self.k_scale, self.v_scale = (torch.full((kv_heads,), 0.05, device="cuda") if fp8_cache else None for _ in range(2))
        self.rope = hq.rope_desc(head_dim, scaling=hq.HQ_ROPE_PARTS, factor=2.0, context=max_context // 2)
        self.table = torch.empty(max_context, head_dim, device="cuda")
        hq.hq_rope_table(self.rope, 0, max_context, self.table)
        i32 = lambda *n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
        self.free = torch.randperm(num_blocks, generator=torch.Generator().manual_seed(seed)).to(torch.int32).cuda()
        self.max_blocks = -(-max_context // block)
        self.blocks = torch.full((max_requests, self.max_blocks), -1, dtype=torch.int32, device="cuda")
        self.cached, self.kv_lens, self.cu, self.taken = i32(max_requests), i32(max_requests), i32(max_requests + 1), i32(1)
        self.prefix_table, self.prefix_len = i32(self.max_blocks), 0
        self.positions, self.slots = i32(max_tokens), torch.zeros(max_tokens, dtype=torch.int64, device="cuda")
        self.lens, self.workspace = [0] * max_requests, torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
        self.x_qkv = torch.empty(max_tokens, self.row, dtype=torch.bfloat16, device="cuda")
        self.q, self.heads = (torch.empty(max_tokens, self.q_row, dtype=torch.bfloat16, device="cuda") for _ in range(2))

    def share_prefix(self, x):
        """Runs the prompt that all requests share (request 0 of an otherwise empty
        block) and keeps its pages as the prefix."""
        if any(self.lens) or self.prefix_len:
            raise ValueError("a prefix is shared before all else")
        out = self.step(x, [x.shape[0]])
        self.prefix_len = x.shape[0]
        self.prefix_table.copy_(self.blocks[0])
        self.blocks[0].fill_(-1)
        self.cached.zero_()
        self.lens = [0] * len(self.lens)
        return out

    def admit(self, x, new):
        """Refuses a step that the buffers do not hold, before anything is launched or
        changed (the library is given addresses: it cannot tell).  Returns the lengths
        after the step and the pages that it takes."""
        T, hidden, context = sum(new), self.qkv.K, self.table.shape[0]
        if (any(n < 0 for n in new) or tuple(x.shape) != (T, hidden) or x.dtype != torch.bfloat16 or not x.is_contiguous()
                or x.device != self.positions.device):
            raise ValueError(f"x must be a contiguous bf16 [{T}][{hidden}] beside the cache: a row for each new token")
        if not 0 < T <= self.positions.numel() or len(new) > len(self.lens):
            raise ValueError(f"{T} tokens of {len(new)} requests: from 1 to {self.positions.numel()} tokens of up to {len(self.lens)} requests fit")
        after = [c + n for c, n in zip(self.lens, new)]
        if self.prefix_len + max(after) > context:
            raise ValueError(f"a request of {max(after)} tokens behind a prefix of {self.prefix_len} exceeds the context of {context}")
        taken = sum(-(-k // self.block) - -(-c // self.block) for c, k in zip(self.lens, after))
        if taken > self.free.numel():
            raise ValueError(f"out of pages: {taken} needed, {self.free.numel()} free")
        return after, taken

    def step(self, x, new):
        """x: hidden states [sum(new)][hidden] of new[r] new tokens of request r."""
        B, T, dt = len(new), x.shape[0], hq.HQ_DT_BF16
        after, taken = self.admit(x, new)
        fresh = torch.tensor(new, dtype=torch.int32, device="cuda")
        hq.hq_kv_slots(self.block, B, T, self.cached, fresh, self.free, self.free.numel(), self.blocks, self.max_blocks, self.cu, self.kv_lens,
                       self.positions, self.slots, self.taken, first_pos=self.prefix_len)
        self.qkv(x, self.x_qkv, self.workspace)
        k, v = self.x_qkv[:, self.q_row:], self.x_qkv[:, self.q_row + self.kv_heads * self.head_dim:]
        hq.hq_rope_kv(self.rope, self.kv, dt, T, self.q_heads, self.x_qkv, self.row, k, self.row, v, self.row, self.positions, self.table,
                      self.table.shape[0], self.slots, self.q, self.q_row, self.k_cache, self.v_cache, self.k_scale, self.v_scale)
        # the host knows the lengths too: it uses them to size the launch
        desc = hq.attn_desc(dt, self.q_heads, max(new), max(after), self.head_dim ** -0.5, total_kv=sum(after))
        need = hq.hq_attn_workspace_bytes(desc, self.kv, B, T, self.prefix_len)
        if need > self.workspace.numel():
            self.workspace = torch.empty(need, dtype=torch.uint8, device="cuda")
        hq.hq_attn(desc, self.kv, B, T, self.q, self.q_row, self.k_cache, self.v_cache, self.prefix_table, self.prefix_len, self.blocks,
                   self.max_blocks, self.kv_lens, self.cu, self.heads, self.q_row, None, self.workspace, self.workspace.numel(), self.k_scale,
                   self.v_scale)
        self.lens[:B] = after
        self.free = self.free[taken:]
        self.cached[:B].copy_(self.kv_lens[:B])
        out = torch.empty(T, self.proj.N, dtype=torch.bfloat16, device="cuda")
        return self.proj(self.heads[:T], out, self.workspace)


def main():
    block = ServedBlock()
    hidden = block.qkv.K
    gen = torch.Generator(device="cuda").manual_seed(1)
    tokens = lambda n: torch.randn(n, hidden, device="cuda", generator=gen).to(torch.bfloat16)  # noqa: E731
    block.share_prefix(tokens(300))
    prompts = [17, 1, 130, 64]
    y = block.step(tokens(sum(prompts)), prompts)
    for i in range(4):
        y = block.step(tokens(len(prompts)), [1] * len(prompts))
        torch.cuda.synchronize()
        print(f"step {i}: lengths {block.lens[:len(prompts)]} behind a prefix of {block.prefix_len}, output rms {y.float().pow(2).mean().sqrt():.3f}")


if __name__ == "__main__":
    main()
