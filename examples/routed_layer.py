"""One mixture-of-experts layer of a served model on the library: FP8 experts with
block scales behind a norm and a router, for the tokens of a step.

    norm       hq_rmsnorm         the residual's addition; 16 bits for the router
    codes      hq_rmsnorm         the same rows as FP8 codes with block scales
    logits     a small product    of torch, in the 16-bit type
    route      hq_moe_route       the experts of each token and their weights
    gate, up   hq_moe_gemm        an expert's two projections side by side
    SwiGLU     hq_silu_mul_quant  FP8 codes with block scales again
    down       hq_moe_gemm        back to the hidden width
    combine    hq_moe_combine     the weighted sum

The experts' rows come in the tokens' order (Indexed), or sorted by expert
(`grouped`: hq_moe_align and hq_moe_gather before, as a layer does whose experts
lie on several cards); either gives the same bits.  All buffers are the layer's
own, so that a step can be captured in a graph.  Run it for a prompt step and a few
single tokens with random weights:

    python3 examples/routed_layer.py
"""
from __future__ import annotations

import os
import sys

import numpy as np
import torch

if __package__ in (None, ""):
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from bit_quantized_gemm_w4a16_amd import hq  # noqa: E402


class Experts:
    """FP8 experts (E4M3 codes, a scale for each 128 x 128) of random weights."""

    def __init__(self, E, N, K, rng):
        self.E, self.N, self.K = E, N, K
        self.desc = hq.desc_moe_fp8_blockwise(E, N, K)
        codes = torch.from_numpy(rng.standard_normal((E, K, N), dtype=np.float32) * 64).to(torch.float8_e4m3fn)
        self.codes, self.scale = codes, (0.5 + rng.random((E, K // 128, -(-N // 128)), dtype=np.float32)) / (64 * K ** 0.5)
        w, s, _ = hq.hq_repack(self.desc, codes.view(torch.uint8).numpy(), self.scale)
        self.w, self.s = torch.from_numpy(w).cuda(), torch.from_numpy(s).cuda()

    def __call__(self, a, sa, ids, offsets, T, top_k, out, workspace):
        mode = hq.HQ_MOE_GROUPED if ids is None else hq.HQ_MOE_INDEXED
        hq.hq_moe_gemm(self.desc, mode, T, top_k, a, sa, ids, offsets, self.w, self.s, None, out, workspace, workspace.numel())


class RoutedLayer:
    def __init__(self, hidden=1024, inner=512, experts=32, top_k=4, groups=4, top_groups=2, max_tokens=512, grouped=False, seed=0):
        rng = np.random.default_rng(seed)
        self.hidden, self.inner, self.experts, self.top_k, self.max_tokens, self.grouped = hidden, inner, experts, top_k, max_tokens, grouped
        self.up, self.down = Experts(experts, 2 * inner, hidden, rng), Experts(experts, hidden, inner, rng)
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.weight = (1 + 0.1 * torch.randn(hidden, device="cuda", generator=gen)).to(torch.bfloat16)
        self.router = (torch.randn(hidden, experts, device="cuda", generator=gen) * hidden ** -0.5).to(torch.bfloat16)
        self.bias = 0.1 * torch.randn(experts, device="cuda", generator=gen)
        dt = hq.HQ_DT_BF16
        self.norm = hq.norm_desc(dt, dt)
        self.norm_codes = hq.norm_desc(dt, hq.HQ_DT_FP8_E4M3, hq.HQ_ASCALE_PER_BLOCK128_F32)
        self.route = hq.route_desc(dt, experts, top_k, sigmoid=True, groups=groups, top_groups=top_groups, group_best=2, scale=2.5)
        T, P, f8 = max_tokens, max_tokens * top_k, torch.float8_e4m3fn
        new = lambda *n, dtype=torch.bfloat16: torch.empty(n, dtype=dtype, device="cuda")  # noqa: E731
        self.y, self.logits, self.out = new(T, hidden), new(T, experts), new(T, hidden)
        self.a, self.sa = new(T, hidden, dtype=f8), new(T, hidden // 128, dtype=torch.float32)
        self.ids, self.weights = new(T, top_k, dtype=torch.int32), new(T, top_k, dtype=torch.float32)
        self.gate_up, self.answers = new(P, 2 * inner), new(P, hidden)
        self.h, self.sh = new(P, inner, dtype=f8), new(P, inner // 128, dtype=torch.float32)
        self.order, self.starts = new(P, dtype=torch.int32), new(experts + 1, dtype=torch.int32)
        self.sorted_a, self.sorted_sa = (new(P, hidden, dtype=f8), new(P, hidden // 128, dtype=torch.float32)) if grouped else (None, None)
        need = max(hq.hq_workspace_bytes(self.up.desc, T, top_k), hq.hq_workspace_bytes(self.down.desc, P, 1), 4 * P)
        self.workspace = new(need, dtype=torch.uint8)

    def admit(self, x, residual):
        """Refuses rows that the buffers do not hold, before anything is launched (the
        library is given addresses: it cannot tell)."""
        for what, t in (("x", x), ("residual", residual)):
            if (t.dim() != 2 or t.shape[1] != self.hidden or t.shape[0] != x.shape[0] or t.dtype != torch.bfloat16 or not t.is_contiguous()
                    or t.device != self.out.device):
                raise ValueError(f"{what} must be a contiguous bf16 [tokens][{self.hidden}] beside the weights")
        if not 0 < x.shape[0] <= self.max_tokens:
            raise ValueError(f"{x.shape[0]} tokens: 1 to {self.max_tokens} fit")
        return x.shape[0]

    def step(self, x, residual):
        """x: what the layer before adds [tokens][hidden]; residual takes it in (residual +=
        x).  Returns what this layer adds: rows of the layer's own buffer, until the
        next step."""
        T, k, P = self.admit(x, residual), self.top_k, x.shape[0] * self.top_k
        hq.hq_rmsnorm(self.norm, T, self.hidden, x, self.hidden, self.weight, self.y, residual=residual, residual_stride=self.hidden,
                      sum_out=residual, sum_stride=self.hidden)
        hq.hq_rmsnorm(self.norm_codes, T, self.hidden, residual, self.hidden, self.weight, self.a, self.sa)
        torch.mm(self.y[:T], self.router, out=self.logits[:T])
        hq.hq_moe_route(self.route, T, self.logits, self.experts, self.bias, self.ids, self.weights)
        if self.grouped:
            hq.hq_moe_align(T, k, self.experts, self.ids, self.starts, self.order, self.workspace, self.workspace.numel())
            hq.hq_moe_gather(hq.HQ_DT_FP8_E4M3, T, k, self.hidden, self.a, self.order, self.sorted_a)
            hq.hq_moe_gather(hq.HQ_DT_FP32, T, k, self.hidden // 128, self.sa, self.order, self.sorted_sa)
            self.up(self.sorted_a, self.sorted_sa, None, self.starts, T, k, self.gate_up, self.workspace)
        else:
            self.up(self.a, self.sa, self.ids, None, T, k, self.gate_up, self.workspace)
        hq.hq_silu_mul_quant(hq.HQ_DT_BF16, hq.HQ_DT_FP8_E4M3, hq.HQ_ASCALE_PER_BLOCK128_F32, P, self.inner, self.gate_up, self.h, self.sh)
        self.down(self.h, self.sh, None if self.grouped else self.ids, self.starts if self.grouped else None, P, 1, self.answers, self.workspace)
        hq.hq_moe_combine(hq.HQ_DT_BF16, T, k, self.hidden, self.answers, self.weights, self.out, sorted_pairs=self.order if self.grouped else None,
                          workspace=self.workspace, ws_bytes=self.workspace.numel())
        return self.out[:T]


def main():
    layer = RoutedLayer()
    gen = torch.Generator(device="cuda").manual_seed(1)
    tokens = lambda n: torch.randn(n, layer.hidden, device="cuda", generator=gen).to(torch.bfloat16)  # noqa: E731
    for i, n in enumerate([300, 5, 5, 1]):
        residual = tokens(n)
        y = layer.step(tokens(n), residual)
        torch.cuda.synchronize()
        used = layer.ids[:n].unique().numel()
        print(f"step {i}: {n} tokens on {used} of {layer.experts} experts, output rms {y.float().pow(2).mean().sqrt():.3f}, residual rms "
              f"{residual.float().pow(2).mean().sqrt():.3f}")


if __name__ == "__main__":
    main()
