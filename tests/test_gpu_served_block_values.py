"""Each operator of the example block against 64 bits on what the block itself holds
before it, so that a bound is that operator's own roundings alone: the cache that
the rotation wrote, the attention over that cache, both projections."""
import os
import sys

import numpy as np
import pytest
import torch

import oracle
from gpu_util import GATE, note
from kv_util import TINY, U
from oracle import kv as okv

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def f64(t):
    return t.double().cpu().numpy()


def weights(b, seed=0):
    """Codes and scales of the block's two layers, as it draws them."""
    rng = np.random.default_rng(seed)
    out = []
    for layer in (b.qkv, b.proj):
        codes = rng.integers(0, 1 << 32, (layer.K // 8, layer.N), dtype=np.uint32)
        out.append((codes, torch.full((layer.K // 128, layer.N), 0.25 / layer.K ** 0.5, dtype=torch.bfloat16).view(torch.int16).numpy()))
    return out


def product(x, layer, w):
    return oracle.gemm_wna16(x.view(torch.int16).cpu().numpy(), *w, None, N=layer.N, K=layer.K, G=128, a_bf16=True, w_signed=True)


def near(got, want):
    return (np.abs(got - want) <= GATE * np.maximum(np.abs(want), np.sqrt(np.mean(want * want)))).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_each_operator_on_what_it_is_given(fp8):
    from served_block import ServedBlock
    note(f"served block values fp8={fp8}")
    b = ServedBlock(fp8_cache=fp8)
    D, Hq, Hk, P = b.head_dim, b.q_heads, b.kv_heads, b.block
    cache = "fp8" if fp8 else "bf16"
    scale = float(np.float32(0.05)) if fp8 else 1.0
    table = f64(b.table)
    w_qkv, w_out = weights(b)
    gen = torch.Generator(device="cuda").manual_seed(3)
    lens, pages = [0] * 3, None

    def held(side, ids, n):  # the first n keys of those pages, as values
        store = f64((b.k_cache, b.v_cache)[side]).reshape(-1, Hk, D) * scale
        return store[[int(ids[i // P]) * P + i % P for i in range(n)]]

    def wrote(rows, pos, ids, first, side):
        """The new tokens' keys (values) in the cache are the projected rows, rotated (as they are) and rounded once."""
        x = rows[:, Hq + side * Hk:Hq + (side + 1) * Hk]
        want = okv.rope(x, table[pos], D, False) if side == 0 else x
        if fp8:
            want = np.clip(want, -448 * scale, 448 * scale)
        got = held(side, ids, first + len(pos))[first:]
        # two products and their sum in 32 bits (cos and sin times the gain are below 1.2), the division by the scale
        tol = U[cache] * np.abs(want) * 1.01 + 2.0 ** -20 * np.abs(x).max(initial=0.0) + TINY[cache] * scale
        assert (np.abs(got - want) <= tol).all(), float((np.abs(got - want) / tol).max())

    def step(new, call):
        T = sum(new)
        x = torch.randn(T, b.qkv.K, device="cuda", generator=gen).to(torch.bfloat16)
        prefix = b.prefix_len
        y = call(x)
        torch.cuda.synchronize()
        rows = f64(b.x_qkv[:T])
        assert near(rows, product(x, b.qkv, w_qkv))
        rows = rows.reshape(T, Hq + 2 * Hk, D)
        cu = np.concatenate([[0], np.cumsum(new)])
        ids = b.prefix_table[None] if pages is None else b.blocks  # (the shared prompt's pages have become the prefix's)
        ids = ids.cpu().numpy()
        pos = np.concatenate([prefix + lens[r] + np.arange(n) for r, n in enumerate(new)])
        for r, n in enumerate(new):
            for side in range(2):
                wrote(rows[cu[r]:cu[r + 1]], pos[cu[r]:cu[r + 1]], ids[r], lens[r], side)
            lens[r] += n
        q = f64(b.q[:T]).reshape(T, Hq, D)
        want = okv.rope(rows[:, :Hq], table[pos], D, False)
        assert (np.abs(q - want) <= U["bf16"] * np.abs(want) * 1.01 + 2.0 ** -20 * np.abs(rows[:, :Hq]).max() + TINY["bf16"]).all()
        shared = f64(b.prefix_table) if prefix else []
        k, v = ([np.concatenate([held(s, shared, prefix), held(s, ids[r], lens[r])]) for r in range(len(new))] for s in range(2))
        out, lse, (mass, qk, seen, vmax) = okv.attention(q, lambda r: k[r], lambda r: v[r], prefix, lens[:len(new)], cu, float(np.float32(D ** -0.5)))
        u = U["bf16"]
        es = 2.0 ** -24 * (D + 8) * qk + 2.0 ** -22 * (1 + np.abs(lse))
        tol = ((u + 2 * es + 2.0 ** -21 + (seen + 64) * 2.0 ** -24)[..., None] * mass + (seen * TINY["bf16"] * vmax)[..., None] + u * np.abs(out)
               + TINY["bf16"]) * (1 + 2.0 ** -6)
        err = np.abs(f64(b.heads[:T]).reshape(T, Hq, D) - out)
        assert (err <= tol).all(), float((err / tol).max())
        assert near(f64(y), product(b.heads[:T], b.proj, w_out))

    step([150], b.share_prefix)
    lens, pages = [0] * 3, b.blocks
    for new in ([20, 1, 70], [1, 1, 1], [1, 30, 0], [1, 1, 1]):
        step(new, lambda x: b.step(x, new))  # noqa: B023
        assert b.lens[:3] == lens == b.kv_lens[:3].tolist()
