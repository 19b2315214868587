"""The example block: its steps on a paged cache give what one pass over each whole
sequence gives, up to the roundings on the way (attention outputs compared, with
the oracle of the attention on the block's own projected rows)."""
import os
import sys

import numpy as np
import pytest
import torch

from gpu_util import note
from kv_util import TINY, U
from oracle import kv as okv

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True])
def test_steps_match_whole_sequences(fp8):
    from served_block import ServedBlock
    note(f"served block fp8={fp8}")
    b = ServedBlock(fp8_cache=fp8)
    gen = torch.Generator(device="cuda").manual_seed(2)
    table = b.table.double().cpu().numpy()
    D, Hq, Hk = b.head_dim, b.q_heads, b.kv_heads

    def rows(n):  # the projected rows of n tokens (the example's own buffer), 64 bits
        return b.x_qkv[:n].double().cpu().numpy().reshape(n, Hq + 2 * Hk, D)

    def rotated(h, pos, rnd):
        q, k, v = h[:, :Hq], h[:, Hq:Hq + Hk], h[:, Hq + Hk:]
        return rnd(okv.rope(q, table[pos], D, False)), okv.rope(k, table[pos], D, False), v

    def rnd(x):
        return torch.from_numpy(x).to(torch.bfloat16).double().numpy()

    def stored(x):  # as the cache holds it
        if not fp8:
            return rnd(x)
        return (torch.from_numpy(x / 0.05).float().clamp(-448, 448).to(torch.float8_e4m3fn).double() * float(np.float32(0.05))).numpy()

    x = torch.randn(150, b.qkv.K, device="cuda", generator=gen).to(torch.bfloat16)
    b.share_prefix(x)
    _, k, v = rotated(rows(150), np.arange(150), rnd)
    pk, pv = stored(k), stored(v)
    held = [(np.zeros((0, Hk, D)), np.zeros((0, Hk, D))) for _ in range(3)]
    for new in ([20, 1, 70], [1, 1, 1], [1, 30, 0], [1, 1, 1]):
        T = sum(new)
        y = b.step(torch.randn(T, b.qkv.K, device="cuda", generator=gen).to(torch.bfloat16), new)
        torch.cuda.synchronize()
        pos = np.concatenate([150 + len(held[r][0]) + np.arange(n) for r, n in enumerate(new)])
        q, k, v = rotated(rows(T), pos, rnd)
        at = 0
        for r, n in enumerate(new):
            held[r] = (np.concatenate([held[r][0], stored(k[at:at + n])]), np.concatenate([held[r][1], stored(v[at:at + n])]))
            at += n
        assert b.kv_lens[:3].tolist() == [len(h[0]) for h in held] == b.lens[:3]
        out, lse, (mass, qk, seen, vmax) = okv.attention(q, lambda r: np.concatenate([pk, held[r][0]]), lambda r: np.concatenate([pv, held[r][1]]),
                                                         150, [len(h[0]) for h in held], np.concatenate([[0], np.cumsum(new)]), float(np.float32(D ** -0.5)))
        got = b.heads[:T].double().cpu().numpy().reshape(T, Hq, D)
        # weights and the output are rounded to bf16; a rotated element whose fp32 value lies next
        # to a rounding boundary may be held as the neighbour, one step off: of q and k that moves
        # a score by at most u |q||k| for one such element (few are), of v the output by u |v|
        u, uc = U["bf16"], U["fp8"] if fp8 else U["bf16"]
        tol = (2 * u + 2.0 ** -16 * (1 + qk[..., None])) * mass + 2 * uc * vmax[..., None] / np.sqrt(seen[..., None]) + u * np.abs(out) + TINY["bf16"]
        assert (np.abs(got - out) <= tol).all(), float((np.abs(got - out) / tol).max())
        assert torch.isfinite(y.float()).all() and y.shape == (T, b.proj.N)


def test_main_runs(capsys):
    import served_block
    note("served block main")
    served_block.main()
    assert "step 3" in capsys.readouterr().out
