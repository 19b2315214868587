"""Blocks whose largest value is a denormal: max / 448 would round to 0, and the block's
zeros to 0 / 0.  The scale is at least the smallest fp32 above 0 (no GPU)."""
import numpy as np
import pytest
import torch

import oracle

UNIT = np.float32(2.0 ** -149)
TOPS = np.arange(1, 700, dtype=np.float32)  # in units; up to 224 the quotient rounds to 0


def rows(K, block):
    """Each row's blocks hold one largest value, a half of it, its negative, and zeros."""
    x = np.zeros((len(TOPS), K // block, block), np.float32)
    x[:, :, 1], x[:, :, block // 2], x[:, :, block - 1] = TOPS[:, None] * UNIT, -np.floor(TOPS / 2)[:, None] * UNIT, -TOPS[:, None] * UNIT
    return x.reshape(len(TOPS), K)


def wanted(x, block):
    parts = x.reshape(len(x), -1, block)
    peak = np.abs(parts).max(2)
    s = np.maximum(peak / np.float32(448), UNIT)
    ratio = np.clip(parts / s[:, :, None], -448, 448)
    return torch.from_numpy(ratio.reshape(x.shape)).to(torch.float8_e4m3fn).view(torch.uint8).numpy(), s


@pytest.mark.parametrize("K,block", [(128, 128), (384, 128), (260, 260), (130, 130)])
def test_oracle_scale_stays_above_zero(K, block):
    x = rows(K, block)
    q, s = oracle.quant_act_e4m3_blocks(x, block)
    want, ws = wanted(x, block)
    assert (s > 0).all() and not ((q & 0x7F) == 0x7F).any()
    np.testing.assert_array_equal(s, ws)
    np.testing.assert_array_equal(q, want)
    assert ((q[x == 0] & 0x7F) == 0).all()  # (a zero keeps its sign)
    if block == K:
        q1, s1 = oracle.quant_act_e4m3(x)
        np.testing.assert_array_equal(q1, q)
        np.testing.assert_array_equal(s1, s[:, 0])
