"""The rotary table far out: 50 digits as the measure, up to the last position."""
import math
from decimal import Decimal, getcontext

import numpy as np
import pytest
import torch

from bit_quantized_gemm_w4a16_amd import hq
from gpu_util import note

pytestmark = pytest.mark.gpu

getcontext().prec = 50
TWO_PI = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582")


def exact_rows(rot, first, count, base, scaling, factor, context):
    """cos and sin of pos * f_d, the angle taken to one turn before it leaves 50 digits."""
    base, factor, context = Decimal(base), Decimal(factor), Decimal(context)
    if scaling == hq.HQ_ROPE_NTK:
        base *= factor ** (Decimal(rot) / Decimal(rot - 2))
    gain = 0.1 * math.log(factor) + 1.0 if scaling == hq.HQ_ROPE_PARTS else 1.0
    out = np.empty((count, rot))
    for d in range(rot // 2):
        f = base ** (Decimal(-2 * d) / Decimal(rot))
        if scaling == hq.HQ_ROPE_LINEAR:
            f /= factor
        if scaling == hq.HQ_ROPE_PARTS:
            g = min(max((context * f / TWO_PI - 1) / Decimal(31), Decimal(0)), Decimal(1))
            f = f * g + f / factor * (1 - g)
        turn = f / TWO_PI
        for i in range(count):
            t = turn * (first + i)
            a = float((t - t.to_integral_value()) * TWO_PI)
            out[i, d], out[i, rot // 2 + d] = math.cos(a) * gain, math.sin(a) * gain
    return out


@pytest.mark.parametrize("scaling", [hq.HQ_ROPE_NONE, hq.HQ_ROPE_LINEAR, hq.HQ_ROPE_NTK, hq.HQ_ROPE_PARTS])
@pytest.mark.parametrize("rot,first,count", [(32, 0, 40), (64, 131072 - 20, 20), (128, (1 << 24) - 5, 37), (64, (1 << 31) - 70, 70), (256, (1 << 31) - 9, 9)])
def test_no_position_loses_accuracy(scaling, rot, first, count):
    """One rounding to fp32 of a value below the gain (half of 2^-24 of it), and 2^-30 of a turn for
    all that is done in 64 bits: the same bound at every position."""
    note(f"rope far {scaling} rot={rot} first={first}")
    p = dict(base=500000.0, factor=6.5 if scaling else 1.0, context=4096.0)
    t = torch.full((count, rot), 9.0).cuda()
    hq.hq_rope_table(hq.rope_desc(rot, p["base"], scaling=scaling, factor=p["factor"], context=p["context"]), first, count, t)
    torch.cuda.synchronize()
    want = exact_rows(rot, first, count, scaling=scaling, **p)
    gain = 0.1 * math.log(p["factor"]) + 1.0 if scaling == hq.HQ_ROPE_PARTS else 1.0
    err = np.abs(t.double().cpu().numpy() - want).max()
    # (half a step of values in [1, 2) where the gain takes them there: 2^-24)
    assert err <= (2.0 ** -24 if gain > 1.0 else 2.0 ** -25) + gain * 2 * math.pi * 2.0 ** -30, err
