"""SwiGLU of gates so far below 0 that e^-|g| is a denormal while the result is not yet 0.

An fp32 value is within SILU_DELTA of the definition's, relative to it: the hardware's exp2
and reciprocal one unit in the last place each (2^-23), the power's argument 2^-24 of e^x,
1 + e, the quotient's and the two other products one rounding each: 2^-23 (1 + 1 + 5/2) <
2^-20.  Below the smallest normal number a value is off by half a unit of 2^-149 more, and
silu's part of that is multiplied by up."""
import numpy as np
import pytest
import torch

from bit_quantized_gemm_w4a16_amd import hq
from gpu_util import note
from layer_util import DT, FORMS, SILU_DELTA, check_rows, f64, outputs
from oracle import layer as ol

pytestmark = pytest.mark.gpu


def swiglu(form, gu, rows, I):
    odt, kind, _, _ = FORMS[form]
    out = outputs(form, "bf16", rows, I)
    hq.hq_silu_mul_quant(DT["bf16"][0], odt, kind, rows, I, gu, out[0], out[1])
    torch.cuda.synchronize()
    return out


def gates(rows, I, lo, hi):
    """One gate for each block of 128."""
    return torch.linspace(lo, hi, rows * I // 128).view(rows, -1).repeat_interleave(128, 1)


@pytest.mark.parametrize("form", ["f8_block", "f8_token", "mx_f8"])
@pytest.mark.parametrize("rows,I", [(7, 1280), (64, 128), (1030, 2048)])
def test_where_the_result_is_a_normal_number(form, rows, I):
    """-91.5 to -86: silu is above 2^-126.  (up of some 2^20, so that the scale is a normal number too)"""
    note(f"swiglu far {form} {rows} x {I}")
    u = torch.randn(rows, I, generator=torch.Generator().manual_seed(I)) * 2.0 ** 20
    gu = torch.cat([gates(rows, I, -91.5, -86.0), u], 1).to(torch.bfloat16)
    y = ol.silu_mul(f64(gu))
    assert (np.abs(y).max(1) > 0).all()
    check_rows(form, "bf16", y, SILU_DELTA, *swiglu(form, gu.cuda(), rows, I))


def test_down_to_nothing():
    """-150 to -84, past where silu rounds to 0 (some -108): scales as the definition's but for the denormal's rounding."""
    note("swiglu far to nothing")
    rows, I = 64, 1280
    u = torch.randn(rows, I, generator=torch.Generator().manual_seed(1)) * 2.0 ** 40
    gu = torch.cat([gates(rows, I, -150.0, -84.0), u], 1).to(torch.bfloat16)
    y, up = ol.silu_mul(f64(gu)), np.abs(f64(gu)[:, I:])
    out, scale, n, ns = swiglu("f8_block", gu.cuda(), rows, I)
    s = f64(scale[:ns].view(torch.float32)).reshape(rows, -1)
    peak, most = (np.abs(v).reshape(rows, -1, 128).max(2) for v in (y, up))
    got = f64(out[:n].view(torch.float8_e4m3fn)).reshape(rows, -1, 128)
    gone = np.abs(got).max(2) == 0
    # silu is off by half a unit and its relative error; times up, over 448
    far = (peak * SILU_DELTA + most * 2.0 ** -150) / 448 * (1 + 2.0 ** -20)
    assert (np.abs(s - peak / 448) <= far + 2.0 ** -149)[~gone].all()
    assert (peak[gone] <= most[gone] * 2.0 ** -149).all() and (s[gone] == 1).all()
    assert gone.any() and not gone[-8:].any()


def test_as_the_product_in_16_bits():
    """The same rows through hq_silu_mul: its 16 bits, within the codes' step."""
    note("swiglu far against hq_silu_mul")
    rows, I = 16, 256
    u = torch.randn(rows, I, generator=torch.Generator().manual_seed(2)) * 2.0 ** 20
    gu = torch.cat([gates(rows, I, -91.0, -87.4), u], 1).to(torch.bfloat16).cuda()
    want = torch.empty(rows, I, dtype=torch.bfloat16, device="cuda")
    hq.hq_silu_mul(hq.HQ_DT_BF16, rows, I, gu, want)
    out, scale, n, ns = swiglu("f8_block", gu, rows, I)
    s = np.repeat(f64(scale[:ns].view(torch.float32)).reshape(rows, -1), 128, 1)
    got = f64(out[:n].view(torch.float8_e4m3fn)).reshape(rows, I)
    w = f64(want) / s
    # half a step of E4M3, a bf16 rounding, and what the two ways to e^x differ by
    assert (np.abs(got - w) <= ol.step_e4m3(np.abs(w) * 1.01) / 2 + np.abs(w) * (2.0 ** -8 + 2.0 ** -18)).all()
    assert np.abs(got).max() == 448


def test_limits():
    note("swiglu limits")
    gu = torch.ones(6, 2 * 128)
    gu[:, 5] = torch.tensor([-torch.inf, -3e38, -150.0, -151.0, -0.0, torch.nan])
    out, scale, n, ns = swiglu("f8_token", gu.to(torch.bfloat16).cuda(), 6, 128)
    codes = out[:n].view(6, 128).cpu()
    assert (codes[:, 5] == torch.tensor([0x7F, 0x80, 0x80, 0x80, 0x80, 0x7F], dtype=torch.uint8)).all()
    assert (codes[:, :5] == 0x7E).all() and (codes[:, 6:] == 0x7E).all()
