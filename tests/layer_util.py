"""Shared by the tests of a routed layer's operators: inputs on both sides, and the
checks of an output against the 64-bit definitions with bounds that count roundings.

An fp32 value here is within DELTA of the definition's, relative to it:
 - norm: the squares (one rounding each) are summed over at most 64 values of a
   thread, 6 steps of a wave and 16 waves, all of one sign: 87 roundings of 2^-24, of
   which the root takes half; x + r, mean + eps, the division by K, root, reciprocal,
   weight + offset and two products: 8 more.  52 * 2^-24 < 2^-18.
 - SwiGLU: expf to 2 units in the last place (4 * 2^-24), 1 + e, two products, one
   quotient: 9 * 2^-24 < 2^-20.
A scale adds one division, a code's ratio another.
"""
from __future__ import annotations

import numpy as np
import torch

from bit_quantized_gemm_w4a16_amd import hq
from oracle import layer as ol

NORM_DELTA, SILU_DELTA = 2.0 ** -18, 2.0 ** -20
DT = {"bf16": (hq.HQ_DT_BF16, torch.bfloat16, 2.0 ** -8), "fp16": (hq.HQ_DT_FP16, torch.float16, 2.0 ** -11), "fp32": (hq.HQ_DT_FP32, torch.float32, 2.0 ** -24)}
# name: output dtype (None: that of the input), scales, block (0: the row), largest code
FORMS = {"same": (None, hq.HQ_ASCALE_NONE, 0, 0), "f8_token": (hq.HQ_DT_FP8_E4M3, hq.HQ_ASCALE_PER_TOKEN_F32, 0, 448.0),
         "i8_token": (hq.HQ_DT_INT8, hq.HQ_ASCALE_PER_TOKEN_F32, 0, 127.0), "f8_block": (hq.HQ_DT_FP8_E4M3, hq.HQ_ASCALE_PER_BLOCK128_F32, 128, 448.0),
         "mx_f8": (hq.HQ_DT_FP8_E4M3, hq.HQ_ASCALE_MX_E8M0, 32, 448.0), "mx_f4": (hq.HQ_DT_FP4_E2M1, hq.HQ_ASCALE_MX_E8M0, 32, 6.0)}
E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])


def f64(t):
    return t.detach().double().cpu().numpy()


def outputs(form, dtype, M, K, guard=64):
    """Output and scale buffers of `form`, filled with a pattern and longer than needed by `guard` bytes."""
    each = {"same": 2 * K, "mx_f4": K // 2}.get(form, K)
    per = {"same": 0, "f8_token": 4, "i8_token": 4, "f8_block": K // 128 * 4}.get(form, K // 32)
    out = torch.full((M * each + guard,), 0x5A, dtype=torch.uint8, device="cuda")
    scale = torch.full((M * per + guard,), 0x5A, dtype=torch.uint8, device="cuda") if per else None
    return out, scale, M * each, M * per


def check_rows(form, dtype, y, delta, out, scale, nout, nscale):
    """The written bytes against y [M][K] in 64 bits; nothing behind them."""
    M, K = y.shape
    for buf, n in ((out, nout), (scale, nscale)):
        if buf is not None:
            assert (buf[n:] == 0x5A).all(), "bytes behind the output were written"
    raw = out[:nout]
    code, tdt, half = DT[dtype]
    if form == "same":
        got = f64(raw.view(tdt).view(M, K))
        tiny = 2.0 ** -25 if dtype == "fp16" else 0.0
        assert (np.abs(got - y) <= np.abs(y) * (half + delta) * (1 + 2.0 ** -10) + tiny).all(), np.abs(got - y).max()
        return got
    _, _, block, top = FORMS[form]
    block = block or K
    if form in ("f8_token", "i8_token", "f8_block"):
        s = f64(scale[:nscale].view(torch.float32).view(M, K // block))
        want = ol.scales(y, block, top)
        assert (np.abs(s - want) <= want * (delta + 2.0 ** -23)).all(), np.abs(s / want - 1).max()
        r = y / np.repeat(s, block, 1)
        got = f64(raw.view(torch.int8 if form == "i8_token" else torch.float8_e4m3fn).view(M, K))
        step = 1.0 if form == "i8_token" else ol.step_e4m3(np.abs(r) * (1 + 2 * delta))
        assert (np.abs(got - r) <= step / 2 + np.abs(r) * 2 * delta).all(), np.abs(got - r).max()
        return got * np.repeat(s, block, 1)
    e = scale[:nscale].cpu().numpy().astype(np.int64).reshape(M, K // 32)
    emax = 8 if form == "mx_f8" else 2
    peak = np.abs(y).reshape(M, -1, 32).max(2)
    lo, hi = (np.where(peak > 0, np.maximum(np.frexp(peak * (1 + d))[1] - 1 - emax + 127, 0), 0) for d in (-delta, delta))
    assert ((e >= lo) & (e <= hi)).all()
    r = y * np.exp2(127.0 - np.repeat(e, 32, 1))
    if form == "mx_f8":
        got, step = f64(raw.view(torch.float8_e4m3fn).view(M, K)), ol.step_e4m3
    else:
        b = raw.cpu().numpy().reshape(M, K // 2)
        got, step = E2M1[np.stack([b & 15, b >> 4], 2).reshape(M, K)], ol.step_e2m1
    r = np.clip(r, -top, top)
    assert (np.abs(got - r) <= step(np.abs(r) * (1 + 2 * delta)) / 2 + np.abs(r) * 2 * delta).all()
    return got * np.exp2(np.repeat(e, 32, 1) - 127.0)


def run_norm(form, dtype, x, res, w, M, K, *, eps=1e-6, offset=0.0, x_stride=None, res_stride=None, sum_out=None, sum_stride=None, stream=None):
    code = DT[dtype][0]
    odt, kind, _, _ = FORMS[form]
    out, scale, nout, nscale = outputs(form, dtype, M, K)
    desc = hq.norm_desc(code, odt or code, kind, eps=eps, weight_dtype=hq.HQ_DT_FP32 if w.dtype == torch.float32 else code, weight_offset=offset)
    hq.hq_rmsnorm(desc, M, K, x, x_stride or K, w, out, scale, residual=res, residual_stride=res_stride or K, sum_out=sum_out,
                  sum_stride=sum_stride or K, stream=stream)
    return out, scale, nout, nscale
