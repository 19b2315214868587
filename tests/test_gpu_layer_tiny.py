"""Norm and SwiGLU where a block's largest value is so small a denormal that its quotient by
the largest code rounds to 0: the scale stays above 0, and zeros stay zeros."""
import numpy as np
import pytest
import torch

from bit_quantized_gemm_w4a16_amd import hq
from gpu_util import note
from layer_util import DT, FORMS, f64, outputs, run_norm
from oracle import layer as ol
from test_quantise_tiny_host import UNIT

pytestmark = pytest.mark.gpu
QUANTISED = ["f8_token", "i8_token", "f8_block"]


def opened(form, out, scale, n, ns, M, K):
    codes = f64(out[:n].view(torch.int8 if form == "i8_token" else torch.float8_e4m3fn)).reshape(M, K)
    return codes, scale[:ns].view(torch.float32).cpu().numpy().reshape(M, -1)


@pytest.mark.parametrize("form,K", [(f, k) for f in QUANTISED for k in (128, 640, 4096, 8192, 16512)] + [(f, k) for f in QUANTISED[:2] for k in (130, 4001)])
def test_norm_of_ones_times_tiny_weights(form, K):
    """x of ones and eps 0 make y the weights themselves: whole units of 2^-149, beside zeros."""
    top = FORMS[form][3]
    for units in (1, 2, 31, 63, 64, 65, 127, 128, 223, 224, 225, 447, 448, 671):
        note(f"norm tiny {form} K={K} units={units}")
        w = np.zeros(K, np.float32)
        w[1::128], w[70::128], w[100::128] = units * UNIT, -(units // 2) * UNIT, -units * UNIT
        x = torch.ones(2, K, dtype=torch.bfloat16, device="cuda")
        got = run_norm(form, "bf16", x, None, torch.from_numpy(w).cuda(), 2, K, eps=0.0)
        torch.cuda.synchronize()
        codes, s = opened(form, *got, 2, K)
        ws = max(np.float32(units) * UNIT / np.float32(top), UNIT)
        assert (s == ws).all(), (s, ws)
        ratio = np.clip(w / ws, -top, top)
        want = np.rint(ratio) if form == "i8_token" else f64(torch.from_numpy(ratio).to(torch.float8_e4m3fn))
        np.testing.assert_array_equal(codes, np.broadcast_to(want, codes.shape))


@pytest.mark.parametrize("form", QUANTISED)
@pytest.mark.parametrize("rows", [3, 1030])
def test_swiglu_products_of_few_units(form, rows):
    """silu(-20) times 2^-125 and its multiples: 0.7 units each, beside zeros."""
    I = 256
    note(f"swiglu tiny {form} rows={rows}")
    gu = torch.zeros(rows, 2 * I)
    gu[:, :I] = -20.0
    gu[:, I + 3::64] = (1 + torch.arange(rows) % 200)[:, None] * 2.0 ** -125
    gu = gu.to(torch.bfloat16)
    y = ol.silu_mul(f64(gu))
    odt, kind, block, top = FORMS[form]
    out = outputs(form, "bf16", rows, I)
    hq.hq_silu_mul_quant(DT["bf16"][0], odt, kind, rows, I, gu.cuda(), out[0], out[1])
    torch.cuda.synchronize()
    codes, s = opened(form, *out, rows, I)
    assert (s > 0).all() and np.isfinite(codes).all()
    assert (codes[y == 0] == 0).all() and (codes[:, 3::64][np.abs(y[:, 3::64]) > UNIT] < 0).all()
    # the scale is within a unit of the largest value's quotient: y is a denormal, rounded to a unit
    peak = np.abs(y).reshape(rows, -1, block or I).max(2)
    assert (np.abs(s - np.maximum(peak / top, UNIT)) <= UNIT).all()
