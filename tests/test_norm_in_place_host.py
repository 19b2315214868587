"""The norm's sum in place of x or the residual: at the same stride, or refused (no GPU).  At another
stride a row's sum would be written over rows that are not read yet."""
import pytest

from bit_quantized_gemm_w4a16_amd import hq
from test_layer_host import A, ALIGN, BAD, NORM, norm, status_of

B, C = A + (1 << 20), A + (2 << 20)


@pytest.mark.parametrize("change", [dict(sum_out=A, sum_stride=264), dict(sum_out=A, x_stride=264), dict(sum_out=A, x_stride=264, sum_stride=272),
                                    dict(sum_out=B, sum_stride=264), dict(sum_out=B, residual_stride=512), dict(x=B, sum_out=B, x_stride=264)])
def test_another_stride_is_refused(change):
    call = {**NORM, "residual": B, "out": C, "out_scale": C, **change}
    assert status_of(hq.hq_rmsnorm, norm(), **call) == BAD
    assert b"sum_out" in hq.lib().hq_last_error()


@pytest.mark.parametrize("change", [dict(sum_out=A), dict(sum_out=B), dict(sum_out=A, x_stride=264, sum_stride=264), dict(sum_out=C, sum_stride=264),
                                    dict(sum_out=A, sum_stride=264, M=1), dict(sum_out=B, residual_stride=512, sum_stride=512),
                                    dict(sum_out=None, sum_stride=300), dict(sum_out=A, residual=None, residual_stride=0)])
def test_the_same_stride_and_one_row_are_taken(change):
    """(past this check: the weight's address is refused)"""
    call = {**NORM, "residual": B, "out": C, "out_scale": C, "weight": A + 4, **change}
    assert status_of(hq.hq_rmsnorm, norm(), **call) == ALIGN
