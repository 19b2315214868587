"""A routed layer's operators on rows at strides of their own, and on workspaces that hold an earlier call's contents."""
import numpy as np
import pytest
import torch

from bit_quantized_gemm_w4a16_amd import hq
from gpu_util import note
from layer_util import DT, NORM_DELTA, check_rows, f64, run_norm
from oracle import layer as ol
from test_gpu_norm import made, weight
from test_gpu_route import bias_of, logits_of, routed

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("form", ["same", "f8_token", "i8_token", "f8_block", "mx_f4"])
@pytest.mark.parametrize("K,M", [(384, 5), (2048, 3), (4096, 1030), (16512, 2)])
def test_norm_strides_of_each_buffer(form, K, M):
    """Wider residual and sum rows than K, each alone and together; odd ones (that alone turn the wide loads off) where
    the form takes them.  What lies between the rows of the sum stays."""
    odd = form in ("same", "f8_token", "i8_token")
    for xs, rs, ss in [(K, K + 8, K), (K, K, K + 64), (K + 16, K + 8, K + 24)] + ([(K, K + 3, K), (K, K, K + 5), (K + 8, K + 1, K + 2)] if odd else []):
        note(f"norm strides {form} M={M} K={K} {xs} {rs} {ss}")
        x, r, w = made(1, M, K, "bf16", xs), made(2, M, K, "bf16", rs), weight(3, K, "bf16")
        total = torch.full((M, ss), 7.0, dtype=torch.bfloat16, device="cuda")
        got = run_norm(form, "bf16", x, r, w, M, K, x_stride=xs, res_stride=rs, sum_out=total, sum_stride=ss)
        h, y = ol.rms_norm(f64(x)[:, :K], f64(r)[:, :K], f64(w), float(np.float32(1e-6)))
        check_rows(form, "bf16", y, NORM_DELTA, *got)
        assert (np.abs(f64(total)[:, :K] - h) <= np.abs(h) * (2.0 ** -8 + 2.0 ** -23)).all()
        assert (total[:, K:] == 7.0).all()


@pytest.mark.parametrize("E,stride", [(256, 260), (256, 512), (252, 256), (64, 68), (128, 1000), (512, 516), (1024, 1028), (4096, 4100), (256, 257), (60, 63)])
def test_route_wide_loads_of_strided_rows(E, stride):
    """Rows of whole 16 bytes inside wider ones (and rows that are not)."""
    note(f"route strided E={E} stride={stride}")
    wide = logits_of(10, 9, stride)
    wide[:, E:] = 1e9  # (not the router's)
    for bias, sigmoid in ((None, False), (bias_of(1, E), True)):
        ids, w = routed(wide, bias, 4, stride=stride, E=E, sigmoid=sigmoid)
        want, ww = ol.route(f64(wide)[:, :E], None if bias is None else f64(bias), 4, sigmoid, True)
        np.testing.assert_array_equal(ids, want)
        assert (np.abs(w - ww) <= ww * (2.0 ** -24 + 2.0 ** -43)).all()


@pytest.mark.parametrize("T,k", [(200, 8), (1025, 1), (40, 50)])
def test_combine_in_a_workspace_that_was_used(T, k):
    """More pairs than a workgroup looks through by itself: places that an earlier call left there, in range, name rows
    of other pairs now."""
    N, P = 64, T * k
    assert P > 1024
    g = torch.Generator().manual_seed(T)
    y = torch.randn(P, N, generator=g).to(torch.bfloat16).cuda()
    w = (torch.rand(T, k, generator=g) + 0.1).cuda()
    out = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(P, dtype=torch.int32, device="cuda")

    def call(order):
        hq.hq_moe_combine(hq.HQ_DT_BF16, T, k, N, y, w, out, sorted_pairs=order.cuda(), workspace=ws, ws_bytes=4 * P)
        torch.cuda.synchronize()

    for i in range(4):
        order = torch.randperm(P, generator=g).to(torch.int32)
        if i == 0:
            call(torch.randperm(P, generator=g).to(torch.int32))  # every place of another order
        else:
            ws.fill_((0, 0, int(order[7]), P - 1)[i])
        gone = torch.randperm(P, generator=g)[:P // 4]
        order[gone[::2]] = -1  # a quarter of the rows belong to no pair any more,
        order[gone[1::2]] = P + 3
        note(f"combine used workspace T={T} k={k} {i}")
        call(order)
        o, at = order.numpy(), np.full(P, -1, np.int64)
        ok = (o >= 0) & (o < P)
        at[o[ok]] = np.nonzero(ok)[0]
        want, S = ol.combine(f64(y), f64(w), None, at.reshape(T, k))
        assert (np.abs(f64(out) - want) <= np.abs(want) * 2.0 ** -8 + S * (2 * k + 2) * 2.0 ** -24).all()
