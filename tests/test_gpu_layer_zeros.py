"""Zeros of either sign and values that round to zero: the norm's codes are the quantisers', byte for byte."""
import pytest
import torch

from bit_quantized_gemm_w4a16_amd import hq
from gpu_util import note
from layer_util import outputs, run_norm

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K", [256, 2048, 8192])
@pytest.mark.parametrize("form", ["f8_token", "f8_block", "mx_f8", "mx_f4"])
def test_signs_of_zeros_are_the_quantisers(form, K):
    """x of ones of both signs and eps 0: y is x times the weights, of which half are zeros or next to nothing."""
    note(f"norm signed zeros {form} K={K}")
    M = 4
    g = torch.Generator().manual_seed(K)
    x = torch.where(torch.rand(M, K, generator=g) < 0.5, -1.0, 1.0).to(torch.bfloat16).cuda()
    w = torch.exp2(torch.randint(-6, 6, (K,), generator=g).float())
    w[torch.randperm(K, generator=g)[:K // 4]] = 0.0
    w[torch.randperm(K, generator=g)[:K // 4]] *= 2.0 ** -40
    y = (x.float() * w.cuda()).contiguous()
    got = run_norm(form, "bf16", x, None, w.cuda(), M, K, eps=0.0)
    q, s, _, _ = outputs(form, "bf16", M, K)
    f8, f4 = hq.HQ_DT_FP8_E4M3, hq.HQ_DT_FP4_E2M1
    {"f8_token": lambda: hq.hq_quantize_act(f8, M, K, y, q, s), "f8_block": lambda: hq.hq_quantize_act_blocks(f8, M, K, 128, y, q, s),
     "mx_f8": lambda: hq.hq_quantize_act_mx(f8, M, K, y, q, s), "mx_f4": lambda: hq.hq_quantize_act_mx(f4, M, K, y, q, s)}[form]()
    torch.cuda.synchronize()
    assert torch.equal(got[0], q) and torch.equal(got[1], s)
