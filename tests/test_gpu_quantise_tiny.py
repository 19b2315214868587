"""The quantisers on blocks whose largest value is a denormal: codes and scales are the
oracle's, and zeros stay zeros."""
import numpy as np
import pytest
import torch

import oracle
from bit_quantized_gemm_w4a16_amd import hq
from gpu_util import dev, empty, note
from test_quantise_tiny_host import rows

pytestmark = pytest.mark.gpu


# K a multiple of 4: the kernel that holds a row; others and longer ones: the one that reads it twice
@pytest.mark.parametrize("K,block", [(128, 128), (384, 128), (260, 260), (130, 130), (8196, 8196)])
def test_scales_stay_above_zero(K, block):
    note(f"quantise tiny K={K} block={block}")
    x = rows(K, block)
    M, n = len(x), K // block
    q, s = empty(M * K), empty(M * n * 4)
    want, ws = oracle.quant_act_e4m3_blocks(x, block)
    calls = [lambda: hq.hq_quantize_act_blocks(hq.HQ_DT_FP8_E4M3, M, K, block, dev(x), q, s)]
    if n == 1:
        calls.append(lambda: hq.hq_quantize_act(hq.HQ_DT_FP8_E4M3, M, K, dev(x), q, s))
    for call in calls:
        call()
        torch.cuda.synchronize()
        got, gs = q[:M * K].cpu().numpy().reshape(M, K), s[:M * n * 4].cpu().numpy().view(np.float32).reshape(M, n)
        np.testing.assert_array_equal(gs.view(np.uint32), ws.view(np.uint32))
        np.testing.assert_array_equal(got, want)
        assert (gs > 0).all() and ((got[x == 0] & 0x7F) == 0).all()
