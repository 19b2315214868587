"""Launch plans of the attention over the whole range of sizes that its checks let
through (host only): a plan or a refusal for each, with a workspace that holds the
plan's parts."""
import itertools
import re

import pytest

from bit_quantized_gemm_w4a16_amd import hq


def ask(B, T, prefix, max_new, max_kv, total, q_heads, kv_heads, dim, fp8=False):
    """(launches, workspace bytes), or None where the library refuses."""
    kv = hq.kv_desc(hq.HQ_DT_FP8_E4M3 if fp8 else hq.HQ_DT_BF16, 64, 16, kv_heads, dim)
    d = hq.attn_desc(hq.HQ_DT_BF16, q_heads, max_new, max_kv, 0.125, total_kv=total)
    try:
        return hq.hq_attn_plan(d, kv, B, T, prefix), hq.hq_attn_workspace_bytes(d, kv, B, T, prefix)
    except hq.HQError as e:
        assert e.status == hq.HQ_ERR_UNSUPPORTED
        return None


@pytest.mark.parametrize("q_heads,kv_heads,dim", [(1, 1, 16), (8, 8, 64), (64, 8, 128), (4096, 1, 256), (1024, 1024, 256), (4096, 1024, 128)])
@pytest.mark.parametrize("B", [1, 2, 513, 4096, 1 << 20])
def test_every_size_is_planned_or_refused(B, q_heads, kv_heads, dim):
    for per, prefix, max_kv, loose, fp8 in itertools.product((1, 5, 3000), (0, 1, 4097, 1 << 29), (0, 1, 5000, 1 << 29), (0, 1), (False, True)):
        T = min(B * per, 1 << 23, ((1 << 30) - 1) // q_heads)  # (requests without a new token among them)
        got = ask(B, T, prefix, per, max_kv, 0 if loose else B * max(max_kv // 3, 1), q_heads, kv_heads, dim, fp8)
        if got is None:
            continue
        (main, *join), need = got
        n = {k: int(v) for k, v in re.findall(r"(\w+)=(\d+)", main)}
        parts = n["prefix"] + max(n["few"], n["many"])
        assert 1 <= n["grid"] < 1 << 24 and 1 <= n["few"] <= 256 and n["prefix"] <= 256 and n["many"] <= 256
        assert n["prefix"] == 0 if n["joint"] or not prefix else n["prefix"] > 0
        assert bool(join) == (parts > 1)
        rows = T * q_heads
        assert need == 0 if not join else need >= parts * rows * (dim + 2) * 4 + T * 4
        assert len(join) <= 1 and (not join or f"parts={parts}" in join[0])
