"""Host side of the paged-cache operators (no GPU): refusals before any HIP call,
workspace sizes and launch plans, and pins of the 64-bit definitions."""
import math

import numpy as np
import pytest

from bit_quantized_gemm_w4a16_amd import hq
from oracle import kv as okv


def status_of(fn, *args, **kw):
    try:
        fn(*args, **kw)
    except hq.HQError as e:
        return e.status
    return hq.HQ_OK


A = 1 << 20                       # stands for an aligned device pointer; no call below gets as far as using it
KV = lambda **k: _with(hq.kv_desc(hq.HQ_DT_BF16, 64, 16, 2, 64), k)  # noqa: E731
ROPE = lambda **k: _with(hq.rope_desc(64), k)  # noqa: E731
ATT = lambda **k: _with(hq.attn_desc(hq.HQ_DT_BF16, 8, 1, 100, 0.125), k)  # noqa: E731


def _with(d, fields):
    for k, v in fields.items():
        setattr(d, k, v)
    return d


# ---------------------------------------------------------------------------
# slot maps
# ---------------------------------------------------------------------------

SLOTS = dict(block_size=16, B=2, T_cap=4, cached_lens=A, new_lens=A, free_blocks=A, n_free=4, block_table=A, max_blocks=8, cu_new=A, kv_lens=A,
             positions=A, slots=A, taken=A, first_pos=0, stream=0)


@pytest.mark.parametrize("change,want", [
    (dict(block_size=0), hq.HQ_ERR_INVALID_ARG), (dict(block_size=65537), hq.HQ_ERR_INVALID_ARG), (dict(B=-1), hq.HQ_ERR_INVALID_ARG),
    (dict(B=4097), hq.HQ_ERR_UNSUPPORTED), (dict(T_cap=-1), hq.HQ_ERR_INVALID_ARG), (dict(max_blocks=-1), hq.HQ_ERR_INVALID_ARG),
    (dict(n_free=-1), hq.HQ_ERR_INVALID_ARG), (dict(first_pos=-1), hq.HQ_ERR_INVALID_ARG), (dict(cached_lens=None), hq.HQ_ERR_INVALID_ARG),
    (dict(new_lens=None), hq.HQ_ERR_INVALID_ARG), (dict(free_blocks=None), hq.HQ_ERR_INVALID_ARG), (dict(block_table=None), hq.HQ_ERR_INVALID_ARG),
    (dict(cu_new=None), hq.HQ_ERR_INVALID_ARG), (dict(kv_lens=None), hq.HQ_ERR_INVALID_ARG), (dict(positions=None), hq.HQ_ERR_INVALID_ARG),
    (dict(slots=None), hq.HQ_ERR_INVALID_ARG), (dict(taken=None), hq.HQ_ERR_INVALID_ARG), (dict(slots=A + 4), hq.HQ_ERR_ALIGNMENT),
    (dict(cached_lens=A + 2), hq.HQ_ERR_ALIGNMENT), (dict(block_table=A + 1), hq.HQ_ERR_ALIGNMENT)])
def test_slots_refusals(change, want):
    a = {**SLOTS, **change}
    assert status_of(hq.hq_kv_slots, **a) == want
    assert hq.lib().hq_last_error()


# ---------------------------------------------------------------------------
# descriptors and refusals of the rotation
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("change,want", [
    (dict(abi_version=9), hq.HQ_ERR_ABI), (dict(rot_dim=8), hq.HQ_ERR_UNSUPPORTED), (dict(rot_dim=40), hq.HQ_ERR_UNSUPPORTED),
    (dict(rot_dim=272), hq.HQ_ERR_UNSUPPORTED), (dict(layout=0), hq.HQ_ERR_INVALID_ARG), (dict(scaling=4), hq.HQ_ERR_INVALID_ARG),
    (dict(base=1.0), hq.HQ_ERR_INVALID_ARG), (dict(base=math.nan), hq.HQ_ERR_INVALID_ARG), (dict(scaling=1, factor=0.5), hq.HQ_ERR_INVALID_ARG),
    (dict(scaling=3, factor=2.0, context=0.0), hq.HQ_ERR_INVALID_ARG), (dict(scaling=3, factor=2.0, context=4096.0, slow=32.0), hq.HQ_ERR_INVALID_ARG),
    (dict(attn_factor=1.0), hq.HQ_ERR_INVALID_ARG), (dict(scaling=3, factor=2.0, context=4096.0, attn_factor=-1.0), hq.HQ_ERR_INVALID_ARG)])
def test_rope_descriptor_refusals(change, want):
    assert status_of(hq.hq_rope_table, ROPE(**change), 0, 4, A, stream=0) == want


def test_rope_table_refusals():
    assert status_of(hq.hq_rope_table, ROPE(), -1, 4, A, stream=0) == hq.HQ_ERR_INVALID_ARG
    assert status_of(hq.hq_rope_table, ROPE(), (1 << 31) - 3, 4, A, stream=0) == hq.HQ_ERR_INVALID_ARG
    assert status_of(hq.hq_rope_table, ROPE(), 0, 4, None, stream=0) == hq.HQ_ERR_INVALID_ARG
    assert status_of(hq.hq_rope_table, ROPE(), 0, 4, A + 4, stream=0) == hq.HQ_ERR_ALIGNMENT
    assert status_of(hq.hq_rope_table, ROPE(), 0, 0, None, stream=0) == hq.HQ_OK


RK = dict(rope=None, kv=None, dtype=hq.HQ_DT_BF16, T=4, q_heads=8, q=A, q_stride=512, k=A, k_stride=128, v=A, v_stride=128, positions=A, table=A,
          table_rows=10, slots=A, q_out=A + 4096, q_out_stride=512, k_cache=A, v_cache=A, k_scale=None, v_scale=None, stream=0)


@pytest.mark.parametrize("change,want", [
    (dict(dtype=hq.HQ_DT_FP32), hq.HQ_ERR_UNSUPPORTED), (dict(dtype=hq.HQ_DT_FP16), hq.HQ_ERR_UNSUPPORTED), (dict(q_heads=0), hq.HQ_ERR_INVALID_ARG),
    (dict(T=-1), hq.HQ_ERR_INVALID_ARG), (dict(T=(1 << 23) + 1), hq.HQ_ERR_INVALID_ARG), (dict(table_rows=0), hq.HQ_ERR_INVALID_ARG),
    (dict(q_stride=511), hq.HQ_ERR_INVALID_ARG), (dict(k_stride=120), hq.HQ_ERR_INVALID_ARG), (dict(v_stride=132), hq.HQ_ERR_INVALID_ARG),
    (dict(q_out_stride=504), hq.HQ_ERR_INVALID_ARG), (dict(k_scale=A), hq.HQ_ERR_INVALID_ARG), (dict(q=None), hq.HQ_ERR_INVALID_ARG),
    (dict(slots=None), hq.HQ_ERR_INVALID_ARG), (dict(k_cache=None), hq.HQ_ERR_INVALID_ARG), (dict(q=A + 8), hq.HQ_ERR_ALIGNMENT),
    (dict(v_cache=A + 8), hq.HQ_ERR_ALIGNMENT), (dict(slots=A + 4), hq.HQ_ERR_ALIGNMENT), (dict(q_out=A, q_out_stride=520), hq.HQ_ERR_INVALID_ARG),
    (dict(rope=ROPE(rot_dim=80)), hq.HQ_ERR_INVALID_ARG), (dict(kv=hq.kv_desc(hq.HQ_DT_FP8_E4M3, 64, 16, 2, 64)), hq.HQ_ERR_INVALID_ARG)])
def test_rope_kv_refusals(change, want):
    a = {**RK, "rope": ROPE(), "kv": KV(), **change}
    assert status_of(hq.hq_rope_kv, **a) == want
    assert status_of(hq.hq_rope_kv, **{**RK, "rope": ROPE(), "kv": KV(), "T": 0}) == hq.HQ_OK


# ---------------------------------------------------------------------------
# refusals of the attention
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("change,want", [
    (dict(abi_version=2), hq.HQ_ERR_ABI), (dict(reserved=1), hq.HQ_ERR_INVALID_ARG), (dict(dtype=hq.HQ_DT_INT8), hq.HQ_ERR_UNSUPPORTED),
    (dict(num_blocks=0), hq.HQ_ERR_INVALID_ARG), (dict(num_blocks=1 << 28), hq.HQ_ERR_UNSUPPORTED), (dict(block_size=0), hq.HQ_ERR_INVALID_ARG),
    (dict(kv_heads=0), hq.HQ_ERR_INVALID_ARG), (dict(head_dim=72), hq.HQ_ERR_UNSUPPORTED), (dict(head_dim=272), hq.HQ_ERR_UNSUPPORTED),
    (dict(block_stride=0), hq.HQ_ERR_INVALID_ARG), (dict(slot_stride=-128), hq.HQ_ERR_INVALID_ARG), (dict(head_stride=72), hq.HQ_ERR_INVALID_ARG),
    (dict(block_stride=1 << 31), hq.HQ_ERR_INVALID_ARG), (dict(dtype=hq.HQ_DT_FP16), hq.HQ_ERR_UNSUPPORTED), (dict(kv_heads=3), hq.HQ_ERR_INVALID_ARG)])
def test_cache_descriptor_refusals(change, want):
    assert status_of(hq.hq_attn_workspace_bytes, ATT(), KV(**change), 2, 2, 0) == want


@pytest.mark.parametrize("change,want", [
    (dict(abi_version=0), hq.HQ_ERR_ABI), (dict(reserved=1), hq.HQ_ERR_INVALID_ARG), (dict(dtype=hq.HQ_DT_FP8_E4M3), hq.HQ_ERR_UNSUPPORTED),
    (dict(q_heads=0), hq.HQ_ERR_INVALID_ARG), (dict(q_heads=7), hq.HQ_ERR_INVALID_ARG), (dict(max_new=0), hq.HQ_ERR_INVALID_ARG),
    (dict(max_kv=-1), hq.HQ_ERR_INVALID_ARG), (dict(max_kv=(1 << 29) + 1), hq.HQ_ERR_INVALID_ARG), (dict(total_kv=-1), hq.HQ_ERR_INVALID_ARG),
    (dict(scale=0.0), hq.HQ_ERR_INVALID_ARG), (dict(scale=math.inf), hq.HQ_ERR_INVALID_ARG), (dict(scale=math.nan), hq.HQ_ERR_INVALID_ARG),
    (dict(softcap=-1.0), hq.HQ_ERR_INVALID_ARG), (dict(softcap=math.nan), hq.HQ_ERR_INVALID_ARG)])
def test_attn_descriptor_refusals(change, want):
    assert status_of(hq.hq_attn_workspace_bytes, ATT(**change), KV(), 2, 2, 0) == want


def test_attn_size_refusals():
    ws = hq.hq_attn_workspace_bytes
    assert status_of(ws, ATT(), KV(), -1, 2, 0) == hq.HQ_ERR_INVALID_ARG
    assert status_of(ws, ATT(), KV(), 2, -1, 0) == hq.HQ_ERR_INVALID_ARG
    assert status_of(ws, ATT(), KV(), 2, 2, -1) == hq.HQ_ERR_INVALID_ARG
    assert status_of(ws, ATT(q_heads=4096), KV(), 2, 1 << 18, 0) == hq.HQ_ERR_UNSUPPORTED
    assert status_of(ws, ATT(q_heads=64), KV(kv_heads=64), 1 << 20, 1 << 20, 0) == hq.HQ_ERR_UNSUPPORTED   # too many workgroups
    assert status_of(ws, ATT(q_heads=64, max_new=1 << 20), KV(), 4096, 1 << 20, 300) == hq.HQ_OK   # as many rows, but none to join
    many = dict(q_heads=64, max_new=1 << 20, max_kv=1000, total_kv=1)
    assert status_of(ws, ATT(**many), KV(), 1, (1 << 20) - 1, 0) == hq.HQ_OK
    assert status_of(ws, ATT(**many), KV(), 1, 1 << 20, 0) == hq.HQ_OK   # one part of the keys: none to join
    assert status_of(ws, ATT(q_heads=64), KV(), 1 << 20, (1 << 20) - 1, 3000) == hq.HQ_OK
    assert status_of(ws, ATT(q_heads=64), KV(), 1 << 20, 1 << 20, 3000) == hq.HQ_ERR_UNSUPPORTED   # too many rows to join


ATTN = dict(desc=None, kv=None, B=2, T=2, q=A, q_stride=512, k_cache=A, v_cache=A, prefix_table=A, prefix_len=600, block_table=A, max_blocks=8,
            kv_lens=A, cu_new=A, out=A, out_stride=512, lse=None, workspace=A, ws_bytes=1 << 30, k_scale=None, v_scale=None, stream=0)


@pytest.mark.parametrize("change,want", [
    (dict(q_stride=500), hq.HQ_ERR_INVALID_ARG), (dict(out_stride=516), hq.HQ_ERR_INVALID_ARG), (dict(k_scale=A, v_scale=A), hq.HQ_ERR_INVALID_ARG),
    (dict(max_blocks=-1), hq.HQ_ERR_INVALID_ARG), (dict(q=None), hq.HQ_ERR_INVALID_ARG), (dict(prefix_table=None), hq.HQ_ERR_INVALID_ARG),
    (dict(block_table=None), hq.HQ_ERR_INVALID_ARG), (dict(cu_new=None), hq.HQ_ERR_INVALID_ARG), (dict(out=None), hq.HQ_ERR_INVALID_ARG),
    (dict(q=A + 8), hq.HQ_ERR_ALIGNMENT), (dict(v_cache=A + 2), hq.HQ_ERR_ALIGNMENT), (dict(kv_lens=A + 2), hq.HQ_ERR_ALIGNMENT),
    (dict(lse=A + 1), hq.HQ_ERR_ALIGNMENT), (dict(workspace=None), hq.HQ_ERR_WORKSPACE), (dict(ws_bytes=16), hq.HQ_ERR_WORKSPACE),
    (dict(workspace=A + 4), hq.HQ_ERR_ALIGNMENT), (dict(kv=hq.kv_desc(hq.HQ_DT_FP8_E4M3, 64, 16, 2, 64)), hq.HQ_ERR_INVALID_ARG)])
def test_attn_refusals(change, want):
    a = {**ATTN, "desc": ATT(), "kv": KV(), **change}
    assert status_of(hq.hq_attn, **a) == want


def test_attn_without_work():
    for k in ("T", "B"):
        a = {**ATTN, "desc": ATT(), "kv": KV(), k: 0, "q": None, "out": None}
        assert status_of(hq.hq_attn, **a) == hq.HQ_OK
        assert hq.hq_attn_workspace_bytes(ATT(), KV(), a["B"], a["T"], 600) == 0
        assert hq.hq_attn_plan(ATT(), KV(), a["B"], a["T"], 600) == []


# ---------------------------------------------------------------------------
# plans
# ---------------------------------------------------------------------------

def plan(B, T, prefix, max_new, max_kv, **k):
    return hq.hq_attn_plan(ATT(max_new=max_new, max_kv=max_kv), KV(**k), B, T, prefix)


def test_plans():
    """One launch where one workgroup a head is enough; a join where keys are cut;
    a prefix for all, and walked by each request where nobody shares it."""
    one = plan(1, 1, 0, 1, 300)
    assert len(one) == 1 and "prefix=0 few=1 many=0" in one[0]
    assert hq.hq_attn_workspace_bytes(ATT(max_kv=300), KV(), 1, 1, 0) == 0
    cut = plan(1, 1, 0, 1, 10000)
    assert len(cut) == 2 and "attn_join" in cut[1]
    assert "joint=1" in plan(1, 1, 5000, 1, 300)[0]
    assert "joint=0" in plan(64, 64, 5000, 1, 300)[0]
    assert "joint=1" in plan(4, 4, 64, 1, 100)[0] and len(plan(4, 4, 64, 1, 100)) == 1
    prompt = plan(2, 2000, 0, 1000, 1000)
    assert "many=0" not in prompt[0]
    for dim, name in ((16, "attn<64,"), (64, "attn<64,"), (80, "attn<128,"), (128, "attn<128,"), (144, "attn<256,"), (256, "attn<256,")):
        assert plan(1, 1, 0, 1, 300, head_dim=dim)[0].startswith(name)


@pytest.mark.parametrize("B,max_kv,prefix", [(1, 1 << 20, 0), (1, 1 << 29, 0), (200, 5000, 1 << 20), (4096, 100000, 300)])
def test_plans_of_long_contexts(B, max_kv, prefix):
    """The number of parts is bounded, and the workspace holds them all."""
    d, kv = ATT(max_kv=max_kv), KV()
    p = hq.hq_attn_plan(d, kv, B, B, prefix)
    parts = int(p[1].split("parts=")[1])
    assert 1 < parts <= 512
    assert hq.hq_attn_workspace_bytes(d, kv, B, B, prefix) >= parts * B * 8 * (64 + 2) * 4


# ---------------------------------------------------------------------------
# pins of the definitions
# ---------------------------------------------------------------------------

def test_slots_by_hand():
    """P = 4: request 0 has 3 of 4 places of page 7 used and takes 3 more (one new page);
    request 1 is new with 5 tokens (two pages); request 2 does nothing."""
    cu, kv, table, pos, slots, taken = okv.slots([3, 0, 4], [3, 5, 0], [20, 21, 22, 23], [[7, -1], [-1, -1], [9, -1]], 4, 9, first_pos=100)
    assert cu.tolist() == [0, 3, 8, 8] and kv.tolist() == [6, 5, 4] and taken == 3
    assert table.tolist() == [[7, 20], [21, 22], [9, -1]]
    assert pos.tolist() == [103, 104, 105, 100, 101, 102, 103, 104, 0]
    assert slots.tolist() == [31, 80, 81, 84, 85, 86, 87, 88, -1]


def test_rope_invariants():
    """Angles add: the product of a query at p and a key at r depends on p - r alone;
    lengths are kept; position 0 is the identity."""
    rng = np.random.default_rng(0)
    t = okv.rope_table(32, 0, 200)
    for inter in (False, True):
        q, k = rng.standard_normal((2, 1, 1, 48))
        dot = [float(np.sum(okv.rope(q, t[p:p + 1], 32, inter) * okv.rope(k, t[r:r + 1], 32, inter))) for p, r in ((5, 2), (103, 100), (3, 0))]
        assert np.allclose(dot, dot[0], rtol=0, atol=1e-12)
        assert np.allclose(okv.rope(q, t[:1], 32, inter), q)
        assert np.isclose(np.linalg.norm(okv.rope(q, t[77:78], 32, inter)), np.linalg.norm(q))
        assert np.array_equal(okv.rope(q, t[9:10], 32, inter)[..., 32:], q[..., 32:])


def test_rope_scalings():
    """Linear stretching reads the plain table at pos / factor; ntk keeps the fastest
    pair and stretches the slowest by the factor; parts keeps fast pairs and
    stretches slow ones."""
    plain = okv.rope_table(64, 0, 400, base=1e4)
    assert np.allclose(okv.rope_table(64, 0, 400, scaling="linear", factor=4.0)[::4], plain[:100])
    ntk = okv.rope_table(64, 0, 400, scaling="ntk", factor=4.0)
    assert np.allclose(ntk[:, [0, 32]], plain[:, [0, 32]]) and np.allclose(ntk[::4][:, [31, 63]], plain[:100][:, [31, 63]])
    parts = okv.rope_table(64, 0, 400, scaling="parts", factor=4.0, context=4096.0, attn_factor=1.0)
    assert np.allclose(parts[:, [0, 32]], plain[:, [0, 32]]) and np.allclose(parts[::4][:, [31, 63]], plain[:100][:, [31, 63]])
    gain = okv.rope_table(64, 0, 1, scaling="parts", factor=4.0, context=4096.0)
    assert np.allclose(gain[0, :32], 0.1 * math.log(4.0) + 1.0)


def test_attention_invariants():
    """Equal keys give the mean of the seen values; a prefix is the same as own keys
    that come first; a shift of all scores changes lse alone."""
    rng = np.random.default_rng(1)
    v = rng.standard_normal((9, 2, 8))
    q = rng.standard_normal((3, 4, 8))
    one = okv.attention(q, lambda r: np.ones((9, 2, 8)), lambda r: v, 4, [5], [0, 3], 0.3)
    for t in range(3):
        assert np.allclose(one[0][t, 0], v[:7 + t, 0].mean(0)) and np.allclose(one[0][t, 3], v[:7 + t, 1].mean(0))
    k = rng.standard_normal((9, 2, 8))
    a = okv.attention(q, lambda r: k, lambda r: v, 4, [5], [0, 3], 0.3)
    b = okv.attention(q, lambda r: k, lambda r: v, 0, [9], [0, 3], 0.3)
    assert np.allclose(a[0], b[0]) and np.allclose(a[1], b[1])
    big = okv.attention(q, lambda r: k, lambda r: v, 4, [5], [0, 3], 0.3, softcap=1e6)
    assert np.allclose(a[0], big[0], atol=1e-6)
