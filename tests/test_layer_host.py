"""Host side of a routed layer's operators (no GPU): refusals before any HIP call,
workspace sizes, and pins of the 64-bit definitions."""
import numpy as np
import pytest

from bit_quantized_gemm_w4a16_amd import hq
from oracle import layer as ol

A = 1 << 20  # stands for an aligned device pointer; no call below gets as far as using it


def status_of(fn, *args, **kw):
    try:
        fn(*args, **kw)
    except hq.HQError as e:
        return e.status
    return hq.HQ_OK


def with_(d, **fields):
    for k, v in fields.items():
        setattr(d, k, v)
    return d


BAD, UNSUP, ALIGN = hq.HQ_ERR_INVALID_ARG, hq.HQ_ERR_UNSUPPORTED, hq.HQ_ERR_ALIGNMENT
BF, F8, I8, F4 = hq.HQ_DT_BF16, hq.HQ_DT_FP8_E4M3, hq.HQ_DT_INT8, hq.HQ_DT_FP4_E2M1
TOKEN, BLOCK, MX = hq.HQ_ASCALE_PER_TOKEN_F32, hq.HQ_ASCALE_PER_BLOCK128_F32, hq.HQ_ASCALE_MX_E8M0
norm = lambda **k: with_(hq.norm_desc(BF, F8, BLOCK), **k)  # noqa: E731
NORM = dict(M=2, K=256, x=A, x_stride=256, weight=A, out=A, out_scale=A, residual=A, residual_stride=256, sum_out=A, sum_stride=256, stream=0)


@pytest.mark.parametrize("desc,change,want", [
    (dict(abi_version=2), {}, hq.HQ_ERR_ABI), (dict(reserved=1), {}, BAD), (dict(dtype=hq.HQ_DT_FP32), {}, UNSUP),
    (dict(weight_dtype=hq.HQ_DT_FP16), {}, UNSUP), (dict(eps=-1.0), {}, BAD), (dict(eps=float("nan")), {}, BAD),
    (dict(weight_offset=float("inf")), {}, BAD), (dict(out_dtype=hq.HQ_DT_FP16), {}, UNSUP), (dict(a_scale=9), {}, UNSUP),
    (dict(out_dtype=I8), {}, UNSUP), (dict(out_dtype=F4), {}, UNSUP), (dict(out_dtype=F4, a_scale=TOKEN), {}, UNSUP),
    ({}, dict(M=-1), BAD), ({}, dict(M=(1 << 22) + 1), BAD), ({}, dict(K=0, x_stride=0), BAD), ({}, dict(K=65664, x_stride=65664), UNSUP),
    ({}, dict(K=200), UNSUP), (dict(a_scale=MX), dict(K=200), UNSUP), ({}, dict(x_stride=255), BAD), ({}, dict(residual_stride=255), BAD),
    ({}, dict(sum_stride=255), BAD), ({}, dict(x_stride=1 << 31), BAD), ({}, dict(x_stride=257), UNSUP), ({}, dict(residual_stride=260), UNSUP),
    (dict(a_scale=MX), dict(sum_stride=258), UNSUP), ({}, dict(x=None), BAD), ({}, dict(weight=None), BAD), ({}, dict(out=None), BAD),
    ({}, dict(out_scale=None), BAD), (dict(out_dtype=BF, a_scale=0), {}, BAD), ({}, dict(x=A + 8), ALIGN), ({}, dict(residual=A + 2), ALIGN),
    ({}, dict(weight=A + 4), ALIGN), ({}, dict(sum_out=A + 8), ALIGN), ({}, dict(out=A + 8), ALIGN), ({}, dict(out_scale=A + 4), ALIGN)])
def test_norm_refusals(desc, change, want):
    assert status_of(hq.hq_rmsnorm, norm(**desc), **{**NORM, **change}) == want
    assert hq.lib().hq_last_error()


def test_empty_calls_are_fine():
    """No rows: nothing is launched and no pointer is looked at."""
    assert status_of(hq.hq_rmsnorm, norm(), 0, 256, None, 256, None, None, stream=0) == hq.HQ_OK
    assert status_of(hq.hq_silu_mul_quant, BF, F8, TOKEN, 0, 64, None, None, None, stream=0) == hq.HQ_OK
    assert status_of(hq.hq_moe_route, route(), 0, None, 64, None, None, None, stream=0) == hq.HQ_OK
    assert status_of(hq.hq_moe_combine, BF, 0, 2, 64, None, None, None, stream=0) == hq.HQ_OK
    d = hq.desc_moe_fp8_blockwise(4, 256, 256)
    assert status_of(hq.hq_moe_gemm, d, hq.HQ_MOE_INDEXED, 0, 2, None, None, None, None, None, None, None, None, stream=0) == hq.HQ_OK


SILU = dict(dtype=BF, out_dtype=F8, a_scale=BLOCK, rows=2, I=256, gate_up=A, out=A, out_scale=A, stream=0)


@pytest.mark.parametrize("change,want", [
    (dict(dtype=hq.HQ_DT_FP32), UNSUP), (dict(rows=-1), BAD), (dict(rows=(1 << 22) + 1), BAD), (dict(I=0), BAD), (dict(I=12), BAD),
    (dict(I=65664), UNSUP), (dict(I=200), UNSUP), (dict(I=200, a_scale=MX), UNSUP), (dict(out_dtype=BF, a_scale=0), UNSUP),
    (dict(out_dtype=I8), UNSUP), (dict(gate_up=None), BAD), (dict(out=None), BAD), (dict(out_scale=None), BAD), (dict(gate_up=A + 8), ALIGN),
    (dict(out=A + 8), ALIGN), (dict(out_scale=A + 8), ALIGN)])
def test_silu_refusals(change, want):
    assert status_of(hq.hq_silu_mul_quant, **{**SILU, **change}) == want
    assert hq.lib().hq_last_error()


route = lambda **k: with_(hq.route_desc(hq.HQ_DT_FP32, 64, 4), **k)  # noqa: E731
ROUTE = dict(T=3, logits=A, logits_stride=64, bias=A, topk_ids=A, topk_weights=A, stream=0)


@pytest.mark.parametrize("desc,change,want", [
    (dict(abi_version=0), {}, hq.HQ_ERR_ABI), (dict(reserved=3), {}, BAD), (dict(dtype=I8), {}, UNSUP), (dict(scoring=0), {}, BAD),
    (dict(renormalize=2), {}, BAD), (dict(scale=float("inf")), {}, BAD), (dict(num_experts=0), {}, BAD), (dict(num_experts=4097), dict(logits_stride=4097), BAD),
    (dict(groups=0), {}, BAD), (dict(groups=7), {}, BAD), (dict(groups=128, num_experts=128), dict(logits_stride=128), BAD),
    (dict(groups=8, top_groups=9), {}, BAD), (dict(groups=8, top_groups=0), {}, BAD), (dict(groups=8, group_best=3), {}, BAD),
    (dict(groups=64, top_groups=8, group_best=2), {}, BAD), (dict(top_k=0), {}, BAD), (dict(top_k=65, num_experts=128), dict(logits_stride=128), BAD),
    (dict(groups=16, top_groups=1, top_k=5), {}, BAD), ({}, dict(T=-1), BAD), ({}, dict(T=(1 << 24) + 1), BAD), ({}, dict(logits_stride=63), BAD),
    ({}, dict(logits_stride=1 << 31), BAD), ({}, dict(logits=None), BAD), ({}, dict(topk_ids=None), BAD), ({}, dict(topk_weights=None), BAD),
    ({}, dict(logits=A + 4), ALIGN), ({}, dict(bias=A + 4), ALIGN), ({}, dict(topk_ids=A + 4), ALIGN), ({}, dict(topk_weights=A + 8), ALIGN)])
def test_route_refusals(desc, change, want):
    assert status_of(hq.hq_moe_route, route(**desc), **{**ROUTE, **change}) == want
    assert hq.lib().hq_last_error()


COMBINE = dict(dtype=BF, T=4, top_k=2, N=64, y=A, topk_weights=A, out=A, add=A, sorted_pairs=A, workspace=A, ws_bytes=32, stream=0)


@pytest.mark.parametrize("change,want", [
    (dict(dtype=hq.HQ_DT_FP32), UNSUP), (dict(T=-1), BAD), (dict(T=(1 << 23) + 1), BAD), (dict(top_k=0), BAD), (dict(top_k=4097), BAD),
    (dict(N=0), BAD), (dict(N=(1 << 21) + 1), BAD), (dict(T=1 << 23, top_k=256), UNSUP), (dict(y=None), BAD), (dict(topk_weights=None), BAD),
    (dict(out=None), BAD), (dict(y=A + 8), ALIGN), (dict(topk_weights=A + 8), ALIGN), (dict(add=A + 2), ALIGN), (dict(sorted_pairs=A + 4), ALIGN),
    (dict(out=A + 2), ALIGN), (dict(workspace=None), hq.HQ_ERR_WORKSPACE), (dict(ws_bytes=31), hq.HQ_ERR_WORKSPACE), (dict(workspace=A + 4), ALIGN)])
def test_combine_refusals(change, want):
    assert status_of(hq.hq_moe_combine, **{**COMBINE, **change}) == want
    assert hq.lib().hq_last_error()


f8 = lambda **k: with_(hq.desc_moe_fp8_blockwise(8, 256, 256), **k)  # noqa: E731
GEMM = dict(mode=hq.HQ_MOE_INDEXED, T=4, top_k=2, A=A, a_scale=A, topk_ids=A, expert_offsets=None, w=A, s=A, z=None, D=A, workspace=A,
            ws_bytes=1 << 20, stream=0)


@pytest.mark.parametrize("desc,change,want", [
    (dict(a_scale=TOKEN), {}, UNSUP), (dict(w_scale_gran=hq.HQ_GRAN_PER_CHANNEL), {}, UNSUP), (dict(out_dtype=hq.HQ_DT_FP16), {}, UNSUP),
    (dict(K=200), {}, UNSUP), (dict(K=1 << 20, N=1 << 11), {}, UNSUP), (dict(flags=hq.HQ_FLAG_BATCH_INVARIANT), {}, UNSUP),
    (dict(num_experts=0), {}, BAD), ({}, dict(a_scale=None), BAD), ({}, dict(z=A), BAD), ({}, dict(mode=3), BAD), ({}, dict(top_k=9), BAD),
    ({}, dict(topk_ids=None), BAD), ({}, dict(expert_offsets=A), BAD), (dict(), dict(mode=hq.HQ_MOE_GROUPED), BAD), ({}, dict(a_scale=A + 8), ALIGN),
    ({}, dict(D=A + 8), ALIGN), ({}, dict(topk_ids=A + 4), ALIGN), ({}, dict(workspace=A + 8), ALIGN), ({}, dict(workspace=None), hq.HQ_ERR_WORKSPACE),
    ({}, dict(ws_bytes=15), hq.HQ_ERR_WORKSPACE), (dict(K=1 << 14), dict(T=1 << 18, top_k=1), UNSUP), ({}, dict(T=1 << 22, top_k=8), UNSUP)])
def test_expert_refusals(desc, change, want):
    assert status_of(hq.hq_moe_gemm, f8(**desc), **{**GEMM, **change}) == want
    assert hq.lib().hq_last_error()


def test_expert_layout_is_the_dense_layout_of_each():
    rng = np.random.default_rng(0)
    E, N, K = 3, 200, 256
    w = rng.integers(0, 127, (E, K, N), dtype=np.uint8)
    s = rng.random((E, K // 128, -(-N // 128)), dtype=np.float32)
    got_w, got_s, _ = hq.hq_repack(hq.desc_moe_fp8_blockwise(E, N, K), w, s)
    each = [hq.hq_repack(hq.desc_fp8_blockwise(N, K), w[e], s[e]) for e in range(E)]
    np.testing.assert_array_equal(got_w, np.concatenate([x[0] for x in each]))
    np.testing.assert_array_equal(got_s, np.concatenate([x[1] for x in each]))


@pytest.mark.parametrize("T,top_k,E", [(1, 1, 1), (4, 8, 256), (9, 8, 8), (1024, 8, 256), (4095, 8, 32), (100000, 8, 512)])
def test_expert_workspace_holds_the_routing(T, top_k, E):
    """The sorted pairs and the tile list at least; a few bytes per pair and expert at most."""
    n = hq.hq_workspace_bytes(hq.desc_moe_fp8_blockwise(E, 256, 256), T, top_k)
    assert T * top_k * 4 <= n <= T * top_k * 12 + E * 64 + (T * top_k // 8192 + 1) * E * 4 + 256


# ---------------------------------------------------------------------------
# the definitions
# ---------------------------------------------------------------------------

def test_route_definition_by_hand():
    x = np.log(np.array([[1.0, 2.0, 4.0, 1.0], [8.0, 8.0, 8.0, 8.0]]))
    ids, w = ol.route(x, None, 2, False, False)
    np.testing.assert_array_equal(ids, [[2, 1], [0, 1]])
    np.testing.assert_allclose(w, [[0.5, 0.25], [0.25, 0.25]], rtol=1e-15)
    ids, w = ol.route(x, None, 2, False, True, scale=3.0)
    np.testing.assert_allclose(w, [[2.0, 1.0], [1.5, 1.5]], rtol=1e-15)
    # a bias changes the choice and not the weight: sigmoid of 0 is a half
    ids, w = ol.route(np.zeros((1, 4)), np.array([0.0, 0.25, -1.0, 0.25]), 2, True, False)
    np.testing.assert_array_equal(ids, [[1, 3]])
    np.testing.assert_array_equal(w, [[0.5, 0.5]])
    # groups: {1, 2} holds the two best together, {3, 0} the single best
    s = np.array([[0.0, 0.4, 0.5, 0.4]])
    ids, _ = ol.route(np.zeros((1, 4)), s[0][[1, 3, 2, 0]], 2, True, False, groups=2, top_groups=1, group_best=2)
    np.testing.assert_array_equal(ids, [[0, 1]])
    ids, _ = ol.route(np.zeros((1, 4)), s[0][[1, 3, 2, 0]], 2, True, False, groups=2, top_groups=1, group_best=1)
    np.testing.assert_array_equal(ids, [[2, 3]])
    # nothing left by the logits: the lowest experts, weights 0
    ids, w = ol.route(np.full((1, 4), -np.inf), None, 2, False, True)
    np.testing.assert_array_equal(ids, [[0, 1]])
    np.testing.assert_array_equal(w, [[0.0, 0.0]])


def test_norm_and_swiglu_definitions_by_hand():
    h, y = ol.rms_norm(np.array([[3.0, 4.0]]), np.array([[0.0, 1.0]]), np.array([1.0, 2.0]), 0.0)
    np.testing.assert_array_equal(h, [[3.0, 5.0]])
    np.testing.assert_allclose(y, [[3 / 17 ** 0.5, 10 / 17 ** 0.5]], rtol=1e-15)
    _, y = ol.rms_norm(np.array([[2.0, 2.0]]), None, np.zeros(2), 0.0, offset=1.0)
    np.testing.assert_allclose(y, [[1.0, 1.0]], rtol=1e-15)
    np.testing.assert_allclose(ol.silu_mul(np.array([[0.0, 2.0, -800.0, 5.0, 3.0, 2.0]])), [[0.0, 2 / (1 + np.exp(-2)) * 3.0, 0.0]], atol=1e-300)
    np.testing.assert_array_equal(ol.scales(np.array([[0.0, 0.0, 8.0, np.nan]]), 2, 4.0), [[1.0, 2.0]])
    np.testing.assert_array_equal(ol.step_e4m3(np.array([0.0, 1.0, 1.9, 2.0, 448.0, 2.0 ** -7])), [2.0 ** -9, 0.125, 0.125, 0.25, 32.0, 2.0 ** -9])
    np.testing.assert_array_equal(ol.step_e2m1(np.array([0.2, 1.0, 2.0, 4.0, 6.0])), [0.5, 0.5, 1.0, 2.0, 2.0])


@pytest.mark.parametrize("T,top_k,E", [(1, 1, 1), (7, 4, 16), (8, 8, 256), (9, 8, 256), (100, 2, 4096), (512, 8, 256), (5000, 8, 32), (65536, 8, 256)])
def test_a_layers_workspace_holds_the_sorting_of_its_routes(T, top_k, E):
    """hq_moe_align takes the workspace of a layer with the same T and top_k (past the check of its size the address is refused)."""
    for desc in (hq.desc_moe_fp8_blockwise(E, 256, 256), hq.desc_moe_mxfp4(E, 256, 256)):
        n = hq.hq_workspace_bytes(desc, T, top_k)
        with pytest.raises(hq.HQError) as e:
            hq.hq_moe_align(T, top_k, E, A, A, A, A + 4, n, stream=0)
        assert e.value.status == hq.HQ_ERR_ALIGNMENT


def test_as_many_rows_as_a_launch_holds():
    """Workgroups times threads stay below 2^32, with up to 1024 threads a row."""
    for M, want in ((1 << 22, BAD), ((1 << 22) - 1, ALIGN)):
        assert status_of(hq.hq_rmsnorm, norm(), **{**NORM, "M": M, "x": A + 8}) == want
        assert status_of(hq.hq_silu_mul_quant, **{**SILU, "rows": M, "gate_up": A + 8}) == want


@pytest.mark.parametrize("E,top_k", [(1, 1), (3, 2), (8, 8), (32, 4), (256, 8), (4096, 1)])
def test_fewer_tokens_never_need_a_larger_workspace(E, top_k):
    """A workspace for the largest step serves every smaller one, whichever kernels take it."""
    desc, before = hq.desc_moe_fp8_blockwise(E, 256, 256), 0
    for T in (*range(2200), 4095, 4096, 4097, 20000, 65535, 65536):
        need = hq.hq_workspace_bytes(desc, T, top_k)
        assert need >= before, T
        before = need
