"""Routing to experts and the weighted sum of their outputs against the definitions in 64 bits."""
import numpy as np
import pytest
import torch

from bit_quantized_gemm_w4a16_amd import hq
from gpu_util import note
from layer_util import DT, f64
from oracle import layer as ol

pytestmark = pytest.mark.gpu


def routed(logits, bias, top_k, *, dtype="fp32", stride=None, T=None, E=None, stream=None, **kw):
    T, E = T or logits.shape[0], E or logits.shape[1]
    ids = torch.full((T * top_k + 8,), -77, dtype=torch.int32, device="cuda")
    w = torch.full((T * top_k + 8,), -77.0, device="cuda")
    hq.hq_moe_route(hq.route_desc(DT[dtype][0], E, top_k, **kw), T, logits, stride or E, bias, ids, w, stream=stream)
    torch.cuda.synchronize()
    assert (ids[T * top_k:] == -77).all() and (w[T * top_k:] == -77).all(), "written behind the last token"
    return ids[:T * top_k].view(T, top_k).cpu().numpy(), f64(w[:T * top_k].view(T, top_k))


def check(logits, bias, top_k, dtype="fp32", **kw):
    ids, w = routed(logits, bias, top_k, dtype=dtype, **kw)
    scale = kw.pop("scale", 1.0)
    kw["renormalize"] = kw.get("renormalize", True)
    kw["sigmoid"] = kw.get("sigmoid", False)
    want, ww = ol.route(f64(logits), None if bias is None else f64(bias), top_k, kw["sigmoid"], kw["renormalize"], kw.get("groups", 1),
                        kw.get("top_groups", 1), kw.get("group_best", 1), float(np.float32(scale)))
    np.testing.assert_array_equal(ids, want)
    # scores, their sum and quotient in 64 bits (under 1000 roundings of 2^-53), one rounding to fp32
    assert (np.abs(w - ww) <= np.abs(ww) * (2.0 ** -24 + 2.0 ** -43) + 2.0 ** -149).all()


def logits_of(seed, T, E, dtype="fp32", std=1.5):
    g = torch.Generator().manual_seed(seed)
    return (std * torch.randn(T, E, generator=g) + 0.5 * torch.randn(E, generator=g)).to(DT[dtype][1]).cuda()


def bias_of(seed, E):
    return (0.2 * torch.randn(E, generator=torch.Generator().manual_seed(seed))).cuda()


@pytest.mark.parametrize("E", [1, 2, 3, 31, 63, 64, 65, 100, 128, 129, 256, 257, 384, 512, 513, 1000, 1024, 1025, 4095, 4096])
def test_route_experts_and_scores(E):
    """Every count of experts per lane, both scorings, with and without a bias, all three dtypes."""
    k = min(E, 8)
    for n, (sigmoid, bias, dtype) in enumerate([(False, False, "fp32"), (True, True, "fp32"), (True, False, "bf16"), (False, True, "fp16")]):
        note(f"route E={E} k={k} sigmoid={sigmoid} bias={bias} {dtype}")
        check(logits_of(n, 13, E, dtype), bias_of(n, E) if bias else None, k, dtype, sigmoid=sigmoid, renormalize=n % 2 == 0, scale=1.0 + 1.5 * (n > 1))


@pytest.mark.parametrize("E,groups,top_groups,best,k", [(256, 8, 4, 2, 8), (256, 8, 1, 1, 32), (160, 8, 3, 1, 6), (64, 64, 5, 1, 5), (120, 60, 7, 2, 9),
                                                       (512, 8, 4, 2, 10), (4096, 64, 2, 2, 64), (96, 3, 3, 2, 8), (1030, 5, 2, 2, 8), (65, 13, 2, 1, 7)])
@pytest.mark.parametrize("bias", [False, True])
def test_route_groups(E, groups, top_groups, best, k, bias):
    for sigmoid in (False, True):
        note(f"route groups E={E} {groups}/{top_groups}/{best} k={k} bias={bias} sigmoid={sigmoid}")
        check(logits_of(5, 21, E), bias_of(6, E) if bias else None, k, sigmoid=sigmoid, groups=groups, top_groups=top_groups, group_best=best)


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 63, 1025])
def test_route_token_counts(T):
    note(f"route T={T}")
    check(logits_of(7, T, 60), None, 4, renormalize=False)


def test_route_all_experts():
    """k = every expert (64 of 64), and one of one."""
    note("route all")
    check(logits_of(8, 7, 64), bias_of(9, 64), 64, sigmoid=True)
    check(logits_of(8, 7, 1), None, 1)


def test_route_strided_rows():
    note("route strided")
    wide = logits_of(10, 9, 300)
    ids, w = routed(wide, None, 4, stride=300, E=150)
    want, ww = ol.route(f64(wide)[:, :150], None, 4, False, True)
    np.testing.assert_array_equal(ids, want)
    assert (np.abs(w - ww) <= ww * (2.0 ** -24 + 2.0 ** -43)).all()


def test_route_ties_go_to_the_lowest():
    """Equal logits, equal sums of score and bias, equal groups; values that fp32 scores cannot tell apart."""
    note("route ties")
    x = torch.zeros(3, 200, device="cuda")
    x[1, 50:] = 2.0
    x[2] = torch.randint(0, 3, (200,), generator=torch.Generator().manual_seed(0)).float().cuda()
    for kw in (dict(), dict(sigmoid=True), dict(groups=8, top_groups=2, group_best=2)):
        check(x, None, 8, **kw)
        check(x, torch.zeros(200, device="cuda"), 8, **kw)
    # logits of one more unit in the last place each, in falling order of their index: all scores round to 1.0
    y = (40.0 + torch.arange(128) * 2.0 ** -18).flip(0)[None].cuda()
    ids, _ = routed(y, None, 4, sigmoid=True)
    np.testing.assert_array_equal(ids, [[0, 1, 2, 3]])
    ids, _ = routed(y.flip(1).contiguous(), None, 4, sigmoid=True)
    np.testing.assert_array_equal(ids, [[127, 126, 125, 124]])
    # biased scores that differ by less than fp32 holds near 8
    z = torch.zeros(1, 64)
    z[0, 40] = 2.0 ** -20  # its sigmoid is 2^-22 above a half
    ids, _ = routed(z.cuda(), torch.full((64,), 8.0, device="cuda"), 1, sigmoid=True)
    assert ids[0, 0] == 40


def test_route_masked_and_not_finite():
    """-inf logits (some, all but fewer than k, all), the type's lowest value, far negative ones; -inf biases; NaN."""
    note("route masked")
    x = logits_of(11, 6, 96)
    x[0, ::2] = -torch.inf
    x[1, 3:] = -torch.inf
    x[2] = -torch.inf
    x[3, 10:] = torch.finfo(torch.float32).min
    x[4] = -700.0 - torch.arange(96).float().cuda()
    for kw in (dict(), dict(renormalize=False), dict(sigmoid=True), dict(groups=4, top_groups=2)):
        check(x, None, 8, **kw)
    b = bias_of(12, 96)
    b[5:90] = -torch.inf
    check(x, b, 8, sigmoid=True)
    check(x, b, 20, sigmoid=True)  # more than the finite ones: the lowest of the others
    y = logits_of(13, 3, 96)
    y[1, 7] = torch.nan
    ids, w = routed(y, None, 8)
    want, ww = ol.route(f64(y)[[0, 2]], None, 8, False, True)
    np.testing.assert_array_equal(ids[[0, 2]], want)
    assert np.isnan(w[1]).all() and 7 not in ids[1] and len(set(ids[1])) == 8
    ids, w = routed(y, None, 8, sigmoid=True)
    assert 7 not in ids[1] and np.isfinite(w).all()
    y[1] = torch.nan
    ids, w = routed(y, None, 8, sigmoid=True)
    np.testing.assert_array_equal(ids[1], np.arange(8))


# ---------------------------------------------------------------------------
# the weighted sum
# ---------------------------------------------------------------------------

def summed(dtype, y, w, add, order, T, k, N, into_add=False):
    out = torch.full((T * N + 32,), 7.0, dtype=DT[dtype][1], device="cuda")
    if into_add:
        out[:T * N] = add.reshape(-1)
        add = out
    ws = torch.full((T * k + 4,), 1 << 30, dtype=torch.int32, device="cuda")  # what it held before does not matter
    hq.hq_moe_combine(DT[dtype][0], T, k, N, y, w, out, add=add, sorted_pairs=order, workspace=ws if order is not None else None, ws_bytes=T * k * 4)
    torch.cuda.synchronize()
    assert (out[T * N:] == 7.0).all() and (ws[T * k:] == 1 << 30).all()
    return f64(out[:T * N].view(T, N))


@pytest.mark.parametrize("N", [1, 7, 8, 100, 1777, 2048, 2056, 7168])
@pytest.mark.parametrize("T,k", [(1, 1), (3, 8), (5, 3), (33, 10)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_combine(dtype, T, k, N):
    g = torch.Generator().manual_seed(N)
    y = torch.randn(T * k, N, generator=g).to(DT[dtype][1]).cuda()
    w = (torch.rand(T, k, generator=g) - 0.2).cuda()
    add = (3 * torch.randn(T, N, generator=g)).to(DT[dtype][1]).cuda()
    order = torch.randperm(T * k, generator=g).to(torch.int32).cuda()
    at = np.empty(T * k, np.int64)
    at[order.cpu().numpy()] = np.arange(T * k)
    for a, o, rows in ((None, None, np.arange(T * k)), (add, None, np.arange(T * k)), (None, order, at), (add, order, at)):
        note(f"combine {dtype} T={T} k={k} N={N} add={a is not None} sorted={o is not None}")
        got = summed(dtype, y, w, a, o, T, k, N)
        want, S = ol.combine(f64(y), f64(w), None if a is None else f64(a), rows.reshape(T, k))
        # one rounding of the result, and k products, k sums and the addition in fp32
        assert (np.abs(got - want) <= np.abs(want) * DT[dtype][2] + S * (2 * k + 2) * 2.0 ** -24 + 2.0 ** -25).all()
        if a is not None:
            assert (summed(dtype, y, w, a, o, T, k, N, into_add=True) == got).all()


def test_combine_rows_that_do_not_count():
    """A weight of 0 keeps a row of NaN out; pairs that sorted_pairs does not name, and names outside, add nothing."""
    note("combine dropped rows")
    T, k, N = 4, 3, 64
    y = torch.randn(T * k, N, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    w = torch.rand(T, k, generator=torch.Generator().manual_seed(2)).cuda() + 0.1
    y[4] = torch.nan
    w[1, 1] = 0.0
    want, S = ol.combine(np.nan_to_num(f64(y)), f64(w), None, np.arange(T * k).reshape(T, k))
    got = summed("bf16", y, w, None, None, T, k, N)
    assert (np.abs(got - want) <= np.abs(want) * 2.0 ** -8 + S * 8 * 2.0 ** -24).all()
    order = torch.arange(T * k, dtype=torch.int32, device="cuda")
    order[[2, 7]] = torch.tensor([-5, 1 << 20], dtype=torch.int32, device="cuda")
    rows = np.arange(T * k)
    rows[[2, 7]] = -1
    for before in (0, 2, 7, 1 << 30):  # whatever the workspace held
        ws = torch.full((T * k,), before, dtype=torch.int32, device="cuda")
        out = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
        hq.hq_moe_combine(hq.HQ_DT_BF16, T, k, N, y, w, out, sorted_pairs=order, workspace=ws, ws_bytes=T * k * 4)
        want, S = ol.combine(np.nan_to_num(f64(y)), f64(w), None, rows.reshape(T, k))
        assert (np.abs(f64(out) - want) <= np.abs(want) * 2.0 ** -8 + S * 8 * 2.0 ** -24).all()


def test_route_and_combine_captured():
    """Both in one graph on a side stream, replayed with new inputs between eager calls."""
    T, E, k, N = 7, 64, 4, 512
    note("route and combine captured")
    x, y = logits_of(30, T, E), torch.randn(T * k, N, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).cuda()
    order = torch.randperm(T * k).to(torch.int32).cuda()
    desc = hq.route_desc(hq.HQ_DT_FP32, E, k)
    bufs = [(torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda"), torch.empty(T, N, dtype=torch.bfloat16, device="cuda"),
             torch.empty(T * k, dtype=torch.int32, device="cuda")) for _ in range(2)]

    def call(ids, w, out, ws):
        hq.hq_moe_route(desc, T, x, E, None, ids, w)
        hq.hq_moe_combine(hq.HQ_DT_BF16, T, k, N, y, w, out, sorted_pairs=order, workspace=ws, ws_bytes=T * k * 4)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(*bufs[0])
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        call(*bufs[0])
    for i in range(3):
        x.copy_(logits_of(31 + i, T, E))
        g.replay()
        call(*bufs[1])
        torch.cuda.synchronize()
        for a, b in zip(bufs[0][:3], bufs[1][:3]):
            assert torch.equal(a, b)
