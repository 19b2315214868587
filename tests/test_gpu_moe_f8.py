"""Experts in FP8 with block scales (hq_moe_gemm) against their definition in 64 bits."""
import numpy as np
import pytest
import torch

import synthetic as syn
from bit_quantized_gemm_w4a16_amd import hq
from gpu_util import note
from layer_util import f64
from oracle import layer as ol

pytestmark = pytest.mark.gpu


class Experts:
    """E experts of random codes and scales, packed, and in 64 bits."""

    def __init__(self, E, N, K, seed=0):
        rng = np.random.default_rng(seed)
        self.E, self.N, self.K = E, N, K
        self.desc = hq.desc_moe_fp8_blockwise(E, N, K)
        w = torch.from_numpy(rng.standard_normal((E, K, N), dtype=np.float32) * 60).clamp(-448, 448).to(torch.float8_e4m3fn)
        self.w, self.sw = w.double().numpy(), np.exp(rng.standard_normal((E, K // 128, -(-N // 128)), dtype=np.float32)) / 60
        wp, sp, _ = hq.hq_repack(self.desc, w.view(torch.uint8).numpy(), self.sw)
        self.wp, self.sp = torch.from_numpy(wp).cuda(), torch.from_numpy(sp).cuda()

    def rows(self, n, seed):
        rng = np.random.default_rng([seed, n])
        a = torch.from_numpy(rng.standard_normal((n, self.K), dtype=np.float32) * 60).clamp(-448, 448).to(torch.float8_e4m3fn)
        return a.cuda(), torch.from_numpy(np.exp(rng.standard_normal((n, self.K // 128), dtype=np.float32)) / 60).cuda()

    def call(self, mode, T, k, a, sa, ids, offsets, out=None, ws=None, stream=None):
        n = hq.hq_workspace_bytes(self.desc, T, k)
        if ws is None:
            ws = torch.full((n + 64,), 0x7B, dtype=torch.uint8, device="cuda")
        own = out is None
        if own:
            out = torch.full((T * k * self.N + 64,), 3.0, dtype=torch.bfloat16, device="cuda")
        hq.hq_moe_gemm(self.desc, mode, T, k, a, sa, ids, offsets, self.wp, self.sp, None, out, ws, n, stream=stream)
        if own:
            torch.cuda.synchronize()
            assert (out[T * k * self.N:] == 3.0).all() and (ws[n:] == 0x7B).all(), "written behind a buffer"
        return out[:T * k * self.N].view(T * k, self.N)

    def check(self, got, a, sa, rows, experts):
        """One rounding to bf16; what the 8-bit MFMA cuts off inside 8 neighbouring K (7 * 2^-13 of their largest
        product); in fp32 the sums of a block's 16 such groups, its scale (two products) and the sum over blocks."""
        want, S, G = ol.experts_f8(f64(a)[rows], f64(sa)[rows], self.w, self.sw, experts)
        bound = np.abs(want) * 2.0 ** -8 + G * 7 * 2.0 ** -13 + S * (16 + 3 + self.K // 128) * 2.0 ** -24
        assert (np.abs(f64(got) - want) <= bound).all(), (np.abs(f64(got) - want) / bound).max()


def both_ways(x, T, k, ids, seed):
    """Indexed and grouped on the same routes."""
    E = x.E
    flat = ids.reshape(-1)
    a, sa = x.rows(T, seed)
    dev = torch.from_numpy(np.ascontiguousarray(ids, dtype=np.int32)).cuda()
    got = x.call(hq.HQ_MOE_INDEXED, T, k, a, sa, dev, None)
    x.check(got, a, sa, np.arange(T * k) // k, flat)
    order = np.argsort(flat, kind="stable")
    start = np.zeros(E + 1, np.int32)
    start[1:] = np.cumsum(np.bincount(flat, minlength=E))
    srt = torch.from_numpy(order.astype(np.int32)).cuda()
    ga, gs = torch.empty(T * k, x.K, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(T * k, x.K // 128, device="cuda")
    hq.hq_moe_gather(hq.HQ_DT_FP8_E4M3, T, k, x.K, a, srt, ga)
    hq.hq_moe_gather(hq.HQ_DT_FP32, T, k, x.K // 128, sa, srt, gs)
    assert torch.equal(ga.view(torch.uint8), a.view(torch.uint8)[torch.from_numpy(order // k).cuda()]) and torch.equal(gs, sa[torch.from_numpy(order // k).cuda()])
    grouped = x.call(hq.HQ_MOE_GROUPED, T, k, ga, gs, None, torch.from_numpy(start).cuda())
    # a row's sums do not depend on its place
    assert torch.equal(grouped, got[torch.from_numpy(order).cuda()])


# one pair and up; up to 64 pairs and above (where the routing changes); counts around a tile's 16, 32, 64 and 128 rows
@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 2, 8), (2, 3, 8), (7, 4, 16), (16, 4, 8), (13, 5, 8), (17, 4, 8), (63, 1, 3), (64, 1, 1), (65, 1, 1),
                                   (200, 2, 4), (129, 8, 8), (300, 3, 200), (1500, 2, 5)])
@pytest.mark.parametrize("N,K", [(256, 256), (200, 640)])
def test_routes_and_counts(T, k, E, N, K):
    note(f"experts f8 T={T} k={k} E={E} N={N} K={K}")
    x = Experts(E, N, K, seed=T)
    both_ways(x, T, k, syn.zipf_topk(T, 5, T, E, k), T)


@pytest.mark.parametrize("N", [1, 15, 16, 17, 127, 128, 129, 1000])
@pytest.mark.parametrize("T", [5, 90])
def test_column_counts(N, T):
    note(f"experts f8 N={N} T={T}")
    both_ways(Experts(4, N, 384, seed=N), T, 2, syn.zipf_topk(T, 5, T, 4, 2), 1)


@pytest.mark.parametrize("K", [128, 256, 384, 512, 640, 8064, 8192, 8320, 8448, 16512])
@pytest.mark.parametrize("T", [3, 40, 150])
def test_depths(K, T):
    """Depths around the pipeline's length and the blocks of scales held at a time."""
    note(f"experts f8 K={K} T={T}")
    both_ways(Experts(2, 144, K, seed=K), T, 1, syn.zipf_topk(T, 5, T, 2, 1), 2)


@pytest.mark.parametrize("rows", [1, 15, 16, 17, 31, 32, 33, 48, 63, 64, 65, 80, 127, 128, 129, 192, 255, 256, 257, 511, 700])
def test_rows_of_one_expert(rows):
    """All rows on the last of three experts, the others empty."""
    note(f"experts f8 rows={rows}")
    x = Experts(3, 272, 512, seed=rows)
    both_ways(x, rows, 1, np.full((rows, 1), 2, np.int32), 3)


def test_many_pairs():
    """More pairs than one routing workgroup takes."""
    T, k, E = 2500, 4, 12
    note(f"experts f8 T={T} k={k} E={E}")
    both_ways(Experts(E, 128, 256), T, k, syn.zipf_topk(T, 5, T, E, k), 4)


def test_rows_do_not_depend_on_the_batch():
    """A token's rows are the same bits alone, in a small batch and in a large one."""
    note("experts f8 batch independence")
    x = Experts(4, 384, 1024)
    a, sa = x.rows(600, 5)
    ids = torch.from_numpy(syn.zipf_topk(1, 5, 600, 4, 2).astype(np.int32)).cuda()
    whole = x.call(hq.HQ_MOE_INDEXED, 600, 2, a, sa, ids, None)
    for T in (1, 5, 31, 33, 150):
        part = x.call(hq.HQ_MOE_INDEXED, T, 2, a[:T].contiguous(), sa[:T].contiguous(), ids[:T].contiguous(), None)
        assert torch.equal(part, whole[:2 * T]), T


@pytest.mark.parametrize("T", [6, 120])
def test_ids_outside_and_repeated(T):
    """Rows of an id outside are left as they were; an expert named twice by a token answers twice."""
    note(f"experts f8 odd ids T={T}")
    x = Experts(4, 160, 256)
    a, sa = x.rows(T, 6)
    ids = np.random.default_rng(0).integers(0, 4, (T, 3)).astype(np.int32)
    ids[1] = [2, 2, 2]
    ids[0, 1], ids[3, 0], ids[5, 2] = -1, 4, 1 << 30
    out = torch.full((T * 3, 160), 9.0, dtype=torch.bfloat16, device="cuda")
    x.call(hq.HQ_MOE_INDEXED, T, 3, a, sa, torch.from_numpy(ids).cuda(), None, out=out)
    torch.cuda.synchronize()
    flat = ids.reshape(-1)
    good = np.nonzero((flat >= 0) & (flat < 4))[0]
    assert (out[torch.from_numpy(np.nonzero((flat < 0) | (flat >= 4))[0]).cuda()] == 9.0).all()
    x.check(out[torch.from_numpy(good).cuda()], a, sa, good // 3, flat[good])
    assert torch.equal(out[3], out[4]) and torch.equal(out[4], out[5])


@pytest.mark.parametrize("T", [4, 100])
def test_offsets_that_are_malformed_stay_inside(T):
    """Offsets past the rows, falling ones, negative ones: no row outside is touched."""
    note(f"experts f8 malformed offsets T={T}")
    x = Experts(4, 160, 256)
    a, sa = x.rows(T, 7)
    for off in ([0, T, 3 * T, 1 << 30, 1 << 30], [-9, 2, 1, T, T], [T, 0, 0, 0, 0], [0, T, 0, T, T]):
        x.call(hq.HQ_MOE_GROUPED, T, 1, a, sa, None, torch.tensor(off, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("T", [3, 200])
def test_nan_stays_in_its_row(T):
    note(f"experts f8 NaN T={T}")
    x = Experts(2, 160, 384)
    a, sa = x.rows(T, 8)
    ids = torch.from_numpy(np.arange(T, dtype=np.int32) % 2).cuda()
    clean = x.call(hq.HQ_MOE_INDEXED, T, 1, a, sa, ids, None).clone()
    a.view(torch.uint8)[1, 200] = 0x7F
    got = x.call(hq.HQ_MOE_INDEXED, T, 1, a, sa, ids, None)
    assert got[1].isnan().all()
    got[1] = clean[1]
    assert torch.equal(got, clean)
    # ... and a NaN scale
    a.view(torch.uint8)[1, 200] = 0
    sa[2, 1] = torch.nan
    assert x.call(hq.HQ_MOE_INDEXED, T, 1, a, sa, ids, None)[2].isnan().all()


@pytest.mark.parametrize("T,k", [(5, 2), (300, 2)])
def test_captured_with_its_workspace(T, k):
    """In a graph on a side stream, replayed with new routes; the workspace is used by eager calls in between."""
    note(f"experts f8 captured T={T}")
    x = Experts(6, 256, 512)
    a, sa = x.rows(T, 9)
    ids = torch.from_numpy(syn.zipf_topk(2, 5, T, 6, k).astype(np.int32)).cuda()
    n = hq.hq_workspace_bytes(x.desc, T, k)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    out = torch.empty(T * k, 256, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        x.call(hq.HQ_MOE_INDEXED, T, k, a, sa, ids, None, out=out, ws=ws)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        x.call(hq.HQ_MOE_INDEXED, T, k, a, sa, ids, None, out=out, ws=ws)
    for i in range(3):
        ids.copy_(torch.from_numpy(syn.zipf_topk(3 + i, 5, T, 6, k).astype(np.int32)))
        g.replay()
        torch.cuda.synchronize()
        kept = out.clone()
        eager = torch.empty_like(out)
        x.call(hq.HQ_MOE_INDEXED, T, k, a, sa, ids, None, out=eager, ws=ws)
        torch.cuda.synchronize()
        assert torch.equal(kept, eager)
