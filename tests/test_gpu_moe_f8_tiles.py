"""FP8 experts in tiles of more than the fewest rows: several unequal experts, more m-tiles of an expert than a group,
columns that end inside a tile, both modes, against the definition in 64 bits."""
import numpy as np
import pytest
import torch

from bit_quantized_gemm_w4a16_amd import hq
from gpu_util import note
from layer_util import f64
from test_gpu_moe_f8 import Experts

pytestmark = pytest.mark.gpu


def tile_rows(P, E, N):
    """Rows of a tile: as few (96 and up, in steps of 32, to 256) as give each of 256 CUs one tile at most, by the mean."""
    held, rows = min(E, P), 96
    while rows < 256 and held * -(-P // (held * rows)) * -(-N // 256) > 256:
        rows += 32
    return rows


def heights(c, most):
    """Subtiles of 32 rows of the tiles that c rows are cut into, evenly."""
    n = -(-c // most)
    step = -(--(-c // 32) // n)
    return {step, -(-(c - (n - 1) * step * 32) // 32)} if n else set()


def sample(counts):
    """Rows (of those sorted by expert) at the ends of every 32 and some between, fewer of the larger experts."""
    rows, first = [], 0
    for c in counts:
        at = {0, 1, c // 2, c - 2, c - 1} | {r for b in range(0, c, 32 * max(1, c // 600)) for r in (b - 1, b)}
        rows += [first + r for r in sorted(at) if 0 <= r < c]
        first += c
    return np.array(rows)


# tokens, each to one of the experts by these shares; every height of a tile (3 to 8 subtiles) is among them
CASES = [(2049, (1,), 256), (1900, (0.9, 0.06, 0.04), 256), (1200, (0.55, 0.35, 0.1), 224), (1000, (0.7, 0.29, 0.01), 192), (800, (0.4, 0.35, 0.25), 160),
         (700, (0.05, 0.9, 0.05), 128), (900, (1,), 160), (1121, (1,), 192), (1500, (1,), 224), (680, (1,), 128)]


@pytest.mark.parametrize("T,shares,want,N,K", [(*c, *[(8199, 384), (8200, 256), (8196, 128), (8448, 640)][(i + j) % 4]) for i, c in enumerate(CASES) for j in (0, 1)])
def test_heights_columns_and_experts(T, shares, want, N, K):
    E = len(shares)
    assert tile_rows(T, E, N) == want
    note(f"experts f8 tiles T={T} E={E} N={N} K={K} rows={want}")
    x = Experts(E, N, K, seed=T)
    ids = np.random.default_rng([T, N]).choice(E, T, p=shares).astype(np.int32)
    ids[:E] = np.arange(E)
    order = np.argsort(ids, kind="stable")
    counts = np.bincount(ids, minlength=E)
    a, sa = x.rows(T, K)
    got = x.call(hq.HQ_MOE_INDEXED, T, 1, a, sa, torch.from_numpy(ids[:, None].copy()).cuda(), None)
    rows = order[sample(counts)]
    x.check(got[torch.from_numpy(rows).cuda()], a, sa, rows, ids[rows])
    # the same rows sorted by expert: the same bits
    at = torch.from_numpy(order).cuda()
    start = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).cuda()
    assert torch.equal(x.call(hq.HQ_MOE_GROUPED, T, 1, a.view(torch.uint8)[at].view(a.dtype), sa[at].contiguous(), None, start), got[at])
    # ... and by themselves, in tiles of the fewest rows
    few = rows[:90]
    alone = x.call(hq.HQ_MOE_INDEXED, len(few), 1, a.view(torch.uint8)[torch.from_numpy(few).cuda()].view(a.dtype), sa[torch.from_numpy(few).cuda()].contiguous(),
                   torch.from_numpy(ids[few][:, None].copy()).cuda(), None)
    assert torch.equal(alone, got[torch.from_numpy(few).cuda()])


def test_every_height_is_met():
    """(by the rule that the cases are checked against, on the counts that they draw)"""
    met = set()
    for T, shares, want in CASES:
        for N in (8199, 8200, 8196, 8448):
            ids = np.random.default_rng([T, N]).choice(len(shares), T, p=shares)
            for c in np.bincount(ids, minlength=len(shares)):
                met |= heights(int(c), want) if N == 8199 else set()
    assert met >= {3, 4, 5, 6, 7, 8}, met


def test_rows_left_out_of_large_tiles():
    """Ids outside among the rows of large tiles, two experts a token: those rows of D stay."""
    note("experts f8 tiles with ids outside")
    E, N, K, T, k = 3, 8200, 256, 800, 2
    assert tile_rows(T * k, E, N) == 256
    x = Experts(E, N, K)
    ids = np.random.default_rng(1).choice([-1, 0, 1, 2, 3, 1 << 30], (T, k), p=[0.1, 0.6, 0.1, 0.1, 0.05, 0.05]).astype(np.int32)
    a, sa = x.rows(T, 1)
    out = torch.full((T * k * N,), 9.0, dtype=torch.bfloat16, device="cuda")
    got = x.call(hq.HQ_MOE_INDEXED, T, k, a, sa, torch.from_numpy(ids).cuda(), None, out=out)
    torch.cuda.synchronize()
    flat = ids.reshape(-1)
    good = np.nonzero((flat >= 0) & (flat < E))[0]
    assert (got[torch.from_numpy(np.nonzero((flat < 0) | (flat >= E))[0]).cuda()] == 9.0).all()
    rows = good[::17]
    x.check(got[torch.from_numpy(rows).cuda()], a, sa, rows // k, flat[rows])
