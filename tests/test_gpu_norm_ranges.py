"""The norm of rows whose squares leave fp32's range at either end: the formula's values."""
import numpy as np
import pytest
import torch

from gpu_util import note
from layer_util import FORMS, NORM_DELTA, check_rows, f64, run_norm
from oracle import layer as ol

pytestmark = pytest.mark.gpu
ANY = ["same", "f8_token", "i8_token"]
# sizes of a row's values (bf16): squares that are 0 or denormals, values that are denormals, and squares past 2^128
SIZES = [1e-19, 2e-23, 1e-30, 1e-37, 2e-39, 3e-40, 4e18, 3e19, 1e30, 2e37]


def made(K, odd=False):
    """A row for each size and, between them, ordinary rows."""
    g = torch.Generator().manual_seed(K)
    x = torch.randn(2 * len(SIZES), K, generator=g).clamp(-4, 4)
    x[::2] *= torch.tensor(SIZES, dtype=torch.float64)[:, None]
    return x.to(torch.bfloat16)


def weight(K):
    return 1 + 0.2 * torch.randn(K, generator=torch.Generator().manual_seed(3))


@pytest.mark.parametrize("form,K", [(f, k) for f in FORMS for k in (128, 384, 2048, 4096, 7168, 16384, 16512)] + [(f, k) for f in ANY for k in (1, 9, 777, 4001, 8193)])
def test_rows_of_every_size_with_eps_0(form, K):
    note(f"norm ranges {form} K={K}")
    x, w = made(K), weight(K)
    _, y = ol.rms_norm(f64(x), None, f64(w), 0.0)
    assert np.isfinite(y).all() or K == 1
    got = run_norm(form, "bf16", x.cuda(), None, w.cuda(), len(x), K, eps=0.0)
    torch.cuda.synchronize()
    check_rows(form, "bf16", y, NORM_DELTA, *got)
    # ... and the ordinary rows have the bits that they have alone
    alone = run_norm(form, "bf16", x[1::2].contiguous().cuda(), None, w.cuda(), len(x) // 2, K, eps=0.0)
    torch.cuda.synchronize()
    for buf, n, one, m in ((got[0], got[2], alone[0], alone[2]), (got[1], got[3], alone[1], alone[3])):
        if buf is not None:
            assert torch.equal(buf[:n].view(len(x), -1)[1::2], one[:m].view(len(x) // 2, -1))


@pytest.mark.parametrize("eps", [1e-45, 1e-40, 1e-35, 1e-30, 1e-20, 1e-6, 1e10])
@pytest.mark.parametrize("form,K", [("same", 384), ("f8_token", 777), ("f8_block", 7168)])
def test_rows_of_every_size_with_an_eps(form, K, eps):
    """eps beside the squares' mean, at every ratio."""
    note(f"norm ranges {form} K={K} eps={eps}")
    x, w = made(K), weight(K)
    _, y = ol.rms_norm(f64(x), None, f64(w), float(np.float32(eps)))
    out, scale, n, ns = run_norm(form, "bf16", x.cuda(), None, w.cuda(), len(x), K, eps=eps)
    torch.cuda.synchronize()
    # (rows whose values or scales are denormals are off by units of 2^-149: not by a share of them)
    keep = np.abs(y).max(1) > 2.0 ** -100 * 448
    assert keep.sum() >= len(x) // 2
    each, per = n // len(x), ns // len(x)
    rows = torch.from_numpy(np.nonzero(keep)[0]).cuda()
    pick = lambda b, k: torch.cat([b[:k * len(x)].view(len(x), k)[rows].reshape(-1), b[:0]]) if b is not None else None  # noqa: E731
    kept = y[keep]
    if form == "same":  # bf16's own denormals
        kept = np.where(np.abs(kept) < 2.0 ** -126, 0, kept)
        assert (np.abs(y[keep] - kept) < 2.0 ** -126).all()
    check_rows(form, "bf16", kept, NORM_DELTA, pick(out, each), pick(scale, per), int(rows.numel()) * each, int(rows.numel()) * per)


@pytest.mark.parametrize("K", [384, 777, 4096])
def test_sum_with_a_residual_is_stored_as_it_is(K):
    note(f"norm ranges residual K={K}")
    x, r, w = made(K), made(K).flip(1).contiguous(), weight(K)
    total = torch.empty(len(x), K, dtype=torch.bfloat16, device="cuda")
    got = run_norm("same", "bf16", x.cuda(), r.cuda(), w.cuda(), len(x), K, eps=0.0, sum_out=total)
    torch.cuda.synchronize()
    h, y = ol.rms_norm(f64(x), f64(r), f64(w), 0.0)
    big = np.abs(h) > 2.0 ** -126
    assert (np.abs(f64(total) - h)[big] <= (np.abs(h) * (2.0 ** -8 + 2.0 ** -23))[big]).all()
    check_rows("same", "bf16", y, NORM_DELTA, *got)  # (h's own rounding is one of those that it counts)


def test_zeros_and_what_is_not_finite():
    """A row of zeros is 0 / 0 with eps 0, zeros with another; an infinity makes its row's others 0, itself NaN."""
    note("norm ranges zeros")
    K = 256
    x = torch.ones(4, K)
    x[0], x[1, 7], x[2, 9] = 0, torch.inf, torch.nan
    x[3] = 1e38
    x[1, 8] = 1e38
    for eps in (0.0, 1e-6):
        out, _, n, _ = run_norm("same", "bf16", x.to(torch.bfloat16).cuda(), None, torch.ones(K).cuda(), 4, K, eps=eps)
        torch.cuda.synchronize()
        y = f64(out[:n].view(torch.bfloat16).view(4, K))
        assert np.isnan(y[0]).all() if eps == 0 else (y[0] == 0).all()
        assert np.isnan(y[1, 7]) and (np.delete(y[1], 7) == 0).all() and np.isnan(y[2]).all()
        assert (np.abs(y[3] - 1) <= 2.0 ** -8).all()
