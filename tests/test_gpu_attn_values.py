"""GPU attention at values where roundings or infinities decide: long flat tails
behind one strong key, rows whose scores are all minus infinity, caps of any size."""
import numpy as np
import pytest
import torch

from gpu_util import note
from kv_util import DT, TINY, U, AttnCase

pytestmark = pytest.mark.gpu


def place(c, side, r, i):
    """(page, slot) of the own key i of request r."""
    return int(c.table[r, i // c.block]), i % c.block


# ---------------------------------------------------------------------------
# weights far below the largest
# ---------------------------------------------------------------------------

def flat_tail(lens, new, cache, **kw):
    """Key 0 of each request has a score of 18.75, all others 0: their weights are
    2^-27 of its own.  Values are 1 in element 1 of key 0 and 256 in element 0 of
    the others."""
    c = AttnCase(lens, new, 4, 1, 64, "fp16", cache, **kw)
    c.q.zero_()
    c.q[..., 0] = 12.5
    c.scales = [torch.ones(1) if cache == "fp8" else None for _ in range(2)]
    k, v = torch.zeros(c.store[0].shape), torch.zeros(c.store[1].shape)
    v[..., 0] = 256.0
    for r in range(len(lens)):
        b, s = place(c, 0, r, 0)
        k[b, s, 0, 0] = 12.0
        v[b, s, 0, 0], v[b, s, 0, 1] = 0.0, 1.0
    c.store = [k.to(DT[cache]), v.to(DT[cache])]
    return c


@pytest.mark.parametrize("cache", ["fp16", "fp8"])
@pytest.mark.parametrize("lens,new", [([300], [1]), ([5000], [1]), ([600], [100]), ([40, 700, 90], [1, 5, 30])])
def test_flat_tail_keeps_its_mass_in_fp16(lens, new, cache):
    """The largest weight of a row is held as 2^7 or more, so a weight errs by at most half the
    smallest 16-bit step, 2^-25, over 2^7, of the largest, however small it is."""
    note(f"attn flat tail {lens} {new} {cache}")
    c = flat_tail(lens, new, cache)
    got, ls, _ = c.run()
    out, lse, (mass, qk, seen, vmax) = c.oracle()
    u = U["fp16"]
    es = 2.0 ** -24 * (c.D + 8) * qk + 2.0 ** -22 * (1 + np.abs(lse))
    rel = (u + 2 * es + 2.0 ** -21 + (seen + 64) * 2.0 ** -24)[..., None]
    tol = rel * mass + (seen * 2.0 ** -32 * vmax)[..., None] + u * np.abs(out) + TINY["fp16"]
    assert out[-1, 0, 0] > 8 * tol[-1, 0, 0]  # the tail is there to be seen
    err = np.abs(got - out)
    assert (err <= tol).all(), float((err / tol).max())
    assert (np.abs(ls - lse) <= es + 2.0 ** -20 + (seen + 64) * 2.0 ** -24).all()


# ---------------------------------------------------------------------------
# scores of minus infinity
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("lens,new,prefix", [([300], [1], 0), ([4000], [1], 0), ([200], [120], 0), ([4000, 1500, 1500], [1, 40, 3], 900)])
def test_rows_whose_scores_are_all_minus_infinity(dtype, lens, new, prefix):
    """A row that sees keys, all of weight 0 / 0, has no softmax: NaN, as the formula gives, and not
    the zeros of a row that sees none.  One finite score among them takes all the weight."""
    note(f"attn minus infinity {dtype} {lens} prefix {prefix}")
    c = AttnCase(lens, new, 4, 1, 64, dtype, prefix=prefix, seed=2)
    c.q[..., 0] = 1.0
    c.store[0][..., 0] = -float("inf")
    got, ls, _ = c.run()
    assert np.isnan(got).all() and np.isnan(ls).all()
    b, s = place(c, 0, 0, 77)  # of the first request: its tokens that see it
    c.store[0][b, s, 0, 0] = 0.0
    got, ls, _ = c.run()
    out, lse, _ = c.oracle()
    assert np.array_equal(np.isnan(got), np.isnan(out)) and np.array_equal(np.isnan(ls), np.isnan(lse))
    seen = ~np.isnan(lse)
    assert seen.any()
    np.testing.assert_array_equal(got[seen], out[seen])  # one key's value, held in the output's type
    assert (np.abs(ls[seen] - lse[seen]) <= 2.0 ** -20 * (1 + np.abs(lse[seen]))).all()


def test_rows_without_keys_next_to_rows_of_minus_infinity():
    note("attn minus infinity, no keys")
    c = AttnCase([2, 40], [5, 1], 4, 2, 64, "bf16", seed=1)
    c.q[..., 0] = 1.0
    c.store[0][..., 0] = -float("inf")
    got, ls, _ = c.run()
    assert (got[:3] == 0).all() and np.isneginf(ls[:3]).all()
    assert np.isnan(got[3:]).all() and np.isnan(ls[3:]).all()


# ---------------------------------------------------------------------------
# caps far above the scores
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("cache", ["fp16", "fp8"])
@pytest.mark.parametrize("softcap", [0.5, 50.0, 1e4, 1e6, 1e12])
@pytest.mark.parametrize("lens,new,prefix", [([300, 41], [1, 9], 50), ([3000, 900], [1, 2], 700), ([260], [130], 0)])
def test_cap_errs_by_a_share_of_the_score(softcap, cache, lens, new, prefix):
    """cap * tanh(x / cap) to 2^-19 of x, whatever the cap (tanh of a quarter and
    more to some 2^-22, below that by its series)."""
    note(f"attn cap {softcap} {cache} {lens} {prefix}")
    c = AttnCase(lens, new, 8, 2, 64, "fp16", cache, prefix=prefix, softcap=softcap, q_gain=3.0, seed=2)
    got, ls, _ = c.run()
    out, lse, (mass, qk, seen, vmax) = c.oracle()
    u = U["fp16"]
    es = (2.0 ** -24 * (c.D + 8) + 2.0 ** -19) * qk + 2.0 ** -22 * (1 + np.abs(lse))
    tol = (u + 2 * es + 2.0 ** -21 + (seen + 64) * 2.0 ** -24)[..., None] * mass + (seen * TINY["fp16"] * vmax)[..., None] + u * np.abs(out) + TINY["fp16"]
    err = np.abs(got - out)
    assert (err <= tol).all(), float((err / tol).max())
    e2, ltol = np.abs(ls - lse), es + 2.0 ** -20 + (seen + 64) * 2.0 ** -24
    assert (e2 <= ltol).all(), float((e2 / ltol).max())


def test_cap_beyond_all_scores_changes_nothing():
    note("attn cap 1e30")
    a = AttnCase([300, 41], [1, 40], 8, 2, 64, "bf16", prefix=50, softcap=1e30, seed=2)
    b = AttnCase([300, 41], [1, 40], 8, 2, 64, "bf16", prefix=50, seed=2)
    x, y = a.run(), b.run()
    assert np.array_equal(x[0], y[0]) and np.array_equal(x[1], y[1])
