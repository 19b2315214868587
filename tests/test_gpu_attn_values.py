"""GPU attention at values where roundings or infinities decide: long flat tails
behind one strong key."""
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
