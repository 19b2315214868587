"""What the example block refuses (no GPU): a step that its buffers do not hold ends
in an error before anything is launched, and leaves its state as it was."""
import os
import sys
from types import SimpleNamespace

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

HIDDEN = 32


def block(lens=(0, 0, 0, 0), free=10, prefix=0):
    """The host's side of a block: 4 requests, 20 tokens a step, a context of 64, pages of 8 tokens."""
    from served_block import ServedBlock
    b = ServedBlock.__new__(ServedBlock)
    b.qkv = SimpleNamespace(K=HIDDEN)
    b.block, b.lens, b.free, b.prefix_len = 8, list(lens), torch.arange(free), prefix
    b.positions, b.cached, b.table = torch.zeros(20), torch.zeros(4), torch.zeros(64, 16)
    return b


def rows(n, dtype=torch.bfloat16, hidden=HIDDEN):
    return torch.zeros(n, hidden, dtype=dtype)


@pytest.mark.parametrize("state,x,new", [
    (dict(), rows(21), [21]),                                         # more tokens than a step holds
    (dict(), rows(5), [1] * 5),                                       # more requests
    (dict(), rows(0), []), (dict(), rows(0), [0, 0]),                 # none
    (dict(), rows(4), [3]), (dict(), rows(2), [3, -1]),               # rows that are not the new tokens'
    (dict(), rows(3, hidden=HIDDEN - 1), [3]), (dict(), rows(3, torch.float32), [3]),
    (dict(), rows(3, hidden=2 * HIDDEN)[:, :HIDDEN], [3]),            # not contiguous
    (dict(), rows(3).to("meta"), [3]),                                # on another device
    (dict(lens=(60, 0, 0, 0)), rows(5), [5]),                         # past the context
    (dict(lens=(40, 0, 0, 0), prefix=20), rows(5), [5]),
    (dict(lens=(8, 0, 0, 0), free=1), rows(10), [1, 9]),              # three pages, one free
])
def test_refusals(state, x, new):
    b = block(**state)
    before = list(b.lens), b.free.clone()
    with pytest.raises(ValueError):
        b.step(x, new)
    assert b.lens == before[0] and torch.equal(b.free, before[1])


def test_the_limits_are_admitted():
    assert block().admit(rows(20), [5, 5, 5, 5]) == ([5, 5, 5, 5], 4)
    assert block(lens=(40, 7, 0, 0), prefix=20, free=1).admit(rows(5), [4, 1]) == ([44, 8], 1)


def test_a_prefix_comes_first():
    with pytest.raises(ValueError):
        block(lens=(1, 0, 0, 0)).share_prefix(rows(3))
    with pytest.raises(ValueError):
        block(prefix=5).share_prefix(rows(3))
    with pytest.raises(ValueError):
        block().share_prefix(rows(0))
