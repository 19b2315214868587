"""What the example layer refuses (no GPU): rows that its buffers do not hold."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def layer():
    from routed_layer import RoutedLayer
    x = RoutedLayer.__new__(RoutedLayer)
    x.hidden, x.max_tokens, x.out = 32, 20, torch.zeros(20, 32)
    return x


def rows(n, hidden=32, dtype=torch.bfloat16):
    return torch.zeros(n, hidden, dtype=dtype)


@pytest.mark.parametrize("x,residual", [(rows(21), rows(21)), (rows(0), rows(0)), (rows(3, 31), rows(3)), (rows(3), rows(3, 31)), (rows(3), rows(4)),
                                        (rows(3, dtype=torch.float32), rows(3)), (rows(3), rows(3, dtype=torch.float16)), (rows(3, 64)[:, :32], rows(3)),
                                        (rows(3), rows(6)[::2]), (rows(3).to("meta"), rows(3)), (rows(3), rows(3).to("meta")), (rows(3)[0], rows(3))])
def test_refusals(x, residual):
    with pytest.raises(ValueError):
        layer().step(x, residual)


def test_the_limits_are_admitted():
    assert layer().admit(rows(20), rows(20)) == 20 and layer().admit(rows(1), rows(1)) == 1
