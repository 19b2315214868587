"""Routing where a workgroup's LDS passes 64 KB: thousands of experts in groups that fill no whole lanes."""
import pytest

from gpu_util import note
from test_gpu_route import bias_of, check, logits_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E,groups", [(3885, 35), (3900, 60), (3904, 61), (4032, 64), (4095, 63), (4095, 7)])
def test_groups_of_thousands_of_experts(E, groups):
    note(f"route LDS E={E} groups={groups}")
    for bias, sigmoid in ((None, False), (bias_of(1, E), True)):
        check(logits_of(2, 9, E), bias, 10, sigmoid=sigmoid, groups=groups, top_groups=min(5, groups), group_best=2)
