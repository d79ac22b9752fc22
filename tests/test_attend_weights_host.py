"""The inputs of test_attend_weights_gpu.py tell weights of one 16-bit number from weights of two."""
from __future__ import annotations

import pytest

from . import _attend_weights as aw

GROUPS = (1, 4, 7, 8, 16)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("group", GROUPS)
@pytest.mark.parametrize("D", [16, 128, 256])
def test_one_part_is_out_of_tolerance_and_two_are_within(dtype, group, D):
    c = aw.case(dtype, group, D, seed=50)
    ref, tol = aw.expected(c)
    assert bool(((aw.modelled(c, 2) - ref).abs() <= tol).all())
    off = (aw.modelled(c, 1) - ref).abs() > tol
    assert bool(off.any(-1).all())  # in every query head
