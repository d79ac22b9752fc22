"""Attention of one token holds its softmax weights in two 16-bit numbers: inputs on which one
would be out of tolerance (test_attend_weights_host.py)."""
from __future__ import annotations

import pytest

import token_decode_attention_gb300 as dattn

from . import _attend_weights as aw
from .test_attend_weights_host import GROUPS

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from token_decode_attention_gb300 import build
    build.build()
    dattn.load()
    yield
    assert dattn.dattn_device_error(clear=True) == 0


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("group", GROUPS)
@pytest.mark.parametrize("D", [16, 128, 256])
def test_weights_of_one_token_keep_two_parts(dtype, group, D):
    c = aw.case(dtype, group, D, seed=50)
    ref, tol = aw.expected(c)
    err = (c.run()[0].double() - ref).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
