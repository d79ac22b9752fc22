"""More calls of attention over a 16-bit cache against the definition in 64 bits: workspaces
at any allowed address, values at the ends of the types, tiles whose last block of channels is
not full, CTAs that take many items."""
from __future__ import annotations

import pytest
import torch

import token_decode_attention_gb300 as dattn
from token_decode_attention_gb300 import _native

from ._attend import TYPES, Case
from .test_attend_gpu import cases_of_calls, workspace_bytes

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from token_decode_attention_gb300 import build
    build.build()
    dattn.load()
    yield
    assert dattn.dattn_device_error(clear=True) == _native.OK


@pytest.mark.parametrize("offset", [16, 48])
@pytest.mark.parametrize("i", range(6))
def test_workspaces_on_16_bytes(i, offset):
    """A workspace need lie on 16 bytes only."""
    c = cases_of_calls()[i]
    n = workspace_bytes(c)
    first = c.run()
    ws = torch.full((max(n, 16) + 128,), 255, dtype=torch.uint8, device="cuda")
    assert ws.data_ptr() % 64 == 0
    out = c.call(c.cuda(), workspace=ws[offset: offset + max(n, 16)])
    assert torch.equal(out.cpu(), first)
    assert bool((ws[:offset] == 255).all()) and bool((ws[offset + max(n, 16):] == 255).all())
