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


# ------------------------------------------------------ values at the ends of the types

FORMS = {"token": dict(S=300, last=[299, 77]), "ragged": dict(S=300, last=[280, 9], counts=[180, 3]),
         "window": dict(S=300, last=[280, 9], counts=[180, 3], window=50, sinks=3),
         "shared": dict(S=40, last=[39, 5, 20], shared=260)}


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype,D", [("f16", 64), ("f16", 128), ("f16", 256), ("bf16", 128)])
def test_the_largest_values_stay_finite(form, dtype, D):
    """A mean of the type's largest value (bf16: 2^80) is that value: weights that are rounded
    up do not carry it beyond."""
    def edit(c):
        top = 65504.0 if dtype == "f16" else 2.0 ** 80
        for x in (c.v, c.vp):
            if x is not None:
                x[:] = top
                x[..., 1::2] = -top
        c.q *= 2
    c = Case(dtype, 8, 2, D, seed=41, edit=edit, **FORMS[form])
    got = c.run()
    assert bool(torch.isfinite(got).all()), int((~torch.isfinite(got)).sum())
    c.check(got)
