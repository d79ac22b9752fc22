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
@pytest.mark.parametrize("dtype,D,q,k", [
    ("f16", 64, 1536.0, 1536.0), ("f16", 128, 2048.0, 2560.0), ("f16", 128, -3000.0, 2500.0),
    ("f16", 128, 5120.0, 5120.0), ("f16", 256, 65504.0, 65504.0), ("f16", 128, -65504.0, 40000.0),
    ("bf16", 64, 2.0 ** 20, 3 * 2.0 ** 17), ("bf16", 128, 2.0 ** 50, 2.0 ** 50), ("bf16", 256, -2.0 ** 30, 2.0 ** 28)])
def test_equal_scores_of_any_size(form, dtype, D, q, k):
    """One key at every position: each weighs the same, however far from 0 its score lies.
    The result is a mean of V, |V| <= size; a weight is rounded once (eps / 2 of it), sums of
    n <= 300 terms are off by n 2^-24 each, the result is rounded once.

    All positions of a call but a shared prefix's are one kernel's, which adds the D equal
    products in one order, so their scores are the same whatever was rounded.  The prefix's and a
    sequence's own are two kernels': their sums agree where no partial sum needs rounding, that
    is where the odd part of q k times D fits 24 bits.  Where it does not (65504^2 = 2^10 x
    4190209: 22 bits, times 256) the scores may differ by D 2^-24 of 10^10, and with them the
    parts' weights as far as the general tolerance says; the result is finite all the same."""
    def edit(c):
        c.q[:] = q
        c.k[:] = k
        if c.kp is not None:
            c.kp[:] = k
    c = Case(dtype, 4, 2, D, seed=40, edit=edit, **FORMS[form])
    got = c.run()
    ref, general = c.expected()  # the scores are equal in 64 bits too
    half = torch.finfo(c.t).eps / 2
    size = max(float(x.double().abs().max()) for x in (c.v, c.vp) if x is not None)
    tol = size * (half + 2 * 300 * 2.0 ** -24)
    tol = tol + (ref.abs() + tol) * half + torch.finfo(c.t).tiny
    odd = int(abs(q)) * int(k)
    odd //= odd & -odd
    if form == "shared" and odd * D >= 2 ** 24:
        tol = torch.maximum(tol, general)
        assert bool(torch.isfinite(got).all())
    bad = ~((got.double() - ref).abs() <= tol)
    assert not bool(bad.any()), (int(bad.sum()), got[bad][0], ref[bad][0])


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
