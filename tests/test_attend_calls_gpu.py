"""More calls of attention over a 16-bit cache against the definition in 64 bits: workspaces
at any allowed address, values at the ends of the types, tiles whose last block of channels is
not full, CTAs that take many items."""
from __future__ import annotations

import pytest
import torch

import token_decode_attention_gb300 as dattn
from token_decode_attention_gb300 import _native

from ._attend import Case, half_step
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


# ------------------------------- tiles whose last block of channels is not full, long walks

def check_fast(c, got):
    """Case.check with a sequence's rows at once."""
    ref, tol = c.out0.double(), torch.zeros(c.out0.shape, dtype=torch.float64)
    group, t, half = c.H // c.Hk, 0, torch.finfo(c.t).eps / 2
    for b in range(c.B):
        n, end = (1 if c.counts is None else c.counts[b]), min(c.last[b], c.S - 1)
        if c.shared and not c.page:
            end += c.shared
        if n == 0:
            continue
        K, V = (x.double().repeat_interleave(group, 1).transpose(0, 1) for x in c.rows(b, range(end + 1)))
        q = c.q[t: t + n].double().transpose(0, 1)  # [H, n, D]
        p, j = torch.arange(end - n + 1, end + 1)[:, None], torch.arange(end + 1)
        sees = j <= p
        if c.window:
            sees &= (j > p - c.window) | (j < c.sinks)
        s = (q @ K.transpose(1, 2) / c.D ** 0.5).masked_fill(~sees, -float("inf"))
        w = torch.softmax(s, -1)
        r, size, m = w @ V, w @ V.abs(), sees.sum(-1)[:, None]
        dot = (q.abs() @ K.abs().transpose(1, 2) / c.D ** 0.5).masked_fill(~sees, 0).amax(-1, keepdim=True)
        most = s.masked_fill(~sees, 0).abs().amax(-1, keepdim=True)
        d = (c.D + 8) * 2.0 ** -24 * dot + 4 * 2.0 ** -24 * most + 2.0 ** -21
        e = size * (2 * (d + m * 2.0 ** -24) + half)
        if c.t is torch.float16:
            e = e + m * 2.0 ** -25 * V.abs().amax(1, keepdim=True)
        ref[t: t + n], tol[t: t + n] = r.transpose(0, 1), (e + half_step(r.abs() + e, c.t)).transpose(0, 1)
        t += n
    bad = ~((got.double() - ref).abs() <= tol)
    assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[0].tolist(), got[bad][0], ref[bad][0], tol[bad][0])


def test_the_fast_check_is_the_other():
    c = Case("f16", 4, 2, 72, 90, [80, 3, 89], counts=[50, 0, 7], window=30, sinks=2, pad=3, seed=42)
    got = c.run()
    check_fast(c, got)
    c.check(got)


@pytest.mark.parametrize("D", [8, 72, 80, 136, 200])
@pytest.mark.parametrize("page", [0, 16, 64])
@pytest.mark.parametrize("window,sinks", [(0, 0), (290, 5)])
def test_boxes_with_a_block_of_channels_in_part(D, page, window, sinks):
    """Whole key tiles inside the window come as boxes of 64 channels, the last one's zero filled."""
    c = Case("bf16" if D % 16 else "f16", 8, 2, D, 704, [700, 510], counts=[150, 3], page=page, window=window,
             sinks=sinks, seed=43)
    check_fast(c, c.run())


@pytest.mark.parametrize("D", [8, 72, 80, 136, 200])
@pytest.mark.parametrize("page", [0, 16, 64])
def test_boxes_of_a_shared_prefix_with_a_block_of_channels_in_part(D, page):
    if page:
        c = Case("f16", 8, 2, D, 768, [700, 640, 767, 512], page=page, shared=512, seed=44)
    else:
        c = Case("bf16", 8, 2, D, 50, [49, 0, 17], shared=517, seed=44)
    check_fast(c, c.run())


@pytest.mark.parametrize("dtype,H,Hk,D,counts", [
    ("bf16", 16, 1, 64, (3, 12, 1, 16, 8, 9, 20, 0, 16, 2)),    # 16 rows a token: one stack up to 8 tokens
    ("f16", 16, 1, 128, (12, 3, 16, 1, 9, 8, 2, 30)),
    ("f16", 12, 1, 72, (12, 3, 16, 1, 21, 11, 10, 2)),          # 12 rows a token: stacks end inside one
    ("bf16", 16, 2, 256, (3, 12, 1, 16, 8, 9)),                 # one stack always
])
@pytest.mark.parametrize("window,sinks,page", [(0, 0, 0), (100, 3, 16)])
def test_ctas_that_take_items_of_one_and_of_two_stacks_in_turn(dtype, H, Hk, D, counts, window, sinks, page):
    """Eight items and more for each CTA, of one and of two stacks in every order."""
    B = 1200
    counts = [counts[(i * 7 + i // 50) % len(counts)] for i in range(B)]
    last = [max(n, 1) - 1 + (i * 37) % (240 - n) for i, n in enumerate(counts)]
    c = Case(dtype, H, Hk, D, 240, last, counts=counts, window=window, sinks=sinks, page=page, seed=45)
    check_fast(c, c.run())


# -------------------------------------------------------------------- pinned host memory

@pytest.mark.parametrize("i", range(6))
def test_queries_positions_and_output_in_pinned_memory(i):
    """What a step brings from the host and takes back, of every form."""
    c = cases_of_calls()[i]
    first = c.run()
    d = c.cuda()
    for name in ("q", "pos", "offsets", "table"):
        if d[name] is not None:
            d[name] = d[name].cpu().pin_memory()
    host = torch.empty_like(c.out0).pin_memory()
    assert c.call(d, out=host) is host
    torch.cuda.synchronize()
    assert torch.equal(host, first)
    out = c.call(d)
    assert out.is_cuda and torch.equal(out.cpu(), first)


# ------------------------------------------------------------- values that are not finite

def prompt(n, H=32, Hk=8, D=128, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(46)
    q, k, v = (torch.randn(s, generator=g, device="cuda").to(dtype) for s in ((n, H, D), (1, n, Hk, D), (1, n, Hk, D)))
    pos, off = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([n - 1], [0, n]))
    return lambda **kw: dattn.attend(q, k, v, pos, token_offsets=off, **kw), q, k, v


@pytest.mark.parametrize("where", ["key", "value", "middle"])
def test_a_value_that_is_not_finite_costs_little(where):
    """A prompt whose tokens see a NaN takes about as long as one whose tokens see none: what
    rows are computed again for is hidden values alone.  (Position by position the whole
    prompt takes 400 times as long; the limit of 20 leaves room for a busy clock.)"""
    n = 4096
    call, q, k, v = prompt(n)
    first = call()

    def ms():
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        times = []
        for _ in range(5):
            start.record()
            call()
            end.record()
            end.synchronize()
            times.append(start.elapsed_time(end))
        return sorted(times)[2]
    plain = ms()
    at = n // 2 if where == "middle" else 0
    (k if where == "key" else v)[0, at, 2, 5] = float("nan")
    got = call()
    hit = torch.zeros_like(first, dtype=torch.bool)
    hit[at:, 8:12, slice(None) if where == "key" else 5] = True  # heads of key/value head 2
    assert bool(torch.isnan(got[hit]).all())
    assert torch.equal(got[~hit], first[~hit])
    assert ms() < 20 * plain


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("D", [64, 256])
def test_values_that_some_rows_of_an_item_see(bad, D):
    """The rows before a bad value, in its own item and the next, come out as without it."""
    n = 700
    call, q, k, v = prompt(n, 8, 2, D, torch.float16)
    first = call()
    for at in (0, 1, 30, 31, 333, 699):
        old = v[0, at, 1].clone()
        v[0, at, 1, 3] = bad
        got = call()
        assert not bool(torch.isfinite(got[at:, 4:, 3]).any())
        keep = torch.ones_like(first, dtype=torch.bool)
        keep[at:, 4:, 3] = False
        # rows that are computed again weigh in fp32 what the others round to f16: 2^-11 of a
        # weight, and the output's own rounding
        off = (got.double() - first.double()).abs()[keep]
        size = float(v[torch.isfinite(v)].abs().max())
        assert bool((off <= size * 2.0 ** -10 + 2.0 ** -10 * first.double().abs()[keep]).all())
        v[0, at, 1] = old
