"""Attention over a 16-bit cache against its definition in 64 bits: one token per sequence,
ragged batches of tokens, windows and sinks, and shared prefixes."""
from __future__ import annotations

import pytest
import torch

import token_decode_attention_gb300 as dattn
from token_decode_attention_gb300 import _native

from ._attend import TYPES, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from token_decode_attention_gb300 import build
    build.build()
    dattn.load()
    yield
    assert dattn.dattn_device_error(clear=True) == _native.OK


def error_is(status):
    assert dattn.dattn_device_error(clear=True) == status


# ------------------------------------------------------------ one token each

HEADS = [(1, 1), (4, 4), (8, 2), (10, 2), (16, 1), (34, 2)]


@pytest.mark.parametrize("H,Hk", HEADS)
@pytest.mark.parametrize("D", [8, 64, 72, 80, 128, 136, 256])
def test_token_heads_and_channels(H, Hk, D):
    dtype = "f16" if (H + D) % 16 else "bf16"
    Case(dtype, H, Hk, D, 50, [49, 0, 16, 31], seed=1).check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("S", [1, 2, 15, 16, 17, 33, 127, 129, 300])
def test_token_lengths(dtype, S):
    Case(dtype, 8, 2, 64, S, [S - 1, 0, S // 2, S // 3, S + 5, 2 ** 31 + 3, 2 ** 32 - 1], seed=2).check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 1), (7, 3), (16, 16), (17, 4), (40, 70), (64, 5),
                                          (200, 9), (2 ** 31 - 1, 2 ** 31 - 1), (5, 2 ** 31 - 1)])
@pytest.mark.parametrize("page", [0, 1, 7, 16])
def test_token_windows(dtype, window, sinks, page):
    Case(dtype, 4, 2, 64, 112, [111, 0, 1, 15, 16, 40, 63, 64, 80], page=page, window=window, sinks=sinks,
         seed=3).check()


@pytest.mark.parametrize("page,S", [(1, 40), (3, 39), (24, 240), (16, 256), (128, 256), (200, 400)])
@pytest.mark.parametrize("D", [64, 80, 256])
def test_token_pages(page, S, D):
    Case("bf16", 10, 2, D, S, [S - 1, 0, S // 2, page, page - 1], page=page, seed=4).check()


@pytest.mark.parametrize("window,sinks,page", [(0, 0, 0), (1024, 4, 0), (1500, 130, 48), (0, 0, 64)])
@pytest.mark.parametrize("dtype", TYPES)
def test_token_long(dtype, window, sinks, page):
    Case(dtype, 8, 1, 128, 4800, [4799, 2000], page=page, window=window, sinks=sinks, seed=5).check()


def test_token_many_sequences():
    Case("bf16", 4, 2, 64, 70, [(i * 37) % 70 for i in range(700)], window=33, sinks=2, seed=6).check()


# ------------------------------------------------------------ ragged batches

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("H,Hk,D", [(4, 4, 64), (8, 2, 128), (10, 2, 80), (16, 1, 256), (34, 2, 72), (3, 3, 8)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (9, 2)])
def test_ragged_heads_and_channels(dtype, H, Hk, D, window, sinks):
    Case(dtype, H, Hk, D, 70, [69, 3, 20, 40, 0], counts=[40, 4, 0, 13, 1], window=window, sinks=sinks,
         seed=7).check()


@pytest.mark.parametrize("page", [0, 1, 24, 64])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (1, 1), (5, 3), (64, 4), (100, 130), (129, 1),
                                          (2 ** 31 - 1, 7)])
def test_ragged_windows(page, window, sinks):
    # more than one tile of rows and of keys; a sequence that brings all, one, none
    Case("bf16", 4, 2, 64, 384, [300, 9, 17, 383, 255], counts=[301, 1, 0, 130, 3], page=page, window=window,
         sinks=sinks, pad=5, seed=8).check()


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 257])
def test_ragged_token_counts(n):
    Case("f16", 8, 2, 64, 300, [n - 1, 299], counts=[n, n], seed=9).check()


@pytest.mark.parametrize("dtype,D", [("f16", 64), ("bf16", 128), ("f16", 256)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (700, 4)])
def test_ragged_chunk_of_a_long_context(dtype, D, window, sinks):
    Case(dtype, 8, 2, D, 3500, [3400, 1111], counts=[40, 1], window=window, sinks=sinks, seed=10).check()


def test_ragged_many_single_tokens():
    Case("f16", 4, 2, 64, 64, [(i * 29) % 64 for i in range(300)], counts=[1] * 300, window=20, sinks=1,
         seed=11).check()


def test_positions_before_the_first_see_nothing():
    error_is(_native.OK)
    c = Case("f16", 4, 2, 64, 64, [2, 5], counts=[6, 6], seed=12)
    c.check()
    error_is(_native.ERR_BAD_POSITION)


def test_padding_rows_are_left():
    c = Case("bf16", 4, 2, 64, 64, [20], counts=[9], pad=150, seed=13)
    got = c.run()
    assert torch.equal(got[9:], c.out0[9:])
    c.check(got)


# ------------------------------------------------------------ shared prefixes

@pytest.mark.parametrize("H,Hk,D", [(4, 4, 64), (8, 2, 128), (10, 2, 80), (16, 1, 256), (34, 2, 72), (3, 3, 8)])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("page", [0, 24])
def test_shared_heads_and_channels(dtype, H, Hk, D, page):
    own = [0, 40, 17, 3]
    if page:
        Case(dtype, H, Hk, D, 144, [70 + x for x in own], page=page, shared=70, seed=14).check()
    else:
        Case(dtype, H, Hk, D, 41, own, shared=70, seed=14).check()


@pytest.mark.parametrize("shared", [1, 2, 127, 128, 129, 300, 1111])
@pytest.mark.parametrize("B", [1, 2, 33, 70])
def test_shared_lengths(shared, B):
    Case("bf16", 4, 1, 64, 30, [i % 31 for i in range(B)], shared=shared, seed=15).check()


@pytest.mark.parametrize("page,S,shared", [(1, 40, 20), (16, 320, 160), (16, 320, 155), (64, 256, 256),
                                           (24, 240, 1), (200, 400, 250)])
def test_shared_pages(page, S, shared):
    # tokens inside the shared positions, at their end, behind them
    last = [S - 1, 0, shared // 2, max(0, shared - 1), min(S - 1, shared), S + 9]
    Case("f16", 8, 2, 128, S, last, page=page, shared=shared, seed=16).check()


def test_shared_pages_of_other_rows_are_not_used():
    def edit(c):
        c.table[1:, : 64 // 16] = -1
    error_is(_native.OK)
    Case("f16", 4, 2, 64, 128, [100, 64, 127, 3], page=16, shared=64, seed=17, edit=edit).check()
    error_is(_native.OK)


# ------------------------------------------------------ values in odd places

def plant(c, b, p, k=None, v=None):
    at = c.at(b, p)
    if k is not None:
        c.k[at] = k
    if v is not None:
        c.v[at] = v


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 6e4])
@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("counts", [None, [1, 1, 1], [90, 0, 12]])
def test_what_no_token_sees_never_enters(bad, page, counts):
    """Rows behind the live ones, and between sinks and window, hold anything."""
    last = [120, 30, 200]

    def edit(c):
        for b, p in enumerate(last):
            n = 1 if counts is None else counts[b]
            for j in range(c.S):
                if j > p or (3 <= j <= p - (n - 1) - 20):
                    plant(c, b, j, bad, bad)
    Case("f16", 4, 2, 64, 256, last, counts=counts, page=page, window=20, sinks=3, seed=18, edit=edit).check()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("window", [0, 10])
def test_what_other_tokens_see_stays_theirs(bad, window):
    """A key and a value that are not finite reach the rows of the tokens that see them only."""
    for where in (0, 13, 40, 70):
        def edit(c):
            c.v[0, where, 0, 5] = bad
            c.k[0, where, 1, 7] = bad
        c = Case("bf16", 4, 2, 64, 80, [70], counts=[60], window=window, sinks=1, seed=19, edit=edit)
        got = c.run()
        ref, tol = c.expected()
        hit = torch.zeros(60, dtype=torch.bool)
        for i in range(60):
            p = 11 + i
            hit[i] = where <= p and (window == 0 or where > p - window or where < 1)
        fine = (got.double() - ref).abs() <= tol
        assert bool(fine[~hit].all())
        assert not bool(torch.isfinite(got[hit][:, :2, 5]).any())
        if bad != bad:
            assert bool(torch.isnan(got[hit][:, 2:]).all())


@pytest.mark.parametrize("shared", [40, 200])
def test_shared_rows_that_are_not_finite(shared):
    def edit(c):
        c.v[c.at(0, 30)][0, 3] = float("inf")  # tokens at 30 and later see it
        for p in range(260, 288):
            for b in range(3):
                plant(c, b, p, float("nan"), float("nan"))
    c = Case("f16", 4, 2, 64, 288, [20, 29, 250], page=24, shared=shared, seed=20, edit=edit)
    got = c.run()
    if shared == 200:  # the first two lie inside the shared positions
        c.check(got)
    ref, tol = c.expected()
    assert bool(((got.double() - ref).abs() <= tol)[:2].all())
    assert bool(torch.isinf(got[2, :2, 3]).all())


@pytest.mark.parametrize("counts", [None, [200, 1]])
@pytest.mark.parametrize("dtype", TYPES)
def test_large_scores(counts, dtype):
    """Scores far from 0, growing and falling along the sequence: the running maximum moves."""
    def edit(c):
        n = c.S
        ramp = torch.linspace(-6, 6, n).view(1, n, 1, 1)
        c.k = (c.k.float() * 0.3 + ramp).to(c.t)
        c.k[1] = c.k[1].flip(0)
    Case(dtype, 4, 2, 64, 300, [280, 299], counts=counts, seed=21, qscale=3.0, edit=edit).check()


@pytest.mark.parametrize("counts", [None, [30]])
def test_one_position_takes_all_weight(counts):
    """The last, the first of the window and the last sink in turn outweigh everything."""
    for where in (99, 80, 3, 60):
        def edit(c):
            c.q[:] = 1.0
            c.k *= 0.1
            c.k[0, where] = 6.0
            c.v[0, where] = 2.0
        Case("bf16", 4, 1, 64, 100, [99], counts=counts, window=20, sinks=4, seed=22, edit=edit).check()


def test_equal_scores_of_the_lowest_value():
    """Keys that give every position the same, very negative score."""
    def edit(c):
        c.q[:] = 100.0
        c.k[:] = -200.0
    Case("bf16", 4, 2, 64, 200, [199, 7], counts=[150, 8], seed=23, edit=edit).check()
    Case("bf16", 4, 2, 64, 200, [199, 7], seed=23, edit=edit).check()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [0, 24, 64])
def test_bad_values_in_pieces_that_ctas_share(D, page):
    """Long contexts of few rows, cut among CTAs: a value that is not finite lies where some
    rows see it and others do not, and behind what any row sees."""
    def edit(c):
        for p, bad in ((2390, float("inf")), (2396, float("nan")), (2402, float("nan")), (700, -float("inf"))):
            at = c.at(0, p)
            c.v[at][:, 3] = bad
            c.k[at][1, 2] = bad
    c = Case("bf16", 8, 2, D, 2496, [2400, 1500], counts=[20, 1], page=page, window=1700, sinks=3, seed=33, edit=edit)
    got, (ref, tol) = c.run(), c.expected()
    fine = (got.double() - ref).abs() <= tol
    for i in range(20):
        p = 2381 + i
        sees = [x for x in (2390, 2396) if x <= p] + ([700] if 700 > p - 1700 else [])
        if not sees:
            assert bool(fine[i].all())
        else:
            assert bool(fine[i, :4, :3].all()) and bool(fine[i, :4, 4:].all())  # the other channels of head 0
            assert not bool(torch.isfinite(got[i, :4, 3]).any())
    assert bool(fine[20].all())


@pytest.mark.parametrize("page", [0, 48])
def test_bad_values_in_a_shared_prefix(page):
    """Tokens inside the shared positions see only what is before them."""
    if page:
        def edit(c):
            c.v[c.at(0, 1000)][0, 5] = float("nan")
            c.v[c.at(0, 1500)][1, 6] = float("inf")
        last = [999, 1000, 1499, 1500, 1700, 3, 1600]
        c = Case("f16", 8, 2, 128, 1728, last, page=page, shared=1600, seed=34, edit=edit)
    else:
        def edit(c):
            c.vp[1000, 0, 5] = float("nan")
            c.v[2, 7, 1, 6] = float("inf")  # behind sequence 2's live positions
        last = [9, 0, 6, 3]
        c = Case("f16", 8, 2, 128, 10, last, shared=1600, seed=34, edit=edit)
    got, (ref, tol) = c.run(), c.expected()
    finite = torch.isfinite(ref)
    assert torch.equal(torch.isnan(ref), torch.isnan(got.double()))
    assert bool(((got.double() - ref).abs() <= tol)[finite].all())


def test_offsets_past_32_bits():
    """Caches of more than 2^32 bytes, the live rows at their far end."""
    S, Hk, D, H = 700000, 8, 256, 16
    k, v = (torch.zeros((2, S, Hk, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    assert k.numel() > 2 ** 31
    small = Case("bf16", H, Hk, D, 128, [127, 100], counts=[3, 2], window=60, sinks=2, seed=35)
    tail = S - 128  # the small case's positions from 64 on lie there, its sinks at the beginning
    for big, x in ((k, small.k), (v, small.v)):
        big[:, tail:] = x.cuda()
        big[:, :2] = x[:, :2].cuda()
    ref, tol = small.expected()
    d = small.cuda()
    pos = d["pos"] + tail
    got = dattn.attend(d["q"], k, v, pos, window=60, sinks=2, token_offsets=d["offsets"]).cpu().double()
    assert bool(((got - ref).abs() <= tol).all())
    # one token each: the last of either sequence
    pick = torch.tensor([2, 4])
    got = dattn.attend(d["q"][pick.cuda()].contiguous(), k, v, pos, window=60, sinks=2).cpu().double()
    assert bool(((got - ref[pick]).abs() <= tol[pick]).all())
    # the same rows as pages of 100 positions
    table = torch.arange(2 * S // 100, dtype=torch.int32, device="cuda").view(2, -1)
    got = dattn.attend(d["q"], k.view(-1, 100, Hk, D), v.view(-1, 100, Hk, D), pos, window=60, sinks=2,
                       token_offsets=d["offsets"], block_table=table).cpu().double()
    assert bool(((got - ref).abs() <= tol).all())


# ----------------------------------------------------------------- the calls

@pytest.mark.parametrize("counts,shared", [(None, 0), ([20, 3], 0), (None, 50)])
def test_q_slice_of_a_projection(counts, shared):
    Case("f16", 8, 2, 64, 64, [40, 60], counts=counts, shared=shared, stride=2 * 2 * 64, seed=24).check()


def test_bad_pages_are_reported():
    for counts, window in ((None, 0), ([5, 1], 0), (None, 20), ([5, 1], 20)):
        c = Case("f16", 4, 2, 64, 128, [100, 90], counts=counts, page=16, window=window, sinks=2, seed=25)
        good = c.table.clone()
        if window:  # pages that the window has left behind may be gone
            c.table[:, 1:4] = -1
            c.run()
            error_is(_native.OK)
        for bad in (-1, 10 ** 6):
            c.table = good.clone()
            c.table[1, 5] = bad
            c.run()
            error_is(_native.ERR_BAD_PAGE)
    c = Case("f16", 4, 2, 64, 128, [100, 90], page=16, shared=40, seed=25)
    c.table[0, 1] = -7
    c.run()
    error_is(_native.ERR_BAD_PAGE)


def cases_of_calls():
    return [Case("f16", 8, 2, 128, 600, [599, 300, 7], seed=26),
            Case("bf16", 8, 2, 128, 600, [599, 300, 7], window=100, sinks=4, seed=26),
            Case("bf16", 8, 2, 64, 600, [599, 300, 7], counts=[300, 1, 4], seed=27),
            Case("f16", 8, 2, 128, 640, [599, 300, 7], counts=[2, 1, 4], page=64, window=50, seed=28),
            Case("f16", 8, 2, 128, 60, [59, 30, 7], shared=700, seed=29),
            Case("bf16", 8, 2, 128, 640, [599, 500, 450], page=64, shared=400, seed=30)]


@pytest.mark.parametrize("i", range(6))
def test_repeated_and_concurrent_calls_agree(i):
    c = cases_of_calls()[i]
    first = c.run()
    c.check(first)
    d = c.cuda()
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    outs = []
    for r in range(4):
        for s in streams:
            outs.append(c.call(d, stream=s))
    with torch.cuda.stream(streams[0]):
        outs.append(c.call(d))
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o.cpu(), first)


@pytest.mark.parametrize("i", range(6))
def test_captured_and_recorded_calls(i):
    c = cases_of_calls()[i]
    first = c.run()
    d = c.cuda()
    out = torch.empty_like(c.out0, device="cuda")
    c.call(d, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.call(d, out=out)
    # the replay reads the buffers as they are then
    d["q"].neg_()
    graph.replay()
    torch.cuda.synchronize()
    other = out.cpu()
    assert not torch.equal(other, first)
    d["q"].neg_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out.cpu(), first)

    stream = torch.cuda.Stream()
    ws = torch.empty(max(workspace_bytes(c), 16), dtype=torch.uint8, device="cuda")
    dattn.dattn_batch_begin(stream)
    try:
        with pytest.raises(ValueError, match="outlive"):
            c.call(d, stream=stream)
        c.call(d, out=out, workspace=ws, stream=stream)
    finally:
        batch = dattn.dattn_batch_end(stream)
    out.zero_()
    torch.cuda.synchronize()
    batch.launch(stream)
    stream.synchronize()
    assert torch.equal(out.cpu(), first)
    batch.close()


def workspace_bytes(c):
    if c.shared:
        own = c.S - c.shared if c.page else c.S
        return dattn.dattn_decode_shared_workspace_bytes(c.B, c.H, c.Hk, c.D, c.shared, own)
    return dattn.dattn_attend_workspace_bytes(c.B, c.q.shape[0], c.counts is not None, c.H, c.Hk, c.D, c.S,
                                              c.window, c.sinks)


@pytest.mark.parametrize("i", range(6))
def test_workspace_contents_do_not_matter(i):
    c = cases_of_calls()[i]
    n = workspace_bytes(c)
    d = c.cuda()
    first = c.run()
    for fill in (0, 255, 127):
        ws = torch.full((n + 64,), fill, dtype=torch.uint8, device="cuda")
        out = c.call(d, workspace=ws[: max(n, 16)])
        assert torch.equal(out.cpu(), first)
        assert bool((ws[n:] == fill).all())
    if n:
        for ws in (ws[: n - 1], ws[8: n + 8]):
            with pytest.raises(_native.DattnError) as e:
                c.call(d, workspace=ws)
            assert e.value.status == _native.ERR_WORKSPACE


def test_pinned_inputs():
    c = Case("f16", 8, 2, 64, 100, [99, 5], seed=31)
    first = c.run()
    d = c.cuda()
    d["q"], d["pos"] = c.q.pin_memory(), d["pos"].cpu().pin_memory()
    out = c.call(d)
    assert out.is_cuda and torch.equal(out.cpu(), first)
    host = torch.empty_like(c.out0).pin_memory()
    c.call(d, out=host)
    torch.cuda.synchronize()
    assert torch.equal(host, first)


# ------------------------------------------------------- as a model uses them

@pytest.mark.parametrize("page", [0, 16])
def test_prompt_then_decode_steps_then_samples(page):
    """A prompt rotated, written to the cache and attended to with a window; decode steps
    behind it; then samples of the prompt that share it."""
    H = Hk = 4
    D, S, n, steps, t = 64, 160, 100, 5, torch.float16
    g = torch.Generator(device="cuda").manual_seed(32)
    new = lambda *s: torch.randn(s, generator=g, device="cuda").to(t)  # noqa: E731
    table = None
    lead, rows = 1, S
    if page:
        lead, rows = S // page, page
        table = torch.randperm(lead, generator=torch.Generator().manual_seed(1)).view(1, -1).to(torch.int32).cuda()
    kc, vc = (torch.zeros((lead, rows, Hk, D), dtype=t, device="cuda") for _ in range(2))

    def dense(x):
        return x.reshape(S, Hk, D) if table is None else x[table[0].long()].reshape(S, Hk, D)

    def expect(q, got, p, window, sinks):
        c = Case("f16", H, Hk, D, S, [p], counts=[q.shape[0]], window=window, sinks=sinks)
        c.q, c.out0 = q.cpu(), got.cpu()
        c.k, c.v = dense(kc).cpu()[None], dense(vc).cpu()[None]
        c.check(got.cpu())

    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    q, k, v = dattn.rope(new(n, H, D), pos), dattn.rope(new(n, Hk, D), pos), new(n, Hk, D)
    at = (torch.zeros(n, dtype=torch.long, device="cuda"), pos.long())
    if page:
        at = (table[0].long()[pos.long() // page], pos.long() % page)
    kc[at], vc[at] = k, v
    last = torch.tensor([n - 1], dtype=torch.int32, device="cuda")
    offsets = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    out = dattn.attend(q, kc, vc, last, window=40, sinks=4, token_offsets=offsets, block_table=table)
    expect(q, out, n - 1, 40, 4)
    for i in range(steps):
        last += 1
        q = dattn.rope_append(new(1, H, D), new(1, Hk, D), new(1, Hk, D), kc, vc, last, block_table=table)
        out = dattn.attend(q, kc, vc, last, window=40, sinks=4, block_table=table)
        expect(q, out, n + i, 40, 4)
    # three samples of the prompt
    B, own = 3, 16
    if page:
        per = n // page + 2
        pool_k, pool_v = (torch.cat([x, torch.zeros((B * 2, page, Hk, D), dtype=t, device="cuda")]) for x in (kc, vc))
        tables = torch.empty((B, per), dtype=torch.int32, device="cuda")
        tables[:, : n // page] = table[0, : n // page]
        tables[:, n // page:] = lead + torch.arange(2 * B, device="cuda").view(B, 2)
        for b in range(B):  # the page that the prompt ends in is each sample's own
            for x in (pool_k, pool_v):
                x[tables[b, n // page].long()] = x[table[0, n // page].long()]
        cp = torch.full((B,), n, dtype=torch.int32, device="cuda")
        q = dattn.rope_append(new(B, H, D), new(B, Hk, D), new(B, Hk, D), pool_k, pool_v, cp, block_table=tables)
        out = dattn.decode_shared_paged(q, pool_k, pool_v, tables, cp, n)
        again = dattn.attend(q, pool_k, pool_v, cp, block_table=tables)
        flat = [[x[tables[b].long()].reshape(-1, Hk, D)[: n + 1] for x in (pool_k, pool_v)] for b in range(B)]
    else:
        ko, vo = (torch.zeros((B, own, Hk, D), dtype=t, device="cuda") for _ in range(2))
        cp = torch.zeros((B,), dtype=torch.int32, device="cuda")
        at = torch.full((B,), n, dtype=torch.int32, device="cuda")
        q, ko[:, 0], vo[:, 0] = dattn.rope(new(B, H, D), at), dattn.rope(new(B, Hk, D), at), new(B, Hk, D)
        out = dattn.decode_shared(q, kc[0, :n], vc[0, :n], ko, vo, cp)
        flat = [[torch.cat([x[0, :n], y[b, :1]]) for x, y in ((kc, ko), (vc, vo))] for b in range(B)]
        again = dattn.attend(q, *(torch.stack([f[i] for f in flat]) for i in range(2)), at)
    for got in (out, again):
        c = Case("f16", H, Hk, D, n + 1, [n] * B)
        c.q, c.out0 = q.cpu(), got.cpu()
        c.k, c.v = (torch.stack([f[i] for f in flat]).cpu() for i in range(2))
        c.check(got.cpu())
