"""Decode attention over an 8-bit KV cache against a plain form in 64 bits."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import token_decode_attention_gb300 as dattn
from token_decode_attention_gb300 import _native

from . import _q8
from ._util import cur_pos_tensor

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from token_decode_attention_gb300 import build
    build.build()
    dattn.load()
    yield
    assert dattn.dattn_device_error(clear=True) == _native.OK


class Case:
    """One decode over a dense or paged cache with its reference."""

    def __init__(self, B, H, Hk, D, S, block, kv, cp, page=0, seed=0, qscale=1.0, spread=1.0,
                 edit=None):
        rng = np.random.default_rng(seed + 1000 * B + H + D)
        self.B, self.D, self.block, self.page, self.kv, self.cp = B, D, block, page, kv, cp
        self.q = (rng.standard_normal((B, H, D)) * qscale).astype(np.float16)
        lead, rows, self.table = B, S, None
        if page:
            per = S // page
            lead, rows = B * per + 3, page
            self.table = rng.permutation(lead)[: B * per].reshape(B, per).astype(np.int32)
        self.kq, self.ks = _q8.random_cache(rng, lead, rows, Hk, D, block, kv, spread)
        self.vq, self.vs = _q8.random_cache(rng, lead, rows, Hk, D, block, kv, spread)
        if edit is not None:
            edit(self)
        self.tq = torch.from_numpy(self.q).cuda()
        self.tk, self.tv = _q8.to_cache(self.kq, kv), _q8.to_cache(self.vq, kv)
        self.tks, self.tvs = torch.from_numpy(self.ks).cuda(), torch.from_numpy(self.vs).cuda()
        self.tcp = cur_pos_tensor(np.asarray(cp, np.int64) % 2 ** 32 - (np.asarray(cp) >= 2 ** 31) * 2 ** 32)
        self.tt = None if self.table is None else torch.from_numpy(self.table).cuda()

    def run(self, **kw):
        if self.tt is None:
            return dattn.decode_q8(self.tq, self.tk, self.tv, self.tks, self.tvs, self.tcp,
                                   self.block, **kw)
        return dattn.decode_paged_q8(self.tq, self.tk, self.tv, self.tks, self.tvs, self.tt,
                                     self.tcp, self.block, **kw)

    def check(self, got, what=""):
        ref, size, dot, top = _q8.decode(self.q, self.kq, self.vq, self.ks, self.vs, self.cp,
                                         self.block, self.table, self.page)
        L = int(max(min(int(c), 2 ** 31) for c in self.cp)) + 1
        bound = _q8.decode_bound(ref, size, dot, top, min(L, 10 ** 6), self.D, self.vs)
        _q8.check(_q8.f64(got), ref, bound, what)


SHAPES = [
    # B, H, Hk, D, S, block, page, current_pos
    (1, 8, 8, 64, 256, 16, 0, [200]),
    (1, 1, 1, 16, 1, 1, 0, [0]),                      # one position, the smallest head
    (1, 2, 1, 128, 40, 16, 0, [0]),                   # one live position of many
    (2, 4, 4, 32, 17, 8, 0, [16, 3]),                 # dense length not a multiple of the block
    (3, 8, 2, 128, 300, 32, 0, [299, 0, 130]),
    (1, 32, 8, 128, 4096, 16, 16, [4095]),
    (4, 32, 32, 128, 160, 16, 32, [159, 31, 32, 0]),
    (5, 20, 4, 80, 216, 8, 24, [215, 0, 23, 24, 100]),  # pages that end inside a tile
    (2, 40, 40, 96, 130, 64, 0, [129, 64]),
    (2, 16, 1, 128, 500, 128, 0, [499, 127]),         # sixteen query heads to one key/value head
    (1, 24, 2, 64, 777, 1, 7, [770]),                 # a scale for each position, odd pages
    (2, 34, 2, 64, 100, 16, 0, [99, 50]),             # groups of 17: one head at a time
    (2, 64, 2, 64, 333, 16, 0, [332, 10]),            # groups of 32: two columns tiles twice
    (2, 8, 2, 256, 200, 16, 16, [199, 55]),
    (1, 12, 1, 256, 70, 32, 0, [69]),
    (1, 12, 4, 192, 90, 16, 0, [88]),
    (33, 6, 3, 112, 64, 32, 64, list(range(0, 64, 2)) + [63]),
    (1, 4, 4, 128, 20000, 64, 0, [19999]),
]


@pytest.mark.parametrize("kv", ["e4m3", "int8"])
@pytest.mark.parametrize("B,H,Hk,D,S,block,page,cp", SHAPES,
                         ids=[f"B{s[0]}H{s[1]}k{s[2]}D{s[3]}S{s[4]}n{s[5]}p{s[6]}" for s in SHAPES])
def test_matches_the_plain_form(B, H, Hk, D, S, block, page, cp, kv):
    if page:
        S = S // page * page
    c = Case(B, H, Hk, D, S, block, kv, cp, page)
    c.check(c.run())


@pytest.mark.parametrize("parts", [1, 2, 3, 7, 40, 1000])
def test_forced_partitions_agree(parts):
    # ranges that end anywhere: inside a tile, a page, a scale block; empty ranges
    c = Case(3, 8, 2, 128, 96, 16, "e4m3", [95, 40, 7], page=24 * 2)
    c.check(c.run(num_partitions=parts), f"{parts} partitions")


def test_large_batch_of_short_sequences():
    # more sequences than threads of a CTA: the live lengths are summed in rounds
    rng = np.random.default_rng(5)
    cp = rng.integers(0, 6, 1100).tolist()
    c = Case(1100, 2, 1, 16, 6, 2, "int8", cp)
    c.check(c.run())


def test_very_large_batch_uses_the_kept_prefix_sums():
    rng = np.random.default_rng(6)
    cp = rng.integers(0, 3, 4500).tolist()
    c = Case(4500, 1, 1, 16, 3, 1, "e4m3", cp)
    c.check(c.run(num_partitions=977))


def test_current_pos_past_the_cache_masks_nothing():
    c = Case(2, 4, 2, 64, 48, 16, "e4m3", [2 ** 32 - 1, 60])
    c.check(c.run())


def test_large_scores_keep_the_softmax_exact():
    # one position far above the rest: weights underflow, the maximum moves late
    def edit(c):
        c.kq[0, 150] = np.sign(c.q[0, :1].astype(np.float64)) * 200.0
    c = Case(1, 1, 1, 64, 256, 16, "e4m3", [255], qscale=4.0, edit=edit)
    c.check(c.run())


def test_rising_scores_move_the_maximum_in_every_tile():
    def edit(c):
        c.q[:] = 1.0
        c.kq[:] = np.minimum(np.arange(c.kq.shape[1]) // 16 * 8, 120).reshape(1, -1, 1, 1)
        c.ks[:] = 0.25
    c = Case(1, 2, 2, 64, 272, 16, "int8", [271], edit=edit)
    c.check(c.run())


@pytest.mark.parametrize("kv", ["e4m3", "int8"])
def test_scales_over_a_wide_range(kv):
    # V's blocks differ by 2^40: a weight is never lost to its scale
    def edit(c):
        e = np.random.default_rng(2).integers(-20, 20, c.vs.shape)
        c.vs[:] = 2.0 ** e * 1.37
        c.ks[:] *= 0.73
    c = Case(2, 8, 4, 128, 200, 8, kv, [199, 30], edit=edit, spread=0.1)
    # values up to 448 2^20 pass f16: compare where the result is representable
    ref, size, dot, top = _q8.decode(c.q, c.kq, c.vq, c.ks, c.vs, c.cp, c.block)
    got = _q8.f64(c.run())
    ok = np.abs(ref) < 60000
    assert ok.any()
    bound = _q8.decode_bound(ref, size, dot, top, 200, c.D, c.vs)
    _q8.check(got[ok], ref[ok], bound[ok], "wide scales")


def test_zero_scales_stand_for_zeros():
    def edit(c):
        c.vs[:, 1] = 0.0
        c.ks[:, 2] = 0.0
    c = Case(1, 4, 2, 64, 96, 16, "e4m3", [95], edit=edit)
    c.check(c.run())

    def all_zero(c):
        c.vs[:] = 0.0
    c = Case(1, 4, 2, 64, 96, 16, "int8", [95], edit=all_zero)
    assert torch.count_nonzero(c.run()) == 0
    assert torch.count_nonzero(c.run(num_partitions=5)) == 0


@pytest.mark.parametrize("parts", [0, 1, 6])
def test_dead_rows_and_scales_have_no_effect(parts):
    cp = [70, 5]
    clean = Case(2, 4, 2, 128, 128, 16, "e4m3", cp)

    def poison(c):
        for b, p in enumerate(cp):
            c.kq[b, p + 1:] = c.vq[b, p + 1:] = np.nan
            c.ks[b, p // 16 + 1:] = np.inf
            c.vs[b, p // 16 + 1:] = np.nan
    bad = Case(2, 4, 2, 128, 128, 16, "e4m3", cp, edit=poison)
    assert torch.isnan(bad.tk.float()).any()
    a, b = clean.run(num_partitions=parts), bad.run(num_partitions=parts)
    assert torch.equal(a, b)
    clean.check(a)


@pytest.mark.parametrize("parts", [1, 5])
def test_nan_of_a_live_row_reaches_its_heads_only(parts):
    def edit(c):
        c.kq[0, 10, 1, 3] = np.nan   # head 1 of sequence 0: every weight is NaN
        c.vq[1, 20, 0, 7] = np.nan   # one channel of head 0 of sequence 1
    c = Case(2, 4, 2, 64, 64, 16, "e4m3", [63, 63], edit=edit)
    got = c.run(num_partitions=parts)
    nan = torch.isnan(got).cpu().numpy()
    want = np.zeros_like(nan)
    want[0, 2:4] = True
    want[1, 0:2, 7] = True
    assert np.array_equal(nan, want)


def test_infinite_query_gives_nan_as_the_definition_does():
    c = Case(1, 2, 2, 64, 40, 8, "int8", [39])
    c.tq[0, 1, 5] = math.inf
    got = c.run()
    assert torch.isnan(got[0, 1]).all() and not torch.isnan(got[0, 0]).any()


def test_shared_pages_and_unused_table_entries():
    c = Case(2, 4, 2, 64, 96, 16, "e4m3", [40, 95], page=32)
    c.table[1, 0] = c.table[0, 0]     # a shared prefix page
    c.table[0, 2] = -7                # past sequence 0's live length
    c.tt = torch.from_numpy(c.table).cuda()
    c.check(c.run())
    assert dattn.dattn_device_error(clear=True) == _native.OK


@pytest.mark.parametrize("entry", [-1, 10 ** 6])
def test_bad_live_page_is_reported(entry):
    c = Case(2, 4, 2, 64, 96, 16, "e4m3", [95, 95], page=32)
    good = c.run()
    c.tt[0, 1] = entry
    got = c.run()
    assert dattn.dattn_device_error(clear=True) == _native.ERR_BAD_PAGE
    assert torch.equal(got[1], good[1])


def test_repeated_calls_are_bit_identical():
    c = Case(5, 32, 8, 128, 700, 16, "e4m3", [699, 3, 400, 128, 64])
    a = c.run()
    for _ in range(5):
        assert torch.equal(a, c.run())


def test_replayed_batch_sees_new_inputs():
    c = Case(2, 8, 2, 128, 256, 16, "int8", [100, 255])
    s = torch.cuda.Stream()
    n = dattn.dattn_decode_q8_workspace_bytes(2, 8, 2, 128, 256)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(c.tq)
    c.run()
    torch.cuda.synchronize()
    dattn.dattn_batch_begin(s)
    try:
        with pytest.raises(ValueError, match="workspace"):
            c.run(stream=s)
        c.run(out=out, workspace=ws, stream=s)
    finally:
        batch = dattn.dattn_batch_end(s)
    for seed in (1, 2):
        g = torch.Generator(device="cuda").manual_seed(seed)
        c.tq.normal_(generator=g)
        c.q = c.tq.cpu().numpy()
        c.cp = [seed * 50, 17]
        c.tcp.copy_(cur_pos_tensor(c.cp))
        torch.cuda.synchronize()
        batch.launch(s)
        s.synchronize()
        c.check(out, f"replay {seed}")
    batch.close()


def test_two_streams_at_once():
    cs = [Case(2, 8, 4, 128, 900, 16, "e4m3", [899, 500], seed=i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    outs = [[c.run(stream=s) for c, s in zip(cs, streams)] for _ in range(6)]
    torch.cuda.synchronize()
    for c, o in zip(cs, zip(*outs)):
        c.check(o[0])
        assert all(torch.equal(o[0], x) for x in o[1:])


def test_graph_of_torch_replays():
    c = Case(3, 8, 2, 64, 400, 16, "e4m3", [399, 10, 200])
    want = c.run()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = c.run()
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_refuses_tensors_of_another_device(monkeypatch):
    c = Case(1, 2, 1, 64, 32, 16, "e4m3", [3])
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    out = torch.empty_like(c.tq)
    with pytest.raises(ValueError, match="current device"):
        dattn.dattn_decode_q8(c.tq, c.tk, c.tv, c.tks, c.tvs, out, c.tcp, 16)


def test_long_cache_offsets_pass_32_bits():
    # 2^32 + bytes of K: the last positions lie behind a 32-bit byte offset
    B, H, Hk, D, page, block = 1, 8, 8, 128, 64, 64
    rows = 2 ** 22 + 128
    k = torch.zeros((rows // page, page, Hk, D), dtype=torch.int8, device="cuda")
    v = torch.zeros_like(k)
    ks = torch.ones((rows // page, 1, Hk), device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    for t in (k, v):
        t[-2:] = torch.randint(-127, 128, t[-2:].shape, generator=g, device="cuda").to(torch.int8)
    table = torch.tensor([[rows // page - 1, rows // page - 2]], dtype=torch.int32, device="cuda")
    q = torch.randn((B, H, D), generator=g, device="cuda").half() * 0.01
    cp = cur_pos_tensor([page * 2 - 1])
    got = dattn.decode_paged_q8(q, k, v, ks, ks, table, cp, block)
    kk, vv = (torch.cat([t[-1], t[-2]]).cpu().double().numpy()[None] for t in (k, v))
    one = np.ones((1, 2, Hk), np.float32)
    ref, size, dot, top = _q8.decode(q.cpu().numpy(), kk, vv, one, one, [page * 2 - 1], block)
    _q8.check(_q8.f64(got), ref, _q8.decode_bound(ref, size, dot, top, 2 * page, D, one), "far rows")


MANY = [
    # B, H, Hk, D, S, block, page: more (sequence, head group) units than CTAs fit at once
    (160, 16, 8, 64, 40, 8, 8),
    (330, 10, 5, 128, 96, 16, 32),     # groups of four heads: the second holds one
    (170, 8, 2, 256, 48, 16, 0),
    (210, 24, 24, 80, 64, 32, 64),
    (640, 3, 3, 32, 200, 1, 0),
    (320, 48, 3, 128, 33, 16, 0),      # sixteen query heads each
    (700, 2, 1, 16, 1, 1, 1),
]


@pytest.mark.parametrize("kv", ["e4m3", "int8"])
@pytest.mark.parametrize("B,H,Hk,D,S,block,page", MANY,
                         ids=[f"B{s[0]}H{s[1]}k{s[2]}D{s[3]}S{s[4]}" for s in MANY])
def test_many_short_sequences_in_several_waves(B, H, Hk, D, S, block, page, kv):
    assert dattn.dattn_decode_q8_workspace_bytes(B, H, Hk, D, S) == 0
    plan = dattn.dattn_decode_q8_plan(B, H, Hk, D, S)
    assert plan["cluster_size"] == 1 and plan["partitions"] > plan["sm_count"] * plan["ctas_per_sm"]
    cp = np.random.default_rng(B).integers(0, S, B).tolist()
    c = Case(B, H, Hk, D, S, block, kv, cp, page)
    got = c.run()
    c.check(got)
    assert torch.equal(got, c.run())
    # any other split of the same work agrees within the bound
    c.check(c.run(num_partitions=100), "split")


def test_bad_page_among_many_short_sequences():
    c = Case(330, 4, 4, 64, 32, 8, "e4m3", [31] * 330, page=16)
    good = c.run()
    c.tt[7, 1] = 10 ** 6
    c.tt[300, 0] = -5
    got = c.run()
    assert dattn.dattn_device_error(clear=True) == _native.ERR_BAD_PAGE
    keep = torch.ones(330, dtype=torch.bool, device="cuda")
    keep[7] = keep[300] = False
    assert torch.equal(got[keep], good[keep])


@pytest.mark.parametrize("B,H,Hk,D,S", [(1, 8, 8, 64, 500), (2, 32, 8, 128, 900), (1, 32, 32, 128, 4096),
                                        (5, 20, 4, 80, 700), (1, 16, 4, 256, 1000), (1, 12, 3, 128, 600)])
@pytest.mark.parametrize("short", [False, True], ids=["full", "ragged"])
def test_clusters_merge_in_shared_memory(B, H, Hk, D, S, short):
    # no workspace: the CTAs of a sequence's head group exchange their states
    assert dattn.dattn_decode_q8_workspace_bytes(B, H, Hk, D, S) == 0
    cp = [S - 1] * B if not short else [(17 * b + 3) % S for b in range(B)]
    c = Case(B, H, Hk, D, S, 16, "e4m3", cp)
    got = c.run()
    c.check(got)
    assert torch.equal(got, c.run())


@pytest.mark.parametrize("S,parts", [(700, 0), (700, 3), (5000, 0)])
def test_out_may_be_the_queries(S, parts):
    c = Case(2, 8, 2, 128, S, 16, "e4m3", [S - 1, 40])
    want = c.run(num_partitions=parts)
    got = c.run(num_partitions=parts, out=c.tq)
    assert got.data_ptr() == c.tq.data_ptr() and torch.equal(got, want)


@pytest.mark.parametrize("kv", ["e4m3", "int8"])
def test_every_8_bit_value(kv):
    # each code but e4m3's NaN, int8's -128 among them
    codes = np.arange(256, dtype=np.uint8)
    t = torch.from_numpy(codes)
    val = (t.view(torch.float8_e4m3fn) if kv == "e4m3" else t.view(torch.int8)).float().numpy()
    val = np.where(np.isnan(val), 1.0, val).astype(np.float64)

    def edit(c):
        for p in range(c.vq.shape[1]):
            c.vq[0, p, 0] = np.roll(val, 5 * p)[: c.D]
            c.kq[0, p, 0] = np.roll(val, 11 * p + 3)[: c.D]
    c = Case(1, 4, 1, 256, 48, 16, kv, [47], edit=edit, qscale=0.01)
    c.check(c.run())


@pytest.mark.parametrize("kv", ["e4m3", "int8"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("parts", [0, 1, 3])
def test_zero_scales_over_a_long_stretch(parts, D, kv):
    # 131072 positions whose V scale is 0, all but the first tile with weights almost as large as
    # they get before the running maximum moves, then 16 positions that count.  One warp has a
    # head's positions where a single CTA does the work.
    S, H = 131072 + 16, 8
    k = torch.zeros((1, S, H, D), dtype=torch.int8, device="cuda")
    k[..., 0] = 1
    v = torch.randint(-100, 100, k.shape, device="cuda").to(torch.int8)
    v[:, -16:] = 96
    # the scores, in powers of two, by K's scales
    s = torch.full((S // 16,), 4.9, dtype=torch.float64)
    s[0], s[-1] = 0.0, 34.9
    ks = (s * math.log(2.0) * math.sqrt(D)).float().cuda()[None, :, None].expand(1, S // 16, H).contiguous()
    vs = torch.zeros_like(ks)
    vs[:, -1] = 1.0
    q = torch.zeros((1, H, D), dtype=torch.float16, device="cuda")
    q[..., 0] = 1.0
    if kv == "e4m3":
        k, v = k.float().to(torch.float8_e4m3fn), v.float().to(torch.float8_e4m3fn)
    plan = dattn.dattn_decode_q8_plan(1, H, H, D, S, 1)
    assert plan["heads_per_cta"] == 8 and plan["threads_per_cta"] == 256
    got = dattn.decode_q8(q, k, v, ks, vs, cur_pos_tensor([S - 1]), 16, num_partitions=parts)
    # 131072 2^4.9 against 16 2^34.9: the zeros weigh 2^-17, 8e-4 of 96, whose step is 2^-4
    assert torch.equal(got, torch.full_like(got, 96.0))


# Weights rounded to f16 would be off by up to 2^-11.  What is left of decode_bound's weight
# without that rounding: a weight held as the sum of two f16 is off by 2^-21 of itself or, times V's
# scale, by 2^-35 of the largest of them, whose 8-bit values are at most 448.
def exact_weight_bound(ref, size, dot, top, L, D, vs):
    bound = _q8.decode_bound(ref, size, dot, top, L, D, vs) + (2.0 ** -21 - 2.0 ** -11) * size
    return bound + L * 2.0 ** -35 * 448 * vs.max()


@pytest.mark.parametrize("kv", ["e4m3", "int8"])
@pytest.mark.parametrize("D", [16, 64, 80, 128, 256])
@pytest.mark.parametrize("H,Hk", [(1, 1), (6, 2), (4, 1), (5, 1), (16, 2), (12, 1), (16, 1), (34, 2)])
def test_weights_keep_more_bits_than_f16(H, Hk, D, kv):
    # In every tile one position of weight 1 and value -60, and fifteen of weight
    # 2^-4 (1 + 0.45 2^-10) and value 64: all but 0.45 2^-10 of it cancels, and that is
    # what a rounding to 11 bits would drop.
    S = 144

    def edit(c):
        at = np.arange(S) % 16 == 0
        c.q[:] = 0.0
        c.q[:, :, 0] = -1.0
        c.kq[:] = 0.0
        c.kq[:, ~at, :, 0] = 1.0
        c.ks[:] = (4.0 - math.log2(1 + 0.45 * 2.0 ** -10)) * math.log(2.0) * math.sqrt(D)
        c.vs[:] = 1.0
        c.vq[:] = np.where(at, -60.0, 64.0)[None, :, None, None]
    c = Case(2, H, Hk, D, S, 1, kv, [S - 1, 15], edit=edit)
    ref, size, dot, top = _q8.decode(c.q, c.kq, c.vq, c.ks, c.vs, c.cp, 1)
    bound = exact_weight_bound(ref, size, dot, top, S, D, c.vs)
    assert (bound < 0.6 * np.abs(ref)).all()     # 0.0136: a result of 0 is outside
    for parts in (0, 1, 9):
        _q8.check(_q8.f64(c.run(num_partitions=parts)), ref, bound, f"{parts} partitions")


@pytest.mark.parametrize("B,H,Hk,D,S,block,page,cp", SHAPES,
                         ids=[f"B{s[0]}H{s[1]}k{s[2]}D{s[3]}S{s[4]}n{s[5]}p{s[6]}" for s in SHAPES])
def test_the_bound_without_a_rounding_of_the_weights(B, H, Hk, D, S, block, page, cp):
    c = Case(B, H, Hk, D, S // page * page if page else S, block, "e4m3", cp, page, seed=3)
    ref, size, dot, top = _q8.decode(c.q, c.kq, c.vq, c.ks, c.vs, c.cp, block, c.table, page)
    _q8.check(_q8.f64(c.run()), ref, exact_weight_bound(ref, size, dot, top, max(cp) + 1, D, c.vs), "")


@pytest.mark.parametrize("page", [0, 16])
def test_writing_to_out_counts_as_a_change_in_place(page):
    c = Case(2, 4, 2, 64, 64, 16, "e4m3", [63, 5], page=page)
    want, out = c.run(), torch.empty_like(c.tq)
    before = out._version
    assert torch.equal(c.run(out=out), want) and out._version > before
    w = torch.ones_like(c.tq, requires_grad=True)
    y = (w * c.tq).sum()
    c.run(out=c.tq)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    with torch.inference_mode():
        c.run(out=torch.empty_like(c.tq))


@pytest.mark.parametrize("page", [0, 16])
def test_gradients_that_would_be_lost_are_refused(page):
    c = Case(2, 4, 2, 64, 64, 16, "e4m3", [63, 5], page=page)
    for name in ("tq", "tks", "tvs"):
        setattr(c, name, getattr(c, name).requires_grad_())
        with pytest.raises(ValueError, match="gradient"):
            c.run()
        setattr(c, name, getattr(c, name).detach())
    with pytest.raises(ValueError, match="gradient"):
        c.run(out=torch.empty_like(c.tq).requires_grad_())
    fwad = torch.autograd.forward_ad
    with fwad.dual_level():
        keep, c.tq = c.tq, fwad.make_dual(c.tq, torch.ones_like(c.tq))
        with pytest.raises(ValueError, match="gradient"):
            c.run()
        c.tq = keep
    c.tq.requires_grad_()
    with torch.no_grad():
        c.check(c.run())


def test_a_wide_table_over_a_small_pool():
    # capacities of 2^20 positions add up to 2^31; the pool holds 8 pages
    B, page = 2048, 256
    rng = np.random.default_rng(9)
    kq, ks = _q8.random_cache(rng, 8, page, 1, 16, 16, "e4m3")
    vq, vs = _q8.random_cache(rng, 8, page, 1, 16, 16, "e4m3")
    table = np.full((B, 2 ** 20 // page), -1, np.int32)     # dead entries are not read
    table[:, :2] = rng.integers(0, 8, (B, 2))
    cp = rng.integers(0, 2 * page, B)
    q = rng.standard_normal((B, 2, 16)).astype(np.float16)
    got = dattn.decode_paged_q8(torch.from_numpy(q).cuda(), _q8.to_cache(kq, "e4m3"), _q8.to_cache(vq, "e4m3"),
                                torch.from_numpy(ks).cuda(), torch.from_numpy(vs).cuda(),
                                torch.from_numpy(table).cuda(), cur_pos_tensor(cp), 16)
    ref, size, dot, top = _q8.decode(q, kq, vq, ks, vs, cp, 16, table, page)
    _q8.check(_q8.f64(got), ref, _q8.decode_bound(ref, size, dot, top, 2 * page, 16, vs), "wide table")


def test_refuses_a_workspace_of_another_device():
    class Elsewhere(torch.Tensor):
        def get_device(self):
            return 1
    c = Case(1, 8, 2, 128, 40000, 16, "e4m3", [39999])
    n = dattn.dattn_decode_q8_workspace_bytes(1, 8, 2, 128, 40000)
    assert n > 0
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError, match="workspace is on cuda:1"):
        c.run(workspace=ws.as_subclass(Elsewhere))
    out = torch.empty_like(c.tq)
    with pytest.raises(ValueError, match="workspace is on cuda:1"):
        dattn.dattn_decode_q8(c.tq, c.tk, c.tv, c.tks, c.tvs, out, c.tcp, 16, ws.as_subclass(Elsewhere))
    c.check(c.run(workspace=ws))
    pinned = torch.empty(n, dtype=torch.uint8, pin_memory=True)
    c.check(c.run(workspace=pinned))
