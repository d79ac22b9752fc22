"""Rotating and appending to an 8-bit KV cache against a plain form in 64 bits."""
from __future__ import annotations

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


class Step:
    """One append to a cache that already holds values, with its reference."""

    def __init__(self, counts, last, H, Hk, D, S, block, kv, page=0, pad=0, rd=0, base=10000.0,
                 trad=False, scaling=None, seed=0, ragged=None, scale=1.0):
        rng = np.random.default_rng(seed + len(counts) + D)
        self.counts, self.last, self.kv, self.block, self.page = counts, last, kv, block, page
        self.B, self.H, self.Hk, self.D, self.S = len(counts), H, Hk, D, S
        self.rope = dict(rope_dims=rd, rope_base=base, traditional=trad, scaling=scaling)
        T = sum(counts)
        rows = T + pad
        self.T = T
        mk = lambda h: (scale * rng.standard_normal((rows, h, D)) * np.exp(rng.standard_normal((rows, h, 1)))).astype(np.float16)  # noqa: E731
        self.q, self.k, self.v = mk(H), mk(Hk), mk(Hk)
        lead, n, self.table = self.B, S, None
        if page:
            per = S // page
            lead, n = self.B * per + 2, page
            self.table = rng.permutation(lead)[: self.B * per].reshape(self.B, per).astype(np.int32)
        self.kq, self.ks = _q8.random_cache(rng, lead, n, Hk, D, block, kv)
        self.vq, self.vs = _q8.random_cache(rng, lead, n, Hk, D, block, kv)
        self.tq, self.tk, self.tv = (torch.from_numpy(x).cuda() for x in (self.q, self.k, self.v))
        self.ck, self.cv = _q8.to_cache(self.kq, kv), _q8.to_cache(self.vq, kv)
        self.sk, self.sv = torch.from_numpy(self.ks).cuda(), torch.from_numpy(self.vs).cuda()
        self.qo = torch.full((rows, H, D), -3.0, dtype=torch.float16, device="cuda")
        off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        ragged = (pad > 0 or any(c != 1 for c in counts)) if ragged is None else ragged
        self.off = torch.from_numpy(off).cuda() if ragged else None
        self.cp = cur_pos_tensor(last)
        self.tt = None if self.table is None else torch.from_numpy(self.table).cuda()

    def run(self, **kw):
        kw = {"q_out": self.qo, **kw}
        return dattn.rope_append_q8(self.tq, self.tk, self.tv, self.ck, self.cv, self.sk, self.sv,
                                    self.cp, self.block, token_offsets=self.off,
                                    block_table=self.tt, **self.rope, **kw)

    def positions(self):
        return np.concatenate([np.arange(l - c + 1, l + 1) for c, l in zip(self.counts, self.last)]
                              ).astype(np.int64) if self.T else np.zeros(0, np.int64)

    def expect(self, x, cache, scales):
        """(values, scales, written rows' exact x/scale) after appending x (64 bits)."""
        cache, scales = cache.copy(), scales.astype(np.float64)
        exact = np.full(cache.shape, np.nan)
        t = 0
        n = self.block
        for b, c in enumerate(self.counts):
            p, p1 = self.last[b] - c + 1, self.last[b] + 1
            while p < p1:
                if p < 0 or p >= self.S:
                    t, p = t + 1, p + 1
                    continue
                stop = min(p1, (p // n + 1) * n, self.S)
                lead, row = (b, p) if not self.page else (self.table[b, p // self.page], p % self.page)
                if not 0 <= lead < cache.shape[0]:
                    t, p = t + stop - p, stop
                    continue
                blk, before = row // n, p % n
                new = x[t: t + stop - p]
                a = np.abs(new)
                s = _q8.need_scale(np.where(np.isfinite(a), a, 0).max(axis=(0, 2)), self.kv)
                if before:
                    old = scales[lead, blk].copy()
                    s = np.maximum(s, old)
                    f = np.float32(1) * (old / s).astype(np.float32)
                    cache[lead, row - before: row] = _q8.round8(
                        cache[lead, row - before: row] * f[:, None], self.kv)
                scales[lead, blk] = s
                exact[lead, row: row + stop - p] = new / s[:, None]
                cache[lead, row: row + stop - p] = _q8.round8(new / s[:, None], self.kv)
                t, p = t + stop - p, stop
        return cache, scales, exact

    def check(self, what=""):
        rd, trad, sc = self.rope["rope_dims"] or self.D, self.rope["traditional"], self.rope["scaling"]
        mag = 1.0 if sc is None else sc.magnitude
        pos = self.positions() % 2 ** 32
        args = (pos, rd, self.rope["rope_base"], trad, sc)
        q = self.q[: self.T].astype(np.float64)
        ref = _q8.rotate(q, *args)
        bound = _q8.ROTATION * _q8.pair_size(q, rd, trad, mag)
        bound += (np.arange(self.D) < rd) * _q8.half_step(np.abs(ref) + bound, 2.0 ** -10, 2.0 ** -24)
        _q8.check(_q8.f64(self.qo[: self.T]), ref, bound, what + " q")
        assert (self.qo[self.T:] == -3.0).all(), what + ": padding rows of q_out were written"
        # V is not rotated: every byte and scale is determined
        cache, scales, _ = self.expect(self.v[: self.T].astype(np.float64), self.vq, self.vs)
        assert np.array_equal(self.sv.cpu().numpy().astype(np.float64), scales), what + " V scales"
        assert np.array_equal(_q8.values(self.cv), cache), what + " V"
        # K: a rotated value within ROTATION of a border may fall on either side
        k = self.k[: self.T].astype(np.float64)
        cache, scales, exact = self.expect(_q8.rotate(k, *args), self.kq, self.ks)
        assert np.array_equal(self.sk.cpu().numpy().astype(np.float64), scales), what + " K scales"
        got = _q8.values(self.ck)
        new = ~np.isnan(exact)
        assert np.array_equal(got[~new], cache[~new]), what + ": a row of K that is not new differs"
        sz = _q8.pair_size(k, rd, trad, mag).max() if self.T else 0.0
        s = np.repeat(scales, self.block, axis=1)[:, : cache.shape[1]][..., None] + 0 * exact
        slack = _q8.ROTATION * sz / s[new]
        x = exact[new]
        top = _q8.QMAX[self.kv]
        err = np.abs(got[new] - np.clip(x, -top, top))
        assert (err <= _q8.half_step8(np.abs(x) + slack, self.kv) + slack).all(), what + " K"
        # and almost all are the nearest ones
        assert np.mean(got[new] != cache[new]) < 1e-3, what + " K"


CASES = [
    # counts, last, H, Hk, D, S, block, page, pad, rope_dims, trad
    ([1], [0], 8, 8, 64, 16, 16, 0, 0, 0, False),
    ([1], [4095], 32, 8, 128, 4096, 16, 16, 0, 0, False),
    ([1, 1, 1], [0, 31, 17], 4, 4, 128, 32, 16, 0, 0, 0, True),
    ([1, 1, 1], [0, 31, 17], 4, 4, 128, 32, 16, 0, 5, 0, False),
    ([5], [4], 8, 2, 128, 64, 16, 0, 0, 0, False),
    ([40], [50], 8, 2, 128, 64, 16, 32, 0, 64, False),
    ([0, 17, 1, 0, 33], [9, 16, 40, 0, 60], 6, 3, 80, 72, 8, 24, 11, 40, True),
    ([100, 3], [120, 2], 4, 1, 256, 128, 128, 0, 0, 0, False),
    ([150], [149], 4, 2, 256, 256, 256, 0, 0, 32, False),   # more rows than registers hold
    ([300, 290], [310, 289], 2, 2, 128, 320, 320, 0, 0, 0, True),
    ([7, 9], [6, 20], 2, 1, 16, 24, 1, 0, 0, 0, False),     # a scale for each position
    ([20, 1], [19, 5], 10, 5, 96, 30, 4, 0, 2, 20, False),  # pairs one by one; S no multiple
    ([64] * 5, [63 + 7 * i for i in range(5)], 40, 40, 128, 128, 32, 64, 0, 0, False),
    ([1] * 70, list(range(70)), 3, 3, 48, 80, 16, 16, 0, 0, False),
    ([2] * 40, [2 * i + 1 for i in range(40)], 2, 1, 112, 96, 32, 0, 1, 0, True),
]


@pytest.mark.parametrize("kv", ["e4m3", "int8"])
@pytest.mark.parametrize("case", CASES, ids=[f"T{sum(c[0])}B{len(c[0])}H{c[2]}k{c[3]}D{c[4]}n{c[6]}p{c[7]}" for c in CASES])
def test_matches_the_plain_form(case, kv):
    counts, last, H, Hk, D, S, block, page, pad, rd, trad = case
    s = Step(counts, last, H, Hk, D, S, block, kv, page, pad, rd, trad=trad)
    s.run()
    s.check()


@pytest.mark.parametrize("kind", ["linear", "base", "by_parts"])
def test_scaled_frequencies(kind):
    sc = dattn.RopeScaling(kind, 4.0, original_len=512, low_turns=1, high_turns=16, magnitude=1.1)
    s = Step([30, 1], [500, 3], 4, 2, 64, 512, 16, "e4m3", page=32, scaling=sc, base=500000.0)
    s.run()
    s.check(kind)


@pytest.mark.parametrize("kv", ["e4m3", "int8"])
def test_growing_scale_requantises_the_earlier_rows(kv):
    # token after token into one block, each twice as large as the one before
    B, H, Hk, D, n = 1, 2, 2, 64, 16
    s = Step([1], [0], H, Hk, D, 32, n, kv)
    for p in range(n + 3):
        s2 = Step([1], [p], H, Hk, D, 32, n, kv, seed=p, scale=2.0 ** (p - 8))
        s2.kq, s2.vq = _q8.values(s.ck), _q8.values(s.cv)
        s2.ks, s2.vs = s.sk.cpu().numpy(), s.sv.cpu().numpy()
        s2.ck, s2.cv, s2.sk, s2.sv = s.ck, s.cv, s.sk, s.sv
        s2.run()
        s2.check(f"position {p}")
        s = s2


def test_a_chunk_fills_the_block_that_another_began():
    s = Step([10], [9], 4, 2, 128, 64, 16, "e4m3")
    s.run()
    s.check("first")
    t = Step([20], [29], 4, 2, 128, 64, 16, "e4m3", seed=3, scale=30.0)
    t.kq, t.vq, t.ks, t.vs = _q8.values(s.ck), _q8.values(s.cv), s.sk.cpu().numpy(), s.sv.cpu().numpy()
    t.ck, t.cv, t.sk, t.sv = s.ck, s.cv, s.sk, s.sv
    t.run()
    t.check("second")


def test_the_same_step_twice_changes_nothing_more():
    s = Step([5, 40], [20, 61], 4, 2, 128, 64, 16, "int8")
    s.run()
    first = [t.clone() for t in (s.ck, s.cv, s.sk, s.sv, s.qo)]
    s.run()
    torch.cuda.synchronize()
    for a, b in zip(first, (s.ck, s.cv, s.sk, s.sv, s.qo)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("kv", ["e4m3", "int8"])
def test_zeros_subnormals_and_the_largest_values(kv):
    s = Step([4], [3], 2, 2, 64, 16, 4, kv)
    v = np.zeros((4, 2, 64), np.float16)
    v[0, 0, 0] = np.float16(2.0 ** -24)
    v[1, 1, :4] = [65504, -65504, 448, 1]
    s.v, s.tv = v, torch.from_numpy(v).cuda()
    s.run()
    s.check("extremes")
    z = Step([4], [3], 2, 2, 64, 16, 4, kv)
    z.v[:] = 0
    z.k[:] = 0
    z.tv.zero_()
    z.tk.zero_()
    z.run()
    z.check("zeros")
    assert (z.sv[0, 0] == 2.0 ** -32).all()


@pytest.mark.parametrize("kv", ["e4m3", "int8"])
def test_infinities_saturate_and_nan_is_kept_or_zero(kv):
    s = Step([3], [2], 1, 1, 32, 8, 8, kv)
    s.tv[0, 0, 0], s.tv[1, 0, 1], s.tv[2, 0, 2] = float("inf"), float("-inf"), float("nan")
    s.run()
    v = _q8.values(s.cv)[0, :3, 0]
    top = _q8.QMAX[kv]
    assert v[0, 0] == top and v[1, 1] == -top
    assert np.isnan(v[2, 2]) if kv == "e4m3" else v[2, 2] == 0
    a = np.abs(s.v[:, 0].astype(np.float64))
    a[0, 0] = a[1, 1] = a[2, 2] = 0
    assert float(s.sv[0, 0, 0]) == _q8.need_scale(a.max(keepdims=True), kv)[0, 0]


def test_positions_outside_the_cache_are_reported_and_not_written():
    # sequence 0 runs past the end, sequence 1 begins before position 0
    s = Step([6, 5, 2], [17, 2, 9], 4, 2, 64, 16, 4, "e4m3")
    assert dattn.dattn_device_error(clear=True) == _native.OK
    s.run()
    assert dattn.dattn_device_error(clear=True) == _native.ERR_BAD_POSITION
    s.check()
    one = Step([1, 1], [16, 3], 4, 2, 64, 16, 4, "int8")
    one.run()
    assert dattn.dattn_device_error(clear=True) == _native.ERR_BAD_POSITION
    one.check()


def test_invalid_pages_are_reported_and_not_written():
    s = Step([20, 4], [35, 3], 4, 2, 64, 64, 8, "e4m3", page=16)
    s.table[0, 1] = -1
    s.table[1, 0] = 10 ** 6
    s.tt = torch.from_numpy(s.table).cuda()
    s.run()
    assert dattn.dattn_device_error(clear=True) == _native.ERR_BAD_PAGE
    s.check()


@pytest.mark.parametrize("offsets", [[0, 0, 0], [3, 1, 5], [0, 9, 2], [-4, 2, 100], [0, 2, -1]])
def test_offsets_that_make_no_sense_stay_in_bounds(offsets):
    # the call promises nothing for them but to stay inside its buffers: the rows
    # and pages around the cache keep their bytes
    s = Step([3, 2], [2, 9], 2, 1, 64, 16, 4, "int8")
    s.off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    big = torch.full((3, 2, 16, 1, 64), 77, dtype=torch.int8, device="cuda")
    big[1] = s.ck
    s.ck = big[1]
    s.run()
    torch.cuda.synchronize()
    assert (big[0] == 77).all() and (big[2] == 77).all()
    dattn.dattn_device_error(clear=True)


def test_slices_of_a_projection_and_in_place_q():
    H, Hk, D, T = 8, 2, 128, 21
    s = Step([20, 1], [30, 0], H, Hk, D, 32, 16, "e4m3")
    qkv = torch.cat([s.tq.view(T, -1), s.tk.view(T, -1), s.tv.view(T, -1)], 1)
    s.tq = qkv[:, : H * D].view(T, H, D)
    s.tk = qkv[:, H * D: (H + Hk) * D].view(T, Hk, D)
    s.tv = qkv[:, (H + Hk) * D:].view(T, Hk, D)
    s.run()
    s.check("slices")
    t = Step([20, 1], [30, 0], H, Hk, D, 32, 16, "e4m3")
    t.run(q_out=t.tq)
    t.qo = t.tq
    t.check("in place")


def test_replayed_step_sees_new_inputs():
    s = Step([3, 1], [2, 9], 4, 2, 64, 32, 8, "e4m3", page=16)
    st = torch.cuda.Stream()
    s.run()
    torch.cuda.synchronize()
    dattn.dattn_batch_begin(st)
    s.run(stream=st)
    batch = dattn.dattn_batch_end(st)
    for i in range(3):
        t = Step([2, 2] if i == 1 else [0, 4], [i + 5, i + 12], 4, 2, 64, 32, 8, "e4m3", page=16, seed=i)
        for a, b in ((s.tq, t.tq), (s.tk, t.tk), (s.tv, t.tv), (s.ck.view(torch.uint8), t.ck.view(torch.uint8)),
                     (s.cv.view(torch.uint8), t.cv.view(torch.uint8)), (s.sk, t.sk), (s.sv, t.sv), (s.cp, t.cp),
                     (s.off, t.off), (s.tt, t.tt), (s.qo, t.qo)):
            a.copy_(b)
        torch.cuda.synchronize()
        batch.launch(st)
        st.synchronize()
        t.ck, t.cv, t.sk, t.sv, t.qo = s.ck, s.cv, s.sk, s.sv, s.qo
        t.check(f"replay {i}")
    batch.close()


def test_refusals():
    s = Step([1, 1], [0, 3], 4, 2, 64, 16, 8, "e4m3")
    run = lambda **k: s.run(**k)  # noqa: E731
    keep = s.tk
    s.tk = keep[:, :1]
    with pytest.raises(ValueError, match="k_new"):
        run()
    s.tk = keep.float()
    with pytest.raises(TypeError, match="k_new"):
        run()
    s.tk = keep
    ck, s.ck = s.ck, s.ck.view(torch.uint8)
    with pytest.raises(TypeError, match="cache"):
        run()
    s.ck = ck
    sk, s.sk = s.sk, s.sk[:, :1]
    with pytest.raises(ValueError, match="K_scale"):
        run()
    s.sk = sk
    s.block = 0
    with pytest.raises(ValueError, match="scale_block"):
        run()
    s.block = 8
    s.off = torch.zeros(2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="token_offsets"):
        run()
    s.off = None
    s.rope["rope_dims"] = 7
    with pytest.raises(_native.DattnError, match="rope_dims"):
        run()
    s.rope["rope_dims"] = 0
    tq, s.tq = s.tq, s.tq.expand(2, 4, 64)[:1]
    with pytest.raises(ValueError):
        run()
    s.tq = tq
    run()
    s.check()


def _mixed(n, top, seed):
    return np.random.default_rng(seed).integers(0, top, n).tolist()


LARGER = [
    # counts, first position's offset, H, Hk, D, S, block, page, pad, rope_dims, trad
    (_mixed(300, 40, 1), 5, 6, 6, 32, 64, 16, 32, 3, 0, False),
    ([2000], 77, 16, 8, 64, 2112, 16, 16, 0, 0, False),
    ([700, 0, 513], 1, 6, 3, 128, 768, 256, 256, 9, 64, True),
    (_mixed(64, 30, 2), 0, 7, 7, 80, 40, 8, 0, 0, 40, False),   # odd heads, pairs one by one
    (_mixed(64, 30, 3), 9, 12, 4, 96, 40, 40, 0, 1, 20, True),
    (_mixed(1500, 4, 4), 2, 2, 1, 16, 8, 4, 4, 0, 0, False),
    ([33] * 9, 31, 40, 20, 256, 64, 64, 64, 0, 128, False),
]


@pytest.mark.parametrize("kv", ["e4m3", "int8"])
@pytest.mark.parametrize("case", LARGER, ids=[f"T{sum(c[0])}B{len(c[0])}H{c[2]}k{c[3]}D{c[4]}n{c[6]}p{c[7]}" for c in LARGER])
def test_larger_batches(case, kv):
    counts, first, H, Hk, D, S, block, page, pad, rd, trad = case
    last = [min(first + i % 3 + c - 1, S - 1) if c else first for i, c in enumerate(counts)]
    s = Step(counts, last, H, Hk, D, S, block, kv, page, pad, rd, trad=trad)
    s.run()
    s.check()


def test_far_pages_pass_32_bits():
    # 2^32 + bytes of each cache: a block of the last page that has earlier rows
    Hk, H, D, page, n = 8, 8, 128, 64, 16
    pages = 2 ** 22 // page + 3
    g = torch.Generator(device="cuda").manual_seed(2)
    k = torch.zeros((pages, page, Hk, D), dtype=torch.int8, device="cuda")
    v = torch.zeros_like(k)
    ks = torch.ones((pages, page // n, Hk), device="cuda")
    vs = torch.ones_like(ks)
    near = [t[:2].clone() for t in (k, v, ks, vs)]   # the same step on pages at the front
    mk = lambda h: torch.randn((20, h, D), generator=g, device="cuda").half()  # noqa: E731
    x = [mk(H), mk(Hk), mk(Hk)]
    off = torch.tensor([0, 20], dtype=torch.int32, device="cuda")
    table = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32, device="cuda")
    small = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda")
    for offsets, cp, take in ((off, 69, 20), (None, 70, 1)):
        args = [t[:take] for t in x]
        dattn.rope_append_q8(*args, k, v, ks, vs, cur_pos_tensor([cp]), n, token_offsets=offsets, block_table=table)
        dattn.rope_append_q8(*args, *near, cur_pos_tensor([cp]), n, token_offsets=offsets, block_table=small)
    for far, t in zip((k, v, ks, vs), near):
        assert torch.equal(far[-2:], t)
    assert torch.count_nonzero(k[:-2]) == 0 and torch.count_nonzero(v[:-2]) == 0


def test_a_recorded_append_needs_its_output():
    s = Step([1, 1], [0, 3], 4, 2, 64, 16, 8, "e4m3")
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    dattn.dattn_batch_begin(st)
    try:
        with pytest.raises(ValueError, match="q_out"):
            s.run(q_out=None, stream=st)
    finally:
        s.run(stream=st)
        dattn.dattn_batch_end(st).close()


@pytest.mark.parametrize("counts,last", [
    ([1] * 30 + [200] + [1] * 20 + [0, 3], [7 * i % 250 for i in range(30)] + [230] + [50 + i for i in range(20)] + [9, 2]),
    ([0, 0, 0, 5], [1, 2, 3, 4]),
    ([0, 64, 0], [0, 63, 0]),
])
@pytest.mark.parametrize("block", [1, 2, 16, 256])
def test_steps_and_a_prompt_in_one_call(counts, last, block):
    s = Step(counts, last, 8, 4, 64, 256, block, "e4m3", ragged=True)
    s.run()
    s.check()


@pytest.mark.parametrize("D,rd", [(256, 20), (128, 20), (256, 40), (48, 12), (96, 6), (256, 250)])
@pytest.mark.parametrize("counts", [[1, 1, 1], [5, 0, 40]])
@pytest.mark.parametrize("trad", [False, True])
def test_rotated_parts_that_16_does_not_divide(D, rd, counts, trad):
    # items of eight, of four (a warp's lanes or too many of them), of single channels
    s = Step(counts, [50, 7, 44], 6, 3, D, 64, 16, "e4m3", rd=rd, trad=trad)
    s.run()
    s.check()


@pytest.mark.parametrize("page", [0, 16])
def test_what_an_append_writes_counts_as_changed(page):
    s = Step([3, 1], [5, 9], 4, 2, 64, 32, 8, "e4m3", page=page)
    written = (s.qo, s.ck, s.cv, s.sk, s.sv)
    before = [t._version for t in written]
    s.run()
    assert all(t._version > b for t, b in zip(written, before))
    s.check()
    with torch.inference_mode():
        s = Step([3, 1], [5, 9], 4, 2, 64, 32, 8, "e4m3", page=page)
        s.run()
    s.check()


def test_a_kept_query_that_is_rotated_in_place_is_noticed():
    s = Step([1, 1], [5, 9], 4, 2, 64, 32, 8, "int8")
    w = torch.ones_like(s.tq, requires_grad=True)
    y = (w * s.tq).sum()
    s.run(q_out=s.tq)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


def test_gradients_that_would_be_lost_are_refused():
    s = Step([1, 1], [5, 9], 4, 2, 64, 32, 8, "e4m3")
    for name in ("tq", "tk", "tv", "sk", "qo"):
        setattr(s, name, getattr(s, name).requires_grad_())
        with pytest.raises(ValueError, match="gradient"):
            s.run()
        setattr(s, name, getattr(s, name).detach())
    fwad = torch.autograd.forward_ad
    with fwad.dual_level():
        keep, s.tk = s.tk, fwad.make_dual(s.tk, torch.ones_like(s.tk))
        with pytest.raises(ValueError, match="gradient"):
            s.run()
        s.tk = keep
    s.tq.requires_grad_()
    with torch.no_grad():
        s.run()
    s.check()


@pytest.mark.parametrize("ragged", [False, True])
def test_q_out_on_the_new_keys_or_values_is_refused(ragged):
    # q is written while k and v are read
    s = Step([1, 1, 1], [5, 9, 2], 2, 2, 64, 32, 8, "e4m3", ragged=ragged)
    for name in ("tk", "tv"):
        with pytest.raises(ValueError, match="q_out"):
            s.run(q_out=getattr(s, name))
        room = torch.empty(6 * 128 + 64, dtype=torch.float16, device="cuda")
        keep = getattr(s, name)
        setattr(s, name, room[: 3 * 128].view(3, 2, 64).copy_(keep))
        with pytest.raises(ValueError, match="q_out"):
            s.run(q_out=room[3 * 128 - 64: 6 * 128 - 64].view(3, 2, 64))
        s.run(q_out=room[3 * 128: 6 * 128].view(3, 2, 64))            # just behind
        # between the first and the second token of a wide projection
        wide = torch.empty((3, 640), dtype=torch.float16, device="cuda")
        setattr(s, name, wide[:, :128].unflatten(1, (2, 64)).copy_(keep))
        s.run(q_out=wide.view(-1)[192: 192 + 384].view(3, 2, 64))
        with pytest.raises(ValueError, match="q_out"):
            s.run(q_out=wide.view(-1)[384: 384 + 384].view(3, 2, 64))
        setattr(s, name, keep)
    s = Step([1, 1, 1], [5, 9, 2], 2, 2, 64, 32, 8, "e4m3", ragged=ragged)
    s.run()
    s.check()
