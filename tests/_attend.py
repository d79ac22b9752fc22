"""Attention over a 16-bit cache in 64 bits, and inputs for its tests."""
from __future__ import annotations

import math

import torch

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def half_step(ref, dtype):
    """Half a step of the type at |ref|."""
    f = torch.finfo(dtype)
    a = ref.abs().clamp(min=f.tiny)
    return f.eps / 2 * torch.exp2(torch.floor(torch.log2(a))) * (1 + 1e-12)


def row(q, K, V, dtype):
    """softmax(q K^T / sqrt(D)) V of one query head in 64 bits and how far a kernel's result
    may be off.

    Before the last rounding the result is sum w_j V_j / sum w_j with w_j = e^(s_j - M):
      score    D products and sums in fp32, 2^-24 each of at most sum |q||k|; the scaled
               score, its difference from M and the exponential round at 2^-24 of |s_j|,
               |s_j - M| and 2^-22 relative: in all `d`, relative, of a weight
      weight   rounded to the cache's type before it meets V: eps / 2 relative, in f16 at
               least 2^-25 of the largest
      sums     of n terms in fp32: n 2^-24 (at most sqrt(n) of that in practice; n here)
    relative to sum w_j |V_j| / sum w_j; the sum of weights is off by as much as the
    scores and the sums are.  Then the result is rounded."""
    n, D = K.shape
    if n == 0:
        z = torch.zeros(q.shape, dtype=torch.float64)
        return z, z
    q, K, V = q.double(), K.double(), V.double()
    s = K @ q / math.sqrt(D)
    w = torch.exp(s - s.max())
    w = w / w.sum()
    ref = w @ V
    dot = (K.abs() @ q.abs()).max() / math.sqrt(D)
    d = (D + 8) * 2.0 ** -24 * dot + 4 * 2.0 ** -24 * s.abs().max() + 2.0 ** -21
    size = w @ V.abs()
    eps = torch.finfo(dtype).eps / 2
    tol = size * (2 * (d + n * 2.0 ** -24) + eps)
    if dtype is torch.float16:
        tol = tol + n * 2.0 ** -25 * V.abs().amax(0)
    return ref, tol + half_step(ref.abs() + tol, dtype)


def seen(p, window, sinks):
    """Positions that a token at p sees."""
    if p < 0:
        return []
    return [j for j in range(p + 1) if window == 0 or j > p - window or j < sinks]


class Case:
    """One call over a dense or paged cache.  counts: new tokens of each sequence (None: one
    each without offsets); last: current_pos, S positions at most; shared: length of a
    prefix, in a tensor of its own (dense) or in the first sequence's pages."""

    def __init__(self, dtype, H, Hk, D, S, last, counts=None, page=0, window=0, sinks=0, shared=0, pad=0,
                 seed=0, qscale=1.0, edit=None, stride=0):
        g = torch.Generator().manual_seed(seed * 7919 + H * 31 + D + S)
        t = TYPES[dtype]
        self.t, self.H, self.Hk, self.D, self.S, self.page = t, H, Hk, D, S, page
        self.last, self.counts, self.window, self.sinks = list(last), counts, window, sinks
        self.shared = shared
        B = self.B = len(self.last)
        n = B if counts is None else sum(counts)
        rand = lambda *s: torch.randn(s, generator=g).to(t)  # noqa: E731
        self.q = (torch.randn((n + pad, H, D), generator=g) * qscale).to(t)
        self.out0 = rand(n + pad, H, D)
        self.stride = stride
        self.table = self.kp = self.vp = None
        lead, rows = B, S
        if page:
            assert S % page == 0
            per = S // page
            lead, rows = B * per + 3, page
            self.table = torch.randperm(lead, generator=g)[: B * per].view(B, per).to(torch.int32)
        elif shared:
            self.kp, self.vp = rand(shared, Hk, D), rand(shared, Hk, D)
        self.k, self.v = rand(lead, rows, Hk, D), rand(lead, rows, Hk, D)
        if edit is not None:
            edit(self)

    # one row of the cache, for tests that plant something there
    def at(self, b, p):
        if self.table is None:
            return b, p
        owner = 0 if p < self.shared else b
        return int(self.table[owner, p // self.page]), p % self.page

    def rows(self, b, positions):
        own = 0 if self.page else self.shared
        K = [self.kp[p] if p < own else self.k[self.at(b, p - own)] for p in positions]
        V = [self.vp[p] if p < own else self.v[self.at(b, p - own)] for p in positions]
        if not K:
            return (torch.zeros((0, self.Hk, self.D), dtype=self.t),) * 2
        return torch.stack(K), torch.stack(V)

    def expected(self):
        """(reference, tolerance) of every row of out; padding keeps what was there."""
        ref, tol = self.out0.double(), torch.zeros(self.out0.shape, dtype=torch.float64)
        t, group = 0, self.H // self.Hk
        for b in range(self.B):
            n = 1 if self.counts is None else self.counts[b]
            end = min(self.last[b], self.S - 1)
            if self.shared and not self.page:
                end += self.shared
            for i in range(n):
                K, V = self.rows(b, seen(end - (n - 1 - i), self.window, self.sinks))
                for h in range(self.H):
                    ref[t, h], tol[t, h] = row(self.q[t, h], K[:, h // group], V[:, h // group], self.t)
                t += 1
        return ref, tol

    def cuda(self):
        """The call's tensors on the GPU."""
        d = {x: getattr(self, x).cuda() for x in ("q", "k", "v")}
        if self.stride:  # q as a slice of a wider projection
            n, H, D = self.q.shape
            wide = torch.full((n, H * D + self.stride), float("nan"), dtype=self.t, device="cuda")
            wide[:, : H * D] = d["q"].view(n, H * D)
            d["q"] = wide[:, : H * D].unflatten(1, (H, D))
        pos = [x - 2 ** 32 if x >= 2 ** 31 else x for x in self.last]
        d["pos"] = torch.tensor(pos, dtype=torch.int32, device="cuda")
        d["table"] = None if self.table is None else self.table.cuda()
        d["offsets"] = None
        if self.counts is not None:
            off = [0]
            for n in self.counts:
                off.append(off[-1] + n)
            d["offsets"] = torch.tensor(off, dtype=torch.int32, device="cuda")
        if self.kp is not None:
            d["kp"], d["vp"] = self.kp.cuda(), self.vp.cuda()
        return d

    def call(self, d, **kw):
        import token_decode_attention_gb300 as dattn
        if self.shared and self.page:
            return dattn.decode_shared_paged(d["q"], d["k"], d["v"], d["table"], d["pos"], self.shared, **kw)
        if self.shared:
            return dattn.decode_shared(d["q"], d["kp"], d["vp"], d["k"], d["v"], d["pos"], **kw)
        return dattn.attend(d["q"], d["k"], d["v"], d["pos"], window=self.window, sinks=self.sinks,
                            token_offsets=d["offsets"], block_table=d["table"], **kw)

    def run(self, **kw):
        out = self.out0.cuda()
        got = self.call(self.cuda(), out=out, **kw)
        assert got is out
        return out.cpu()

    def check(self, got=None, what=""):
        got = self.run() if got is None else got
        ref, tol = self.expected()
        err = (got.double() - ref).abs()
        same_nan = torch.isnan(got.double()) == torch.isnan(ref)
        inf = torch.isinf(ref) & (got.double() == ref)
        ok = same_nan & (torch.isnan(ref) | inf | (err <= tol))
        assert bool(ok.all()), (f"{what}: {int((~ok).sum())} of {ok.numel()} out of tolerance, first at "
                                f"{(~ok).nonzero()[0].tolist()}: got {got[~ok][0]}, expected {ref[~ok][0]}"
                                f" +- {tol[~ok][0]}")
