"""Inputs whose error is that of the softmax weights' rounding, for attention of one token over
a 16-bit cache: V holds 1 where rounding a weight to the type moves it up and -1 where it moves
it down, so that the errors of weights held in one 16-bit number add up instead of cancelling
(but for the smallest errors, whose signs balance the sum).

The kernel holds a weight as 2^(s - M) with M ten (log2) below the largest score that its warp
had met: every 16th position has the largest score, so that all have the same M and the
rounding of w 2^10 / max(w) is that of w / max(w)."""
from __future__ import annotations

import math

import torch

from ._attend import TYPES, Case, half_step

N = 256
# relative error of a weight that is the sum of two numbers of the type: the first is rounded
# down from (1 - eps) w and leaves at most 3/2 eps w, whose rounding is eps / 2 of that; f16
# has steps of 2^-24 besides, in units of which the largest weight is 2^10
TWO_PARTS = {torch.float16: 1.5 * 2.0 ** -21, torch.bfloat16: 1.5 * 2.0 ** -15}


def weights(q, K, D):
    s = (K.double() @ q.double()) / math.sqrt(D)
    w = torch.exp(s - s.max())
    return s, w


def rounded(w, t):
    """w in one number of the type, as if 2^10 were the largest."""
    return (w * 1024).to(t).double() / 1024


def case(dtype, group, D, seed):
    """One sequence, `group` query heads on one key/value head; channel c goes by the weights of
    query head c % group."""
    t = TYPES[dtype]

    def edit(c):
        # query head h looks at channel h of the keys: scores from -1 to 0, and 0 every 16 positions
        c.q[:] = 0
        for h in range(group):
            c.q[0, h, h] = math.sqrt(D)
        c.k[:] = -c.k.abs() / c.k.abs().amax()
        c.k[0, ::16] = 0
        for h in range(group):
            _, w = weights(c.q[0, h], c.k[0, :, 0], D)
            assert float(w[0]) == 1.0  # the largest
            err = rounded(w, t) - w
            up = torch.where(err > 0, 1.0, -1.0).double()
            for j in err.abs().argsort().tolist():  # and sum w V near 0, whose own rounding is small
                if (w @ up) * up[j] > w[j]:
                    up[j] = -up[j]
            c.v[0, :, 0, h::group] = up.to(t)[:, None]
    return Case(dtype, group, 1, D, N, [N - 1], seed=seed, edit=edit)


def expected(c):
    """(reference, tolerance with weights of two parts), [heads, D]: the bound of _attend.row with
    the weights' own part in place of eps / 2."""
    ref, tol = torch.empty((2, c.H, c.D), dtype=torch.float64)
    K, V = c.k[0, :, 0], c.v[0, :, 0].double()
    for h in range(c.H):
        s, w = weights(c.q[0, h], K, c.D)
        w = w / w.sum()
        ref[h] = w @ V
        dot = (K.double().abs() @ c.q[0, h].double().abs()).max() / math.sqrt(c.D)
        d = (c.D + 8) * 2.0 ** -24 * dot + 4 * 2.0 ** -24 * s.abs().max() + 2.0 ** -21
        e = (w @ V.abs()) * (2 * (d + N * 2.0 ** -24) + TWO_PARTS[c.t])
        if c.t is torch.float16:
            e = e + N * 2.0 ** -35
        tol[h] = e + half_step(ref[h].abs() + e, c.t)
    return ref, tol


def modelled(c, parts):
    """The result with weights rounded to `parts` numbers of the type, exact otherwise but for
    its own rounding."""
    out = torch.empty((c.H, c.D), dtype=torch.float64)
    less = 1 - torch.finfo(c.t).eps
    for h in range(c.H):
        _, w = weights(c.q[0, h], c.k[0, :, 0], c.D)
        r = rounded(w, c.t)
        if parts == 2:
            r = rounded(w * less, c.t)
            r = r + rounded(w - r, c.t)
        out[h] = (r @ c.v[0, :, 0].double()) / w.sum()
    return out.to(c.t).double()
