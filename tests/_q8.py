"""Plain 64-bit forms of the rotary operator and the 8-bit KV cache (numpy), and
inputs for their tests."""
from __future__ import annotations

import math

import numpy as np
import torch

QMAX = {"e4m3": 448.0, "int8": 127.0}
TORCH = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}


# ------------------------------------------------------------------ rotation

def theta(rope_dims: int, base: float, scaling=None) -> np.ndarray:
    d = rope_dims
    i = np.arange(d // 2, dtype=np.float64)
    kind = None if scaling is None else scaling.kind
    if kind == "base":
        base = base * scaling.factor ** (d / (d - 2))
    t = base ** (-2.0 * i / d)
    if kind == "linear":
        t = t / scaling.factor
    if kind == "by_parts":
        r = scaling.original_len * t / (2 * np.pi)
        g = np.clip((r - scaling.low_turns) / (scaling.high_turns - scaling.low_turns), 0, 1)
        t = t * (g + (1 - g) / scaling.factor)
    return t


def rotate(x: np.ndarray, pos, rope_dims: int = 0, base: float = 10000.0, trad: bool = False,
           scaling=None, gradient: bool = False) -> np.ndarray:
    """x [tokens, heads, dim] (any float type) rotated in 64 bits."""
    x = np.asarray(x, dtype=np.float64)
    d = rope_dims or x.shape[-1]
    # p theta reduced modulo 2 pi in extended precision: in 64 bits the product at
    # positions near 2^32 is off by 2^-21
    turns = np.multiply.outer(np.asarray(pos, np.longdouble),
                              theta(d, base, scaling).astype(np.longdouble))
    a = np.fmod(turns, 2 * np.longdouble("3.14159265358979323846264338327950288"))
    a = a.astype(np.float64)[:, None, :]
    m = 1.0 if scaling is None else scaling.magnitude
    c, s = m * np.cos(a), m * np.sin(a) * (-1 if gradient else 1)
    y = x.copy()
    if trad:
        u, w = x[..., 0:d:2], x[..., 1:d:2]
        y[..., 0:d:2], y[..., 1:d:2] = u * c - w * s, u * s + w * c
    else:
        u, w = x[..., : d // 2], x[..., d // 2: d]
        y[..., : d // 2], y[..., d // 2: d] = u * c - w * s, u * s + w * c
    return y


def pair_size(x, rope_dims: int, trad: bool, magnitude: float = 1.0) -> np.ndarray:
    """magnitude (|u| + |w|) of the pair each channel belongs to; 0 past rope_dims."""
    a = np.abs(np.asarray(x, np.float64)) * magnitude
    m = np.zeros_like(a)
    h = rope_dims // 2
    if trad:
        s = a[..., 0:rope_dims:2] + a[..., 1:rope_dims:2]
        m[..., 0:rope_dims:2] = m[..., 1:rope_dims:2] = s
    else:
        s = a[..., :h] + a[..., h:rope_dims]
        m[..., :h] = m[..., h:rope_dims] = s
    return m


# Error of a rotated element before its rounding, relative to |u| + |w|: cos and
# sin are off by at most 1.5e-7, cos and sin times the magnitude and the two products
# round by 2^-24 each (at most 2.4e-7 together).
ROTATION = 4e-7


def half_step(ref: np.ndarray, eps: float, tiny: float) -> np.ndarray:
    """Half a step of a float type at |ref|: eps / 2 relative to the power of two
    below it, half of `tiny` in the subnormal range."""
    a = np.maximum(np.abs(ref), tiny / eps)
    return eps / 2 * 2.0 ** np.floor(np.log2(a)) * (1 + 1e-12)


# --------------------------------------------------------------- 8-bit cache

def values(cache: torch.Tensor) -> np.ndarray:
    return cache.cpu().float().numpy().astype(np.float64)


def round8(x: np.ndarray, kv: str) -> np.ndarray:
    """The 8-bit value nearest to x, ties to even, saturating."""
    x = np.asarray(x, np.float64)
    if kv == "int8":
        return np.clip(np.rint(np.nan_to_num(x, nan=0.0, posinf=127, neginf=-127)), -127, 127)
    with np.errstate(invalid="ignore"):
        e = np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -6)))
        step = 2.0 ** (np.minimum(e, 8) - 3)
        return np.clip(np.rint(x / step) * step, -448, 448)


def half_step8(x: np.ndarray, kv: str) -> np.ndarray:
    """Half the distance of neighbouring 8-bit values at x."""
    if kv == "int8":
        return np.full_like(np.asarray(x, np.float64), 0.5)
    return 2.0 ** (np.floor(np.log2(np.clip(np.abs(x), 2.0 ** -6, 448.0))) - 4)


def need_scale(amax: np.ndarray, kv: str) -> np.ndarray:
    s = np.full(np.shape(amax), 2.0 ** -32)
    while (amax > QMAX[kv] * s).any():
        s = np.where(amax > QMAX[kv] * s, 2 * s, s)
    return s


def to_cache(x: np.ndarray, kv: str, device="cuda") -> torch.Tensor:
    """8-bit values (exact) as a tensor of the cache's type."""
    t = torch.from_numpy(np.ascontiguousarray(x))
    return (t.to(torch.int8) if kv == "int8" else t.float().to(torch.float8_e4m3fn)).to(device)


def random_cache(rng, lead: int, rows: int, hk: int, d: int, block: int, kv: str, spread=1.0):
    """Values and scales of a cache whose blocks hold normal values of different
    size: (values [lead, rows, hk, d] in 8-bit units, scales)."""
    nb = -(-rows // block)
    x = rng.standard_normal((lead, nb * block, hk, d))
    x = x.reshape(lead, nb, block, hk, d) * np.exp(spread * rng.standard_normal((lead, nb, 1, hk, 1)))
    s = need_scale(np.abs(x).max(axis=(2, 4)), kv)
    q = round8(x / s[:, :, None, :, None], kv).reshape(lead, nb * block, hk, d)[:, :rows]
    return q, s.astype(np.float32)


def decode(q, kq, vq, ks, vs, cur_pos, block: int, table=None, page: int = 0):
    """out [B, H, D] in 64 bits and, per element, sum_p w_p |v_p|; per (b, h) the
    largest sum |q_i k_i| and the largest |s|, which bound the error of the scores.
    kq, vq: 8-bit values as float64; ks, vs: scales."""
    q = np.asarray(q, np.float64)
    B, H, D = q.shape
    hk = kq.shape[2]
    g = H // hk
    out, size = np.zeros((B, H, D)), np.zeros((B, H, D))
    dot, top = np.zeros((B, H)), np.zeros((B, H))
    cap = kq.shape[1] if table is None else page * table.shape[1]
    for b in range(B):
        L = min(int(cur_pos[b]), cap - 1) + 1
        p = np.arange(L)
        lead = np.full(L, b) if table is None else table[b, p // page]
        row = p if table is None else p % page
        k = kq[lead, row] * ks[lead, row // block][..., None].astype(np.float64)
        v = vq[lead, row] * vs[lead, row // block][..., None].astype(np.float64)
        for h in range(H):
            e = h // g
            s = k[:, e] @ q[b, h] / math.sqrt(D)
            w = np.exp(s - s.max())
            w /= w.sum()
            out[b, h], size[b, h] = w @ v[:, e], w @ np.abs(v[:, e])
            dot[b, h] = (np.abs(k[:, e]) @ np.abs(q[b, h])).max() / math.sqrt(D)
            top[b, h] = np.abs(s).max()
    return out, size, dot, top


def decode_bound(ref, size, dot, top, L: int, D: int, vs) -> np.ndarray:
    """How far the kernel may be from `ref`: each weight carries the rounding of P
    to f16 (2^-11), the error of its score (D products and sums in fp32, the scale
    and the exponent's fused sum, whose size is |s| log2e plus |log2 vs|), ex2 and
    lg2 (2^-21 together); numerator and denominator both; L fp32 additions; then
    the output's own rounding to f16."""
    lv = np.abs(np.log2(np.maximum(vs, 2.0 ** -100))).max()
    score = (D + 4) * 2.0 ** -24 * dot + 2.0 ** -23 * (1.5 * top + lv) + 2.0 ** -21
    weight = 2.0 ** -11 + 2 * score + 2 * L * 2.0 ** -24
    return weight[..., None] * size + half_step(ref, 2.0 ** -10, 2.0 ** -24)


def check(got: np.ndarray, ref: np.ndarray, bound: np.ndarray, what: str) -> None:
    assert got.shape == ref.shape, f"{what}: shape {got.shape}, expected {ref.shape}"
    err = np.abs(got - ref)
    bad = ~(err <= bound)
    if bad.any():
        i = tuple(int(v) for v in np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} outside the bound, first at {i}: "
                             f"got {got[i]!r}, expected {ref[i]!r}, bound {bound[i]:.3g}")


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().to(torch.float64).numpy()
