"""Cases, plain forms and 64-bit definitions of three operators of a decode step
whose KV cache is held in 8 bits:

  rope     rotary positions of many tokens: both pair layouts, part of the head,
           frequencies scaled for long contexts, and the gradient
  append   rotate the new tokens of a ragged batch and append their keys and
           values to an 8-bit cache (dense or paged) that has one scale for each
           block of tokens and head
  decode   single-query attention over that cache, query heads sharing key/value
           heads in groups

``run`` is the plain form in elementary torch operations while ``own`` is false,
and the package's calls while it is true.
"""
from __future__ import annotations

import math

import torch

own = False

QMAX = {"e4m3": 448.0, "int8": 127.0}  # largest magnitude of the 8-bit types
MIN_EXP = -32  # scales are powers of two, 2^-32 at least
DEV = "cuda"


# --------------------------------------------------------------------- cases

def listed():
    return [
        # one token of a decode step, 32 heads of 128: latency
        dict(name="rope_token", op="rope", dtype="f16", tokens=1, heads=32, dim=128,
             rope_dims=128, trad=False, scaling="none", base=10000.0, grad=False),
        # a prompt chunk of 8192 tokens in a model run past its trained length
        dict(name="rope_prompt", op="rope", dtype="bf16", tokens=8192, heads=32, dim=128,
             rope_dims=128, trad=False, scaling="by_parts", base=500000.0, grad=False),
        # the backward pass of a training batch, half of each head rotated,
        # adjacent pairs, f32 gradients
        dict(name="rope_grad", op="rope", dtype="f32", tokens=4095, heads=40, dim=128,
             rope_dims=64, trad=True, scaling="linear", base=10000.0, grad=True),
        # one token of one sequence, the 7B-class step (32 heads of 128, 4096 positions)
        dict(name="append_token", op="append", kv="e4m3", batch=1, tokens=1, ragged=False,
             heads=32, kv_heads=32, dim=128, seq_len=4096, page=0, block=16, pad=0,
             rope_dims=128, trad=False, scaling="none", base=10000.0),
        # one token for each of 256 sequences, 40 heads, a paged cache
        dict(name="append_batch", op="append", kv="e4m3", batch=256, tokens=256, ragged=False,
             heads=40, kv_heads=40, dim=128, seq_len=128, page=16, block=16, pad=0,
             rope_dims=128, trad=False, scaling="linear", base=10000.0),
        # prompt chunks of four sequences, 8192 tokens together, grouped heads
        dict(name="append_prompt", op="append", kv="e4m3", batch=4, tokens=8192, ragged=True,
             heads=32, kv_heads=8, dim=128, seq_len=8192, page=64, block=32, pad=0,
             rope_dims=128, trad=False, scaling="by_parts", base=500000.0),
        # a mixed step in int8: some sequences bring a chunk, some one token,
        # some none; the rows of the batch are padded to a fixed count
        dict(name="append_int8", op="append", kv="int8", batch=13, tokens=301, ragged=True,
             heads=20, kv_heads=4, dim=80, seq_len=216, page=24, block=8, pad=19,
             rope_dims=40, trad=True, scaling="none", base=10000.0),
        # the smallest decode step
        dict(name="decode_small", op="decode", kv="e4m3", batch=1, heads=8, kv_heads=8, dim=64,
             seq_len=256, live=201, page=0, block=16),
        # the 7B-class step with four query heads to a key/value head, small pages
        dict(name="decode_7b", op="decode", kv="int8", batch=1, heads=32, kv_heads=8, dim=128,
             seq_len=4096, live=4096, page=16, block=16),
        # a ragged batch of odd shape
        dict(name="decode_odd", op="decode", kv="int8", batch=37, heads=20, kv_heads=4, dim=80,
             seq_len=1992, live=0, page=24, block=8),
        # a ragged batch of 64 sequences, 32 heads, pages of 128
        dict(name="decode_ragged", op="decode", kv="e4m3", batch=64, heads=32, kv_heads=32,
             dim=128, seq_len=2048, live=0, page=128, block=32),
        # one long context, 1 GiB of cache
        dict(name="decode_long", op="decode", kv="e4m3", batch=1, heads=32, kv_heads=32, dim=128,
             seq_len=131072, live=131072, page=0, block=64),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("rope", "append", "decode", "decode"))
    dim = rng.choice((64, 80, 96, 128, 128, 256))
    scaling = rng.choice(("none", "linear", "base", "by_parts"))
    base = rng.choice((10000.0, 500000.0, 1e6))
    trad = rng.random() < 0.5
    rope_dims = rng.choice((dim, dim, dim // 2, dim // 4))
    if op == "rope":
        heads = _log(rng, 1, 64)
        return dict(op=op, dtype=rng.choice(("f16", "bf16", "f32")),
                    tokens=_log(rng, 1, 16 * 2 ** 20 // (heads * dim)), heads=heads, dim=dim,
                    rope_dims=rope_dims, trad=trad, scaling=scaling, base=base,
                    grad=rng.random() < 0.4)
    kv_heads = rng.choice((1, 2, 4, 8, 8, 16, 32, 40))
    heads = kv_heads * rng.choice([g for g in (1, 2, 3, 4, 5, 8, 16) if g * kv_heads <= 64])
    kv = rng.choice(("e4m3", "int8"))
    block = rng.choice((1, 8, 16, 32, 64, 128))
    page = rng.choice((0, block, 2 * block, 3 * block))
    if op == "append":
        batch = _log(rng, 1, 64)
        ragged = rng.random() < 0.6
        tokens = batch if not ragged else _log(rng, batch, max(batch, 2 ** 22 // (kv_heads * dim)))
        longest = -(-3 * tokens // batch) if ragged else 1
        unit = page or block
        seq_len = unit * max(1, -(-(longest + rng.randrange(1, 200)) // unit))
        return dict(op=op, kv=kv, batch=batch, tokens=tokens, ragged=ragged, heads=heads,
                    kv_heads=kv_heads, dim=dim, seq_len=seq_len, page=page, block=block,
                    pad=rng.choice((0, 0, 7)), rope_dims=rope_dims, trad=trad, scaling=scaling,
                    base=base)
    batch = _log(rng, 1, 256)
    most = max(1, 2 ** 27 // (batch * kv_heads * dim))
    seq_len = _log(rng, 1, min(131072, most))
    if page:
        seq_len = page * max(1, seq_len // page)
    return dict(op=op, kv=kv, batch=batch, heads=heads, kv_heads=kv_heads, dim=dim,
                seq_len=seq_len, live=0 if batch > 1 else seq_len - rng.randrange(0, seq_len),
                page=page, block=block)


# ------------------------------------------------- sizes that a case stands for

def _live(c):
    """Live lengths of a decode case: the given one, or spread evenly over 1 .. seq_len."""
    if c["live"]:
        return [c["live"]] * c["batch"]
    return [1 + (2 * i + 1) * (c["seq_len"] - 1) // (2 * c["batch"]) for i in range(c["batch"])]


def _counts(c):
    """New tokens of each sequence of an append case: one, or shares of the total
    in the ratio 3 : 0 : 2 : 1 : ... around a mean of tokens / batch."""
    B, T = c["batch"], c["tokens"]
    if not c["ragged"]:
        return [1] * B
    w = [(3.0, 0.0, 2.0, 1.0)[i % 4] for i in range(B)]
    n = [int(T * x / sum(w)) for x in w]
    left = T - sum(n)
    return [n[i] + (left if i == 0 else 0) for i in range(B)]


def _scaling(c):
    """(kind, factor, original length, low turns, high turns, magnitude)."""
    return {"none": ("none", 1.0, 0.0, 0.0, 0.0, 1.0),
            "linear": ("linear", 4.0, 0.0, 0.0, 0.0, 1.0),
            "base": ("base", 8.0, 0.0, 0.0, 0.0, 1.0),
            "by_parts": ("by_parts", 8.0, 8192.0, 1.0, 32.0, 0.1 * math.log(8.0) + 1.0),
            }[c["scaling"]]


def _nblk(c):
    return -(-c["seq_len"] // c["block"])


def work(c):
    if c["op"] == "rope":
        n, e = c["tokens"] * c["heads"], {"f16": 2, "bf16": 2, "f32": 4}[c["dtype"]]
        return {"bytes": 2 * n * c["dim"] * e + 4 * c["tokens"], "flops": 3 * n * c["rope_dims"]}
    if c["op"] == "append":
        T, D = sum(_counts(c)), c["dim"]
        new = T * c["kv_heads"] * D
        blocks = sum(-(-n // c["block"]) for n in _counts(c)) * c["kv_heads"]
        return {"bytes": 4 * T * c["heads"] * D + 2 * new * 3 + 2 * 4 * blocks + 4 * c["batch"],
                "flops": 3 * T * (c["heads"] + c["kv_heads"]) * c["rope_dims"] + 4 * new}
    live = sum(_live(c))
    blocks = sum(-(-n // c["block"]) for n in _live(c))
    return {"bytes": 2 * live * c["kv_heads"] * c["dim"] + 8 * blocks * c["kv_heads"]
            + 4 * c["batch"] * c["heads"] * c["dim"], "flops": 4 * live * c["heads"] * c["dim"]}


# -------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(shape, g, dtype):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)


def _filled_cache(c, lead, slots, g):
    """A cache [lead, slots, kv_heads, dim] in 8 bits and its block scales, as
    appending normal values block after block leaves it."""
    H, D, blk, top = c["kv_heads"], c["dim"], c["block"], QMAX[c["kv"]]
    nb = -(-slots // blk)
    x = torch.randn((lead, nb, blk, H, D), generator=g, device=DEV, dtype=torch.float32)
    x *= torch.exp(0.5 * torch.randn((lead, nb, 1, H, 1), generator=g, device=DEV))
    amax = x.abs().amax(dim=(2, 4))
    scale = torch.exp2(torch.ceil(torch.log2(amax / top)))
    x = (x / scale[:, :, None, :, None]).clamp_(-top, top)
    q = x.round_().to(torch.int8) if c["kv"] == "int8" else x.to(torch.float8_e4m3fn)
    return q.view(lead, nb * blk, H, D)[:, :slots].contiguous(), scale.contiguous()


def _table(c, g, spare):
    """A block table of distinct pages in random order, and the pool's size."""
    per = c["seq_len"] // c["page"]
    n = c["batch"] * per + spare
    order = torch.randperm(n, generator=g, device=DEV)[: c["batch"] * per]
    return order.view(c["batch"], per).to(torch.int32), n


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": c}
    host = torch.Generator().manual_seed(seed)
    if c["op"] == "rope":
        dtype = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}[c["dtype"]]
        s["x"] = _randn((c["tokens"], c["heads"], c["dim"]), g, dtype)
        first = int(torch.randint(0, 100000, (1,), generator=host))
        s["pos"] = (torch.arange(c["tokens"], device=DEV) + first).to(torch.int32)
        return s
    B, H, Hk, D = c["batch"], c["heads"], c["kv_heads"], c["dim"]
    turn = torch.randperm(B, generator=host).tolist()
    if c["op"] == "append":
        n = [_counts(c)[i] for i in turn]
        T = sum(n)
        rows = T + c["pad"]
        s["count"] = T
        s["q"], s["q_out"] = _randn((rows, H, D), g, torch.float16), _randn((rows, H, D), g, torch.float16)
        s["k"], s["v"] = (_randn((rows, Hk, D), g, torch.float16) for _ in range(2))
        last = [int(torch.randint(max(x, 1) - 1, c["seq_len"], (1,), generator=host)) for x in n]
        s["pos"] = torch.tensor(last, dtype=torch.int32, device=DEV)
        s["offsets"] = None
        if c["ragged"] or c["pad"]:
            off = [0]
            for x in n:
                off.append(off[-1] + x)
            s["offsets"] = torch.tensor(off, dtype=torch.int32, device=DEV)
    else:
        s["q"] = _randn((B, H, D), g, torch.float16)
        s["pos"] = torch.tensor([_live(c)[i] - 1 for i in turn], dtype=torch.int32, device=DEV)
    s["table"] = None
    lead, slots = B, c["seq_len"]
    if c["page"]:
        s["table"], lead = _table(c, g, 3)
        slots = c["page"]
    s["kc"], s["ks"] = _filled_cache(c, lead, slots, g)
    s["vc"], s["vs"] = _filled_cache(c, lead, slots, g)
    return s


# --------------------------------------------------------------- plain forms

def _theta(c):
    """theta_i of the pairs in 64 bits, and the magnitude."""
    kind, factor, length, low, high, mag = _scaling(c)
    d = c["rope_dims"]
    i = torch.arange(d // 2, device=DEV, dtype=torch.float64)
    base = c["base"] * (factor ** (d / (d - 2)) if kind == "base" else 1.0)
    theta = torch.exp(-2.0 * i / d * math.log(base))
    if kind == "linear":
        theta = theta / factor
    if kind == "by_parts":
        keep = ((length * theta / (2 * math.pi) - low) / (high - low)).clamp(0.0, 1.0)
        theta = theta * keep + theta / factor * (1.0 - keep)
    return theta, mag


def _turned(x, pos, c, sign):
    """x [T, heads, dim] in 32 bits, rotated by sign * pos * theta."""
    theta, mag = _theta(c)
    a = pos.to(torch.float64)[:, None, None] * theta
    cos, sin = (mag * a.cos()).float(), (sign * mag * a.sin()).float()
    d = c["rope_dims"]
    x = x.float()
    y = x.clone()
    if c["trad"]:
        u, w = x[..., 0:d:2], x[..., 1:d:2]
        y[..., 0:d:2], y[..., 1:d:2] = u * cos - w * sin, u * sin + w * cos
    else:
        u, w = x[..., : d // 2], x[..., d // 2: d]
        y[..., : d // 2], y[..., d // 2: d] = u * cos - w * sin, u * sin + w * cos
    return y


def _to8(x, kv):
    x = x.clamp(-QMAX[kv], QMAX[kv])
    return x.round().to(torch.int8) if kv == "int8" else x.to(torch.float8_e4m3fn)


def _put(cache, scale, x, blk, row, before, slot, c):
    """Append x [T, Hk, D] to rows `row` of `cache`, in block `blk` of `scale` each;
    `slot` and `before`: for each sequence the block that its first new token is
    in and how many rows of it were there before."""
    H, D, n, kv = c["kv_heads"], c["dim"], c["block"], c["kv"]
    flat, scales = cache.view(torch.uint8).view(-1, H, D), scale.view(-1, H)
    amax = torch.zeros_like(scales)
    amax.scatter_reduce_(0, blk[:, None].expand(-1, H), x.abs().amax(-1), "amax")
    m, e = torch.frexp(amax)  # amax = m 2^e with m in [1/2, 1), or 0
    top_m, top_e = math.frexp(QMAX[kv])
    e = torch.where(m <= top_m, e - top_e, e - top_e + 1).clamp(min=MIN_EXP)
    e = torch.where(amax > 0, e, MIN_EXP)
    new = ((e + 127) << 23).view(torch.float32)  # 2^e
    # a block that has rows from before keeps its scale unless it has to grow
    has = torch.zeros(scales.shape[0], 1, dtype=torch.bool, device=DEV)
    has[slot] = (before > 0)[:, None]
    new = torch.where(has, torch.maximum(scales, new), new)
    # those rows on the new scale; the other rows of the block are left out by
    # writing its first row once more
    per = c["page"] // n if c["page"] else _nblk(c)
    lead = slot // per * (c["page"] or c["seq_len"]) + slot % per * n
    r = torch.arange(n, device=DEV)
    at = lead[:, None] + torch.where(r < before[:, None], r, 0)
    was = flat[at]
    now = _to8(was.view(cache.dtype).float() * (scales / new)[slot][:, None, :, None], kv)
    flat[at] = torch.where((before > 0)[:, None, None, None], now.view(torch.uint8), was)
    flat[row] = _to8(x / new[blk][:, :, None], kv).view(torch.uint8)
    scales[blk] = new[blk]


def _places(s):
    """For each new token its sequence and position, and (row, block) of the cache."""
    c = s["case"]
    B, T = c["batch"], s["count"]
    off = s["offsets"].long() if s["offsets"] is not None else torch.arange(B + 1, device=DEV)
    t = torch.arange(T, device=DEV)
    b = torch.searchsorted(off, t, right=True) - 1
    first = s["pos"].long() - (off[1:] - off[:-1]) + 1
    return b, first[b] + t - off[b], first, off[1:] > off[:-1]


def _where(b, p, s):
    c = s["case"]
    n = c["block"]
    if not c["page"]:
        return b * c["seq_len"] + p, b * _nblk(c) + p // n
    page = s["table"].long()[b, p // c["page"]]
    return page * c["page"] + p % c["page"], page * (c["page"] // n) + p % c["page"] // n


def _plain_append(s):
    c = s["case"]
    T = s["count"]
    b, p, first, any_new = _places(s)
    k = _turned(s["k"][:T], p, c, 1.0)
    s["q_out"][:T] = _turned(s["q"][:T], p, c, 1.0).half()
    row, blk = _where(b, p, s)
    one = torch.arange(c["batch"], device=DEV)
    start = torch.where(any_new, first, 0)
    before = torch.where(any_new, start % c["block"], 0)
    _, slot = _where(one, start, s)
    _put(s["kc"], s["ks"], k, blk, row, before, slot, c)
    _put(s["vc"], s["vs"], s["v"][:T].float(), blk, row, before, slot, c)


def _values(cache, scale, c):
    """The 16-bit values that an 8-bit cache stands for."""
    n = c["block"]
    lead, slots = cache.shape[:2]
    s = scale.repeat_interleave(n, dim=1)[:, :slots]
    return cache.float().mul_(s[..., None]).half()


def _plain_decode(s):
    c = s["case"]
    B, H, Hk, D, n = c["batch"], c["heads"], c["kv_heads"], c["dim"], c["block"]
    kc, vc, ks, vs = s["kc"], s["vc"], s["ks"], s["vs"]
    if s["table"] is not None:
        t = s["table"].long()
        kc, vc = (x.view(torch.uint8)[t].view(x.dtype).view(B, -1, Hk, D) for x in (kc, vc))
        ks, vs = (x[t].view(B, -1, Hk) for x in (ks, vs))
    S = kc.shape[1]
    q = s["q"].float().view(B, Hk, H // Hk, D)
    score = q @ kc.permute(0, 2, 3, 1).float()  # [B, Hk, group, S]
    score *= ks.repeat_interleave(n, dim=1)[:, :S].permute(0, 2, 1)[:, :, None] / math.sqrt(D)
    dead = torch.arange(S, device=DEV) > s["pos"].long()[:, None]
    score.masked_fill_(dead[:, None, None], -math.inf)
    w = torch.exp(score - score.amax(-1, keepdim=True))
    total = w.sum(-1, keepdim=True)
    w *= vs.repeat_interleave(n, dim=1)[:, :S].permute(0, 2, 1)[:, :, None]
    return ((w @ vc.permute(0, 2, 1, 3).float()) / total).half().view(B, H, D)


def run(state):
    s, c = state, state["case"]
    if own:
        import token_decode_attention_gb300 as dattn
        if c["op"] != "decode":
            kind, factor, length, low, high, mag = _scaling(c)
            scaling = None if kind == "none" else dattn.RopeScaling(
                kind, factor, original_len=length, low_turns=low, high_turns=high, magnitude=mag)
        if c["op"] == "rope":
            return dattn.rope(s["x"], s["pos"], c["rope_dims"], c["base"], c["trad"], scaling,
                              gradient=c["grad"])
        if c["op"] == "append":
            dattn.rope_append_q8(s["q"], s["k"], s["v"], s["kc"], s["vc"], s["ks"], s["vs"],
                                 s["pos"], c["block"], token_offsets=s["offsets"],
                                 rope_dims=c["rope_dims"], rope_base=c["base"],
                                 traditional=c["trad"], scaling=scaling,
                                 block_table=s["table"], q_out=s["q_out"])
        elif s["table"] is None:
            return dattn.decode_q8(s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["pos"],
                                   c["block"])
        else:
            return dattn.decode_paged_q8(s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"],
                                         s["pos"], c["block"])
    elif c["op"] == "rope":
        return _turned(s["x"], s["pos"], c, -1.0 if c["grad"] else 1.0).to(s["x"].dtype)
    elif c["op"] == "append":
        _plain_append(s)
    else:
        return _plain_decode(s)
    if c["kv"] == "int8":  # whole numbers on a scale: the values they stand for
        return [s["q_out"], _values(s["kc"], s["ks"], c), _values(s["vc"], s["vs"], c), s["ks"], s["vs"]]
    return [s["q_out"], s["kc"], s["vc"], s["ks"], s["vs"]]


# ------------------------------------------------------ 64-bit definitions

def _exact_angles(c, pos):
    kind, factor, length, low, high, mag = _scaling(c)
    d, base = c["rope_dims"], c["base"]
    if kind == "base":
        base *= factor ** (d / (d - 2))
    rows = []
    for i in range(d // 2):
        th = base ** (-2.0 * i / d)
        if kind == "linear":
            th /= factor
        if kind == "by_parts":
            turns = length * th / (2.0 * math.pi)
            g = min(1.0, max(0.0, (turns - low) / (high - low)))
            th = (1.0 - g) * th / factor + g * th
        rows.append(th)
    return torch.outer(pos.double(), torch.tensor(rows, dtype=torch.float64, device=pos.device)), mag


def _exact_turn(x, pos, c, back):
    """Pairs as complex numbers times mag e^(+-i angle)."""
    a, mag = _exact_angles(c, pos)
    d, x = c["rope_dims"], x.double()
    z = torch.polar(torch.full_like(a, mag), -a if back else a)[:, None]
    head = x[..., :d]
    if c["trad"]:
        p = head.unflatten(-1, (d // 2, 2))
    else:
        p = head.unflatten(-1, (2, d // 2)).transpose(-1, -2)
    y = torch.view_as_real(torch.complex(p[..., 0].contiguous(), p[..., 1].contiguous()) * z)
    y = y.flatten(-2) if c["trad"] else y.transpose(-1, -2).flatten(-2)
    return torch.cat([y, x[..., d:]], -1)


def _exact_round8(x, kv):
    """To the nearest value of the type, ties to even, saturating."""
    if kv == "int8":
        return torch.round(x).clamp(-127, 127)
    _, e = torch.frexp(x)
    step = (((e.long() - 4).clamp(min=-9) + 1023) << 52).view(torch.float64)  # 2^(e - 4)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _exact_scale(amax, kv):
    """Smallest power of two s >= 2^-32 with amax <= QMAX s."""
    s = torch.full_like(amax, 2.0 ** MIN_EXP)
    while bool((amax > QMAX[kv] * s).any()):
        s = torch.where(amax > QMAX[kv] * s, 2 * s, s)
    return s


def _exact_append(c, s):
    kv, n, T, page = c["kv"], c["block"], s["count"], c["page"]
    off = s["offsets"].tolist() if s["offsets"] is not None else list(range(c["batch"] + 1))
    last = s["pos"].tolist()
    pos = [last[b] - (off[b + 1] - off[b]) + 1 + j for b in range(c["batch"]) for j in range(off[b + 1] - off[b])]
    pos = torch.tensor(pos, dtype=torch.int64, device=DEV)
    q_out = s["q_out"].double()
    q_out[:T] = _exact_turn(s["q"][:T], pos, c, False)
    out = []
    for cache, scale, x in ((s["kc"], s["ks"], _exact_turn(s["k"][:T], pos, c, False)),
                            (s["vc"], s["vs"], s["v"][:T].double())):
        C, S = cache.double(), scale.double()
        for b in range(c["batch"]):
            t, p1 = off[b], last[b] + 1
            p = p1 - (off[b + 1] - off[b])
            while p < p1:
                blk, stop = p // n, min(p1, (p // n + 1) * n)
                lead = b if not page else int(s["table"][b, p // page])
                row, sb = (p, blk) if not page else (p % page, p % page // n)
                was, start = p - blk * n, row - (p - blk * n)
                new = x[t: t + stop - p]
                sc = _exact_scale(new.abs().amax((0, 2)), kv)
                if was:
                    sc = torch.maximum(sc, S[lead, sb])
                    C[lead, start: row] = _exact_round8(C[lead, start: row] * (S[lead, sb] / sc)[:, None], kv)
                S[lead, sb] = sc
                C[lead, row: row + stop - p] = _exact_round8(new / sc[:, None], kv)
                t, p = t + stop - p, stop
        out.append((C, S))
    (K, ks), (V, vs) = out
    if kv == "int8":
        slots = K.shape[1]
        at = torch.arange(slots, device=DEV) // n
        K, V = K * ks[:, at][..., None], V * vs[:, at][..., None]
    return [q_out, K, V, ks, vs]


def _exact_decode(c, s):
    B, H, Hk, D, n, page = (c[k] for k in ("batch", "heads", "kv_heads", "dim", "block", "page"))
    out = torch.empty((B, H, D), dtype=torch.float64, device=DEV)
    for b in range(B):
        L = min(int(s["pos"][b]) + 1, c["seq_len"])
        p = torch.arange(L, device=DEV)
        lead = torch.full_like(p, b) if not page else s["table"][b].long()[p // page]
        row = p if not page else p % page
        for h in range(Hk):
            K, V = (x.view(torch.uint8)[lead, row, h].view(x.dtype).double() for x in (s["kc"], s["vc"]))
            K = K * s["ks"][lead, row // n, h].double()[:, None]
            V = V * s["vs"][lead, row // n, h].double()[:, None]
            g = slice(h * (H // Hk), (h + 1) * (H // Hk))
            w = torch.softmax(s["q"][b, g].double() @ K.T / D ** 0.5, -1)
            out[b, g] = w @ V
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_turn(s["x"], s["pos"], case, case["grad"])
    return _exact_append(case, s) if case["op"] == "append" else _exact_decode(case, s)
