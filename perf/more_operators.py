"""Cases, plain forms and 64-bit definitions of two forms of attention over a 16-bit
(f16 or bf16) KV cache with grouped heads, dense or paged:

  attend   one token per sequence, or the ragged tokens of a prompt or a mixed step,
           each seeing the positions up to its own: all of them, or a sliding window
           and a few first tokens that stay visible (sinks)
  shared   one token per sequence for a batch whose sequences share a long prefix,
           which is read once for all

``run`` is the plain form in elementary torch operations while ``own`` is false,
and the package's calls while it is true.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
ROWS = 1024  # query tokens that the plain form of a prompt takes at a time


# --------------------------------------------------------------------- cases

def listed():
    return [
        # one token of a 7B-class step with four query heads to a key/value head: latency
        dict(name="window_token", op="attend", dtype="f16", batch=1, tokens=1, ragged=False,
             heads=32, kv_heads=8, dim=128, seq_len=4096, live=4096, page=0, window=1024, sinks=4,
             pad=0, fresh=False),
        # one token for each of 64 sequences behind a window, a cache in pages
        dict(name="window_batch", op="attend", dtype="bf16", batch=64, tokens=64, ragged=False,
             heads=32, kv_heads=8, dim=128, seq_len=8192, live=0, page=64, window=4096, sinks=4,
             pad=0, fresh=False),
        # a ragged batch of odd shape, pages that divide nothing
        dict(name="window_odd", op="attend", dtype="f16", batch=37, tokens=37, ragged=False,
             heads=20, kv_heads=4, dim=80, seq_len=1992, live=0, page=24, window=333, sinks=5,
             pad=0, fresh=False),
        # one long context, every position visible
        dict(name="long_token", op="attend", dtype="bf16", batch=1, tokens=1, ragged=False,
             heads=64, kv_heads=8, dim=128, seq_len=131072, live=131072, page=0, window=0, sinks=0,
             pad=0, fresh=False),
        # a small mixed step of odd shape, padded to a fixed count of rows
        dict(name="prompt_odd", op="attend", dtype="f16", batch=13, tokens=301, ragged=True,
             heads=20, kv_heads=4, dim=80, seq_len=216, live=0, page=24, window=77, sinks=3,
             pad=19, fresh=False),
        # a prompt of 8192 tokens in a model with windows and sinks
        dict(name="prompt_window", op="attend", dtype="bf16", batch=1, tokens=8192, ragged=True,
             heads=32, kv_heads=8, dim=128, seq_len=8192, live=0, page=0, window=1024, sinks=4,
             pad=0, fresh=True),
        # chunks of four sequences' prompts behind what is cached of them, in pages
        dict(name="prompt_chunks", op="attend", dtype="f16", batch=4, tokens=2048, ragged=True,
             heads=32, kv_heads=8, dim=128, seq_len=8192, live=0, page=64, window=0, sinks=0,
             pad=0, fresh=False),
        # a whole prompt of 16384 tokens
        dict(name="prompt_long", op="attend", dtype="bf16", batch=1, tokens=16384, ragged=True,
             heads=32, kv_heads=8, dim=128, seq_len=16384, live=0, page=0, window=0, sinks=0,
             pad=0, fresh=True),
        # four samples of one short prompt
        dict(name="shared_small", op="shared", dtype="f16", batch=4, heads=32, kv_heads=8, dim=128,
             prefix=512, own=64, page=0),
        # 64 requests behind one system prompt, a cache in pages
        dict(name="shared_batch", op="shared", dtype="bf16", batch=64, heads=32, kv_heads=8,
             dim=128, prefix=8192, own=512, page=64),
        # odd shape: a prefix that ends inside a page
        dict(name="shared_odd", op="shared", dtype="f16", batch=37, heads=20, kv_heads=4, dim=80,
             prefix=1000, own=77, page=24),
        # 256 sequences of 40 heads, each with its own key/value head
        dict(name="shared_large", op="shared", dtype="f16", batch=256, heads=40, kv_heads=40,
             dim=128, prefix=8192, own=256, page=0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """A case whose bytes and operations are both within those of the largest listed ones."""
    most = [max(work(c)[k] for c in listed()) for k in ("bytes", "flops")]
    while True:
        c = _any_case(rng)
        w = work(c)
        if w["bytes"] <= most[0] and w["flops"] <= most[1]:
            return c


def _any_case(rng):
    kind = rng.choice(("token", "token", "ragged", "ragged", "shared", "shared"))
    dim = rng.choice((64, 80, 96, 128, 128, 256))
    kv_heads = rng.choice((1, 2, 4, 8, 8, 16, 32, 40))
    heads = kv_heads * rng.choice([g for g in (1, 2, 3, 4, 5, 8, 16) if g * kv_heads <= 64])
    c = dict(op="shared" if kind == "shared" else "attend", dtype=rng.choice(("f16", "bf16")),
             heads=heads, kv_heads=kv_heads, dim=dim)
    page = rng.choice((0, 0, 1, 16, 24, 64, 128))
    batch = _log(rng, 1, 64 if kind == "ragged" else 256)
    room = 2 ** 28 // (kv_heads * dim)  # positions of all sequences together
    if kind == "shared":
        own_len = _log(rng, 1, max(1, min(1024, room // batch)))
        most = 2 ** 36 // (batch * heads * dim)
        return dict(c, batch=batch, prefix=_log(rng, 1, max(2, min(65536, most, room // 2))),
                    own=own_len, page=page)
    window = rng.choice((0, 1, 1, 1))
    sinks = rng.choice((0, 1, 4, 4, 7, 130))
    if kind == "token":
        seq_len = _log(rng, 1, max(1, min(131072, room // batch)))
        tokens, ragged, pad, fresh = batch, False, 0, False
    else:
        most = min(16384, room // 4, int(math.sqrt(2 ** 42 / (heads * dim))))
        tokens = _log(rng, 1, max(1, most))
        longest = -(-3 * tokens // batch) + 1
        more = max(1, min(16384, room // batch, 2 ** 40 // (heads * dim * tokens)))
        fresh = rng.random() < 0.4
        seq_len = longest + (0 if fresh else _log(rng, 1, more))
        ragged, pad = True, rng.choice((0, 0, 7))
    if page:
        seq_len = page * -(-seq_len // page)
    if window:
        window = _log(rng, 1, seq_len)
    live = seq_len - rng.randrange(0, seq_len) if kind == "token" and batch == 1 else 0
    return dict(c, batch=batch, tokens=tokens, ragged=ragged, seq_len=seq_len, live=live, page=page,
                window=window, sinks=sinks, pad=pad, fresh=fresh)


# ------------------------------------------------- sizes that a case stands for

def _spread(lo, hi, i, n):
    """The i-th of n values spread evenly over lo .. hi."""
    return lo + (2 * i + 1) * (hi - lo) // (2 * n)


def _bring(c):
    """(new tokens, position of the last one) of each sequence of an attend case.  Ragged:
    shares of the tokens in the ratio 3 : 0 : 2 : 1 : ..., none for a few."""
    B, S = c["batch"], c["seq_len"]
    if not c["ragged"]:
        return [(1, (c["live"] or _spread(1, S, i, B)) - 1) for i in range(B)]
    w = [(3.0, 0.0, 2.0, 1.0)[i % 4] for i in range(B)]
    n = [int(c["tokens"] * x / sum(w)) for x in w]
    n[0] += c["tokens"] - sum(n)
    return [(x, max(x, 1) - 1 if c["fresh"] else _spread(max(x, 1) - 1, S - 1, i, B))
            for i, x in enumerate(n)]


def _first(c, p):
    """First position of the window of a token at p."""
    return max(0, p - c["window"] + 1) if c["window"] else 0


def _own_lengths(c):
    """Positions of each sequence behind the shared prefix."""
    return [_spread(1, c["own"], i, c["batch"]) for i in range(c["batch"])]


def work(c):
    H, Hk, D = c["heads"], c["kv_heads"], c["dim"]
    if c["op"] == "shared":
        keys, q = c["prefix"] + sum(_own_lengths(c)), c["batch"]
        pairs = c["batch"] * c["prefix"] + sum(_own_lengths(c))
    else:
        keys = pairs = 0
        q = c["tokens"]
        for n, last in _bring(c):
            if n:
                lo = _first(c, last - n + 1)
                keys += last + 1 - lo + min(c["sinks"], lo)
            for p in range(last - n + 1, last + 1):
                lo = _first(c, p)
                pairs += p + 1 - lo + min(c["sinks"], lo)
    return {"bytes": 4 * keys * Hk * D + 4 * q * H * D, "flops": 4 * pairs * H * D}


# -------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(shape, g, dtype):
    return torch.randn(shape, generator=g, device=DEV, dtype=dtype)


def prepare(case, seed):
    c, g = case, _gen(seed)
    host = torch.Generator().manual_seed(seed)
    B, H, Hk, D, page, dtype = (c["batch"], c["heads"], c["kv_heads"], c["dim"], c["page"],
                                DTYPES[c["dtype"]])
    s = {"case": c, "table": None}
    turn = torch.randperm(B, generator=host).tolist()
    if c["op"] == "shared":
        P = c["prefix"]
        lens = [_own_lengths(c)[i] for i in turn]
        s["q"] = _randn((B, H, D), g, dtype)
        s["lens"] = lens
        if not page:
            s["kp"], s["vp"] = (_randn((P, Hk, D), g, dtype) for _ in range(2))
            s["k"], s["v"] = (_randn((B, c["own"], Hk, D), g, dtype) for _ in range(2))
            s["pos"] = torch.tensor([n - 1 for n in lens], dtype=torch.int32, device=DEV)
            return s
        # the prefix's whole pages are every sequence's; the page that it ends in is copied
        whole, per = P // page, -(-(P + c["own"]) // page)
        n = whole + B * (per - whole) + 3
        order = torch.randperm(n, generator=g, device=DEV)
        table = torch.empty((B, per), dtype=torch.int64, device=DEV)
        table[:, :whole] = order[:whole]
        table[:, whole:] = order[whole: n - 3].view(B, per - whole)
        s["k"], s["v"] = (_randn((n, page, Hk, D), g, dtype) for _ in range(2))
        if P % page:
            for x in (s["k"], s["v"]):
                x[table[:, whole], : P % page] = x[table[0, whole], : P % page].clone()
        s["table"] = table.to(torch.int32)
        s["pos"] = torch.tensor([P + n - 1 for n in lens], dtype=torch.int32, device=DEV)
        return s
    bring = [_bring(c)[i] for i in turn]
    rows = c["tokens"] + c["pad"]
    s["bring"] = bring
    s["q"], s["out"] = (_randn((rows, H, D), g, dtype) for _ in range(2))
    s["pos"] = torch.tensor([last for _, last in bring], dtype=torch.int32, device=DEV)
    s["offsets"] = None
    if c["ragged"]:
        off = [0]
        for n, _ in bring:
            off.append(off[-1] + n)
        s["offsets"] = torch.tensor(off, dtype=torch.int32, device=DEV)
    lead, slots = B, c["seq_len"]
    if page:
        per = c["seq_len"] // page
        lead, slots = B * per + 3, page
        order = torch.randperm(lead, generator=g, device=DEV)[: B * per]
        s["table"] = order.view(B, per).to(torch.int32)
    s["k"], s["v"] = (_randn((lead, slots, Hk, D), g, dtype) for _ in range(2))
    return s


# --------------------------------------------------------------- plain forms

def _rows(cache, table, b, p):
    """Rows of the cache in 32 bits: positions p of sequences b (index tensors)."""
    if table is None:
        return cache[b, p].float()
    n = cache.shape[1]
    return cache[table.long()[b, p // n], p % n].float()


def _weigh(score, seen):
    """Softmax over the last axis of what is seen."""
    score = score.masked_fill(~seen, -math.inf)
    e = torch.exp(score - score.amax(-1, keepdim=True))
    return e / e.sum(-1, keepdim=True)


def _plain_token(s):
    c = s["case"]
    B, H, Hk, D = c["batch"], c["heads"], c["kv_heads"], c["dim"]
    most = max(last + 1 - _first(c, last) + min(c["sinks"], _first(c, last)) for _, last in s["bring"])
    p = s["pos"].long()
    lo = (p - c["window"] + 1).clamp(min=0) if c["window"] else torch.zeros_like(p)
    first = lo.clamp(max=c["sinks"])  # sinks before the window
    i = torch.arange(most, device=DEV)
    at = torch.where(i < first[:, None], i, i + (lo - first)[:, None])
    seen = at <= p[:, None]
    at = torch.where(seen, at, 0)
    b = torch.arange(B, device=DEV)[:, None]
    K, V = (_rows(s[x], s["table"], b, at).transpose(1, 2) for x in "kv")  # [B, Hk, most, D]
    score = s["q"].float().view(B, Hk, H // Hk, D) @ K.transpose(-1, -2) / math.sqrt(D)
    return (_weigh(score, seen[:, None, None]) @ V).view(B, H, D).to(s["q"].dtype)


def _plain_ragged(s):
    c = s["case"]
    H, Hk, D, w = c["heads"], c["kv_heads"], c["dim"], c["window"]
    out, t = s["out"].clone(), 0
    for b, (n, last) in enumerate(s["bring"]):
        for t0 in range(0, n, ROWS):
            m = min(ROWS, n - t0)
            p0 = last - n + 1 + t0
            lo = _first(c, p0)
            at = torch.cat([torch.arange(min(c["sinks"], lo), device=DEV),
                            torch.arange(lo, p0 + m, device=DEV)])
            p = torch.arange(p0, p0 + m, device=DEV)[:, None]
            seen = at <= p
            if w:
                seen &= (at > p - w) | (at < c["sinks"])
            K, V = (_rows(s[x], s["table"], torch.full_like(at, b), at).transpose(0, 1) for x in "kv")
            q = s["q"][t + t0: t + t0 + m].float().view(m, Hk, H // Hk, D).permute(1, 2, 0, 3)
            for h in range(Hk):  # [G, m, keys] scores of one key/value head
                y = _weigh(q[h] @ K[h].T / math.sqrt(D), seen) @ V[h]
                out[t + t0: t + t0 + m, h * (H // Hk): (h + 1) * (H // Hk)] = y.transpose(0, 1).to(out.dtype)
        t += n
    return out


def _plain_shared(s):
    c = s["case"]
    B, H, Hk, D, P, page = (c[k] for k in ("batch", "heads", "kv_heads", "dim", "prefix", "page"))
    G = H // Hk
    b = torch.arange(B, device=DEV)[:, None]
    i = torch.arange(max(s["lens"]), device=DEV)
    own_pos = s["pos"].long() - (P if page else 0)
    seen = i <= own_pos[:, None]
    at = torch.where(seen, i, 0)
    if page:
        zero, p = torch.zeros(P, dtype=torch.long, device=DEV), torch.arange(P, device=DEV)
        K0, V0 = (_rows(s[x], s["table"], zero, p) for x in "kv")
        at = at + P
    else:
        K0, V0 = s["kp"].float(), s["vp"].float()
    K1, V1 = (_rows(s[x], s["table"], b, at).transpose(1, 2) for x in "kv")
    q = s["q"].float().view(B, Hk, G, D)
    # the prefix's scores of all sequences in one product per key/value head
    s0 = q.transpose(0, 1).reshape(Hk, B * G, D) @ K0.permute(1, 2, 0)
    s0 = s0.view(Hk, B, G, P).transpose(0, 1) / math.sqrt(D)
    s1 = (q @ K1.transpose(-1, -2) / math.sqrt(D)).masked_fill(~seen[:, None, None], -math.inf)
    top = torch.maximum(s0.amax(-1, keepdim=True), s1.amax(-1, keepdim=True))
    e0, e1 = torch.exp(s0 - top), torch.exp(s1 - top)
    y = (e0.transpose(0, 1).reshape(Hk, B * G, P) @ V0.transpose(0, 1)).view(Hk, B, G, D).transpose(0, 1)
    y = (y + e1 @ V1) / (e0.sum(-1, keepdim=True) + e1.sum(-1, keepdim=True))
    return y.reshape(B, H, D).to(s["q"].dtype)


# ----------------------------------------------------------------- the calls

def run(state):
    s, c = state, state["case"]
    if own:
        import token_decode_attention_gb300 as dattn
        if c["op"] == "shared":
            if c["page"]:
                return dattn.decode_shared_paged(s["q"], s["k"], s["v"], s["table"], s["pos"], c["prefix"])
            return dattn.decode_shared(s["q"], s["kp"], s["vp"], s["k"], s["v"], s["pos"])
        return dattn.attend(s["q"], s["k"], s["v"], s["pos"], window=c["window"], sinks=c["sinks"],
                            token_offsets=s["offsets"], block_table=s["table"],
                            out=s["out"] if c["pad"] else None)
    if c["op"] == "shared":
        return _plain_shared(s)
    return _plain_ragged(s) if c["ragged"] else _plain_token(s)


# ------------------------------------------------------ 64-bit definitions

def _exact_keys(s, b, h, upto):
    """K and V of positions 0 .. upto of sequence b, key/value head h, in 64 bits."""
    c = s["case"]
    out = []
    for x in (s["k"], s["v"]):
        if c["page"]:
            used = s["table"][b, : upto // c["page"] + 1].long()
            out.append(x[used, :, h].reshape(-1, c["dim"])[: upto + 1].double())
        else:
            out.append(x[b, : upto + 1, h].double())
    return out


def _exact_attend(c, s):
    H, Hk, w = c["heads"], c["kv_heads"], c["window"]
    out = s["out"].double()
    t = 0
    for b, (n, last) in enumerate(s["bring"]):
        for h in range(Hk if n else 0):
            K, V = _exact_keys(s, b, h, last)
            for r in range(0, n, 2048):
                p = torch.arange(last - n + 1 + r, min(last - n + 1 + r + 2048, last + 1), device=DEV)
                j = torch.arange(int(p[-1]) + 1, device=DEV)
                behind = p[:, None] - j  # how far back a key lies
                hidden = behind < 0
                if w:
                    hidden |= (behind >= w) & (j >= c["sinks"])
                for e in range(h * (H // Hk), (h + 1) * (H // Hk)):
                    x = s["q"][t + r: t + r + len(p), e].double() @ K[: len(j)].T / c["dim"] ** 0.5
                    x[hidden] = -math.inf
                    out[t + r: t + r + len(p), e] = torch.softmax(x, -1) @ V[: len(j)]
        t += n
    return out


def _exact_shared(c, s):
    B, H, Hk, D = c["batch"], c["heads"], c["kv_heads"], c["dim"]
    out = torch.empty((B, H, D), dtype=torch.float64, device=DEV)
    for h in range(Hk):
        if not c["page"]:
            K0, V0 = s["kp"][:, h].double(), s["vp"][:, h].double()
        for b in range(B):
            K, V = _exact_keys(s, b, h, int(s["lens"][b]) - 1 + (c["prefix"] if c["page"] else 0))
            if not c["page"]:
                K, V = torch.cat([K0, K]), torch.cat([V0, V])
            g = slice(h * (H // Hk), (h + 1) * (H // Hk))
            out[b, g] = torch.softmax(s["q"][b, g].double() @ K.T / D ** 0.5, -1) @ V
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_shared(case, s) if case["op"] == "shared" else _exact_attend(case, s)
