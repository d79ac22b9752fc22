"""The 8-bit cache as a decoder uses it: a prompt appended in chunks, then decode
steps, each an append and a decode on the cache it left."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import token_decode_attention_gb300 as dattn
from token_decode_attention_gb300 import _native

from . import _q8
from ._util import cur_pos_tensor

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv,page", [("e4m3", 32), ("int8", 32), ("e4m3", 0)])
def test_prompt_then_decode_steps(kv, page):
    from token_decode_attention_gb300 import build
    build.build()
    B, H, Hk, D, S, n = 3, 8, 2, 128, 256, 16
    g = torch.Generator(device="cuda").manual_seed(11)
    sc = dattn.RopeScaling("by_parts", 4.0, original_len=64, low_turns=1, high_turns=8,
                           magnitude=1.14)
    rope = dict(rope_base=500000.0, scaling=sc)
    lead, rows, table, tn = B, S, None, None
    if page:
        lead, rows = B * S // page, page
        tn = np.random.default_rng(0).permutation(lead).reshape(B, -1).astype(np.int32)
        table = torch.from_numpy(tn).cuda()
    kc, vc = (torch.zeros((lead, rows, Hk, D), dtype=_q8.TORCH[kv], device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((lead, rows // n, Hk), device="cuda") for _ in range(2))
    new = lambda t, h: torch.randn((t, h, D), generator=g, device="cuda").half()  # noqa: E731

    assert dattn.dattn_device_error(clear=True) == _native.OK
    K = [np.zeros((0, Hk, D)) for _ in range(B)]  # what the cache stands for, unrounded
    V = [np.zeros((0, Hk, D)) for _ in range(B)]
    length = [0, 0, 0]

    def append(counts):
        off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        q, k, v = new(int(off[-1]), H), new(int(off[-1]), Hk), new(int(off[-1]), Hk)
        for b, c in enumerate(counts):
            p = np.arange(length[b], length[b] + c)
            kr = _q8.rotate(_q8.f64(k)[off[b]: off[b + 1]], p, 0, 500000.0, False, sc)
            K[b], V[b] = np.concatenate([K[b], kr]), np.concatenate([V[b], _q8.f64(v)[off[b]: off[b + 1]]])
            length[b] += c
        cp = cur_pos_tensor([x - 1 for x in length])
        one = all(c == 1 for c in counts)
        q = dattn.rope_append_q8(q, k, v, kc, vc, ks, vs, cp, n,
                                 token_offsets=None if one else torch.from_numpy(off).cuda(),
                                 block_table=table, **rope)
        return q, cp

    append([100, 7, 33])
    append([30, 0, 1])
    for step in range(4):
        q, cp = append([1, 1, 1])
        if page:
            out = dattn.decode_paged_q8(q, kc, vc, ks, vs, table, cp, n)
        else:
            out = dattn.decode_q8(q, kc, vc, ks, vs, cp, n)
        kq, vq = _q8.values(kc), _q8.values(vc)
        ksn, vsn, cpn = ks.cpu().numpy(), vs.cpu().numpy(), [x - 1 for x in length]
        ref, size, dot, top = _q8.decode(q.cpu().numpy(), kq, vq, ksn, vsn, cpn, n, tn, page)
        _q8.check(_q8.f64(out), ref, _q8.decode_bound(ref, size, dot, top, max(length), D,
                                                      np.maximum(vsn, 2.0 ** -32)), f"step {step}")
        # the cache stands for the tokens, to the 8-bit type's rounding of the
        # block's largest value (int8: half a step of scale <= amax / 63.5, and as
        # much again for each doubling of the scale, at most amax / 63.5 in all)
        for b in range(B):
            p = np.arange(length[b])
            ld = np.full(length[b], b) if tn is None else tn[b, p // page]
            rw = p if tn is None else p % page
            for x, c, s in ((K[b], kq, ksn), (V[b], vq, vsn)):
                got = c[ld, rw] * s[ld, rw // n][..., None]
                blk = np.zeros((-(-length[b] // n), Hk))
                np.maximum.at(blk, p // n, np.abs(x).max(axis=2))
                amax = blk[p // n][..., None]
                lim = amax / 63.5 if kv == "int8" else np.abs(x) * 2.0 ** -4 + amax * 2.0 ** -16
                assert (np.abs(got - x) <= lim * 1.0001).all(), f"step {step}, sequence {b}"
    assert dattn.dattn_device_error(clear=True) == _native.OK


def test_steps_back_to_back_without_host_sync():
    B, H, Hk, D, S, n, steps = 2, 8, 4, 64, 64, 8, 12
    g = torch.Generator(device="cuda").manual_seed(12)
    kc, vc = (torch.zeros((B, S, Hk, D), dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((B, S // n, Hk), device="cuda") for _ in range(2))
    toks = [[torch.randn((B, h, D), generator=g, device="cuda").half() for h in (H, Hk, Hk)]
            for _ in range(steps)]
    cps = [cur_pos_tensor([t, t]) for t in range(steps)]
    torch.cuda.synchronize()

    def go(sync):
        for t in (kc, vc, ks, vs):
            t.view(torch.uint8).zero_()
        outs = []
        for (q, k, v), cp in zip(toks, cps):
            qr = dattn.rope_append_q8(q, k, v, kc, vc, ks, vs, cp, n)
            outs.append(dattn.decode_q8(qr, kc, vc, ks, vs, cp, n))
            if sync:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return outs

    for a, b in zip(go(True), go(False)):
        assert torch.equal(a, b)


def test_inputs_in_pinned_memory_without_an_output():
    # the small inputs of a step may lie in pinned host memory; fresh results are on the device
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn((2, h, 64), generator=g).half().pin_memory() for h in (4, 2, 2))
    cp = torch.tensor([5, 9], dtype=torch.int32).pin_memory()
    dev = [t.cuda() for t in (q, k, v, cp)]
    kc, vc = (torch.zeros((2, 32, 2, 64), dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((2, 2, 2), device="cuda") for _ in range(2))
    caches = [t.clone() for t in (kc, vc, ks, vs)]
    want = dattn.rope_append_q8(*dev[:3], *caches, dev[3], 16)
    got = dattn.rope_append_q8(q, k, v, kc, vc, ks, vs, cp, 16)
    assert got.is_cuda and torch.equal(got, want)
    assert all(torch.equal(a, b) for a, b in zip((kc, vc, ks, vs), caches))
    assert torch.equal(dattn.decode_q8(q, kc, vc, ks, vs, cp, 16), dattn.decode_q8(dev[0], kc, vc, ks, vs, dev[3], 16))
    y = dattn.rope(q, cp)
    assert y.is_cuda and torch.equal(y, dattn.rope(dev[0], dev[3]))
    s = torch.cuda.Stream()
    y = dattn.rope(q, cp, stream=s)
    s.synchronize()
    assert torch.equal(y, dattn.rope(dev[0], dev[3]))
