"""Rotary positions of many tokens against a plain form in 64 bits."""
from __future__ import annotations

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import token_decode_attention_gb300 as dattn
from token_decode_attention_gb300 import _native

from . import _q8

pytestmark = pytest.mark.gpu

# (eps, smallest subnormal) of the output type
STEP = {torch.float16: (2.0 ** -10, 2.0 ** -24), torch.bfloat16: (2.0 ** -7, 2.0 ** -133),
        torch.float32: (2.0 ** -23, 2.0 ** -149)}
SCALINGS = {
    "none": None,
    "linear": dattn.RopeScaling("linear", 4.0),
    "base": dattn.RopeScaling("base", 8.0),
    "by_parts": dattn.RopeScaling("by_parts", 8.0, original_len=4096, low_turns=1, high_turns=32,
                                  magnitude=1.2079441541679836),
}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from token_decode_attention_gb300 import build
    build.build()
    dattn.load()
    yield
    assert dattn.dattn_device_error(clear=True) == _native.OK


def positions(p) -> torch.Tensor:
    return torch.from_numpy(np.asarray(p, np.int64).astype(np.uint32).view(np.int32)).cuda()


def check(got, x, p, rd, base, trad, scaling, gradient, what=""):
    rd = rd or x.shape[-1]
    xn = _q8.f64(x)
    ref = _q8.rotate(xn, p, rd, base, trad, scaling, gradient)
    mag = 1.0 if scaling is None else scaling.magnitude
    bound = _q8.ROTATION * _q8.pair_size(xn, rd, trad, mag)
    eps, tiny = STEP[x.dtype]
    bound = bound + (np.arange(x.shape[-1]) < rd) * _q8.half_step(np.abs(ref) + bound, eps, tiny)
    _q8.check(_q8.f64(got), ref, bound, what)


CASES = [
    # tokens, H, D, rope_dims, base
    (1, 32, 128, 0, 10000.0),
    (1, 1, 8, 0, 10000.0),
    (3, 5, 64, 20, 10000.0),      # pairs read one by one
    (7, 3, 24, 16, 10000.0),      # a head of 24 channels: no whole vectors past the rotated ones
    (130, 40, 128, 64, 500000.0),
    (33, 2, 256, 0, 1e6),
    (1000, 8, 80, 32, 10000.0),
    (65, 17, 96, 96, 10000.0),
    (2, 600, 64, 48, 10000.0),    # more heads than a CTA takes
    (4097, 1, 128, 2, 10000.0),
]


@pytest.mark.parametrize("dtype", list(STEP), ids=["f16", "bf16", "f32"])
@pytest.mark.parametrize("trad", [False, True], ids=["half", "adjacent"])
@pytest.mark.parametrize("n,H,D,rd,base", CASES, ids=[f"T{c[0]}H{c[1]}D{c[2]}r{c[3]}" for c in CASES])
def test_matches_the_plain_form(n, H, D, rd, base, trad, dtype):
    g = torch.Generator(device="cuda").manual_seed(n + H + D)
    x = (2 * torch.randn((n, H, D), generator=g, device="cuda")).to(dtype)
    p = np.random.default_rng(n).integers(0, 200000, n)
    check(dattn.rope(x, positions(p), rd, base, trad), x, p, rd, base, trad, None, False)


@pytest.mark.parametrize("gradient", [False, True])
@pytest.mark.parametrize("kind", list(SCALINGS))
def test_scaled_frequencies(kind, gradient):
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn((50, 4, 128), generator=g, device="cuda")
    p = np.arange(50) * 1777
    for trad in (False, True):
        check(dattn.rope(x, positions(p), 0, 10000.0, trad, SCALINGS[kind], gradient), x, p, 0,
              10000.0, trad, SCALINGS[kind], gradient, f"{kind} {trad}")


def test_far_positions_keep_their_digits():
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((6, 3, 64), generator=g, device="cuda")
    p = [0, 1, 2 ** 24 + 1, 2 ** 31 - 1, 2 ** 31, 2 ** 32 - 1]
    # theta_i itself is rounded to 64 bits: p theta_i is off by up to 2^32 2^-53 rad,
    # which the plain form shares (it uses the same theta)
    check(dattn.rope(x, positions(p)), x, p, 0, 10000.0, False, None, False)


def test_gradient_is_the_transpose():
    g = torch.Generator(device="cuda").manual_seed(6)
    x, y = (torch.randn((40, 3, 64), generator=g, device="cuda") for _ in range(2))
    p = positions(np.arange(40) * 911)
    s = SCALINGS["by_parts"]
    for trad in (False, True):
        fx = dattn.rope(x, p, 48, 1e4, trad, s)
        gy = dattn.rope(y, p, 48, 1e4, trad, s, gradient=True)
        a, b = (fx.double() * y.double()).sum((1, 2)), (x.double() * gy.double()).sum((1, 2))
        # per element at most ROTATION (|u| + |w|) of error on either side, 192 of them
        size = (x.double().abs().sum((1, 2)) * y.double().abs().amax((1, 2)) * 2 * s.magnitude)
        assert ((a - b).abs() <= 4 * _q8.ROTATION * size).all()


def test_gradient_agrees_with_differences():
    g = torch.Generator(device="cuda").manual_seed(7)
    x, y, d = (torch.randn((5, 2, 32), generator=g, device="cuda") for _ in range(3))
    p = positions([3, 70, 1000, 9, 0])
    s = SCALINGS["by_parts"]
    f = lambda t: (dattn.rope(t, p, 24, 1e4, False, s).double() * y.double()).sum()  # noqa: E731
    grad = dattn.rope(y, p, 24, 1e4, False, s, gradient=True)
    # the map is linear: a difference over a step of 1 has no truncation error
    num, ana = float(f(x + d) - f(x - d)) / 2, float((grad.double() * d.double()).sum())
    bound = 8 * 2.0 ** -23 * float((y.double().abs() * (x.double().abs() + d.double().abs())).sum()) * 4
    assert abs(num - ana) <= bound


def test_in_place_and_slices_of_a_projection():
    g = torch.Generator(device="cuda").manual_seed(8)
    H, Hk, D, n = 8, 2, 128, 77
    qkv = torch.randn((n, (H + 2 * Hk) * D), generator=g, device="cuda").half()
    keep = qkv.clone()
    q = qkv[:, : H * D].view(n, H, D)
    k = qkv[:, H * D: (H + Hk) * D].view(n, Hk, D)
    p = np.arange(n) + 5
    got_k = dattn.rope(k, positions(p))
    check(got_k, k, p, 0, 1e4, False, None, False, "k")
    x = q.clone()
    dattn.rope(q, positions(p), out=q)
    check(q, x, p, 0, 1e4, False, None, False, "q in place")
    assert torch.equal(qkv[:, H * D:], keep[:, H * D:])


def test_special_values_stay_in_their_pair():
    x = torch.ones((2, 1, 32), device="cuda")
    x[0, 0, 3] = float("nan")
    x[1, 0, 20] = float("inf")
    y = dattn.rope(x, positions([5, 0]), 16)
    bad = ~torch.isfinite(y)
    want = torch.zeros_like(bad)
    want[0, 0, [3, 11]] = True
    want[1, 0, 20] = True  # passes through
    assert torch.equal(bad, want)


def test_agrees_with_the_append_of_one_token():
    # the rotation of dattn_rope_append_f16, up to one rounding of f16
    g = torch.Generator(device="cuda").manual_seed(9)
    B, H, D = 4, 8, 128
    q = torch.randn((B, H, D), generator=g, device="cuda").half()
    cache = torch.zeros((B, 600, H, D), dtype=torch.float16, device="cuda")
    p = [0, 599, 17, 300]
    a = dattn.rope_append(q, q, q, cache, cache.clone(), positions(p))
    b = dattn.rope(q, positions(p))
    step = _q8.half_step(_q8.f64(b), 2.0 ** -10, 2.0 ** -24) * 2
    _q8.check(_q8.f64(a), _q8.f64(b), step + 1e-6, "one token")


def test_graph_replay_and_streams():
    g = torch.Generator(device="cuda").manual_seed(10)
    x = torch.randn((100, 4, 64), generator=g, device="cuda").half()
    p = np.arange(100)
    tp = positions(p)
    s = torch.cuda.Stream()
    out = torch.empty_like(x)
    torch.cuda.synchronize()
    dattn.dattn_batch_begin(s)
    dattn.rope(x, tp, out=out, stream=s)
    batch = dattn.dattn_batch_end(s)
    for k in (3, 40):
        x.normal_(generator=g)
        tp.copy_(positions(p + k))
        torch.cuda.synchronize()
        batch.launch(s)
        s.synchronize()
        check(out, x, p + k, 0, 1e4, False, None, False)
    batch.close()


def test_refusals():
    x = torch.zeros((4, 2, 64), device="cuda")
    p = positions([0, 1, 2, 3])
    with pytest.raises(TypeError, match="float16"):
        dattn.rope(x.double(), p)
    with pytest.raises(ValueError, match="positions"):
        dattn.rope(x, p[:3])
    with pytest.raises(TypeError, match="positions"):
        dattn.rope(x, p.long())
    with pytest.raises(ValueError, match="contiguous"):
        dattn.rope(x.transpose(1, 2), p)
    with pytest.raises(ValueError, match="out"):
        dattn.rope(x, p, out=x[:, :1])
    with pytest.raises(_native.DattnError, match="16-byte"):
        dattn.rope(torch.zeros(4 * 130 + 8, device="cuda")[: 4 * 130].view(4, 130)[:, :128].view(4, 2, 64), p)
    with pytest.raises(_native.DattnError, match="rope_dims"):
        dattn.rope(x, p, 66)
    with pytest.raises(_native.DattnError, match="INVALID_ARG"):
        dattn.rope(x[:0], p[:0])
    with pytest.raises(TypeError, match="RopeScaling"):
        dattn.rope(x, p, scaling="linear")


@pytest.mark.parametrize("dtype", list(STEP), ids=["f16", "bf16", "f32"])
@pytest.mark.parametrize("n,H,D,rd,trad", [
    (20011, 4, 64, 0, False),      # several tiles for each CTA, four heads at a time
    (9001, 6, 32, 32, True),       # two at a time
    (7003, 7, 48, 16, False),      # one
    (5001, 4, 80, 40, True),       # pairs one by one
    (5001, 4, 80, 20, False),
    (3001, 6, 40, 12, False),
    (501, 130, 128, 0, False),     # more heads than a tile
])
def test_many_tiles_in_place_of_a_slice(n, H, D, rd, trad, dtype):
    g = torch.Generator(device="cuda").manual_seed(n + H)
    whole = torch.randn((n, H + 3, D), generator=g, device="cuda").to(dtype)
    keep = whole.clone()
    x = whole[:, 1: H + 1]
    p = torch.arange(n, dtype=torch.int32, device="cuda") * 7
    kw = dict(rope_dims=rd, traditional=trad)
    apart = dattn.rope(x, p, **kw)
    same = dattn.rope(x, p, out=x, **kw)
    assert same.data_ptr() == x.data_ptr() and torch.equal(same, apart)
    assert torch.equal(whole[:, :1], keep[:, :1]) and torch.equal(whole[:, H + 1:], keep[:, H + 1:])
    rows = np.unique(np.r_[0:70, n // 2: n // 2 + 70, n - 70: n])
    check(apart[rows], keep[:, 1: H + 1][rows], rows * 7, rd, 10000.0, trad, None, False)


def test_offsets_pass_32_bits():
    # 2^31 elements and more: the last tokens lie behind a 32-bit element count
    n, H, D = 2 ** 21 + 37, 8, 128
    x = torch.zeros((n, H, D), dtype=torch.float16, device="cuda")
    tail = torch.randn((37, H, D), device="cuda").half()
    x[-37:] = tail
    p = torch.full((n,), 5, dtype=torch.int32, device="cuda")
    p[-37:] = torch.arange(37, device="cuda", dtype=torch.int32) + 1000
    y = dattn.rope(x, p, out=x)
    assert torch.count_nonzero(y[:-37]) == 0
    check(y[-37:], tail, np.arange(37) + 1000, 0, 1e4, False, None, False)


def test_a_recorded_call_needs_its_output():
    x = torch.zeros((2, 1, 64), dtype=torch.float16, device="cuda")
    p = positions([0, 1])
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    dattn.dattn_batch_begin(s)
    try:
        with pytest.raises(ValueError, match="out"):
            dattn.rope(x, p, stream=s)
        dattn.rope(x, p, out=x, stream=s)
    finally:
        dattn.dattn_batch_end(s).close()


def test_threads_launch_at_the_same_time():
    # shapes that ask for different amounts of shared memory of the same kernels
    import threading
    cases, bad = [], []
    for i, (n, H, D, rd) in enumerate([(3000, 8, 128, 0), (3000, 8, 80, 40), (5000, 4, 80, 40),
                                       (2000, 16, 128, 128)]):
        g = torch.Generator(device="cuda").manual_seed(i)
        x = torch.randn((n, H, D), generator=g, device="cuda")
        p = torch.arange(n, dtype=torch.int32, device="cuda")
        cases.append((x, p, rd, dattn.rope(x, p, rd)))
    torch.cuda.synchronize()

    def work(x, p, rd, want):
        s = torch.cuda.Stream()
        for _ in range(50):
            try:
                got = dattn.rope(x, p, rd, stream=s)
                s.synchronize()
                if not torch.equal(got, want):
                    bad.append("differs")
            except Exception as e:  # noqa: BLE001
                bad.append(repr(e))
    threads = [threading.Thread(target=work, args=c) for c in cases]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, bad[:3]


@pytest.mark.parametrize("dtype", list(STEP), ids=["f16", "bf16", "f32"])
@pytest.mark.parametrize("gradient", [False, True])
def test_torch_finds_the_gradient(dtype, gradient):
    g = torch.Generator(device="cuda").manual_seed(11)
    x = torch.randn((9, 3, 64), generator=g, device="cuda").to(dtype).requires_grad_()
    w = torch.randn((9, 3, 64), generator=g, device="cuda").to(dtype)
    p = positions(np.arange(9) * 1000)
    s = SCALINGS["by_parts"]
    kw = dict(rope_dims=32, traditional=True, scaling=s)
    y = dattn.rope(x, p, gradient=gradient, **kw)
    with torch.no_grad():
        assert torch.equal(y, dattn.rope(x, p, gradient=gradient, **kw))
    (y * w).sum().backward()
    # of y * w the gradient is w itself
    assert torch.equal(x.grad, dattn.rope(w, p, gradient=not gradient, **kw))
    x.grad = None
    dattn.rope(x, p, gradient=gradient, **kw).sum().backward()      # ones of stride 0
    assert torch.equal(x.grad, dattn.rope(torch.ones_like(w), p, gradient=not gradient, **kw))


def test_second_derivatives_and_slices():
    g = torch.Generator(device="cuda").manual_seed(12)
    qkv = torch.randn((6, 5 * 32), generator=g, device="cuda", requires_grad=True)
    p = positions(np.arange(6))
    y = dattn.rope(qkv[:, 32: 96].view(6, 2, 32), p)
    d, = torch.autograd.grad((y ** 3).sum(), qkv, create_graph=True)
    assert torch.count_nonzero(d[:, :32]) == 0 and torch.count_nonzero(d[:, 96:]) == 0
    v = torch.randn((6, 2, 32), generator=g, device="cuda")
    hv, = torch.autograd.grad((d[:, 32: 96].view(6, 2, 32) * v).sum(), qkv)
    # R^T (6 y . (R v))
    want = dattn.rope(6 * y.detach() * dattn.rope(v, p), p, gradient=True)
    # products and rotations in fp32: a few roundings of terms of |6 y R v|
    size = float((6 * y.detach() * dattn.rope(v, p)).abs().max())
    assert float((hv[:, 32: 96].view(6, 2, 32) - want).abs().max()) <= 16 * 2.0 ** -24 * 2 * size


def test_out_and_stream_are_refused_for_a_gradient():
    x = torch.zeros((2, 1, 64), device="cuda", requires_grad=True)
    p = positions([0, 1])
    with pytest.raises(ValueError, match="gradient"):
        dattn.rope(x, p, out=torch.empty_like(x))
    with pytest.raises(ValueError, match="gradient"):
        dattn.rope(x, p, stream=torch.cuda.Stream())
    with pytest.raises(TypeError, match="float16"):
        dattn.rope(x.double(), p)
    with torch.no_grad():
        assert not dattn.rope(x, p, out=torch.empty_like(x)).requires_grad


def test_a_captured_step_takes_its_gradient_by_hand():
    x = torch.randn((5, 2, 64), device="cuda").requires_grad_()
    w = torch.randn((5, 2, 64), device="cuda")
    p = positions(range(5))
    y = dattn.rope(x, p)   # an eager graph of the same leaf is alive
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(ValueError, match="captured"):
            dattn.rope(x, p)
        with torch.no_grad():
            out = dattn.rope(x, p)
            grad = dattn.rope(w, p, gradient=True)
    out.zero_()
    grad.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, y)
    y.backward(w)
    assert torch.equal(grad, x.grad)


def test_one_head_with_a_part_rotated_launches_in_a_fresh_process():
    # rings and tables of 46 to 48 KB in all, each launched before anything larger could have
    # raised its kernel's limit on shared memory
    code = """
import torch, token_decode_attention_gb300 as dattn
p = torch.arange(4096, dtype=torch.int32, device="cuda")
for dtype in (torch.float16, torch.bfloat16):
    for d, rd in ((64, 48), (112, 80), (128, 96), (144, 96), (160, 112), (192, 128), (208, 144),
                  (224, 144), (240, 160), (256, 192)):
        x = torch.ones((4096, 1, d), dtype=dtype, device="cuda")
        y = dattn.rope(x, p, rd)
        assert torch.equal(y[0], x[0]) and torch.equal(y[:, :, rd:], x[:, :, rd:]), (d, rd)
print("launched")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and "launched" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("dtype", list(STEP), ids=["f16", "bf16", "f32"])
def test_forward_mode_rotates_the_tangent(dtype):
    g = torch.Generator(device="cuda").manual_seed(13)
    x, t = (torch.randn((9, 3, 64), generator=g, device="cuda").to(dtype) for _ in range(2))
    p = positions(np.arange(9) * 1000)
    kw = dict(rope_dims=32, traditional=True, scaling=SCALINGS["by_parts"])
    fwad = torch.autograd.forward_ad
    with fwad.dual_level():
        for tangent in (t, t[:1].expand(9, 3, 64)):
            y = fwad.unpack_dual(dattn.rope(fwad.make_dual(x, tangent), p, **kw))
            assert torch.equal(y.primal, dattn.rope(x, p, **kw))
            assert torch.equal(y.tangent, dattn.rope(tangent.contiguous(), p, **kw))
