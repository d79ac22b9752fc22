"""The rotary operator and the 8-bit cache on the host: what the C ABI and the
binding refuse before any CUDA call, and the division by multiplication that the
kernels use (fake pointers are never dereferenced)."""
from __future__ import annotations

import ctypes
import os
import subprocess

import pytest
import torch

import token_decode_attention_gb300 as dattn
from token_decode_attention_gb300 import _native, build

A = 0x10000
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _native.load()


def params(rd=64, trad=0, base=10000.0, scaling=0, factor=1.0, length=0.0, low=0.0, high=0.0, mag=1.0):
    return _native.RopeParams(rd, trad, base, scaling, factor, length, low, high, mag)


INVALID, UNSUPPORTED, MISALIGNED = (_native.ERR_INVALID_ARG, _native.ERR_UNSUPPORTED,
                                    _native.ERR_MISALIGNED)
NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), INVALID), (dict(out=None), INVALID), (dict(pos=None), INVALID),
    (dict(x=A + 8), MISALIGNED), (dict(out=A + 2), MISALIGNED), (dict(pos=A + 2), MISALIGNED),
    (dict(dtype=0), INVALID), (dict(dtype=4), INVALID),
    (dict(T=0), INVALID), (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(D=0), INVALID),
    (dict(D=12), UNSUPPORTED), (dict(D=264), UNSUPPORTED), (dict(T=1 << 31), UNSUPPORTED),
    (dict(xs=100), INVALID), (dict(xs=130), MISALIGNED), (dict(os=132), MISALIGNED),
    (dict(xs=1 << 41), INVALID), (dict(out=A, x=A, xs=136), INVALID),
])
def test_rope_refuses(lib, kw, status):
    a = dict(x=A, out=2 * A, dtype=1, T=4, H=2, D=64, xs=128, os=128, pos=A)
    a.update(kw)
    st = lib.dattn_rope(a["x"], a["out"], a["dtype"], a["T"], a["H"], a["D"], a["xs"], a["os"],
                        a["pos"], params(rd=8), 0, None)
    assert st == status
    assert lib.dattn_last_error()


@pytest.mark.parametrize("kw", [
    dict(rd=0), dict(rd=7), dict(rd=66), dict(rd=-2), dict(base=1.0), dict(base=INF), dict(base=NAN),
    dict(mag=0.0), dict(mag=-1.0), dict(mag=NAN), dict(mag=INF), dict(scaling=4), dict(scaling=-1),
    dict(scaling=1, factor=0.5), dict(scaling=1, factor=NAN), dict(scaling=2, factor=INF),
    dict(scaling=2, factor=2.0, rd=2),
    dict(scaling=3, factor=2.0, length=0.0, low=1, high=2), dict(scaling=3, factor=2.0, length=INF, low=1, high=2),
    dict(scaling=3, factor=2.0, length=8.0, low=2, high=2), dict(scaling=3, factor=2.0, length=8.0, low=-1, high=2),
    dict(scaling=3, factor=2.0, length=8.0, low=1, high=NAN),
])
def test_rotation_parameters_are_checked(lib, kw):
    assert lib.dattn_rope(A, 2 * A, 1, 4, 2, 64, 128, 128, A, params(**kw), 0, None) == INVALID
    assert append(lib, rope=params(**kw)) == INVALID
    assert lib.dattn_rope(A, 2 * A, 1, 4, 2, 64, 128, 128, A, None, 0, None) == INVALID


def append(lib, q=A, k=A, v=A, qo=A, K=A, V=A, ks=A, vs=A, kv=1, n=16, B=4, T=4, off=None, qs=128,
           kstr=64, vstr=64, H=2, Hk=1, D=64, S=64, rope="", cp=A):
    return lib.dattn_rope_append_q8(q, k, v, qo, K, V, ks, vs, kv, n, B, T, off, qs, kstr, vstr, H, Hk,
                                    D, S, params() if rope == "" else rope, cp, None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(qo=None), INVALID),
    (dict(K=None), INVALID), (dict(V=None), INVALID), (dict(ks=None), INVALID), (dict(vs=None), INVALID),
    (dict(cp=None), INVALID), (dict(rope=None), INVALID), (dict(K=A + 8), MISALIGNED),
    (dict(ks=A + 2), MISALIGNED), (dict(cp=A + 1), MISALIGNED), (dict(off=A + 2), MISALIGNED),
    (dict(kv=0), INVALID), (dict(kv=3), INVALID), (dict(n=0), INVALID), (dict(n=-16), INVALID),
    (dict(B=0), INVALID), (dict(T=0, off=A), INVALID), (dict(T=5), INVALID), (dict(H=0), INVALID),
    (dict(Hk=0), INVALID), (dict(H=3, Hk=2), INVALID), (dict(S=0), INVALID), (dict(D=24), UNSUPPORTED),
    (dict(D=272), UNSUPPORTED), (dict(qs=64), INVALID), (dict(kstr=63), INVALID), (dict(vstr=68), MISALIGNED),
])
def test_append_refuses(lib, kw, status):
    assert append(lib, **kw) == status
    assert lib.dattn_last_error()


def test_paged_append_refuses(lib):
    def call(ps=32, mp=4, npages=9, table=A, n=16):
        return lib.dattn_rope_append_paged_q8(A, A, A, A, A, A, A, A, 1, n, 4, 4, None, 128, 64, 64, 2,
                                              1, 64, ps, mp, npages, table, params(), A, None)
    assert call(table=None) == INVALID
    assert call(table=A + 1) == MISALIGNED
    assert call(ps=0) == call(mp=0) == call(npages=-1) == INVALID
    assert call(n=24) == INVALID
    assert call(n=0) == INVALID
    assert call(ps=1 << 20, mp=1 << 12) == UNSUPPORTED


def decode(lib, q=A, K=A, V=A, ks=A, vs=A, out=A, kv=1, n=16, B=2, H=4, Hk=2, D=64, S=64, cp=A, parts=0):
    return lib.dattn_decode_q8(q, K, V, ks, vs, out, kv, n, B, H, Hk, D, S, cp, A, 1 << 30, parts, None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INVALID), (dict(K=None), INVALID), (dict(V=None), INVALID), (dict(ks=None), INVALID),
    (dict(vs=None), INVALID), (dict(out=None), INVALID), (dict(cp=None), INVALID),
    (dict(q=A + 8), MISALIGNED), (dict(vs=A + 1), MISALIGNED), (dict(cp=A + 2), MISALIGNED),
    (dict(kv=7), INVALID), (dict(n=0), INVALID), (dict(B=-1), INVALID), (dict(H=5), INVALID),
    (dict(Hk=0), INVALID), (dict(S=0), INVALID), (dict(D=40), UNSUPPORTED), (dict(D=512), UNSUPPORTED),
    (dict(parts=-1), INVALID),
])
def test_decode_refuses(lib, kw, status):
    assert decode(lib, **kw) == status


def test_paged_decode_and_queries_refuse(lib):
    def call(ps=32, mp=4, npages=9, table=A, n=16):
        return lib.dattn_decode_paged_q8(A, A, A, A, A, A, 1, n, 2, 4, 2, 64, ps, mp, npages, table, A, A,
                                         1 << 30, 0, None)
    assert call(table=None) == INVALID
    assert call(ps=-1) == call(npages=0) == INVALID
    assert call(n=5) == INVALID
    assert call(ps=1 << 30, mp=2) == UNSUPPORTED
    size, plan = ctypes.c_size_t(0), _native.Plan()
    assert lib.dattn_decode_q8_workspace_bytes(1, 4, 2, 64, 64, 0, None) == INVALID
    assert lib.dattn_decode_q8_workspace_bytes(1, 4, 3, 64, 64, 0, ctypes.byref(size)) == INVALID
    assert lib.dattn_decode_q8_workspace_bytes(1, 4, 2, 72, 64, 0, ctypes.byref(size)) == UNSUPPORTED
    assert lib.dattn_decode_q8_plan(1, 4, 2, 64, 64, 0, None) == INVALID
    assert lib.dattn_decode_q8_plan(1, 4, 2, 64, 0, 0, ctypes.byref(plan)) == INVALID
    assert lib.dattn_decode_q8_plan(1, 4, 2, 64, 64, -2, ctypes.byref(plan)) == INVALID


def test_binding_refuses_without_a_device():
    h = torch.zeros((2, 4, 64), dtype=torch.float16)
    kc = torch.zeros((2, 32, 2, 64), dtype=torch.int8)
    ks = torch.zeros((2, 2, 2))
    cp = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        dattn.rope(h, cp)
    with pytest.raises(TypeError, match="float8"):
        dattn.dattn_decode_q8(h, kc.float(), kc, ks, ks, h, cp, 16)
    with pytest.raises(ValueError, match="sequences"):
        dattn.dattn_decode_q8(h, kc[:1], kc, ks, ks, h, cp, 16)
    with pytest.raises(ValueError, match="CUDA"):
        dattn.dattn_decode_q8(h, kc, kc, ks, ks, h, cp, 16)


def test_rope_scaling_is_checked_and_immutable():
    with pytest.raises(ValueError, match="kind"):
        dattn.RopeScaling("other", 2.0)
    s = dattn.RopeScaling("linear", 2)
    with pytest.raises(AttributeError):
        s.factor = 3.0
    assert s == dattn.RopeScaling("linear", 2.0) and hash(s) == hash(dattn.RopeScaling("linear", 2.0))
    assert s != dattn.RopeScaling("base", 2.0)


def test_division_by_multiplication(tmp_path):
    src = tmp_path / "div.cpp"
    src.write_text("""
#include "dattn_internal.h"
#include <cstdio>
static long long fast(long long n, dattn::FastDiv d) { return (long long)(((unsigned long long)n * d.mul) >> d.shift); }
int main() {
    const long long top = 0x7fffffffLL;
    const int ds[] = {1, 2, 3, 5, 7, 10, 16, 24, 31, 33, 100, 127, 128, 641, 1000, 4097, 65535, 65537,
                      (1 << 20) - 1, 123456789, (1 << 30) - 1, 1 << 30, (1 << 30) + 1, 0x7ffffffe, 0x7fffffff};
    for (int d : ds) {
        const dattn::FastDiv f = dattn::fast_div_of(d);
        for (long long q = 0; q <= top / d; q += 1 + top / d / 5000)
            for (long long n : {q * d, q * d + d - 1, q * d + d / 2})
                if (n <= top && fast(n, f) != n / d) return std::printf("%lld / %d\\n", n, d), 1;
        for (long long n = top; n > top - 1000 && n >= 0; --n)
            if (fast(n, f) != n / d) return std::printf("%lld / %d\\n", n, d), 1;
    }
    for (int d = 1; d < 3000; ++d)
        for (long long n = 0; n < 5000; ++n)
            if (fast(n, dattn::fast_div_of(d)) != n / d) return std::printf("%lld / %d\\n", n, d), 1;
    return 0;
}
""")
    exe = tmp_path / "div"
    cuda = os.path.join(os.path.dirname(os.path.dirname(build.nvcc())), "include")
    subprocess.run(["g++", "-O2", "-std=c++17", f"-I{build.CSRC}", f"-I{build.INCLUDE}", f"-I{cuda}",
                    str(src), "-o", str(exe)], check=True)
    subprocess.run([str(exe)], check=True)


@pytest.mark.parametrize("x,xs,out,os,T,bad", [
    (A, 128, A + 16, 128, 4, True),          # shifted by half a row
    (A, 128, A + 256, 128, 4, True),         # by a token
    (A + 256, 128, A, 128, 4, True),
    (A, 256, A + 256, 256, 4, False),        # neighbouring slices of one buffer
    (A + 256, 256, A, 256, 4, False),
    (A, 256, A + 240, 256, 4, True),         # that touch
    (A, 256, A + 272, 256, 4, True),         # the second reaches into the first's next token
    (A, 136, A, 128, 4, True),               # the same start, other strides
    (A, 136, A, 128, 1, False),              # of one token
    (A, 128, A + 1024, 128, 4, False),       # one behind the other
    (A, 128, A + 1008, 128, 4, True),
    (A, 1 << 40, A + 16, 1 << 40, 1 << 30, True),
])
def test_rope_refuses_tensors_that_overlap(lib, x, xs, out, os, T, bad):
    # rows of 2 x 64 f16; what is let through fails later, without a device
    st = lib.dattn_rope(x, out, 1, T, 2, 64, xs, os, A, params(rd=8), 0, None)
    assert (st == INVALID) == bad
    if bad:
        assert b"overlap" in lib.dattn_last_error() or b"too large" in lib.dattn_last_error()


def test_append_refuses_q_out_inside_q_new(lib):
    assert append(lib, q=A, qo=A + 16) == INVALID
    assert append(lib, q=A, qo=A, qs=256) == INVALID      # a projection's slice, not dense
    assert append(lib, q=A, qo=A + 256, qs=256) == INVALID
    assert append(lib, q=A, qo=A) != INVALID
    assert append(lib, q=A, qo=A + 4 * 256) != INVALID


def test_rope_scaling_can_be_copied_and_pickled():
    # as a part of a model's configuration it is
    import copy
    import pickle
    s = dattn.RopeScaling("by_parts", 8.0, original_len=8192, low_turns=1, high_turns=32, magnitude=1.2)
    for t in (copy.copy(s), copy.deepcopy({"a": [s]})["a"][0], pickle.loads(pickle.dumps(s))):
        assert t == s and hash(t) == hash(s) and repr(t) == repr(s)
        with pytest.raises(AttributeError):
            t.factor = 3.0


def test_workspace_sizes_are_kept_for_a_bounded_number_of_shapes(monkeypatch):
    class Lib:
        asked = 0

        def dattn_decode_q8_workspace_bytes(self, b, h, hk, d, s, parts, out):
            self.asked += 1
            out._obj.value = 16 * s
            return 0
    lib = Lib()
    monkeypatch.setattr(_native, "load", lambda: lib)
    monkeypatch.setattr(_native, "_Q8_WORKSPACE", {})
    for s in range(1, 20001):
        assert dattn.dattn_decode_q8_workspace_bytes(1, 8, 8, 64, s) == 16 * s
    assert len(_native._Q8_WORKSPACE) < 2000
    lib.asked = 0
    assert dattn.dattn_decode_q8_workspace_bytes(1, 8, 8, 64, 20000) == 16 * 20000 and lib.asked == 0
    assert dattn.dattn_decode_q8_workspace_bytes(1, 8, 8, 64, 1) == 16 and lib.asked == 1
