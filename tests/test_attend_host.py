"""The C entry points of attention over a 16-bit cache over stand-ins for the device and the
launches (what is refused, workspaces, which kernels a call takes), and what the binding
refuses by itself."""
from __future__ import annotations

import os
import subprocess

import pytest
import torch

import token_decode_attention_gb300 as dattn
from token_decode_attention_gb300 import build

STANDINS = r"""
#include "dattn.h"
#include "dattn_internal.h"
#include <cstdio>
#include <cstdlib>
#include <new>
#include <string>

static std::string g_message;
static int g_token = 0, g_tiles = 0, g_merge = 0, g_maps = 0;
static bool g_no_memory = false;
static dattn::AttendArgs g_a;
static dattn::TokenArgs g_w;
static dattn::TileArgs g_t;
static dattn::TileMaps g_m;

namespace dattn {
int set_last_error(int status, const char *m) { g_message = m; return status; }
int device_facts(DeviceFacts *out) {
    if (g_no_memory) throw std::bad_alloc();
    static unsigned word;
    *out = DeviceFacts{152, 232448, &word};
    return DATTN_OK;
}
cudaError_t attend_token_configure(int) { return cudaSuccess; }
cudaError_t attend_tiles_configure(int) { return cudaSuccess; }
cudaError_t attend_token_max_clusters(int, int, bool, int, int cluster, int *n) { *n = 304 / cluster; return cudaSuccess; }
int encode_head_rows(CUtensorMap *, const void *, long long, long long, int, int, int, int, int) { ++g_maps; return DATTN_OK; }
cudaError_t launch_attend_token(const AttendArgs &a, const TokenArgs &w, int, int, int, cudaStream_t) {
    g_a = a; g_w = w; ++g_token; return cudaSuccess;
}
cudaError_t launch_attend_tiles(const AttendArgs &a, const TileArgs &t, const TileMaps &m, int, int, cudaStream_t) {
    g_a = a; g_t = t; g_m = m; ++g_tiles; return cudaSuccess;
}
cudaError_t launch_attend_merge(const AttendArgs &, const TokenArgs &, const TileArgs *, int, int, cudaStream_t) { ++g_merge; return cudaSuccess; }
}
extern "C" {
cudaError_t cudaGetDevice(int *d) { *d = 0; return cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
const char *cudaGetErrorName(cudaError_t) { return ""; }
const char *cudaGetErrorString(cudaError_t) { return ""; }
}
static char *const A = reinterpret_cast<char *>(0x10000);      // inputs: 64 KB at most in these calls
static char *const O = reinterpret_cast<char *>(0x40000000);   // outputs and workspaces
static char *const W = reinterpret_cast<char *>(0x50000000);
#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s (%s)\n", __LINE__, #x, g_message.c_str()); return 1; } } while (0)

struct Call {  // a decode of two sequences of 64 positions, 4 heads on 2, 64 channels
    char *q = A, *k = A, *v = A, *out = O, *ws = W, *cp = A, *off = nullptr, *table = A, *kp = A, *vp = A;
    int dtype = DATTN_F16, B = 2, T = 2, H = 4, Hk = 2, D = 64, S = 64, window = 0, sinks = 0, page = 16, per = 4, shared = 16;
    long long qs = 256, pages = 8;
    size_t bytes = size_t(1) << 30;
    int dense() {
        return dattn_attend(q, k, v, out, dtype, B, T, (int32_t *)off, qs, H, Hk, D, S, window, sinks, (uint32_t *)cp, ws, bytes, nullptr);
    }
    int paged() {
        return dattn_attend_paged(q, k, v, out, dtype, B, T, (int32_t *)off, qs, H, Hk, D, page, per, pages, (int32_t *)table, window,
                                  sinks, (uint32_t *)cp, ws, bytes, nullptr);
    }
    int prefix() {
        return dattn_decode_shared(q, kp, vp, k, v, out, dtype, B, qs, H, Hk, D, shared, S, (uint32_t *)cp, ws, bytes, nullptr);
    }
    int pool() {
        return dattn_decode_shared_paged(q, k, v, out, dtype, B, qs, H, Hk, D, page, per, pages, (int32_t *)table, shared, (uint32_t *)cp,
                                         ws, bytes, nullptr);
    }
    size_t need() {
        size_t n = 0;
        return dattn_attend_workspace_bytes(B, T, off != nullptr, H, Hk, D, S, window, sinks, &n) == DATTN_OK ? n : ~size_t(0);
    }
    size_t need_shared(int own) {
        size_t n = 0;
        return dattn_decode_shared_workspace_bytes(B, H, Hk, D, shared, own, &n) == DATTN_OK ? n : ~size_t(0);
    }
};
"""


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    tmp = tmp_path_factory.mktemp("attend")

    def go(body: str) -> None:
        src, exe = tmp / "t.cpp", tmp / "t"
        src.write_text(STANDINS + "int main() {\n" + body + "\nreturn 0;\n}\n")
        cuda = os.path.join(os.path.dirname(os.path.dirname(build.nvcc())), "include")
        subprocess.run(["g++", "-O1", "-std=c++17", f"-I{build.CSRC}", f"-I{build.INCLUDE}", f"-I{cuda}",
                        str(src), os.path.join(build.CSRC, "attend_api.cpp"), "-o", str(exe)], check=True)
        r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
        assert r.returncode == 0, r.stdout + r.stderr
    return go


def test_each_call_takes_its_kernels(run):
    run("""
    Call c;
    CHECK(c.dense() == DATTN_OK && g_token == 1 && g_tiles == 0 && g_merge == 0 && g_maps == 0);
    CHECK(c.paged() == DATTN_OK && g_token == 2 && g_tiles == 0);
    c.off = A;
    c.T = 9;
    CHECK(c.dense() == DATTN_OK && g_tiles == 1 && g_token == 2 && g_maps == 3 && g_t.plan != nullptr);
    CHECK(g_m.box_rows == 128 && g_t.align == 1 && g_m.q_tokens == 64);
    CHECK(c.paged() == DATTN_OK && g_tiles == 2 && g_m.box_rows == 16 && g_t.align == 16);
    c.page = 3;   // no box divides it
    CHECK(c.paged() == DATTN_OK && g_tiles == 3 && g_m.box_rows == 0 && g_t.align == 1 && g_maps == 7);
    c.H = 6;      // a stack is no whole number of tokens
    c.qs = 384;
    CHECK(c.dense() == DATTN_OK && g_m.q_tokens == 0 && g_maps == 9);
    g_tiles = 3;
    Call s;
    CHECK(s.prefix() == DATTN_OK && g_tiles == 4 && g_token == 3 && g_merge == 1);
    CHECK(g_t.plan == nullptr && g_t.bound_ends == 0 && g_w.own_only == 1 && g_a.own_base == 16 && g_a.S == 80);
    CHECK(s.pool() == DATTN_OK && g_tiles == 5 && g_token == 4 && g_merge == 2);
    CHECK(g_t.bound_ends == 1 && g_a.own_base == 0 && g_a.S == 64 && g_a.shared == 16);
    Call l;   // one long sequence: chunks and their merge
    l.B = l.T = 1, l.S = 1 << 20;
    CHECK(l.dense() == DATTN_OK && g_merge == 3 && g_w.chunks > 1 && !g_w.cluster);
    CHECK((long long)g_w.chunks * g_w.chunk_tiles * 16 >= 1 << 20);
    """)


def test_refusals(run):
    run("""
    #define REFUSED(field, value, status) do { \
        Call a; a.field = value; CHECK(a.dense() == status); \
        Call p; p.field = value; CHECK(p.paged() == status); \
        Call s; s.field = value; CHECK(s.prefix() == status); \
        Call t; t.field = value; CHECK(t.pool() == status); } while (0)
    REFUSED(q, nullptr, DATTN_ERR_INVALID_ARG);
    REFUSED(k, nullptr, DATTN_ERR_INVALID_ARG);
    REFUSED(v, nullptr, DATTN_ERR_INVALID_ARG);
    REFUSED(out, nullptr, DATTN_ERR_INVALID_ARG);
    REFUSED(cp, nullptr, DATTN_ERR_INVALID_ARG);
    REFUSED(q, A + 8, DATTN_ERR_MISALIGNED);
    REFUSED(k, A + 2, DATTN_ERR_MISALIGNED);
    REFUSED(v, A + 2, DATTN_ERR_MISALIGNED);
    REFUSED(out, O + 8, DATTN_ERR_MISALIGNED);
    REFUSED(cp, A + 2, DATTN_ERR_MISALIGNED);
    REFUSED(dtype, DATTN_F32, DATTN_ERR_INVALID_ARG);
    REFUSED(dtype, 0, DATTN_ERR_INVALID_ARG);
    REFUSED(B, 0, DATTN_ERR_INVALID_ARG);
    REFUSED(H, -4, DATTN_ERR_INVALID_ARG);
    REFUSED(H, 5, DATTN_ERR_INVALID_ARG);
    REFUSED(Hk, 0, DATTN_ERR_INVALID_ARG);
    REFUSED(Hk, 3, DATTN_ERR_INVALID_ARG);
    REFUSED(D, 0, DATTN_ERR_INVALID_ARG);
    REFUSED(D, 60, DATTN_ERR_UNSUPPORTED);
    REFUSED(D, 264, DATTN_ERR_UNSUPPORTED);
    REFUSED(qs, 255, DATTN_ERR_INVALID_ARG);
    REFUSED(qs, 260, DATTN_ERR_MISALIGNED);
    REFUSED(qs, 1LL << 50, DATTN_ERR_INVALID_ARG);
    #define ALONE(call, field, value, status) do { Call a; a.field = value; CHECK(a.call() == status); } while (0)
    ALONE(dense, T, 3, DATTN_ERR_INVALID_ARG);    // not one token each
    ALONE(dense, S, 0, DATTN_ERR_INVALID_ARG);
    ALONE(dense, window, -1, DATTN_ERR_INVALID_ARG);
    ALONE(paged, sinks, -1, DATTN_ERR_INVALID_ARG);
    ALONE(dense, S, 0x7fffff00, DATTN_ERR_UNSUPPORTED);
    ALONE(paged, page, 0, DATTN_ERR_INVALID_ARG);
    ALONE(paged, per, 0, DATTN_ERR_INVALID_ARG);
    ALONE(pool, pages, 0, DATTN_ERR_INVALID_ARG);
    ALONE(paged, per, 1 << 28, DATTN_ERR_UNSUPPORTED);
    ALONE(paged, pages, 1LL << 28, DATTN_ERR_UNSUPPORTED);
    ALONE(paged, table, nullptr, DATTN_ERR_INVALID_ARG);
    ALONE(pool, table, A + 2, DATTN_ERR_MISALIGNED);
    ALONE(prefix, kp, nullptr, DATTN_ERR_INVALID_ARG);
    ALONE(prefix, vp, A + 8, DATTN_ERR_MISALIGNED);
    ALONE(prefix, shared, 0, DATTN_ERR_INVALID_ARG);
    ALONE(pool, shared, -1, DATTN_ERR_INVALID_ARG);
    ALONE(pool, shared, 65, DATTN_ERR_INVALID_ARG);
    ALONE(prefix, shared, 0x7fffff00, DATTN_ERR_UNSUPPORTED);
    Call r;
    r.off = A + 2;
    CHECK(r.dense() == DATTN_ERR_MISALIGNED);
    r.off = A, r.T = 0;
    CHECK(r.dense() == DATTN_ERR_INVALID_ARG);
    Call big;
    big.B = big.T = 1 << 20, big.H = 1 << 12, big.Hk = 1, big.qs = 1 << 18;
    CHECK(big.dense() == DATTN_ERR_UNSUPPORTED);
    CHECK(g_token + g_tiles + g_merge == 0);
    """)


def test_out_shares_nothing_with_the_inputs(run):
    # q and out 2 x 4 x 64 f16 (1024 bytes), the cache 2 x 64 x 2 x 64 (32768), the prefix 16 x 2 x 64 (4096)
    run("""
    #define AT(call, q_, k_, v_, kp_, vp_, out_) ([&] { Call c; c.q = q_, c.k = k_, c.v = v_, c.kp = kp_, c.vp = vp_, c.out = out_; return c.call(); }())
    char *const X = O + (1 << 20);
    CHECK(AT(dense, O, X, X, X, X, O) == DATTN_ERR_INVALID_ARG);
    CHECK(AT(dense, O, X, X, X, X, O + 1008) == DATTN_ERR_INVALID_ARG);
    CHECK(AT(dense, O, X, X, X, X, O + 1024) == DATTN_OK);
    CHECK(AT(dense, O + 1024, X, X, X, X, O) == DATTN_OK);
    CHECK(AT(dense, X, O, X, X, X, O + 32752) == DATTN_ERR_INVALID_ARG);
    CHECK(AT(dense, X, O, X, X, X, O + 32768) == DATTN_OK);
    CHECK(AT(dense, X, X, O, X, X, O + 16) == DATTN_ERR_INVALID_ARG);
    CHECK(AT(prefix, X, X, X, O, X, O + 4080) == DATTN_ERR_INVALID_ARG);
    CHECK(AT(prefix, X, X, X, X, O, O + 4080) == DATTN_ERR_INVALID_ARG);
    CHECK(AT(prefix, X, X, X, X, O, O + 4096) == DATTN_OK);
    CHECK(AT(paged, X, O, X, X, X, O + 32752) == DATTN_ERR_INVALID_ARG);   // a pool of 8 pages of 16
    CHECK(AT(paged, X, O, X, X, X, O + 32768) == DATTN_OK);
    """)


def test_workspaces(run):
    run("""
    for (int ragged = 0; ragged < 2; ++ragged)
        for (int B : {1, 2, 300})
            for (int S : {16, 1024, 40000})
                for (int window : {0, 5, 700}) {
                    Call c;
                    c.B = B, c.S = S, c.window = window, c.sinks = 4;
                    c.T = ragged ? 3 * B : B;
                    c.off = ragged ? A : nullptr;
                    c.out = reinterpret_cast<char *>(0x7000000000);
                    const size_t n = c.need();
                    CHECK(n != ~size_t(0));
                    c.bytes = n;
                    CHECK(c.dense() == DATTN_OK);
                    c.page = 8, c.per = S / 8, c.pages = 5;   // a pool smaller than what the tables could name
                    CHECK(c.paged() == DATTN_OK);
                    if (n == 0) { c.ws = nullptr; CHECK(c.dense() == DATTN_OK); continue; }
                    c.bytes = n - 1;
                    CHECK(c.dense() == DATTN_ERR_WORKSPACE && c.paged() == DATTN_ERR_WORKSPACE);
                    c.bytes = n, c.ws = W + 8;
                    CHECK(c.dense() == DATTN_ERR_WORKSPACE);
                    c.ws = nullptr;
                    CHECK(c.dense() == DATTN_ERR_WORKSPACE);
                }
    for (int B : {1, 2, 300})
        for (int shared : {1, 130, 9000}) {
            Call c;
            c.B = B, c.T = B, c.shared = shared;
            c.out = reinterpret_cast<char *>(0x7000000000);
            c.bytes = c.need_shared(c.S);
            CHECK(c.bytes != ~size_t(0) && c.bytes > 0 && c.prefix() == DATTN_OK);
            c.bytes -= 1;
            CHECK(c.prefix() == DATTN_ERR_WORKSPACE);
            c.per = shared / 16 + 5;
            c.bytes = c.need_shared(c.per * 16 - shared);
            CHECK(c.pool() == DATTN_OK);
            c.bytes -= 1;
            CHECK(c.pool() == DATTN_ERR_WORKSPACE);
        }
    Call whole;   // nothing but shared positions
    whole.shared = 64;
    whole.bytes = whole.need_shared(0);
    CHECK(whole.pool() == DATTN_OK);
    size_t n;
    CHECK(dattn_attend_workspace_bytes(2, 2, 0, 4, 2, 64, 64, 0, 0, nullptr) == DATTN_ERR_INVALID_ARG);
    CHECK(dattn_attend_workspace_bytes(2, 3, 0, 4, 2, 64, 64, 0, 0, &n) == DATTN_ERR_INVALID_ARG);
    CHECK(dattn_attend_workspace_bytes(2, 3, 1, 4, 2, 64, 0, 0, 0, &n) == DATTN_ERR_INVALID_ARG);
    CHECK(dattn_decode_shared_workspace_bytes(2, 4, 2, 64, 0, 64, &n) == DATTN_ERR_INVALID_ARG);
    CHECK(dattn_decode_shared_workspace_bytes(2, 4, 2, 64, 5, -1, &n) == DATTN_ERR_INVALID_ARG);
    """)


def test_a_size_holds_when_other_shapes_were_asked_for_meanwhile(run):
    """Sizes depend on a call's own shape, not on which shapes came before it."""
    run("""
    auto need = [](int S, int window) { Call c; c.B = c.T = 1, c.T = 40, c.off = A, c.S = S, c.window = window; return c.need(); };
    const size_t small = need(128, 100), large = need(1 << 20, 100);
    for (int i = 0; i < 1100; ++i) need(200 + i, 0);      // all that were kept are dropped
    CHECK(need(1 << 20, 100) == large);
    CHECK(need(128, 100) == small);
    for (int i = 0; i < 1100; ++i) need(200 + i, 0);
    CHECK(need(128, 100) == small);
    CHECK(need(1 << 20, 100) == large);
    """)


def test_a_failure_of_the_host_has_its_own_message(run):
    run("""
    Call c;
    g_message = "of an earlier call";
    g_no_memory = true;
    CHECK(c.dense() == DATTN_ERR_CUDA && c.paged() == DATTN_ERR_CUDA && c.prefix() == DATTN_ERR_CUDA && c.pool() == DATTN_ERR_CUDA);
    CHECK(c.need() == ~size_t(0) && c.need_shared(4) == ~size_t(0));
    CHECK(g_message.find("earlier") == std::string::npos && !g_message.empty());
    CHECK(g_token + g_tiles == 0);
    """)


# ------------------------------------------------------------------ the binding

def tensors(**kw):
    d = dict(q=torch.zeros(2, 4, 64, dtype=torch.float16), k=torch.zeros(2, 64, 2, 64, dtype=torch.float16),
             v=torch.zeros(2, 64, 2, 64, dtype=torch.float16), pos=torch.zeros(2, dtype=torch.int32))
    d.update(kw)
    return d["q"], d["k"], d["v"], d["pos"]


@pytest.mark.parametrize("kw,error", [
    (dict(q=torch.zeros(2, 4, 64)), TypeError), (dict(q=None), TypeError), (dict(pos=[0, 0]), TypeError),
    (dict(q=torch.zeros(4, 64, dtype=torch.float16)), ValueError),
    (dict(k=torch.zeros(2, 64, 2, 64)), (TypeError, ValueError)),
    (dict(q=torch.zeros(2, 4, 64, dtype=torch.float16, requires_grad=True)), ValueError),
])
def test_binding_names_what_is_wrong(kw, error):
    with pytest.raises(error):
        dattn.attend(*tensors(**kw))


@pytest.mark.parametrize("kw", [dict(window=2 ** 31), dict(sinks=2 ** 32 + 4), dict(window=-1), dict(sinks=-5)])
def test_binding_refuses_what_32_bits_would_change(kw):
    with pytest.raises(ValueError, match="2\\^31"):
        dattn.attend(*tensors(), **kw)
    q, k, v, pos = tensors()
    with pytest.raises(ValueError, match="2\\^31"):
        dattn.decode_shared_paged(q, k, v, torch.zeros(2, 4, dtype=torch.int32), pos, 2 ** 32 + 1)


def test_binding_refuses_host_tensors_and_missing_tables():
    with pytest.raises((ValueError, RuntimeError)):
        dattn.attend(*tensors())
    q, k, v, pos = tensors()
    with pytest.raises(TypeError):
        dattn.decode_shared_paged(q, k, v, None, pos, 16)
