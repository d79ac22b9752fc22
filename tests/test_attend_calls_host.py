"""More of the C entry points of attention over a 16-bit cache over stand-ins for the device
and the launches: where the parts of a workspace lie, what overlaps, and refusals of the binding."""
from __future__ import annotations

import pytest
import torch

import token_decode_attention_gb300 as dattn

from .test_attend_host import run, tensors  # noqa: F401  (`run` is the fixture)


def test_states_lie_on_32_bytes_whatever_the_workspace_starts_on(run):  # noqa: F811
    """The kernels store states of many tokens 32 bytes at a time; a workspace need lie on 16."""
    run("""
    auto aligned = [](const void *p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; };
    for (int ofs : {0, 16, 32, 48, 112}) {
        for (int D : {8, 64, 72, 128, 136, 256}) {
            Call c;   // a ragged batch
            c.D = D, c.qs = 4 * D, c.T = 9, c.off = A, c.ws = W + ofs;
            c.bytes = c.need();
            CHECK(c.dense() == DATTN_OK && aligned(g_t.acc) && aligned(g_t.ml));
            const char *const end = reinterpret_cast<const char *>(g_t.ml + 2 * (size_t)g_t.ctas * dattn::tile_rows(D <= 64 ? 64 : D <= 128 ? 128 : 256));
            CHECK(reinterpret_cast<const char *>(g_t.plan) >= c.ws && end <= c.ws + c.bytes);
            c.page = 16, c.per = 4;
            CHECK(c.paged() == DATTN_OK && aligned(g_t.acc));
            Call s;   // a shared prefix: the states of whole items too, and of the sequences' own positions
            s.D = D, s.qs = 4 * D, s.ws = W + ofs;
            s.bytes = s.need_shared(s.S);
            CHECK(s.prefix() == DATTN_OK && aligned(g_t.acc) && aligned(g_t.whole_acc) && aligned(g_w.ws_acc));
            CHECK(reinterpret_cast<const char *>(g_w.ws_ml + (size_t)s.B * s.H * g_w.chunks) <= s.ws + s.bytes);
            CHECK(reinterpret_cast<const char *>(g_t.whole_acc) >= s.ws);
            s.bytes = s.need_shared(48);
            CHECK(s.pool() == DATTN_OK && aligned(g_t.acc) && aligned(g_t.whole_acc));
        }
    }
    """)



def test_a_call_writes_over_nothing_that_it_reads(run):  # noqa: F811
    """out and workspace share no byte with the inputs that a kernel reads, nor with each other."""
    run("""
    #define ON(call, status, ...) do { Call c; c.off = OFF; c.T = OFF ? 9 : 2; __VA_ARGS__; CHECK(c.call() == status); } while (0)
    char *const X = O + (1 << 24);
    for (char *OFF : {(char *)nullptr, A}) {
        // q and out 1024 bytes (4608 of 9 tokens), positions 8, offsets 12, a table 32
        ON(dense, DATTN_OK, c.cp = O - 8);
        ON(dense, DATTN_ERR_INVALID_ARG, c.cp = O - 4);
        ON(dense, DATTN_ERR_INVALID_ARG, c.cp = O + 512);
        ON(paged, DATTN_ERR_INVALID_ARG, c.cp = O);
        ON(paged, DATTN_ERR_INVALID_ARG, c.table = O + 64);
        ON(paged, DATTN_ERR_INVALID_ARG, c.table = O - 28);
        ON(paged, DATTN_OK, c.table = O - 32);
    }
    #undef ON
    #define ON(call, status, ...) do { Call c; __VA_ARGS__; CHECK(c.call() == status); } while (0)
    ON(dense, DATTN_ERR_INVALID_ARG, c.T = 9; c.off = O + 16);
    ON(paged, DATTN_ERR_INVALID_ARG, c.T = 9; c.off = O - 8);
    ON(dense, DATTN_OK, c.T = 9; c.off = O - 12);
    ON(prefix, DATTN_ERR_INVALID_ARG, c.cp = O);
    ON(pool, DATTN_ERR_INVALID_ARG, c.table = O);
    // what the workspace of a ragged call and of a shared prefix may not lie on
    size_t n;
    { Call c; c.T = 9; c.off = A; n = c.need(); }
    #undef ON
    #define ON(status, ...) do { Call c; c.T = 9; c.off = A; c.ws = X; c.bytes = n; __VA_ARGS__; CHECK(c.dense() == status); } while (0)
    ON(DATTN_OK, (void)0);
    ON(DATTN_ERR_INVALID_ARG, c.out = X);
    ON(DATTN_ERR_INVALID_ARG, c.out = X - 4592);
    ON(DATTN_OK, c.out = X - 4608);
    ON(DATTN_ERR_INVALID_ARG, c.out = X + (n - 16) / 16 * 16);
    ON(DATTN_OK, c.out = X + (n + 15) / 16 * 16);
    ON(DATTN_ERR_INVALID_ARG, c.q = X + 1024);
    ON(DATTN_ERR_INVALID_ARG, c.cp = X + n - 4);
    ON(DATTN_ERR_INVALID_ARG, c.off = X);
    ON(DATTN_ERR_INVALID_ARG, c.off = X - 8);
    { Call c; n = c.need_shared(c.S); }
    #define SHARED(status, ...) do { Call c; c.ws = X; c.bytes = n; __VA_ARGS__; CHECK(c.prefix() == status); } while (0)
    SHARED(DATTN_OK, (void)0);
    SHARED(DATTN_ERR_INVALID_ARG, c.kp = X);
    SHARED(DATTN_ERR_INVALID_ARG, c.vp = X - 4080);
    SHARED(DATTN_OK, c.vp = X - 4096);
    SHARED(DATTN_ERR_INVALID_ARG, c.out = X + 16);
    { Call c; n = c.need_shared(48); c.ws = X; c.bytes = n; c.table = X + 32; CHECK(c.pool() == DATTN_ERR_INVALID_ARG); }
    { Call c; c.ws = O; CHECK(c.dense() == DATTN_OK); }   // none is needed: not looked at
    """)


# ------------------------------------------------------------------ the binding

@pytest.mark.parametrize("call", ["function", "entry"])
def test_a_shared_call_needs_its_length(call):
    """No shared_len is not "nothing shared": that would be another operator."""
    q, k, v, pos = tensors()
    table = torch.zeros(2, 4, dtype=torch.int32)
    with pytest.raises(TypeError, match="shared_len"):
        if call == "function":
            dattn.decode_shared_paged(q, k, v, table, pos, None)
        else:
            dattn.dattn_decode_shared_paged(q, k, v, torch.empty_like(q), table, pos, None)


def test_a_workspace_on_the_caches_is_refused(monkeypatch):
    """The binding's own check, ahead of the C entry's of the other tensors."""
    native = dattn.attend.__globals__
    q, k, v, pos = tensors()
    for n in ("_tensor", "_on_device"):
        monkeypatch.setitem(native, n, lambda t, *a: t.data_ptr() if isinstance(t, torch.Tensor) else None)
    apart = native["_apart_from_caches"]
    apart(torch.zeros(4096, dtype=torch.uint8), k, v)
    for cache in (k, v):
        raw = cache.view(-1).view(torch.uint8)
        for part in (raw[:64], raw[-16:], raw):
            with pytest.raises(ValueError, match="workspace overlaps"):
                apart(part, k, v)
        apart(raw[:0], k, v)
    whole = torch.zeros(3 * 32768, dtype=torch.uint8)  # K, workspace, V side by side
    k, v = (x.view(torch.float16).view(2, 64, 2, 64) for x in (whole[:32768], whole[65536:]))
    apart(whole[32768:65536], k, v)
    with pytest.raises(ValueError, match="V cache"):
        apart(whole[32768:65552], k, v)
