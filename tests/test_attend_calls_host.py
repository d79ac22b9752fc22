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
