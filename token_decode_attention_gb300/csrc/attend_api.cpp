// attend_api.cpp -- C ABI of attention over a 16-bit cache with grouped heads
// (include/dattn.h): argument validation before anything is launched.
#include "dattn.h"

#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "api_checks.h"
#include "dattn_internal.h"

namespace {

constexpr int kMaxHeadDim = 256;

// What the batch and its cache are; `rows` positions of a sequence's own.
struct Shape {
    int batch, tokens, n_heads, n_kv_heads, head_dim;
    int rows = 0;
    int shared = 0;     // positions that all sequences share
    bool apart = false;  // they lie in a tensor of their own, ahead of the cache's rows
    bool ragged = false;
    int window = 0, sinks = 0;
    int page_size = 0, max_pages = 0;  // 0: dense
    long long num_pages = 0;
    const int32_t *block_table = nullptr;
};

int check_shape(const Shape &s) {
    if (s.batch <= 0 || s.tokens <= 0 || s.n_heads <= 0 || s.n_kv_heads <= 0 || s.head_dim <= 0 || s.rows <= 0)
        return fail(DATTN_ERR_INVALID_ARG,
                    "sizes must be positive (batch=%d tokens=%d n_heads=%d n_kv_heads=%d head_dim=%d "
                    "seq_len=%d)",
                    s.batch, s.tokens, s.n_heads, s.n_kv_heads, s.head_dim, s.rows);
    if (s.n_heads % s.n_kv_heads != 0)
        return fail(DATTN_ERR_INVALID_ARG, "n_heads=%d must be a multiple of n_kv_heads=%d", s.n_heads,
                    s.n_kv_heads);
    if (s.head_dim % 8 != 0 || s.head_dim > kMaxHeadDim)
        return fail(DATTN_ERR_UNSUPPORTED, "head_dim=%d: must be a multiple of 8 and <= %d", s.head_dim,
                    kMaxHeadDim);
    if (!s.ragged && s.tokens != s.batch)
        return fail(DATTN_ERR_INVALID_ARG,
                    "without token_offsets each sequence brings one token: tokens=%d, batch=%d", s.tokens,
                    s.batch);
    if (s.window < 0 || s.sinks < 0)
        return fail(DATTN_ERR_INVALID_ARG, "window=%d and sinks=%d must not be negative", s.window, s.sinks);
    if (static_cast<double>(s.tokens) * s.n_heads >= 2147483648.0)
        return fail(DATTN_ERR_UNSUPPORTED, "tokens x n_heads must stay below 2^31");
    if (static_cast<double>(s.n_kv_heads) * s.head_dim >= 2147483648.0)
        return fail(DATTN_ERR_UNSUPPORTED, "a position must hold fewer than 2^31 elements");
    if (static_cast<double>(s.rows) + (s.apart ? s.shared : 0) >= 2147483648.0 - 1024)
        return fail(DATTN_ERR_UNSUPPORTED, "a sequence must hold fewer than 2^31 - 1024 positions");
    return DATTN_OK;
}

// The paged form's own arguments; s->rows receives the capacity of a sequence.
int check_pages(Shape *s) {
    if (int st = check_words(s->block_table, "block_table")) return st;
    if (s->page_size <= 0 || s->max_pages <= 0 || s->num_pages <= 0)
        return fail(DATTN_ERR_INVALID_ARG, "page_size=%d, max_pages=%d and num_pages=%lld must be positive",
                    s->page_size, s->max_pages, s->num_pages);
    const long long cap = static_cast<long long>(s->page_size) * s->max_pages;
    if (cap > 0x7fffffffLL)
        return fail(DATTN_ERR_UNSUPPORTED, "page_size x max_pages = %lld exceeds 2^31 - 1", cap);
    s->rows = static_cast<int>(cap);
    return DATTN_OK;
}

// `out` may share no byte with what the call reads.
int check_apart(const void *out, double out_bytes, const void *p, double bytes, const char *name) {
    const double a = static_cast<double>(reinterpret_cast<uintptr_t>(out));
    const double b = static_cast<double>(reinterpret_cast<uintptr_t>(p));
    if (a < b + bytes && b < a + out_bytes)
        return fail(DATTN_ERR_INVALID_ARG, "out overlaps %s", name);
    return DATTN_OK;
}

int attend(const void *Q, const void *Kp, const void *Vp, const void *K, const void *V, void *out, int dtype,
           const Shape &s, long long q_stride, const int32_t *token_offsets, const uint32_t *current_pos,
           void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    if (int st = check_tensor(Q, "Q")) return st;
    if (s.apart) {
        if (int st = check_tensor(Kp, "K_prefix")) return st;
        if (int st = check_tensor(Vp, "V_prefix")) return st;
    }
    if (int st = check_tensor(K, "K cache")) return st;
    if (int st = check_tensor(V, "V cache")) return st;
    if (int st = check_tensor(out, "out")) return st;
    if (int st = check_words(current_pos, "current_pos")) return st;
    if (s.ragged)
        if (int st = check_words(token_offsets, "token_offsets")) return st;
    if (dtype != DATTN_F16 && dtype != DATTN_BF16)
        return fail(DATTN_ERR_INVALID_ARG, "dtype=%d must be DATTN_F16 or DATTN_BF16", dtype);
    if (int st = check_shape(s)) return st;
    const long long q_row = static_cast<long long>(s.n_heads) * s.head_dim;
    const long long kv_row = static_cast<long long>(s.n_kv_heads) * s.head_dim;
    if (int st = check_stride(q_stride, q_row, 2, "q_stride")) return st;
    const double rows = s.page_size > 0 ? static_cast<double>(s.num_pages) * s.page_size
                                        : static_cast<double>(s.batch) * s.rows;
    if (rows * kv_row > 4.0e18 || static_cast<double>(s.tokens) * q_stride > 4.0e18)
        return fail(DATTN_ERR_INVALID_ARG, "the tensors are too large");
    const double out_bytes = 2.0 * s.tokens * q_row, kv_bytes = 2.0 * rows * kv_row;
    if (int st = check_apart(out, out_bytes, Q, 2.0 * ((s.tokens - 1.0) * q_stride + q_row), "Q")) return st;
    if (int st = check_apart(out, out_bytes, K, kv_bytes, "the K cache")) return st;
    if (int st = check_apart(out, out_bytes, V, kv_bytes, "the V cache")) return st;
    if (s.apart) {
        if (int st = check_apart(out, out_bytes, Kp, 2.0 * s.shared * kv_row, "K_prefix")) return st;
        if (int st = check_apart(out, out_bytes, Vp, 2.0 * s.shared * kv_row, "V_prefix")) return st;
    }
    (void)workspace;
    (void)workspace_bytes;
    dattn::DeviceFacts df;
    if (int st = dattn::device_facts(&df)) return st;
    dattn::AttendArgs a{};
    a.Q = Q;
    a.K = K;
    a.V = V;
    a.Kp = s.apart ? Kp : nullptr;
    a.Vp = s.apart ? Vp : nullptr;
    a.out = out;
    a.block_table = s.block_table;
    a.num_pages = s.num_pages;
    a.page_size = s.page_size;
    a.max_pages = s.max_pages;
    a.div_page = dattn::fast_div_of(std::max(1, s.page_size));
    a.offsets = token_offsets;
    a.cur_pos = current_pos;
    a.err = df.err_word;
    a.q_stride = q_stride;
    a.tokens = s.tokens;
    a.B = s.batch;
    a.H = s.n_heads;
    a.Hk = s.n_kv_heads;
    a.D = s.head_dim;
    a.group = s.n_heads / s.n_kv_heads;
    a.shared = s.shared;
    a.own_base = s.apart ? s.shared : 0;
    a.S = a.own_base + s.rows;
    a.window = s.window;
    a.sinks = s.sinks;
    a.qscale = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(s.head_dim)));
    const cudaError_t e = dattn::launch_attend(a, dtype, stream);
    return e == cudaSuccess ? DATTN_OK : fail_cuda(e, "attention kernel launch");
}

int workspace_of(const Shape &s, size_t *bytes) {
    if (bytes == nullptr) return fail(DATTN_ERR_INVALID_ARG, "bytes is NULL");
    if (int st = check_shape(s)) return st;
    *bytes = 0;
    return DATTN_OK;
}

Shape shape_of(int batch, int tokens, bool ragged, int n_heads, int n_kv_heads, int head_dim) {
    Shape s{};
    s.batch = batch;
    s.tokens = tokens;
    s.ragged = ragged;
    s.n_heads = n_heads;
    s.n_kv_heads = n_kv_heads;
    s.head_dim = head_dim;
    return s;
}

int check_shared(int shared_len) {
    if (shared_len <= 0) return fail(DATTN_ERR_INVALID_ARG, "shared_len=%d must be positive", shared_len);
    return DATTN_OK;
}

}  // namespace

extern "C" {

int dattn_attend_workspace_bytes(int batch, int tokens, int ragged, int n_heads, int n_kv_heads, int head_dim,
                                 int seq_len, int window, int sinks, size_t *bytes) {
    return guarded([&]() -> int {
        Shape s = shape_of(batch, tokens, ragged != 0, n_heads, n_kv_heads, head_dim);
        s.rows = seq_len;
        s.window = window;
        s.sinks = sinks;
        return workspace_of(s, bytes);
    });
}

int dattn_attend(const void *Q, const void *K_cache, const void *V_cache, void *out, int dtype, int batch,
                 int tokens, const int32_t *token_offsets, long long q_stride, int n_heads, int n_kv_heads,
                 int head_dim, int seq_len, int window, int sinks, const uint32_t *current_pos,
                 void *workspace, size_t workspace_bytes, dattn_stream_t stream) {
    return guarded([&]() -> int {
        Shape s = shape_of(batch, tokens, token_offsets != nullptr, n_heads, n_kv_heads, head_dim);
        s.rows = seq_len;
        s.window = window;
        s.sinks = sinks;
        return attend(Q, nullptr, nullptr, K_cache, V_cache, out, dtype, s, q_stride, token_offsets,
                      current_pos, workspace, workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
    });
}

int dattn_attend_paged(const void *Q, const void *K_pages, const void *V_pages, void *out, int dtype, int batch,
                       int tokens, const int32_t *token_offsets, long long q_stride, int n_heads,
                       int n_kv_heads, int head_dim, int page_size, int max_pages, long long num_pages,
                       const int32_t *block_table, int window, int sinks, const uint32_t *current_pos,
                       void *workspace, size_t workspace_bytes, dattn_stream_t stream) {
    return guarded([&]() -> int {
        Shape s = shape_of(batch, tokens, token_offsets != nullptr, n_heads, n_kv_heads, head_dim);
        s.page_size = page_size;
        s.max_pages = max_pages;
        s.num_pages = num_pages;
        s.block_table = block_table;
        if (int st = check_pages(&s)) return st;
        s.window = window;
        s.sinks = sinks;
        return attend(Q, nullptr, nullptr, K_pages, V_pages, out, dtype, s, q_stride, token_offsets,
                      current_pos, workspace, workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
    });
}

int dattn_decode_shared_workspace_bytes(int batch, int n_heads, int n_kv_heads, int head_dim, int shared_len,
                                        int own_len, size_t *bytes) {
    return guarded([&]() -> int {
        if (int st = check_shared(shared_len)) return st;
        Shape s = shape_of(batch, batch, false, n_heads, n_kv_heads, head_dim);
        s.shared = shared_len;
        s.rows = own_len;
        return workspace_of(s, bytes);
    });
}

int dattn_decode_shared(const void *Q, const void *K_prefix, const void *V_prefix, const void *K_cache,
                        const void *V_cache, void *out, int dtype, int batch, long long q_stride, int n_heads,
                        int n_kv_heads, int head_dim, int shared_len, int seq_len,
                        const uint32_t *current_pos, void *workspace, size_t workspace_bytes,
                        dattn_stream_t stream) {
    return guarded([&]() -> int {
        if (int st = check_shared(shared_len)) return st;
        Shape s = shape_of(batch, batch, false, n_heads, n_kv_heads, head_dim);
        s.shared = shared_len;
        s.apart = true;
        s.rows = seq_len;
        return attend(Q, K_prefix, V_prefix, K_cache, V_cache, out, dtype, s, q_stride, nullptr, current_pos,
                      workspace, workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
    });
}

int dattn_decode_shared_paged(const void *Q, const void *K_pages, const void *V_pages, void *out, int dtype,
                              int batch, long long q_stride, int n_heads, int n_kv_heads, int head_dim,
                              int page_size, int max_pages, long long num_pages, const int32_t *block_table,
                              int shared_len, const uint32_t *current_pos, void *workspace,
                              size_t workspace_bytes, dattn_stream_t stream) {
    return guarded([&]() -> int {
        if (int st = check_shared(shared_len)) return st;
        Shape s = shape_of(batch, batch, false, n_heads, n_kv_heads, head_dim);
        s.page_size = page_size;
        s.max_pages = max_pages;
        s.num_pages = num_pages;
        s.block_table = block_table;
        if (int st = check_pages(&s)) return st;
        if (shared_len > s.rows)
            return fail(DATTN_ERR_INVALID_ARG, "shared_len=%d exceeds the %d positions of a sequence",
                        shared_len, s.rows);
        s.shared = shared_len;
        return attend(Q, nullptr, nullptr, K_pages, V_pages, out, dtype, s, q_stride, nullptr, current_pos,
                      workspace, workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
    });
}

}  // extern "C"
