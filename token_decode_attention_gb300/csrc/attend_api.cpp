// attend_api.cpp -- C ABI of attention over a 16-bit cache with grouped heads
// (include/dattn.h): argument validation before anything is launched.
#include "dattn.h"

#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <map>
#include <mutex>
#include <tuple>
#include <type_traits>
#include <utility>

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
    if (static_cast<double>(s.n_kv_heads) * s.head_dim >= 1073741824.0)
        return fail(DATTN_ERR_UNSUPPORTED, "a position must hold fewer than 2^30 elements");
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

// What a call writes may share no byte with what it reads, nor `out` with the workspace.
struct Written {
    const void *at;
    double bytes;
    const char *name;

    int apart(const void *p, double n, const char *what) const {
        if (p == nullptr) return DATTN_OK;
        const double a = static_cast<double>(reinterpret_cast<uintptr_t>(at));
        const double b = static_cast<double>(reinterpret_cast<uintptr_t>(p));
        if (a < b + n && b < a + bytes) return fail(DATTN_ERR_INVALID_ARG, "%s overlaps %s", name, what);
        return DATTN_OK;
    }
};

// ------------------------------------------------------------------- plans

size_t round_up(size_t x, size_t m) { return (x + m - 1) / m * m; }

struct Plan {
    int dp = 0, slots = 0, smem = 0;
    bool tiles = false, token = false;  // which kernels run
    dattn::TokenArgs w{};
    dattn::TileArgs t{};
    size_t ws_bytes = 0;
    // where the parts of the workspace begin
    size_t ws_acc = 0, ws_ml = 0, t_plan = 0, t_items = 0, t_before = 0, t_seq = 0, t_cuts = 0, t_acc = 0, t_ml = 0,
           t_whole_acc = 0, t_whole_ml = 0;

    size_t take(size_t bytes) {
        const size_t at = ws_bytes;
        ws_bytes = at + round_up(bytes, 256);
        return at;
    }
};

constexpr double kTileUs = 1.9;      // of an SM, for a key tile of 256 rows of 128 channels
constexpr double kBytesUs = 6.8e6;   // of the GPU
constexpr long long kMaxMapStride = 1LL << 38;  // elements between rows that a tensor map takes
constexpr int kBoxRows = 8;  // fewest rows of a page's box
constexpr int kMaxColumns = 16;  // query heads of a key/value head in one CTA
constexpr int kStaticSmem = 1024;  // the kernel's static shared memory at most
constexpr size_t kWorkspaceAlign = 16;  // what a caller's workspace lies on
constexpr size_t kStateAlign = 32;      // what states of many tokens lie on, stored 32 bytes at a time
constexpr size_t kKeptPlans = 1024;  // a program that never repeats a shape starts anew

// One token per sequence, `cap` positions seen at most.  Measured (graph replay, inputs
// larger than L2 in all), us:
//  - Key/value heads of a CTA: the fewest of 1, 2, 4 with which all units are resident at
//    once, as each further wave of CTAs costs its start.  64 sequences of 8 heads, window
//    4096: 1, 2 heads 128, 119; 222 of 2, 240 positions, 15.7, 14.2; 168 of 16, 128
//    positions: 1, 2, 4 heads 34.9, 26.8, 23.2.
//  - Where that leaves most SMs idle, clusters of CTAs share a unit, as many as leave a warp
//    3/2 tiles on average: one sequence of 8 heads, window 1024 (65 tiles): 4, 8, 16 CTAs
//    5.9, 5.5, 5.7; 7 sequences of 32 heads, 8 tiles, D = 64: 1, 2 CTAs 3.9, 4.4.
//  - Up to kClusterTiles tiles a warp the merge in the same launch wins; beyond, chunks that
//    a second kernel merges: 3/2 as many as are resident for a batch, whose lengths differ
//    (19 sequences of 4 heads, 295 tiles: clusters of 4 19.5, 6 chunks 18.1), 3/4 for one
//    sequence (8 heads, 131072 positions: clusters of 16 91.6, chunks for 1/2, 3/4, 1 of
//    the slots 84.8, 83.0, 86.6).
constexpr long long kClusterTiles = 16;

int token_plan(const Shape &s, int cap, const dattn::DeviceFacts &df, Plan *p) {
    dattn::TokenArgs &w = p->w;
    const int group = s.n_heads / s.n_kv_heads;
    w.vheads_per_kv = (group + kMaxColumns - 1) / kMaxColumns;
    while (group % w.vheads_per_kv != 0) ++w.vheads_per_kv;
    w.gq = group / w.vheads_per_kv;
    w.div_gq = dattn::fast_div_of(w.gq);
    w.vheads = s.n_kv_heads * w.vheads_per_kv;
    w.own_only = s.shared > 0 ? 1 : 0;
    p->token = true;
    const long long slots = static_cast<long long>(df.sms) * dattn::token_ctas_per_sm(p->dp);
    const long long tiles = (static_cast<long long>(cap) + dattn::kTokenTile - 1) / dattn::kTokenTile;
    int hg = 1;
    auto units_of = [&](int heads) {
        return static_cast<long long>(s.batch) * ((w.vheads + heads - 1) / heads);
    };
    while (hg < dattn::kTokenWarps && 2 * hg <= w.vheads && units_of(hg) > slots) hg *= 2;
    const long long units = units_of(hg);
    w.heads_per_cta = hg;
    w.head_groups = (w.vheads + hg - 1) / hg;
    w.phases = dattn::kTokenWarps / hg;
    auto per_warp = [&](long long C) { return ((tiles + C - 1) / C + w.phases - 1) / w.phases; };
    long long C = 1;
    while (C < 16 && units * C * 2 <= slots && 2 * tiles >= 3 * w.phases * C * 2) C *= 2;
    if (w.own_only && per_warp(1) <= kClusterTiles) C = 1;  // its states are merged in any case
    const bool chunked = per_warp(C) > kClusterTiles || (w.own_only && C > 1);
    if (chunked) {
        C = std::max(1LL, s.batch == 1 ? slots * 3 / 4 / units : slots * 3 / 2 / units);
        w.chunk_tiles = static_cast<int>(std::max<long long>(4 * w.phases, (tiles + C - 1) / C));
        C = (tiles + w.chunk_tiles - 1) / w.chunk_tiles;
    }
    p->slots = dattn::kTokenSlots;  // a chunk has tiles for all of them
    p->smem = dattn::token_smem(p->dp, p->slots, w.gq);
    if (!chunked) {
        const int nt = w.gq > 8 ? 2 : 1;
        for (; C > 1; C /= 2) {
            p->slots = static_cast<int>(std::min<long long>(dattn::kTokenSlots, per_warp(C)));
            const long long rec = (hg * w.gq * (p->dp / 2) + C - 1) / C * C * 16LL;
            const long long smem = dattn::token_smem(p->dp, p->slots, w.gq) + rec;
            if (smem > df.max_smem_optin - kStaticSmem) continue;
            int fit = 0;
            if (dattn::attend_token_max_clusters(p->dp, nt, w.gq <= 4, static_cast<int>(smem), static_cast<int>(C),
                                                 &fit) != cudaSuccess) {
                cudaGetLastError();  // this cluster size is not available
                continue;
            }
            if (fit < units) continue;
            p->smem = static_cast<int>(smem);
            w.cluster = 1;
            break;
        }
        if (C == 1) {
            p->slots = static_cast<int>(std::min<long long>(dattn::kTokenSlots, per_warp(1)));
            p->smem = dattn::token_smem(p->dp, p->slots, w.gq);
        }
        w.chunk_tiles = static_cast<int>(tiles);
    }
    w.ring_bytes = dattn::token_ring_bytes(p->dp, p->slots, w.gq);
    w.chunks = static_cast<int>(C);
    if (!w.cluster && (w.chunks > 1 || w.own_only)) {
        const size_t states = static_cast<size_t>(s.batch) * s.n_heads * w.chunks;
        p->ws_acc = p->take(states * s.head_dim * sizeof(float));
        p->ws_ml = p->take(states * sizeof(float2));
    }
    if (units * C > 0x7fffffffLL) return fail(DATTN_ERR_UNSUPPORTED, "batch x n_kv_heads is too large");
    return DATTN_OK;
}

// Many tokens (or the shared positions), `cap` positions seen at most by one token.
int tiles_plan(const Shape &s, int cap, const dattn::DeviceFacts &df, Plan *p) {
    dattn::TileArgs &t = p->t;
    const int group = s.n_heads / s.n_kv_heads, rows = dattn::tile_rows(p->dp), keys = dattn::tile_keys(p->dp);
    const long long all_rows = static_cast<long long>(s.tokens) * group;
    p->tiles = true;
    t.div_group = dattn::fast_div_of(group);
    const long long items = (all_rows + rows - 1) / rows + (s.ragged ? s.batch : 0);
    if (items > 0x7fffff00LL) return fail(DATTN_ERR_UNSUPPORTED, "the batch is too large");
    t.max_items = static_cast<int>(items);
    // key tiles of an item at most: what its first token sees and the tokens behind it
    const long long seen = s.shared > 0 ? s.shared : std::min<long long>(s.rows, static_cast<long long>(cap) + rows);
    const double units = static_cast<double>(items) * s.n_kv_heads * ((seen + keys - 1) / keys + 1);
    if (units * 1024.0 > 4.0e18) return fail(DATTN_ERR_UNSUPPORTED, "the batch is too large");
    double ctas = df.sms;
    if (s.shared > 0) {
        // The sequences' own positions are worked on at the same time, on the other SMs: as
        // many for each as it has work, a key tile against the bytes of sequences half full.
        const double own_bytes = 2.0 * cap * s.batch * s.n_kv_heads * s.head_dim;
        const double tiles_us = units * kTileUs * p->dp / 128, own_us = own_bytes / kBytesUs * df.sms;
        ctas = std::max(1.0, df.sms * tiles_us / (tiles_us + own_us));
    }
    t.ctas = static_cast<int>(std::max(1.0, std::min(ctas, units / dattn::kTileMinUnits)));
    if (s.ragged) {
        p->t_plan = p->take(sizeof(dattn::TilePlan));
        p->t_items = p->take(sizeof(dattn::TileItem) * items);
        p->t_before = p->take(sizeof(long long) * (items + 1));
        p->t_cuts = p->take(sizeof(dattn::TileCut) * t.ctas);
        p->t_seq = p->take(sizeof(int) * (static_cast<size_t>(s.batch) + 1));
    } else {
        const size_t states = static_cast<size_t>(s.batch) * s.n_heads;
        p->t_whole_acc = p->take(states * s.head_dim * sizeof(float));
        p->t_whole_ml = p->take(states * sizeof(float2));
    }
    p->t_acc = p->take(2 * static_cast<size_t>(t.ctas) * rows * s.head_dim * sizeof(float));
    p->t_ml = p->take(2 * static_cast<size_t>(t.ctas) * rows * sizeof(float2));
    return DATTN_OK;
}

int make_plan(const Shape &s, Plan *out) {
    dattn::DeviceFacts df;
    if (int st = dattn::device_facts(&df)) return st;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return fail_cuda(e, "cudaGetDevice");
    // positions of its own that a sequence's token sees at most
    const int cap = s.shared > 0 ? std::max(1, s.apart ? s.rows : s.rows - s.shared)
                    : s.window > 0 && s.window < s.rows
                        ? static_cast<int>(std::min<long long>(s.rows, static_cast<long long>(s.window) + s.sinks))
                        : s.rows;
    using Key = std::tuple<int, int, int, bool, int, int, int, int, int, int>;
    static std::mutex mutex;
    static std::map<Key, Plan> plans;
    static std::map<int, bool> configured;
    const Key key{dev, s.batch, s.tokens, s.ragged, s.n_heads, s.n_kv_heads, s.head_dim, cap,
                  s.shared > 0 ? 0 : s.rows, s.shared};
    std::lock_guard<std::mutex> lock(mutex);
    const auto it = plans.find(key);
    if (it != plans.end()) {
        *out = it->second;
        return DATTN_OK;
    }
    if (!configured[dev]) {
        e = dattn::attend_token_configure(df.max_smem_optin);
        if (e == cudaSuccess) e = dattn::attend_tiles_configure(df.max_smem_optin);
        if (e != cudaSuccess) return fail_cuda(e, "cudaFuncSetAttribute(attention kernel)");
        configured[dev] = true;
    }
    Plan p;
    p.dp = s.head_dim <= 64 ? 64 : s.head_dim <= 128 ? 128 : 256;
    if (s.ragged || s.shared > 0)
        if (int st = tiles_plan(s, cap, df, &p)) return st;
    if (!s.ragged)
        if (int st = token_plan(s, cap, df, &p)) return st;
    if (p.tiles) p.ws_bytes += kStateAlign - kWorkspaceAlign;  // the parts begin on kStateAlign
    if (plans.size() >= kKeptPlans) plans.clear();
    plans[key] = p;
    *out = p;
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
    if (rows >= 2147483648.0)
        return fail(DATTN_ERR_UNSUPPORTED, "the cache must hold fewer than 2^31 positions in all");
    if (rows * kv_row > 4.0e18 || static_cast<double>(s.tokens) * q_stride > 4.0e18)
        return fail(DATTN_ERR_INVALID_ARG, "the tensors are too large");
    const double kv_bytes = 2.0 * rows * kv_row;
    const Written result{out, 2.0 * s.tokens * q_row, "out"};
    // the inputs but the cache
    auto apart = [&](const Written &w) {
        if (int st = w.apart(Q, 2.0 * ((s.tokens - 1.0) * q_stride + q_row), "Q")) return st;
        if (int st = w.apart(current_pos, 4.0 * s.batch, "current_pos")) return st;
        if (int st = w.apart(token_offsets, 4.0 * (s.batch + 1.0), "token_offsets")) return st;
        if (int st = w.apart(s.block_table, 4.0 * s.batch * s.max_pages, "block_table")) return st;
        if (!s.apart) return static_cast<int>(DATTN_OK);
        if (int st = w.apart(Kp, 2.0 * s.shared * kv_row, "K_prefix")) return st;
        return w.apart(Vp, 2.0 * s.shared * kv_row, "V_prefix");
    };
    if (int st = apart(result)) return st;
    if (int st = result.apart(K, kv_bytes, "the K cache")) return st;
    if (int st = result.apart(V, kv_bytes, "the V cache")) return st;
    Plan p;
    if (int st = make_plan(s, &p)) return st;
    if (p.ws_bytes > 0) {
        if (workspace == nullptr)
            return fail(DATTN_ERR_WORKSPACE, "workspace of %zu bytes required, got NULL", p.ws_bytes);
        if (reinterpret_cast<uintptr_t>(workspace) % kWorkspaceAlign != 0)
            return fail(DATTN_ERR_WORKSPACE, "workspace is not 16-byte aligned");
        if (workspace_bytes < p.ws_bytes)
            return fail(DATTN_ERR_WORKSPACE, "workspace of %zu bytes required, got %zu", p.ws_bytes,
                        workspace_bytes);
        const Written scratch{workspace, static_cast<double>(p.ws_bytes), "the workspace"};
        if (int st = apart(scratch)) return st;
        if (int st = scratch.apart(out, result.bytes, "out")) return st;
    }
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
    const size_t align = p.tiles ? kStateAlign : kWorkspaceAlign;
    char *const ws = reinterpret_cast<char *>(round_up(reinterpret_cast<uintptr_t>(workspace), align));
    auto at = [&](size_t offset, auto *&part) {
        part = reinterpret_cast<std::remove_reference_t<decltype(part)>>(ws + offset);
    };
    dattn::TokenArgs w = p.w;
    dattn::TileArgs t = p.t;
    cudaError_t e = cudaSuccess;
    if (p.tiles) {
        t.bound_ends = s.shared > 0 && !s.apart ? 1 : 0;
        if (s.ragged) {
            at(p.t_plan, t.plan);
            at(p.t_items, t.items);
            at(p.t_before, t.before);
            at(p.t_seq, t.seq_items);
            at(p.t_cuts, t.cuts);
        } else {
            at(p.t_whole_acc, t.whole_acc);
            at(p.t_whole_ml, t.whole_ml);
        }
        // A dense cache's tiles are one box each; a paged one's as many rows as divide a page.
        dattn::TileMaps m{};
        m.box_rows = dattn::tile_keys(p.dp);
        if (s.page_size > 0)
            while (s.page_size % m.box_rows != 0) m.box_rows /= 2;
        if (m.box_rows < kBoxRows) m.box_rows = 0;
        t.align = s.page_size > 0 && m.box_rows > 0 ? m.box_rows : 1;
        t.out_32 = s.head_dim % 16 == 0 && (reinterpret_cast<uintptr_t>(out) & 31u) == 0 ? 1 : 0;
        if (m.box_rows > 0) {
            const long long map_rows = s.apart ? s.shared : static_cast<long long>(rows);
            for (auto &[map, base] : {std::pair{&m.k, s.apart ? Kp : K}, std::pair{&m.v, s.apart ? Vp : V}})
                if (int st = dattn::encode_head_rows(map, base, map_rows, kv_row, s.n_kv_heads, s.head_dim, m.box_rows,
                                                     1, dtype))
                    return st;
        }
        if (128 % a.group == 0 && q_stride < kMaxMapStride) {
            m.q_tokens = 128 / a.group;
            if (int st = dattn::encode_head_rows(&m.q, Q, s.tokens, q_stride, s.n_heads, s.head_dim, m.q_tokens,
                                                 a.group, dtype))
                return st;
        }
        at(p.t_acc, t.acc);
        at(p.t_ml, t.ml);
        e = dattn::launch_attend_tiles(a, t, m, dtype, p.dp, stream);
        if (e != cudaSuccess) return fail_cuda(e, "attention kernel launch");
    }
    if (p.token) {
        const bool states = !w.cluster && (w.chunks > 1 || w.own_only);
        if (states) {
            at(p.ws_acc, w.ws_acc);
            at(p.ws_ml, w.ws_ml);
        }
        e = dattn::launch_attend_token(a, w, dtype, p.dp, p.smem, stream);
        if (e != cudaSuccess) return fail_cuda(e, "attention kernel launch");
        if (states) {
            e = dattn::launch_attend_merge(a, w, p.tiles ? &t : nullptr, dtype, p.dp, stream);
            if (e != cudaSuccess) return fail_cuda(e, "merge kernel launch");
        }
    }
    return DATTN_OK;
}

int workspace_of(const Shape &s, size_t *bytes) {
    if (bytes == nullptr) return fail(DATTN_ERR_INVALID_ARG, "bytes is NULL");
    if (int st = check_shape(s)) return st;
    Plan p;
    if (int st = make_plan(s, &p)) return st;
    *bytes = p.ws_bytes;
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
        if (own_len < 0) return fail(DATTN_ERR_INVALID_ARG, "own_len=%d must not be negative", own_len);
        Shape s = shape_of(batch, batch, false, n_heads, n_kv_heads, head_dim);
        s.shared = shared_len;
        s.apart = true;
        s.rows = std::max(1, own_len);
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
