// q8_api.cpp -- C ABI of the rotary operator and of the 8-bit KV cache
// (include/dattn.h): argument validation before anything is launched, the
// table of turn fractions of a rotation, and the plan of the 8-bit decode.
#include "dattn.h"

#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <map>
#include <mutex>
#include <tuple>

#include "api_checks.h"
#include "dattn_internal.h"

namespace {

constexpr int kMaxHeadDim = 256;
constexpr int kMaxPartitions = 65535;
constexpr int kMaxColumns = 16;  // query heads of a key/value head in one CTA
constexpr int kStaticSmem = 4096;  // the decode kernel's static shared memory at most
// Tiles of a warp up to which the cluster plan is taken.  Measured here and below with one
// f16 per weight (the second adds 0 to 7 %, under either plan): (cluster, split)
// one 7B-class step of 8 key/value heads, 2 tiles, 8.4 and 8.7 us; of 32, 4 tiles, 9.9
// and 12.1; 32 ragged sequences of 8 heads, 8 tiles, 13.6 and 16.0; 37 of 4 heads, 8
// tiles, 14.7 and 16.2; 64 query on 8 key/value heads over 32768 positions, 16 tiles
// and 7 in the split plan, 26.6 and 18.1.
constexpr long long kClusterTiles = 8;
constexpr long long kUnitTiles = 16;  // the same with a CTA for each unit
constexpr long long kShortUnitTiles = 10;
constexpr size_t kKeptPlans = 1024;  // a program that never repeats a shape starts anew

// ------------------------------------------------------------------ rotation

int check_rope(const dattn_rope_params *r, int head_dim) {
    if (r == nullptr) return fail(DATTN_ERR_INVALID_ARG, "rope is NULL");
    if (r->rope_dims < 2 || r->rope_dims > head_dim || r->rope_dims % 2 != 0)
        return fail(DATTN_ERR_INVALID_ARG, "rope_dims=%d must be even and in [2, head_dim=%d]",
                    r->rope_dims, head_dim);
    if (!(r->rope_base > 1.0) || !std::isfinite(r->rope_base))
        return fail(DATTN_ERR_INVALID_ARG, "rope_base must be a finite number above 1");
    if (!(r->magnitude > 0.0) || !(r->magnitude < 1e30))
        return fail(DATTN_ERR_INVALID_ARG, "magnitude must be a positive number below 1e30");
    if (r->scaling == DATTN_ROPE_UNSCALED) return DATTN_OK;
    if (r->scaling != DATTN_ROPE_LINEAR && r->scaling != DATTN_ROPE_BASE &&
        r->scaling != DATTN_ROPE_BY_PARTS)
        return fail(DATTN_ERR_INVALID_ARG, "scaling=%d is not a dattn_rope_scaling", r->scaling);
    if (!(r->factor >= 1.0) || !(r->factor < 1e9))
        return fail(DATTN_ERR_INVALID_ARG, "factor must be in [1, 1e9)");
    if (r->scaling == DATTN_ROPE_BASE && r->rope_dims == 2)
        return fail(DATTN_ERR_INVALID_ARG, "scaling the base needs rope_dims above 2");
    if (r->scaling == DATTN_ROPE_BY_PARTS) {
        if (!(r->original_len > 0.0) || !std::isfinite(r->original_len))
            return fail(DATTN_ERR_INVALID_ARG, "original_len must be positive and finite");
        if (!(r->low_turns >= 0.0) || !(r->high_turns > r->low_turns) || !std::isfinite(r->high_turns))
            return fail(DATTN_ERR_INVALID_ARG, "turns must satisfy 0 <= low_turns < high_turns");
    }
    return DATTN_OK;
}

// The table depends on the parameters only and a decode loop passes the same
// ones every step: the last one is kept per thread (long double is software
// arithmetic on some hosts).
void rope_table(const dattn_rope_params &r, dattn::RopeTable *out) {
    struct Kept {
        int dims = 0, scaling = 0;
        double base = 0, factor = 0, len = 0, low = 0, high = 0;
        unsigned long long frac[kMaxHeadDim / 2];
    };
    thread_local Kept k;
    if (k.dims != r.rope_dims || k.scaling != r.scaling || k.base != r.rope_base ||
        k.factor != r.factor || k.len != r.original_len || k.low != r.low_turns ||
        k.high != r.high_turns) {
        const int d = r.rope_dims;
        const double base = r.scaling == DATTN_ROPE_BASE
                                ? r.rope_base * std::pow(r.factor, static_cast<double>(d) / (d - 2))
                                : r.rope_base;
        const long double two_pi = 6.283185307179586476925286766559005768L;
        for (int i = 0; i < d / 2; ++i) {
            double theta = std::pow(base, -2.0 * i / d);
            if (r.scaling == DATTN_ROPE_LINEAR) theta /= r.factor;
            if (r.scaling == DATTN_ROPE_BY_PARTS) {
                const double turns = r.original_len * theta / static_cast<double>(two_pi);
                const double keep =
                    std::min(1.0, std::max(0.0, (turns - r.low_turns) / (r.high_turns - r.low_turns)));
                theta = theta * keep + theta / r.factor * (1.0 - keep);
            }
            // theta <= 1: theta / (2 pi) 2^64 fits in 62 bits
            k.frac[i] = static_cast<unsigned long long>(
                std::llroundl(std::ldexp(static_cast<long double>(theta) / two_pi, 64)));
        }
        k.dims = d;
        k.scaling = r.scaling;
        k.base = r.rope_base;
        k.factor = r.factor;
        k.len = r.original_len;
        k.low = r.low_turns;
        k.high = r.high_turns;
    }
    std::memcpy(out->turn_frac, k.frac, sizeof(k.frac[0]) * (r.rope_dims / 2));
    out->magnitude = static_cast<float>(r.magnitude);
    out->rope_dims = r.rope_dims;
    out->traditional = r.traditional ? 1 : 0;
}

// ------------------------------------------------------------- 8-bit caches

// Shape of a cache: `rows` is seq_len (dense) or page_size (paged).
struct Cache {
    int kv_type, scale_block;
    int page_size = 0, max_pages = 0;  // 0: dense
    long long num_pages = 0;
    const int32_t *block_table = nullptr;
};

// The sizes of a batch.  The queries know no more: what a paged cache's tables can name
// may be more than its pool holds.
int check_sizes(int batch, int n_heads, int n_kv_heads, int head_dim, int seq_len) {
    if (batch <= 0 || n_heads <= 0 || n_kv_heads <= 0 || head_dim <= 0 || seq_len <= 0)
        return fail(DATTN_ERR_INVALID_ARG,
                    "sizes must be positive (batch=%d n_heads=%d n_kv_heads=%d head_dim=%d "
                    "seq_len=%d)",
                    batch, n_heads, n_kv_heads, head_dim, seq_len);
    if (n_heads % n_kv_heads != 0)
        return fail(DATTN_ERR_INVALID_ARG, "n_heads=%d must be a multiple of n_kv_heads=%d", n_heads,
                    n_kv_heads);
    if (head_dim % 16 != 0 || head_dim > kMaxHeadDim)
        return fail(DATTN_ERR_UNSUPPORTED, "head_dim=%d: must be a multiple of 16 and <= %d",
                    head_dim, kMaxHeadDim);
    if (static_cast<double>(n_kv_heads) * head_dim >= 2147483648.0)
        return fail(DATTN_ERR_UNSUPPORTED, "a position must hold fewer than 2^31 elements");
    if (static_cast<double>(batch) * n_heads * head_dim > 4.0e18)
        return fail(DATTN_ERR_INVALID_ARG, "the batch is too large");
    return DATTN_OK;
}

int check_cache(int batch, int n_heads, int n_kv_heads, int head_dim, int seq_len, const Cache &c) {
    if (c.kv_type != DATTN_KV_E4M3 && c.kv_type != DATTN_KV_INT8)
        return fail(DATTN_ERR_INVALID_ARG, "kv_type=%d is not a dattn_kv_type", c.kv_type);
    if (int st = check_sizes(batch, n_heads, n_kv_heads, head_dim, seq_len)) return st;
    if (c.scale_block <= 0)
        return fail(DATTN_ERR_INVALID_ARG, "scale_block=%d must be positive", c.scale_block);
    // rows of the cache are counted in 31 bits
    const double lead = c.page_size > 0 ? static_cast<double>(c.num_pages) * c.page_size
                                        : static_cast<double>(batch) * seq_len;
    if (lead >= 2147483648.0)
        return fail(DATTN_ERR_UNSUPPORTED, "the cache must hold fewer than 2^31 positions in all");
    if (lead * n_kv_heads * head_dim > 4.0e18)
        return fail(DATTN_ERR_INVALID_ARG, "the cache is too large");
    return DATTN_OK;
}

// The paged form's own arguments; *seq_len receives the capacity of a sequence.
int check_pages(const Cache &c, int *seq_len) {
    if (int st = check_words(c.block_table, "block_table")) return st;
    if (c.page_size <= 0 || c.max_pages <= 0 || c.num_pages <= 0)
        return fail(DATTN_ERR_INVALID_ARG,
                    "page_size=%d, max_pages=%d and num_pages=%lld must be positive", c.page_size,
                    c.max_pages, c.num_pages);
    const long long cap = static_cast<long long>(c.page_size) * c.max_pages;
    if (cap > 0x7fffffffLL)
        return fail(DATTN_ERR_UNSUPPORTED, "page_size x max_pages = %lld exceeds 2^31 - 1", cap);
    if (c.scale_block > 0 && c.page_size % c.scale_block != 0)
        return fail(DATTN_ERR_INVALID_ARG, "page_size=%d must be a multiple of scale_block=%d",
                    c.page_size, c.scale_block);
    *seq_len = static_cast<int>(cap);
    return DATTN_OK;
}

int scale_rows_of(const Cache &c, int seq_len) {
    const int rows = c.page_size > 0 ? c.page_size : seq_len;
    return (rows - 1) / c.scale_block + 1;
}

struct Plan {
    int dp = 0, nt = 0, warps = 0, slots = 0;
    int gq = 0, vheads = 0, vheads_per_kv = 0;
    int HG = 0, NHG = 0, PH = 0, G = 0, sms = 0;
    int cluster = 0, smem = 0, ctas_per_sm = 1, extra = 0;
    int combine_chunk = 0, combine_inflight = 0;
    size_t prefix_bytes = 0, acc_bytes = 0, ws_bytes = 0;
};

size_t round_up(size_t x, size_t m) { return (x + m - 1) / m * m; }

// A plan without partial states in memory in place of the split plan *p, where that is
// faster: a CTA, or a cluster of them that merges in shared memory, takes a (sequence,
// group of hg heads) unit whole.
//
// Units of their own CTAs, as many waves of them as it takes, where there are enough to
// fill most of the SMs' slots and a warp's tiles of a full sequence are at most
// kUnitTiles: the most heads for which both hold.  Short runs of the cache per position
// cost more than the split plan's merge, so no fewer than an eighth of the heads, or a
// twentieth where a warp's tiles are at most kShortUnitTiles.  Measured with ragged
// lengths, these units and the split plan, us: 512 sequences of 8 heads up to 128
// positions 28.0, 62.2; 256 of 8 up to 1024 56.8, 70.7; 128 of 32 up to 512 55.8, 59.2;
// 256 of 8 up to 2048, one head per CTA, 98.2, 108.8; 16 of 40 up to 576, two heads,
// 17.1, 18.4.  What the last rule excludes: 64 of 32 up to 1024, two heads, 54.2, 53.7; 16
// of 40 up to 996, two heads, 25.0, 23.8.
//
// With fewer units, calls bound by latency: clusters of C CTAs, all resident at once.  Of
// the head groups and cluster sizes that fit, the one with the fewest tiles for a warp at
// full length; then fewer CTAs.
int cluster_plan(int B, int D, long long tiles, const dattn::DeviceFacts &df, Plan *p) {
    const long long slots = static_cast<long long>(df.sms) * p->ctas_per_sm;
    auto use = [&](int hg, int C, long long smem) {
        p->HG = hg;
        p->NHG = (p->vheads + hg - 1) / hg;
        p->PH = p->warps / hg;
        p->cluster = C;
        p->G = static_cast<int>(static_cast<long long>(B) * p->NHG * C);
        p->smem = static_cast<int>(smem);
    };
    const long long ring = static_cast<long long>(p->warps) * p->slots * dattn::q8_tile_bytes(p->dp);
    for (int hg = 8; hg >= 1 && hg * 20 >= p->vheads; hg /= 2) {
        if (hg > std::min(p->vheads, p->warps)) continue;
        const long long units = static_cast<long long>(B) * ((p->vheads + hg - 1) / hg);
        const long long per_warp = (tiles + p->warps / hg - 1) / (p->warps / hg);
        if (10 * units < 7 * slots || units > 0x7fffffffLL) continue;
        if (per_warp > (hg * 8 >= p->vheads ? kUnitTiles : kShortUnitTiles)) continue;
        use(hg, 1, ring);
        return DATTN_OK;
    }
    long long best = 0, best_smem = 0;
    int best_hg = 0, best_C = 0;
    for (int hg = 1; hg <= std::min(p->vheads, p->warps); hg *= 2) {
        const long long units = static_cast<long long>(B) * ((p->vheads + hg - 1) / hg);
        const int ph = p->warps / hg;
        for (int C = 1; C <= 16 && units * C <= slots; C *= 2) {
            const long long per_warp = ((tiles + C - 1) / C + ph - 1) / ph;
            if (best != 0 && per_warp >= best) continue;
            // the records of a CTA's share of the unit's (query head, channel pair) outputs
            const long long rec = C > 1 ? (hg * p->gq * (p->dp / 2) + C - 1) / C * C * 16LL : 0;
            if (ring + rec > df.max_smem_optin - kStaticSmem) continue;
            int fit = 0;
            if (dattn::decode_q8_max_clusters(p->dp, p->nt, dattn::q8_pair(p->gq),
                                              static_cast<int>(ring + rec), C, &fit) != cudaSuccess) {
                cudaGetLastError();  // this cluster size is not available
                continue;
            }
            if (fit < units) continue;
            best = per_warp;
            best_smem = ring + rec;
            best_hg = hg;
            best_C = C;
        }
    }
    // The split plan costs a second launch and the states' way through memory, about
    // two tiles of a warp; the cluster plan waits for its longest sequence.
    const double split = static_cast<double>(B) * p->NHG * tiles / (static_cast<double>(p->G) * p->PH);
    if (best > 0 && best <= kClusterTiles && best <= split + 2.0) use(best_hg, best_C, best_smem);
    return DATTN_OK;
}

int make_plan(int B, int H, int Hk, int D, int S, int num_partitions, Plan *out) {
    if (num_partitions < 0)
        return fail(DATTN_ERR_INVALID_ARG, "num_partitions=%d must be >= 0", num_partitions);
    dattn::DeviceFacts df;
    if (int st = dattn::device_facts(&df)) return st;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return fail_cuda(e, "cudaGetDevice");
    using Key = std::tuple<int, int, int, int, int, int, int>;
    static std::mutex mutex;
    static std::map<Key, Plan> plans;
    static std::map<int, bool> configured;
    const Key key{dev, B, H, Hk, D, S, num_partitions};
    std::lock_guard<std::mutex> lock(mutex);
    const auto it = plans.find(key);
    if (it != plans.end()) {
        *out = it->second;
        return DATTN_OK;
    }
    if (!configured[dev]) {
        e = dattn::decode_q8_configure(df.max_smem_optin);
        if (e != cudaSuccess) return fail_cuda(e, "cudaFuncSetAttribute(8-bit decode kernel)");
        configured[dev] = true;
    }
    Plan p;
    p.sms = df.sms;
    // virtual heads: the query heads of a key/value head, in equal groups of at
    // most kMaxColumns
    const int group = H / Hk;
    p.vheads_per_kv = (group + kMaxColumns - 1) / kMaxColumns;
    while (group % p.vheads_per_kv != 0) ++p.vheads_per_kv;
    p.gq = group / p.vheads_per_kv;
    p.vheads = Hk * p.vheads_per_kv;
    p.nt = p.gq > 8 ? 2 : 1;
    p.dp = D <= 64 ? 64 : D <= 128 ? 128 : 256;
    p.warps = dattn::kQ8Warps;
    p.slots = dattn::q8_slots(p.dp, p.nt);
    p.ctas_per_sm = dattn::q8_ctas_per_sm(p.dp, p.nt);
    // Heads per CTA, of those that keep the most warps busy.  More heads make longer
    // runs of the cache per position (one 1 GiB sequence of 32 heads: 158 us with 8,
    // 171 with 4, 169 with 2, 189 with 1), fewer make fewer partial states to write
    // and merge, (G + U) HG gq D floats of them (64 query on 8 key/value heads, 32768
    // positions: 29 us with 8, 21 with 4, 19 with 2, 18 with 1).  Taken: the most
    // heads whose states, written and read, stay within 2 % of the cache's capacity;
    // else one.  With 1, 2, 4 and 8 %, us: 16 sequences of 40 heads up to 996 positions
    // 26.5, 23.3, 23.3, 23.3; 14 of 16 up to 2880 26.2, 23.2, 22.4, 23.3; 32 of 8 up to
    // 4096 32.6, 31.3, 32.0, 34.9; one of 8 with 131072 47.5, 49.1, 51.4, 51.5.
    const long long slots = static_cast<long long>(df.sms) * p.ctas_per_sm;
    const double cache_bytes = 2.0 * B * S * static_cast<double>(Hk) * D;
    double best = 0.0;
    for (int hg = 1; hg <= std::min(p.vheads, p.warps); ++hg) {
        const int nhg = (p.vheads + hg - 1) / hg;
        const double busy = static_cast<double>(p.vheads) / (static_cast<double>(nhg) * hg) *
                            (p.warps / hg * hg) / p.warps;
        const double states = (slots + static_cast<double>(B) * nhg) * hg * p.gq * D * 8.0;
        if (busy > best + 1e-9 || (busy > best - 1e-9 && states <= 0.02 * cache_bytes)) {
            best = std::max(best, busy);
            p.HG = hg;
            p.NHG = nhg;
        }
    }
    p.PH = p.warps / p.HG;
    p.smem = p.warps * p.slots * dattn::q8_tile_bytes(p.dp);
    const long long tiles = (static_cast<long long>(S) + dattn::kQ8Tile - 1) / dattn::kQ8Tile;
    // What beginning a unit costs a CTA (the first tiles' latency, the epilogue), in
    // tiles of a warp.  Measured with 0, 2, 4 and 6: 64 ragged sequences of 32 heads
    // 99, 92, 90.6, 92 us; 37 of 4 heads 21.1, 17.2, 16.4, 16.5 us.
    p.extra = 4 * p.PH;
    const double capacity = static_cast<double>(B) * p.NHG * tiles;
    if (static_cast<double>(p.NHG) * (tiles + p.extra) >= 2147483648.0)
        return fail(DATTN_ERR_UNSUPPORTED, "head groups x seq_len must stay below 2^35");
    if (num_partitions > 0) {
        p.G = std::min(num_partitions, kMaxPartitions);
    } else {
        // every resident CTA slot; fewer when a partition would hold less than one
        // tile per warp
        const long long by_work = static_cast<long long>(capacity) / p.PH;
        p.G = static_cast<int>(
            std::max(1LL, std::min<long long>(slots, by_work)));
    }
    if (static_cast<double>(B) * p.NHG * (tiles + p.extra) * (p.G + 1.0) > 4.0e18)
        return fail(DATTN_ERR_UNSUPPORTED, "batch of %.3g tiles is too large", capacity);
    if (num_partitions == 0)
        if (int st = cluster_plan(B, D, tiles, df, &p)) return st;
    if (p.G > 1 && p.cluster == 0) {
        const size_t units = static_cast<size_t>(B) * p.NHG;
        const size_t rows = (static_cast<size_t>(p.G) + units) * p.HG * p.gq;
        p.prefix_bytes = round_up((static_cast<size_t>(B) + 1) * sizeof(long long), 256);
        p.acc_bytes = round_up(rows * D * sizeof(float), 256);
        p.ws_bytes = p.prefix_bytes + p.acc_bytes + rows * sizeof(float2);
        dattn::combine_shape(D, p.G, static_cast<long long>(units), &p.combine_chunk,
                             &p.combine_inflight);
        if (static_cast<double>(B) * H * ((D + p.combine_chunk - 1) / p.combine_chunk) > 2147483647.0)
            return fail(DATTN_ERR_UNSUPPORTED, "batch x n_heads is too large");
    }
    if (plans.size() >= kKeptPlans) plans.clear();
    plans[key] = p;
    *out = p;
    return DATTN_OK;
}

int decode(const void *Q, const void *K, const void *V, const float *K_scale, const float *V_scale,
           void *out, int batch, int n_heads, int n_kv_heads, int head_dim, int seq_len,
           const Cache &c, const uint32_t *current_pos, void *workspace, size_t workspace_bytes,
           int num_partitions, cudaStream_t stream) {
    if (int st = check_tensor(Q, "Q")) return st;
    if (int st = check_tensor(K, "K cache")) return st;
    if (int st = check_tensor(V, "V cache")) return st;
    if (int st = check_words(K_scale, "K_scale")) return st;
    if (int st = check_words(V_scale, "V_scale")) return st;
    if (int st = check_tensor(out, "out")) return st;
    if (int st = check_words(current_pos, "current_pos")) return st;
    if (int st = check_cache(batch, n_heads, n_kv_heads, head_dim, seq_len, c)) return st;
    Plan p;
    if (int st = make_plan(batch, n_heads, n_kv_heads, head_dim, seq_len, num_partitions, &p)) return st;
    if (p.ws_bytes > 0) {
        if (workspace == nullptr)
            return fail(DATTN_ERR_WORKSPACE, "workspace of %zu bytes required, got NULL", p.ws_bytes);
        if (reinterpret_cast<uintptr_t>(workspace) & 15u)
            return fail(DATTN_ERR_WORKSPACE, "workspace is not 16-byte aligned");
        if (workspace_bytes < p.ws_bytes)
            return fail(DATTN_ERR_WORKSPACE, "workspace of %zu bytes required, got %zu", p.ws_bytes,
                        workspace_bytes);
    }
    dattn::DeviceFacts df;
    if (int st = dattn::device_facts(&df)) return st;
    char *ws = static_cast<char *>(workspace);
    dattn::Q8DecodeArgs a{};
    a.Q = Q;
    a.K = static_cast<const unsigned char *>(K);
    a.V = static_cast<const unsigned char *>(V);
    a.ks = K_scale;
    a.vs = V_scale;
    a.out = out;
    a.cur_pos = current_pos;
    const bool split = p.G > 1 && p.cluster == 0;  // partial states go through the workspace
    if (split) {
        a.ws_prefix = reinterpret_cast<long long *>(ws);
        a.ws_acc = reinterpret_cast<float *>(ws + p.prefix_bytes);
        a.ws_ml = reinterpret_cast<float2 *>(ws + p.prefix_bytes + p.acc_bytes);
    }
    a.err = df.err_word;
    a.block_table = c.block_table;
    a.num_pages = c.num_pages;
    a.page_size = c.page_size;
    a.max_pages = c.max_pages;
    a.scale_rows = scale_rows_of(c, seq_len);
    a.div_page = dattn::fast_div_of(std::max(1, c.page_size));
    a.div_block = dattn::fast_div_of(c.scale_block);
    a.B = batch;
    a.H = n_heads;
    a.D = head_dim;
    a.S = seq_len;
    a.kv_heads = n_kv_heads;
    a.gq = p.gq;
    a.div_gq = dattn::fast_div_of(p.gq);
    a.vheads = p.vheads;
    a.vheads_per_kv = p.vheads_per_kv;
    a.heads_per_cta = p.HG;
    a.head_groups = p.NHG;
    a.phases = p.PH;
    a.partitions = p.G;
    a.cluster = p.cluster;
    a.extra = p.extra;
    a.tile_in_page = c.page_size % dattn::kQ8Tile == 0 ? 1 : 0;
    a.qscale = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(head_dim)));
    cudaError_t e = dattn::launch_decode_q8(a, p.dp, p.nt, c.kv_type, p.smem, stream);
    if (e != cudaSuccess) return fail_cuda(e, "8-bit decode kernel launch");
    if (split) {
        dattn::CombineArgs m{};
        m.ws_acc = a.ws_acc;
        m.ws_ml = a.ws_ml;
        m.ws_prefix = a.ws_prefix;
        m.cur_pos = current_pos;
        m.out = out;
        m.B = batch;
        m.H = n_heads;
        m.D = head_dim;
        m.S = seq_len;
        m.heads_per_cta = p.HG * p.gq;
        m.head_groups = p.NHG;
        m.partitions = p.G;
        m.chunk = p.combine_chunk;
        m.inflight = p.combine_inflight;
        m.shift = dattn::kQ8TileShift;
        m.extra = p.extra;
        e = dattn::launch_combine(m, stream);
        if (e != cudaSuccess) return fail_cuda(e, "combine kernel launch");
    }
    return DATTN_OK;
}

int append(const void *q_new, const void *k_new, const void *v_new, void *q_out, void *K, void *V,
           float *K_scale, float *V_scale, int batch, int tokens, const int32_t *token_offsets,
           long long q_stride, long long k_stride, long long v_stride, int n_heads, int n_kv_heads,
           int head_dim, int seq_len, const Cache &c, const dattn_rope_params *rope,
           const uint32_t *current_pos, cudaStream_t stream) {
    if (int st = check_tensor(q_new, "q_new")) return st;
    if (int st = check_tensor(k_new, "k_new")) return st;
    if (int st = check_tensor(v_new, "v_new")) return st;
    if (int st = check_tensor(q_out, "q_out")) return st;
    if (int st = check_tensor(K, "K cache")) return st;
    if (int st = check_tensor(V, "V cache")) return st;
    if (int st = check_words(K_scale, "K_scale")) return st;
    if (int st = check_words(V_scale, "V_scale")) return st;
    if (int st = check_words(current_pos, "current_pos")) return st;
    if (token_offsets != nullptr)
        if (int st = check_words(token_offsets, "token_offsets")) return st;
    if (int st = check_cache(batch, n_heads, n_kv_heads, head_dim, seq_len, c)) return st;
    if (tokens <= 0) return fail(DATTN_ERR_INVALID_ARG, "tokens=%d must be positive", tokens);
    if (token_offsets == nullptr && tokens != batch)
        return fail(DATTN_ERR_INVALID_ARG,
                    "without token_offsets each sequence brings one token: tokens=%d, batch=%d", tokens,
                    batch);
    if (int st = check_stride(q_stride, static_cast<long long>(n_heads) * head_dim, 2, "q_stride")) return st;
    if (int st = check_stride(k_stride, static_cast<long long>(n_kv_heads) * head_dim, 2, "k_stride")) return st;
    if (int st = check_stride(v_stride, static_cast<long long>(n_kv_heads) * head_dim, 2, "v_stride")) return st;
    const long long q_row = static_cast<long long>(n_heads) * head_dim;
    if (int st = check_overlap(q_new, q_out, tokens, q_row * 2, q_stride * 2, q_row * 2, "q_new and q_out"))
        return st;
    if (int st = check_rope(rope, head_dim)) return st;
    dattn::DeviceFacts df;
    if (int st = dattn::device_facts(&df)) return st;
    dattn::Q8AppendArgs a{};
    rope_table(*rope, &a.rope);
    a.q = q_new;
    a.k = k_new;
    a.v = v_new;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.q_out = q_out;
    a.K = static_cast<unsigned char *>(K);
    a.V = static_cast<unsigned char *>(V);
    a.ks = K_scale;
    a.vs = V_scale;
    a.block_table = c.block_table;
    a.num_pages = c.num_pages;
    a.page_size = c.page_size;
    a.max_pages = c.max_pages;
    a.scale_rows = scale_rows_of(c, seq_len);
    a.scale_block = c.scale_block;
    a.div_page = dattn::fast_div_of(std::max(1, c.page_size));
    a.div_block = dattn::fast_div_of(c.scale_block);
    a.offsets = token_offsets;
    a.cur_pos = current_pos;
    a.err = df.err_word;
    a.tokens = tokens;
    a.B = batch;
    a.H = n_heads;
    a.kv_heads = n_kv_heads;
    a.D = head_dim;
    a.S = seq_len;
    const cudaError_t e = dattn::launch_append_q8(a, c.kv_type, df.sms, stream);
    return e == cudaSuccess ? DATTN_OK : fail_cuda(e, "8-bit append kernel launch");
}

}  // namespace

extern "C" {

int dattn_rope(const void *x, void *out, int dtype, long long tokens, int n_heads, int head_dim,
               long long x_stride, long long out_stride, const uint32_t *positions,
               const dattn_rope_params *rope, int gradient, dattn_stream_t stream) {
    return guarded([&]() -> int {
        if (int st = check_tensor(x, "x")) return st;
        if (int st = check_tensor(out, "out")) return st;
        if (int st = check_words(positions, "positions")) return st;
        if (dtype != DATTN_F16 && dtype != DATTN_BF16 && dtype != DATTN_F32)
            return fail(DATTN_ERR_INVALID_ARG, "dtype=%d is not a dattn_dtype", dtype);
        if (tokens <= 0 || n_heads <= 0 || head_dim <= 0)
            return fail(DATTN_ERR_INVALID_ARG,
                        "sizes must be positive (tokens=%lld n_heads=%d head_dim=%d)", tokens, n_heads,
                        head_dim);
        if (head_dim % 8 != 0 || head_dim > kMaxHeadDim)
            return fail(DATTN_ERR_UNSUPPORTED, "head_dim=%d: must be a multiple of 8 and <= %d",
                        head_dim, kMaxHeadDim);
        if (tokens > 0x7ffffc00LL || n_heads > (1 << 20))
            return fail(DATTN_ERR_UNSUPPORTED, "at most 2^31-1024 tokens of 2^20 heads");
        const long long row = static_cast<long long>(n_heads) * head_dim;
        const int elem = dtype == DATTN_F32 ? 4 : 2;
        if (int st = check_stride(x_stride, row, elem, "x_stride")) return st;
        if (int st = check_stride(out_stride, row, elem, "out_stride")) return st;
        if (int st = check_overlap(x, out, tokens, row * elem, x_stride * elem, out_stride * elem, "x and out"))
            return st;
        if (int st = check_rope(rope, head_dim)) return st;
        dattn::DeviceFacts df;
        if (int st = dattn::device_facts(&df)) return st;
        dattn::RopeArgs a{};
        rope_table(*rope, &a.rope);
        a.x = x;
        a.out = out;
        a.positions = positions;
        a.x_stride = x_stride;
        a.out_stride = out_stride;
        a.tokens = tokens;
        a.H = n_heads;
        a.D = head_dim;
        a.gradient = gradient ? 1 : 0;
        const cudaError_t e =
            dattn::launch_rope(a, dtype, df.sms, reinterpret_cast<cudaStream_t>(stream));
        return e == cudaSuccess ? DATTN_OK : fail_cuda(e, "rope kernel launch");
    });
}

int dattn_rope_append_q8(const void *q_new, const void *k_new, const void *v_new, void *q_out,
                         void *K_cache, void *V_cache, float *K_scale, float *V_scale, int kv_type,
                         int scale_block, int batch, int tokens, const int32_t *token_offsets,
                         long long q_stride, long long k_stride, long long v_stride, int n_heads,
                         int n_kv_heads, int head_dim, int seq_len, const dattn_rope_params *rope,
                         const uint32_t *current_pos, dattn_stream_t stream) {
    return guarded([&]() -> int {
        const Cache c{kv_type, scale_block};
        return append(q_new, k_new, v_new, q_out, K_cache, V_cache, K_scale, V_scale, batch, tokens,
                      token_offsets, q_stride, k_stride, v_stride, n_heads, n_kv_heads, head_dim,
                      seq_len, c, rope, current_pos, reinterpret_cast<cudaStream_t>(stream));
    });
}

int dattn_rope_append_paged_q8(const void *q_new, const void *k_new, const void *v_new, void *q_out,
                               void *K_pages, void *V_pages, float *K_scale, float *V_scale,
                               int kv_type, int scale_block, int batch, int tokens,
                               const int32_t *token_offsets, long long q_stride, long long k_stride,
                               long long v_stride, int n_heads, int n_kv_heads, int head_dim,
                               int page_size, int max_pages, long long num_pages,
                               const int32_t *block_table, const dattn_rope_params *rope,
                               const uint32_t *current_pos, dattn_stream_t stream) {
    return guarded([&]() -> int {
        Cache c{kv_type, scale_block};
        c.page_size = page_size;
        c.max_pages = max_pages;
        c.num_pages = num_pages;
        c.block_table = block_table;
        int seq_len = 0;
        if (int st = check_pages(c, &seq_len)) return st;
        return append(q_new, k_new, v_new, q_out, K_pages, V_pages, K_scale, V_scale, batch, tokens,
                      token_offsets, q_stride, k_stride, v_stride, n_heads, n_kv_heads, head_dim,
                      seq_len, c, rope, current_pos, reinterpret_cast<cudaStream_t>(stream));
    });
}

int dattn_decode_q8_plan(int batch, int n_heads, int n_kv_heads, int head_dim, int seq_len,
                         int num_partitions, dattn_plan *plan) {
    return guarded([&]() -> int {
        if (plan == nullptr) return fail(DATTN_ERR_INVALID_ARG, "plan is NULL");
        if (int st = check_sizes(batch, n_heads, n_kv_heads, head_dim, seq_len)) return st;
        Plan p;
        if (int st = make_plan(batch, n_heads, n_kv_heads, head_dim, seq_len, num_partitions, &p)) return st;
        plan->partitions = p.G;
        plan->heads_per_cta = p.HG * p.gq;
        plan->head_groups = p.NHG;
        plan->stage_positions = dattn::kQ8Tile;
        plan->stages = p.slots;
        plan->threads_per_cta = p.warps * 32;
        plan->smem_bytes = p.smem;
        plan->ctas_per_sm = p.ctas_per_sm;
        plan->sm_count = p.sms;
        plan->workspace_bytes = p.ws_bytes;
        plan->cluster_size = p.cluster;
        return DATTN_OK;
    });
}

int dattn_decode_q8_workspace_bytes(int batch, int n_heads, int n_kv_heads, int head_dim,
                                    int seq_len, int num_partitions, size_t *bytes) {
    return guarded([&]() -> int {
        if (bytes == nullptr) return fail(DATTN_ERR_INVALID_ARG, "bytes is NULL");
        if (int st = check_sizes(batch, n_heads, n_kv_heads, head_dim, seq_len)) return st;
        Plan p;
        if (int st = make_plan(batch, n_heads, n_kv_heads, head_dim, seq_len, num_partitions, &p)) return st;
        *bytes = p.ws_bytes;
        return DATTN_OK;
    });
}

int dattn_decode_q8(const void *Q, const void *K_cache, const void *V_cache, const float *K_scale,
                    const float *V_scale, void *out, int kv_type, int scale_block, int batch,
                    int n_heads, int n_kv_heads, int head_dim, int seq_len,
                    const uint32_t *current_pos, void *workspace, size_t workspace_bytes,
                    int num_partitions, dattn_stream_t stream) {
    return guarded([&]() -> int {
        const Cache c{kv_type, scale_block};
        return decode(Q, K_cache, V_cache, K_scale, V_scale, out, batch, n_heads, n_kv_heads, head_dim,
                      seq_len, c, current_pos, workspace, workspace_bytes, num_partitions,
                      reinterpret_cast<cudaStream_t>(stream));
    });
}

int dattn_decode_paged_q8(const void *Q, const void *K_pages, const void *V_pages,
                          const float *K_scale, const float *V_scale, void *out, int kv_type,
                          int scale_block, int batch, int n_heads, int n_kv_heads, int head_dim,
                          int page_size, int max_pages, long long num_pages,
                          const int32_t *block_table, const uint32_t *current_pos, void *workspace,
                          size_t workspace_bytes, int num_partitions, dattn_stream_t stream) {
    return guarded([&]() -> int {
        Cache c{kv_type, scale_block};
        c.page_size = page_size;
        c.max_pages = max_pages;
        c.num_pages = num_pages;
        c.block_table = block_table;
        int seq_len = 0;
        if (int st = check_pages(c, &seq_len)) return st;
        return decode(Q, K_pages, V_pages, K_scale, V_scale, out, batch, n_heads, n_kv_heads, head_dim,
                      seq_len, c, current_pos, workspace, workspace_bytes, num_partitions,
                      reinterpret_cast<cudaStream_t>(stream));
    });
}

}  // extern "C"
