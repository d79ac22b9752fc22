// dattn_internal.h -- kernel argument blocks and launchers shared between the
// C-ABI layer (dattn_api.cpp) and the CUDA translation units.  Host-side types.
#pragma once

#include <cuda.h>  // CUtensorMap (a plain struct; the driver library is not linked)
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace dattn {

// Threads of a decode CTA with `nwc` consumer warps: one more warp issues the
// bulk copies.  Eight consumer warps run two CTAs per SM, sixteen run one.
__host__ __device__ constexpr int decode_threads(int nwc) { return (nwc + 1) * 32; }
__host__ __device__ constexpr int decode_min_blocks(int nwc) { return nwc <= 8 ? 2 : 1; }

// Error codes a kernel records in the device error word.
constexpr unsigned kErrConsumerWait = 1u;
constexpr unsigned kErrProducerWait = 2u;
constexpr unsigned kErrDrainWait = 4u;
constexpr unsigned kErrSelftestWait = 8u;
constexpr unsigned kErrPageIndex = 16u;  // a block-table entry outside [0, num_pages)
constexpr unsigned kErrAppendPosition = 32u;  // an append position outside the cache

// Time limit of the pipeline waits in the library's kernels (attend_tiles_kernel.cuh: ten times that).
constexpr unsigned long long kWaitLimitNs = 1000000000ull;  // one second

// Arguments of the stream-K decode kernel.
//
// Units are (sequence b, head group g), u = b * head_groups + g, each holding
// the L_b live positions of heads [g*heads_per_cta, min(H, (g+1)*heads_per_cta)).
// Their positions, flattened unit after unit (W in total), are cut into
// `partitions` equal ranges, one per CTA (see streamk.h).  A CTA writes the
// f16 output of every unit it covers entirely and a partial softmax state for
// the others.
struct DecodeArgs {
    // Cluster mode (cluster > 0) with a head group smaller than H: tiled tensor
    // maps of K and V as [rows, H, D] (innermost D), box {D, HG, box_pos}: for a
    // dense cache the B*S positions and one full stage of a head group, for a
    // paged cache the num_pages*page_size rows of the pool and one page.
    CUtensorMap tmap_k, tmap_v;
    const void *Q;            // f16 [B,H,D]
    const void *K;            // f16 [B,S,H,D]
    const void *V;            // f16 [B,S,H,D]
    void *out;                // f16 [B,H,D]
    const uint32_t *cur_pos;  // [B]
    long long *ws_prefix;     // [B+1] live positions before each sequence (written by CTA 0)
    float *ws_acc;            // [(G+U), HG, D] unnormalised partial outputs
    float2 *ws_ml;            // [(G+U), HG]    partial (running max, log2 units; sum)
    unsigned *err;            // device error word
    // Paged cache (block_table != nullptr): K and V are pages
    // [num_pages, page_size, H, D] and position p of sequence b lives in page
    // block_table[b * max_pages + p / page_size], row p % page_size.  S is then
    // page_size * max_pages.
    const int *block_table;
    long long num_pages;
    int page_size, max_pages;
    int B, H, D, S;
    int heads_per_cta;  // HG
    int head_groups;    // NHG
    int phases;         // PHI: lane groups sharing one head interleave positions
    int stage_pos;      // P: positions per pipeline stage (a multiple of PHI)
    int stages;         // NST: pipeline depth
    int partitions;     // G: CTAs
    int active_warps;   // consumer warps holding at least one (head, phase) slot
    int merge_offset;   // byte offset of the phase-merge area in dynamic smem
    int bar_offset;     // byte offset of the mbarriers in dynamic smem
    float qscale;       // log2(e) / sqrt(D), applied to each dot product
    // Positions of its first stages each CTA prefetches into L2 before waiting
    // on the kernel before it (0 = none).
    int prefetch_positions;
    // Cluster mode: 0 = stream-K over the batch (above).  C > 0: the grid is
    // head_groups * B clusters of C CTAs; cluster u takes unit u = (b, g) whole,
    // CTA r of it the positions [r L_b / C, (r+1) L_b / C) of that unit, and
    // the C partial states are merged through distributed shared memory into
    // `out`.  No workspace and no second kernel.
    int cluster;
    int use_tmap;      // full stages (pages) of a head group are copied as tensor boxes
    int box_pos;       // positions of a tensor box: a stage (dense) or a page (paged)
    int prefetch_lanes;  // paged cache: lanes of warp 0 that read the prefetch window's pages (1..32)
    // Cluster mode: byte offset of this CTA's record [HG][D + 2] of its
    // partial state (m, l, acc) per head, read by the cluster's other CTAs.
    int rec_offset;
};

// Arguments of the combine kernel (log-sum-exp merge of the pieces of a unit).
struct CombineArgs {
    const float *ws_acc;
    const float2 *ws_ml;
    const long long *ws_prefix;
    const uint32_t *cur_pos;
    void *out;
    int B, H, D, S;
    int heads_per_cta;
    int head_groups;
    int partitions;
    int chunk;     // channels per combine CTA (a multiple of 8)
    int inflight;  // piece loads per thread per round: 2, 4 or 8
    int shift;     // the ranges are cut in units of 2^shift positions (0 or kQ8TileShift)
    int extra;     // units ahead of a unit's own that belong to no piece
};

// Compile-time shape of one decode-kernel instance.
struct DecodeVariant {
    int bdx;   // lanes per KV row: 1, 2, 4, 8 (chunks = 1) or 8, 16 (chunks = 2)
    int ch;    // 8-element chunks per lane: 1 or 2
    int kmax;  // (head, phase) slots per lane group: 1..2 (1 when ch = 2)
    int nwc;   // consumer warps: 8 or 16
};

// Launch the decode kernel.  smem = dynamic shared memory bytes.
cudaError_t launch_decode(const DecodeArgs &a, DecodeVariant v, int smem, cudaStream_t stream);
// Resident CTAs per SM for a variant at a given dynamic shared memory size.
cudaError_t decode_occupancy(DecodeVariant v, int smem, int *ctas_per_sm);
// Clusters of `cluster` CTAs of a variant that can be resident at once.
cudaError_t decode_max_clusters(DecodeVariant v, int smem, int cluster, bool paged, int *clusters);
// Raise the dynamic shared memory limit of every variant (once per device).
cudaError_t decode_configure_smem(int max_smem);
// Launch the combine kernel with programmatic dependent launch on `stream`.
cudaError_t launch_combine(const CombineArgs &a, cudaStream_t stream);
// Device error word of the current device.
cudaError_t device_error_word(unsigned **ptr);

// Record `message` as the calling thread's dattn_last_error() text and return
// `status` (for entry points defined outside dattn_api.cpp).
int set_last_error(int status, const char *message);

// Failure-detection self-test: one CTA waits (bounded) on an mbarrier that
// nothing arrives on and records kErrSelftestWait in `err` when the wait runs out.
cudaError_t launch_wait_timeout_selftest(unsigned *err, cudaStream_t stream);

// Arguments of the fused rotary-embedding + KV-append kernel (passed by value;
// the frequency table travels in the kernel's parameter space).
constexpr int kRopeMaxPairs = 256;  // rope_dims / 2 for head_dim up to 512
struct RopeAppendArgs {
    // theta_i / (2 pi) as a binary fraction in units of 2^-64, theta_i =
    // rope_base^(-2 i / rope_dims)
    unsigned long long turn_frac[kRopeMaxPairs];
    const void *q_new, *k_new, *v_new;  // f16 [B,H,D]
    void *q_out;                        // f16 [B,H,D] (may be q_new)
    void *K, *V;                        // cache: [B,S,H,D] or pages [num_pages,page_size,H,D]
    const int *block_table;             // nullptr: dense cache
    long long num_pages;
    int page_size, max_pages;
    const uint32_t *cur_pos;            // [B] position of the new token
    unsigned *err;
    int B, H, D, S;
    int rope_dims;
    int traditional;
    int heads_per_cta;
};
cudaError_t launch_rope_append(const RopeAppendArgs &a, cudaStream_t stream);

// Row softmax over the last dimension of a f32 [rows, cols] matrix.
cudaError_t launch_softmax(const float *x, float *out, long long rows, int cols,
                           unsigned *err, cudaStream_t stream);

// Page-faithful split calls.
cudaError_t launch_qk(const void *Q, const void *K, void *scores, int B, int H, int D, int S,
                      const uint32_t *cur_pos, cudaStream_t stream);
cudaError_t launch_pv(const void *scores, const void *V, void *out, int B, int H, int D,
                      int S, cudaStream_t stream);

// n / d by a multiplication, exact for 0 <= n < 2^31 (d >= 1): with l = ceil(log2 d),
// mul = ceil(2^(31+l) / d) <= 2^32 - 1 exceeds 2^(31+l) / d by less than 2^l / d,
// which n < 2^31 cannot carry into the next integer.
struct FastDiv {
    uint32_t mul;
    int shift;
};
inline FastDiv fast_div_of(int d) {
    int l = 0;
    while ((1LL << l) < d) ++l;
    const unsigned long long p = 1ull << (31 + l);
    return FastDiv{static_cast<uint32_t>((p + d - 1) / d), 31 + l};
}

#ifdef __CUDACC__
// n / d for 0 <= n < 2^31 by one multiplication.
__device__ __forceinline__ int fast_div(int n, FastDiv d) {
    return static_cast<int>((static_cast<unsigned long long>(static_cast<unsigned>(n)) * d.mul) >>
                            d.shift);
}
#endif

// 8-bit cache types (enum dattn_kv_type).
constexpr int kKvE4m3 = 1, kKvInt8 = 2;

constexpr int kQ8Tile = 16, kQ8TileShift = 4;  // positions per tile of the 8-bit decode

// Bytes of one ring slot of the 8-bit decode: 16 positions of K and V, DP bytes
// per row, and their 32 scales.
__host__ __device__ constexpr int q8_tile_bytes(int dp) { return 32 * dp + 128; }

// Warps of a decode CTA, CTAs of an SM and ring slots of a warp, by the row size and
// the 8-column tiles of query heads.
constexpr int kQ8Warps = 8;
__host__ __device__ constexpr int q8_ctas_per_sm(int dp, int nt) { return dp * nt <= 128 ? 2 : 1; }
__host__ __device__ constexpr int q8_slots(int dp, int nt) {
    return 212 * 1024 / (kQ8Warps * q8_ctas_per_sm(dp, nt)) / q8_tile_bytes(dp);
}

// Whether the eight columns hold each of gq query heads twice.
__host__ __device__ constexpr bool q8_pair(int gq) { return gq <= 4; }

// Arguments of the decode kernel over an 8-bit cache (decode_q8.cu).  A virtual
// head is a group of gq query heads of one key/value head (a key/value head has
// vheads_per_kv of them); units are (sequence, group of heads_per_cta virtual
// heads) and the flattened tiles of kQ8Tile positions are cut as DecodeArgs cuts
// positions.
struct Q8DecodeArgs {
    const void *Q;               // f16 [B,H,D]
    const unsigned char *K, *V;  // [B,S,Hk,D], or pages [num_pages,page_size,Hk,D]
    const float *ks, *vs;        // [B,ceil(S/n),Hk], or [num_pages,page_size/n,Hk]
    void *out;                   // f16 [B,H,D]
    const uint32_t *cur_pos;     // [B]
    long long *ws_prefix;        // as in DecodeArgs
    float *ws_acc;               // [(G+U), heads_per_cta * gq, D]
    float2 *ws_ml;               // [(G+U), heads_per_cta * gq]
    unsigned *err;
    const int *block_table;      // nullptr: dense cache
    long long num_pages;
    int page_size, max_pages;
    int scale_rows;              // scale blocks of a sequence (dense) or of a page
    FastDiv div_page, div_block, div_gq;
    int tile_in_page;            // no tile crosses a page (always, in a dense cache)
    int B, H, D, S;
    int kv_heads, gq, vheads, vheads_per_kv;
    int heads_per_cta;           // virtual heads of a CTA
    int head_groups;
    int phases;                  // warps that share a virtual head
    int partitions;              // CTAs
    int extra;                   // split plan: tiles that a unit counts beyond its own
    int cluster;                 // CTAs per unit, merged in shared memory; 0: the split plan
    float qscale;                // log2(e) / sqrt(D)
};
cudaError_t decode_q8_configure(int max_smem);
// Clusters of `cluster` CTAs that can be resident at once.
cudaError_t decode_q8_max_clusters(int dp, int nt, bool pair, int smem, int cluster, int *clusters);
cudaError_t launch_decode_q8(const Q8DecodeArgs &a, int dp, int nt, int kv, int smem,
                             cudaStream_t stream);

// The combine kernel's launch shape for G partitions over `units` units: the
// chunk of channels per CTA (at most ~8 pieces per thread of a 128-thread CTA,
// given the expected pieces per unit, (G + U) / U) and a thread's expected
// pieces in one round as loads in flight.
inline void combine_shape(int D, long long partitions, long long units, int *chunk, int *inflight) {
    const double pieces = static_cast<double>(partitions + units) / static_cast<double>(units);
    int p2 = 1;
    while (p2 < D) p2 <<= 1;
    int cw = p2 < 256 ? p2 : 256;
    while (cw > 8 && pieces * cw / 512.0 > 8.0) cw /= 2;
    const double per_thread = pieces / (128.0 / (cw / 4));
    *chunk = cw;
    *inflight = per_thread <= 2.0 ? 2 : (per_thread <= 4.0 ? 4 : 8);
}

// What entry points outside dattn_api.cpp need of the current device.
struct DeviceFacts {
    int sms;
    int max_smem_optin;
    unsigned *err_word;
};
int device_facts(DeviceFacts *out);  // a dattn_status, the message recorded

// Tensor map of [rows, H, D] 16-bit elements, rows `stride` elements apart, whose box, box_rows
// rows of box_heads heads and 64 channels, lands swizzled by 128 bytes; a dattn_status, the
// message recorded.
int encode_head_rows(CUtensorMap *map, const void *base, long long rows, long long stride, int H, int D,
                     int box_rows, int box_heads, int dtype);

// Rotation of pair i of a token at position p: by the angle p theta_i, cos and
// sin both multiplied by `magnitude`.  theta_i / (2 pi) travels as a binary
// fraction in units of 2^-64.
struct RopeTable {
    unsigned long long turn_frac[128];  // rope_dims / 2 entries, head_dim <= 256
    float magnitude;
    int rope_dims;
    int traditional;
};

// Rotation of x [tokens, H, D] (dtype f16, bf16 or f32) by explicit positions.
struct RopeArgs {
    RopeTable rope;
    const void *x;
    void *out;
    const uint32_t *positions;  // [tokens], or nullptr: from a ragged batch
    const int *offsets;         // [B+1], or nullptr: one token per sequence
    const uint32_t *cur_pos;    // [B] position of each sequence's last token
    int B;
    long long x_stride, out_stride;  // elements from token to token
    long long tokens;
    int H, D;
    int gradient;
};
constexpr int kDtypeF16 = 1, kDtypeBf16 = 2, kDtypeF32 = 3;
cudaError_t launch_rope(const RopeArgs &a, int dtype, int sms, cudaStream_t stream);

// Rotation of new tokens and their append to an 8-bit cache (append_q8.cu).
struct Q8AppendArgs {
    RopeTable rope;
    const void *q, *k, *v;                    // f16 [tokens, H or Hk, D]
    long long q_stride, k_stride, v_stride;   // elements from token to token
    void *q_out;                              // f16 [tokens, H, D]
    unsigned char *K, *V;
    float *ks, *vs;
    const int *block_table;                   // nullptr: dense cache
    long long num_pages;
    int page_size, max_pages;
    int scale_rows;
    int scale_block;
    FastDiv div_page, div_block;
    const int *offsets;                       // [B+1] or nullptr: one token per sequence
    const uint32_t *cur_pos;                  // [B] position of each sequence's last new token
    unsigned *err;
    long long tokens;
    int B, H, kv_heads, D, S;
};
cudaError_t launch_append_q8(const Q8AppendArgs &a, int kv, int sms, cudaStream_t stream);

// Arguments of attention over a 16-bit cache (attend_*.cu).  Positions 0 .. S-1 of a
// sequence; the `shared` first ones are the same for every sequence, in a tensor of their
// own (Kp, Vp; the cache then begins at position `own_base` = shared) or through the
// first sequence's pages (own_base = 0).
struct AttendArgs {
    const void *Q;               // [tokens,H,D], tokens q_stride elements apart
    const void *K, *V;           // [B,S - own_base,Hk,D], or pages [num_pages,page_size,Hk,D]
    const void *Kp, *Vp;         // [shared,Hk,D] or nullptr
    void *out;                   // [tokens,H,D]
    const int *block_table;      // nullptr: dense cache
    long long num_pages;
    int page_size, max_pages;
    FastDiv div_page;
    const int *offsets;          // [B+1], or nullptr: one token per sequence
    const uint32_t *cur_pos;     // [B] cache row of each sequence's last token
    unsigned *err;
    long long q_stride;
    int tokens, B, H, Hk, D, S;
    int group;                   // query heads of a key/value head
    int shared, own_base;
    int window;                  // positions that a token sees up to its own; 0: all
    int sinks;                   // first positions that stay visible
    float qscale;                // log2(e) / sqrt(D)
};
// One token per sequence (attend_token.cu): warps of a CTA, ring slots of a warp at most
// (a slot holds K and V of a tile), CTAs of an SM by the row size.  A warp's ring holds no
// more slots than it has tiles, and the states of its query heads at the end.
constexpr int kTokenTile = 16;  // positions
constexpr int kTokenWarps = 4, kTokenSlots = 3;
__host__ __device__ constexpr int token_ctas_per_sm(int dp) { return 256 / dp; }
__host__ __device__ constexpr int token_ring_bytes(int dp, int slots, int gq) {
    const int ring = slots * 2 * kTokenTile * dp * 2, states = (gq * (dp + 4) * 4 + 127) / 128 * 128;
    return ring > states ? ring : states;
}
__host__ __device__ constexpr int token_smem(int dp, int slots, int gq) {
    return kTokenWarps * token_ring_bytes(dp, slots, gq);
}
// A virtual head is a group of gq query heads of one key/value head (a key/value head has
// vheads_per_kv of them); units are (sequence, heads_per_cta virtual heads).
struct TokenArgs {
    float *ws_acc;      // [B,H,chunks,D] states of the chunks of units of several
    float2 *ws_ml;      // [B,H,chunks]   (running max, log2 units; sum)
    int gq, vheads, vheads_per_kv;
    FastDiv div_gq;
    int heads_per_cta;
    int head_groups;
    int phases;         // warps that share a virtual head
    int chunks;         // CTAs of a unit
    int chunk_tiles;    // tiles of a chunk (not of a cluster's: equal runs of what is seen)
    int cluster;        // the chunks of a unit are a cluster and merge in shared memory
    int ring_bytes;     // a warp's ring
    int own_only;       // the shared positions are left out and every chunk leaves its state
};
cudaError_t attend_token_configure(int max_smem);
cudaError_t attend_token_max_clusters(int dp, int nt, bool pair, int smem, int cluster, int *clusters);
cudaError_t launch_attend_token(const AttendArgs &a, const TokenArgs &w, int dtype, int dp, int smem,
                                cudaStream_t stream);

// Many tokens at a time (attend_tiles.cu): query rows are a sequence's tokens times the
// query heads of a key/value head, cut into items of tile_rows(dp), each over the
// key tiles that one of its tokens sees.
__host__ __device__ constexpr int tile_stacks(int dp) { return dp <= 128 ? 2 : 1; }  // of 128 rows
__host__ __device__ constexpr int tile_rows(int dp) { return 128 * tile_stacks(dp); }
__host__ __device__ constexpr int tile_keys(int dp) { return dp <= 128 ? 128 : 64; }
constexpr int kTileMinUnits = 2;  // key tiles (and what an item adds) of a CTA, of which there are
                                  // fewer for less work
// Items of one key/value head (the same for each).
struct TileItem {
    int b, token;     // sequence, first row's token
    int head, rows;   // first row's query head within the group, rows
    int p0;           // first token's position
    int lo, first;    // positions that some row sees: n - first from `lo` on, then [0, first)
    int n;
};
// An item of key/value head kvh that CTAs first .. last share; first -1: none.
struct TileCut {
    int kvh, item, first, last;
};
// What the planning kernel leaves ahead of the items.
struct TilePlan {
    long long total;  // key tiles of the items of one key/value head, and what an item adds
    int items;
    int ctas;         // CTAs that share them
};
struct TileArgs {
    TilePlan *plan;          // nullptr: rows of all sequences over the shared positions
    TileItem *items;
    long long *before;       // [items + 1] tiles (and what an item adds) ahead of each item
    int *seq_items;          // [B + 1] items ahead of each sequence
    int max_items;
    TileCut *cuts;           // [ctas] what the beginning of a CTA's share is the first to cut
    float *acc;              // [2 ctas, tile_rows, D] states of pieces of items
    float2 *ml;              // [2 ctas, tile_rows]
    float *whole_acc;        // shared: [B,H,D] states of items that one CTA held
    float2 *whole_ml;        // shared: [B,H]
    FastDiv div_group;
    int ctas;                // CTAs at most
    int bound_ends;          // shared: a token may lie inside the shared positions
    int out_32;              // rows of out begin on 32-byte boundaries
    int align;               // an item's `lo` is a multiple (a power of two)
};
// Tensor maps of K and V (of the shared positions' own tensors where there are such) as
// [rows, Hk, D], a box of box_rows rows of one head and 64 channels; box_rows 0: none.  Of Q
// as [tokens, H, D], a box of q_tokens tokens of a group's heads, 128 rows; q_tokens 0: none.
struct TileMaps {
    CUtensorMap k, v, q;
    int box_rows, q_tokens;
};
cudaError_t attend_tiles_configure(int max_smem);
cudaError_t launch_attend_tiles(const AttendArgs &a, const TileArgs &t, const TileMaps &m, int dtype, int dp,
                                cudaStream_t stream);

// Merge of the chunks' states into `out`, with those of the shared positions where `t` is given.
cudaError_t launch_attend_merge(const AttendArgs &a, const TokenArgs &w, const TileArgs *t, int dtype, int dp,
                                cudaStream_t stream);

}  // namespace dattn
