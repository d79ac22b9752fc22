// append_q8_kernel.cuh -- rotate the new tokens of a ragged batch and append their keys
// and values to a KV cache held in 8 bits (e4m3 or int8) with one fp32 scale
// for each block of `scale_block` positions and key/value head.
//
// Sequence b brings tokens offsets[b] .. offsets[b+1]-1 (n_b of them; one when
// offsets is null), the last of them at position current_pos[b].  q and k are
// rotated at their positions (rope.cu's map) in fp32; q is rounded to f16 into
// q_out, k and v go to the cache.  For a block that receives rows:
//   amax  = largest finite |x| of the new rows of the head
//   need  = smallest power of two s >= 2^-32 with amax <= QMAX s   (448 or 127)
//   scale = need, or max(old scale, need) where the sequence has earlier rows in
//           the block; those rows are requantised when the scale grows
//   row   = nearest 8-bit value to x / scale, ties to even, saturating
// A power of two keeps all of e4m3's relative precision, makes x / scale exact
// and a requantisation of e4m3 exact down to its subnormals; for int8 it costs
// up to one of its seven bits.  Infinities saturate; NaN stays NaN in e4m3 and
// becomes 0 in int8.
//
// What bounds it: 2 bytes read per new element and one written for k and v, two
// and two for q; a step of one token is bound by latency, a prompt by instructions: a
// rotated element is converted and turned twice, for the maximum and for the store,
// and needs a cosine.  A thread holds one row's item of 16 channels of kHeads
// heads, so a (row, pair)'s cosine is made once, in registers, for all of them, and the
// maximum of a (block, head) pair is joined by warp reductions and one exchange in
// shared memory: no second launch, no atomics.  Each input is read once unless a block
// has more rows than its warps.  A block is the work of a set of warps, as many as its
// rows and heads fill (at most a CTA's eight); the sets of a CTA go their own ways.  The
// grid cannot know the ragged lengths, so it is cut by tokens: a set looks through a
// window of the flattened tokens for those that open a block (the first of a sequence,
// or a position at a multiple of scale_block) and takes their blocks.  K and V go to
// different CTAs.  q is rotated by further CTAs of the same launch (rope_tiles.cuh),
// which stream while the others compute.
//
// Measured (graph replay): 8192 tokens of 32 query and 8 key/value heads of 128, 185 MB,
// 36.4 us, 5.1 TB/s (k and v alone 22, q alone 29.5); one token each of 256 sequences of
// 40 heads, 13 MB, 5.9 us; one token of one sequence 2.6 us.  The instances that read
// element by element (a rotated part that four do not divide) spill 220 bytes.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "dattn_internal.h"
#include "ptx.cuh"
#include "rope_tiles.cuh"

namespace dattn {
namespace {

constexpr int kThreads = kRopeThreads, kWarps = kThreads / 32;
constexpr int kMinExp = -32;  // scales are at least 2^-32

// Heads of a thread.  8192 tokens of 32 query and 8 key/value heads: 36.4 us with four;
// 42.4 with two; 45.6 with four and three CTAs per SM, whose 80 registers spill.
constexpr int kHeads = 4;

struct AppendGrid {
    int items_k, items_v;  // per row
    int lanes;             // lanes of a row: a power of two, items_k and items_v at least
    int rows;              // rows of a block side by side in a segment of lanes
    int groups_per_warp;   // segments of a warp, kHeads heads each
    int warps;             // warps that share the rows of their heads
    int set;               // warps that work on a block together: a power of two
    int heads_per_set;
    int head_chunks;
    int window;            // tokens a set looks through
    unsigned jobs;         // windows x head_chunks
    unsigned kv_ctas, q_ctas;
};

// Smallest power of two s >= 2^kMinExp with amax <= QMAX s, from the bits of
// amax: QMAX is 1.75 2^8 (e4m3) or 1.984375 2^6 (int8).
template <int KV>
__device__ __forceinline__ float need_scale(uint32_t amax_bits) {
    constexpr uint32_t kTop = KV == kKvE4m3 ? 0x600000u : 0x7e0000u;
    constexpr int kExp = KV == kKvE4m3 ? 8 : 6;
    int e = static_cast<int>(amax_bits >> 23) - 127 - kExp;
    if ((amax_bits & 0x7fffffu) > kTop) ++e;
    if (amax_bits == 0 || e < kMinExp) e = kMinExp;
    return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// x / scale is x times the reciprocal, exactly, where the scale is a power of two; its
// reciprocal is found in the exponent (for 2^-126 .. 2^126).
struct Divider {
    float inv;
    bool exact;
};
__device__ __forceinline__ Divider divider(float scale) {
    const uint32_t bits = __float_as_uint(scale);
    return Divider{__uint_as_float((254u << 23) - bits),
                   (bits & 0x807fffffu) == 0 && bits - (1u << 23) < (253u << 23)};
}

template <int KV>
__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
    uint32_t r;
    if constexpr (KV == kKvE4m3) {
        asm("{\n\t.reg .b16 l, h;\n\t"
            "cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
            "mov.b32 %0, {l, h};\n\t}"
            : "=r"(r)
            : "f"(a), "f"(b), "f"(c), "f"(d));
    } else {
        auto q = [](float x) {
            const int i = __float2int_rn(fminf(fmaxf(x, -127.f), 127.f));
            return static_cast<uint32_t>(x != x ? 0 : i) & 255u;
        };
        r = q(a) | q(b) << 8 | q(c) << 16 | q(d) << 24;
    }
    return r;
}

template <int KV>
__device__ __forceinline__ float value_of(unsigned char x) {
    if constexpr (KV == kKvE4m3) {
        uint32_t h;
        asm("{\n\t.reg .b16 b;\n\tcvt.u16.u32 b, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, b;\n\t}"
            : "=r"(h)
            : "r"(static_cast<uint32_t>(x)));
        return __half2float(__ushort_as_half(static_cast<unsigned short>(h)));
    } else {
        return static_cast<float>(static_cast<signed char>(x));
    }
}

// Put `before` earlier rows of a (block, head) on a scale `f` times finer to coarser:
// value * f, rounded again.  Lane `item` of `lanes` and row `r0`, r0 + hop, ... are this
// thread's; sixteen neighbouring channels at a time, whatever the pairs are.
template <int KV>
__device__ __forceinline__ void requantise(unsigned char *block0, size_t row_elems, int D, int before,
                                           float f, int item, int lanes, int r0, int hop) {
    for (int r = r0; r < before; r += hop) {
        for (int c = item * 16; c < D; c += lanes * 16) {
            uint4 *v = reinterpret_cast<uint4 *>(block0 + r * row_elems + c);
            uint4 x = *v;
            uint32_t *w = reinterpret_cast<uint32_t *>(&x);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                w[e] = pack4<KV>(value_of<KV>(w[e] & 255u) * f, value_of<KV>(w[e] >> 8 & 255u) * f,
                                 value_of<KV>(w[e] >> 16 & 255u) * f, value_of<KV>(w[e] >> 24) * f);
            *v = x;
        }
    }
}

// Largest finite magnitude of an item (0 if it has none).
template <int E>
__device__ __forceinline__ float item_max(const float *y) {
    float m = 0.f;  // fmaxf passes over NaN
#pragma unroll
    for (int e = 0; e < E; ++e) m = fmaxf(m, fabsf(y[e]));
    if (m == INFINITY) {  // among infinities only the finite ones count
        m = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) m = fabsf(y[e]) < INFINITY ? fmaxf(m, fabsf(y[e])) : m;
    }
    return m;
}

// y / scale in 8 bits into the item's channels of row o.
template <int KV, int N>
__device__ __forceinline__ void store_item(const Item<__half, N> &it, unsigned char *o, float *y,
                                           float scale, const Divider &div) {
    constexpr int E = 2 * kPairs<N>;
    if (div.exact) {
#pragma unroll
        for (int e = 0; e < E; ++e) y[e] *= div.inv;
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e) y[e] = y[e] / scale;
    }
    uint32_t w[E / 4];
#pragma unroll
    for (int e = 0; e < E / 4; ++e) w[e] = pack4<KV>(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
    unsigned char *const u = o + it.first, *const v = u + it.hop;  // the two runs
    if constexpr (N == 16) {
        *reinterpret_cast<uint2 *>(u) = make_uint2(w[0], w[1]);
        *reinterpret_cast<uint2 *>(v) = make_uint2(w[2], w[3]);
    } else if constexpr (N == 8) {
        *reinterpret_cast<uint32_t *>(u) = w[0];
        *reinterpret_cast<uint32_t *>(v) = w[1];
    } else if constexpr (N == 4) {
        *reinterpret_cast<unsigned short *>(u) = static_cast<unsigned short>(w[0]);
        *reinterpret_cast<unsigned short *>(v) = static_cast<unsigned short>(w[0] >> 16);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (k < it.n0) u[k] = static_cast<unsigned char>(w[k >> 2] >> (8 * (k & 3)));
            if (k < it.n1) v[k] = static_cast<unsigned char>(w[2 + (k >> 2)] >> (8 * (k & 3)));
        }
    }
}

// The place of position `pos` of sequence b: the first row of its scale block and the
// block's row of scales.  False where the page is not in the pool.
__device__ __forceinline__ bool block_place(const Q8AppendArgs &a, int b, int pos, int blk, int before,
                                            long long *row0, long long *srow) {
    if (a.block_table == nullptr) {
        *row0 = static_cast<long long>(b) * a.S + pos - before;
        *srow = static_cast<long long>(b) * a.scale_rows + blk;
        return true;
    }
    const int pi = fast_div(pos, a.div_page);
    const long long page = __ldg(a.block_table + static_cast<long long>(b) * a.max_pages + pi);
    *row0 = page * a.page_size + (pos - pi * a.page_size - before);
    *srow = page * a.scale_rows + blk - pi * a.scale_rows;
    return page >= 0 && page < a.num_pages;
}

// The block that a set works on: its first new token, position and row, how many rows are
// new and how many the sequence has in it from before, and its row of scales.
struct Unit {
    long long token, row0, srow;
    int pos, n, before;
};

// The next block that a token of [tok, end) opens (by one warp; lane 0 reports tokens that
// cannot be appended).  tok is left behind the block; false: none is left.
__device__ __forceinline__ bool next_unit(const Q8AppendArgs &a, long long used, long long &tok,
                                          long long end, int lane, Unit &u) {
    while (tok < end) {
        const int b = find_sequence(a.offsets, a.B, tok, lane);
        const long long s0 = __ldg(a.offsets + b), s1 = __ldg(a.offsets + b + 1);  // its tokens
        const long long stop = min(s1, used);
        if (stop <= tok) {  // offsets that do not ascend: no token of a sequence
            ++tok;
            continue;
        }
        const long long p = static_cast<long long>(__ldg(a.cur_pos + b)) - (s1 - 1 - tok);
        if (p < 0 || p >= a.S) {
            if (lane == 0) atomicOr(a.err, kErrAppendPosition);
            tok = p < 0 ? min(tok - p, stop) : stop;
            continue;
        }
        u.token = tok;
        u.pos = static_cast<int>(p);
        const int blk = fast_div(u.pos, a.div_block);
        u.before = u.pos - blk * a.scale_block;
        u.n = static_cast<int>(min(min(static_cast<long long>(a.scale_block - u.before), stop - tok),
                                   static_cast<long long>(a.S - u.pos)));
        tok += u.n;
        if (u.before != 0 && u.token != s0) continue;  // inside a block that an earlier token opens
        if (block_place(a, b, u.pos, blk, u.before, &u.row0, &u.srow)) return true;
        if (lane == 0) atomicOr(a.err, kErrPageIndex);
    }
    return false;
}

struct AppendShared {
    unsigned long long frac[128];           // turn fraction of each slot, an item's side by side
    Unit unit[kWarps];                      // of each set
    int more[kWarps];
    float mx[kHeads * 32 * kWarps];         // of each head of a set, by each of its warps
    float now[kHeads * 32 * kWarps], old[kHeads * 32 * kWarps];  // its scale, and before
};

// ONE: the CTA is one set.
template <bool ONE>
__device__ __forceinline__ void sync_set(int set, int warps) {
    if constexpr (ONE) __syncthreads();
    else if (warps == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(set + 1), "r"(warps * 32) : "memory");
}

template <int KV, int N, bool IS_V, bool ONE>
__device__ __forceinline__ void append_kv(const Q8AppendArgs &a, const AppendGrid &gr, unsigned cta,
                                          AppendShared &sh) {
    const int warps = ONE ? kWarps : gr.set;  // of the set
    const int set = ONE ? 0 : (threadIdx.x >> 5) / warps;
    const unsigned job = ONE ? cta : cta * (kWarps / warps) + set;
    if (job >= gr.jobs) return;
    const unsigned window = job / static_cast<unsigned>(gr.head_chunks);
    const int chunk = static_cast<int>(job - window * gr.head_chunks);
    const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & (warps - 1);
    const int thread = warp * 32 + lane, threads = warps * 32;
    const int s_off = set * warps * (kHeads * 32);
    float *const s_mx = sh.mx + s_off, *const s_now = sh.now + s_off, *const s_old = sh.old + s_off;
    const int D = a.D, rd = IS_V ? 0 : a.rope.rope_dims;
    const int seg = gr.lanes * gr.rows;  // lanes of a group of heads: a power of two
    const int item = lane & (gr.lanes - 1), rs = (lane & (seg - 1)) / gr.lanes;
    const int wr = warp & (gr.warps - 1);  // a power of two
    const int local = (warp / gr.warps * gr.groups_per_warp + lane / seg) * kHeads;
    const int first_head = chunk * gr.heads_per_set, head0 = first_head + local;
    const int nh = min(kHeads, a.kv_heads - head0);  // 0 or less: no heads
    const bool mine = item < (IS_V ? gr.items_v : gr.items_k);
    const int myrow = wr * gr.rows + rs, span = gr.rows * gr.warps;  // rows of a pass
    const size_t row_elems = static_cast<size_t>(a.kv_heads) * D;
    const Item<__half, N> it(item, rd, D, a.rope.traditional != 0);
    const __half *const src = reinterpret_cast<const __half *>(IS_V ? a.v : a.k) + static_cast<long long>(head0) * D;
    const long long stride = IS_V ? a.v_stride : a.k_stride;
    const float mag = a.rope.magnitude;

    const long long used = used_tokens(a.offsets, a.B, a.tokens);
    long long tok = static_cast<long long>(window) * gr.window;
    const long long end = min(tok + gr.window, used);
    for (;;) {
        if (warp == 0) {
            Unit u;
            const bool more = next_unit(a, used, tok, end, lane, u);
            if (lane == 0) {
                sh.more[set] = more;
                if (more) sh.unit[set] = u;
            }
        }
        sync_set<ONE>(set, warps);
        if (!sh.more[set]) return;
        const Unit u = sh.unit[set];
        const int n = u.n, before = u.before;

        // this thread's row of a pass: the inputs of its heads, and its cosines
        ItemData<__half, N> d[kHeads];
        float2 cs[kPairs<N>];
        auto load_row = [&](int r0) {
            const int row = r0 + myrow;
            if (!mine || row >= n) return;
            const __half *x = src + (u.token + row) * stride;
#pragma unroll
            for (int h = 0; h < kHeads; ++h)
                if (h < nh) it.load(x + h * D, d[h]);
            if (!IS_V && it.rot) {
#pragma unroll
                for (int e = 0; e < kPairs<N>; ++e) {
                    const float2 c =
                        turn_cos_sin(static_cast<uint32_t>(u.pos + row), sh.frac[item * kPairs<N> + e]);
                    cs[e] = make_float2(c.x * mag, c.y * mag);
                }
            }
        };

        // ---- pass 1: largest finite magnitude of each head's rotated rows ----
        float mx[kHeads];
#pragma unroll
        for (int h = 0; h < kHeads; ++h) mx[h] = 0.f;
        for (int r0 = 0; r0 < n; r0 += span) {
            load_row(r0);
            if (!mine || r0 + myrow >= n) continue;
#pragma unroll
            for (int h = 0; h < kHeads; ++h) {
                if (h >= nh) break;
                float y[2 * kPairs<N>];
                it.values(d[h], cs, 1, y);
                mx[h] = fmaxf(mx[h], item_max<2 * kPairs<N>>(y));
            }
        }
#pragma unroll
        for (int h = 0; h < kHeads; ++h) {
            if (seg == 32) {  // not negative: they order as their bits do
                mx[h] = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mx[h])));
            } else {
                for (int o = seg / 2; o > 0; o >>= 1)
                    mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], o));
            }
        }
        if ((lane & (seg - 1)) == 0) {
#pragma unroll
            for (int h = 0; h < kHeads; ++h) s_mx[(local + h) * gr.warps + wr] = mx[h];
        }
        sync_set<ONE>(set, warps);
        // ---- each head's scale, by one thread ----
        for (int i = thread; i < min(gr.heads_per_set, a.kv_heads - first_head); i += threads) {
            float *const scale = (IS_V ? a.vs : a.ks) + u.srow * a.kv_heads + first_head + i;
            const float old = before > 0 ? *scale : 0.f;
            float m = 0.f;
            for (int w = 0; w < gr.warps; ++w) m = fmaxf(m, s_mx[i * gr.warps + w]);
            const float need = need_scale<KV>(__float_as_uint(m));
            const float now = before > 0 ? fmaxf(old, need) : need;
            s_now[i] = now;
            s_old[i] = before > 0 ? old : now;
            *scale = now;
        }
        sync_set<ONE>(set, warps);
        // ---- earlier rows on the new scale; pass 2: the new rows ----
        unsigned char *const block0 = (IS_V ? a.V : a.K) + static_cast<size_t>(u.row0) * row_elems +
                                      static_cast<size_t>(head0) * D;
        if (before > 0) {
            for (int h = 0; h < nh; ++h) {
                const float now = s_now[local + h], old = s_old[local + h];
                if (now != old)
                    requantise<KV>(block0 + h * D, row_elems, D, before, old / now, item, gr.lanes, myrow, span);
            }
        }
        for (int r0 = 0; r0 < n; r0 += span) {
            if (n > span) load_row(r0);  // more rows than the warps hold: read them again
            if (!mine || r0 + myrow >= n) continue;
            unsigned char *o = block0 + static_cast<size_t>(before + r0 + myrow) * row_elems;
#pragma unroll
            for (int h = 0; h < kHeads; ++h) {
                if (h >= nh) break;
                const float now = s_now[local + h];
                float y[2 * kPairs<N>];
                it.values(d[h], cs, 1, y);
                store_item<KV, N>(it, o + h * D, y, now, divider(now));
            }
        }
    }
}

// CTAs [0, q_ctas) rotate q and stay while K's blocks and then V's, which take less time,
// go through the other slots (K and V alternating left every other SM with K only).  HP:
// heads of a thread that rotates q.
template <int KV, int N, bool FIXED, int HP>
__global__ void __launch_bounds__(kThreads, 2)
    append_q8_kernel(const __grid_constant__ Q8AppendArgs a, const __grid_constant__ RopeArgs q,
                     const AppendGrid gr, const RopeGrid qgr) {
    extern __shared__ __align__(16) unsigned char smem[];
    union Shared {
        AppendShared kv;
        uint32_t pos[2][kRopeThreads];
    };
    __shared__ Shared sh;
    pdl_launch_dependents();
    const unsigned q_ctas = gr.q_ctas;
    if (blockIdx.x < q_ctas) {
        pdl_wait_primary();
        rope_tiles<__half, N, FIXED, HP>(q, a.rope, qgr, blockIdx.x, q_ctas, smem, sh.pos);
        return;
    }
    const int ir = rope_items(a.rope.rope_dims, N);
    for (int i = threadIdx.x; i < kPairs<N> * ir; i += kThreads) {
        const int j = i / kPairs<N>;
        const int pair = Item<__half, N>::pair_of(i - j * kPairs<N>, j, a.rope.rope_dims, a.rope.traditional != 0);
        sh.kv.frac[i] = a.rope.turn_frac[min(pair, a.rope.rope_dims / 2 - 1)];
    }
    __syncthreads();
    pdl_wait_primary();
    const unsigned i = blockIdx.x - q_ctas, half = gr.kv_ctas / 2;
    if (gr.set == kWarps) {
        if (i < half) append_kv<KV, N, false, true>(a, gr, i, sh.kv);
        else append_kv<KV, N, true, true>(a, gr, i - half, sh.kv);
    } else {
        if (i < half) append_kv<KV, N, false, false>(a, gr, i, sh.kv);
        else append_kv<KV, N, true, false>(a, gr, i - half, sh.kv);
    }
}

struct Instance {
    const void *fn;
    int ring_bytes;
};
template <int KV, int N, bool FIXED, int HP>
Instance instance() {
    return Instance{reinterpret_cast<const void *>(append_q8_kernel<KV, N, FIXED, HP>), kRingBytes<__half, N, HP>};
}
template <int KV, int N>
Instance instance_of(int hp) {
    return hp == 4 ? instance<KV, N, false, 4>() : hp == 2 ? instance<KV, N, false, 2>() : instance<KV, N, false, 1>();
}
template <int KV>
Instance instance_of(int width, bool fixed, int hp) {
    if (width == 1) return instance<KV, 1, false, 1>();
    if (width == 4) return instance_of<KV, 4>(hp);
    if (width == 8) return instance_of<KV, 8>(hp);
    if (fixed) return hp == 2 ? instance<KV, 16, true, 2>() : instance<KV, 16, true, 1>();
    return hp == 2 ? instance<KV, 16, false, 2>() : instance<KV, 16, false, 1>();
}

// One token per sequence (a decode step), bound by latency: a CTA takes some of the
// heads of q, k and v of a token, one item per thread, the lanes of a head side by side
// in a warp.  The inputs' addresses need no position, so they are under way while the
// position, the page and the old scales are looked up one after another.  (Three items
// per thread, a CTA for all heads: 7.4 against 7.0 us for 256 tokens of 40 heads.)
struct TokenGrid {
    int items_k, items_v;  // per row of q and k; of v
    int lanes;             // lanes of a head, a power of two
    int chunks;            // CTAs of a token
};

template <int KV, int N>
__global__ void __launch_bounds__(kThreads, 3)
    append_token_kernel(const __grid_constant__ Q8AppendArgs a, const TokenGrid gr) {
    __shared__ float2 table[128];  // rope_dims / 2 entries at most, in slots of eight
    pdl_launch_dependents();
    pdl_wait_primary();
    const unsigned ub = blockIdx.x / static_cast<unsigned>(gr.chunks);
    const int b = static_cast<int>(ub), chunk = static_cast<int>(blockIdx.x - ub * gr.chunks);
    const int D = a.D, ir = rope_items(a.rope.rope_dims, N);
    const int item = threadIdx.x & (gr.lanes - 1);
    const uint32_t p = __ldg(a.cur_pos + b);

    // heads are numbered q, k, v one after another
    int head = chunk * (kThreads / gr.lanes) + threadIdx.x / gr.lanes;
    const bool is_q = head < a.H, is_v = head >= a.H + a.kv_heads;
    const int items = is_v ? gr.items_v : gr.items_k;
    const bool mine = head < a.H + 2 * a.kv_heads && item < items;
    if (!is_q) head -= is_v ? a.H + a.kv_heads : a.H;
    const Item<__half, N> it(item, is_v ? 0 : a.rope.rope_dims, D, a.rope.traditional != 0);
    ItemData<__half, N> d;
    if (mine) {
        const __half *src = reinterpret_cast<const __half *>(is_q ? a.q : is_v ? a.v : a.k);
        const long long stride = is_q ? a.q_stride : is_v ? a.v_stride : a.k_stride;
        it.load(src + b * stride + static_cast<long long>(head) * D, d);
    }
    // The rotation is defined at every position; an append outside the cache is reported.
    RopeFiller<__half, N>(ir, a.rope, false).fill(table, 1, [&](int) { return p; });
    bool ok = p < static_cast<uint32_t>(a.S);
    long long row0 = 0, srow = 0;
    int before = 0;
    if (ok) {
        const int pos = static_cast<int>(p), blk = fast_div(pos, a.div_block);
        before = pos - blk * a.scale_block;
        ok = block_place(a, b, pos, blk, before, &row0, &srow);
        if (!ok && threadIdx.x == 0) atomicOr(a.err, kErrPageIndex);
    } else if (threadIdx.x == 0) {
        atomicOr(a.err, kErrAppendPosition);
    }
    float *const scale = (is_v ? a.vs : a.ks) + srow * a.kv_heads + head;
    const float old = ok && before > 0 && mine && !is_q ? *scale : 0.f;
    __syncthreads();
    float y[2 * kPairs<N>], mx = 0.f;
    if (mine) {
        it.values(d, table + item, ir, y);
        if (!is_q) mx = item_max<2 * kPairs<N>>(y);
    }
    for (int o = gr.lanes / 2; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if (!mine) return;
    if (is_q) {
        round_item(y, d);
        it.store(reinterpret_cast<__half *>(a.q_out) + (static_cast<long long>(b) * a.H + head) * D, d);
        return;
    }
    if (!ok) return;
    const float need = need_scale<KV>(__float_as_uint(mx));
    const float now = before > 0 ? fmaxf(old, need) : need;
    const size_t row_elems = static_cast<size_t>(a.kv_heads) * D;
    unsigned char *const block0 =
        (is_v ? a.V : a.K) + static_cast<size_t>(row0) * row_elems + static_cast<size_t>(head) * D;
    if (before > 0 && now != old)
        requantise<KV>(block0, row_elems, D, before, old / now, item, items, 0, 1);
    if (item == 0) *scale = now;
    store_item<KV, N>(it, block0 + before * row_elems, y, now, divider(now));
}

template <int KV>
const void *token_kernel_of(int width) {
    if (width == 16) return reinterpret_cast<const void *>(append_token_kernel<KV, 16>);
    if (width == 8) return reinterpret_cast<const void *>(append_token_kernel<KV, 8>);
    if (width == 4) return reinterpret_cast<const void *>(append_token_kernel<KV, 4>);
    return reinterpret_cast<const void *>(append_token_kernel<KV, 1>);
}

}  // namespace
}  // namespace dattn
