// decode_q8_kernel.cuh -- single-query attention over a KV cache held in 8 bits (e4m3
// or int8), with one fp32 scale for each block of `scale_block` positions and
// key/value head, and query heads sharing key/value heads in groups.
//
// For sequence b, query head h of key/value head e and L_b = min(cp_b, S-1)+1:
//   s_p = (Q[b,h,:] . Kq[b,p,e,:]) ks[b,p/n,e] / sqrt(D)              p < L_b
//   out = sum_p 2^(s_p log2e) vs[b,p/n,e] Vq[b,p,e,:] / sum_p 2^(s_p log2e)
// in one pass with a running maximum.  The scale of V enters the exponent:
// with t_p = s_p log2e + log2 vs the accumulator holds sum 2^(t_p - M) Vq and
// the sum 2^(t_p - M) / vs, M running over max t_p, so no weight exceeds a
// known bound whatever the scales are, and states of different positions merge
// as in any log-sum-exp (combine.cu merges them unchanged).
//
// What bounds it: the cache is read once, 2 D bytes per position and key/value
// head for 4 G D flops (G query heads to a key/value head).  8-bit elements
// have to be widened and multiplied at ~24 elements per clock and SM to keep up
// with HBM, which scalar FMAs do not reach for G above 2.  The products
// therefore run on the tensor cores with the cache as the 16-row operand
// (mma.sync m16n8k16, f16 in, fp32 accumulate): S^T = K Q^T over 16 positions
// and out^T = V^T P^T over 16 channels, with the query heads in the 8 columns.
// A tcgen05 instruction wants 128 (or 64) rows and both operands through shared
// memory; a decode has at most 16 query heads to share a fetched key, so
// the widened cache would have to be written back to shared memory first, which
// costs more than the products.  8-bit values are exact in f16, Q is f16 already
// and the products accumulate in fp32.  P is fp32 and enters as the sum of two f16,
// the nearest one and what that leaves: a relative 2^-22, where one alone is 2^-11 and
// left the outputs of 64 ragged sequences 2.4e-4 (rms, relative) from the definition; now
// 2.1e-4, what their own rounding to f16 makes.  With at most four query heads the second
// takes the columns that they leave free, at no further product; with more it takes a
// product of its own per 16 channels.  One and two f16, us: 64 ragged sequences of 32 heads
// 90.5, 90.8; 32 on 8 heads, 4096 positions 8.4, 8.7; 64 on 8 heads, 32768 positions 18.2,
// 18.3; 32 on 2 heads (16 columns), 65536 positions 14.6, 15.6.
//
// Fragments straight from 16-byte loads: the sum over channels (and over
// positions) may run in any order, so the channel (position) that a fragment
// slot stands for is chosen to make each lane's elements contiguous in the
// cache row, for K one 16-byte chunk per four k-steps, for V two neighbouring
// positions' words whose bytes are paired with prmt.  P^T is the S^T
// accumulator in its two f16, transposed with movmatrix.
//
// Work split: tiles of 16 positions.  Split plan: as in the f16 decode
// (streamk.h), the live tiles of all (sequence, head group) units, flattened, are
// cut into equal ranges, one per CTA, and combine.cu merges the units that span
// several.  Cluster plan: a thread-block cluster takes a unit whole, its CTAs equal
// runs of its tiles, and they merge through distributed shared memory in the same
// launch; clusters of several CTAs for batches small enough to be bound by latency,
// of one, in as many waves as it takes, for many short sequences.  In a CTA each
// warp owns one head (heads_per_cta of them) and one phase: tiles go to the
// phases in turn.  Every warp streams its own tiles through a private ring in
// shared memory with 16-byte cp.async, so the main loop has no CTA-wide barrier;
// rows past the live length are zero filled and never read from memory.
//
// Measured (graph replay, inputs larger than L2 in all): one sequence of 131072
// positions and 32 heads of 128, 1 GiB, 158 us, 6.8 TB/s, as fast as a copy; 64 ragged
// ones of up to 2048, 538 MB, 90.8 us, 5.9 TB/s, where the units' beginnings, ends and
// merge show; one of 4096 positions, 8 key/value heads, 8.4 MB, 8.7 us, bound by latency
// (launch, position, page, first tiles, exchange).
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "dattn_internal.h"
#include "ptx.cuh"
#include "streamk.h"

namespace dattn {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kTile = kQ8Tile;    // positions per tile
constexpr int kMaxCluster = 16;  // CTAs per cluster (8 is the portable limit)

// The running maximum M is kept kHeadroom (log2) below the largest exponent at
// the time it was set, and moved only when an exponent exceeds M + kTrigger:
// weights then lie below 2^15 (f16 holds up to 65504), and their two f16 keep 22 bits
// down to 2^-13 of the largest, further down 2^-35 of it.
constexpr float kHeadroom = 10.f, kTrigger = 15.f;
// log2 of the smallest scale of V that takes part (a scale of 0 stands for
// values of zero; it is read as 2^-60, which leaves them below any f16).  The sum over
// such positions holds weights of up to 2^15 times 2^60: below 2^107 for as many as there
// can be.
constexpr float kMinLogScale = -60.f;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two neighbouring 8-bit values (the low or high half of a word) as f16x2.
// e4m3: one conversion, exact (NaN stays NaN).  int8: the byte with its sign
// bit flipped is v + 128; put under the exponent of 1024 it reads 1152 + v.
template <int KV>
__device__ __forceinline__ void widen(uint32_t w, uint32_t &lo, uint32_t &hi) {
    if constexpr (KV == kKvE4m3) {
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
            : "=r"(lo), "=r"(hi)
            : "r"(w));
    } else {
        const uint32_t u = w ^ 0x80808080u;
        const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140);
        const uint32_t b = __byte_perm(u, 0x64646464u, 0x4342);
        const __half2 bias = __half2half2(__ushort_as_half(0x6480));  // 1152
        const __half2 x = __hsub2(*reinterpret_cast<const __half2 *>(&a), bias);
        const __half2 y = __hsub2(*reinterpret_cast<const __half2 *>(&b), bias);
        lo = *reinterpret_cast<const uint32_t *>(&x);
        hi = *reinterpret_cast<const uint32_t *>(&y);
    }
}

__device__ __forceinline__ void mma16816(float *c, uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 8x8 transpose of 16-bit elements across the warp.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
    return v;
}
__device__ __forceinline__ float lds32(uint32_t addr) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr));
    return v;
}

__device__ __forceinline__ int live_len(const uint32_t *cp, long long b, int S) {
    const uint32_t c = __ldg(cp + b);
    return c >= static_cast<uint32_t>(S - 1) ? S : static_cast<int>(c) + 1;
}

__device__ __forceinline__ int live_tiles(const uint32_t *cp, long long b, int S) {
    return (live_len(cp, b, S) + kTile - 1) / kTile;
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
// What pack2's rounding left of the two.
__device__ __forceinline__ uint32_t rest2(float lo, float hi, uint32_t packed) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&packed));
    return pack2(lo - f.x, hi - f.y);
}

// Shared-memory row of MMA row r (0..7) within a group of 8 tile rows, chosen
// so that both fragment patterns below are free of bank conflicts under the
// swizzle: rows of 128 bytes and more need rows 2i, 2i+1 to differ in bit 2 and
// the even (odd) rows to differ in bits 1-2; rows of 64 bytes need rows 2i, 2i+1
// to differ in bit 0.
template <int DP>
__device__ __forceinline__ int tile_row(int r) {
    if constexpr (DP >= 128) return (r & 1) ? ((r + 4) & 7) : r;
    const int i = r >> 1;               // pairs (0,3) (1,2) (4,7) (5,6)
    const int first = (i & 1) + (i >> 1) * 4;
    return (r & 1) ? first ^ 3 : first;
}

// Byte offset of 16-byte chunk c of row r in a tile of rows of DP bytes.
template <int DP>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
    if constexpr (DP >= 128) return r * DP + (((c & ~7) | ((c ^ r) & 7)) << 4);
    return r * DP + ((c ^ ((r >> 1) & 3)) << 4);
}

// DP: head_dim rounded up to 64, 128 or 256 (channels above head_dim are zero
// filled).  NT: 8-column tiles of query heads.  NS: ring slots.
// PAIR (NT = 1): at most four query heads, each in columns h and h + 4.
template <int DP, int NT, bool PAIR, int KV, int NS, bool CLUSTER>
__global__ void __launch_bounds__(kQ8Warps * 32, q8_ctas_per_sm(DP, NT)) decode_q8_kernel(const Q8DecodeArgs a) {
    constexpr int NJ = DP / 64;           // 64-channel spans of a row
    constexpr int NM = DP / 16;           // 16-channel tiles of the output
    constexpr int NW = kQ8Warps, kThreads = NW * 32;
    constexpr int kTileBytes = q8_tile_bytes(DP);
    constexpr int CPR = DP / 16;          // 16-byte chunks per row
    constexpr int RPI = 32 / CPR;         // rows per warp-wide copy
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ long long s_warp[NW];
    __shared__ long long s_b0, s_base0;
    __shared__ float2 s_ml[NW][NT * 8];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, t = lane & 3;
    const int D = a.D;
    const long long nhg = a.head_groups;

    if constexpr (CLUSTER) cluster_arrive_relaxed();
    pdl_wait_primary();

    // ---- this CTA's range [x, x1) of the flattened tiles ----
    // b: the sequence that x lies in, base: its first flattened tile, T: its tiles of
    // one head group, L: its live positions.  In the split plan each unit counts
    // `extra` tiles more than it has, ahead of its own: what beginning a unit costs
    // a CTA, so that CTAs with several short units get fewer tiles.  Divisions are 32-bit ones (the grid and
    // a sequence's tiles are), except where the batch holds 2^32 tiles or more.
    long long x, x1, b = 0, base = 0;
    const unsigned c = blockIdx.x;
    int grp0 = 0;  // cluster plan: the CTA's group of heads
    if constexpr (CLUSTER) {
        const unsigned u = c / static_cast<unsigned>(a.cluster), r = c - u * a.cluster;
        const unsigned ub = u / static_cast<unsigned>(a.head_groups);
        b = ub;
        grp0 = static_cast<int>(u - ub * a.head_groups);
        const unsigned T = live_tiles(a.cur_pos, b, a.S);
        x = static_cast<unsigned long long>(r) * T / static_cast<unsigned>(a.cluster);
        x1 = static_cast<unsigned long long>(r + 1) * T / static_cast<unsigned>(a.cluster);
    } else {
        const unsigned G = a.partitions;
        auto cut = [&](long long W) {
            if (W < 0x100000000LL) {
                const unsigned wq = static_cast<unsigned>(W) / G, wr = static_cast<unsigned>(W) - wq * G;
                x = range_begin_split(c, wq, wr, G);
                x1 = range_begin_split(c + 1, wq, wr, G);
            } else {
                x = range_begin(c, W, G);
                x1 = range_begin(c + 1, W, G);
            }
        };
        const bool keep = c == 0 && a.ws_prefix != nullptr;
        long long total = 0;  // tiles of the batch, per head group
        if (a.B == 1) {
            total = live_tiles(a.cur_pos, 0, a.S) + a.extra;
            cut(nhg * total);
        } else {
            // Rounds of one sequence per thread: an inclusive scan of their tiles.  A
            // batch of one round needs no pass before it for the total.
            const bool one_round = a.B <= kThreads;
            if (!one_round) {
                long long sum = 0;
                for (int i = tid; i < a.B; i += kThreads) sum += live_tiles(a.cur_pos, i, a.S) + a.extra;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
                if (lane == 0) s_warp[warp] = sum;
                __syncthreads();
                for (int w = 0; w < NW; ++w) total += s_warp[w];
                cut(nhg * total);
            }
            long long carry = 0;
            for (int i0 = 0; i0 < a.B; i0 += kThreads) {
                const int i = i0 + tid;
                const int T = i < a.B ? live_tiles(a.cur_pos, i, a.S) + a.extra : 0;
                long long pre = T;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const long long y = __shfl_up_sync(kFull, pre, o);
                    if (lane >= o) pre += y;
                }
                if (!one_round) __syncthreads();  // s_warp of the round before has been read
                if (lane == 31) s_warp[warp] = pre;
                __syncthreads();
                long long round = 0;
                for (int w = 0; w < NW; ++w) {
                    if (w < warp) pre += s_warp[w];
                    round += s_warp[w];
                }
                if (one_round) cut(nhg * round);
                pre += carry;  // tiles up to and including sequence i
                if (i < a.B) {
                    if (keep) {
                        if (i == 0) a.ws_prefix[0] = 0;
                        a.ws_prefix[i + 1] = pre;
                    }
                    if (x >= nhg * (pre - T) && x < nhg * pre) {
                        s_b0 = i;
                        s_base0 = nhg * (pre - T);
                    }
                }
                carry += round;
                if (!keep && x < nhg * carry) break;  // the same in every thread
            }
            __syncthreads();
            b = s_b0;
            base = s_base0;
        }
        if (x >= x1) return;
    }

    const int HG = a.heads_per_cta, PH = a.phases;
    const int hl = warp % HG, ph = warp / HG;
    const uint32_t ring = smem_addr(smem) + warp * (NS * kTileBytes);
    const unsigned row_bytes = static_cast<unsigned>(a.kv_heads) * D;
    const int r0 = tile_row<DP>(g);                               // K: rows r0 and r0 + 8
    const int v0 = tile_row<DP>(2 * t), v1 = tile_row<DP>(2 * t + 1);  // V: and 8 rows on
    const int crow = lane / CPR, cchunk = lane % CPR;             // copies: this lane's row and chunk
    const bool in_head = cchunk * 16 < D;
    int L = live_len(a.cur_pos, b, a.S);
    int T = (L + kTile - 1) / kTile;

    do {
        // ---- the next piece: tiles [off, off + len) of unit (b, grp); a CTA of a
        // cluster has one piece, perhaps of no tiles ----
        int grp, off, len;
        if constexpr (CLUSTER) {
            grp = grp0;
            off = static_cast<int>(x);
            len = static_cast<int>(x1 - x);
        } else {
            while (x >= base + nhg * (T + a.extra)) {
                base += nhg * (T + a.extra);
                ++b;
                L = live_len(a.cur_pos, b, a.S);
                T = (L + kTile - 1) / kTile;
            }
            const unsigned rel = static_cast<unsigned>(x - base), span = T + a.extra;
            grp = static_cast<int>(rel / span);
            const int from = static_cast<int>(rel - static_cast<unsigned>(grp) * span);
            const int take = static_cast<int>(x1 - x < static_cast<long long>(span) - from ? x1 - x : span - from);
            off = max(0, from - a.extra);
            len = from + take - a.extra - off;
            x += take;
            if (len <= 0) continue;  // none of the unit's own tiles
        }
        [[maybe_unused]] const long long u = b * nhg + grp;

        const int vh = grp * HG + hl;  // virtual head: gq query heads of one key/value head
        const bool active = ph < PH && vh < a.vheads;
        const int kvh = active ? vh / a.vheads_per_kv : 0;
        const int ntiles = active && ph < len ? (len - ph + PH - 1) / PH : 0;
        const int first = (off + ph) * kTile, step = PH * kTile;
        // this lane's chunk of cache row 0 and the bytes between rows; lanes past
        // head_dim write zeros and read nothing
        const size_t col = in_head ? static_cast<size_t>(kvh) * D + cchunk * 16 : 0;
        const unsigned rb = in_head ? row_bytes : 0u;
        const unsigned char *const k0 = a.K + col, *const v0p = a.V + col;
        const float *const scales = (lane < 16 ? a.ks : a.vs) + kvh;

        // Copy tile i of this warp into its ring slot; `page` is the table entry of
        // the tile where tiles do not cross pages.
        auto issue = [&](int i, int slot, int page) {
            const int p0 = first + i * step;
            const uint32_t dst = ring + slot * kTileBytes;
            const int pos = p0 + (lane & 15);
            const bool live = pos < L;
            if (a.tile_in_page) {
                // rows p0 .. p0 + 15 are neighbours
                unsigned row = static_cast<unsigned>(b) * a.S + p0;
                unsigned srow = static_cast<unsigned>(b) * a.scale_rows;
                int in = pos;
                if (a.block_table != nullptr) {
                    const int at = p0 - fast_div(p0, a.div_page) * a.page_size;
                    if (page < 0 || page >= a.num_pages) {
                        atomicOr(a.err, kErrPageIndex);
                        page = 0;
                    }
                    row = static_cast<unsigned>(page) * a.page_size + at;
                    srow = static_cast<unsigned>(page) * a.scale_rows;
                    in = at + (lane & 15);
                }
                srow = live ? srow + fast_div(in, a.div_block) : 0u;
                cp_async4(dst + 32 * DP + lane * 4,
                          scales + static_cast<unsigned long long>(srow) * a.kv_heads, live ? 4 : 0);
                const unsigned long long at0 = static_cast<unsigned long long>(row + crow) * rb;
                const unsigned char *k = k0 + at0, *v = v0p + at0;
                if (p0 + kTile <= L) {
                    const int bytes = in_head ? 16 : 0;
#pragma unroll
                    for (int j = 0; j < kTile / RPI; ++j) {
                        const uint32_t o = dst + chunk_at<DP>(j * RPI + crow, cchunk);
                        cp_async16(o, k + static_cast<unsigned long long>(rb) * (j * RPI), bytes);
                        cp_async16(o + 16 * DP, v + static_cast<unsigned long long>(rb) * (j * RPI), bytes);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < kTile / RPI; ++j) {
                        const bool there = in_head && p0 + j * RPI + crow < L;
                        const size_t hop = there ? static_cast<size_t>(rb) * (j * RPI) + at0 : 0;
                        const uint32_t o = dst + chunk_at<DP>(j * RPI + crow, cchunk);
                        cp_async16(o, k0 + hop, there ? 16 : 0);
                        cp_async16(o + 16 * DP, v0p + hop, there ? 16 : 0);
                    }
                }
                return;
            }
            // Pages of any size: lanes l and l + 16 find the row of tile position l
            // through the block table and hand it to the lanes that copy it.
            unsigned row = 0, srow = 0;
            if (live) {
                const int pi = fast_div(pos, a.div_page);
                const int in = pos - pi * a.page_size;
                int pg = __ldg(a.block_table + b * a.max_pages + pi);
                if (pg < 0 || pg >= a.num_pages) {
                    atomicOr(a.err, kErrPageIndex);
                    pg = 0;
                }
                row = static_cast<unsigned>(pg) * a.page_size + in;
                srow = static_cast<unsigned>(pg) * a.scale_rows + fast_div(in, a.div_block);
            }
            cp_async4(dst + 32 * DP + lane * 4,
                      scales + static_cast<unsigned long long>(srow) * a.kv_heads, live ? 4 : 0);
#pragma unroll
            for (int j = 0; j < kTile / RPI; ++j) {
                const int r = j * RPI + crow;
                const unsigned rr = __shfl_sync(kFull, row, r);
                const bool there = in_head && p0 + r < L;
                const unsigned long long at = there ? static_cast<unsigned long long>(rr) * rb : 0;
                cp_async16(dst + chunk_at<DP>(r, cchunk), k0 + at, there ? 16 : 0);
                cp_async16(dst + 16 * DP + chunk_at<DP>(r, cchunk), v0p + at, there ? 16 : 0);
            }
        };
        // The table entry of tile i (one tile ahead of its copies, so that the copies
        // do not wait for it).
        const bool lookup = a.tile_in_page && a.block_table != nullptr;
        auto page_of = [&](int i) {
            return lookup && i < ntiles
                       ? __ldg(a.block_table + b * a.max_pages + fast_div(first + i * step, a.div_page))
                       : 0;
        };

        // Q^T fragments: column n = query head (modulo 4 where two columns share one),
        // channels as in K's chunks.
        uint32_t qf[NT][NJ][4][2];
        if (ntiles > 0) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int h = PAIR ? g & 3 : n * 8 + g;
                const __half *qrow = reinterpret_cast<const __half *>(a.Q) +
                                     (b * a.H + static_cast<long long>(vh) * a.gq + h) * D;
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    const int ch = 16 * (t + 4 * j);
                    uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
                    if (h < a.gq && ch < D) {
                        lo = __ldg(reinterpret_cast<const uint4 *>(qrow + ch));
                        hi = __ldg(reinterpret_cast<const uint4 *>(qrow + ch + 8));
                    }
                    qf[n][j][0][0] = lo.x, qf[n][j][0][1] = lo.y;
                    qf[n][j][1][0] = lo.z, qf[n][j][1][1] = lo.w;
                    qf[n][j][2][0] = hi.x, qf[n][j][2][1] = hi.y;
                    qf[n][j][3][0] = hi.z, qf[n][j][3][1] = hi.w;
                }
            }
        }

        float acc[NT][NM][4];
        float M[NT][2], l[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int m = 0; m < NM; ++m)
                acc[n][m][0] = acc[n][m][1] = acc[n][m][2] = acc[n][m][3] = 0.f;
            M[n][0] = M[n][1] = -INFINITY;
            l[n][0] = l[n][1] = 0.f;
        }

        // Once its last tile is under way, a warp asks for the first tiles of the piece
        // after this one to be brought into L2 (a hint), lane l the rows of tile
        // position l & 15, of K or of V.
        auto prefetch_next = [&]() {
            if (x >= x1 || !active) return;
            long long nb = b, nbase = base;
            int nL = L;
            int span = (nL + kTile - 1) / kTile + a.extra;
            if (x >= nbase + nhg * span) {
                nbase += nhg * span;
                ++nb;
                nL = live_len(a.cur_pos, nb, a.S);
                span = (nL + kTile - 1) / kTile + a.extra;
            }
            const unsigned nrel = static_cast<unsigned>(x - nbase);
            const int ngrp = static_cast<int>(nrel / static_cast<unsigned>(span));
            const int nvh = ngrp * HG + hl;
            if (nvh >= a.vheads) return;
            const unsigned char *cache = (lane < 16 ? a.K : a.V) + static_cast<size_t>(nvh / a.vheads_per_kv) * D;
            for (int i = 0; i < NS - 1; ++i) {
                const int pos = (ph + i * PH) * kTile + (lane & 15);
                if (pos >= nL) break;
                unsigned row = static_cast<unsigned>(nb) * a.S + pos;
                if (a.block_table != nullptr) {
                    const int pi = fast_div(pos, a.div_page);
                    const int pg = __ldg(a.block_table + nb * a.max_pages + pi);
                    if (pg < 0 || pg >= a.num_pages) break;
                    row = static_cast<unsigned>(pg) * a.page_size + (pos - pi * a.page_size);
                }
                const unsigned char *at = cache + static_cast<unsigned long long>(row) * row_bytes;
                for (int o = 0; o < D; o += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(at + o));
            }
        };

        // Step j issues the copies of tile j and computes on tile j - (NS - 1): one
        // place for each, so that a call of few tiles fetches little code.
        int page = page_of(0), fill = 0, slot = 0;
        for (int j = 0; j < ntiles + NS - 1; ++j) {
            const int i = j - (NS - 1);
            if (i >= 0) {
                cp_async_wait<NS - 2>();
                __syncwarp();  // every lane's copies of tile i are visible, tile i - 1 is read
            }
            if (j < ntiles) {
                const int now = page;
                page = page_of(j + 1);
                issue(j, fill, now);
                fill = fill + 1 == NS ? 0 : fill + 1;
            }
            cp_async_commit();
            if (!CLUSTER && j == ntiles) prefetch_next();
            if (i < 0) continue;
            const uint32_t kt = ring + slot * kTileBytes, vt = kt + 16 * DP, sc = kt + 32 * DP;
            slot = slot + 1 == NS ? 0 : slot + 1;

            // S^T over the tile: rows (positions) g and g + 8, columns 2t, 2t + 1
            float s[NT][2][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[n][0][e] = s[n][1][e] = 0.f;
#pragma unroll
            for (int jj = 0; jj < NJ; ++jj) {
                const uint4 ka = lds128(kt + chunk_at<DP>(r0, t + 4 * jj));
                const uint4 kb = lds128(kt + 8 * DP + chunk_at<DP>(r0, t + 4 * jj));
                const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t a0, a1, a2, a3;
                    widen<KV>(wa[q], a0, a2);
                    widen<KV>(wb[q], a1, a3);
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        mma16816(s[n][q & 1], a0, a1, a2, a3, qf[n][jj][q][0], qf[n][jj][q][1]);
                }
            }

            // exponents t = s log2e / sqrt(D) + log2 vs
            const float ks0 = lds32(sc + r0 * 4) * a.qscale, ks1 = lds32(sc + 32 + r0 * 4) * a.qscale;
            const float lv0 = fmaxf(lg2(lds32(sc + 64 + r0 * 4)), kMinLogScale);
            const float lv1 = fmaxf(lg2(lds32(sc + 96 + r0 * 4)), kMinLogScale);
            const float iv0 = ex2(-lv0), iv1 = ex2(-lv1);
            const int p0 = first + i * step;
            const bool in0 = p0 + r0 < L, in1 = p0 + 8 + r0 < L;
            bool grow = false;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float z = s[n][0][e] + s[n][1][e];
                    const float y = e < 2 ? fmaf(z, ks0, lv0) : fmaf(z, ks1, lv1);
                    s[n][0][e] = (e < 2 ? in0 : in1) ? y : -INFINITY;
                    grow |= s[n][0][e] > M[n][e & 1] + kTrigger;
                }
            }
            if (__any_sync(kFull, grow)) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float mx = fmaxf(s[n][0][e], s[n][0][e + 2]);
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
                        const float nm = fmaxf(M[n][e], mx - kHeadroom);
                        const float f = M[n][e] == -INFINITY ? 0.f : ex2(M[n][e] - nm);
                        M[n][e] = nm;
                        l[n][e] *= f;
#pragma unroll
                        for (int m = 0; m < NM; ++m) {
                            acc[n][m][e] *= f;
                            acc[n][m][e + 2] *= f;
                        }
                    }
            }
            // the weights as f16 and, columns 4 to 7 of a pair or pr, what that leaves
            uint32_t pf[NT][2];
            [[maybe_unused]] uint32_t pr[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float m0 = M[n][0] == -INFINITY ? 0.f : M[n][0];
                const float m1 = M[n][1] == -INFINITY ? 0.f : M[n][1];
                const float e0 = ex2(s[n][0][0] - m0), e1 = ex2(s[n][0][1] - m1);
                const float e2 = ex2(s[n][0][2] - m0), e3 = ex2(s[n][0][3] - m1);
                l[n][0] = fmaf(e0, iv0, fmaf(e2, iv1, l[n][0]));
                l[n][1] = fmaf(e1, iv0, fmaf(e3, iv1, l[n][1]));
                const uint32_t h0 = pack2(e0, e1), h1 = pack2(e2, e3);
                const uint32_t left0 = rest2(e0, e1, h0), left1 = rest2(e2, e3, h1);
                if constexpr (PAIR) {
                    pf[n][0] = transpose8x8(t & 2 ? left0 : h0);
                    pf[n][1] = transpose8x8(t & 2 ? left1 : h1);
                } else {
                    pf[n][0] = transpose8x8(h0);
                    pf[n][1] = transpose8x8(h1);
                    pr[n][0] = transpose8x8(left0);
                    pr[n][1] = transpose8x8(left1);
                }
            }

            // out^T += V^T P^T: positions v0, v1 and 8 rows on; channels by lane group
#pragma unroll
            for (int hf = 0; hf < (DP == 256 ? 2 : 1); ++hf) {
                uint32_t w[4][4];
                if constexpr (DP == 64) {
                    const int rr[4] = {v0, v1, v0 + 8, v1 + 8};
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint2 y = lds64(vt + chunk_at<DP>(rr[q], g >> 1) + (g & 1) * 8);
                        w[q][0] = y.x, w[q][1] = y.y;
                    }
                } else {
                    const int cv = g + 8 * hf;
                    const uint4 y0 = lds128(vt + chunk_at<DP>(v0, cv));
                    const uint4 y1 = lds128(vt + chunk_at<DP>(v1, cv));
                    const uint4 y2 = lds128(vt + 8 * DP + chunk_at<DP>(v0, cv));
                    const uint4 y3 = lds128(vt + 8 * DP + chunk_at<DP>(v1, cv));
                    w[0][0] = y0.x, w[0][1] = y0.y, w[0][2] = y0.z, w[0][3] = y0.w;
                    w[1][0] = y1.x, w[1][1] = y1.y, w[1][2] = y1.z, w[1][3] = y1.w;
                    w[2][0] = y2.x, w[2][1] = y2.y, w[2][2] = y2.z, w[2][3] = y2.w;
                    w[3][0] = y3.x, w[3][1] = y3.y, w[3][2] = y3.z, w[3][3] = y3.w;
                }
#pragma unroll
                for (int q = 0; q < (DP == 64 ? 2 : 4); ++q) {
                    // bytes of positions v0, v1 paired per channel
                    const uint32_t x0 = __byte_perm(w[0][q], w[1][q], 0x5140);
                    const uint32_t x2 = __byte_perm(w[0][q], w[1][q], 0x7362);
                    const uint32_t z0 = __byte_perm(w[2][q], w[3][q], 0x5140);
                    const uint32_t z2 = __byte_perm(w[2][q], w[3][q], 0x7362);
                    uint32_t a0, a1, a2, a3;
                    const int m = hf * 8 + q * 2;
                    widen<KV>(x0, a0, a1);
                    widen<KV>(z0, a2, a3);
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        mma16816(acc[n][m], a0, a1, a2, a3, pf[n][0], pf[n][1]);
                    if constexpr (!PAIR) {
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            mma16816(acc[n][m], a0, a1, a2, a3, pr[n][0], pr[n][1]);
                    }
                    widen<KV>(x2, a0, a1);
                    widen<KV>(z2, a2, a3);
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        mma16816(acc[n][m + 1], a0, a1, a2, a3, pf[n][0], pf[n][1]);
                    if constexpr (!PAIR) {
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            mma16816(acc[n][m + 1], a0, a1, a2, a3, pr[n][0], pr[n][1]);
                    }
                }
            }
        }

        // the kernel after this one may begin launching during the last epilogue
        if (CLUSTER || x >= x1) pdl_launch_dependents();

        // ---- the piece's state: sum over the lanes, merge the phases, store ----
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) l[n][e] += __shfl_xor_sync(kFull, l[n][e], o);

        const bool whole = len == T;
        // Each warp leaves (M, l) and its accumulators in its idle ring, a row of
        // kRow floats per query head: channel pair (m, g) at 2 (8 m + g), which makes
        // both the stores here and the loads below free of bank conflicts.
        constexpr int kRow = DP + 4;
        float *const my_rows = reinterpret_cast<float *>(smem + warp * (NS * kTileBytes));
        __syncwarp();  // the last tile has been read
        if constexpr (PAIR) {
            // The two columns of a query head together: lanes t and t ^ 2 hold the same two
            // heads and finish one each.
            const bool second = t & 2;
            const int h = 2 * (t & 1) + (second ? 1 : 0);
            float *const row = my_rows + h * kRow + 2 * g;
            const bool mine = active && h < a.gq;
            if (mine && g == 0)
                s_ml[warp][h] = second ? make_float2(M[0][1], l[0][1]) : make_float2(M[0][0], l[0][0]);
#pragma unroll
            for (int m = 0; m < NM; ++m) {
                const float *c = acc[0][m];
                const float y0 = __shfl_xor_sync(kFull, second ? c[0] : c[1], 2);
                const float y1 = __shfl_xor_sync(kFull, second ? c[2] : c[3], 2);
                if (mine)
                    *reinterpret_cast<float2 *>(row + 16 * m) =
                        make_float2((second ? c[1] : c[0]) + y0, (second ? c[3] : c[2]) + y1);
            }
        } else if (active) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int h = n * 8 + 2 * t + e;
                    if (h >= a.gq) continue;
                    if (g == 0) s_ml[warp][h] = make_float2(M[n][e], l[n][e]);
#pragma unroll
                    for (int m = 0; m < NM; ++m)
                        *reinterpret_cast<float2 *>(my_rows + h * kRow + 2 * (8 * m + g)) =
                            make_float2(acc[n][m][e], acc[n][m][e + 2]);
                }
        }
        __syncthreads();
        // Merge the phases: a thread takes a (query head, channel pair) of the unit.
        const int heads = min(HG, a.vheads - grp * HG) * a.gq;
        const long long out_row = b * a.H + static_cast<long long>(grp) * HG * a.gq;
        [[maybe_unused]] const uint32_t rec = smem_addr(smem) + NW * NS * kTileBytes;
        [[maybe_unused]] int share = 0, rank = 0;
        if (CLUSTER && a.cluster > 1) {
            // each CTA of the cluster finishes an equal share of the outputs
            share = (heads * (DP / 2) + a.cluster - 1) / a.cluster;
            rank = static_cast<int>(cluster_ctarank());
        }
        // every CTA of the cluster has started: its shared memory may be written
        if constexpr (CLUSTER) cluster_wait();
        for (int i = tid; i < heads * (DP / 2); i += kThreads) {
            const int hq = i / (DP / 2), pair = i % (DP / 2);  // DP is a power of two
            const int w0 = fast_div(hq, a.div_gq);
            const int h = hq - w0 * a.gq;
            const int m = pair >> 3, pg = pair & 7;
            const int ch = DP == 64 ? 8 * pg + 2 * m : (m >> 3) * 128 + 16 * pg + 2 * (m & 7);
            float top = -INFINITY, lsum = 0.f, y0 = 0.f, y1 = 0.f;
#pragma unroll 4
            for (int p = 0; p < PH; ++p) top = fmaxf(top, s_ml[p * HG + w0][h].x);
#pragma unroll 4
            for (int p = 0; p < PH; ++p) {
                const int w = p * HG + w0;
                const float2 ml = s_ml[w][h];
                const float2 y = *reinterpret_cast<const float2 *>(
                    smem + w * (NS * kTileBytes) + (h * kRow + 2 * pair) * 4);
                const float f = ml.x == -INFINITY ? 0.f : ex2(ml.x - top);
                lsum = fmaf(f, ml.y, lsum);
                y0 = fmaf(f, y.x, y0);
                y1 = fmaf(f, y.y, y1);
            }
            if (ch >= D) continue;
            if (CLUSTER && a.cluster > 1) {
                // to the CTA that finishes this output: slot (its pair, this CTA)
                const int to = i / share;
                st_shared_cluster_f4(cluster_map_shared(rec + ((i - to * share) * a.cluster + rank) * 16, to),
                                     make_float4(y0, y1, top, lsum));
            } else if (CLUSTER || whole) {
                const float inv = 1.f / lsum;
                *reinterpret_cast<__half2 *>(reinterpret_cast<__half *>(a.out) + (out_row + hq) * D + ch) =
                    __floats2half2_rn(y0 * inv, y1 * inv);
            } else {
                const size_t row = static_cast<size_t>(piece_slot(c, u)) * (HG * a.gq) + hq;
                *reinterpret_cast<float2 *>(a.ws_acc + row * D + ch) = make_float2(y0, y1);
                // a NaN sum is kept as a state that makes the merged sum NaN
                if (pair == 0)
                    a.ws_ml[row] = lsum == lsum ? make_float2(top, lsum) : make_float2(INFINITY, 1.f);
            }
        }
        if constexpr (!CLUSTER) {
            __syncthreads();  // the ring is free again
        } else if (a.cluster > 1) {
            cluster_sync_all();  // every record has arrived
            for (int j = tid; j < share; j += kThreads) {
                const int i = rank * share + j;
                const int hq = i / (DP / 2), pair = i % (DP / 2);
                const int m = pair >> 3, pg = pair & 7;
                const int ch = DP == 64 ? 8 * pg + 2 * m : (m >> 3) * 128 + 16 * pg + 2 * (m & 7);
                if (hq >= heads || ch >= D) continue;
                const float4 *r = reinterpret_cast<const float4 *>(smem + NW * NS * kTileBytes) + j * a.cluster;
                float top = -INFINITY, lsum = 0.f, y0 = 0.f, y1 = 0.f;
#pragma unroll 4
                for (int q = 0; q < a.cluster; ++q) top = fmaxf(top, r[q].z);
#pragma unroll 4
                for (int q = 0; q < a.cluster; ++q) {
                    const float4 v = r[q];
                    const float f = v.z == -INFINITY ? 0.f : ex2(v.z - top);
                    lsum = fmaf(f, v.w, lsum);
                    y0 = fmaf(f, v.x, y0);
                    y1 = fmaf(f, v.y, y1);
                }
                const float inv = 1.f / lsum;
                *reinterpret_cast<__half2 *>(reinterpret_cast<__half *>(a.out) + (out_row + hq) * D + ch) =
                    __floats2half2_rn(y0 * inv, y1 * inv);
            }
        }
    } while (!CLUSTER && x < x1);
}

struct Q8Instance {
    int dp, nt;
    bool pair;
    const void *split, *cluster;
};

// The instances of one 8-bit type: 16 warps on an SM where a thread's accumulators
// and query fragments leave room for 128 registers, 8 otherwise; ring slots that
// fill ~200 KB of an SM's shared memory.  256 channels with 9 to 16 query heads need
// more than the 255 registers that there are and spill 32 to 84 bytes; no other does.
template <int KV>
const Q8Instance *q8_instance(int dp, int nt, bool pair) {
#define DATTN_Q8(DP, NT, PAIR)                                                                      \
    {DP, NT, PAIR,                                                                                  \
     reinterpret_cast<const void *>(decode_q8_kernel<DP, NT, PAIR, KV, q8_slots(DP, NT), false>),   \
     reinterpret_cast<const void *>(decode_q8_kernel<DP, NT, PAIR, KV, q8_slots(DP, NT), true>)}
    static const Q8Instance table[] = {
        DATTN_Q8(64, 1, true),  DATTN_Q8(64, 1, false),  DATTN_Q8(64, 2, false),
        DATTN_Q8(128, 1, true), DATTN_Q8(128, 1, false), DATTN_Q8(128, 2, false),
        DATTN_Q8(256, 1, true), DATTN_Q8(256, 1, false), DATTN_Q8(256, 2, false)};
#undef DATTN_Q8
    for (const Q8Instance &i : table)
        if (i.dp == dp && i.nt == nt && i.pair == pair) return &i;
    return nullptr;
}

}  // namespace
}  // namespace dattn
