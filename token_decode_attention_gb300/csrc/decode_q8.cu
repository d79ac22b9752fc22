// decode_q8.cu -- single-query attention over a KV cache held in 8 bits (e4m3
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
// and the products accumulate in fp32; P is rounded to f16 (a relative 2^-11).
//
// Fragments straight from 16-byte loads: the sum over channels (and over
// positions) may run in any order, so the channel (position) that a fragment
// slot stands for is chosen to make each lane's elements contiguous in the
// cache row, for K one 16-byte chunk per four k-steps, for V two neighbouring
// positions' words whose bytes are paired with prmt.  P^T is the S^T
// accumulator rounded to f16 and transposed with movmatrix.
//
// Work split: as in the f16 decode (streamk.h), the live positions of all
// (sequence, head group) units, flattened, are cut into equal ranges, one per
// CTA.  In a CTA each warp owns one head (heads_per_cta of them) and one phase:
// tiles of 16 positions go to the phases in turn.  Every warp streams its own
// tiles through a private ring in shared memory with 16-byte cp.async, so the
// main loop has no CTA-wide barrier; rows past the end of a piece are zero
// filled and never read from memory.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "dattn_internal.h"
#include "ptx.cuh"
#include "streamk.h"

namespace dattn {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kTile = 16;  // positions per tile

// The running maximum M is kept kHeadroom (log2) below the largest exponent at
// the time it was set, and moved only when an exponent exceeds M + kTrigger:
// weights then lie below 2^15 (f16 holds up to 65504) and keep f16's full
// precision down to 2^-24 of the largest.
constexpr float kHeadroom = 10.f, kTrigger = 15.f;
// log2 of the smallest scale of V that takes part (a scale of 0 stands for
// values of zero; it is read as 2^-100, which leaves them below any f16).
constexpr float kMinLogScale = -100.f;

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

// n / d for 0 <= n < 2^31 by one multiplication (d's constants from the host).
__device__ __forceinline__ int fast_div(int n, FastDiv d) {
    return static_cast<int>((static_cast<unsigned long long>(static_cast<unsigned>(n)) * d.mul) >>
                            d.shift);
}

// bytes == 0: the 16 bytes are zero filled and src is not read.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
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
// filled).  NT: 8-column tiles of query heads.  NW: warps.  NS: ring slots.
template <int DP, int NT, int KV, int NW, int NS>
__global__ void __launch_bounds__(NW * 32, 1) decode_q8_kernel(const Q8DecodeArgs a) {
    constexpr int NJ = DP / 64;           // 64-channel spans of a row
    constexpr int NM = DP / 16;           // 16-channel tiles of the output
    constexpr int kThreads = NW * 32;
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
    const long long G = a.partitions;

    pdl_wait_primary();

    // ---- this CTA's range [x0, x1) of the flattened positions ----
    long long W, b = 0, base = 0;
    if (a.B == 1) {
        W = nhg * live_len(a.cur_pos, 0, a.S);
    } else {
        long long sum = 0;
        for (int i = tid; i < a.B; i += kThreads) sum += live_len(a.cur_pos, i, a.S);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
        if (lane == 0) s_warp[warp] = sum;
        __syncthreads();
        W = 0;
#pragma unroll
        for (int w = 0; w < NW; ++w) W += s_warp[w];
        W *= nhg;
    }
    const long long c = blockIdx.x;
    long long x = range_begin(c, W, G);
    const long long x1 = range_begin(c + 1, W, G);
    if (a.B > 1) {
        const bool keep = c == 0 && a.ws_prefix != nullptr;
        if (x >= x1 && !keep) return;
        long long carry = 0;
        for (int i0 = 0; i0 < a.B; i0 += kThreads) {
            const int i = i0 + tid;
            const long long L = i < a.B ? live_len(a.cur_pos, i, a.S) : 0;
            long long pre = L;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(kFull, pre, o);
                if (lane >= o) pre += y;
            }
            __syncthreads();  // s_warp of the round before has been read
            if (lane == 31) s_warp[warp] = pre;
            __syncthreads();
            long long total = 0;
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                if (w < warp) pre += s_warp[w];
                total += s_warp[w];
            }
            pre += carry;  // positions up to and including sequence i
            if (i < a.B) {
                if (keep) {
                    if (i == 0) a.ws_prefix[0] = 0;
                    a.ws_prefix[i + 1] = pre;
                }
                if (x >= nhg * (pre - L) && x < nhg * pre) {
                    s_b0 = i;
                    s_base0 = nhg * (pre - L);
                }
            }
            carry += total;
            if (!keep && x < nhg * carry) break;  // the same in every thread
        }
        __syncthreads();
        b = s_b0;
        base = s_base0;
    }
    if (x >= x1) return;

    const int HG = a.heads_per_cta, PH = a.phases;
    const int hl = warp % HG, ph = warp / HG;
    const uint32_t ring = smem_addr(smem) + warp * (NS * kTileBytes);
    const int step = kTile * PH;
    const size_t row_bytes = static_cast<size_t>(a.kv_heads) * D;
    const int r0 = tile_row<DP>(g);                               // K: rows r0 and r0 + 8
    const int v0 = tile_row<DP>(2 * t), v1 = tile_row<DP>(2 * t + 1);  // V: and 8 rows on
    int L = live_len(a.cur_pos, b, a.S);

    while (x < x1) {
        // ---- the next piece: positions [off, end) of unit (b, grp) ----
        while (x >= base + nhg * L) {
            base += nhg * L;
            ++b;
            L = live_len(a.cur_pos, b, a.S);
        }
        const unsigned rel = static_cast<unsigned>(x - base);
        const int grp = static_cast<int>(rel / static_cast<unsigned>(L));
        const int off = static_cast<int>(rel - static_cast<unsigned>(grp) * static_cast<unsigned>(L));
        const int len = static_cast<int>(x1 - x < L - off ? x1 - x : L - off);
        const int end = off + len;
        const long long u = b * nhg + grp;
        x += len;

        const int vh = grp * HG + hl;  // virtual head: gq query heads of one key/value head
        const bool active = ph < PH && vh < a.vheads;
        const int kvh = active ? vh / a.vheads_per_kv : 0;
        const int first = off + kTile * ph;
        const int ntiles = active && first < end ? (end - first + step - 1) / step : 0;

        // Copy tile i of this warp into its ring slot.  Lanes l and l + 16 find
        // the cache row of tile position l (through the block table) and copy
        // its scales of K and V; the rows' bytes are dealt out RPI rows at a time.
        auto issue = [&](int i, int slot) {
            const int p0 = first + i * step;
            const uint32_t dst = ring + slot * kTileBytes;
            const int pos = p0 + (lane & 15);
            const bool live = pos < end;
            long long row = 0, srow = 0;
            if (live) {
                if (a.block_table == nullptr) {
                    row = b * a.S + pos;
                    srow = b * a.scale_rows + fast_div(pos, a.div_block);
                } else {
                    const int pi = fast_div(pos, a.div_page);
                    const int in = pos - pi * a.page_size;
                    long long page = __ldg(a.block_table + b * a.max_pages + pi);
                    if (page < 0 || page >= a.num_pages) {
                        atomicOr(a.err, kErrPageIndex);
                        page = 0;
                    }
                    row = page * a.page_size + in;
                    srow = page * a.scale_rows + fast_div(in, a.div_block);
                }
            }
            const float *scale = (lane < 16 ? a.ks : a.vs) + srow * a.kv_heads + kvh;
            cp_async4(dst + 32 * DP + lane * 4, scale, live ? 4 : 0);
            const int ch = lane % CPR;
            const size_t col = static_cast<size_t>(kvh) * D + ch * 16;
            const bool in_head = ch * 16 < D;
#pragma unroll
            for (int j = 0; j < kTile / RPI; ++j) {
                const int r = j * RPI + lane / CPR;
                const long long rr = __shfl_sync(kFull, row, r);
                const int bytes = in_head && p0 + r < end ? 16 : 0;
                const size_t at = bytes ? static_cast<size_t>(rr) * row_bytes + col : 0;
                cp_async16(dst + chunk_at<DP>(r, ch), a.K + at, bytes);
                cp_async16(dst + 16 * DP + chunk_at<DP>(r, ch), a.V + at, bytes);
            }
        };

#pragma unroll
        for (int i = 0; i < NS - 1; ++i) {
            if (i < ntiles) issue(i, i);
            cp_async_commit();
        }

        // Q^T fragments: column n = query head, channels as in K's chunks.
        uint32_t qf[NT][NJ][4][2];
        if (ntiles > 0) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int h = n * 8 + g;
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

        int slot = 0;
        for (int i = 0; i < ntiles; ++i) {
            cp_async_wait<NS - 2>();
            __syncwarp();  // every lane's copies of tile i are visible, tile i - 1 is read
            {
                const int nxt = i + NS - 1;
                const int ns = slot == 0 ? NS - 1 : slot - 1;
                if (nxt < ntiles) issue(nxt, ns);
                cp_async_commit();
            }
            const uint32_t kt = ring + slot * kTileBytes, vt = kt + 16 * DP, sc = kt + 32 * DP;
            slot = slot + 1 == NS ? 0 : slot + 1;

            // S^T over the tile: rows (positions) g and g + 8, columns 2t, 2t + 1
            float s[NT][2][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[n][0][e] = s[n][1][e] = 0.f;
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                const uint4 ka = lds128(kt + chunk_at<DP>(r0, t + 4 * j));
                const uint4 kb = lds128(kt + 8 * DP + chunk_at<DP>(r0, t + 4 * j));
                const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t a0, a1, a2, a3;
                    widen<KV>(wa[q], a0, a2);
                    widen<KV>(wb[q], a1, a3);
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        mma16816(s[n][q & 1], a0, a1, a2, a3, qf[n][j][q][0], qf[n][j][q][1]);
                }
            }

            // exponents t = s log2e / sqrt(D) + log2 vs
            const float ks0 = lds32(sc + r0 * 4) * a.qscale, ks1 = lds32(sc + 32 + r0 * 4) * a.qscale;
            const float lv0 = fmaxf(lg2(lds32(sc + 64 + r0 * 4)), kMinLogScale);
            const float lv1 = fmaxf(lg2(lds32(sc + 96 + r0 * 4)), kMinLogScale);
            const float iv0 = ex2(-lv0), iv1 = ex2(-lv1);
            const int p0 = first + i * step;
            const bool in0 = p0 + r0 < end, in1 = p0 + 8 + r0 < end;
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
            uint32_t pf[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float m0 = M[n][0] == -INFINITY ? 0.f : M[n][0];
                const float m1 = M[n][1] == -INFINITY ? 0.f : M[n][1];
                const float e0 = ex2(s[n][0][0] - m0), e1 = ex2(s[n][0][1] - m1);
                const float e2 = ex2(s[n][0][2] - m0), e3 = ex2(s[n][0][3] - m1);
                l[n][0] = fmaf(e0, iv0, fmaf(e2, iv1, l[n][0]));
                l[n][1] = fmaf(e1, iv0, fmaf(e3, iv1, l[n][1]));
                pf[n][0] = transpose8x8(pack2(e0, e1));
                pf[n][1] = transpose8x8(pack2(e2, e3));
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
                    widen<KV>(x2, a0, a1);
                    widen<KV>(z2, a2, a3);
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        mma16816(acc[n][m + 1], a0, a1, a2, a3, pf[n][0], pf[n][1]);
                }
            }
        }

        // ---- the piece's state: sum over the lanes, merge the phases, store ----
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) l[n][e] += __shfl_xor_sync(kFull, l[n][e], o);

        const bool whole = len == L;
        const size_t hgs = static_cast<size_t>(HG) * a.gq;
        // channels of tile m in this lane: two neighbours from channel(m) on
        auto channel = [&](int m) {
            return DP == 64 ? 8 * g + 2 * m : (m >> 3) * 128 + 16 * g + 2 * (m & 7);
        };
        auto store = [&](int n, int e, int m, float lsum, float y0, float y1) {
            const int h = n * 8 + 2 * t + e, ch = channel(m);
            if (h >= a.gq || ch >= D) return;
            if (whole) {
                const float inv = 1.f / lsum;
                __half *o = reinterpret_cast<__half *>(a.out) +
                            (b * a.H + static_cast<long long>(vh) * a.gq + h) * D + ch;
                *reinterpret_cast<__half2 *>(o) = __floats2half2_rn(y0 * inv, y1 * inv);
            } else {
                const size_t row = static_cast<size_t>(piece_slot(c, u)) * hgs + hl * a.gq + h;
                *reinterpret_cast<float2 *>(a.ws_acc + row * D + ch) = make_float2(y0, y1);
            }
        };
        auto store_ml = [&](int n, int e, float m, float lsum) {
            const int h = n * 8 + 2 * t + e;
            if (whole || h >= a.gq) return;
            const size_t row = static_cast<size_t>(piece_slot(c, u)) * hgs + hl * a.gq + h;
            // a NaN sum is kept as a state that makes the merged sum NaN
            a.ws_ml[row] = lsum == lsum ? make_float2(m, lsum) : make_float2(INFINITY, 1.f);
        };
        if (PH == 1) {
            if (active) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        if (g == 0) store_ml(n, e, M[n][e], l[n][e]);
#pragma unroll
                        for (int m = 0; m < NM; ++m)
                            store(n, e, m, l[n][e], acc[n][m][e], acc[n][m][e + 2]);
                    }
            }
            __syncwarp();
            continue;
        }
        // The ring is idle: each warp leaves its accumulator there, register by
        // register, and phase ph of a head merges the output tiles ph, ph + PH, ...
        float *dump = reinterpret_cast<float *>(smem + warp * (NS * kTileBytes));
        __syncwarp();
        if (active) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int m = 0; m < NM; ++m)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        dump[((n * NM + m) * 4 + e) * 32 + lane] = acc[n][m][e];
                if (g == 0) {
                    s_ml[warp][n * 8 + 2 * t] = make_float2(M[n][0], l[n][0]);
                    s_ml[warp][n * 8 + 2 * t + 1] = make_float2(M[n][1], l[n][1]);
                }
            }
        }
        __syncthreads();
        if (active) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int col = n * 8 + 2 * t + e;
                    float mx = -INFINITY, lsum = 0.f;
                    for (int p = 0; p < PH; ++p) mx = fmaxf(mx, s_ml[p * HG + hl][col].x);
                    for (int p = 0; p < PH; ++p) {
                        const float2 ml = s_ml[p * HG + hl][col];
                        lsum = fmaf(ml.x == -INFINITY ? 0.f : ex2(ml.x - mx), ml.y, lsum);
                    }
                    if (ph == 0 && g == 0) store_ml(n, e, mx, lsum);
                    for (int m = ph; m < NM; m += PH) {
                        float y0 = 0.f, y1 = 0.f;
                        for (int p = 0; p < PH; ++p) {
                            const int w = p * HG + hl;
                            const float mw = s_ml[w][col].x;
                            const float f = mw == -INFINITY ? 0.f : ex2(mw - mx);
                            const float *d = reinterpret_cast<const float *>(smem + w * (NS * kTileBytes)) +
                                             ((n * NM + m) * 4 + e) * 32 + lane;
                            y0 = fmaf(f, d[0], y0);
                            y1 = fmaf(f, d[64], y1);
                        }
                        store(n, e, m, lsum, y0, y1);
                    }
                }
        }
        __syncthreads();  // the ring is free again
    }
    pdl_launch_dependents();
}

struct Instance {
    int dp, nt, kv, nw, ns;
    const void *fn;
};

#define DATTN_Q8(DP, NT, NW, NS)                                                           \
    {DP, NT, kKvE4m3, NW, NS,                                                              \
     reinterpret_cast<const void *>(decode_q8_kernel<DP, NT, kKvE4m3, NW, NS>)},           \
        {DP, NT, kKvInt8, NW, NS,                                                          \
         reinterpret_cast<const void *>(decode_q8_kernel<DP, NT, kKvInt8, NW, NS>)}
const Instance kInstances[] = {
    DATTN_Q8(64, 1, 16, 6), DATTN_Q8(64, 2, 16, 6),  DATTN_Q8(128, 1, 16, 3),
    DATTN_Q8(128, 2, 8, 6), DATTN_Q8(256, 1, 8, 3), DATTN_Q8(256, 2, 8, 3),
};
#undef DATTN_Q8

const Instance *find(int dp, int nt, int kv) {
    for (const Instance &i : kInstances)
        if (i.dp == dp && i.nt == nt && i.kv == kv) return &i;
    return nullptr;
}

}  // namespace

bool decode_q8_shape(int dp, int nt, int *warps, int *slots) {
    const Instance *i = find(dp, nt, kKvE4m3);
    if (i == nullptr) return false;
    *warps = i->nw;
    *slots = i->ns;
    return true;
}

cudaError_t decode_q8_configure() {
    for (const Instance &i : kInstances) {
        const cudaError_t e =
            cudaFuncSetAttribute(i.fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 i.nw * i.ns * q8_tile_bytes(i.dp));
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t launch_decode_q8(const Q8DecodeArgs &a, int dp, int nt, int kv, cudaStream_t stream) {
    const Instance *i = find(dp, nt, kv);
    if (i == nullptr || a.partitions <= 0) return cudaErrorInvalidValue;
    void *args[] = {const_cast<Q8DecodeArgs *>(&a)};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.partitions));
    cfg.blockDim = dim3(i->nw * 32);
    cfg.dynamicSmemBytes = static_cast<size_t>(i->nw) * i->ns * q8_tile_bytes(dp);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelExC(&cfg, i->fn, args);
}

}  // namespace dattn
