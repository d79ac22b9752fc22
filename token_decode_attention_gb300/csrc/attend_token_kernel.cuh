// attend_token_kernel.cuh -- attention of one token per sequence over a 16-bit cache, query
// heads sharing key/value heads in groups, over the positions that a window and sinks leave.
//
//   out[b,h,:] = sum_j 2^(s_j) V[j] / sum_j 2^(s_j),  s_j = (Q[b,h,:] . K[j]) log2e / sqrt(D)
//
// in one pass with a running maximum.  What bounds it: every key and value that is seen is
// read once, 4 D bytes a position and key/value head for 4 G D flops (G query heads to one).
// The products run on the tensor cores with the cache as the 16-row operand (mma.sync
// m16n8k16): S^T = K Q^T over 16 positions and out^T = V^T P^T over 16 channels, the query
// heads in the 8 columns.  A tcgen05 instruction wants 64 rows at least; a decode has as
// many as query heads share a key, and at HBM's rate the tensor pipe idles either way.
// P enters as the sum of two 16-bit numbers, so that the weights are off by at most 1.5 x 2^-15
// (bf16) or 1.5 x 2^-21 (f16) where one number is off by up to 2^-8 or 2^-11: their rounding
// alone would move outputs by as much as the outputs' own rounding does.  Both parts are
// positive wherever the weight is (the first is rounded down from slightly less than it): an
// infinite V stays infinite.
//
// Work split: the seen positions are counted through (attend_rows.cuh) and cut into tiles
// of 16.  A CTA takes a chunk of one unit, a (sequence, group of key/value heads); each of
// its warps one head and every PH-th tile, through a ring of its own in shared memory,
// filled with 16-byte cp.async, so the main loop has no CTA-wide barrier.  A unit of one chunk is
// finished by its CTA; the chunks of a cluster merge through distributed shared memory in
// the same launch; other units leave their chunks' states to attend_merge.cu.
//
// Measured (graph replay, inputs larger than L2 in all): 64 sequences of 8 key/value heads of
// 128 behind a window of 4096, bf16 in pages of 64, 807 MB, 119 us, 6.8 TB/s, a copy's rate
// (a read-only stream can reach 7.5); one of 131072 positions, 537 MB, 83.4 us, 6.4 TB/s; one
// of 1028, 4.2 MB, 5.7 us, bound by latency (launch, position, first tiles, exchange).
#pragma once

#include <type_traits>

#include "attend_rows.cuh"

namespace dattn {
namespace {

using attend::ex2;
using attend::Pair;
using attend::Seen;

constexpr unsigned kFull = 0xffffffffu;
constexpr int kTile = kTokenTile;

// The running maximum M is kept kHeadroom (log2) below the largest exponent at the time it
// was set and moved only when an exponent exceeds M + kTrigger: weights lie below 2^15
// (f16 holds up to 65504) and the largest is at least 2^10.
constexpr float kHeadroom = 10.f, kTrigger = 15.f;

template <typename T>
__device__ __forceinline__ void mma16816(float *c, const uint32_t *a, uint32_t b0, uint32_t b1) {
    if constexpr (std::is_same<T, __half>::value)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
                     "{%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
                     "{%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldmatrix4(uint32_t *r, uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t *r, uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
// 8x8 transpose of 16-bit elements across the warp.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// Two weights as two words of 16-bit pairs whose sum they are: the first a little below
// the weight, the second what that leaves, positive where the weight is.
template <typename T>
__device__ __forceinline__ void split2(float x, float y, uint32_t &most, uint32_t &rest) {
    constexpr float kLess = std::is_same<T, __half>::value ? 1.f - 0x1p-10f : 1.f - 0x1p-7f;
    most = Pair<T>::narrow(x * kLess, y * kLess);
    const float2 f = Pair<T>::wide(most);
    rest = Pair<T>::narrow(x - f.x, y - f.y);
}

// Byte offset of 16-byte chunk c of row r in a tile of rows of `row` bytes: the chunks of
// 128 bytes are swapped by the row, so that ldmatrix reads 8 rows without bank conflicts.
__device__ __forceinline__ uint32_t chunk_at(int row, int r, int c) {
    return r * row + (((c & ~7) | ((c ^ r) & 7)) << 4);
}

// DP: head_dim rounded up to 64, 128 or 256 (channels above head_dim are zero filled).
// NT: 8-column tiles of query heads.  PAIR (NT = 1): at most four query heads, each in
// columns h and h + 4, which hold the two parts of its weights.
template <typename T, int DP, int NT, bool PAIR, bool CLUSTER>
__global__ void __launch_bounds__(kTokenWarps * 32, token_ctas_per_sm(DP))
    attend_token_kernel(const AttendArgs a, const TokenArgs w) {
    constexpr int NK = DP / 16;  // 16-channel steps
    constexpr int NW = kTokenWarps, kThreads = NW * 32, NS = kTokenSlots;
    constexpr int kRow = DP * 2;                // bytes of a row
    constexpr int kTileBytes = 2 * kTile * kRow;  // K and V
    constexpr int CPR = kRow / 16;              // 16-byte chunks of a row
    constexpr int RPI = CPR >= 32 ? 1 : 32 / CPR;  // rows per warp-wide copy
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ float2 s_ml[NW][NT * 8];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, t = lane & 3;
    const int D = a.D;
    const unsigned unit = blockIdx.x / static_cast<unsigned>(w.chunks);
    const int chunk = static_cast<int>(blockIdx.x - unit * w.chunks);
    const int b = static_cast<int>(unit / static_cast<unsigned>(w.head_groups));
    const int grp = static_cast<int>(unit) - b * w.head_groups;

    if constexpr (CLUSTER) cluster_arrive_relaxed();
    // Beside the kernel of the shared positions, which began when everything before it was
    // done, nothing is waited for; the last CTA alone stays until that kernel has ended, so
    // that what waits for this one has both.
    const bool stays = w.own_only && blockIdx.x == gridDim.x - 1;
    if (!w.own_only) pdl_wait_primary();

    Seen v = attend::seen_by(a, attend::live_end(a, b) - 1);
    if (w.own_only) v.lo = min(a.shared, v.end);  // the shared positions are another kernel's
    const int n = v.count();
    const int tiles = (n + kTile - 1) / kTile;
    int from, to;
    if constexpr (CLUSTER) {
        from = static_cast<int>(static_cast<long long>(chunk) * tiles / w.chunks);
        to = static_cast<int>(static_cast<long long>(chunk + 1) * tiles / w.chunks);
    } else {
        from = min(chunk * w.chunk_tiles, tiles);
        to = min(from + w.chunk_tiles, tiles);
        if (from >= to && chunk > 0) {  // the merge knows how many chunks there are
            if (stays) pdl_wait_primary();
            return;
        }
    }

    const int HG = w.heads_per_cta, PH = w.phases;
    const int hl = warp % HG, ph = warp / HG;
    const int vh = grp * HG + hl;  // virtual head: gq query heads of one key/value head
    const bool active = ph < PH && vh < w.vheads;
    const int kvh = active ? vh / w.vheads_per_kv : 0;
    const int ntiles = active && ph < to - from ? (to - from - ph + PH - 1) / PH : 0;
    const int first = (from + ph) * kTile, step = PH * kTile;
    const uint32_t ring = smem_addr(smem) + warp * w.ring_bytes;
    const int crow = CPR >= 32 ? 0 : lane / CPR, cchunk = CPR >= 32 ? lane : lane % CPR;
    const bool in_head = cchunk * 8 < D;
    const unsigned row_bytes = static_cast<unsigned>(a.Hk) * D * 2;
    const size_t col = in_head ? (static_cast<size_t>(kvh) * D + cchunk * 8) * 2 : 0;
    const unsigned char *const k0 = static_cast<const unsigned char *>(a.K) + col;
    const unsigned char *const v0 = static_cast<const unsigned char *>(a.V) + col;

    // The cache row of position l of tile i, lanes l and l + 16; found a tile ahead of the copies.
    auto row_in_tile = [&](int i) -> unsigned {
        const int at = first + i * step + (lane & 15);
        return i < ntiles && at < n ? static_cast<unsigned>(attend::row_of(a, b, v.at(at))) : 0u;
    };
    auto issue = [&](int i, int slot, unsigned row) {
        const int at0 = first + i * step;
        const uint32_t dst = ring + slot * kTileBytes;
#pragma unroll
        for (int j = 0; j < kTile / RPI; ++j) {
            const int r = j * RPI + crow;
            const unsigned rr = __shfl_sync(kFull, row, r);
            const bool there = in_head && at0 + r < n;
            const size_t off = there ? static_cast<size_t>(rr) * row_bytes : 0;
            const uint32_t o = dst + chunk_at(kRow, r, cchunk);
            cp_async16(o, k0 + off, there ? 16 : 0);
            cp_async16(o + kTile * kRow, v0 + off, there ? 16 : 0);
        }
    };

    // Q^T fragments: column = query head (modulo 4 where two columns share one)
    uint32_t qf[NT][NK][2];
    unsigned row = row_in_tile(0);
    int fill = 0;
    int issued = 0;
    // the first tiles are under way before Q is read
#pragma unroll
    for (int j = 0; j < NS - 1; ++j) {
        if (j < ntiles) {
            const unsigned now = row;
            row = row_in_tile(j + 1);
            issue(j, fill, now);
            fill = fill + 1 == NS ? 0 : fill + 1;
            ++issued;
        }
        cp_async_commit();
    }
#pragma unroll
    for (int nn = 0; nn < NT; ++nn) {
        const int h = PAIR ? g & 3 : nn * 8 + g;
        const T *q = static_cast<const T *>(a.Q) + b * a.q_stride + (static_cast<long long>(vh) * w.gq + h) * D;
#pragma unroll
        for (int k = 0; k < NK; ++k) {
            const int ch = 16 * k + 2 * t;
            const bool in = ntiles > 0 && h < w.gq;
            qf[nn][k][0] = in && ch < D ? __ldg(reinterpret_cast<const uint32_t *>(q + ch)) : 0u;
            qf[nn][k][1] = in && ch + 8 < D ? __ldg(reinterpret_cast<const uint32_t *>(q + ch + 8)) : 0u;
        }
    }

    float acc[NT][NK][4];
    float M[NT][2], l[NT][2];
#pragma unroll
    for (int nn = 0; nn < NT; ++nn) {
#pragma unroll
        for (int m = 0; m < NK; ++m) acc[nn][m][0] = acc[nn][m][1] = acc[nn][m][2] = acc[nn][m][3] = 0.f;
        M[nn][0] = M[nn][1] = -INFINITY;
        l[nn][0] = l[nn][1] = 0.f;
    }

    int slot = 0;
    for (int i = 0; i < ntiles; ++i) {
        cp_async_wait<NS - 2>();
        __syncwarp();  // every lane's copies of tile i are visible, tile i - 1 is read
        if (issued < ntiles) {
            const unsigned now = row;
            row = row_in_tile(issued + 1);
            issue(issued, fill, now);
            fill = fill + 1 == NS ? 0 : fill + 1;
            ++issued;
        }
        cp_async_commit();
        const uint32_t kt = ring + slot * kTileBytes, vt = kt + kTile * kRow;
        slot = slot + 1 == NS ? 0 : slot + 1;

        // S^T over the tile: rows (positions) g and g + 8, columns 2t, 2t + 1
        float s[NT][2][4];
#pragma unroll
        for (int nn = 0; nn < NT; ++nn)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[nn][0][e] = s[nn][1][e] = 0.f;
#pragma unroll
        for (int k = 0; k < NK; ++k) {
            uint32_t ka[4];
            ldmatrix4(ka, kt + chunk_at(kRow, lane & 15, 2 * k + (lane >> 4)));
#pragma unroll
            for (int nn = 0; nn < NT; ++nn) mma16816<T>(s[nn][k & 1], ka, qf[nn][k][0], qf[nn][k][1]);
        }
        const int at0 = first + i * step;
        const bool in0 = at0 + g < n, in1 = at0 + 8 + g < n;
        bool grow = false;
#pragma unroll
        for (int nn = 0; nn < NT; ++nn)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float z = (s[nn][0][e] + s[nn][1][e]) * a.qscale;
                s[nn][0][e] = (e < 2 ? in0 : in1) ? z : -INFINITY;
                grow |= s[nn][0][e] > M[nn][e & 1] + kTrigger;
            }
        if (__any_sync(kFull, grow)) {
#pragma unroll
            for (int nn = 0; nn < NT; ++nn)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float mx = fmaxf(s[nn][0][e], s[nn][0][e + 2]);
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
                    const float nm = fmaxf(M[nn][e], mx - kHeadroom);
                    const float f = M[nn][e] == -INFINITY ? 0.f : ex2(M[nn][e] - nm);
                    M[nn][e] = nm;
                    l[nn][e] *= f;
#pragma unroll
                    for (int m = 0; m < NK; ++m) {
                        acc[nn][m][e] *= f;
                        acc[nn][m][e + 2] *= f;
                    }
                }
        }
        // the weights in two parts: columns 0 to 3 and 4 to 7 of a pair, or pf and pr
        uint32_t pf[NT][2];
        [[maybe_unused]] uint32_t pr[NT][2];
#pragma unroll
        for (int nn = 0; nn < NT; ++nn) {
            const float m0 = M[nn][0] == -INFINITY ? 0.f : M[nn][0];
            const float m1 = M[nn][1] == -INFINITY ? 0.f : M[nn][1];
            const float e0 = ex2(s[nn][0][0] - m0), e1 = ex2(s[nn][0][1] - m1);
            const float e2 = ex2(s[nn][0][2] - m0), e3 = ex2(s[nn][0][3] - m1);
            l[nn][0] += e0 + e2;
            l[nn][1] += e1 + e3;
            uint32_t h0, h1, r0, r1;
            split2<T>(e0, e1, h0, r0);
            split2<T>(e2, e3, h1, r1);
            if constexpr (PAIR) {
                pf[nn][0] = transpose8x8(t & 2 ? r0 : h0);
                pf[nn][1] = transpose8x8(t & 2 ? r1 : h1);
            } else {
                pf[nn][0] = transpose8x8(h0);
                pf[nn][1] = transpose8x8(h1);
                pr[nn][0] = transpose8x8(r0);
                pr[nn][1] = transpose8x8(r1);
            }
        }
        // out^T += V^T P^T
#pragma unroll
        for (int m = 0; m < NK; ++m) {
            uint32_t va[4];
            ldmatrix4_trans(va, vt + chunk_at(kRow, (lane & 7) + ((lane >> 4) << 3), 2 * m + ((lane >> 3) & 1)));
#pragma unroll
            for (int nn = 0; nn < NT; ++nn) {
                mma16816<T>(acc[nn][m], va, pf[nn][0], pf[nn][1]);
                if constexpr (!PAIR) mma16816<T>(acc[nn][m], va, pr[nn][0], pr[nn][1]);
            }
        }
    }

    pdl_launch_dependents();

    // ---- the chunk's state: sum over the lanes, merge the phases, store ----
#pragma unroll
    for (int nn = 0; nn < NT; ++nn)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) l[nn][e] += __shfl_xor_sync(kFull, l[nn][e], o);

    // Each warp leaves (M, l) and its accumulators in its idle ring, a row of kStage floats
    // per query head; kStage makes the stores free of bank conflicts.
    constexpr int kStage = DP + 4;
    float *const rows = reinterpret_cast<float *>(smem + warp * w.ring_bytes);
    cp_async_wait<0>();
    __syncwarp();  // the last tile has been read
    if constexpr (PAIR) {
        // the two columns of a query head together: lanes t and t ^ 2 hold the same two
        // heads and finish one each
        const bool second = t & 2;
        const int h = 2 * (t & 1) + (second ? 1 : 0);
        const bool mine = active && h < w.gq;
        // columns h and h + 4 count the same weights: l is that of either
        if (mine && g == 0)
            s_ml[warp][h] = second ? make_float2(M[0][1], l[0][1]) : make_float2(M[0][0], l[0][0]);
#pragma unroll
        for (int m = 0; m < NK; ++m) {
            const float *c = acc[0][m];
            const float y0 = __shfl_xor_sync(kFull, second ? c[0] : c[1], 2);
            const float y1 = __shfl_xor_sync(kFull, second ? c[2] : c[3], 2);
            if (mine) {
                rows[h * kStage + 16 * m + g] = (second ? c[1] : c[0]) + y0;
                rows[h * kStage + 16 * m + g + 8] = (second ? c[3] : c[2]) + y1;
            }
        }
    } else if (active) {
#pragma unroll
        for (int nn = 0; nn < NT; ++nn)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int h = nn * 8 + 2 * t + e;
                if (h >= w.gq) continue;
                if (g == 0) s_ml[warp][h] = make_float2(M[nn][e], l[nn][e]);
#pragma unroll
                for (int m = 0; m < NK; ++m) {
                    rows[h * kStage + 16 * m + g] = acc[nn][m][e];
                    rows[h * kStage + 16 * m + g + 8] = acc[nn][m][e + 2];
                }
            }
    }
    __syncthreads();
    // A thread takes a (query head, channel pair) of the unit.
    const int heads = min(HG, w.vheads - grp * HG) * w.gq;
    const long long out_row = static_cast<long long>(b) * a.H + static_cast<long long>(grp) * HG * w.gq;
    const bool partial = w.own_only || (!CLUSTER && w.chunks > 1);
    [[maybe_unused]] const uint32_t rec = smem_addr(smem) + NW * w.ring_bytes;
    [[maybe_unused]] int share = 0, rank = 0;
    if constexpr (CLUSTER) {
        // each CTA of the cluster finishes an equal share of the outputs
        share = (heads * (DP / 2) + w.chunks - 1) / w.chunks;
        rank = static_cast<int>(cluster_ctarank());
        cluster_wait();  // every CTA of the cluster has started: its shared memory may be written
    }
    T *const out = static_cast<T *>(a.out);
    for (int i = tid; i < heads * (DP / 2); i += kThreads) {
        const int hq = i / (DP / 2), ch = 2 * (i % (DP / 2));  // DP is a power of two
        const int w0 = fast_div(hq, w.div_gq);
        const int h = hq - w0 * w.gq;
        float top = -INFINITY, lsum = 0.f, y0 = 0.f, y1 = 0.f;
#pragma unroll 4
        for (int p = 0; p < PH; ++p) top = fmaxf(top, s_ml[p * HG + w0][h].x);
#pragma unroll 4
        for (int p = 0; p < PH; ++p) {
            const int from_warp = p * HG + w0;
            const float2 ml = s_ml[from_warp][h];
            const float2 y = *reinterpret_cast<const float2 *>(
                reinterpret_cast<const float *>(smem + from_warp * w.ring_bytes) + h * kStage + ch);
            const float f = ml.x == -INFINITY ? 0.f : ex2(ml.x - top);
            lsum = fmaf(f, ml.y, lsum);
            y0 = fmaf(f, y.x, y0);
            y1 = fmaf(f, y.y, y1);
        }
        if (ch >= D) continue;
        if constexpr (CLUSTER) {
            // to the CTA that finishes this output: slot (its pair, this CTA)
            const int dst = i / share;
            st_shared_cluster_f4(cluster_map_shared(rec + ((i - dst * share) * w.chunks + rank) * 16, dst),
                                 make_float4(y0, y1, top, lsum));
        } else if (!partial) {
            const float inv = 1.f / lsum;
            *reinterpret_cast<uint32_t *>(out + (out_row + hq) * D + ch) = Pair<T>::narrow(y0 * inv, y1 * inv);
        } else {
            const long long r = (out_row + hq) * w.chunks + chunk;
            *reinterpret_cast<float2 *>(w.ws_acc + r * D + ch) = make_float2(y0, y1);
            if (ch == 0) w.ws_ml[r] = make_float2(top, lsum);
        }
    }
    if (stays) pdl_wait_primary();
    if constexpr (CLUSTER) {
        cluster_sync_all();  // every record has arrived
        for (int j = tid; j < share; j += kThreads) {
            const int i = rank * share + j;
            const int hq = i / (DP / 2), ch = 2 * (i % (DP / 2));
            if (hq >= heads || ch >= D) continue;
            const float4 *r = reinterpret_cast<const float4 *>(smem + NW * w.ring_bytes) + j * w.chunks;
            float top = -INFINITY, lsum = 0.f, y0 = 0.f, y1 = 0.f;
#pragma unroll 4
            for (int q = 0; q < w.chunks; ++q) top = fmaxf(top, r[q].z);
#pragma unroll 4
            for (int q = 0; q < w.chunks; ++q) {
                const float4 x = r[q];
                const float f = x.z == -INFINITY ? 0.f : ex2(x.z - top);
                lsum = fmaf(f, x.w, lsum);
                y0 = fmaf(f, x.x, y0);
                y1 = fmaf(f, x.y, y1);
            }
            const float inv = 1.f / lsum;
            *reinterpret_cast<uint32_t *>(out + (out_row + hq) * D + ch) = Pair<T>::narrow(y0 * inv, y1 * inv);
        }
    }
}

template <typename T>
const void *token_instance(int dp, int nt, bool pair, bool cluster) {
    struct Instance {
        int dp, nt;
        bool pair;
        const void *chunks, *cluster;
    };
#define DATTN_TOKEN(DP, NT, PAIR)                                                              \
    {DP, NT, PAIR, reinterpret_cast<const void *>(attend_token_kernel<T, DP, NT, PAIR, false>), \
     reinterpret_cast<const void *>(attend_token_kernel<T, DP, NT, PAIR, true>)}
    static const Instance table[] = {
        DATTN_TOKEN(64, 1, true),  DATTN_TOKEN(64, 1, false),  DATTN_TOKEN(64, 2, false),
        DATTN_TOKEN(128, 1, true), DATTN_TOKEN(128, 1, false), DATTN_TOKEN(128, 2, false),
        DATTN_TOKEN(256, 1, true), DATTN_TOKEN(256, 1, false), DATTN_TOKEN(256, 2, false)};
#undef DATTN_TOKEN
    for (const Instance &i : table)
        if (i.dp == dp && i.nt == nt && i.pair == pair) return cluster ? i.cluster : i.chunks;
    return nullptr;
}

}  // namespace
}  // namespace dattn
