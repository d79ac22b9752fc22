// rope_items.cuh -- the pieces of a head row that the rotary kernels work on.
//
// A row of D channels, the first rope_dims of them rotated in pairs, is cut
// into items of N = 16, 8 or 4 channels, the most that divide rope_dims and D, one
// thread each: N / 2 pairs (u, w), channels (i, i + rope_dims/2) in the half layout
// and (2i, 2i + 1) in the interleaved one, or N channels that pass through.  A thread
// needs no other thread's data.  An item is two runs or four (16 channels in 32 bits)
// of at most 16 bytes, spread evenly over the rotated (or the passing) channels, so
// that in either layout neighbouring threads read and write neighbouring runs.
// Where four do not divide rope_dims (N = 1) an item has up to 16 channels, read one
// by one.  Measured on 8192 tokens of 32 heads in f16, us: 80 channels with 16, 20 and 6
// rotated (N = 16, 4, 1) 18.9, 22.1, 110; 96 channels with 24 rotated (N = 8) 23.7, one by
// one 135.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "dattn_internal.h"

namespace dattn {

// cos and sin of the angle p * theta_i from the turn fraction f = theta_i / 2pi
// (units of 2^-64).  p * f mod 1 is an exact wrapping product.  Its top 32 bits
// are split into the nearest quarter turn and a rest within an eighth of a turn
// either way, that into its top 24 bits, a float, and the six below.  The angle in
// radians is z + e, z the nearest float of the former's and e all that is left; sine
// and cosine are their Taylor series in z (|z| <= pi / 4: the first term left out is
// below 2e-9) and their first-order terms in e, summed so that the last addition is
// the only rounding near an ulp; then the quarter turns by exchange and sign.
// Over all angles both are within 4.4e-8 of the exact values and 1.47e-8 rms, where
// rounding those once gives 1.46e-8; without the terms in e and in what the roundings of
// z * z and 1 - z * z / 2 lose, 1.7e-7 and 4.4e-8.  (Within an eighth of a turn, before
// the exchange, the sine's series is 1.15e-8 rms off and the cosine's 1.73e-8.)  A general
// sincospif takes more instructions still: it reduces its argument once more.
__device__ __forceinline__ float2 turn_cos_sin(uint32_t p, unsigned long long f) {
    constexpr float kTurn = 6.28318548f * 0x1p-32f, kTurnLow = -1.74845553e-7f * 0x1p-32f;  // 2 pi
    const uint32_t turn =
        static_cast<uint32_t>((static_cast<unsigned long long>(p) * f) >> 32);
    const uint32_t quarter = (turn + 0x20000000u) >> 30;
    const int rest = static_cast<int>(turn - (quarter << 30));
    const float x = static_cast<float>(rest & ~63);
    const float low = __uint_as_float(0x4b000000u | (rest & 63)) - 8388608.f;  // the six bits
    const float z = __fmul_rn(x, kTurn);
    const float e = fmaf(low, kTurn, fmaf(x, kTurnLow, fmaf(x, kTurn, -z)));
    const float w = __fmul_rn(z, z), half = 0.5f * w;
    const float ps = fmaf(w, fmaf(w, fmaf(w, 1.f / 362880, -1.f / 5040), 1.f / 120), -1.f / 6);
    const float s = z + fmaf(z * w, ps, fmaf(-half, e, e));
    const float pc = fmaf(w, fmaf(w, fmaf(w, -1.f / 3628800, 1.f / 40320), -1.f / 720), 1.f / 24);
    const float c0 = 1.f - half, c1 = (1.f - c0) - half;
    const float lost = fmaf(z, e, 0.5f * fmaf(z, z, -w));
    const float c = c0 + fmaf(w * w, pc, c1 - lost);
    const float u = quarter & 1u ? s : c, v = quarter & 1u ? c : s;
    // quarter turns 0: (c, s)  1: (-s, c)  2: (-c, -s)  3: (s, -c)
    return make_float2((quarter == 1u || quarter == 2u) ? -u : u, quarter & 2u ? -v : v);
}

// The sequence of flattened token t: the largest b with offsets[b] <= t, by a
// warp-wide search (every lane returns it).  t lies below offsets[B].
__device__ __forceinline__ int find_sequence(const int *offsets, int B, long long t, int lane) {
    int lo = 0, n = B;  // the answer is in [lo, lo + n)
    while (n > 1) {
        const int step = (n + 31) / 32;
        const int i = lo + lane * step;
        const bool le = i < lo + n && __ldg(offsets + i) <= t;
        const int k = max(__popc(__ballot_sync(0xffffffffu, le)), 1) - 1;
        n = min(step, n - k * step);
        lo += k * step;
    }
    return lo;
}

// Tokens of a ragged batch that belong to a sequence.
__device__ __forceinline__ long long used_tokens(const int *offsets, int B, long long tokens) {
    return offsets ? min(tokens, max(0LL, static_cast<long long>(__ldg(offsets + B)))) : tokens;
}

// Channels of an item; 1: up to 16, one by one.
__host__ __device__ inline int item_width(int rope_dims, int D) {
    return (rope_dims | D) % 16 == 0 ? 16 : (rope_dims | D) % 8 == 0 ? 8 : (rope_dims | D) % 4 == 0 ? 4 : 1;
}
__host__ __device__ inline int rope_items(int rope_dims, int width) {
    return width > 1 ? rope_dims / width : (rope_dims / 2 + 7) / 8;
}
// Items of a row: the rotated ones, then those of the channels that pass through.
__host__ __device__ inline int row_items(int rope_dims, int D, int width) {
    return rope_items(rope_dims, width) + (width > 1 ? (D - rope_dims) / width : (D - rope_dims + 15) / 16);
}

// Pairs of an item, at most.
template <int N>
constexpr int kPairs = N == 1 ? 8 : N / 2;

// The elements of an item.
template <typename T, int N>
struct __align__(16) ItemData {
    T e[2 * kPairs<N>];
};

// fp32 values rounded to T.
template <int N>
__device__ __forceinline__ void round_item(const float *y, ItemData<__half, N> &x) {
    __half2 *h = reinterpret_cast<__half2 *>(x.e);
#pragma unroll
    for (int i = 0; i < kPairs<N>; ++i) h[i] = __floats2half2_rn(y[2 * i], y[2 * i + 1]);
}
template <int N>
__device__ __forceinline__ void round_item(const float *y, ItemData<__nv_bfloat16, N> &x) {
    __nv_bfloat162 *h = reinterpret_cast<__nv_bfloat162 *>(x.e);
#pragma unroll
    for (int i = 0; i < kPairs<N>; ++i) h[i] = __floats2bfloat162_rn(y[2 * i], y[2 * i + 1]);
}
template <int N>
__device__ __forceinline__ void round_item(const float *y, ItemData<float, N> &x) {
#pragma unroll
    for (int i = 0; i < 2 * kPairs<N>; ++i) x.e[i] = y[i];
}

// BYTES moved at once.
template <int BYTES>
struct PieceOf;
template <>
struct PieceOf<4> {
    using type = uint32_t;
};
template <>
struct PieceOf<8> {
    using type = uint2;
};
template <>
struct PieceOf<16> {
    using type = uint4;
};

__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(float x) { return x; }
template <typename T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ __half from_float<__half>(float x) {
    return __float2half_rn(x);
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) {
    return __float2bfloat16_rn(x);
}
template <>
__device__ __forceinline__ float from_float<float>(float x) {
    return x;
}

// Item j of a row of T.  Elements k = 0 .. 2 P - 1, P = kPairs<N>: in the half layout u
// of pair e is element e and w element e + P, in the interleaved one 2e and 2e + 1.
template <typename T, int N>
struct Item {
    static constexpr bool kVec = N > 1;
    static constexpr int P = kPairs<N>;
    static constexpr int kRuns = N * sizeof(T) > 32 ? 4 : 2, kRun = 2 * P / kRuns;
    static constexpr int kRunBytes = kVec ? kRun * static_cast<int>(sizeof(T)) : 16;
    using Run = typename PieceOf<kRunBytes>::type;
    int j, rope_dims, D;
    bool rot, trad;
    int first, hop;  // kVec: channel of run r: first + r hop; else two runs of eight
                     // channels at most, at first and first + hop, n0 and n1 long
    int n0, n1;

    __device__ __forceinline__ Item(int j_, int rope_dims_, int D_, bool trad_)
        : j(j_), rope_dims(rope_dims_), D(D_), trad(trad_) {
        const int ir = rope_items(rope_dims, N);
        rot = j < ir;
        if constexpr (kVec) {
            first = rot ? kRun * j : rope_dims + kRun * (j - ir);
            hop = (rot ? rope_dims : D - rope_dims) / kRuns;
            n0 = n1 = kRun;
        } else {
            const bool halves = rot && !trad;
            first = halves ? 8 * j : rot ? 16 * j : rope_dims + 16 * (j - ir);
            hop = halves ? rope_dims / 2 : 8;
            const int left = halves ? rope_dims / 2 - first : (rot ? rope_dims : D) - first;
            n0 = min(left, 8);
            n1 = halves ? n0 : min(max(left - 8, 0), 8);
        }
    }
    // The pair that slot e of item j rotates, or one past the last.
    static __device__ __forceinline__ int pair_of(int e, int j, int rope_dims, bool trad) {
        if constexpr (kVec) {
            const int k = trad ? 2 * e : e;
            const int c = k / kRun * (rope_dims / kRuns) + kRun * j + k % kRun;
            return trad ? c >> 1 : c;
        }
        return 8 * j + e;
    }
    __device__ __forceinline__ void load(const T *row, ItemData<T, N> &x) const {
        if constexpr (kVec) {
#pragma unroll
            for (int r = 0; r < kRuns; ++r)
                reinterpret_cast<Run *>(x.e)[r] = __ldg(reinterpret_cast<const Run *>(row + first + r * hop));
        } else {
            // without branches, so that all sixteen are in flight: what is past the
            // end of a run (which may be empty, but for the first) is read elsewhere
            const T *u = row + first, *w = n1 > 0 ? u + hop : u;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                x.e[k] = u[k < n0 ? k : 0];
                x.e[k + 8] = w[k < n1 ? k : 0];
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                x.e[k] = k < n0 ? x.e[k] : from_float<T>(0.f);
                x.e[k + 8] = k < n1 ? x.e[k + 8] : from_float<T>(0.f);
            }
        }
    }
    __device__ __forceinline__ void store(T *row, const ItemData<T, N> &x) const {
        if constexpr (kVec) {
#pragma unroll
            for (int r = 0; r < kRuns; ++r)
                *reinterpret_cast<Run *>(row + first + r * hop) = reinterpret_cast<const Run *>(x.e)[r];
        } else {
            T *u = row + first, *w = u + hop;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                if (k < n0) u[k] = x.e[k];
                if (k < n1) w[k] = x.e[k + 8];
            }
        }
    }
    // The elements in fp32, those of a rotated item turned by the (cos, sin) of its
    // slots, at table[0], table[items], ...
    __device__ __forceinline__ void values(const ItemData<T, N> &x, const float2 *table, int items,
                                           float *y) const {
        if (!rot) {
#pragma unroll
            for (int k = 0; k < 2 * P; ++k) y[k] = to_float(x.e[k]);
        } else if (trad) {
#pragma unroll
            for (int k = 0; k < P; ++k) {
                const float2 cs = table[k * items];
                const float u = to_float(x.e[2 * k]), w = to_float(x.e[2 * k + 1]);
                y[2 * k] = u * cs.x - w * cs.y;
                y[2 * k + 1] = u * cs.y + w * cs.x;
            }
        } else {
#pragma unroll
            for (int k = 0; k < P; ++k) {
                const float2 cs = table[k * items];
                const float u = to_float(x.e[k]), w = to_float(x.e[k + P]);
                y[k] = u * cs.x - w * cs.y;
                y[k + P] = u * cs.y + w * cs.x;
            }
        }
    }
};

// A thread's part in building the cos/sin tables of some positions, kPairs<N> * items entries
// each: slot e of item j at e * items + j, so that threads on neighbouring items read
// neighbouring entries.  The CTA's threads (a power of two, 256 or more) keep one slot
// each and go through the positions; the turn fraction, which neighbouring threads
// fetch from different places of the parameters, is fetched once.
template <typename T, int N>
struct RopeFiller {
    int entries, slot, row0, hop;  // row0 < 0: no part
    float mag_c, mag_s;
    unsigned long long frac;

    __device__ __forceinline__ RopeFiller(int items, const RopeTable &r, bool gradient)
        : entries(kPairs<N> * items), slot(0), row0(-1), hop(1), mag_c(r.magnitude),
          mag_s(gradient ? -r.magnitude : r.magnitude), frac(0) {
        if (items == 0) return;
        int lanes = 1;
        while (lanes < entries) lanes *= 2;
        slot = threadIdx.x & (lanes - 1);
        hop = blockDim.x / lanes;
        const int e = slot / items;
        const int pair = Item<T, N>::pair_of(e, slot - e * items, r.rope_dims, r.traditional != 0);
        if (slot < entries && pair < r.rope_dims / 2) {
            row0 = threadIdx.x / lanes;
            frac = r.turn_frac[pair];
        }
    }
    template <typename Pos>
    __device__ __forceinline__ void fill(float2 *table, int rows, Pos position) const {
        if (row0 < 0) return;
        for (int row = row0; row < rows; row += hop) {
            const float2 cs = turn_cos_sin(position(row), frac);
            table[row * entries + slot] = make_float2(cs.x * mag_c, cs.y * mag_s);
        }
    }
};

}  // namespace dattn
