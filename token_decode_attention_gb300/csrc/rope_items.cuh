// rope_items.cuh -- the pieces of a head row that the rotary kernels work on.
//
// A row of D channels, the first rope_dims of them rotated in pairs, is cut
// into items of 16 channels, one thread each: an item holds eight pairs (u, w),
// channels (i, i + rope_dims/2) in the half layout and (2i, 2i + 1) in the
// interleaved one, or 16 channels that pass through.  In either layout an
// item is two runs of eight channels, so a thread reads 16-byte vectors and
// needs no other thread's data.  VEC: rope_dims and D are multiples of 16, and
// the runs are whole vectors; otherwise the elements are read one by one.
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
// either way, which a float holds to 2^-27 of a half turn; sincospif of the
// rest, then the quarter turns by exchange and sign.  The error is that of
// sincospif plus 2.4e-8 rad at every position.
__device__ __forceinline__ float2 turn_cos_sin(uint32_t p, unsigned long long f) {
    const uint32_t turn =
        static_cast<uint32_t>((static_cast<unsigned long long>(p) * f) >> 32);
    const uint32_t quarter = (turn + 0x20000000u) >> 30;
    const int rest = static_cast<int>(turn - (quarter << 30));
    float s, c;
    sincospif(static_cast<float>(rest) * 0x1p-31f, &s, &c);
    const float x = quarter & 1u ? s : c, y = quarter & 1u ? c : s;
    // quarter turns 0: (c, s)  1: (-s, c)  2: (-c, -s)  3: (s, -c)
    return make_float2((quarter == 1u || quarter == 2u) ? -x : x, quarter & 2u ? -y : y);
}

__host__ __device__ inline int rope_items(int rope_dims, bool vec) {
    return vec ? rope_dims / 16 : (rope_dims / 2 + 7) / 8;
}
// Items of a row: the rotated ones, then those of the channels that pass through.
__host__ __device__ inline int row_items(int rope_dims, int D, bool vec) {
    return rope_items(rope_dims, vec) + (D - rope_dims + 15) / 16;
}

// Sixteen elements of an item: runs x[0..7] and x[8..15].
template <typename T>
struct ItemData {
    uint4 v[sizeof(T)];
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

// Item j of a row.
template <bool VEC>
struct Item {
    int j, rope_dims, D;
    bool rot, trad;
    int o0, o1;  // VEC: first channels of the two runs

    __device__ __forceinline__ Item(int j_, int rope_dims_, int D_, bool trad_)
        : j(j_), rope_dims(rope_dims_), D(D_), trad(trad_) {
        const int ir = rope_items(rope_dims, VEC);
        rot = j < ir;
        if (rot) {
            o0 = trad ? 16 * j : 8 * j;
            o1 = trad ? o0 + 8 : rope_dims / 2 + o0;
        } else {
            o0 = rope_dims + 16 * (j - ir);
            o1 = o0 + 8;
        }
    }
    // Channel of element k, or -1 past the item's end (the scalar form).
    __device__ __forceinline__ int channel(int k) const {
        if (!rot) return o0 + k < D ? o0 + k : -1;
        const int half = rope_dims / 2;
        const int pair = 8 * j + (trad ? k >> 1 : k & 7);
        if (pair >= half) return -1;
        return trad ? 2 * pair + (k & 1) : pair + (k >> 3) * half;
    }
    template <typename T>
    __device__ __forceinline__ void load(const T *row, ItemData<T> &x) const {
        if constexpr (VEC) {
            constexpr int N = sizeof(T) / 2;
            const uint4 *a = reinterpret_cast<const uint4 *>(row + o0);
            const uint4 *b = reinterpret_cast<const uint4 *>(row + o1);
#pragma unroll
            for (int i = 0; i < N; ++i) x.v[i] = a[i], x.v[N + i] = b[i];
        } else {
            T *e = reinterpret_cast<T *>(x.v);
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const int c = channel(k);
                e[k] = c >= 0 ? row[c] : from_float<T>(0.f);
            }
        }
    }
    template <typename T>
    __device__ __forceinline__ void store(T *row, const ItemData<T> &x) const {
        if constexpr (VEC) {
            constexpr int N = sizeof(T) / 2;
            uint4 *a = reinterpret_cast<uint4 *>(row + o0);
            uint4 *b = reinterpret_cast<uint4 *>(row + o1);
#pragma unroll
            for (int i = 0; i < N; ++i) a[i] = x.v[i], b[i] = x.v[N + i];
        } else {
            const T *e = reinterpret_cast<const T *>(x.v);
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const int c = channel(k);
                if (c >= 0) row[c] = e[k];
            }
        }
    }
};

// The sixteen elements in fp32, rotated by (cos, sin) = cs[e] of pair e.
template <bool VEC, typename T>
__device__ __forceinline__ void rotate_item(const Item<VEC> &it, const ItemData<T> &x,
                                            const float2 *cs, float *y) {
    const T *e = reinterpret_cast<const T *>(x.v);
    if (!it.rot) {
#pragma unroll
        for (int k = 0; k < 16; ++k) y[k] = to_float(e[k]);
    } else if (it.trad) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float u = to_float(e[2 * k]), w = to_float(e[2 * k + 1]);
            y[2 * k] = u * cs[k].x - w * cs[k].y;
            y[2 * k + 1] = u * cs[k].y + w * cs[k].x;
        }
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float u = to_float(e[k]), w = to_float(e[k + 8]);
            y[k] = u * cs[k].x - w * cs[k].y;
            y[k + 8] = u * cs[k].y + w * cs[k].x;
        }
    }
}

// cos/sin table of one position: pair 8 j + e at index e * items + j, so that
// threads on neighbouring items read neighbouring entries.
__device__ __forceinline__ void rope_table_entry(float2 *table, int items, int i, uint32_t pos,
                                                 const RopeTable &r, bool gradient) {
    float2 cs = turn_cos_sin(pos, r.turn_frac[i]);
    cs.x *= r.magnitude;
    cs.y *= gradient ? -r.magnitude : r.magnitude;
    table[(i & 7) * items + (i >> 3)] = cs;
}

}  // namespace dattn
