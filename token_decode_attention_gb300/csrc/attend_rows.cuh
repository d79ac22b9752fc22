// attend_rows.cuh -- what the kernels of attention over a 16-bit cache share: which
// positions a token sees, where their rows lie, and one query head's attention by a warp.
//
// A token at position p sees [0, first) and [lo, p]: lo = max(0, p - window + 1) (0
// without a window) and first = min(sinks, lo).  The n = first + p + 1 - lo positions it
// sees are counted through: the i-th is i below `first` and i - first + lo from there on,
// so the kernels walk what is seen and nothing else.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "dattn_internal.h"
#include "ptx.cuh"

namespace dattn {
namespace attend {

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 16-bit types: two values of a word to fp32, two fp32 to a word (to nearest).  result: of
// outputs whose weights were rounded to the type while their sum was not, so that a mean of
// f16 values may come out up to 2^-11 too large, and infinite: no mean of finite values is
// beyond the largest one.
template <typename T>
struct Pair;
template <>
struct Pair<__half> {
    static __device__ __forceinline__ float2 wide(uint32_t w) {
        return __half22float2(*reinterpret_cast<const __half2 *>(&w));
    }
    static __device__ __forceinline__ uint32_t narrow(float x, float y) {
        const __half2 h = __floats2half2_rn(x, y);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    static constexpr float kLargest = 65504.f;
    static __device__ __forceinline__ float bounded(float x) {
        return fabsf(x) < INFINITY ? fminf(fmaxf(x, -kLargest), kLargest) : x;
    }
    static __device__ __forceinline__ uint32_t result(float x, float y) { return narrow(bounded(x), bounded(y)); }
};
template <>
struct Pair<__nv_bfloat16> {
    static __device__ __forceinline__ float2 wide(uint32_t w) {
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
    static __device__ __forceinline__ uint32_t narrow(float x, float y) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    static constexpr float kLargest = INFINITY;  // outputs that overflow did so in fp32
    static __device__ __forceinline__ float bounded(float x) { return x; }
    static __device__ __forceinline__ uint32_t result(float x, float y) { return narrow(x, y); }
};

struct Seen {
    int first, lo, end;  // [0, first) and [lo, end)
    __device__ __forceinline__ int count() const { return first + end - lo; }
    __device__ __forceinline__ int at(int i) const { return i < first ? i : i - first + lo; }
};

// Positions of sequence b: its last token's, plus one.
__device__ __forceinline__ int live_end(const AttendArgs &a, int b) {
    const uint32_t c = __ldg(a.cur_pos + b), top = static_cast<uint32_t>(a.S - a.own_base - 1);
    return a.own_base + static_cast<int>(c < top ? c : top) + 1;
}

// What a token at position p sees (nothing at a position before the first).
__device__ __forceinline__ Seen seen_by(const AttendArgs &a, int p) {
    Seen v;
    v.end = max(p + 1, 0);
    v.lo = a.window > 0 ? max(0, v.end - a.window) : 0;
    v.first = min(a.sinks, v.lo);
    return v;
}

// Row of position pos of sequence b in the cache (or in the tensor of the shared
// positions, where they have one), in rows of Hk x D elements.  A page outside the pool
// is recorded and page 0 read in its place.
__device__ __forceinline__ long long row_of(const AttendArgs &a, int b, int pos) {
    if (a.block_table == nullptr)
        return pos < a.own_base ? pos : static_cast<long long>(b) * (a.S - a.own_base) + (pos - a.own_base);
    const int pi = fast_div(pos, a.div_page);
    const int owner = pos < a.shared ? 0 : b;
    int page = __ldg(a.block_table + static_cast<long long>(owner) * a.max_pages + pi);
    if (page < 0 || page >= a.num_pages) {
        atomicOr(a.err, kErrPageIndex);
        page = 0;
    }
    return static_cast<long long>(page) * a.page_size + (pos - pi * a.page_size);
}

// The positions that some token of a group sees, counted: `window` from lo on, then the
// sinks from 0 on.
struct Counted {
    int lo, window;
    __device__ __forceinline__ int at(int i) const { return i < window ? lo + i : i - window; }
};

// State of one query head over the positions counted i0 .. i1-1 of `v` that its own token,
// which sees [0, sinks) and [lo, end), sees too: running
// maximum (log2 units), sum of weights and weighted values of channels 2 (lane + 32 c), by
// one warp, 32 positions at a time: a lane each for the scores, channels over the lanes for V.
struct RowState {
    float M, l, acc[4][2];
};
template <typename T>
__device__ void row_state(const AttendArgs &a, int b, int kvh, const T *q, Counted v, int i0, int i1, int lo, int end,
                          int lane, RowState &r) {
    constexpr unsigned kAll = 0xffffffffu;
    const long long head = static_cast<long long>(kvh) * a.D;
    const long long row_elems = static_cast<long long>(a.Hk) * a.D;
    r.M = -INFINITY;
    r.l = 0.f;
#pragma unroll
    for (int c = 0; c < 4; ++c) r.acc[c][0] = r.acc[c][1] = 0.f;
    for (; i0 < i1; i0 += 32) {
        const int i = i0 + lane;
        const int pos = v.at(i);
        const bool sees = i < i1 && pos < end && (pos >= lo || pos < a.sinks);
        float s = -INFINITY;
        long long at = 0;
        int apart = 0;
        if (sees) {
            apart = a.Kp != nullptr && pos < a.own_base;
            at = row_of(a, b, pos) * row_elems + head;
            const T *k = static_cast<const T *>(apart ? a.Kp : a.K) + at;
            float dot = 0.f;
            for (int c = 0; c < a.D; c += 8) {
                const uint4 kw = __ldg(reinterpret_cast<const uint4 *>(k + c));
                const uint4 qw = __ldg(reinterpret_cast<const uint4 *>(q + c));
                const uint32_t ks[4] = {kw.x, kw.y, kw.z, kw.w}, qs[4] = {qw.x, qw.y, qw.z, qw.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 x = Pair<T>::wide(ks[e]), y = Pair<T>::wide(qs[e]);
                    dot = fmaf(x.x, y.x, dot);
                    dot = fmaf(x.y, y.y, dot);
                }
            }
            s = dot * a.qscale;
        }
        const unsigned who = __ballot_sync(kAll, sees);
        float top = s;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
        const float nm = fmaxf(r.M, top), ref = nm == -INFINITY ? 0.f : nm;
        const float f = ex2(r.M - ref);  // 0 before the first
        const float p = sees ? ex2(s - ref) : 0.f;
        r.M = nm;
        r.l = fmaf(r.l, f, p);
#pragma unroll
        for (int c = 0; c < 4; ++c) r.acc[c][0] *= f, r.acc[c][1] *= f;
        // eight positions' loads in flight
#pragma unroll 1
        for (int j0 = 0; j0 < 32; j0 += 8) {
            if ((who >> j0 & 0xffu) == 0) continue;
            uint32_t x[8][4];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const long long row = __shfl_sync(kAll, at, j0 + u);
                const int there = __shfl_sync(kAll, apart, j0 + u);
                const T *vr = static_cast<const T *>(there ? a.Vp : a.V) + row;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int ch = 2 * (lane + 32 * c);
                    x[u][c] = (who >> (j0 + u) & 1) && ch < a.D ? __ldg(reinterpret_cast<const uint32_t *>(vr + ch)) : 0u;
                }
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const float w = __shfl_sync(kAll, p, j0 + u);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const float2 y = Pair<T>::wide(x[u][c]);
                    r.acc[c][0] = fmaf(w, y.x, r.acc[c][0]);
                    r.acc[c][1] = fmaf(w, y.y, r.acc[c][1]);
                }
            }
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) r.l += __shfl_xor_sync(kAll, r.l, o);
}

// Whether the value of position pos of sequence b holds something that is not finite.  Not
// inlined: hardly ever called, from a kernel whose code is large already (16384 tokens 1.60
// and 1.58 ms).
template <typename T>
__device__ __noinline__ bool value_not_finite(const AttendArgs &a, int b, int kvh, int pos) {
    const bool apart = a.Kp != nullptr && pos < a.own_base;
    const T *v = static_cast<const T *>(apart ? a.Vp : a.V) +
                 row_of(a, b, pos) * static_cast<long long>(a.Hk) * a.D + static_cast<long long>(kvh) * a.D;
    bool bad = false;
    for (int c = 0; c < a.D; c += 8) {
        const uint4 x = __ldg(reinterpret_cast<const uint4 *>(v + c));
        const uint32_t words[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 y = Pair<T>::wide(words[e]);
            bad |= !(fabsf(y.x) < INFINITY) || !(fabsf(y.y) < INFINITY);
        }
    }
    return bad;
}

}  // namespace attend
}  // namespace dattn
