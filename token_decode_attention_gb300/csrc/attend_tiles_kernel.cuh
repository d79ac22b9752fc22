// attend_tiles_kernel.cuh -- attention of many query rows at a time on the fifth-generation
// tensor cores: the tokens of prompts and mixed steps, or one token of each sequence over
// the positions that all share.
//
//   S = Q K^T,  P = 2^(S log2e / sqrt(D) - M),  O = sum P V,  out = O / sum P
// over 128 query rows (a token's query heads of one key/value head are neighbouring rows, so
// they share its keys) and key tiles of 128 (64 above 128 channels), M a running maximum.
// What bounds it: 4 D flops for each query row and key; a key tile is loaded once for 256 rows.
//
// Roles of a CTA's 12 warps, one CTA on an SM:
//   0-3, 4-7  softmax of the first and second 128 rows (the stacks): a thread a row.  S comes
//             from tensor memory, P goes back there in 16 bits over S; O stays there too
//             and is rescaled only when a maximum grows by more than 2^kTrigger, so most
//             tiles never touch it.
//   8-10      loads: cp.async of 16 bytes into swizzled tiles, a ring of slots for K and V.
//             Row addresses may be any (pages, sinks ahead of a window), positions that no
//             row sees are not read and zero.
//   11        issues the products: S of the next tile while softmax works on the last one.
// While one stack's softmax runs, the tensor cores work for the other.
//
// A hidden position gets weight zero; 0 times a V that is not finite would still reach the
// row.  The loading warps look for such values in tiles that some row sees in part (no
// other tile can hold a hidden one); where there are any, the piece's rows are computed
// again position by position (attend::row_state), which touches what they see only.
//
// Work split: attend_tiles.cuh.  Pieces of items leave their states to the merge kernels.
#pragma once

#include <type_traits>

#include "attend_tiles.cuh"
#include "tcgen05.cuh"

namespace dattn {
namespace {

using attend::ex2;
using attend::Pair;
using attend::Seen;

constexpr unsigned kFull = 0xffffffffu;
constexpr int kSoftmaxThreads = 128;  // of a stack
constexpr int kLoadWarps = 3, kThreads = 384;
constexpr unsigned kNoRow = 0xffffffffu;  // zeros (a cache has fewer than 2^31 rows)
// The running maximum M is kept kHeadroom (log2) below the largest exponent when it was set
// and moved when one exceeds M + kTrigger: weights lie below 2^12 (f16 holds up to 65504)
// and the largest is at least 2^4, which keeps f16 weights normal down to 2^-18 of it.
constexpr float kHeadroom = 4.f, kTrigger = 12.f;

template <int DP>
struct TileShape {
    static constexpr int kStacks = tile_stacks(DP), kKeys = tile_keys(DP);
    static constexpr int kBlocks = DP / 64;            // 64-channel blocks of a row
    static constexpr int kQBytes = 128 * DP * 2;       // of a stack
    static constexpr int kSlotBytes = kKeys * DP * 2;  // K or V of a tile
    static constexpr int kSlots = DP == 64 ? 8 : DP == 128 ? 5 : 5;
    static constexpr int kColS = 0, kColO = 2 * kKeys;  // tensor memory columns
    static constexpr int kBars = 2 * kSlots + 16;
    static constexpr int kSmem = kStacks * kQBytes + kSlots * kSlotBytes + 1024;
};

// Byte offset of 16-byte chunk c of row r in a tile of blocks of `rows` rows.
__device__ __forceinline__ uint32_t swizzled(int rows, int r, int c) {
    return (c >> 3) * (rows * 128) + r * 128 + (((c ^ r) & 7) << 4);
}

// Pairs of fp32 in one instruction; the largest of three (NaN left aside).
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    unsigned long long x, y, z, r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b.x), "f"(b.y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(z) : "f"(c.x), "f"(c.y));
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
    float2 d;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(r));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    unsigned long long x, y, r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b.x), "f"(b.y));
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    float2 d;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(r));
    return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// Whether a word holds a 16-bit value whose exponent is all ones.
template <typename T>
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
    if constexpr (std::is_same<T, __half>::value) return ((w & 0x7c007c00u) + 0x04000400u) & 0x80008000u;
    return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
}

// Hidden positions of an item's rows, in the item's count: a row sees i < end that is at
// least `lo` or below `sinks`.
struct Edges {
    int lo, end, sinks;
    __device__ __forceinline__ bool hides(int i) const { return i >= end || (i < lo && i >= sinks); }
};

// A row of token `tok` rows behind the item's first one.
__device__ __forceinline__ Edges edges_of(const AttendArgs &a, const TileArgs &t, const TileItem &it, int tok,
                                          bool uniform) {
    Edges e;
    if (uniform) {
        e.lo = 0;
        e.sinks = 0;
        e.end = t.bound_ends ? min(a.shared, attend::live_end(a, it.token + tok)) : a.shared;
        return e;
    }
    const int shift = it.first - it.lo;  // position to count, from `lo` on
    const Seen v = attend::seen_by(a, it.p0 + tok);
    e.lo = v.lo + shift;
    e.end = v.end + shift;
    // sinks past the item's `lo` are seen by rows whose window has moved past them
    e.sinks = a.sinks > it.lo ? a.sinks + shift : it.first;
    return e;
}

template <typename T, int DP>
__global__ void __launch_bounds__(kThreads, 1) attend_tiles_kernel(const AttendArgs a, const TileArgs t) {
    using Z = TileShape<DP>;
    constexpr int kKeys = Z::kKeys;
    constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
    extern __shared__ unsigned char smem_raw[];
    __shared__ uint64_t bars[Z::kBars];
    __shared__ uint32_t s_tmem;
    __shared__ int s_bad[4];  // number of the last item (modulo 4) with values that are not finite

    uint64_t *const kv_full = bars, *const kv_free = bars + Z::kSlots;
    uint64_t *const q_full = bars + 2 * Z::kSlots, *const q_free = q_full + 1;
    uint64_t *const s_two = q_full + 2;   // [2] S of a stack is there (items of two stacks)
    uint64_t *const s_one = q_full + 4;   // [2] S of a buffer is there (items of one)
    uint64_t *const p_full = q_full + 6;  // [2] P of a buffer is there
    uint64_t *const o_done = q_full + 8;  // [2] O of a stack has its last tile
    uint64_t *const drained = q_full + 10;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t q_smem = (smem_addr(smem_raw) + 1023u) & ~1023u;
    const uint32_t ring = q_smem + Z::kStacks * Z::kQBytes;

    if (warp == 11) tc::alloc(&s_tmem);
    if (tid == 0) {
        for (int i = 0; i < Z::kSlots; ++i) {
            mbar_init(kv_full + i, kLoadWarps * 32);
            mbar_init(kv_free + i, 1);
        }
        mbar_init(q_full, kLoadWarps * 32);
        mbar_init(q_free, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(s_two + i, 1);
            mbar_init(s_one + i, 1);
            mbar_init(p_full + i, kSoftmaxThreads);
            mbar_init(o_done + i, 1);
        }
        mbar_init(drained, 1);
        fence_barrier_init();
        s_bad[0] = s_bad[1] = s_bad[2] = s_bad[3] = -1;
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = s_tmem;
    pdl_wait_primary();
    pdl_launch_dependents();

    const attend::Shares shares = attend::shares_of(a, t, DP);
    const bool uniform = shares.uniform != 0;
    const int cta = blockIdx.x;
    attend::Walk walk{};
    const bool some = cta < shares.ctas && shares.items > 0;
    if (some) walk.start(t, shares, cta);

    // A wait that ran out is recorded; every role then leaves its loop, warps as a whole.
    auto wait = [&](uint64_t *bar, uint32_t parity, unsigned code) {
        if (mbar_wait_bounded(bar, parity, kWaitLimitNs)) return true;
        atomicOr(a.err, code);
        return false;
    };
    auto wait_warp = [&](uint64_t *bar, uint32_t parity, unsigned code) {
        return __all_sync(kFull, wait(bar, parity, code)) != 0;
    };
    auto stacks_of = [&](const TileItem &it) { return Z::kStacks == 2 && it.rows > 128 ? 2 : 1; };
    // What rows [r0, r1) of the item all see; a tile that goes past it is hidden in part.
    auto seen_by_all = [&](const TileItem &it, int r0, int r1, int min_end) {
        if (uniform) return Edges{0, min_end, 0};
        const Edges first = edges_of(a, t, it, fast_div(it.head + r0, t.div_group), false);
        Edges last = edges_of(a, t, it, fast_div(it.head + r1 - 1, t.div_group), false);
        last.end = first.end;
        return last;
    };
    auto in_part = [&](const Edges &all, int x0, int x1) {
        return x1 > all.end || (x0 < all.lo && x1 > all.sinks);
    };

    // A softmax thread holds a row's scores of a tile; the registers come from the others:
    // 256 x 200 + 128 x 104 = 384 x 168, what the launch gave.
    if (warp < 8)
        asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    else
        asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    if (warp < 8) {
        // ------------------------------------------------------------ softmax
        const int stack = warp >> 2, row = tid & 127;
        const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // lane 32 (warp % 4)
        const uint32_t col_o = tmem + lanes + Z::kColO + stack * DP;
        uint32_t n_two = 0, n_one[2] = {0, 0}, n_o = 0;
        int number = 0;
        bool ok = true;
        while (ok && some && walk.next(t, shares)) {
            const int my_number = number++;
            const TileItem it = attend::item_of(a, t, shares, tile_rows(DP), walk.item);
            const int stacks = stacks_of(it);
            if (stack >= stacks) continue;
            const int r0 = stack * 128, r1 = min(it.rows, r0 + 128);
            const int tok = fast_div(it.head + r0 + row, t.div_group);
            const bool mine = r0 + row < it.rows;
            Edges e{0, 0, 0};
            if (mine) e = edges_of(a, t, it, tok, uniform);
            int min_end = a.shared;
            if (uniform && t.bound_ends) {
                min_end = mine ? e.end : a.shared;
                min_end = __reduce_min_sync(kFull, min_end);  // of the warp's own rows
            }
            const Edges all = seen_by_all(it, r0, r1, min_end);
            float M = -INFINITY, l = 0.f;
            for (int j = walk.j0; j < walk.j1; ++j) {
                const int n = j - walk.j0;
                const int buf = stacks == 2 ? stack : n & 1;
                uint64_t *const full = stacks == 2 ? s_two + stack : s_one + buf;
                uint32_t &phase = stacks == 2 ? n_two : n_one[buf];
                if (!(ok = wait_warp(full, phase & 1, kErrConsumerWait))) break;
                ++phase;
                tc::fence_after();
                const uint32_t col_s = tmem + lanes + Z::kColS + buf * kKeys;
                uint32_t sv[kKeys];
#pragma unroll
                for (int c = 0; c < kKeys; c += 32) tc::ld32(sv + c, col_s + c);
                tc::wait_ld();
                const int x0 = j * kKeys;
                if (in_part(all, x0, x0 + kKeys)) {
#pragma unroll
                    for (int c = 0; c < kKeys; ++c)
                        if (e.hides(x0 + c)) sv[c] = 0xff800000u;  // -infinity
                }
                float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int c = 0; c < kKeys; c += 2)
                    m4[(c >> 1) & 3] = max3(m4[(c >> 1) & 3], __uint_as_float(sv[c]), __uint_as_float(sv[c + 1]));
                const float top = max3(fmaxf(m4[0], m4[1]), m4[2], m4[3]) * a.qscale;
                // With one stack the last product with V may still run, with two it is done:
                // this S was issued behind it.
                bool running = stacks == 1 && n > 0;
                n_o += n > 0;
                auto product_done = [&]() {
                    running = false;
                    ok = wait_warp(o_done + stack, (n_o - 1) & 1, kErrConsumerWait);
                    tc::fence_after();
                    return ok;
                };
                const bool grow = top > M + kTrigger;
                if (__any_sync(kFull, grow)) {
                    const float nm = fmaxf(M, top - kHeadroom);
                    const float f = M == -INFINITY ? 0.f : ex2(M - nm);
                    M = nm;
                    l *= f;
                    if (running && !product_done()) break;
                    if (n > 0) {
#pragma unroll
                        for (int c = 0; c < DP; c += 32) {
                            if (c >= a.D) break;
                            uint32_t o[32];
                            tc::ld32(o, col_o + c);
                            tc::wait_ld();
#pragma unroll
                            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                            tc::st32(col_o + c, o);
                        }
                    }
                }
                const float ref = M == -INFINITY ? 0.f : M;
                const float2 scale2 = make_float2(a.qscale, a.qscale), ref2 = make_float2(-ref, -ref);
                float2 l2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int c = 0; c < kKeys; c += 2) {
                    float2 p = fma2(make_float2(__uint_as_float(sv[c]), __uint_as_float(sv[c + 1])), scale2, ref2);
                    p.x = ex2(p.x);
                    p.y = ex2(p.y);
                    l2[(c >> 1) & 1] = add2(l2[(c >> 1) & 1], p);
                    sv[c / 2] = Pair<T>::narrow(p.x, p.y);
                }
                l2[0] = add2(l2[0], l2[1]);
                l += l2[0].x + l2[0].y;
#pragma unroll
                for (int c = 0; c < kKeys / 2; c += 32) tc::st32(col_s + c, sv + c);
                tc::wait_st();
                if (running && !product_done()) break;  // its phases are not to be passed over
                tc::fence_before();
                mbar_arrive(p_full + buf);
            }
            if (!ok) break;
            // ---- the piece's rows ----
            if (!(ok = wait_warp(o_done + stack, n_o & 1, kErrConsumerWait))) break;
            ++n_o;
            tc::fence_after();
            const bool whole = walk.begins && walk.ends;
            const int kvh = walk.kvh;
            const int q_head = it.head + r0 + row - tok * a.group;
            const long long token = it.token + static_cast<long long>(tok);
            const long long out_row = token * a.H + static_cast<long long>(kvh) * a.group + q_head;
            const long long slot_row =
                static_cast<long long>(2 * cta + (walk.begins ? 1 : 0)) * tile_rows(DP) + r0 + row;
            const bool bad = *const_cast<volatile int *>(&s_bad[my_number & 3]) == my_number;
            const float inv = e.end > 0 ? 1.f / l : 0.f;
            float *const state = uniform && whole ? t.whole_acc + out_row * a.D : t.acc + slot_row * a.D;
            float2 *const state_ml = uniform && whole ? t.whole_ml + out_row : t.ml + slot_row;
            const bool to_out = whole && !uniform;
#pragma unroll
            for (int c = 0; c < DP; c += 32) {
                if (c >= a.D) break;
                uint32_t o[32];
                tc::ld32(o, col_o + c);
                tc::wait_ld();
                if (!mine || bad) continue;
#pragma unroll
                for (int k = 0; k < 32; k += 8) {
                    if (c + k >= a.D) break;
                    float y[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) y[i] = __uint_as_float(o[k + i]);
                    if (to_out) {
                        uint4 w;
                        w.x = Pair<T>::narrow(y[0] * inv, y[1] * inv);
                        w.y = Pair<T>::narrow(y[2] * inv, y[3] * inv);
                        w.z = Pair<T>::narrow(y[4] * inv, y[5] * inv);
                        w.w = Pair<T>::narrow(y[6] * inv, y[7] * inv);
                        *reinterpret_cast<uint4 *>(static_cast<T *>(a.out) + out_row * a.D + c + k) = w;
                    } else {
                        *reinterpret_cast<float4 *>(state + c + k) = make_float4(y[0], y[1], y[2], y[3]);
                        *reinterpret_cast<float4 *>(state + c + k + 4) = make_float4(y[4], y[5], y[6], y[7]);
                    }
                }
            }
            tc::fence_before();  // O has been read before the next item's first P is handed over
            if (mine && !bad && !to_out) *state_ml = make_float2(M, l);
            if (bad) {
                // position by position, a row after the other of the warp's
                const Seen counted{it.first, it.lo, it.lo + it.n - it.first};
                const int i0 = walk.j0 * kKeys, i1 = min(it.n, walk.j1 * kKeys);
                for (int r = 0; r < 32; ++r) {
                    if (r0 + (row & 96) + r >= it.rows) break;
                    const int rtok = __shfl_sync(kFull, tok, r), rhead = __shfl_sync(kFull, q_head, r);
                    const long long rtoken = it.token + static_cast<long long>(rtok);
                    const int h = kvh * a.group + rhead;
                    int lo = 0, end = __shfl_sync(kFull, e.end, r);
                    if (!uniform) {
                        const Seen v = attend::seen_by(a, it.p0 + rtok);
                        lo = v.lo;
                        end = v.end;
                    }
                    attend::RowState y;
                    attend::row_state<T>(a, it.b, kvh,
                                         static_cast<const T *>(a.Q) + rtoken * a.q_stride +
                                             static_cast<long long>(h) * a.D,
                                         counted, i0, i1, lo, end, lane, y);
                    const long long row_out = rtoken * a.H + h;
                    const long long row_slot = __shfl_sync(kFull, slot_row, r);
                    float *const to = uniform && whole ? t.whole_acc + row_out * a.D : t.acc + row_slot * a.D;
                    const float rinv = end > 0 ? 1.f / y.l : 0.f;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int ch = 2 * (lane + 32 * c);
                        if (ch >= a.D) continue;
                        if (to_out)
                            *reinterpret_cast<uint32_t *>(static_cast<T *>(a.out) + row_out * a.D + ch) =
                                Pair<T>::narrow(y.acc[c][0] * rinv, y.acc[c][1] * rinv);
                        else
                            *reinterpret_cast<float2 *>(to + ch) = make_float2(y.acc[c][0], y.acc[c][1]);
                    }
                    if (lane == 0 && !to_out)
                        *(uniform && whole ? t.whole_ml + row_out : t.ml + row_slot) = make_float2(y.M, y.l);
                }
            }
        }
    } else if (warp < 8 + kLoadWarps) {
        // ------------------------------------------------------------ loads
        const int lw = warp - 8;
        const int chunks = (a.D + 15) / 16 * 2;  // 16-byte chunks of a row that the products read
        constexpr int CPR = DP / 8;              // of a full row
        constexpr int kLanesRow = CPR < 32 ? CPR : 32, kRowsCopy = 32 / kLanesRow;
        const int crow = lane / kLanesRow, cc = lane % kLanesRow;
        int number = 0;
        bool ok = true;
        // Whether this lane's own copies of a tile hold a value that is not finite.
        auto look_through = [&](int slot) {
            const uint32_t base = ring + slot * Z::kSlotBytes;
            uint32_t any = 0;
            for (int g = lw; g < kKeys / 16; g += kLoadWarps)
#pragma unroll 4
                for (int i = 0; i < 16 / kRowsCopy; ++i) {
                    if (cc >= chunks) continue;
                    const uint4 w = lds128(base + swizzled(kKeys, g * 16 + i * kRowsCopy + crow, cc));
                    any |= not_finite<T>(w.x) | not_finite<T>(w.y) | not_finite<T>(w.z) | not_finite<T>(w.w);
                }
            return any != 0;
        };
        constexpr int kCopies = 16 / kRowsCopy;  // warp-wide copies of 16 rows
        const bool in_row = cc < chunks, in_head = cc * 8 < a.D;
        // 16 rows from r0 on; lane l (and l + 16) knows row l's address, or nullptr for zeros
        auto copy16 = [&](uint32_t tile, int rows, int r0, const unsigned char *row) {
            unsigned long long p[kCopies];
#pragma unroll
            for (int i = 0; i < kCopies; ++i)
                p[i] = __shfl_sync(kFull, reinterpret_cast<unsigned long long>(row), i * kRowsCopy + crow);
            if (!in_row) return;
#pragma unroll
            for (int i = 0; i < kCopies; ++i) {
                const bool there = p[i] != 0 && in_head;
                const void *src = there ? reinterpret_cast<const void *>(p[i] + cc * 16) : a.Q;
                cp_async16(tile + swizzled(rows, r0 + i * kRowsCopy + crow, cc), src, there ? 16 : 0);
            }
        };
        uint32_t used = 0;  // slots handed out
        while (ok && some && walk.next(t, shares)) {
            const int my_number = number++;
            const TileItem it = attend::item_of(a, t, shares, tile_rows(DP), walk.item);
            const int stacks = stacks_of(it);
            if (my_number > 0 && !(ok = wait_warp(q_free, (my_number - 1) & 1, kErrProducerWait))) break;
            for (int g = lw; g < stacks * 8; g += kLoadWarps) {
                const int r = g * 16 + (lane & 15);
                const unsigned char *row = nullptr;
                if (r < it.rows) {
                    const int tok = fast_div(it.head + r, t.div_group);
                    const int h = walk.kvh * a.group + (it.head + r - tok * a.group);
                    row = static_cast<const unsigned char *>(a.Q) +
                          ((it.token + static_cast<long long>(tok)) * a.q_stride + static_cast<long long>(h) * a.D) * 2;
                }
                copy16(q_smem + (g >> 3) * Z::kQBytes, 128, (g & 7) * 16, row);
            }
            cp_async_arrive(q_full);
            int min_end = a.shared;
            if (uniform && t.bound_ends) {
                const int toks = fast_div(it.head + it.rows - 1, t.div_group) + 1;
                for (int k = lane; k < toks; k += 32) min_end = min(min_end, attend::live_end(a, it.token + k));
                min_end = __reduce_min_sync(kFull, min_end);
            }
            const Seen counted{it.first, it.lo, it.lo + it.n - it.first};
            const Edges all = seen_by_all(it, 0, it.rows, min_end);
            const unsigned row_bytes = static_cast<unsigned>(a.Hk) * a.D * 2;
            const size_t col = (static_cast<size_t>(walk.kvh) * a.D + (in_head ? cc * 8 : 0)) * 2;
            const unsigned char *const from_k = static_cast<const unsigned char *>(a.Kp ? a.Kp : a.K) + col;
            const unsigned char *const from_v = static_cast<const unsigned char *>(a.Kp ? a.Vp : a.V) + col;
            for (int j = walk.j0; j < walk.j1 && ok; ++j) {
                // the rows that this lane copies from, of each of the warp's groups of 16
                constexpr int kGroups = (kKeys / 16 + kLoadWarps - 1) / kLoadWarps;
                unsigned at[kGroups][kCopies];
#pragma unroll
                for (int i = 0; i < kGroups; ++i) {
                    const int g = lw + i * kLoadWarps;
                    const int x = j * kKeys + g * 16 + (lane & 15);
                    unsigned row = kNoRow;
                    if (g < kKeys / 16 && x < it.n) row = static_cast<unsigned>(attend::row_of(a, it.b, counted.at(x)));
#pragma unroll
                    for (int c = 0; c < kCopies; ++c) {
                        at[i][c] = __shfl_sync(kFull, row, c * kRowsCopy + crow);
                        if (!in_head) at[i][c] = kNoRow;
                    }
                }
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
                    const int slot = used % Z::kSlots;
                    const uint32_t round = used / Z::kSlots;
                    ++used;
                    if (round > 0 && !(ok = wait_warp(kv_free + slot, (round - 1) & 1, kErrProducerWait))) break;
                    const unsigned char *const from = kv == 0 ? from_k : from_v;
                    const uint32_t tile = ring + slot * Z::kSlotBytes;
#pragma unroll
                    for (int i = 0; i < kGroups; ++i) {
                        const int g = lw + i * kLoadWarps;
                        if (g >= kKeys / 16 || !in_row) break;
#pragma unroll
                        for (int c = 0; c < kCopies; ++c) {
                            const bool there = at[i][c] != kNoRow;
                            const unsigned row = there ? at[i][c] : 0u;
                            cp_async16(tile + swizzled(kKeys, g * 16 + c * kRowsCopy + crow, cc),
                                       from + static_cast<size_t>(row) * row_bytes, there ? 16 : 0);
                        }
                    }
                    if (kv == 1 && in_part(all, j * kKeys, min(it.n, (j + 1) * kKeys))) {
                        cp_async_commit();
                        cp_async_wait<0>();
                        if (look_through(slot)) *const_cast<volatile int *>(&s_bad[my_number & 3]) = my_number;
                        mbar_arrive(kv_full + slot);
                    } else {
                        cp_async_arrive(kv_full + slot);
                    }
                }
            }
        }
        cp_async_commit();
        cp_async_wait<0>();
    } else {
        // ---------------------------------------------------------- products
        if (tc::elect_one()) {
            constexpr uint32_t kIdescS = tc::instr_desc(128, kKeys, kBf16, false);
            const uint32_t idesc_o = tc::instr_desc(128, (a.D + 15) / 16 * 16, kBf16, true);
            const int ksteps = (a.D + 15) / 16;
            const uint64_t q_desc = tc::smem_desc(q_smem, 0), k_desc = tc::smem_desc(ring, 0);
            const uint64_t v_desc = tc::smem_desc(ring, kKeys * 128);
            uint32_t used = 0, n_p[2] = {0, 0};
            int number = 0;
            bool ok = true;
            while (ok && some && walk.next(t, shares)) {
                const TileItem it = attend::item_of(a, t, shares, tile_rows(DP), walk.item);
                const int stacks = stacks_of(it);
                const int steps = stacks * (walk.j1 - walk.j0);
                auto scores = [&](int n) {
                    const int j = stacks == 2 ? n >> 1 : n, stack = stacks == 2 ? n & 1 : 0, buf = n & 1;
                    const uint32_t u = used + 2 * j;
                    const int slot = u % Z::kSlots;
                    if (stack == 0 && !wait(kv_full + slot, (u / Z::kSlots) & 1, kErrConsumerWait)) return false;
                    tc::fence_async();  // what the copies wrote is visible to the tensor cores
                    tc::fence_after();
                    const uint64_t qd = q_desc + stack * (Z::kQBytes >> 4), kd = k_desc + slot * (Z::kSlotBytes >> 4);
                    const uint32_t to = tmem + Z::kColS + buf * kKeys;
#pragma unroll
                    for (int k = 0; k < DP / 16; ++k) {
                        if (k >= ksteps) break;
                        tc::mma(to, qd + (((k >> 2) * (128 * 128) + (k & 3) * 32) >> 4),
                                kd + (((k >> 2) * (kKeys * 128) + (k & 3) * 32) >> 4), kIdescS, k > 0);
                    }
                    tc::commit((stacks == 2 ? s_two : s_one) + buf);
                    if (stack == stacks - 1) tc::commit(kv_free + slot);
                    if (n == steps - 1) tc::commit(q_free);
                    return true;
                };
                auto values = [&](int n) {
                    const int j = stacks == 2 ? n >> 1 : n, stack = stacks == 2 ? n & 1 : 0, buf = n & 1;
                    const uint32_t u = used + 2 * j + 1;
                    const int slot = u % Z::kSlots;
                    if (stack == 0 && !wait(kv_full + slot, (u / Z::kSlots) & 1, kErrConsumerWait)) return false;
                    if (!wait(p_full + buf, n_p[buf] & 1, kErrConsumerWait)) return false;
                    ++n_p[buf];
                    tc::fence_async();
                    tc::fence_after();
                    const uint64_t vd = v_desc + slot * (Z::kSlotBytes >> 4);
                    const uint32_t to = tmem + Z::kColO + stack * DP, from = tmem + Z::kColS + buf * kKeys;
#pragma unroll
                    for (int k = 0; k < kKeys / 16; ++k)
                        tc::mma_tmem(to, from + k * 8, vd + k * (2048 >> 4), idesc_o, j > 0 || k > 0);
                    tc::commit(o_done + stack);
                    if (stack == stacks - 1) tc::commit(kv_free + slot);
                    return true;
                };
                ok = wait(q_full, number & 1, kErrConsumerWait) && scores(0) && (steps < 2 || scores(1));
                for (int n = 0; n < steps && ok; ++n) ok = values(n) && (n + 2 >= steps || scores(n + 2));
                used += 2 * (walk.j1 - walk.j0);
                ++number;
            }
            // nothing runs on when the tensor memory is given back
            tc::commit(drained);
            wait(drained, 0, kErrDrainWait);
        }
        __syncwarp();
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (warp == 11) tc::dealloc(tmem);
}

}  // namespace
}  // namespace dattn
