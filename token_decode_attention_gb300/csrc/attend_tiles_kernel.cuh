// attend_tiles_kernel.cuh -- attention of many query rows at a time on the fifth-generation
// tensor cores: the tokens of prompts and mixed steps, or one token of each sequence over
// the positions that all share.
//
//   S = Q K^T,  P = 2^(S log2e / sqrt(D) - M),  O = sum P V,  out = O / sum P
// over 128 query rows (a token's query heads of one key/value head are neighbouring rows, so
// they share its keys) and key tiles of 128 (64 above 128 channels), M a running maximum.
// What bounds it: 4 D flops for each query row and key; a key tile is loaded once for 256 rows.
// P is rounded to the cache's type, the type of V's product (2^-8 or 2^-11 of a weight at most;
// the sum of weights keeps them unrounded): errors of many weights mostly cancel, the rms error
// of outputs is about 1.4 times what their own rounding makes, and a second part as in the
// one-token kernel would be half as many products again.
//
// Roles of a CTA's 12 warps, one CTA on an SM:
//   0-3, 4-7  softmax of the first and second 128 rows (the stacks): a thread a row.  S comes
//             from tensor memory, P goes back there in 16 bits over S; O stays there too
//             and is rescaled only when a maximum grows by more than 2^kTrigger, so most
//             tiles never touch it.
//   8-10      loads: K and V tiles into a ring of slots, Q once an item.  Tiles inside the
//             window are boxes of TMA (a whole tile of a dense cache, of a paged one as many
//             rows as divide a page), a stack's Q too where it is whole tokens.  Others are
//             16-byte cp.async of any rows (sinks, the item's end, odd pages): positions that
//             no row sees are not read and zero.
//   11        issues the products, one thread: S of the next tile while softmax works on
//             the last one, into the next item.
// While one stack's softmax runs, the tensor cores work for the other.
//
// Measured (graph replay): 16384 tokens, 32 heads on 8 of 128, bf16, 1.58 ms, 1390 TFLOP/s, 72 %
// of a large matrix product's burst; tensor pipe busy half of the cycles.  Bound by the chain
// S, softmax, P, V of a stack and its hand-overs, not by bytes: half of them loaded, or the
// softmax left out, it takes 1.5 ms.  Tried, ms: tiles by 16-byte copies 1.88, by TMA
// gathers of four rows 4.5; P handed over in halves 1.66, in quarters 1.72; registers
// shared evenly 1.86; every role's loops unrolled 2.0 (instruction fetch).  168 bytes of the
// softmax role's registers and up to 72 of the loads' are spilled.
//
// A hidden position gets weight zero; 0 times a V that is not finite still makes the row's
// O a NaN.  Where a position that some rows of a piece do not see holds such a value, the
// piece's rows with a NaN are computed again position by position (attend::row_state), which
// touches what they see only.  So are rows whose scores lie beyond kFar.
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
constexpr int kLoadWarps = 3, kThreads = 384;
// Time limit of a wait: a warp that computes 32 rows of a context of millions of positions
// again (below) keeps the other roles waiting for seconds.
constexpr unsigned long long kTileWaitLimitNs = 10 * kWaitLimitNs;
constexpr unsigned kNoRow = 0xffffffffu;  // zeros (a cache has fewer than 2^31 rows)
// The running maximum M is kept kHeadroom (log2) below the largest exponent when it was set
// and moved when one exceeds M + kTrigger: weights lie below 2^12 (f16 holds up to 65504)
// and the largest is at least 2^4, which keeps f16 weights normal down to 2^-18 of it.
constexpr float kHeadroom = 4.f, kTrigger = 12.f;
// An exponent is the exact product of score and scale less M, and M a rounded one: from
// scores of 2^26 on (log2 units), where fp32 goes in steps of 8, the largest exponent can
// pass f16's range.  Rows whose M reached kFar are computed again with the rounded score less
// M, as the one-token kernel does; below it the two differ by 2^-10 at most.
constexpr float kFar = 16384.f;

template <int DP>
struct TileShape {
    static constexpr int kStacks = tile_stacks(DP), kKeys = tile_keys(DP);
    static constexpr int kQBytes = 128 * DP * 2;       // of a stack
    static constexpr int kSlotBytes = kKeys * DP * 2;  // K or V of a tile
    static constexpr int kSlots = DP == 64 ? 8 : 5;    // what shared memory holds
    static constexpr int kColS = 0, kColO = 2 * kKeys;  // tensor memory columns
    static constexpr int kBars = 2 * kSlots + 11;
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

// The largest of three absolute values, NaN where one is.
__device__ __forceinline__ float max3_abs_nan(float a, float b, float c) {
    float d;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// What a row sees of an item's positions, in the item's count: of the `window` ones from
// the item's `lo` on those in [lo, end) and below `sinks`; the sinks behind them, up to n, all.
struct Edges {
    int lo, end, sinks, window, n;
    // The hidden ones of positions x0 .. x0 + 31, a bit each.
    __device__ __forceinline__ uint32_t hidden32(int x0) const {
        return range32(end - x0, window - x0) | range32(sinks - x0, min(lo, window) - x0) | ~below32(n - x0);
    }
    static __device__ __forceinline__ uint32_t below32(int k) { return k >= 32 ? ~0u : k <= 0 ? 0u : (1u << k) - 1u; }
    static __device__ __forceinline__ uint32_t range32(int k0, int k1) { return below32(k1) & ~below32(k0); }
    // Whether rows that all see this much see [x0, x1) in part.
    __device__ __forceinline__ bool cuts(int x0, int x1) const {
        const int w1 = min(x1, window);
        return w1 > max(end, x0) || (x0 < lo && min(w1, lo) > max(sinks, x0)) || x1 > n;
    }
};

// The row of the item's token `tok`.
__device__ __forceinline__ Edges edges_of(const AttendArgs &a, const TileArgs &t, const TileItem &it, int tok,
                                          bool uniform) {
    Edges e;
    e.window = it.n - it.first;
    e.n = it.n;
    if (uniform) {
        e.lo = 0;
        e.sinks = 0;
        e.end = t.bound_ends ? min(a.shared, attend::live_end(a, it.token + tok)) : a.shared;
        return e;
    }
    const Seen v = attend::seen_by(a, it.p0 + tok);
    e.lo = v.lo - it.lo;
    e.end = v.end - it.lo;
    e.sinks = max(a.sinks - it.lo, 0);
    return e;
}

template <typename T, int DP>
__global__ void __launch_bounds__(kThreads, 1) attend_tiles_kernel(const AttendArgs a, const TileArgs t,
                                                                  const __grid_constant__ TileMaps maps) {
    using Z = TileShape<DP>;
    constexpr int kKeys = Z::kKeys;
    constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
    extern __shared__ unsigned char smem_raw[];
    __shared__ uint64_t bars[Z::kBars];
    __shared__ uint32_t s_tmem;

    uint64_t *const kv_full = bars, *const kv_free = bars + Z::kSlots;
    uint64_t *const q_full = bars + 2 * Z::kSlots, *const q_free = q_full + 1;
    uint64_t *const s_two = q_full + 2;   // [2] S of a stack is there (items of two stacks)
    uint64_t *const s_one = q_full + 4;   // [2] S of a buffer is there (items of one)
    uint64_t *const o_done = q_full + 6;  // [2] O of a stack has its last tile (items of one stack: each)
    uint64_t *const drained = q_full + 8;
    uint64_t *const p_full = q_full + 9;  // [2] P of a buffer is there

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t q_smem = (smem_addr(smem_raw) + 1023u) & ~1023u;
    const uint32_t ring = q_smem + Z::kStacks * Z::kQBytes;

    if (warp == 11) tc::alloc(&s_tmem);
    if (tid == 0) {
        for (int i = 0; i < Z::kSlots; ++i) {
            mbar_init(kv_full + i, kLoadWarps);
            mbar_init(kv_free + i, 1);
        }
        mbar_init(q_full, kLoadWarps);
        mbar_init(q_free, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(s_two + i, 1);
            mbar_init(s_one + i, 1);
            mbar_init(p_full + i, 4);  // the stack's warps
            mbar_init(o_done + i, 1);
        }
        mbar_init(drained, 1);
        fence_barrier_init();
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
    if (!uniform && tid == kThreads - 1) {
        // an item whose first tiles are the CTA's before has its pieces merged by join_kernel
        TileCut cut{0, 0, -1, 0};
        if (some && cta > 0 && walk.x < walk.x1) {
            const int2 who = attend::holders(shares, walk.kvh, walk.at, walk.end);
            if (who.x == cta - 1 && who.y >= cta) cut = TileCut{walk.kvh, walk.item, who.x, who.y};
        }
        t.cuts[cta] = cut;
    }

    // A wait that ran out is recorded; every role then leaves its loop, warps as a whole.
    auto wait = [&](uint64_t *bar, uint32_t parity, unsigned code) {
        if (mbar_wait_bounded(bar, parity, kTileWaitLimitNs)) return true;
        atomicOr(a.err, code);
        return false;
    };
    auto wait_warp = [&](uint64_t *bar, uint32_t parity, unsigned code) {
        return __all_sync(kFull, wait(bar, parity, code)) != 0;
    };
    auto stacks_of = [&](const TileItem &it) { return Z::kStacks == 2 && it.rows > 128 ? 2 : 1; };
    // What rows [r0, r1) of the item all see.
    auto seen_by_all = [&](const TileItem &it, int r0, int r1, int min_end) {
        const Edges first = edges_of(a, t, it, fast_div(it.head + r0, t.div_group), uniform);
        Edges last = edges_of(a, t, it, fast_div(it.head + r1 - 1, t.div_group), uniform);
        last.end = uniform ? min_end : first.end;
        return last;
    };

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
        uint32_t n_two = 0, n_one[2] = {0, 0}, n_o = 0, base = 0;
        bool ok = true;
        while (ok && some && walk.next(t, shares)) {
            const TileItem it = attend::item_of(a, t, shares, tile_rows(DP), walk.item);
            const int stacks = stacks_of(it);
            const uint32_t begun = base;  // steps of the CTA before the item's
            base += stacks * (walk.j1 - walk.j0);
            if (stack >= stacks) continue;
            const int r0 = stack * 128, r1 = min(it.rows, r0 + 128);
            const int tok = fast_div(it.head + r0 + row, t.div_group);
            const bool mine = r0 + row < it.rows;
            Edges e{0, 0, 0, it.n, it.n};
            if (mine) e = edges_of(a, t, it, tok, uniform);
            int min_end = a.shared;
            if (uniform && t.bound_ends) {
                min_end = mine ? e.end : a.shared;
                min_end = __reduce_min_sync(kFull, min_end);  // of the warp's own rows
            }
            const Edges all = seen_by_all(it, r0, r1, min_end);
            float M = -INFINITY, l = 0.f;
            bool hidden = false;  // some row of the warp does not see some position
            bool far = false;     // the row's M was beyond kFar
            for (int j = walk.j0; j < walk.j1; ++j) {
                const int n = j - walk.j0;
                const int buf = (begun + (stacks == 2 ? stack : n)) & 1;
                uint64_t *const full = stacks == 2 ? s_two + stack : s_one + buf;
                uint32_t &phase = stacks == 2 ? n_two : n_one[buf];
                if (!(ok = wait_warp(full, phase & 1, kErrConsumerWait))) break;
                ++phase;
                tc::fence_after();
                const uint32_t col_s = tmem + lanes + Z::kColS + buf * kKeys;
                // The loads bring the row's maximum along.  Tiles with hidden positions, a few
                // of an item, are masked in a small loop of their own, in tensor memory:
                // code that is large in all roles together starves for instructions.
                uint32_t sv[kKeys];
                const int x0 = j * kKeys;
                if (all.cuts(x0, x0 + kKeys)) {
                    hidden = true;
#pragma unroll 1
                    for (int c = 0; c < kKeys; c += 32) {
                        tc::ld32(sv, col_s + c);
                        const uint32_t h = e.hidden32(x0 + c);
                        tc::wait_ld();
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            if (h >> k & 1) sv[k] = 0xff800000u;  // -infinity
                        tc::st32(col_s + c, sv);
                    }
                    tc::wait_st();
                }
                float m[kKeys / 32];
#pragma unroll
                for (int c = 0; c < kKeys / 32; ++c) m[c] = tc::ld32_max(sv + 32 * c, col_s + 32 * c);
                tc::wait_ld();
                float top = fmaxf(m[0], m[1]);
                if constexpr (kKeys == 128) top = max3(top, m[2], m[3]);
                top *= a.qscale;
                // With one stack the last product with V may still run, with two it is done:
                // this S was issued behind it.
                bool running = stacks == 1 && n > 0;
                n_o += running;
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
                    far |= fabsf(nm) >= kFar && nm != -INFINITY;
                    if (running && !product_done()) break;
                    if (n > 0) {
#pragma unroll 1
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
                for (int part = 0; part < kKeys; part += 32) {
#pragma unroll
                    for (int c = part; c < part + 32; c += 2) {
                        float2 p = fma2(make_float2(__uint_as_float(sv[c]), __uint_as_float(sv[c + 1])), scale2, ref2);
                        p.x = ex2(p.x);
                        p.y = ex2(p.y);
                        l2[(c >> 1) & 1] = add2(l2[(c >> 1) & 1], p);
                        sv[c / 2] = Pair<T>::narrow(p.x, p.y);
                    }
                    tc::st16(col_s + part / 2, sv + part / 2);  // over S
                }
                tc::wait_st();
                if (running && !product_done()) break;  // its phases are not to be passed over
                tc::fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full + buf);
                l2[0] = add2(l2[0], l2[1]);
                l += l2[0].x + l2[0].y;
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
            bool nan = false;
            const float inv = e.end > 0 ? 1.f / l : 0.f;
            float *const state = uniform && whole ? t.whole_acc + out_row * a.D : t.acc + slot_row * a.D;
            float2 *const state_ml = uniform && whole ? t.whole_ml + out_row : t.ml + slot_row;
            const bool to_out = whole && !uniform;
#pragma unroll 1
            for (int c = 0; c < DP; c += 32) {
                if (c >= a.D) break;
                uint32_t o[32];
                tc::ld32(o, col_o + c);
                tc::wait_ld();
                if (!mine) continue;
                float big = 0.f;  // the largest absolute value, NaN where one is
#pragma unroll
                for (int k = 0; k < 32; k += 8)
                    if (c + k < a.D)
#pragma unroll
                        for (int h = k; h < k + 8; h += 2)
                            big = max3_abs_nan(big, __uint_as_float(o[h]), __uint_as_float(o[h + 1]));
                nan |= big != big;
                if (!to_out) {
#pragma unroll
                    for (int k = 0; k < 32; k += 8)
                        if (c + k < a.D) st_global_v8(state + c + k, o + k);
                    continue;
                }
                T *const out = static_cast<T *>(a.out) + out_row * a.D + c;
                float times = inv;
                if (!kBf16 && big * inv > Pair<T>::kLargest) {  // rare: see Pair::result
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(Pair<T>::bounded(__uint_as_float(o[k]) * inv));
                    times = 1.f;
                }
#pragma unroll
                for (int k = 0; k < 32; k += 2)
                    o[k / 2] = Pair<T>::narrow(__uint_as_float(o[k]) * times, __uint_as_float(o[k + 1]) * times);
#pragma unroll
                for (int k = 0; k < 32; k += 16) {
                    if (t.out_32 && c + k + 8 < a.D) {
                        st_global_v8(out + k, o + k / 2);
                        continue;
                    }
#pragma unroll
                    for (int h = 0; h < 16; h += 8)
                        if (c + k + h < a.D)
                            *reinterpret_cast<uint4 *>(out + k + h) =
                                make_uint4(o[(k + h) / 2], o[(k + h) / 2 + 1], o[(k + h) / 2 + 2], o[(k + h) / 2 + 3]);
                }
            }
            tc::fence_before();  // O has been read before the next item's first P is handed over
            if (mine && !to_out) *state_ml = make_float2(M, l);
            // A sum of weights that is NaN comes of a score that the row sees, and all of its
            // outputs are; other NaN may come of a hidden value, where there is one.
            bool doubt = mine && nan && l == l;
            if (hidden && __any_sync(kFull, doubt)) {
                bool bad = false;
                for (int x = walk.j0 * kKeys; x < walk.j1 * kKeys && !bad; x += 32) {
                    const unsigned h = all.hidden32(x);
                    const bool there = x + lane < it.n && (h >> lane & 1) != 0;
                    const attend::Counted counted{it.lo, it.n - it.first};
                    if (h != 0) bad = __any_sync(kFull, there && attend::value_not_finite<T>(a, it.b, kvh, counted.at(x + lane)));
                }
                doubt &= bad;
            } else {
                doubt = false;
            }
            unsigned again = __ballot_sync(kFull, mine && (far || doubt));
            if (again != 0) {
                // position by position, a row after the other, over what was just written
                __syncwarp();
                const int i0 = walk.j0 * kKeys, i1 = min(it.n, walk.j1 * kKeys);
                for (; again != 0; again &= again - 1) {
                    const int r = __ffs(again) - 1;
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
                                         attend::Counted{it.lo, it.n - it.first}, i0, i1, lo, end, lane, y);
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
        const int blocks = (a.D + 63) / 64;      // 64-channel blocks
        constexpr int CPR = DP / 8;              // chunks of a full row
        constexpr int kLanesRow = CPR < 32 ? CPR : 32, kRowsCopy = 32 / kLanesRow;
        constexpr int kCopies = 16 / kRowsCopy;  // warp-wide copies of 16 rows
        const int crow = lane / kLanesRow, cc = lane % kLanesRow;
        const bool in_row = cc < chunks, in_head = cc * 8 < a.D;
        // the warp's copies so far are done, and what it had to do for the tile
        auto arrive = [&](uint64_t *bar) {
            cp_async_hold(bar);
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
        };
        int number = 0;
        uint32_t used = 0;  // slots handed out
        bool ok = true;
        while (ok && some && walk.next(t, shares)) {
            const TileItem it = attend::item_of(a, t, shares, tile_rows(DP), walk.item);
            const int stacks = stacks_of(it);
            const attend::Counted counted{it.lo, it.n - it.first};
            const unsigned row_bytes = static_cast<unsigned>(a.Hk) * a.D * 2;
            const size_t col = (static_cast<size_t>(walk.kvh) * a.D + (in_head ? cc * 8 : 0)) * 2;
            const unsigned char *const from_k = static_cast<const unsigned char *>(a.Kp ? a.Kp : a.K) + col;
            const unsigned char *const from_v = static_cast<const unsigned char *>(a.Kp ? a.Vp : a.V) + col;
            for (int j = walk.j0; j < walk.j1 && ok; ++j) {
                constexpr int kGroups = (kKeys / 16 + kLoadWarps - 1) / kLoadWarps;
                const bool boxes = maps.box_rows > 0 && (j + 1) * kKeys <= counted.window;
                unsigned at[kGroups][kCopies];
                int box_row = 0;
                if (boxes) {
                    // lane l of the first warp: the first row of the tile's l-th box
                    if (lw == 0 && lane * maps.box_rows < kKeys)
                        box_row = static_cast<int>(
                            attend::row_of(a, it.b, counted.at(j * kKeys + lane * maps.box_rows)));
                } else {
                    // the rows that this lane copies from, of each of the warp's groups of 16
#pragma unroll
                    for (int i = 0; i < kGroups; ++i) {
                        const int g = lw + i * kLoadWarps;
                        const int x = j * kKeys + g * 16 + (lane & 15);
                        unsigned row = kNoRow;
                        if (g < kKeys / 16 && x < it.n)
                            row = static_cast<unsigned>(attend::row_of(a, it.b, counted.at(x)));
#pragma unroll
                        for (int c = 0; c < kCopies; ++c) {
                            at[i][c] = __shfl_sync(kFull, row, c * kRowsCopy + crow);
                            if (!in_head) at[i][c] = kNoRow;
                        }
                    }
                }
#pragma unroll 1
                for (int kv = 0; kv < 2; ++kv) {
                    const int slot = used % Z::kSlots;
                    const uint32_t round = used / Z::kSlots;
                    ++used;
                    if (round > 0 && !(ok = wait_warp(kv_free + slot, (round - 1) & 1, kErrProducerWait))) break;
                    const uint32_t tile = ring + slot * Z::kSlotBytes;
                    if (boxes) {
                        if (lane == 0) {
                            if (lw == 0) mbar_arrive_expect_tx(kv_full + slot, blocks * kKeys * 128);
                            else mbar_arrive(kv_full + slot);
                        }
                        __syncwarp();
                        if (lw == 0 && lane * maps.box_rows < kKeys)
                            for (int c = 0; c < blocks; ++c)
                                box_g2s(tile + c * (kKeys * 128) + lane * maps.box_rows * 128,
                                        kv == 0 ? &maps.k : &maps.v, c * 64, walk.kvh, box_row, kv_full + slot);
                        continue;
                    }
                    const unsigned char *const from = kv == 0 ? from_k : from_v;
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
                    arrive(kv_full + slot);
                }
                if (!ok) break;
                if (j > walk.j0) continue;
                // the item's queries, behind its first tile: the last item's products may still
                // read theirs
                if (number > 0 && !(ok = wait_warp(q_free, (number - 1) & 1, kErrProducerWait))) break;
                ++number;
                if (maps.q_tokens > 0) {
                    // a stack is whole tokens: 64 channels of its rows are a box
                    if (lane == 0) {
                        if (lw == 0) mbar_arrive_expect_tx(q_full, stacks * blocks * 128 * 128);
                        else mbar_arrive(q_full);
                    }
                    __syncwarp();
                    if (lw == 0 && lane < stacks * blocks) {
                        const int st = lane / blocks, c = lane - st * blocks;
                        box_g2s(q_smem + st * Z::kQBytes + c * (128 * 128), &maps.q, c * 64, walk.kvh * a.group,
                                it.token + st * maps.q_tokens, q_full);
                    }
                    continue;
                }
                for (int g = lw; g < stacks * 8; g += kLoadWarps) {
                    // 16 rows: lane l (and l + 16) finds row l's address, 0 for zeros
                    const int r = g * 16 + (lane & 15);
                    unsigned long long row = 0;
                    if (r < it.rows) {
                        const int tok = fast_div(it.head + r, t.div_group);
                        const int h = walk.kvh * a.group + (it.head + r - tok * a.group);
                        row = reinterpret_cast<unsigned long long>(a.Q) +
                              ((it.token + static_cast<long long>(tok)) * a.q_stride + static_cast<long long>(h) * a.D) * 2;
                    }
                    const uint32_t tile = q_smem + (g >> 3) * Z::kQBytes;
                    unsigned long long from[kCopies];
#pragma unroll
                    for (int i = 0; i < kCopies; ++i) from[i] = __shfl_sync(kFull, row, i * kRowsCopy + crow);
                    if (!in_row) continue;
#pragma unroll
                    for (int i = 0; i < kCopies; ++i) {
                        const bool there = from[i] != 0 && in_head;
                        cp_async16(tile + swizzled(128, (g & 7) * 16 + i * kRowsCopy + crow, cc),
                                   there ? reinterpret_cast<const void *>(from[i] + cc * 16) : a.Q, there ? 16 : 0);
                    }
                }
                arrive(q_full);
            }
        }
        // what was asked for has arrived before the shared memory is given up
        cp_async_commit();
        cp_async_wait<0>();
        if (number > 0) wait_warp(q_full, (number - 1) & 1, kErrDrainWait);
        for (int i = 0; i < Z::kSlots; ++i) {
            const uint32_t rounds = (used + Z::kSlots - 1 - i) / Z::kSlots;
            if (rounds > 0) wait_warp(kv_full + i, (rounds - 1) & 1, kErrDrainWait);
        }
    } else {
        // ---------------------------------------------------------- products
        if (tc::elect_one()) {
            constexpr uint32_t kIdescS = tc::instr_desc(128, kKeys, kBf16, false);
            const uint32_t idesc_o = tc::instr_desc(128, (a.D + 15) / 16 * 16, kBf16, true);
            const int ksteps = (a.D + 15) / 16;
            const uint32_t q_desc = tc::smem_desc(q_smem, 0), k_desc = tc::smem_desc(ring, 0);
            const uint32_t v_desc = tc::smem_desc(ring, kKeys * 128);
            // Steps are a tile of a stack.  Scores run two steps ahead of values and into the
            // next item: while softmax works on an item's last tiles, the first products of
            // the next are under way.  A step has the buffer of its parity in the CTA.
            struct Steps {
                attend::Walk walk;
                int stacks, left;  // of the item; steps to come
                int stack, first;  // the next step's; whether its tile is the piece's first
                uint32_t buf, use;  // its buffer; its tile's use of the ring
            };
            auto begin = [&](Steps &x) {  // the next item, if there is one
                if (!some || !x.walk.next(t, shares)) return false;
                x.stacks = stacks_of(attend::item_of(a, t, shares, tile_rows(DP), x.walk.item));
                x.left = x.stacks * (x.walk.j1 - x.walk.j0);
                x.stack = 0;
                x.first = 1;
                return true;
            };
            auto arrived = [&](uint32_t use) {
                if (!wait(kv_full + use % Z::kSlots, use / Z::kSlots & 1, kErrConsumerWait)) return false;
                tc::fence_async();  // what cp.async wrote is visible to the tensor cores
                tc::fence_after();
                return true;
            };
            auto step_done = [&](Steps &x) {
                x.buf ^= 1;
                --x.left;
                if (++x.stack < x.stacks) return;
                tc::commit(kv_free + x.use % Z::kSlots);
                x.use += 2;
                x.stack = 0;
                x.first = 0;
            };
            Steps sc{walk, 1, 0, 0, 1, 0, 0}, va{walk, 1, 0, 0, 1, 0, 1};
            uint32_t p_phase = 0;  // bit b: parity of buffer b's next P
            int ahead = 0, number = 0;
            bool more = some;
            while (true) {
                if (ahead < 2 && more) {
                    if (sc.left == 0) {
                        if (!(more = begin(sc))) continue;
                        if (!wait(q_full, number++ & 1, kErrConsumerWait)) break;
                    }
                    if (sc.stack == 0 && !arrived(sc.use)) break;
                    uint32_t qd = q_desc + sc.stack * (Z::kQBytes >> 4);
                    uint32_t kd = k_desc + sc.use % Z::kSlots * (Z::kSlotBytes >> 4);
                    const uint32_t to = tmem + Z::kColS + sc.buf * kKeys;
#pragma unroll 1
                    for (int k = 0; k < ksteps; k += 4) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (k + i < ksteps) tc::mma(to, qd + 2 * i, kd + 2 * i, kIdescS, k + i > 0);
                        qd += 128 * 128 >> 4;
                        kd += kKeys * 128 >> 4;
                    }
                    tc::commit(sc.stacks == 2 ? s_two + sc.stack : s_one + sc.buf);
                    step_done(sc);
                    if (sc.left == 0) tc::commit(q_free);
                    ++ahead;
                } else if (ahead > 0) {
                    if (va.left == 0 && !begin(va)) break;
                    if (va.stack == 0 && !arrived(va.use)) break;
                    uint32_t vd = v_desc + va.use % Z::kSlots * (Z::kSlotBytes >> 4);
                    uint32_t from = tmem + Z::kColS + va.buf * kKeys;
                    const uint32_t to = tmem + Z::kColO + va.stack * DP, phase = p_phase >> va.buf & 1;
                    p_phase ^= 1u << va.buf;
                    if (!wait(p_full + va.buf, phase, kErrConsumerWait)) break;
                    tc::fence_after();
#pragma unroll 1
                    for (int k = 0; k < kKeys / 16; k += 2) {
                        tc::mma_tmem(to, from, vd, idesc_o, k > 0 || !va.first);
                        tc::mma_tmem(to, from + 8, vd + (2048 >> 4), idesc_o, 1);
                        from += 16;
                        vd += 4096 >> 4;
                    }
                    if (va.stacks == 1 || va.left <= 2) tc::commit(o_done + va.stack);  // a stack's last
                    step_done(va);
                    --ahead;
                } else {
                    break;
                }
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
