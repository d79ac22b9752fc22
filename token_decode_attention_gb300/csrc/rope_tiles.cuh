// rope_tiles.cuh -- the rotation of many tokens, by equal runs of tiles per CTA: all of
// rope.cu, and the queries of append_q8_kernel.cuh.
//
// What bounds it: each element is read once and written once, 3 flops each; the
// cosines depend on (token, pair) only.  The items of all tokens, flattened, are cut
// into tiles of one per thread and every resident CTA takes an equal run of tiles:
// while it rotates and stores one, the next ones are on their way into a ring in
// shared memory (each thread copies, waits for and reads its own items), and the
// cos/sin table of the next one's tokens is built in the other half of a double
// buffer, from positions fetched one tile earlier still.  Measured (graph replay): 8192
// tokens of 32 heads of 128 in bf16, 134 MB, 24.2 us, 5.5 TB/s; 4095 of 40 heads in f32,
// half of each rotated, 168 MB, 29.9 us, 5.6 TB/s (a copy of 4 GB runs at 6.8).
#pragma once

#include <cuda_runtime.h>

#include "dattn_internal.h"
#include "ptx.cuh"
#include "rope_items.cuh"

namespace dattn {
namespace {

constexpr int kRopeThreads = 256;
// A thread's share of a tile is the same item of HP neighbouring heads: their cosines
// are fetched once and the bookkeeping of a tile is paid once.
// Bytes of a tile, stages of the ring and CTAs of an SM, which keep up to 190 KB of
// an SM's shared memory and its registers busy.
template <typename T, int N, int HP>
constexpr int kTileBytes = kRopeThreads * HP * static_cast<int>(sizeof(ItemData<T, N>::e));
template <typename T, int N, int HP>
constexpr int kStages = N == 1 ? 0 : kTileBytes<T, N, HP> > 16384 ? 2 : kTileBytes<T, N, HP> < 8192 ? 4 : 3;
template <typename T, int N, int HP>
constexpr int kRopeBlocks = N == 16 && HP == 4 ? 2 : N == 16 && sizeof(T) == 4 ? 3 : 4;
template <typename T, int N, int HP>
constexpr int kRingBytes = kStages<T, N, HP> * kTileBytes<T, N, HP>;

struct RopeGrid {
    long long tiles;
    int items, per_token;  // items of a row; of a token, HP heads in one
    int max_tokens;        // tokens that a tile may touch
    FastDiv div_token;
};

// FIXED: a thread's item is the same in every tile (the items of a row divide the
// threads), so what depends on it is computed once.
// CTA `cta` of `ctas` (kRopeThreads threads) rotates its run of tiles; smem: rope_smem()
// bytes.
template <typename T, int N, bool FIXED, int HP>
__device__ __forceinline__ void rope_tiles(const RopeArgs &a, const RopeTable &rope, const RopeGrid &gr,
                                           unsigned cta, unsigned ctas, unsigned char *smem,
                                           uint32_t (*s_pos)[kRopeThreads]) {
    using It = Item<T, N>;
    constexpr int kRing = kStages<T, N, HP>;
    constexpr bool kVec = It::kVec;
    // behind the ring: [2][max_tokens][pairs of an item * rotated items]
    float2 *const table = reinterpret_cast<float2 *>(smem + kRingBytes<T, N, HP>);
    const int D = a.D, rd = rope.rope_dims, tid = threadIdx.x;
    const bool trad = rope.traditional != 0;
    const int ir = rope_items(rd, N), entries = kPairs<N> * ir;
    // token numbers fit 31 bits
    const int used = static_cast<int>(used_tokens(a.offsets, a.B, a.tokens));
    const int first = static_cast<int>(gr.tiles * cta / ctas);
    const int count = static_cast<int>(gr.tiles * (cta + 1) / ctas) - first;

    // Tokens and places are carried from tile to tile: 256 items on are step_tokens
    // tokens, step_heads heads and step_items items on, with carries.
    const int step_tokens = kRopeThreads / gr.per_token, step_in = kRopeThreads - step_tokens * gr.per_token;
    const int step_heads = step_in / gr.items, step_items = FIXED ? 0 : step_in - step_heads * gr.items;
    // A tile's first token and the place of its first item in that token.
    struct Tile {
        int token, skip;
    } cur;
    auto next = [&](Tile &t) {
        t.token += step_tokens;
        t.skip += step_in;
        if (t.skip >= gr.per_token) {
            t.skip -= gr.per_token;
            ++t.token;
        }
    };
    // This thread's item, and the first elements of its row in x and out.
    struct Place {
        int token, head, item;
        const T *x;
        T *out;
    } p;
    const long long x_step = step_tokens * a.x_stride + static_cast<long long>(step_heads) * (HP * D);
    const long long x_wrap = a.x_stride - static_cast<long long>(a.H) * D;
    const long long out_step = step_tokens * a.out_stride + static_cast<long long>(step_heads) * (HP * D);
    const long long out_wrap = a.out_stride - static_cast<long long>(a.H) * D;
    const int heads = a.H / HP;
    auto step = [&](Place &q) {
        q.head += step_heads;
        q.token += step_tokens;
        q.x += x_step;
        q.out += out_step;
        if constexpr (!FIXED) {
            q.item += step_items;
            if (q.item >= gr.items) {
                q.item -= gr.items;
                ++q.head;
                q.x += HP * D;
                q.out += HP * D;
            }
        }
        if (q.head >= heads) {
            q.head -= heads;
            ++q.token;
            q.x += x_wrap;
            q.out += out_wrap;
        }
    };
    {
        const long long n = static_cast<long long>(first) * kRopeThreads, t = n / gr.per_token;
        cur = Tile{static_cast<int>(t), static_cast<int>(n - t * gr.per_token)};
        const int in = cur.skip + tid, whole = in / gr.per_token, rest = in - whole * gr.per_token;
        p.token = cur.token + whole;
        p.head = rest / gr.items;
        p.item = rest - p.head * gr.items;
        p.x = reinterpret_cast<const T *>(a.x) + p.token * a.x_stride + static_cast<long long>(p.head) * (HP * D);
        p.out = reinterpret_cast<T *>(a.out) + p.token * a.out_stride + static_cast<long long>(p.head) * (HP * D);
    }
    // Position of the tile's token number tid.  In a ragged batch the thread keeps
    // the sequence it found last: [lo, hi) its tokens, the position of token t
    // being from + t.
    int lo = 0, hi = 0;
    uint32_t from = 0;  // modulo 2^32, as positions are
    auto position = [&](const Tile &t) -> uint32_t {
        if (tid >= gr.max_tokens) return 0;
        const int n = t.token + tid;
        if (n >= used) return 0;
        if (a.positions != nullptr) return __ldg(a.positions + n);
        if (a.offsets == nullptr) return __ldg(a.cur_pos + n);
        if (n < lo || n >= hi) {
            int b = 0, e = a.B;  // the largest b with offsets[b] <= n
            while (e - b > 1) {
                const int m = (b + e) / 2;
                if (__ldg(a.offsets + m) <= n) b = m;
                else e = m;
            }
            lo = __ldg(a.offsets + b);
            hi = __ldg(a.offsets + b + 1);
            from = __ldg(a.cur_pos + b) - static_cast<uint32_t>(hi) + 1u;
        }
        return from + static_cast<uint32_t>(n);
    };
    const RopeFiller<T, N> filler(ir, rope, a.gradient != 0);
    auto fill = [&](const Tile &t, int half) {
        const int touched = min(gr.max_tokens, fast_div(t.skip + kRopeThreads - 1, gr.div_token) + 1);
        filler.fill(table + half * gr.max_tokens * entries, touched, [&](int s) { return s_pos[half][s]; });
    };
    const It fixed(p.item, rd, D, trad);
    auto item_of = [&](const Place &x) {
        if constexpr (FIXED) return fixed;
        return It(x.item, rd, D, trad);
    };
    // run r of head h of this thread's item in a stage of the ring
    auto slot = [&](int stage, int h, int r) {
        return (((stage * HP + h) * It::kRuns + r) * kRopeThreads + tid) * It::kRunBytes;
    };
    const uint32_t ring = smem_addr(smem);
    auto fetch = [&](const Place &q, int stage) {
        if (q.token < used) {
            const It it = item_of(q);
            const T *x = q.x + it.first;
#pragma unroll
            for (int h = 0; h < HP; ++h)
#pragma unroll
                for (int r = 0; r < It::kRuns; ++r)
                    cp_async<It::kRunBytes>(ring + slot(stage, h, r), x + h * D + r * it.hop);
        }
    };

    if (count <= 0) return;
    Place pf = p;  // the item that is fetched next
    if constexpr (kVec) {
#pragma unroll
        for (int i = 0; i < kRing - 1; ++i) {
            if (i < count) fetch(pf, i);
            cp_async_commit();
            step(pf);
        }
    }
    Tile ahead = cur;
    s_pos[0][tid] = position(cur);
    next(ahead);
    s_pos[1][tid] = position(ahead);
    __syncthreads();
    fill(cur, 0);
    __syncthreads();
    int stage = 0;
    for (int k = 0; k < count; ++k) {
        const int half = k & 1;
        if constexpr (kVec) {
            const int into = stage == 0 ? kRing - 1 : stage - 1;
            if (k + kRing - 1 < count) fetch(pf, into);
            cp_async_commit();
            step(pf);
            cp_async_wait<kRing - 1>();
        }
        next(ahead);  // two tiles on
        const uint32_t pos = k + 2 < count ? position(ahead) : 0u;
        if (p.token < used) {
            const It it = item_of(p);
            const float2 *const entry = table + (half * gr.max_tokens + p.token - cur.token) * entries + it.j;
            float2 cs[kPairs<N>];
            if (it.rot) {
#pragma unroll
                for (int e = 0; e < kPairs<N>; ++e) cs[e] = entry[e * ir];
            }
#pragma unroll
            for (int h = 0; h < HP; ++h) {
                ItemData<T, N> d;
                if constexpr (kVec) {
#pragma unroll
                    for (int r = 0; r < It::kRuns; ++r)
                        reinterpret_cast<typename It::Run *>(d.e)[r] =
                            *reinterpret_cast<const typename It::Run *>(smem + slot(stage, h, r));
                } else {
                    it.load(p.x + h * D, d);
                }
                float y[2 * kPairs<N>];
                it.values(d, cs, 1, y);
                round_item(y, d);
                it.store(p.out + h * D, d);
            }
        }
        if constexpr (kVec) stage = stage + 1 == kRing ? 0 : stage + 1;
        if (k + 1 == count) break;
        step(p);
        next(cur);
        fill(cur, half ^ 1);
        if (tid < gr.max_tokens) s_pos[half][tid] = pos;  // last read before the barrier before this one
        __syncthreads();
    }
}

// The launch of rows of `elem_bytes`: the heads of a thread, as many as divide the heads
// (at most `most`) and leave every SM two CTAs, and the cut of the tokens into tiles.
inline bool rope_grid(long long tokens, int H, int D, int rope_dims, int most, int sms, RopeGrid *gr,
                      int *hp, int width, bool *fixed) {
    gr->items = row_items(rope_dims, D, width);
    if (static_cast<long long>(H) * gr->items > (1 << 30) || tokens > 0x7ffffc00LL) return false;
    *fixed = kRopeThreads % gr->items == 0;
    *hp = width > 1 ? most : 1;
    while (*hp > 1 && (H % *hp != 0 || tokens * H * gr->items < 2LL * sms * kRopeThreads * *hp)) *hp /= 2;
    gr->per_token = H / *hp * gr->items;
    gr->tiles = (tokens * gr->per_token + kRopeThreads - 1) / kRopeThreads;
    if (gr->tiles > 0x7fffffffLL) return false;
    gr->max_tokens = kRopeThreads % gr->per_token == 0 ? kRopeThreads / gr->per_token
                                                       : (kRopeThreads - 2) / gr->per_token + 2;
    gr->div_token = fast_div_of(gr->per_token);
    return true;
}

// What a kernel that may need more than the default limit asks for: one value for all
// its launches, so that threads that launch it at the same time agree.  With the static
// part (16 KB at most) below the 227 KB of a CTA.
constexpr int kMaxDynamicSmem = 208 * 1024;

// Shared memory behind a ring of `ring_bytes`: two tables of at most (256 / items + 2)
// tokens of 8 entries for 16 channels, 36 KB.
inline size_t rope_smem(const RopeGrid &gr, int rope_dims, int width, int ring_bytes) {
    const int entries = (width > 1 ? width / 2 : 8) * rope_items(rope_dims, width);
    return ring_bytes + static_cast<size_t>(2) * gr.max_tokens * entries * sizeof(float2);
}

}  // namespace
}  // namespace dattn
