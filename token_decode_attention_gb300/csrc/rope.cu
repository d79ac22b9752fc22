// rope.cu -- rotary positions of many tokens at once.
//
// For token t at position p, head h and pair i < rope_dims / 2:
//   (u, w) -> magnitude (u cos a - w sin a, u sin a + w cos a),  a = p theta_i,
// channels from rope_dims on are copied; the gradient is the transposed map,
// the rotation by -a times the same magnitude.  fp32 arithmetic, one rounding
// to the tensor's type.  theta_i (scaled for long contexts or not) is made on
// the host; the angle is reduced exactly (rope_items.cuh).  p is positions[t], or
// for a ragged batch (the queries of an append) counted back from the position
// of the last token of t's sequence.
//
// What bounds it: each element is read once and written once, 3 flops each; the
// cosines depend on (token, pair) only.  The items of all tokens, flattened, are cut
// into tiles of one per thread and every resident CTA takes an equal run of tiles:
// while it rotates and stores one, the next one's loads are in flight, and the
// cos/sin table of the next one's tokens is built in the other half of a double
// buffer, from positions fetched one tile earlier still.
#include <cuda_runtime.h>

#include <algorithm>

#include "dattn_internal.h"
#include "ptx.cuh"
#include "rope_items.cuh"

namespace dattn {
namespace {

constexpr int kThreads = 256;
// CTAs of an SM: f32 items take twice the registers.
template <typename T>
constexpr int kMinBlocks = sizeof(T) == 4 ? 3 : 4;

struct RopeGrid {
    long long tiles;
    int items, per_token;  // items of a row, of a token
    int max_tokens;        // tokens that a tile may touch
    FastDiv div_token;
};

// FIXED: a thread's item is the same in every tile (the items of a row divide the
// threads), so what depends on it is computed once.
template <typename T, bool VEC, bool FIXED>
__global__ void __launch_bounds__(kThreads, kMinBlocks<T>)
    rope_kernel(const __grid_constant__ RopeArgs a, const RopeGrid gr) {
    extern __shared__ float2 table[];  // [2][max_tokens][8 * rotated items]
    __shared__ uint32_t s_pos[2][kThreads];
    pdl_launch_dependents();
    pdl_wait_primary();
    const int D = a.D, rd = a.rope.rope_dims, tid = threadIdx.x;
    const bool trad = a.rope.traditional != 0;
    const int ir = rope_items(rd, VEC), entries = 8 * ir;
    const long long used = used_tokens(a.offsets, a.B, a.tokens);
    const long long first = gr.tiles * blockIdx.x / gridDim.x;
    const long long last = gr.tiles * (blockIdx.x + 1) / gridDim.x;

    // Tokens and places are carried from tile to tile: 256 items on are step_tokens
    // tokens, step_heads heads and step_items items on, with carries.
    const int step_tokens = kThreads / gr.per_token, step_in = kThreads - step_tokens * gr.per_token;
    const int step_heads = step_in / gr.items, step_items = FIXED ? 0 : step_in - step_heads * gr.items;
    // A tile's first token and the place of its first item in that token.
    struct Tile {
        long long token;
        int skip;
    } cur;
    auto next = [&](Tile &t) {
        t.token += step_tokens;
        t.skip += step_in;
        if (t.skip >= gr.per_token) {
            t.skip -= gr.per_token;
            ++t.token;
        }
    };
    // This thread's item.
    struct Place {
        long long token;
        int head, item;
    } p;
    auto step = [&](Place &x) {
        x.head += step_heads;
        x.token += step_tokens;
        if constexpr (!FIXED) {
            x.item += step_items;
            if (x.item >= gr.items) {
                x.item -= gr.items;
                ++x.head;
            }
        }
        if (x.head >= a.H) {
            x.head -= a.H;
            ++x.token;
        }
    };
    {
        const long long n = first * kThreads, t = n / gr.per_token;
        cur = Tile{t, static_cast<int>(n - t * gr.per_token)};
        const int in = cur.skip + tid, whole = in / gr.per_token, rest = in - whole * gr.per_token;
        p.token = t + whole;
        p.head = rest / gr.items;
        p.item = rest - p.head * gr.items;
    }
    // Position of the tile's token number tid.  In a ragged batch the thread keeps
    // the sequence it found last: [lo, hi) its tokens, the position of token t
    // being from + t.
    long long lo = 0, hi = 0, from = 0;
    auto position = [&](const Tile &t) -> uint32_t {
        if (tid >= gr.max_tokens) return 0;
        const long long n = t.token + tid;
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
            from = static_cast<long long>(__ldg(a.cur_pos + b)) - (hi - 1);
        }
        return static_cast<uint32_t>(from + n);
    };
    const RopeFiller<T, VEC> filler(ir, a.rope, a.gradient != 0);
    auto fill = [&](const Tile &t, int half) {
        const int touched = min(gr.max_tokens, fast_div(t.skip + kThreads - 1, gr.div_token) + 1);
        filler.fill(table + half * gr.max_tokens * entries, touched, [&](int s) { return s_pos[half][s]; });
    };
    const Item<T, VEC> fixed(p.item, rd, D, trad);
    auto item_of = [&](const Place &x) {
        if constexpr (FIXED) return fixed;
        return Item<T, VEC>(x.item, rd, D, trad);
    };
    auto load = [&](const Place &x, ItemData<T> &d) {
        if (x.token < used)
            item_of(x).load(reinterpret_cast<const T *>(a.x) + x.token * a.x_stride + x.head * D, d);
    };

    if (first >= last) return;
    ItemData<T> d, dn;
    load(p, d);
    Tile ahead = cur;
    s_pos[0][tid] = position(cur);
    next(ahead);
    s_pos[1][tid] = position(ahead);
    __syncthreads();
    fill(cur, 0);
    __syncthreads();
    const int count = static_cast<int>(last - first);  // tiles fit 31 bits
    for (int k = 0; k < count; ++k) {
        const int half = k & 1;
        Place pn = p;
        step(pn);
        const bool more = k + 1 < count;
        if (more) load(pn, dn);
        next(ahead);  // two tiles on
        const uint32_t pos = k + 2 < count ? position(ahead) : 0u;
        if (p.token < used) {
            const Item<T, VEC> it = item_of(p);
            float y[16];
            it.values(d, table + (half * gr.max_tokens + static_cast<int>(p.token - cur.token)) * entries + it.j,
                      ir, y);
            T *e = reinterpret_cast<T *>(d.v);
#pragma unroll
            for (int i = 0; i < 16; ++i) e[i] = from_float<T>(y[i]);
            it.store(reinterpret_cast<T *>(a.out) + p.token * a.out_stride + p.head * D, d);
        }
        if (!more) break;
        next(cur);
        fill(cur, half ^ 1);
        if (tid < gr.max_tokens) s_pos[half][tid] = pos;  // last read before the barrier before this one
        __syncthreads();
        p = pn;
        d = dn;
    }
}

template <typename T>
const void *kernel_of(bool vec, bool fixed) {
    if (!vec) return reinterpret_cast<const void *>(rope_kernel<T, false, false>);
    return fixed ? reinterpret_cast<const void *>(rope_kernel<T, true, true>)
                 : reinterpret_cast<const void *>(rope_kernel<T, true, false>);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs &a, int dtype, int sms, cudaStream_t stream) {
    const bool vec = a.rope.rope_dims % 16 == 0 && a.D % 16 == 0;
    RopeGrid gr{};
    gr.items = row_items(a.rope.rope_dims, a.D, vec);
    const long long per_token = static_cast<long long>(a.H) * gr.items;
    if (per_token > (1 << 30) || a.tokens > 0x7fffffffLL) return cudaErrorInvalidValue;
    gr.per_token = static_cast<int>(per_token);
    gr.tiles = (a.tokens * per_token + kThreads - 1) / kThreads;
    gr.max_tokens = kThreads % gr.per_token == 0 ? kThreads / gr.per_token
                                                 : (kThreads - 2) / gr.per_token + 2;
    const int ir = rope_items(a.rope.rope_dims, vec);
    gr.div_token = fast_div_of(gr.per_token);
    const long long slots = static_cast<long long>(sms) * (dtype == kDtypeF32 ? kMinBlocks<float> : kMinBlocks<__half>);
    const long long ctas = std::min(gr.tiles, slots);
    if (gr.tiles > 0x7fffffffLL) return cudaErrorInvalidValue;
    const bool fixed = kThreads % gr.items == 0;
    const void *fn = dtype == kDtypeF16    ? kernel_of<__half>(vec, fixed)
                     : dtype == kDtypeBf16 ? kernel_of<__nv_bfloat16>(vec, fixed)
                                           : kernel_of<float>(vec, fixed);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(kThreads);
    // at most 2 x (256 / items + 2) tokens x 8 items entries: 36 KB
    cfg.dynamicSmemBytes = static_cast<size_t>(2) * gr.max_tokens * 8 * ir * sizeof(float2);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void *args[] = {const_cast<RopeArgs *>(&a), &gr};
    return cudaLaunchKernelExC(&cfg, fn, args);
}

}  // namespace dattn
