// append_q8.cu -- rotate the new tokens of a ragged batch and append their keys
// and values to a KV cache held in 8 bits (e4m3 or int8) with one fp32 scale
// for each block of `scale_block` positions and key/value head.
//
// Sequence b brings tokens offsets[b] .. offsets[b+1]-1 (n_b of them; one when
// offsets is null), the last of them at position current_pos[b].  q and k are
// rotated at their positions (rope.cu's map) in fp32; q is rounded to f16 into
// q_out, k and v go to the cache.  For a block that receives rows:
//   amax  = largest finite |x| of the new rows of the head
//   need  = smallest power of two s >= 2^-32 with amax <= QMAX s   (448 or 127)
//   scale = need, or max(old scale, need) where the sequence has earlier rows in
//           the block; those rows are requantised when the scale grows
//   row   = nearest 8-bit value to x / scale, ties to even, saturating
// A power of two keeps all of e4m3's relative precision, makes x / scale exact
// and a requantisation of e4m3 exact down to its subnormals; for int8 it costs
// up to one of its seven bits.  Infinities saturate; NaN stays NaN in e4m3 and
// becomes 0 in int8.
//
// What bounds it: 2 bytes read per new element and one written for k and v, two
// and two for q; a step of one token is bound by latency.  A segment of a warp (or
// a warp) owns a (block, head) pair, so the maximum needs no second launch and no
// atomics: its lanes hold the block's new rows in registers
// (an item of 16 channels per row), join their maxima with shuffles and write the
// 8-bit rows; large blocks take several warps.  Each input is read once unless a
// block has more rows than its warps hold.  The CTA shares one cos/sin table of the block's positions, K and V go to
// different CTAs.  The grid cannot know the ragged lengths, so it is cut by tokens:
// a CTA looks through a window of the flattened tokens for those that open a block
// (the first of a sequence, or a position at a multiple of scale_block) and takes
// their blocks.  q is rotated by further CTAs of the same launch, or, when it is
// large, by the kernel of rope.cu, whose CTAs need fewer registers.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "dattn_internal.h"
#include "ptx.cuh"
#include "rope_items.cuh"

namespace dattn {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMinExp = -32;  // scales are at least 2^-32
constexpr int kQTokens = 4;   // tokens of a CTA that rotates q
constexpr long long kQApart = 4 << 20;  // elements of q from which rope.cu's kernel takes it

struct AppendGrid {
    int items_k, items_v, items_q;  // per row
    int lanes;             // lanes of a row: a power of two, items_k and items_v at most
    int rows;              // rows of a block side by side in a segment of lanes
    int heads_per_warp;    // segments of a warp
    int warps_per_head;    // warps that share the rows of their heads
    int heads_per_cta;
    int head_chunks;
    int window;            // tokens a CTA looks through
    long long kv_ctas;
    int q_tokens, q_heads, q_chunks;
};

// Smallest power of two s >= 2^kMinExp with amax <= QMAX s, from the bits of
// amax: QMAX is 1.75 2^8 (e4m3) or 1.984375 2^6 (int8).
template <int KV>
__device__ __forceinline__ float need_scale(uint32_t amax_bits) {
    constexpr uint32_t kTop = KV == kKvE4m3 ? 0x600000u : 0x7e0000u;
    constexpr int kExp = KV == kKvE4m3 ? 8 : 6;
    int e = static_cast<int>(amax_bits >> 23) - 127 - kExp;
    if ((amax_bits & 0x7fffffu) > kTop) ++e;
    if (amax_bits == 0 || e < kMinExp) e = kMinExp;
    return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// x / scale is x times the reciprocal, exactly, where the scale is a power of two (or
// infinite or NaN).
struct Divider {
    float inv;
    bool exact;
};
__device__ __forceinline__ Divider divider(float scale) {
    return Divider{1.f / scale, (__float_as_uint(scale) & 0x7fffffu) == 0};
}

template <int KV>
__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
    uint32_t r;
    if constexpr (KV == kKvE4m3) {
        asm("{\n\t.reg .b16 l, h;\n\t"
            "cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
            "mov.b32 %0, {l, h};\n\t}"
            : "=r"(r)
            : "f"(a), "f"(b), "f"(c), "f"(d));
    } else {
        auto q = [](float x) {
            const int i = __float2int_rn(fminf(fmaxf(x, -127.f), 127.f));
            return static_cast<uint32_t>(x != x ? 0 : i) & 255u;
        };
        r = q(a) | q(b) << 8 | q(c) << 16 | q(d) << 24;
    }
    return r;
}

template <int KV>
__device__ __forceinline__ float value_of(unsigned char x) {
    if constexpr (KV == kKvE4m3) {
        uint32_t h;
        asm("{\n\t.reg .b16 b;\n\tcvt.u16.u32 b, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, b;\n\t}"
            : "=r"(h)
            : "r"(static_cast<uint32_t>(x)));
        return __half2float(__ushort_as_half(static_cast<unsigned short>(h)));
    } else {
        return static_cast<float>(static_cast<signed char>(x));
    }
}

// RPT rows per lane held in registers.
template <int KV, int RPT, bool VEC>
__device__ __forceinline__ void append_kv(const Q8AppendArgs &a, const AppendGrid &gr, bool is_v,
                                          long long window, int chunk, float2 *table,
                                          float *s_mx) {
    using It = Item<__half, VEC>;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int D = a.D, n_block = a.scale_block;
    const int rd = is_v ? 0 : a.rope.rope_dims;
    const int ir = rope_items(rd, VEC);
    const int items = is_v ? gr.items_v : gr.items_k;
    const int seg = gr.lanes * gr.rows;  // lanes of a head: a power of two
    const int item = lane & (gr.lanes - 1), rs = (lane & (seg - 1)) / gr.lanes;
    const int wph = gr.warps_per_head, wr = warp & (wph - 1);  // a power of two
    const int head = chunk * gr.heads_per_cta + warp / wph * gr.heads_per_warp + lane / seg;
    const int rs0 = wr * gr.rows * RPT + rs;  // this lane's first row of a pass
    const bool mine = item < items && head < a.kv_heads;
    const It it(item, rd, D, a.rope.traditional != 0);
    const __half *src = reinterpret_cast<const __half *>(is_v ? a.v : a.k) + static_cast<long long>(head) * D;
    const long long stride = is_v ? a.v_stride : a.k_stride;
    unsigned char *cache = (is_v ? a.V : a.K) + static_cast<size_t>(head) * D;
    float *scales = (is_v ? a.vs : a.ks) + head;
    const int span = gr.rows * RPT * wph;  // rows of a pass

    const RopeFiller<__half, VEC> filler(ir, a.rope, false);
    const long long used = used_tokens(a.offsets, a.B, a.tokens);
    long long tok = window * gr.window;
    const long long w1 = min(tok + gr.window, used);
    while (tok < w1) {
        // ---- the sequence and position of token tok ----
        int b;
        long long s0, s1;  // its sequence's tokens
        if (a.offsets == nullptr) {
            b = static_cast<int>(tok);
            s0 = tok;
            s1 = tok + 1;
        } else {
            b = find_sequence(a.offsets, a.B, tok, lane);
            s0 = __ldg(a.offsets + b);
            s1 = __ldg(a.offsets + b + 1);
        }
        const long long stop = min(s1, used);
        if (stop <= tok) {  // offsets that do not ascend: no token of a sequence
            ++tok;
            continue;
        }
        const long long p = static_cast<long long>(__ldg(a.cur_pos + b)) - (s1 - 1 - tok);
        if (p < 0 || p >= a.S) {
            if (threadIdx.x == 0) atomicOr(a.err, kErrAppendPosition);
            tok = p < 0 ? min(tok - p, stop) : stop;
            continue;
        }
        const int pos = static_cast<int>(p);
        const int blk = fast_div(pos, a.div_block);
        const int before = pos - blk * n_block;  // rows of the block before this one
        const int n = static_cast<int>(min(min(static_cast<long long>(n_block - before), stop - tok),
                                           static_cast<long long>(a.S - pos)));
        if (before != 0 && tok != s0) {  // inside a block that an earlier token opens
            tok += n;
            continue;
        }

        // ---- load the first rows; the block's first row and its scale's row ----
        ItemData<__half> d[RPT];
        auto load_pass = [&](int r0) {
#pragma unroll
            for (int r = 0; r < RPT; ++r) {
                const int row = r0 + rs0 + r * gr.rows;
                if (mine && row < n) it.load(src + (tok + row) * stride, d[r]);
            }
        };
        load_pass(0);
        long long row0, srow;
        bool ok = true;
        if (a.block_table == nullptr) {
            row0 = static_cast<long long>(b) * a.S + pos - before;
            srow = static_cast<long long>(b) * a.scale_rows + blk;
        } else {
            const int pi = fast_div(pos, a.div_page);
            const long long page = __ldg(a.block_table + static_cast<long long>(b) * a.max_pages + pi);
            ok = page >= 0 && page < a.num_pages;
            if (!ok && threadIdx.x == 0) atomicOr(a.err, kErrPageIndex);
            row0 = page * a.page_size + (pos - pi * a.page_size - before);
            srow = page * a.scale_rows + blk - pi * a.scale_rows;
        }
        if (!ok) {
            tok += n;
            continue;
        }
        float *const scale = scales + srow * a.kv_heads;
        const float old = before > 0 && head < a.kv_heads ? *scale : 0.f;

        // ---- pass 1: rotate, largest finite magnitude of the head ----
        auto fill_table = [&](int r0) {
            filler.fill(table, min(span, n - r0), [&](int r) { return static_cast<uint32_t>(pos + r0 + r); });
        };
        float mx = 0.f;
        for (int r0 = 0; r0 < n; r0 += span) {
            if (r0 > 0) {
                load_pass(r0);
                if (ir > 0) __syncthreads();  // the table of the pass before has been read
            }
            if (ir > 0) {
                fill_table(r0);
                __syncthreads();
            }
#pragma unroll
            for (int r = 0; r < RPT; ++r) {
                const int row = rs0 + r * gr.rows;
                if (mine && r0 + row < n) {
                    float y[16];
                    it.values(d[r], table + row * 8 * ir + item, ir, y);
                    float m = 0.f;  // fmaxf passes over NaN
#pragma unroll
                    for (int e = 0; e < 16; ++e) m = fmaxf(m, fabsf(y[e]));
                    if (m == INFINITY) {  // among infinities only the finite ones count
                        m = 0.f;
#pragma unroll
                        for (int e = 0; e < 16; ++e) m = fabsf(y[e]) < INFINITY ? fmaxf(m, fabsf(y[e])) : m;
                    }
                    mx = fmaxf(mx, m);
                }
            }
        }
        for (int o = seg / 2; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        if (wph > 1) {  // then a warp is one segment
            if (lane == 0) s_mx[warp] = mx;
            __syncthreads();
            for (int w = 0; w < wph; ++w) mx = fmaxf(mx, s_mx[(warp & ~(wph - 1)) + w]);
        }

        // ---- the head's scale; its earlier rows on the new scale ----
        const float need = need_scale<KV>(__float_as_uint(mx));
        const float now = before > 0 ? fmaxf(old, need) : need;
        if (head < a.kv_heads && wr == 0 && (lane & (seg - 1)) == 0) *scale = now;
        const size_t row_elems = static_cast<size_t>(a.kv_heads) * D;
        unsigned char *const block0 = cache + static_cast<size_t>(row0) * row_elems;
        if (before > 0 && now != old && head < a.kv_heads) {
            const float f = old / now;
            for (int r = wr * gr.rows + rs; r < before; r += gr.rows * wph) {
                // sixteen neighbouring channels, whatever the pairs are
                for (int c = item * 16; c < D; c += gr.lanes * 16) {
                    uint4 *v = reinterpret_cast<uint4 *>(block0 + r * row_elems + c);
                    uint4 x = *v;
                    uint32_t *w = reinterpret_cast<uint32_t *>(&x);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        w[e] = pack4<KV>(value_of<KV>(w[e] & 255u) * f, value_of<KV>(w[e] >> 8 & 255u) * f,
                                         value_of<KV>(w[e] >> 16 & 255u) * f, value_of<KV>(w[e] >> 24) * f);
                    *v = x;
                }
            }
        }
        // ---- pass 2: the new rows ----
        const Divider div = divider(now);
        for (int r0 = 0; r0 < n; r0 += span) {
            if (n > span) {  // more rows than the lanes hold: read them again
                load_pass(r0);
                if (ir > 0) {
                    __syncthreads();
                    fill_table(r0);
                    __syncthreads();
                }
            }
#pragma unroll
            for (int r = 0; r < RPT; ++r) {
                const int row = rs0 + r * gr.rows;
                if (!mine || r0 + row >= n) continue;
                float y[16];
                it.values(d[r], table + row * 8 * ir + item, ir, y);
                if (div.exact) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) y[e] *= div.inv;
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e) y[e] = y[e] / now;
                }
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    w[e] = pack4<KV>(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
                unsigned char *o = block0 + static_cast<size_t>(before + r0 + row) * row_elems;
                if constexpr (VEC) {
                    *reinterpret_cast<uint2 *>(o + it.first) = make_uint2(w[0], w[1]);
                    *reinterpret_cast<uint2 *>(o + it.first + it.hop) = make_uint2(w[2], w[3]);
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const int ch = it.channel(e);
                        if (ch >= 0) o[ch] = static_cast<unsigned char>(w[e >> 2] >> (8 * (e & 3)));
                    }
                }
            }
        }
        tok += n;
        if (ir > 0 || wph > 1) __syncthreads();  // the table and s_mx may be written again
    }
}

// q: some tokens with some of their heads.
template <bool VEC>
__device__ __forceinline__ void rotate_q(const Q8AppendArgs &a, const AppendGrid &gr,
                                         long long cta, float2 *table, uint32_t *s_pos) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int D = a.D, rd = a.rope.rope_dims;
    const int ir = rope_items(rd, VEC);
    const long long t0 = cta / gr.q_chunks * gr.q_tokens;
    const int h0 = static_cast<int>(cta % gr.q_chunks) * gr.q_heads;
    const int nh = min(gr.q_heads, a.H - h0);
    const long long used = used_tokens(a.offsets, a.B, a.tokens);
    const int nt = static_cast<int>(min(static_cast<long long>(gr.q_tokens), used - t0));
    if (nt <= 0) return;
    for (int s = warp; s < nt; s += kWarps) {
        const long long t = t0 + s;
        long long p;
        if (a.offsets == nullptr) {
            p = __ldg(a.cur_pos + t);
        } else {
            const int b = find_sequence(a.offsets, a.B, t, lane);
            p = static_cast<long long>(__ldg(a.cur_pos + b)) - (__ldg(a.offsets + b + 1) - 1 - t);
        }
        // the rotation is defined at every position; the append reports those
        // outside the cache
        if (lane == 0) s_pos[s] = static_cast<uint32_t>(p);
    }
    __syncthreads();
    RopeFiller<__half, VEC>(ir, a.rope, false).fill(table, nt, [&](int s) { return s_pos[s]; });
    __syncthreads();
    const __half *q = reinterpret_cast<const __half *>(a.q);
    __half *out = reinterpret_cast<__half *>(a.q_out);
    const int total = nt * nh * gr.items_q;
    for (int n = threadIdx.x; n < total; n += kThreads) {
        const int th = n / gr.items_q, item = n - th * gr.items_q;
        const int s = th / nh, head = h0 + th - s * nh;
        const Item<__half, VEC> it(item, rd, D, a.rope.traditional != 0);
        ItemData<__half> d;
        it.load(q + (t0 + s) * a.q_stride + static_cast<long long>(head) * D, d);
        float y[16];
        it.values(d, table + s * 8 * ir + item, ir, y);
        __half *e = reinterpret_cast<__half *>(d.v);
#pragma unroll
        for (int i = 0; i < 16; ++i) e[i] = __float2half_rn(y[i]);
        it.store(out + ((t0 + s) * a.H + head) * D, d);
    }
}

template <int KV, int RPT, bool VEC>
__global__ void __launch_bounds__(kThreads, 3)
    append_q8_kernel(const __grid_constant__ Q8AppendArgs a, const AppendGrid gr) {
    extern __shared__ float2 table[];
    __shared__ uint32_t s_pos[kQTokens];
    __shared__ float s_mx[kWarps];
    pdl_launch_dependents();
    pdl_wait_primary();
    const long long cta = blockIdx.x;
    if (cta < gr.kv_ctas) {
        const unsigned rest = static_cast<unsigned>(cta >> 1), w = rest / static_cast<unsigned>(gr.head_chunks);
        append_kv<KV, RPT, VEC>(a, gr, (cta & 1) != 0, w, static_cast<int>(rest - w * gr.head_chunks), table,
                               s_mx);
    } else {
        rotate_q<VEC>(a, gr, cta - gr.kv_ctas, table, s_pos);
    }
}

template <int KV, bool VEC>
const void *kernel_of(int rpt) {
    if (rpt == 1) return reinterpret_cast<const void *>(append_q8_kernel<KV, 1, VEC>);
    if (rpt == 2) return reinterpret_cast<const void *>(append_q8_kernel<KV, 2, VEC>);
    // elements read one by one take too many registers for more rows
    if constexpr (VEC) return reinterpret_cast<const void *>(append_q8_kernel<KV, 4, VEC>);
    return nullptr;
}

}  // namespace

cudaError_t launch_append_q8(const Q8AppendArgs &a, int kv, int sms, cudaStream_t stream) {
    const int rd = a.rope.rope_dims;
    const bool vec = rd % 16 == 0;  // D is a multiple of 16
    AppendGrid gr{};
    gr.items_k = row_items(rd, a.D, vec);
    gr.items_v = row_items(0, a.D, vec);
    gr.items_q = gr.items_k;
    gr.lanes = 1;
    while (gr.lanes < std::max(gr.items_k, gr.items_v)) gr.lanes *= 2;
    // rows of a block: side by side in the lanes of a warp first, then up to four in a
    // lane's registers, then in more warps; one in a step of one token per sequence
    const int want = a.offsets == nullptr ? 1 : a.scale_block;
    gr.rows = 1;
    while (gr.rows < want && 2 * gr.rows * gr.lanes <= 32) gr.rows *= 2;
    int rpt = 1;
    while (rpt < (vec ? 4 : 2) && rpt * gr.rows < want) rpt *= 2;
    gr.warps_per_head = 1;
    while (gr.warps_per_head < kWarps && gr.warps_per_head * rpt * gr.rows < want) gr.warps_per_head *= 2;
    gr.heads_per_warp = 32 / (gr.lanes * gr.rows);
    gr.heads_per_cta = gr.heads_per_warp * (kWarps / gr.warps_per_head);
    gr.head_chunks = (a.kv_heads + gr.heads_per_cta - 1) / gr.heads_per_cta;
    // about one block per window when sequences are long, one token when short
    const long long mean = std::max(1LL, a.tokens / a.B);
    gr.window = static_cast<int>(a.offsets == nullptr ? 1 : std::min<long long>(mean, a.scale_block));
    const long long windows = (a.tokens + gr.window - 1) / gr.window;
    gr.kv_ctas = windows * gr.head_chunks * 2;
    // q with the kernel of rope.cu where it is large enough for the second launch
    const bool apart = a.tokens * a.H * static_cast<long long>(a.D) >= kQApart;
    if (apart) {
        RopeArgs r{};
        r.rope = a.rope;
        r.x = a.q;
        r.out = a.q_out;
        r.offsets = a.offsets;
        r.cur_pos = a.cur_pos;
        r.B = a.B;
        r.x_stride = a.q_stride;
        r.out_stride = static_cast<long long>(a.H) * a.D;
        r.tokens = a.tokens;
        r.H = a.H;
        r.D = a.D;
        const cudaError_t e = launch_rope(r, kDtypeF16, sms, stream);
        if (e != cudaSuccess) return e;
    }
    gr.q_tokens = a.tokens >= 4LL * sms * kQTokens ? kQTokens : 1;
    gr.q_heads = a.H;
    while (gr.q_heads > 1 && a.tokens / gr.q_tokens * ((a.H + gr.q_heads - 1) / gr.q_heads) < 2LL * sms &&
           gr.q_heads * gr.items_q > 64)
        gr.q_heads = (gr.q_heads + 1) / 2;
    gr.q_chunks = (a.H + gr.q_heads - 1) / gr.q_heads;
    const long long q_ctas = apart ? 0 : (a.tokens + gr.q_tokens - 1) / gr.q_tokens * gr.q_chunks;
    const long long blocks = gr.kv_ctas + q_ctas;
    if (blocks <= 0 || blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    const void *fn = kv == kKvE4m3 ? (vec ? kernel_of<kKvE4m3, true>(rpt) : kernel_of<kKvE4m3, false>(rpt))
                                   : (vec ? kernel_of<kKvInt8, true>(rpt) : kernel_of<kKvInt8, false>(rpt));
    // the table: at most 8 warps x 32 lanes x 4 rows of them x 8 pairs, 64 KB
    const int rows = std::max(std::min(gr.rows * rpt * gr.warps_per_head, want), gr.q_tokens);
    const size_t smem = static_cast<size_t>(rows) * 8 * rope_items(rd, vec) * sizeof(float2);
    if (smem > 48 * 1024) {
        const cudaError_t e =
            cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void *args[] = {const_cast<Q8AppendArgs *>(&a), &gr};
    return cudaLaunchKernelExC(&cfg, fn, args);
}

}  // namespace dattn
