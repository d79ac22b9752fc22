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
// and two for q; a step of one token is bound by latency.  A CTA owns whole
// (block, head) pairs, so the maximum needs no second launch and no global
// atomics: its threads hold the block's new rows of some heads in registers
// (16 channels each), join their maxima in shared memory and write the 8-bit
// rows; each input is read once.  The grid cannot know the ragged lengths, so
// it is cut by tokens: a CTA looks through a window of the flattened tokens for
// those that open a block (the first of a sequence, or a position at a
// multiple of scale_block) and takes their blocks.  K and V go to different
// CTAs; further CTAs rotate q.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "dattn_internal.h"
#include "ptx.cuh"
#include "rope_items.cuh"

namespace dattn {
namespace {

constexpr int kThreads = 256;
constexpr int kMinExp = -32;     // scales are at least 2^-32
constexpr int kQTokens = 4;      // tokens of a CTA that rotates q
constexpr int kMaxHeads = 256;   // heads of a CTA

struct AppendGrid {
    int items_k, items_v, items_q;  // per row
    int rows;              // rows of a block side by side in a CTA
    int heads;             // heads side by side in a CTA
    int heads_per_cta;
    int head_chunks;
    int window;            // tokens a CTA looks through
    long long kv_ctas;
    int q_tokens, q_heads, q_chunks;
};

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

// x / scale; the reciprocal of a power of two is exact.
struct Divider {
    float s, inv;
    bool exact;
    __device__ __forceinline__ float operator()(float x) const { return exact ? x * inv : x / s; }
};
__device__ __forceinline__ Divider divider(float scale) {
    return Divider{scale, 1.f / scale, (__float_as_uint(scale) & 0x7fffffu) == 0};
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

// RPT rows and HPT heads per thread held in registers.
template <int KV, int RPT, int HPT, bool VEC>
__device__ __forceinline__ void append_kv(const Q8AppendArgs &a, const AppendGrid &gr, bool is_v,
                                          long long window, int chunk, float2 *table,
                                          uint32_t *s_amax, float *s_scale) {
    const int lane = threadIdx.x & 31;
    const int D = a.D, n_block = a.scale_block;
    const int rd = is_v ? 0 : a.rope.rope_dims, half = rd / 2;
    const bool trad = a.rope.traditional != 0;
    const int ir = rope_items(rd, VEC);
    const int items = is_v ? gr.items_v : gr.items_k;
    const int item = threadIdx.x % items;
    const int rs = threadIdx.x / items % gr.rows;
    const int hs = threadIdx.x / (items * gr.rows);
    const int h0 = chunk * gr.heads_per_cta;
    const int nh = min(gr.heads_per_cta, a.kv_heads - h0);
    const Item<VEC> it(item, rd, D, trad);
    const __half *src = reinterpret_cast<const __half *>(is_v ? a.v : a.k);
    const long long stride = is_v ? a.v_stride : a.k_stride;
    unsigned char *cache = is_v ? a.V : a.K;
    float *scales = is_v ? a.vs : a.ks;
    const int span = gr.rows * RPT;  // rows of a pass

    const long long used =
        a.offsets ? min(a.tokens, max(0LL, static_cast<long long>(__ldg(a.offsets + a.B)))) : a.tokens;
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
        const int blk = static_cast<int>((static_cast<unsigned long long>(pos) * a.div_block.mul) >> a.div_block.shift);
        const int before_blk = pos - blk * n_block;  // rows of the block before this one
        const int room = static_cast<int>(
            min(min(static_cast<long long>(n_block - before_blk), stop - tok), static_cast<long long>(a.S - pos)));
        if (before_blk != 0 && tok != s0) {  // inside a block that an earlier token opens
            tok += room;
            continue;
        }
        const int n = room, before = before_blk;

        // ---- the block's first row and its scale's row ----
        long long row0, srow;
        bool ok = true;
        if (a.block_table == nullptr) {
            row0 = static_cast<long long>(b) * a.S + pos - before;
            srow = static_cast<long long>(b) * a.scale_rows + blk;
        } else {
            const int pi = static_cast<int>((static_cast<unsigned long long>(pos) * a.div_page.mul) >> a.div_page.shift);
            const int in = pos - pi * a.page_size - before;
            const long long page = __ldg(a.block_table + static_cast<long long>(b) * a.max_pages + pi);
            ok = page >= 0 && page < a.num_pages;
            if (!ok && threadIdx.x == 0) atomicOr(a.err, kErrPageIndex);
            row0 = page * a.page_size + in;
            srow = page * a.scale_rows + blk - pi * a.scale_rows;
        }
        if (!ok) {
            tok += n;
            continue;
        }

        // ---- pass 1: load, rotate, largest magnitude per head ----
        for (int i = threadIdx.x; i < gr.heads_per_cta; i += kThreads) s_amax[i] = 0u;
        ItemData<__half> d[RPT][HPT];
        float mx[HPT];
#pragma unroll
        for (int h = 0; h < HPT; ++h) mx[h] = 0.f;
        auto load_pass = [&](int r0) {
#pragma unroll
            for (int r = 0; r < RPT; ++r)
#pragma unroll
                for (int h = 0; h < HPT; ++h) {
                    const int row = r0 + rs + r * gr.rows, head = hs + h * gr.heads;
                    if (row < n && head < nh && hs < gr.heads)
                        it.load(src + (tok + row) * stride + static_cast<long long>(h0 + head) * D, d[r][h]);
                }
        };
        auto fill_table = [&](int r0) {
            const int rows = min(span, n - r0);
            for (int i = threadIdx.x; i < rows * half; i += kThreads) {
                const int r = i / half;
                rope_table_entry(table + r * 8 * ir, ir, i - r * half, static_cast<uint32_t>(pos + r0 + r),
                                 a.rope, false);
            }
        };
        // the values of slot (r, h), rotated
        auto values = [&](int r, int h, float *y) {
            float2 cs[8];
            if (it.rot) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    cs[e] = table[(rs + r * gr.rows) * 8 * ir + e * ir + item];
            }
            rotate_item(it, d[r][h], cs, y);
        };
        for (int r0 = 0; r0 < n; r0 += span) {
            load_pass(r0);
            if (r0 > 0) __syncthreads();  // the table of the pass before has been read
            fill_table(r0);
            __syncthreads();
#pragma unroll
            for (int r = 0; r < RPT; ++r)
#pragma unroll
                for (int h = 0; h < HPT; ++h) {
                    const int row = r0 + rs + r * gr.rows, head = hs + h * gr.heads;
                    if (row < n && head < nh && hs < gr.heads) {
                        float y[16];
                        values(r, h, y);
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const float m = fabsf(y[e]);
                            if (m < INFINITY) mx[h] = fmaxf(mx[h], m);
                        }
                    }
                }
        }
        // lanes of one head: whole warps, or groups of a power of two of them
        const int seg = items * gr.rows;
#pragma unroll
        for (int h = 0; h < HPT; ++h) {
            uint32_t m = __float_as_uint(mx[h]);
            bool lead = hs < gr.heads && hs + h * gr.heads < nh;
            if ((seg & 31) == 0) {
                m = __reduce_max_sync(0xffffffffu, m);
                lead = lead && lane == 0;
            } else if ((seg & (seg - 1)) == 0) {
                for (int o = seg / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
                lead = lead && (lane & (seg - 1)) == 0;
            }
            if (lead) atomicMax(&s_amax[hs + h * gr.heads], m);
        }
        __syncthreads();

        // ---- the scale of each head; earlier rows on the new scale ----
        for (int i = threadIdx.x; i < nh; i += kThreads) {
            float *at = scales + srow * a.kv_heads + h0 + i;
            const float need = need_scale<KV>(s_amax[i]);
            const float old = before > 0 ? *at : need;
            const float now = before > 0 ? fmaxf(old, need) : need;
            s_scale[i] = now;
            s_scale[kMaxHeads + i] = old;
            *at = now;
        }
        __syncthreads();
        const size_t row_elems = static_cast<size_t>(a.kv_heads) * D;
        unsigned char *block0 = cache + static_cast<size_t>(row0) * row_elems + static_cast<size_t>(h0) * D;
        if (before > 0) {
#pragma unroll
            for (int h = 0; h < HPT; ++h) {
                const int head = hs + h * gr.heads;
                if (head >= nh || hs >= gr.heads) continue;
                const float now = s_scale[head], old = s_scale[kMaxHeads + head];
                if (!(now != old)) continue;
                const float f = old / now;
                for (int r = rs; r < before; r += gr.rows) {
                    // sixteen neighbouring channels, whatever the pairs are
                    for (int c = item * 16; c < D; c += items * 16) {
                        uint4 *v = reinterpret_cast<uint4 *>(block0 + r * row_elems + static_cast<size_t>(head) * D + c);
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
        }
        // ---- pass 2: the new rows ----
        for (int r0 = 0; r0 < n; r0 += span) {
            if (n > span) {  // more rows than the registers hold: read them again
                __syncthreads();
                load_pass(r0);
                fill_table(r0);
                __syncthreads();
            }
#pragma unroll
            for (int r = 0; r < RPT; ++r)
#pragma unroll
                for (int h = 0; h < HPT; ++h) {
                    const int row = r0 + rs + r * gr.rows, head = hs + h * gr.heads;
                    if (row >= n || head >= nh || hs >= gr.heads) continue;
                    float y[16];
                    values(r, h, y);
                    const Divider div = divider(s_scale[head]);
#pragma unroll
                    for (int e = 0; e < 16; ++e) y[e] = div(y[e]);
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        w[e] = pack4<KV>(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
                    unsigned char *o = block0 + static_cast<size_t>(before + row) * row_elems + static_cast<size_t>(head) * D;
                    if constexpr (VEC) {
                        if (it.o1 == it.o0 + 8 && it.o0 % 16 == 0) {
                            *reinterpret_cast<uint4 *>(o + it.o0) = make_uint4(w[0], w[1], w[2], w[3]);
                        } else {
                            *reinterpret_cast<uint2 *>(o + it.o0) = make_uint2(w[0], w[1]);
                            *reinterpret_cast<uint2 *>(o + it.o1) = make_uint2(w[2], w[3]);
                        }
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
        __syncthreads();  // the table and s_amax may be written again
    }
}

// q: some tokens with some of their heads.
template <bool VEC>
__device__ __forceinline__ void rotate_q(const Q8AppendArgs &a, const AppendGrid &gr,
                                         long long cta, float2 *table, int *s_pos) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int D = a.D, rd = a.rope.rope_dims, half = rd / 2;
    const bool trad = a.rope.traditional != 0;
    const int ir = rope_items(rd, VEC);
    const long long t0 = cta / gr.q_chunks * gr.q_tokens;
    const int h0 = static_cast<int>(cta % gr.q_chunks) * gr.q_heads;
    const int nh = min(gr.q_heads, a.H - h0);
    const long long used =
        a.offsets ? min(a.tokens, max(0LL, static_cast<long long>(__ldg(a.offsets + a.B)))) : a.tokens;
    const int nt = static_cast<int>(min(static_cast<long long>(gr.q_tokens), used - t0));
    if (nt <= 0) return;
    for (int s = warp; s < nt; s += kThreads / 32) {
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
        if (lane == 0) s_pos[s] = static_cast<int>(static_cast<uint32_t>(p));
    }
    __syncthreads();
    for (int i = threadIdx.x; i < nt * half; i += kThreads) {
        const int s = i / half;
        rope_table_entry(table + s * 8 * ir, ir, i - s * half, static_cast<uint32_t>(s_pos[s]), a.rope, false);
    }
    __syncthreads();
    const __half *q = reinterpret_cast<const __half *>(a.q);
    __half *out = reinterpret_cast<__half *>(a.q_out);
    const int total = nt * nh * gr.items_q;
#pragma unroll 4
    for (int n = threadIdx.x; n < total; n += kThreads) {
        const int th = n / gr.items_q, item = n - th * gr.items_q;
        const int s = th / nh, head = h0 + th - s * nh;
        const Item<VEC> it(item, rd, D, trad);
        ItemData<__half> d;
        it.load(q + (t0 + s) * a.q_stride + static_cast<long long>(head) * D, d);
        float2 cs[8];
        if (it.rot) {
#pragma unroll
            for (int e = 0; e < 8; ++e) cs[e] = table[s * 8 * ir + e * ir + item];
        }
        float y[16];
        rotate_item(it, d, cs, y);
        ItemData<__half> r;
        __half *e = reinterpret_cast<__half *>(r.v);
#pragma unroll
        for (int i = 0; i < 16; ++i) e[i] = __float2half_rn(y[i]);
        it.store(out + ((t0 + s) * a.H + head) * D, r);
    }
}

template <int KV, int RPT, int HPT, bool VEC>
__global__ void __launch_bounds__(kThreads)
    append_q8_kernel(const __grid_constant__ Q8AppendArgs a, const AppendGrid gr) {
    extern __shared__ float2 table[];
    __shared__ uint32_t s_amax[kMaxHeads];
    __shared__ float s_scale[2 * kMaxHeads];
    __shared__ int s_pos[kQTokens];
    pdl_launch_dependents();
    pdl_wait_primary();
    const long long cta = blockIdx.x;
    if (cta < gr.kv_ctas) {
        const bool is_v = (cta & 1) != 0;
        const long long rest = cta >> 1;
        append_kv<KV, RPT, HPT, VEC>(a, gr, is_v, rest / gr.head_chunks,
                                     static_cast<int>(rest % gr.head_chunks), table, s_amax, s_scale);
    } else {
        rotate_q<VEC>(a, gr, cta - gr.kv_ctas, table, s_pos);
    }
}

template <int KV, bool VEC>
const void *kernel_of(int rpt, int hpt) {
    if (rpt == 1 && hpt == 1) return reinterpret_cast<const void *>(append_q8_kernel<KV, 1, 1, VEC>);
    if (rpt == 1) return reinterpret_cast<const void *>(append_q8_kernel<KV, 1, 4, VEC>);
    if (rpt == 2) return reinterpret_cast<const void *>(append_q8_kernel<KV, 2, 2, VEC>);
    return reinterpret_cast<const void *>(append_q8_kernel<KV, 4, 1, VEC>);
}

}  // namespace

cudaError_t launch_append_q8(const Q8AppendArgs &a, int kv, int sms, cudaStream_t stream) {
    const int rd = a.rope.rope_dims;
    const bool vec = rd % 16 == 0;  // D is a multiple of 16
    AppendGrid gr{};
    gr.items_k = row_items(rd, a.D, vec);
    gr.items_v = row_items(0, a.D, vec);
    gr.items_q = gr.items_k;
    const int items = std::max(gr.items_k, gr.items_v);
    // rows of a block side by side: all of them if they fit, one in a step of
    // one token per sequence
    const int want = a.offsets == nullptr ? 1 : a.scale_block;
    gr.rows = 1;
    while (gr.rows < want && 2 * gr.rows * items <= kThreads) gr.rows *= 2;
    gr.heads = std::min({kThreads / (items * gr.rows), a.kv_heads, kMaxHeads / 4});
    // slots of a thread: the block's rows first, then heads
    int rpt = 1, hpt = 1;
    if (a.offsets != nullptr) {
        while (rpt < 4 && rpt * gr.rows < a.scale_block) rpt *= 2;
        hpt = 4 / rpt;
    }
    gr.heads_per_cta = std::min(gr.heads * hpt, a.kv_heads);
    gr.head_chunks = (a.kv_heads + gr.heads_per_cta - 1) / gr.heads_per_cta;
    // about one block per window when sequences are long, one token when short
    const long long mean = std::max(1LL, a.tokens / a.B);
    gr.window = static_cast<int>(a.offsets == nullptr ? 1 : std::min<long long>(mean, a.scale_block));
    const long long windows = (a.tokens + gr.window - 1) / gr.window;
    gr.kv_ctas = windows * gr.head_chunks * 2;
    gr.q_tokens = a.tokens >= 4LL * sms * kQTokens ? kQTokens : 1;
    gr.q_heads = a.H;
    while (gr.q_heads > 1 && a.tokens / gr.q_tokens * ((a.H + gr.q_heads - 1) / gr.q_heads) < 2LL * sms &&
           gr.q_heads * gr.items_q > 64)
        gr.q_heads = (gr.q_heads + 1) / 2;
    gr.q_chunks = (a.H + gr.q_heads - 1) / gr.q_heads;
    const long long q_ctas = (a.tokens + gr.q_tokens - 1) / gr.q_tokens * gr.q_chunks;
    const long long blocks = gr.kv_ctas + q_ctas;
    if (blocks <= 0 || blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    const void *fn = kv == kKvE4m3 ? (vec ? kernel_of<kKvE4m3, true>(rpt, hpt) : kernel_of<kKvE4m3, false>(rpt, hpt))
                                   : (vec ? kernel_of<kKvInt8, true>(rpt, hpt) : kernel_of<kKvInt8, false>(rpt, hpt));
    const int rows = std::max(std::min(gr.rows * rpt, a.offsets ? a.scale_block : 1), gr.q_tokens);
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
