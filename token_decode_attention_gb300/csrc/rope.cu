// rope.cu -- rotary positions of many tokens at once.
//
// For token t at position p = positions[t], head h and pair i < rope_dims / 2:
//   (u, w) -> magnitude (u cos a - w sin a, u sin a + w cos a),  a = p theta_i,
// channels from rope_dims on are copied; the gradient is the transposed map,
// the rotation by -a times the same magnitude.  fp32 arithmetic, one rounding
// to the tensor's type.  theta_i (scaled for long contexts or not) is made on
// the host; the angle is reduced exactly (rope_items.cuh).
//
// What bounds it: each element is read once and written once, 3 flops each; the
// cosines depend on (token, pair) only.  A CTA takes a few tokens with all or
// some of their heads: it issues its first loads, builds the cos/sin table of
// its tokens in shared memory while they are in flight, and rotates.
#include <cuda_runtime.h>

#include <algorithm>

#include "dattn_internal.h"
#include "ptx.cuh"
#include "rope_items.cuh"

namespace dattn {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;      // items whose loads a thread issues together
constexpr int kMaxTokens = 16;  // tokens of a CTA

struct RopeGrid {
    int tokens_per_cta, heads_per_cta;
    int items;  // per row
    FastDiv div_items, div_heads;
};

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads)
    rope_kernel(const __grid_constant__ RopeArgs a, const RopeGrid gr) {
    extern __shared__ float2 table[];  // [tokens_per_cta][8 * rotated items]
    pdl_launch_dependents();
    pdl_wait_primary();
    const int D = a.D, rd = a.rope.rope_dims, half = rd / 2;
    const bool trad = a.rope.traditional != 0;
    const int ir = rope_items(rd, VEC);
    const long long t0 = static_cast<long long>(blockIdx.x) * gr.tokens_per_cta;
    const int nt = static_cast<int>(min(static_cast<long long>(gr.tokens_per_cta), a.tokens - t0));
    const int h0 = blockIdx.y * gr.heads_per_cta;
    const int nh = min(gr.heads_per_cta, a.H - h0);
    const int total = nt * gr.heads_per_cta * gr.items;
    const T *x = reinterpret_cast<const T *>(a.x);
    T *out = reinterpret_cast<T *>(a.out);

    for (int base = 0; base < total; base += kThreads * kUnroll) {
        ItemData<T> d[kUnroll];
        int tok[kUnroll], head[kUnroll], item[kUnroll];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            const int n = base + k * kThreads + static_cast<int>(threadIdx.x);
            const int th = static_cast<int>((static_cast<unsigned long long>(n) * gr.div_items.mul) >> gr.div_items.shift);
            item[k] = n - th * gr.items;
            tok[k] = static_cast<int>((static_cast<unsigned long long>(th) * gr.div_heads.mul) >> gr.div_heads.shift);
            head[k] = th - tok[k] * gr.heads_per_cta;
            if (tok[k] >= nt || head[k] >= nh) {
                tok[k] = -1;
                continue;
            }
            const Item<VEC> it(item[k], rd, D, trad);
            it.load(x + (t0 + tok[k]) * a.x_stride + static_cast<long long>(h0 + head[k]) * D, d[k]);
        }
        if (base == 0) {
            for (int i = threadIdx.x; i < nt * half; i += kThreads) {
                const int s = i / half;
                rope_table_entry(table + s * 8 * ir, ir, i - s * half, __ldg(a.positions + t0 + s),
                                 a.rope, a.gradient != 0);
            }
            __syncthreads();
        }
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            if (tok[k] < 0) continue;
            const Item<VEC> it(item[k], rd, D, trad);
            float2 cs[8];
            if (it.rot) {
#pragma unroll
                for (int e = 0; e < 8; ++e) cs[e] = table[tok[k] * 8 * ir + e * ir + item[k]];
            }
            float y[16];
            rotate_item(it, d[k], cs, y);
            ItemData<T> r;
            T *e = reinterpret_cast<T *>(r.v);
#pragma unroll
            for (int i = 0; i < 16; ++i) e[i] = from_float<T>(y[i]);
            it.store(out + (t0 + tok[k]) * a.out_stride + static_cast<long long>(h0 + head[k]) * D, r);
        }
    }
}

template <typename T>
const void *kernel_of(bool vec) {
    return vec ? reinterpret_cast<const void *>(rope_kernel<T, true>)
               : reinterpret_cast<const void *>(rope_kernel<T, false>);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs &a, int dtype, int sms, cudaStream_t stream) {
    const bool vec = a.rope.rope_dims % 16 == 0 && a.D % 16 == 0;
    RopeGrid gr{};
    gr.items = row_items(a.rope.rope_dims, a.D, vec);
    // A CTA takes one round of kUnroll items per thread: several tokens when
    // heads are few, part of the heads when they are many or when whole tokens
    // would leave SMs without work.
    const int per_cta = kThreads * kUnroll;
    gr.heads_per_cta = std::min(a.H, std::max(1, per_cta / gr.items));
    gr.tokens_per_cta = std::max(
        1, std::min(kMaxTokens, per_cta / (gr.items * gr.heads_per_cta)));
    while (gr.tokens_per_cta > 1 &&
           (a.tokens + gr.tokens_per_cta - 1) / gr.tokens_per_cta < 2LL * sms)
        gr.tokens_per_cta /= 2;
    while (gr.heads_per_cta > 1 && gr.tokens_per_cta == 1 &&
           a.tokens * ((a.H + gr.heads_per_cta - 1) / gr.heads_per_cta) < 2LL * sms &&
           gr.heads_per_cta * gr.items > 32)
        gr.heads_per_cta = (gr.heads_per_cta + 1) / 2;
    gr.div_items = fast_div_of(gr.items);
    gr.div_heads = fast_div_of(gr.heads_per_cta);
    const long long gx = (a.tokens + gr.tokens_per_cta - 1) / gr.tokens_per_cta;
    const long long gy = (a.H + gr.heads_per_cta - 1) / gr.heads_per_cta;
    if (gx <= 0 || gx > 0x7fffffffLL || gy > 65535) return cudaErrorInvalidValue;
    const void *fn = dtype == kDtypeF16    ? kernel_of<__half>(vec)
                     : dtype == kDtypeBf16 ? kernel_of<__nv_bfloat16>(vec)
                                           : kernel_of<float>(vec);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(gx), static_cast<unsigned>(gy));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes =
        static_cast<size_t>(gr.tokens_per_cta) * 8 * rope_items(a.rope.rope_dims, vec) * sizeof(float2);
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
