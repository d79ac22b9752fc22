// attend_merge.cu -- the states of a query head's chunks into its output:
//   out = sum_j 2^(m_j - M) acc_j / sum_j 2^(m_j - M) l_j,   M = max_j m_j,
// m_j the chunk's running maximum (log2 units), l_j and acc_j its sums, in the chunks'
// order.  One warp a query head, or four that take the chunks in turn where there are
// many; lanes hold four channels each.
#include "attend_rows.cuh"

namespace dattn {
namespace {

using attend::ex2;
using attend::Pair;

constexpr unsigned kFull = 0xffffffffu;
constexpr int kWarps = 4;

template <typename T, int WPR>
__global__ void __launch_bounds__(kWarps * 32) merge_kernel(const AttendArgs a, const TokenArgs w) {
    __shared__ float4 s_acc[WPR > 1 ? kWarps : 1][64];
    __shared__ float s_l[kWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = warp % WPR;
    const long long row = static_cast<long long>(blockIdx.x) * (kWarps / WPR) + warp / WPR;
    if (row >= static_cast<long long>(a.B) * a.H) return;  // whole CTAs where warps share a row
    const int b = static_cast<int>(row / a.H);
    pdl_wait_primary();
    pdl_launch_dependents();
    attend::Seen v = attend::seen_by(a, attend::live_end(a, b) - 1);
    if (w.own_only) v.lo = min(a.shared, v.end);
    const int tiles = (v.count() + kTokenTile - 1) / kTokenTile;
    const int n = max(1, (tiles + w.chunk_tiles - 1) / w.chunk_tiles);
    const float2 *ml = w.ws_ml + row * w.chunks;
    const float *acc = w.ws_acc + row * w.chunks * a.D;
    float top = -INFINITY;
    for (int q = lane; q < n; q += 32) top = fmaxf(top, ml[q].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
    float4 y[2] = {};
    float l = 0.f;
#pragma unroll 4
    for (int q = sub; q < n; q += WPR) {
        const float2 x = ml[q];
        const float f = x.x == -INFINITY ? 0.f : ex2(x.x - top);
        l = fmaf(f, x.y, l);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int ch = 4 * lane + 128 * j;
            if (ch >= a.D) continue;
            const float4 z = *reinterpret_cast<const float4 *>(acc + static_cast<long long>(q) * a.D + ch);
            y[j].x = fmaf(f, z.x, y[j].x);
            y[j].y = fmaf(f, z.y, y[j].y);
            y[j].z = fmaf(f, z.z, y[j].z);
            y[j].w = fmaf(f, z.w, y[j].w);
        }
    }
    if constexpr (WPR > 1) {
        s_acc[warp][lane] = y[0];
        s_acc[warp][lane + 32] = y[1];
        if (lane == 0) s_l[warp] = l;
        __syncthreads();
        if (warp != 0) return;
#pragma unroll
        for (int o = 1; o < WPR; ++o) {
            l += s_l[o];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float4 z = s_acc[o][lane + 32 * j];
                y[j].x += z.x, y[j].y += z.y, y[j].z += z.z, y[j].w += z.w;
            }
        }
    }
    const float inv = 1.f / l;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int ch = 4 * lane + 128 * j;
        if (ch < a.D)
            *reinterpret_cast<uint2 *>(static_cast<T *>(a.out) + row * a.D + ch) =
                make_uint2(Pair<T>::narrow(y[j].x * inv, y[j].y * inv), Pair<T>::narrow(y[j].z * inv, y[j].w * inv));
    }
}

template <typename T>
cudaError_t launch(const AttendArgs &a, const TokenArgs &w, cudaStream_t stream) {
    const long long rows = static_cast<long long>(a.B) * a.H;
    const bool many = w.chunks > 8;
    const long long blocks = many ? rows : (rows + kWarps - 1) / kWarps;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(kWarps * 32);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return many ? cudaLaunchKernelEx(&cfg, merge_kernel<T, kWarps>, a, w)
                : cudaLaunchKernelEx(&cfg, merge_kernel<T, 1>, a, w);
}

}  // namespace

cudaError_t launch_attend_merge(const AttendArgs &a, const TokenArgs &w, int dtype, cudaStream_t stream) {
    return dtype == kDtypeF16 ? launch<__half>(a, w, stream) : launch<__nv_bfloat16>(a, w, stream);
}

}  // namespace dattn
