// attend_merge.cu -- the states of a query head's chunks into its output:
//   out = sum_j 2^(m_j - M) acc_j / sum_j 2^(m_j - M) l_j,   M = max_j m_j,
// m_j the chunk's running maximum (log2 units), l_j and acc_j its sums, in the chunks'
// order, after those of the shared positions where there are such (attend_tiles.cuh; a
// piece or several).  One warp a query head, or four that take the chunks in turn where there are
// many; lanes hold four channels each.
#include "attend_tiles.cuh"

namespace dattn {
namespace {

using attend::ex2;
using attend::Pair;

constexpr unsigned kFull = 0xffffffffu;
constexpr int kWarps = 4;

template <typename T, int WPR>
__global__ void __launch_bounds__(kWarps * 32) merge_kernel(const AttendArgs a, const TokenArgs w,
                                                           const TileArgs t, int dp) {
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
    // state q: of the shared positions for q < pieces, then of the sequence's own
    const float2 *ml = w.ws_ml + row * w.chunks;
    const float *acc = w.ws_acc + row * w.chunks * a.D;
    int pieces = 0, c0 = 0, r = 0;
    bool whole = false;
    if (w.own_only) {
        const attend::Shares s = attend::shares_of(a, t, dp);
        const int h = static_cast<int>(row - static_cast<long long>(b) * a.H);
        const int kvh = fast_div(h, t.div_group);
        const int rr = b * a.group + (h - kvh * a.group), item = rr / tile_rows(dp);
        r = rr - item * tile_rows(dp);
        const int2 who = attend::holders(s, kvh, attend::units_before(t, s, item),
                                         attend::units_before(t, s, item + 1));
        c0 = who.x;
        pieces = who.y - who.x + 1;
        whole = pieces == 1;
    }
    auto slot = [&](int q) {
        return static_cast<long long>(2 * (c0 + q) + (q == 0 ? 1 : 0)) * tile_rows(dp) + r;
    };
    auto ml_of = [&](int q) {
        if (q >= pieces) return ml[q - pieces];
        return whole ? t.whole_ml[row] : t.ml[slot(q)];
    };
    auto acc_of = [&](int q) -> const float * {
        if (q >= pieces) return acc + static_cast<long long>(q - pieces) * a.D;
        return whole ? t.whole_acc + row * a.D : t.acc + slot(q) * a.D;
    };
    const int states = pieces + n;
    float top = -INFINITY;
    for (int q = lane; q < states; q += 32) top = fmaxf(top, ml_of(q).x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
    float4 y[2] = {};
    float l = 0.f;
#pragma unroll 4
    for (int q = sub; q < states; q += WPR) {
        const float2 x = ml_of(q);
        const float *from = acc_of(q);
        const float f = x.x == -INFINITY ? 0.f : ex2(x.x - top);
        l = fmaf(f, x.y, l);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int ch = 4 * lane + 128 * j;
            if (ch >= a.D) continue;
            const float4 z = *reinterpret_cast<const float4 *>(from + ch);
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
                make_uint2(Pair<T>::result(y[j].x * inv, y[j].y * inv), Pair<T>::result(y[j].z * inv, y[j].w * inv));
    }
}

template <typename T>
cudaError_t launch(const AttendArgs &a, const TokenArgs &w, const TileArgs &t, int dp, cudaStream_t stream) {
    const long long rows = static_cast<long long>(a.B) * a.H;
    // states of a row: its chunks, and about as many pieces as CTAs share an item
    long long states = w.chunks;
    if (w.own_only) {
        const long long items = (static_cast<long long>(a.B) * a.group + tile_rows(dp) - 1) / tile_rows(dp) * a.Hk;
        states += 1 + t.ctas / items;
    }
    const bool many = states > 8;
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
    return many ? cudaLaunchKernelEx(&cfg, merge_kernel<T, kWarps>, a, w, t, dp)
                : cudaLaunchKernelEx(&cfg, merge_kernel<T, 1>, a, w, t, dp);
}

}  // namespace

cudaError_t launch_attend_merge(const AttendArgs &a, const TokenArgs &w, const TileArgs *t, int dtype, int dp,
                                cudaStream_t stream) {
    const TileArgs tiles = t != nullptr ? *t : TileArgs{};
    return dtype == kDtypeF16 ? launch<__half>(a, w, tiles, dp, stream)
                              : launch<__nv_bfloat16>(a, w, tiles, dp, stream);
}

}  // namespace dattn
