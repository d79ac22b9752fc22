// attend_tiles.cu -- launchers of attention of many tokens (attend_tiles_kernel.cuh; the bf16
// instances are in attend_tiles_bf16.cu), the kernel that plans a ragged batch, and the one
// that merges the pieces of items that several CTAs shared.
#include "attend_tiles_kernel.cuh"

namespace dattn {

const void *attend_tiles_bf16_fn(int dp);

namespace {

constexpr int kPlanThreads = 1024;

// Inclusive sum over the block's threads, and the block's total.
__device__ long long block_scan(long long x, long long *s_warp, long long *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(kFull, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();  // s_warp of the call before has been read
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    long long sum = 0;
    for (int w = 0; w < kPlanThreads / 32; ++w) {
        if (w == warp) x += sum;
        sum += s_warp[w];
    }
    *total = sum;
    return x;
}

// Tokens of sequence b, in [0, tokens] whatever the offsets are.
__device__ __forceinline__ int2 tokens_of(const AttendArgs &a, int b) {
    const int begin = min(max(__ldg(a.offsets + b), 0), a.tokens);
    return make_int2(begin, min(max(__ldg(a.offsets + b + 1), begin), a.tokens));
}

// One CTA: the items of a ragged batch and the units ahead of each.
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const AttendArgs a, const TileArgs t, int rows,
                                                            int keys) {
    __shared__ long long s_warp[kPlanThreads / 32];
    const int tid = threadIdx.x;
    pdl_wait_primary();
    pdl_launch_dependents();
    long long total = 0, carry = 0;
    if (tid == 0) t.seq_items[0] = 0;
    for (int i0 = 0; i0 < a.B; i0 += kPlanThreads) {
        const int b = i0 + tid;
        long long items = 0;
        if (b < a.B) {
            const int2 own = tokens_of(a, b);
            const int n = own.y - own.x;
            items = (static_cast<long long>(n) * a.group + rows - 1) / rows;
            if (n > attend::live_end(a, b)) atomicOr(a.err, kErrAppendPosition);
        }
        const long long upto = carry + block_scan(items, s_warp, &total);
        // offsets that do not ascend may name more items than there is room for
        if (b < a.B) t.seq_items[b + 1] = static_cast<int>(min(upto, static_cast<long long>(t.max_items)));
        carry += total;
    }
    const int items = static_cast<int>(min(carry, static_cast<long long>(t.max_items)));
    __syncthreads();
    carry = 0;
    if (tid == 0) t.before[0] = 0;
    for (int s0 = 0; s0 < items; s0 += kPlanThreads) {
        const int s = s0 + tid;
        long long units = 0;
        if (s < items) {
            int lo = 0, hi = a.B;  // the last sequence whose items begin at or before s
            while (hi - lo > 1) {
                const int mid = (lo + hi) / 2;
                (t.seq_items[mid] <= s ? lo : hi) = mid;
            }
            const int2 own = tokens_of(a, lo);
            const int row = (s - t.seq_items[lo]) * rows;  // below the sequence's tokens x group
            const int tok = fast_div(row, t.div_group), all = (own.y - own.x) * a.group;
            TileItem it;
            it.b = lo;
            it.token = own.x + tok;
            it.head = row - tok * a.group;
            it.rows = min(rows, all - row);
            const int last = fast_div(row + it.rows - 1, t.div_group);
            it.p0 = attend::live_end(a, lo) - (own.y - own.x) + tok;
            it.lo = attend::seen_by(a, it.p0).lo & ~(t.align - 1);
            it.first = min(a.sinks, it.lo);
            it.n = max(it.p0 + (last - tok) + 1, 0) - it.lo + it.first;
            int4 *at = reinterpret_cast<int4 *>(t.items + s);
            at[0] = make_int4(it.b, it.token, it.head, it.rows);
            at[1] = make_int4(it.p0, it.lo, it.first, it.n);
            units = attend::key_tiles(it.n, keys) + attend::kItemExtra;
        }
        const long long upto = carry + block_scan(units, s_warp, &total);
        if (s < items) t.before[s + 1] = upto;
        carry += total;
    }
    if (tid == 0) {
        t.plan->total = carry;
        t.plan->items = items;
        t.plan->ctas = static_cast<int>(
            max(1LL, min(static_cast<long long>(t.ctas), carry * a.Hk / kTileMinUnits)));
    }
}

constexpr int kJoinWarps = 4, kJoinRows = 8;  // rows of a CTA

// The pieces of the item that the beginning of CTA c's share is the first to cut, into
// `out`.  A warp takes a row, lanes four channels each.
template <typename T>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const AttendArgs a, const TileArgs t, int dp) {
    const int parts = tile_rows(dp) / kJoinRows;
    const int c = 1 + blockIdx.x / parts, part = blockIdx.x % parts;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait_primary();
    pdl_launch_dependents();
    const TileCut cut = t.cuts[c];
    if (cut.first < 0) return;
    const int2 who = make_int2(cut.first, cut.last);
    const int kvh = cut.kvh;
    const int4 *const at = reinterpret_cast<const int4 *>(t.items + cut.item);
    const int4 x0 = at[0], x1 = at[1];
    const TileItem it{x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
    for (int r = part * kJoinRows + warp; r < min(it.rows, (part + 1) * kJoinRows); r += kJoinWarps) {
        const int tok = fast_div(it.head + r, t.div_group);
        const long long row = (it.token + static_cast<long long>(tok)) * a.H +
                              static_cast<long long>(kvh) * a.group + (it.head + r - tok * a.group);
        auto slot = [&](int q) { return static_cast<long long>(2 * q + (q == who.x ? 1 : 0)) * tile_rows(dp) + r; };
        float top = -INFINITY;
        for (int q = who.x + lane; q <= who.y; q += 32) top = fmaxf(top, t.ml[slot(q)].x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
        float4 y[2] = {};
        float l = 0.f;
#pragma unroll 4
        for (int q = who.x; q <= who.y; ++q) {
            const float2 ml = t.ml[slot(q)];
            const float f = ml.x == -INFINITY ? 0.f : ex2(ml.x - top);
            l = fmaf(f, ml.y, l);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int ch = 4 * lane + 128 * j;
                if (ch >= a.D) continue;
                const float4 z = *reinterpret_cast<const float4 *>(t.acc + slot(q) * a.D + ch);
                y[j].x = fmaf(f, z.x, y[j].x);
                y[j].y = fmaf(f, z.y, y[j].y);
                y[j].z = fmaf(f, z.z, y[j].z);
                y[j].w = fmaf(f, z.w, y[j].w);
            }
        }
        const float inv = it.p0 + tok >= 0 ? 1.f / l : 0.f;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int ch = 4 * lane + 128 * j;
            if (ch < a.D)
                *reinterpret_cast<uint2 *>(static_cast<T *>(a.out) + row * a.D + ch) = make_uint2(
                    Pair<T>::result(y[j].x * inv, y[j].y * inv), Pair<T>::result(y[j].z * inv, y[j].w * inv));
        }
    }
}

const void *kernel_of(int dtype, int dp) {
    if (dtype == kDtypeBf16) return attend_tiles_bf16_fn(dp);
    return dp == 64    ? reinterpret_cast<const void *>(attend_tiles_kernel<__half, 64>)
           : dp == 128 ? reinterpret_cast<const void *>(attend_tiles_kernel<__half, 128>)
                       : reinterpret_cast<const void *>(attend_tiles_kernel<__half, 256>);
}

int smem_of(int dp) {
    return dp == 64 ? TileShape<64>::kSmem : dp == 128 ? TileShape<128>::kSmem : TileShape<256>::kSmem;
}

}  // namespace

cudaError_t attend_tiles_configure(int max_smem) {
    for (int dtype : {kDtypeF16, kDtypeBf16})
        for (int dp = 64; dp <= 256; dp *= 2) {
            if (smem_of(dp) > max_smem) return cudaErrorInvalidValue;
            const cudaError_t e = cudaFuncSetAttribute(kernel_of(dtype, dp),
                                                       cudaFuncAttributeMaxDynamicSharedMemorySize, smem_of(dp));
            if (e != cudaSuccess) return e;
        }
    return cudaSuccess;
}

cudaError_t launch_attend_tiles(const AttendArgs &a, const TileArgs &t, const TileMaps &m, int dtype, int dp,
                                cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (t.plan != nullptr) {
        cfg.gridDim = dim3(1);
        cfg.blockDim = dim3(kPlanThreads);
        const cudaError_t e = cudaLaunchKernelEx(&cfg, plan_kernel, a, t, tile_rows(dp), tile_keys(dp));
        if (e != cudaSuccess) return e;
    }
    void *args[] = {const_cast<AttendArgs *>(&a), const_cast<TileArgs *>(&t), const_cast<TileMaps *>(&m)};
    cfg.gridDim = dim3(static_cast<unsigned>(t.ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem_of(dp));
    cudaError_t e = cudaLaunchKernelExC(&cfg, kernel_of(dtype, dp), args);
    if (e != cudaSuccess || t.plan == nullptr || t.ctas == 1) return e;
    cfg.gridDim = dim3(static_cast<unsigned>((t.ctas - 1) * (tile_rows(dp) / kJoinRows)));
    cfg.blockDim = dim3(kJoinWarps * 32);
    cfg.dynamicSmemBytes = 0;
    return dtype == kDtypeF16 ? cudaLaunchKernelEx(&cfg, join_kernel<__half>, a, t, dp)
                              : cudaLaunchKernelEx(&cfg, join_kernel<__nv_bfloat16>, a, t, dp);
}

}  // namespace dattn
