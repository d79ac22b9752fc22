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
// The work of a CTA is rope_tiles.cuh's.
#include <cuda_runtime.h>

#include <algorithm>

#include "dattn_internal.h"
#include "ptx.cuh"
#include "rope_tiles.cuh"

namespace dattn {
namespace {

constexpr size_t kPosBytes = 2 * kRopeThreads * sizeof(uint32_t);

template <typename T, int N, bool FIXED, int HP>
__global__ void __launch_bounds__(kRopeThreads, (kRopeBlocks<T, N, HP>))
    rope_kernel(const __grid_constant__ RopeArgs a, const RopeGrid gr) {
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ uint32_t s_pos[2][kRopeThreads];  // kPosBytes
    pdl_launch_dependents();
    pdl_wait_primary();
    rope_tiles<T, N, FIXED, HP>(a, a.rope, gr, blockIdx.x, gridDim.x, smem, s_pos);
}

struct Instance {
    const void *fn;
    int min_blocks, ring_bytes;
};

template <typename T, int N, bool FIXED, int HP>
Instance instance() {
    return Instance{reinterpret_cast<const void *>(rope_kernel<T, N, FIXED, HP>), kRopeBlocks<T, N, HP>,
                    kRingBytes<T, N, HP>};
}

template <typename T, int N>
Instance instance_of(int hp) {
    return hp == 4 ? instance<T, N, false, 4>() : hp == 2 ? instance<T, N, false, 2>() : instance<T, N, false, 1>();
}
template <typename T>
Instance instance_of(int width, bool fixed, int hp) {
    if (width == 1) return instance<T, 1, false, 1>();
    if (width == 4) return instance_of<T, 4>(hp);
    if (width == 8) return instance_of<T, 8>(hp);
    if constexpr (sizeof(T) == 2)
        if (fixed && hp == 4) return instance<T, 16, true, 4>();
    if (fixed) return hp == 2 ? instance<T, 16, true, 2>() : instance<T, 16, true, 1>();
    return hp == 2 ? instance<T, 16, false, 2>() : instance<T, 16, false, 1>();
}

}  // namespace

cudaError_t launch_rope(const RopeArgs &a, int dtype, int sms, cudaStream_t stream) {
    RopeGrid gr{};
    int hp = 1;
    bool fixed = false;
    const int width = item_width(a.rope.rope_dims, a.D);
    // of items of 16 channels four heads in 16 bits where a thread's item is fixed, two
    // otherwise; of smaller items four
    int most = width < 16 ? 4 : 2;
    if (dtype != kDtypeF32 && width == 16 && kRopeThreads % (a.D / 16) == 0) most = 4;
    if (!rope_grid(a.tokens, a.H, a.D, a.rope.rope_dims, most, sms, &gr, &hp, width, &fixed))
        return cudaErrorInvalidValue;
    const Instance in = dtype == kDtypeF16    ? instance_of<__half>(width, fixed, hp)
                        : dtype == kDtypeBf16 ? instance_of<__nv_bfloat16>(width, fixed, hp)
                                              : instance_of<float>(width, fixed, hp);
    const size_t smem = rope_smem(gr, a.rope.rope_dims, width, in.ring_bytes);
    // resident CTAs: 228 KB an SM, 2 KB of positions and 1 KB of the system's for each
    const long long fit = 228 * 1024 / (static_cast<long long>(smem) + 3 * 1024);
    const long long ctas = std::min(gr.tiles, sms * std::max(1LL, std::min<long long>(in.min_blocks, fit)));
    if (smem + kPosBytes > 48 * 1024) {  // the default limit holds for both parts together
        const cudaError_t e =
            cudaFuncSetAttribute(in.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxDynamicSmem);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(kRopeThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void *args[] = {const_cast<RopeArgs *>(&a), &gr};
    return cudaLaunchKernelExC(&cfg, in.fn, args);
}

}  // namespace dattn
