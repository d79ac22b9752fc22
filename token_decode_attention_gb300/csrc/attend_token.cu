// attend_token.cu -- launchers of attention of one token per sequence
// (attend_token_kernel.cuh) and its f16 instances; the bf16 ones are in
// attend_token_bf16.cu.
#include "attend_token_kernel.cuh"

namespace dattn {

const void *attend_token_bf16_fn(int dp, int nt, bool pair, bool cluster);

namespace {

const void *kernel_of(int dtype, int dp, int nt, bool pair, bool cluster) {
    return dtype == kDtypeF16 ? token_instance<__half>(dp, nt, pair, cluster)
                              : attend_token_bf16_fn(dp, nt, pair, cluster);
}

}  // namespace

cudaError_t attend_token_configure(int max_smem) {
    for (int dtype : {kDtypeF16, kDtypeBf16})
        for (int dp = 64; dp <= 256; dp *= 2)
            for (int columns : {4, 8, 16})
                for (bool cluster : {false, true}) {
                    const void *fn = kernel_of(dtype, dp, columns > 8 ? 2 : 1, columns == 4, cluster);
                    cudaFuncAttributes attr{};
                    cudaError_t e = cudaFuncGetAttributes(&attr, fn);
                    if (e != cudaSuccess) return e;
                    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             max_smem - static_cast<int>(attr.sharedSizeBytes));
                    if (e == cudaSuccess && cluster)
                        e = cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
                    if (e != cudaSuccess) return e;
                }
    return cudaSuccess;
}

cudaError_t attend_token_max_clusters(int dp, int nt, bool pair, int smem, int cluster, int *clusters) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(cluster));
    cfg.blockDim = dim3(kTokenWarps * 32);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaOccupancyMaxActiveClusters(clusters, kernel_of(kDtypeF16, dp, nt, pair, true), &cfg);
}

cudaError_t launch_attend_token(const AttendArgs &a, const TokenArgs &w, int dtype, int dp, int smem,
                                cudaStream_t stream) {
    const void *fn = kernel_of(dtype, dp, w.gq > 8 ? 2 : 1, w.gq <= 4, w.cluster != 0);
    const long long blocks = static_cast<long long>(a.B) * w.head_groups * w.chunks;
    if (fn == nullptr || blocks <= 0 || blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    void *args[] = {const_cast<AttendArgs *>(&a), const_cast<TokenArgs *>(&w)};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(kTokenWarps * 32);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (w.cluster) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = static_cast<unsigned>(w.chunks);
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
    }
    return cudaLaunchKernelExC(&cfg, fn, args);
}

}  // namespace dattn
