// decode_q8.cu -- launchers of the decode over an 8-bit cache
// (decode_q8_kernel.cuh) and its e4m3 instances; the int8 ones are in
// decode_q8_int8.cu.
#include "decode_q8_kernel.cuh"

namespace dattn {

bool decode_q8_int8_fn(int dp, int nt, bool pair, const void **split, const void **cluster);

namespace {

const void *kernel_of(int dp, int nt, bool pair, int kv, bool cluster) {
    const void *s = nullptr, *c = nullptr;
    if (kv == kKvInt8) {
        if (!decode_q8_int8_fn(dp, nt, pair, &s, &c)) return nullptr;
    } else if (const Q8Instance *i = q8_instance<kKvE4m3>(dp, nt, pair)) {
        s = i->split;
        c = i->cluster;
    }
    return cluster ? c : s;
}

}  // namespace

cudaError_t decode_q8_configure(int max_smem) {
    for (int dp = 64; dp <= 256; dp *= 2)
        for (int columns : {4, 8, 16})
            for (int kv : {kKvE4m3, kKvInt8})
                for (bool cluster : {false, true}) {
                    const void *fn = kernel_of(dp, columns > 8 ? 2 : 1, columns == 4, kv, cluster);
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

cudaError_t decode_q8_max_clusters(int dp, int nt, bool pair, int smem, int cluster, int *clusters) {
    const Q8Instance *i = q8_instance<kKvE4m3>(dp, nt, pair);
    if (i == nullptr) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(cluster));
    cfg.blockDim = dim3(kQ8Warps * 32);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaOccupancyMaxActiveClusters(clusters, i->cluster, &cfg);
}

cudaError_t launch_decode_q8(const Q8DecodeArgs &a, int dp, int nt, int kv, int smem,
                             cudaStream_t stream) {
    const void *fn = kernel_of(dp, nt, q8_pair(a.gq), kv, a.cluster > 0);
    if (fn == nullptr || a.partitions <= 0 || a.cluster > kMaxCluster)
        return cudaErrorInvalidValue;
    void *args[] = {const_cast<Q8DecodeArgs *>(&a)};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.partitions));
    cfg.blockDim = dim3(kQ8Warps * 32);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (a.cluster > 0) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = static_cast<unsigned>(a.cluster);
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
    }
    return cudaLaunchKernelExC(&cfg, fn, args);
}

}  // namespace dattn
