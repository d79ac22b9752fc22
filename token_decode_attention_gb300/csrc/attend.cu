// attend.cu -- attention over a 16-bit cache with grouped heads, a warp for each token and
// query head:
//   out[t,h,:] = sum_j softmax_j( Q[t,h,:] . K[j] / sqrt(D) ) V[j],  j the positions that t sees
// in fp32 with a running maximum.
#include "attend_rows.cuh"

namespace dattn {
namespace {

constexpr int kWarps = 8;

template <typename T>
__global__ void __launch_bounds__(kWarps * 32) attend_kernel(const AttendArgs a) {
    const int lane = threadIdx.x & 31;
    const long long u = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const long long t = u / a.H;
    const int h = static_cast<int>(u - t * a.H);
    if (t >= a.tokens) return;
    int b = static_cast<int>(t), back = 0;  // tokens of the sequence behind this one
    if (a.offsets != nullptr) {
        int lo = 0, hi = a.B;  // the last sequence that begins at or before t
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            (__ldg(a.offsets + mid) <= t ? lo : hi) = mid;
        }
        b = lo;
        const int begin = __ldg(a.offsets + b), end = __ldg(a.offsets + b + 1);
        if (t < begin || t >= end) return;  // padding
        back = static_cast<int>(end - 1 - t);
    }
    const int p = attend::live_end(a, b) - 1 - back;
    if (p < 0 && h == 0 && lane == 0) atomicOr(a.err, kErrAppendPosition);
    attend::attend_row<T>(a, b, t, h, attend::seen_by(a, p), lane);
}

}  // namespace

cudaError_t launch_attend(const AttendArgs &a, int dtype, cudaStream_t stream) {
    const long long warps = static_cast<long long>(a.tokens) * a.H;
    const long long blocks = (warps + kWarps - 1) / kWarps;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    if (dtype == kDtypeF16)
        attend_kernel<__half><<<static_cast<unsigned>(blocks), kWarps * 32, 0, stream>>>(a);
    else
        attend_kernel<__nv_bfloat16><<<static_cast<unsigned>(blocks), kWarps * 32, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace dattn
