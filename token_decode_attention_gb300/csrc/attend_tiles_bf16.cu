// attend_tiles_bf16.cu -- the bf16 instances of attention of many tokens.
#include "attend_tiles_kernel.cuh"

namespace dattn {

const void *attend_tiles_bf16_fn(int dp) {
    return dp == 64    ? reinterpret_cast<const void *>(attend_tiles_kernel<__nv_bfloat16, 64>)
           : dp == 128 ? reinterpret_cast<const void *>(attend_tiles_kernel<__nv_bfloat16, 128>)
                       : reinterpret_cast<const void *>(attend_tiles_kernel<__nv_bfloat16, 256>);
}

}  // namespace dattn
