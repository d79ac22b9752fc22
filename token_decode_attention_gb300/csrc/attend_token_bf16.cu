// attend_token_bf16.cu -- the bf16 instances of attention of one token per sequence.
#include "attend_token_kernel.cuh"

namespace dattn {

const void *attend_token_bf16_fn(int dp, int nt, bool pair, bool cluster) {
    return token_instance<__nv_bfloat16>(dp, nt, pair, cluster);
}

}  // namespace dattn
