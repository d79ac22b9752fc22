// append_q8_int8.cu -- the int8 instances of the append to an 8-bit cache, apart from the
// e4m3 ones so that they compile in parallel.
#include "append_q8_kernel.cuh"

namespace dattn {

const void *append_q8_int8_fn(int width, bool fixed, int hp) { return instance_of<kKvInt8>(width, fixed, hp).fn; }
const void *append_token_int8_fn(int width) { return token_kernel_of<kKvInt8>(width); }

}  // namespace dattn
