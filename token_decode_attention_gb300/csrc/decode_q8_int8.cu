// decode_q8_int8.cu -- the int8 instances of the decode over an 8-bit cache, apart
// from the e4m3 ones so that they compile in parallel.
#include "decode_q8_kernel.cuh"

namespace dattn {

bool decode_q8_int8_fn(int dp, int nt, bool pair, const void **split, const void **cluster) {
    const Q8Instance *i = q8_instance<kKvInt8>(dp, nt, pair);
    if (i == nullptr) return false;
    *split = i->split;
    *cluster = i->cluster;
    return true;
}

}  // namespace dattn
