// The mixture-of-experts kernels for bf16 activations and int8 weights, in a
// translation unit of its own so the library builds in parallel.
#include "moe.hpp"

namespace libgemm {
hipError_t launch_moe_bf16_i8(const MoeParams &p, int cus, bool vec, hipStream_t s) {
    return vec ? moe_launch<IT_BF16, true, true>(p, cus, s)
               : moe_launch<IT_BF16, true, false>(p, cus, s);
}
}  // namespace libgemm
