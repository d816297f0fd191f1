// The mixture-of-experts kernels for bf16 activations and weights of the same type, in a
// translation unit of its own so the library builds in parallel.
#include "moe.hpp"

namespace libgemm {
hipError_t launch_moe_bf16(const MoeParams &p, int cus, bool vec, hipStream_t s) {
    return vec ? moe_launch<IT_BF16, false, true>(p, cus, s)
               : moe_launch<IT_BF16, false, false>(p, cus, s);
}
}  // namespace libgemm
