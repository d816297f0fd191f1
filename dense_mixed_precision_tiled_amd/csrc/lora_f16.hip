// The adapters' kernels with f16 inputs, in a translation unit of their own so the
// library builds in parallel.
#include "lora_launch.hpp"

namespace libgemm {
hipError_t launch_lora_f16(const LoraParams &p, int out_dtype, bool few, bool vec_xa, bool vec_b,
                          hipStream_t s) {
    return launch_lora<IT_F16>(p, out_dtype, few, vec_xa, vec_b, s);
}
}  // namespace libgemm
