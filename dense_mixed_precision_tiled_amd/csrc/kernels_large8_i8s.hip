// Kernel instantiations of the "large8" int8 tile with scaled sums (int8 inputs,
// int32 accumulator, float output; all operand layouts and load paths), in a
// translation unit of its own so the library builds in parallel.
#include "gemm_configs.hpp"

namespace libgemm {
hipError_t launch_large8_i8s(const Params &p, int, int akc, int bkc, dim3 grid, hipStream_t s) {
    return launch_layouts<CfgLarge8I8, IT_I8S>(p, akc, bkc, grid, s);
}
}  // namespace libgemm
