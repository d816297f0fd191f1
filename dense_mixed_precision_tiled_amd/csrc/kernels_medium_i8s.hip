// Kernel instantiations of the "medium" int8 tile with scaled sums (int8 inputs,
// int32 accumulator, float output; all operand layouts and load paths), in a
// translation unit of its own so the library builds in parallel.
#include "gemm_configs.hpp"

namespace libgemm {
hipError_t launch_medium_i8s(const Params &p, int, int akc, int bkc, dim3 grid, hipStream_t s) {
    return launch_layouts<CfgMediumI8, IT_I8S>(p, akc, bkc, grid, s);
}
}  // namespace libgemm
