// Kernel instantiations of the four-wave LDS-DMA int8 tile (16x16x64 MFMA)
// with scaled sums (float output; K-contiguous A and B only), in a
// translation unit of its own so the library builds in parallel.
#include "gemm_configs.hpp"

namespace libgemm {
hipError_t launch_large_dma16_i8s(const Params &p, int, int akc, int bkc, dim3 grid,
                                  hipStream_t s) {
    // the host sends no other layout here
    if (!akc || !bkc) return hipErrorInvalidValue;
    return launch_dma_one<CfgLargeDmaI8_16, IT_I8S, true, true>(p, grid, s);
}
}  // namespace libgemm
