// Kernel instantiations of the four-wave LDS-DMA int8 tile (16x16x64 MFMA)
// with scaled sums (float output; K-contiguous A and B only), in a
// translation unit of its own so the library builds in parallel.
#include "gemm_configs.hpp"

namespace libgemm {
hipError_t launch_large_dma16_i8s(const Params &p, int, int akc, int bkc, dim3 grid,
                                  hipStream_t s) {
    using CF = CfgLargeDmaI8_16;
    // the host sends no other layout, alignment or K here
    if (!akc || !bkc || !p.vec_ok || p.K % CF::BK != 0) return hipErrorInvalidValue;
    return launch_params(gemm_dma_kernel<CF, IT_I8S, true, true, false>, grid, dim3(CF::THREADS), p,
                         s);
}
}  // namespace libgemm
