// gemm_quantize_rows: rows of fp16, bf16 or fp32 values to int8 with one scale
// for each row.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/libgemm.h"
#include "gemm_host.hpp"
#include "gemm_kernels.hpp"
#include "gemm_validate.hpp"

namespace libgemm {

struct QuantParams {
    const uint8_t *X;
    uint8_t *Q;
    float *scales;
    int64_t ldx, ldq;  // elements
    int M, K;
};

template <int IN>
__device__ __forceinline__ float quant_load(const uint8_t *row, int64_t k) {
    if constexpr (IN == DT_F32) return reinterpret_cast<const float *>(row)[k];
    else return from_out16<IN>(reinterpret_cast<const uint16_t *>(row)[k]);
}

// One workgroup for each row, in two passes over it.
template <int IN>
__global__ void __launch_bounds__(256) quantize_rows_kernel(QuantParams p) {
    constexpr int ES = IN == DT_F32 ? 4 : 2;
    __shared__ float part[4];
    const int tid = threadIdx.x;
    for (int64_t i = blockIdx.x; i < p.M; i += gridDim.x) {
        const uint8_t *row = p.X + i * p.ldx * ES;
        float a = 0.0f;
        bool bad = false;
        for (int64_t k = tid; k < p.K; k += 256) {
            const float x = quant_load<IN>(row, k);
            bad = bad || !(__builtin_fabsf(x) <= 3.402823466e38f);
            a = fmaxf(a, __builtin_fabsf(x));
        }
        if (bad) a = __builtin_inff();
        for (int m = 32; m; m >>= 1) a = fmaxf(a, __shfl_xor(a, m));
        if ((tid & 63) == 0) part[tid >> 6] = a;
        __syncthreads();
        a = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
        __syncthreads();
        const bool finite = a <= 3.402823466e38f;
        if (tid == 0) p.scales[i] = finite ? a / 127.0f : __builtin_nanf("");
        for (int64_t k = tid; k < p.K; k += 256) {
            const double q = (double)quant_load<IN>(row, k) * 127.0 / (double)a;
            p.Q[i * p.ldq + k] = finite && a > 0.0f ? (uint8_t)(int)rint(q) : 0;
        }
    }
}

}  // namespace libgemm

using namespace libgemm;
using namespace libgemm_host;

extern "C" {

int gemm_validate_quantize_rows(int64_t M, int64_t K, const void *X, int64_t ldx, int in_dtype,
                                const void *Q, int64_t ldq, const float *scales) {
    return validate_quantize_rows(M, K, X, ldx, in_dtype, Q, ldq, scales);
}

int gemm_quantize_rows(int64_t M, int64_t K, const void *X, int64_t ldx, int in_dtype, void *Q,
                       int64_t ldq, float *scales, void *stream) {
    const int st = validate_quantize_rows(M, K, X, ldx, in_dtype, Q, ldq, scales);
    if (st != GEMM_OK) return st;
    if (M == 0) return GEMM_OK;
    QuantParams p{};
    p.X = static_cast<const uint8_t *>(X);
    p.Q = static_cast<uint8_t *>(Q);
    p.scales = scales;
    p.ldx = ldx;
    p.ldq = ldq;
    p.M = (int)M;
    p.K = (int)K;
    void *args[] = {&p};
    const void *f = in_dtype == GEMM_F32   ? (const void *)quantize_rows_kernel<DT_F32>
                    : in_dtype == GEMM_F16 ? (const void *)quantize_rows_kernel<DT_F16>
                                           : (const void *)quantize_rows_kernel<DT_BF16>;
    const dim3 grid((unsigned)(M < (1 << 20) ? M : 1 << 20));
    return hipLaunchKernel(f, grid, dim3(256), args, 0, static_cast<hipStream_t>(stream)) ==
                   hipSuccess
               ? GEMM_OK
               : GEMM_ERR_HIP;
}

}  // extern "C"
