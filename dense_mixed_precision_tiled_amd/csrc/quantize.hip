// gemm_quantize_rows: rows of fp16, bf16 or fp32 values to int8 with one scale
// for each row.
//
// Bound by memory (a row is read once and held in registers between the
// maximum and the rounding), so the arithmetic for each value is kept to six
// instructions for 16-bit inputs.  Rows of bf16: 4096 x 16384 in 45 us (4.4 TB/s),
// 2048 x 4096 in 8.2, up to 256 rows of up to 8192 in 3 to 4 (a launch); of fp32: 4096
// x 16384 in 67 (5.0 TB/s), 2048 x 4096 in 9.4, 64 x 16384 in 5.1.
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
struct QuantRow {
    static constexpr int ES = IN == DT_F32 ? 4 : 2;
    static constexpr int NV = ES;  // 16-byte loads of a chunk of 16 values

    // Magnitudes are compared as bit patterns with the sign cleared: their
    // order is that of the values, with Inf and then NaN above all of them,
    // so one maximum finds both the largest value and whether all are finite.
    static constexpr uint32_t kLargest =
        IN == DT_F32 ? 0x7f7fffffu : (IN == DT_F16 ? 0x7bffu : 0x7f7fu);
    __device__ __forceinline__ static uint32_t bits_of(const u32x4 (&v)[NV], int e) {
        if constexpr (ES == 4) return v[e / 4][e % 4] & 0x7fffffffu;
        else return half_of(v[e / 8], e % 8) & 0x7fffu;
    }
    __device__ __forceinline__ static uint32_t largest_bits(const u32x4 (&v)[NV]) {
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < 16; ++e) m = max(m, bits_of(v, e));
        return m;
    }
    __device__ __forceinline__ static float value_of(const u32x4 (&v)[NV], int e) {
        if constexpr (ES == 4) return __uint_as_float(v[e / 4][e % 4]);
        else return from_out16<IN>(half_of(v[e / 8], e % 8));
    }
    __device__ __forceinline__ static float from_bits(uint32_t b) {
        if constexpr (ES == 4) return __uint_as_float(b);
        else return from_out16<IN>(b);
    }

    // The row's factor 127 / a, and the rounding of x * 127 / a.
    //
    // The product of x with the rounded factor is off by at most 3 units of
    // its last place, which only matters next to a tie.  Distinct from a tie,
    // 127 x / a is at least 32 units away from it: |254 x - (2 n + 1) a| is a
    // multiple of x's last place, and a has at most 11 significant bits (fp16;
    // bf16 has 8).  So rounding the product to a multiple of 16 units first puts
    // every tie back in its place and moves nothing across one.  fp32 inputs
    // do the same in 64 bits, dropping 16 of the bits that a distance of 2^20
    // units leaves free.  A row of bf16 values so small that 127 / a would
    // leave the range of fp32 is scaled by 2^64 first, which is exact.
    struct Factor {
        float f, pre;
        double d;
    };
    __device__ __forceinline__ static Factor factor(float a) {
        Factor r{0.0f, 1.0f, 0.0};
        if constexpr (ES == 4) {
            r.d = 127.0 / (double)a;
        } else {
            if (IN == DT_BF16 && a < 0x1p-64f) r.pre = 0x1p64f;
            r.f = 127.0f / (a * r.pre);
        }
        return r;
    }
    // the rounded value in the low byte
    __device__ __forceinline__ static uint32_t round(float x, const Factor &r) {
        if constexpr (ES == 4) {
            const uint64_t b = __builtin_bit_cast(uint64_t, (double)x * r.d);
            const double t = __builtin_bit_cast(double, (b + 0x8000u) & ~(uint64_t)0xffffu);
            return (uint32_t)(int)__builtin_rint(t);
        } else {
            const uint32_t b = __float_as_uint((IN == DT_BF16 ? x * r.pre : x) * r.f);
            // adding 1.5 * 2^23 rounds to an integer (ties to even) in the low bits
            return __float_as_uint(__uint_as_float((b + 8u) & ~15u) + 12582912.0f);
        }
    }
};

// Maximum over the TPR threads of a row (part: one word for each wave).
template <int TPR>
__device__ __forceinline__ uint32_t row_max(uint32_t m, uint32_t *part) {
#pragma unroll
    for (int s = 32; s; s >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, s));
    if constexpr (TPR > 64) {
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) part[wave] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < TPR / 64; ++w) m = max(m, part[w]);
    }
    return m;
}

// TPR threads take one row (256 / TPR rows for a workgroup of 256), C chunks of
// 16 values each: K <= 16 * TPR * C, 16-byte aligned rows of X and Q.  Chunks
// past K, and the values of a last chunk past K, are zero.
template <int IN, int TPR, int C>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) quantize_rows_kernel(QuantParams p) {
    using R = QuantRow<IN>;
    constexpr int NV = R::NV, ROWS = TPR < 256 ? 256 / TPR : 1;
    __shared__ uint32_t part[16];
    const int t = threadIdx.x % TPR;
    const int64_t i = (int64_t)blockIdx.x * ROWS + threadIdx.x / TPR;
    if (i >= p.M) return;  // whole waves: a wave holds one row (TPR >= 64)
    const uint8_t *row = p.X + i * p.ldx * R::ES;
    u32x4 v[C][NV];
    uint32_t m = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int k = (c * TPR + t) * 16;
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            const int kq = k + q * (16 / R::ES), n = min(max(p.K - kq, 0), 16 / R::ES);
            u32x4 w = {0u, 0u, 0u, 0u};
            if (n > 0) w = *reinterpret_cast<const u32x4 *>(row + (int64_t)kq * R::ES);
            v[c][q] = keep_first_bytes(w, n * R::ES);
        }
    }
#pragma unroll
    for (int c = 0; c < C; ++c) m = max(m, R::largest_bits(v[c]));
    m = row_max<TPR>(m, part);
    const bool finite = m <= R::kLargest;
    const float a = R::from_bits(m);
    if (t == 0) p.scales[i] = finite ? a / 127.0f : __builtin_nanf("");
    const bool zero = !finite || m == 0;
    const typename R::Factor f = R::factor(zero ? 1.0f : a);
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int k = (c * TPR + t) * 16;
        if (k >= p.K) continue;
        u32x4 q;
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            uint32_t b[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) b[e] = R::round(R::value_of(v[c], 4 * d + e), f);
            const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400u);
            const uint32_t hi = __builtin_amdgcn_perm(b[3], b[2], 0x04000c0cu);
            q[d] = zero ? 0u : lo | hi;
        }
        uint8_t *dst = p.Q + i * p.ldq + k;
        if (k + 16 <= p.K) {
            *reinterpret_cast<u32x4 *>(dst) = q;
        } else {
            for (int e = 0; e < p.K - k; ++e) dst[e] = (uint8_t)(q[e / 4] >> (8 * (e % 4)));
        }
    }
}

// Any alignment and length: one workgroup for each row, which is read twice.
template <int IN>
__global__ void __launch_bounds__(256) quantize_long_rows_kernel(QuantParams p) {
    using R = QuantRow<IN>;
    __shared__ uint32_t part[16];
    const int tid = threadIdx.x;
    const int64_t i = blockIdx.x;
    const uint8_t *row = p.X + i * p.ldx * R::ES;
    auto bits = [&](int64_t k) -> uint32_t {
        if constexpr (IN == DT_F32) return reinterpret_cast<const uint32_t *>(row)[k];
        else return reinterpret_cast<const uint16_t *>(row)[k];
    };
    uint32_t m = 0;
    for (int64_t k = tid; k < p.K; k += 256)
        m = max(m, bits(k) & (IN == DT_F32 ? 0x7fffffffu : 0x7fffu));
    m = row_max<256>(m, part);
    const bool finite = m <= R::kLargest;
    const float a = R::from_bits(m);
    if (tid == 0) p.scales[i] = finite ? a / 127.0f : __builtin_nanf("");
    const bool zero = !finite || m == 0;
    const typename R::Factor f = R::factor(zero ? 1.0f : a);
    for (int64_t k = tid; k < p.K; k += 256)
        p.Q[i * p.ldq + k] = zero ? 0 : (uint8_t)R::round(R::from_bits(bits(k)), f);
}

}  // namespace libgemm

using namespace libgemm;
using namespace libgemm_host;

namespace {

// Threads for a row and chunks for a thread, the least that hold the row.  Each rule
// against the next larger one, us:
//   64 x 1 up to 1024:    4096 x 512   4.5 (256 x 1: 7.1)
//   256 x 1 up to 4096:   4096 x 4096 11.7 (256 x 2: 13.8)
//   256 x 2 up to 8192:   4096 x 8192 21.0 (1024 x 2: 35.5)
//   1024 x 2 up to 32768: 256 x 16384  5.8, 4096 x 16384 45 (read twice: 29, 115)
template <int IN>
hipError_t launch_quantize(const QuantParams &p, bool aligned, hipStream_t s) {
    QuantParams arg = p;
    void *args[] = {&arg};
    const unsigned M = (unsigned)p.M;
    if (!aligned || p.K > 32768)
        return hipLaunchKernel((const void *)quantize_long_rows_kernel<IN>, dim3(M), dim3(256),
                               args, 0, s);
    if (p.K <= 1024)
        return hipLaunchKernel((const void *)quantize_rows_kernel<IN, 64, 1>, dim3((M + 3) / 4),
                               dim3(256), args, 0, s);
    if (p.K <= 4096)
        return hipLaunchKernel((const void *)quantize_rows_kernel<IN, 256, 1>, dim3(M), dim3(256),
                               args, 0, s);
    if (p.K <= 8192)
        return hipLaunchKernel((const void *)quantize_rows_kernel<IN, 256, 2>, dim3(M), dim3(256),
                               args, 0, s);
    return hipLaunchKernel((const void *)quantize_rows_kernel<IN, 1024, 2>, dim3(M), dim3(1024),
                           args, 0, s);
}

}  // namespace

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
    p.ldx = ldx;
    p.ldq = ldq;
    p.K = (int)K;
    const int es = in_dtype == GEMM_F32 ? 4 : 2;
    const bool aligned = (uintptr_t)X % 16 == 0 && (uintptr_t)Q % 16 == 0 &&
                         (ldx * es) % 16 == 0 && ldq % 16 == 0;
    hipStream_t s = static_cast<hipStream_t>(stream);
    // a grid holds fewer than 2^32 threads: 2^21 rows for each launch
    const int64_t most = (int64_t)1 << 21;
    for (int64_t i = 0; i < M; i += most) {
        p.X = static_cast<const uint8_t *>(X) + i * ldx * es;
        p.Q = static_cast<uint8_t *>(Q) + i * ldq;
        p.scales = scales + i;
        p.M = (int)(M - i < most ? M - i : most);
        const hipError_t e = in_dtype == GEMM_F32   ? launch_quantize<DT_F32>(p, aligned, s)
                             : in_dtype == GEMM_F16 ? launch_quantize<DT_F16>(p, aligned, s)
                                                    : launch_quantize<DT_BF16>(p, aligned, s);
        if (e != hipSuccess) return GEMM_ERR_HIP;
    }
    return GEMM_OK;
}

}  // extern "C"
