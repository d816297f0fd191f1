// gemm_checkpoint_pack, _unpack and _act_grad: activations to and from the 8-bit
// format of checkpoint.hpp.
//
// One pass over the data, bound by memory: a lane takes 8 values of a row (16 bytes
// of a 16-bit type, 8 of Q), four lanes a block of 32.  The row of an item is found
// with one multiplication, so that short and odd rows fill the waves too.  4096 x 16384
// values of bf16, call after call: packed in 41 us (5.0 TB/s, a copy's rate; fp32 61, 5.5 TB/s),
// unpacked in 38 (5.3), D = G * gelu'(X^) in 68 to 74 (5.0 to 4.6; about 30 vector instructions for
// each value beside the memory), with ReLU or SiLU 62 to 64.  Lines that are not whole 16 bytes
// take three times as long (packing 113 us).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/libgemm.h"
#include "checkpoint.hpp"
#include "gemm_host.hpp"
#include "gemm_validate.hpp"
#include "moe.hpp"

namespace libgemm {

struct CkParams {
    const uint8_t *X;  // pack: X; act_grad: G
    uint8_t *Q, *S, *D;
    int64_t ldx, ldq, lds, ldd;  // elements
    uint32_t items;              // rows * lanes, below 2^31
    uint32_t lanes;              // lanes of a row: four for each block
    CkDivisor div;               // by lanes
    int K;
};

// Items of a thread, 256 apart.  (us of 4096 x 16384 values, packing, unpacking and with GELU: two
// 42, 39 and 73, one 43, 49 and 74, four 47, 44 and 78, eight 49, 92 and 148; packing 100 x 4104 one
// 3.4, two 4.3, four 6.3.)
constexpr int kCkItems = 2;

template <int DT>
constexpr int ck_size = DT == DT_F32 ? 4 : 2;

// Values k .. k+7 of a row (n of them, 0 to 8), the others 0.
template <int DT, bool VEC>
__device__ __forceinline__ void ck_load8(const uint8_t *row, int64_t k, int n, u32x4 (&v)[ck_size<DT> / 2]) {
    constexpr int ES = ck_size<DT>, PER = 16 / ES;
#pragma unroll
    for (int q = 0; q < ES / 2; ++q) {
        u32x4 w = {0u, 0u, 0u, 0u};
        const int m = min(max(n - q * PER, 0), PER);
        if constexpr (VEC) {
            if (m > 0) w = *reinterpret_cast<const u32x4 *>(row + (k + q * PER) * ES);
            w = keep_first_bytes(w, m * ES);
        } else {
#pragma unroll
            for (int e = 0; e < PER; ++e) {
                if (e >= m) continue;
                if constexpr (ES == 4)
                    w[e] = reinterpret_cast<const uint32_t *>(row)[k + q * PER + e];
                else
                    w[e / 2] |= (uint32_t)reinterpret_cast<const uint16_t *>(row)[k + e]
                                << (16 * (e % 2));
            }
        }
        v[q] = w;
    }
}
template <int DT>
__device__ __forceinline__ float ck_value(const u32x4 (&v)[ck_size<DT> / 2], int e) {
    if constexpr (DT == DT_F32) return __uint_as_float(v[e / 4][e % 4]);
    else return from_out16<DT>(half_of(v[0], e));
}

// Largest magnitude bits of the four lanes of a quad.
__device__ __forceinline__ uint32_t quad_max(uint32_t m) {
    m = max(m, quad_xor<1>(m));
    return max(m, quad_xor<2>(m));
}

template <int IN, bool VEC>
__global__ void __launch_bounds__(256) checkpoint_pack_kernel(CkParams p) {
    constexpr int ES = ck_size<IN>;
    constexpr uint32_t kLargest = IN == DT_F32 ? 0x7f7fffffu : (IN == DT_F16 ? 0x7bffu : 0x7f7fu);
    const uint32_t base = blockIdx.x * (256u * kCkItems) + threadIdx.x;
    u32x4 v[kCkItems][ES / 2];
    uint32_t row[kCkItems], lane[kCkItems];
#pragma unroll
    for (int u = 0; u < kCkItems; ++u) {
        // (items past the last are the last quad's again; they store nothing)
        const uint32_t i = min(base + u * 256u, p.items - 4u + (threadIdx.x & 3u));
        row[u] = ck_div(i, p.div);
        lane[u] = i - row[u] * p.lanes;
        const int64_t k = (int64_t)lane[u] * 8;
        ck_load8<IN, VEC>(p.X + row[u] * p.ldx * ES, k, (int)min(max(p.K - k, (int64_t)0), (int64_t)8),
                          v[u]);
    }
#pragma unroll
    for (int u = 0; u < kCkItems; ++u) {
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if constexpr (ES == 4) m = max(m, v[u][e / 4][e % 4] & 0x7fffffffu);
            else m = max(m, half_of(v[u][0], e) & 0x7fffu);
        }
        m = quad_max(m);
        const bool finite = m <= kLargest;
        // the exponent field of the largest value is 127 + floor(log2), 0 below 2^-126
        uint32_t S;
        if constexpr (IN == DT_F16) S = __float_as_uint(from_out16<IN>(m)) >> 23;
        else S = m >> (IN == DT_F32 ? 23 : 7);
        S = finite ? S : 255u;
        const int up = 133 - (int)S;
        u32x2 q;
#pragma unroll
        for (int d = 0; d < 2; ++d) {
            uint32_t b[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                // a power of two: exact but for what rounds to 0 anyway.  Adding
                // 1.5 * 2^23 rounds to an integer, ties to even, in the low byte
                float x = __builtin_ldexpf(ck_value<IN>(v[u], 4 * d + e), up);
                x = __builtin_amdgcn_fmed3f(x, -127.0f, 127.0f);
                b[e] = __float_as_uint(x + 12582912.0f);
            }
            const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400u);
            const uint32_t hi = __builtin_amdgcn_perm(b[3], b[2], 0x04000c0cu);
            q[d] = finite ? lo | hi : 0u;
        }
        if (base + u * 256u >= p.items) continue;
        const int64_t k = (int64_t)lane[u] * 8;
        uint8_t *dst = p.Q + row[u] * p.ldq + k;
        if (VEC && k + 8 <= p.K) {
            *reinterpret_cast<u32x2 *>(dst) = q;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (k + e < p.K) dst[e] = (uint8_t)(q[e / 4] >> (8 * (e % 4)));
        }
        if ((lane[u] & 3) == 0) p.S[row[u] * p.lds + lane[u] / 4] = (uint8_t)S;
    }
}

// exp(a^2 / 2) erfc(a / sqrt 2) / 2 for a >= 0 as a polynomial in t = 1 / (1 + 0.35 a),
// fitted over a in [0, 14] to the least largest error relative to itself + a / sqrt(2 pi)
// (Lawson's iteration on 4000 Chebyshev points): off by at most 9e-8 of that, 3.2e-7 as
// evaluated.  Past that the exponential it is multiplied with is 0 in fp32.
__device__ __forceinline__ float ck_tail(float a) {
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(a, 0.35f, 1.0f));
    float r = 0.044291477650403976f;
    r = __builtin_fmaf(r, t, -0.18242865800857544f);
    r = __builtin_fmaf(r, t, 0.2062307447195053f);
    r = __builtin_fmaf(r, t, 0.014985134825110435f);
    r = __builtin_fmaf(r, t, 0.13894817233085632f);
    r = __builtin_fmaf(r, t, 0.1384863704442978f);
    r = __builtin_fmaf(r, t, 0.13946348428726196f);
    r = __builtin_fmaf(r, t, 2.3313299607252702e-05f);
    return r;
}

// g times the slope of an activation function at x.
template <int ACT>
__device__ __forceinline__ float ck_grad(float g, float x) {
    if constexpr (ACT == ACT_RELU) {
        // selected: an Inf or a NaN of g where the slope is 0 has no part in it
        return x > 0.0f ? g : (x != x ? x : 0.0f);
    } else if constexpr (ACT == ACT_GELU) {
        // Phi(x) + x phi(x), from y = Phi(-a) - a phi(a) = exp(-a^2 / 2) (tail(a) - a / sqrt(2 pi)),
        // a = |x|: y itself for x < 0, so that it keeps its relative precision as it goes to 0,
        // and 1 - y for the others.  (x is finite, or NaN; x^2 is exact, x having seven bits, and
        // its product with the constant is rounded: x^2 2^-24 relatively)
        const float a = __builtin_fabsf(x), e = __builtin_amdgcn_exp2f(x * x * -0.72134752f);
        const float r = __builtin_fmaf(a, -0.39894228f, ck_tail(a));
        return g * (x < 0.0f ? e * r : __builtin_fmaf(-e, r, 1.0f));
    } else {
        // from exp(-|x|), so that neither s nor 1 - s cancels
        const float e = __expf(-__builtin_fabsf(x));
        const float high = __builtin_amdgcn_rcpf(1.0f + e), low = e * high;
        return g * __builtin_fmaf(x * high, low, x < 0.0f ? low : high);
    }
}

// Eight values to a row: n of them.
template <int DT, bool VEC>
__device__ __forceinline__ void ck_store8(uint8_t *row, int64_t k, int n, const float (&y)[8]) {
    if constexpr (DT == DT_F32) {
        float *d = reinterpret_cast<float *>(row) + k;
        if (VEC && n >= 8) {
            reinterpret_cast<f32x4 *>(d)[0] = f32x4{y[0], y[1], y[2], y[3]};
            reinterpret_cast<f32x4 *>(d)[1] = f32x4{y[4], y[5], y[6], y[7]};
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < n) d[e] = y[e];
        }
    } else {
        uint16_t *d = reinterpret_cast<uint16_t *>(row) + k;
        uint32_t h[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] = to_out16<DT>(y[e], false);
        if (VEC && n >= 8) {
            *reinterpret_cast<u32x4 *>(d) = u32x4{h[0] | (h[1] << 16), h[2] | (h[3] << 16),
                                                  h[4] | (h[5] << 16), h[6] | (h[7] << 16)};
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < n) d[e] = (uint16_t)h[e];
        }
    }
}

// ACT_NONE: D = X^; otherwise D = G * act'(X^).
template <int DT, int ACT, bool VEC>
__global__ void __launch_bounds__(256) checkpoint_use_kernel(CkParams p) {
    constexpr int ES = ck_size<DT>;
    const uint32_t base = blockIdx.x * (256u * kCkItems) + threadIdx.x;
    u32x4 g[ACT == ACT_NONE ? 1 : kCkItems][ES / 2];
    u32x2 q[kCkItems];
    uint32_t S[kCkItems], row[kCkItems], lane[kCkItems];
#pragma unroll
    for (int u = 0; u < kCkItems; ++u) {
        const uint32_t i = min(base + u * 256u, p.items - 1u);
        row[u] = ck_div(i, p.div);
        lane[u] = i - row[u] * p.lanes;
        const int64_t k = (int64_t)lane[u] * 8;
        const int n = (int)min(max(p.K - k, (int64_t)0), (int64_t)8);
        S[u] = p.S[row[u] * p.lds + lane[u] / 4];
        const uint8_t *src = p.Q + row[u] * p.ldq + k;
        q[u] = u32x2{0u, 0u};
        if constexpr (VEC) {
            if (n > 0) q[u] = *reinterpret_cast<const u32x2 *>(src);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < n) q[u][e / 4] |= (uint32_t)src[e] << (8 * (e % 4));
        }
        if constexpr (ACT != ACT_NONE)
            ck_load8<DT, VEC>(p.X + row[u] * p.ldx * ES, k, n, g[u]);
    }
#pragma unroll
    for (int u = 0; u < kCkItems; ++u) {
        const float unit = ck_unit(S[u]);
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float x = ck_int(q[u][e / 4], e % 4) * unit;
            if constexpr (ACT == ACT_NONE) y[e] = x;
            else y[e] = ck_grad<ACT>(ck_value<DT>(g[u], e), x);
        }
        if (base + u * 256u >= p.items) continue;
        const int64_t k = (int64_t)lane[u] * 8;
        ck_store8<DT, VEC>(p.D + row[u] * p.ldd * ES, k,
                           (int)min(max(p.K - k, (int64_t)0), (int64_t)8), y);
    }
}

}  // namespace libgemm

using namespace libgemm;
using namespace libgemm_host;

namespace {

typedef void (*ck_kernel)(CkParams);

// Launches over all rows, fewer than 2^31 items at a time.
int ck_launch(ck_kernel kernel, CkParams p, int64_t M, int64_t K, int xsz, int dsz,
              hipStream_t s) {
    p.K = (int)K;
    p.lanes = (uint32_t)(checkpoint_blocks(K) * 4);
    p.div = ck_divisor(p.lanes);
    const int64_t most = 0x7fffffff / p.lanes;  // (lanes <= 2^28)
    for (int64_t i = 0; i < M; i += most) {
        const int64_t rows = M - i < most ? M - i : most;
        CkParams q = p;
        q.items = (uint32_t)(rows * p.lanes);
        q.X = p.X + i * p.ldx * xsz;
        q.Q = p.Q + i * p.ldq;
        q.S = p.S + i * p.lds;
        q.D = p.D + i * p.ldd * dsz;
        void *args[] = {&q};
        const unsigned blocks = (unsigned)cdiv(q.items, 256 * kCkItems);
        if (hipLaunchKernel((const void *)kernel, dim3(blocks), dim3(256), args, 0, s) != hipSuccess)
            return GEMM_ERR_HIP;
    }
    return GEMM_OK;
}

template <int DT>
ck_kernel use_kernel(int act, bool vec) {
    switch (act) {
    case GEMM_ACT_RELU:
        return vec ? checkpoint_use_kernel<DT, ACT_RELU, true> : checkpoint_use_kernel<DT, ACT_RELU, false>;
    case GEMM_ACT_GELU:
        return vec ? checkpoint_use_kernel<DT, ACT_GELU, true> : checkpoint_use_kernel<DT, ACT_GELU, false>;
    case GEMM_ACT_SILU:
        return vec ? checkpoint_use_kernel<DT, MOE_SILU, true> : checkpoint_use_kernel<DT, MOE_SILU, false>;
    default:
        return vec ? checkpoint_use_kernel<DT, ACT_NONE, true> : checkpoint_use_kernel<DT, ACT_NONE, false>;
    }
}

int run_use(int64_t M, int64_t K, const void *Q, int64_t ldq, const uint8_t *S, int64_t lds,
            const void *G, int64_t ldg, int act, void *D, int64_t ldd, int dtype, void *stream) {
    if (M == 0 || K == 0) return GEMM_OK;
    CkParams p{};
    p.X = static_cast<const uint8_t *>(G);
    p.Q = static_cast<uint8_t *>(const_cast<void *>(Q));
    p.S = const_cast<uint8_t *>(S);
    p.D = static_cast<uint8_t *>(D);
    p.ldx = ldg;
    p.ldq = ldq;
    p.lds = lds;
    p.ldd = ldd;
    const int sz = out_size(dtype);
    const bool vec = (uintptr_t)Q % 16 == 0 && ldq % 16 == 0 && (uintptr_t)D % 16 == 0 &&
                     ldd * sz % 16 == 0 && (uintptr_t)G % 16 == 0 && ldg * sz % 16 == 0;
    const ck_kernel k = dtype == GEMM_F32   ? use_kernel<DT_F32>(act, vec)
                        : dtype == GEMM_F16 ? use_kernel<DT_F16>(act, vec)
                                            : use_kernel<DT_BF16>(act, vec);
    return ck_launch(k, p, M, K, sz, sz, static_cast<hipStream_t>(stream));
}

}  // namespace

extern "C" {

int gemm_validate_checkpoint_pack(int64_t M, int64_t K, const void *X, int64_t ldx, int in_dtype,
                                  const void *Q, int64_t ldq, const uint8_t *S, int64_t lds) {
    return validate_checkpoint_pack(M, K, X, ldx, in_dtype, Q, ldq, S, lds);
}

int gemm_validate_checkpoint_unpack(int64_t M, int64_t K, const void *Q, int64_t ldq,
                                    const uint8_t *S, int64_t lds, const void *D, int64_t ldd,
                                    int out_dtype) {
    return validate_checkpoint_unpack(M, K, Q, ldq, S, lds, D, ldd, out_dtype);
}

int gemm_validate_checkpoint_act_grad(int64_t M, int64_t K, const void *Q, int64_t ldq,
                                      const uint8_t *S, int64_t lds, const void *G, int64_t ldg,
                                      int activation, const void *D, int64_t ldd, int dtype) {
    return validate_checkpoint_act_grad(M, K, Q, ldq, S, lds, G, ldg, activation, D, ldd, dtype);
}

int gemm_checkpoint_pack(int64_t M, int64_t K, const void *X, int64_t ldx, int in_dtype, void *Q,
                         int64_t ldq, uint8_t *S, int64_t lds, void *stream) {
    const int st = validate_checkpoint_pack(M, K, X, ldx, in_dtype, Q, ldq, S, lds);
    if (st != GEMM_OK) return st;
    if (M == 0 || K == 0) return GEMM_OK;
    CkParams p{};
    p.X = static_cast<const uint8_t *>(X);
    p.Q = static_cast<uint8_t *>(Q);
    p.S = S;
    p.ldx = ldx;
    p.ldq = ldq;
    p.lds = lds;
    const int sz = out_size(in_dtype);
    const bool vec = (uintptr_t)Q % 16 == 0 && ldq % 16 == 0 && (uintptr_t)X % 16 == 0 &&
                     ldx * sz % 16 == 0;
    ck_kernel k;
    if (in_dtype == GEMM_F32)
        k = vec ? checkpoint_pack_kernel<DT_F32, true> : checkpoint_pack_kernel<DT_F32, false>;
    else if (in_dtype == GEMM_F16)
        k = vec ? checkpoint_pack_kernel<DT_F16, true> : checkpoint_pack_kernel<DT_F16, false>;
    else
        k = vec ? checkpoint_pack_kernel<DT_BF16, true> : checkpoint_pack_kernel<DT_BF16, false>;
    return ck_launch(k, p, M, K, sz, 0, static_cast<hipStream_t>(stream));
}

int gemm_checkpoint_unpack(int64_t M, int64_t K, const void *Q, int64_t ldq, const uint8_t *S,
                           int64_t lds, void *D, int64_t ldd, int out_dtype, void *stream) {
    const int st = validate_checkpoint_unpack(M, K, Q, ldq, S, lds, D, ldd, out_dtype);
    if (st != GEMM_OK) return st;
    return run_use(M, K, Q, ldq, S, lds, nullptr, 0, GEMM_ACT_NONE, D, ldd, out_dtype, stream);
}

int gemm_checkpoint_act_grad(int64_t M, int64_t K, const void *Q, int64_t ldq, const uint8_t *S,
                             int64_t lds, const void *G, int64_t ldg, int activation, void *D,
                             int64_t ldd, int dtype, void *stream) {
    const int st = validate_checkpoint_act_grad(M, K, Q, ldq, S, lds, G, ldg, activation, D, ldd,
                                                dtype);
    if (st != GEMM_OK) return st;
    return run_use(M, K, Q, ldq, S, lds, G, ldg, activation, D, ldd, dtype, stream);
}

}  // extern "C"
