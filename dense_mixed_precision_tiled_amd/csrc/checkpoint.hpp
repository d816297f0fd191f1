// The 8-bit format of activation checkpoints (MXINT8 of the OCP Microscaling
// Formats specification): 32 consecutive values of a row share the power of two
// 2^(S - 127), and each value is 2^(S - 127) * Q / 64 with Q an int8.
#pragma once

#include "gemm_kernels.hpp"

namespace libgemm {

constexpr int kCkBlock = 32;  // values that share a scale

// 2^(S - 133), the value of one unit of Q, in fp32 (below 2^-126 as a subnormal, which
// is exact); S = 255 stands for NaN.
__device__ __forceinline__ float ck_unit(uint32_t S) {
    return S == 255 ? __uint_as_float(0x7fc00000u) : __builtin_ldexpf(1.0f, (int)S - 133);
}

// Byte e of a dword as a signed integer in fp32 (one conversion that selects its byte).
__device__ __forceinline__ float ck_int(uint32_t d, int e) {
    return (float)(int8_t)(uint8_t)(d >> (8 * e));
}

// Two exact values of IT's type from fp32 ones, the first in the low half.  bf16 takes
// the upper halves: the values of a block have at most seven significant bits.
template <int IT>
__device__ __forceinline__ uint32_t ck_pair(float a, float b) {
    if constexpr (IT == IT_BF16) {
        return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
    } else {
        return (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)a) |
               ((uint32_t)__builtin_bit_cast(uint16_t, (_Float16)b) << 16);
    }
}

// Quotient by a divisor d in [2, 2^31) of numbers below 2^31 (a multiplication by
// ceil(2^(31+l) / d), 2^(l-1) < d <= 2^l: its excess stays below 1/d).
struct CkDivisor {
    uint32_t mul;
    int shift;
};
inline CkDivisor ck_divisor(uint32_t d) {
    int l = 1;
    while (((uint64_t)1 << l) < d) ++l;
    const unsigned __int128 p = (unsigned __int128)1 << (31 + l);
    return CkDivisor{(uint32_t)((p + d - 1) / d), l - 1};
}
__device__ __forceinline__ uint32_t ck_div(uint32_t n, const CkDivisor &d) {
    return __umulhi(n, d.mul) >> d.shift;
}

}  // namespace libgemm
