// Products of a few rows with a weight matrix that is read once.
//
// y(r, j) = sum_k x(r, k) w(j, k) for up to 16 * MT rows of x: the arithmetic
// for each byte of w is so little that the rate at which w arrives from memory
// is all that counts.  So w goes from memory straight to the matrix units'
// operand registers: a wave takes 16 rows of w (output channels) as the MFMA's
// first operand and 16 rows of x as its second.  Lane l holds row l % 16 and,
// of each block of 64 bytes of w's rows, the 16-byte chunk l / 16; it loads the
// same k of its x row.  Staging w in LDS would add a write, a read and a wait
// to every byte without saving a load: no two waves share a byte of w.  x is
// small and comes from the caches, once for every 16 * NF channels.
//
// The k of a block pair up lane by lane, so any order of k inside the block is
// right as long as x and w take the same one.  The waves of a workgroup take
// consecutive parts of K and add their sums up in LDS, in a fixed order: the
// same call gives the same bits.
#pragma once

#include "gemm_kernels.hpp"

namespace libgemm {

// x of type XT (IT_F16, IT_BF16 or IT_I8); w of the same type, or int8 (W8)
// under 16-bit x, converted on the way (exact: |w| <= 128 fits fp16 and bf16).
template <int XT, bool W8>
struct StreamTypes {
    static constexpr int XES = XT == IT_I8 ? 1 : 2;
    static constexpr int WES = (W8 || XT == IT_I8) ? 1 : 2;
    static constexpr int EPC = 16 / WES;       // k values of one 16-byte chunk of w
    static constexpr int KB = 4 * EPC;         // k values of a block (64 bytes of a row of w)
    static constexpr int XC = EPC * XES / 16;  // 16-byte chunks of x that go with it
};

// The 16 bytes of `row` that hold elements k, k+1, ... of ES bytes, those at
// and past K zero.  VEC: one load (the row is 16-byte aligned and k a multiple
// of a chunk; a chunk wholly past K reads the row's first instead, so every
// chunk read holds an element of the row).  Otherwise one load per element.
template <int ES, bool VEC>
__device__ __forceinline__ u32x4 stream_chunk(const uint8_t *row, int k, int K) {
    constexpr int EPC = 16 / ES;
    const int n = min(max(K - k, 0), EPC);
    if constexpr (VEC) {
        const u32x4 v = *reinterpret_cast<const u32x4 *>(row + (int64_t)(n > 0 ? k : 0) * ES);
        return ES == 2 ? keep_first(v, n) : keep_first_bytes(v, n);
    } else {
        u32x4 v = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int e = 0; e < EPC; ++e) {
            if (e < n) {
                const uint32_t h = ES == 2 ? (uint32_t)reinterpret_cast<const uint16_t *>(row)[k + e]
                                           : (uint32_t)row[k + e];
                v[e * ES / 4] |= h << (8 * ES * (e % (4 / ES)));
            }
        }
        return v;
    }
}

// Eight int8 values (two dwords) as eight fp16 or bf16 values, exactly.
template <int XT>
__device__ __forceinline__ u32x4 stream_widen(uint32_t lo, uint32_t hi) {
    u32x4 v;
    if constexpr (XT == IT_F16) {
        // the byte plus 128 in the low mantissa bits of 1024.0 is 1152 + the value
        typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
        const f16x2 off = {(_Float16)1152.0f, (_Float16)1152.0f};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t u = (h ? hi : lo) ^ 0x80808080u;
            const uint32_t a = __builtin_amdgcn_perm(0x64646464u, u, 0x04010400u);
            const uint32_t b = __builtin_amdgcn_perm(0x64646464u, u, 0x04030402u);
            v[2 * h] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, a) - off);
            v[2 * h + 1] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, b) - off);
        }
    } else {
        // through fp32, whose upper half is the bf16 value: an integer of at
        // most 8 bits has no bits below it
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t d = h ? hi : lo;
            uint32_t f[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                f[e] = __float_as_uint((float)(int8_t)(uint8_t)(d >> (8 * e)));
            v[2 * h] = __builtin_amdgcn_perm(f[1], f[0], 0x07060302u);
            v[2 * h + 1] = __builtin_amdgcn_perm(f[3], f[2], 0x07060302u);
        }
    }
    return v;
}

// acc[t][f] += the products of blocks [bbeg, bend) of K: w[f] points at the
// lane's row of channel group f, x[t] at its row of row group t, both at the
// lane's chunk of block 0 (k0 = EPC * (lane / 16) elements into the row; wrow
// and xrow are the row starts).  XV, WV: x, w allow 16-byte loads.  U blocks are
// in flight while the U before them are multiplied.
template <int XT, bool W8, int MT, int NF, int U, bool XV, bool WV>
struct Stream {
    using S = StreamTypes<XT, W8>;
    static constexpr int XC = S::XC;
    u32x4 w[2][U][NF], x[2][U][MT][XC];

    template <int SL>
    __device__ __forceinline__ void load_whole(const uint8_t *const (&wr)[NF],
                                               const uint8_t *const (&xr)[MT], int lg, int b) {
        Unroll<0, U>::run([&](auto uu) {
            constexpr int u = decltype(uu)::value;
            const int64_t wo = (int64_t)(b + u) * 64 + lg * 16;
#pragma unroll
            for (int f = 0; f < NF; ++f)
                w[SL][u][f] = *reinterpret_cast<const u32x4 *>(wr[f] + wo);
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int c = 0; c < XC; ++c)
                    x[SL][u][t][c] = *reinterpret_cast<const u32x4 *>(xr[t] + wo * XC + 16 * c);
        });
    }
    template <int SL>
    __device__ __forceinline__ void load_some(const uint8_t *const (&wr)[NF],
                                              const uint8_t *const (&xr)[MT], int lg, int b,
                                              int K) {
        Unroll<0, U>::run([&](auto uu) {
            constexpr int u = decltype(uu)::value;
            const int k = (b + u) * S::KB + lg * S::EPC;
#pragma unroll
            for (int f = 0; f < NF; ++f) w[SL][u][f] = stream_chunk<S::WES, WV>(wr[f], k, K);
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int c = 0; c < XC; ++c)
                    x[SL][u][t][c] = stream_chunk<S::XES, XV>(xr[t], k + c * (16 / S::XES), K);
        });
    }
    template <int SL>
    __device__ __forceinline__ void multiply(f32x4 (&acc)[MT][NF]) {
        Unroll<0, U>::run([&](auto uu) {
            constexpr int u = decltype(uu)::value;
            Unroll<0, NF>::run([&](auto ff) {
                constexpr int f = decltype(ff)::value;
                if constexpr (W8) {
                    const u32x4 v = w[SL][u][f];
                    const u32x4 a = stream_widen<XT>(v[0], v[1]), b = stream_widen<XT>(v[2], v[3]);
                    Unroll<0, MT>::run([&](auto tt) {
                        constexpr int t = decltype(tt)::value;
                        acc[t][f] = mfma16_1<XT>(a, x[SL][u][t][0], acc[t][f]);
                        acc[t][f] = mfma16_1<XT>(b, x[SL][u][t][XC - 1], acc[t][f]);
                    });
                } else {
                    Unroll<0, MT>::run([&](auto tt) {
                        constexpr int t = decltype(tt)::value;
                        acc[t][f] = mfma16_1<XT>(w[SL][u][f], x[SL][u][t][0], acc[t][f]);
                    });
                }
            });
        });
    }
    __device__ __forceinline__ void run(const uint8_t *const (&wr)[NF],
                                        const uint8_t *const (&xr)[MT], int lane, int bbeg,
                                        int bend, int K, f32x4 (&acc)[MT][NF]) {
        const int lg = lane >> 4;
        int b = bbeg;
        if constexpr (XV && WV) {
            // groups of U blocks that lie wholly below K
            const int groups = max(min(bend, K / S::KB) - bbeg, 0) / U;
            if (groups > 0) load_whole<0>(wr, xr, lg, b);
            int g = 0;
            for (; g + 2 <= groups; g += 2) {
                load_whole<1>(wr, xr, lg, b + U);
                __builtin_amdgcn_sched_barrier(0);
                multiply<0>(acc);
                __builtin_amdgcn_sched_barrier(0);
                if (g + 2 < groups) load_whole<0>(wr, xr, lg, b + 2 * U);
                __builtin_amdgcn_sched_barrier(0);
                multiply<1>(acc);
                __builtin_amdgcn_sched_barrier(0);
                b += 2 * U;
            }
            if (g < groups) {
                multiply<0>(acc);
                b += U;
            }
        }
        for (; b < bend; b += U) {
            load_some<0>(wr, xr, lg, b, min(K, bend * S::KB));
            multiply<0>(acc);
        }
    }
};

}  // namespace libgemm
