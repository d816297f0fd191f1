// Low-rank adapters of many requests at once: D(t) = C(t) + s_a (x_t A_a^T) B_a^T with
// a = ids[t], in two kernels.
//
//   lora_down_kernel: h_t = x_t A_a^T, fp32, into the workspace (parts of K by different
//     workgroups each their own sums);
//   lora_up_kernel: D = C + s_a h_t B_a^T.
//
// Both take 16 consecutive tokens at a time, the columns of the 16x16x32 MFMA, whose rows
// are rows of A (ranks) or of B (outputs).  Which adapters the tokens use is found by every
// wave from the 16 ids: a round of the loop takes the first token left, its adapter and
// all the tokens that share it.  Packed prompts have one round almost everywhere, and a
// decoding batch one for each request; no sort, no list in memory, and no launch of its
// own.  A column of an MFMA holds one token, so nothing of an adapter reaches another's
// tokens, which take no part in the round's stores.
//
// What bounds both is memory: X is read once and D written once, the weights once for
// each tile that uses them.
#pragma once

#include "stream.hpp"

namespace libgemm {

struct LoraParams {
    const uint8_t *X, *A, *B;
    const int *ids, *ranks;
    const float *scales;
    const uint8_t *C;
    uint8_t *D;
    int64_t ldx, lda, ldb, ldc, ldd;  // elements
    int T, K, N, adapters, rank;
    int in_place;   // C == D: tokens without an adapter are left alone
    int vec_cd;     // 16-byte accesses to rows of C and D
    float *h;       // [splits][T][ldh]
    int ldh, splits, k_per_split;  // k_per_split: a multiple of 128
};

// Tokens of a tile that share an adapter.
struct LoraGroup {
    int adapter;       // -1: tokens without one
    uint32_t members;  // bit t: token t of the tile
};

// The ids of the tile's 16 tokens (lane t % 16), -1 for none, -2 past the last token.
__device__ __forceinline__ int lora_id(const LoraParams &p, int tile, int lane) {
    const int t = tile * 16 + (lane & 15);
    const int id = t < p.T ? p.ids[t] : -2;
    return t < p.T && (id < 0 || id >= p.adapters) ? -1 : id;
}

// The groups of a tile, one for each adapter in the order of their first tokens, then
// the tokens without one: calls f(group) for groups first, first + step, ...
template <class F>
__device__ __forceinline__ void lora_groups(int id, int lane, int first, int step, bool none, F &&f) {
    uint32_t left = (uint32_t)__ballot(lane < 16 && id >= 0);
    int g = 0;
    while (left) {
        const int lead = __builtin_ctz(left);
        const int a = __builtin_amdgcn_readlane(id, lead);
        const uint32_t members = (uint32_t)__ballot(lane < 16 && id == a);
        left &= ~members;
        if (g == first) {
            f(LoraGroup{a, members});
            first += step;
        }
        ++g;
    }
    if (none && g == first) {
        const uint32_t members = (uint32_t)__ballot(lane < 16 && id == -1);
        if (members) f(LoraGroup{-1, members});
    }
}

// An adapter's own rank.
__device__ __forceinline__ int lora_rank(const LoraParams &p, int a) {
    return p.ranks ? min(max(uniform(p.ranks[a]), 0), p.rank) : p.rank;
}

// h of one tile and adapter at a time; a workgroup of four waves, which take
// consecutive parts of its part of K.  RT row tiles of 16 ranks at once.
// Grid: x tiles, y groups of a tile, z parts of K times chunks of 16 RT ranks.
template <int IT, int RT, bool VEC>
__global__ void __launch_bounds__(256) lora_down_kernel(LoraParams p) {
    __shared__ f32x4 part[3][RT][64];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int split = blockIdx.z % p.splits, r0 = blockIdx.z / p.splits * 16 * RT;
    const int id = lora_id(p, blockIdx.x, lane);
    const int t = blockIdx.x * 16 + (lane & 15), chunk = 8 * (lane >> 4);
    const uint8_t *x = p.X + (int64_t)min(t, p.T - 1) * p.ldx * 2;
    const int k_end = min(p.K, (split + 1) * p.k_per_split);
    const int per = p.k_per_split / 4, kb = split * p.k_per_split + wave * per;
    const int ke = min(k_end, kb + per);
    lora_groups(id, lane, blockIdx.y, gridDim.y, false, [&](const LoraGroup &g) {
        const int rank = lora_rank(p, g.adapter);
        // (rows past the adapter's rank read its first; their sums are not kept)
        const uint8_t *a[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            const int r = r0 + 16 * i + (lane & 15);
            a[i] = p.A + ((int64_t)g.adapter * p.rank + (r < rank ? r : 0)) * p.lda * 2;
        }
        f32x4 acc[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i) acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if (r0 < rank) {
            int k = kb;
            if constexpr (VEC) {
                for (; k + 128 <= ke; k += 128) {
                    u32x4 xv[4], av[RT][4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int64_t at = (int64_t)(k + 32 * q + chunk) * 2;
                        xv[q] = *reinterpret_cast<const u32x4 *>(x + at);
#pragma unroll
                        for (int i = 0; i < RT; ++i)
                            av[i][q] = *reinterpret_cast<const u32x4 *>(a[i] + at);
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q)
#pragma unroll
                        for (int i = 0; i < RT; ++i) acc[i] = mfma16_1<IT>(av[i][q], xv[q], acc[i]);
                }
            }
            for (; k < ke; k += 32) {
                const u32x4 xv = stream_chunk<2, VEC>(x, k + chunk, ke);
#pragma unroll
                for (int i = 0; i < RT; ++i)
                    acc[i] = mfma16_1<IT>(stream_chunk<2, VEC>(a[i], k + chunk, ke), xv, acc[i]);
            }
        }
        // the four waves' sums, in order
        if (wave > 0) {
#pragma unroll
            for (int i = 0; i < RT; ++i) part[wave - 1][i][lane] = acc[i];
        }
        __syncthreads();
        if (wave == 0 && (g.members >> (lane & 15) & 1)) {
            float *h = p.h + ((int64_t)split * p.T + t) * p.ldh;
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                f32x4 s = acc[i];
#pragma unroll
                for (int w = 0; w < 3; ++w) s += part[w][i][lane];
                const int r = r0 + 16 * i + 4 * (lane >> 4);
#pragma unroll
                for (int e = 0; e < 4; ++e) s[e] = r + e < rank ? s[e] : 0.0f;
                if (r < p.ldh) *reinterpret_cast<f32x4 *>(h + r) = s;
            }
        }
        __syncthreads();
    });
}

// 2^e for e in [-126, 127].
__device__ __forceinline__ float lora_pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// D of one tile and adapter at a time: a wave takes 64 columns.  Its four row tiles
// interleave the columns by fours, so that a lane ends up with 16 consecutive ones:
// row i of tile j is column 16 (i / 4) + 4 j + i % 4.
//
// h goes into the MFMA as PARTS values of the 16-bit type, laid end to end along the
// product's depth (a rank of 16 in two parts fills its 32 exactly), B's row being read
// once for each part.  fp16 parts are those of h times a power of two that brings the
// token's largest |h| to [2^8, 2^9).
// Grid: x tiles, y groups of a tile, z blocks of 256 columns.
template <int IT, int OUT, bool VEC>
__global__ void __launch_bounds__(256) lora_up_kernel(LoraParams p) {
    constexpr int PARTS = OUT == DT_F32 ? 3 : 2;
    constexpr int DT = IT == IT_F16 ? DT_F16 : DT_BF16;
    constexpr int OSZ = OUT == DT_F32 ? 4 : 2;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int64_t n0 = (int64_t)blockIdx.z * 256 + wave * 64;
    if (n0 >= p.N) return;
    const int id = lora_id(p, blockIdx.x, lane);
    const int t = blockIdx.x * 16 + (lane & 15), lg = lane >> 4;
    const int64_t n = n0 + 16 * lg;  // this lane's 16 columns
    const int left = (int)min(max(p.N - n, (int64_t)0), (int64_t)16);
    const int chunks = p.ldh / 8;    // of 8 ranks
    lora_groups(id, lane, blockIdx.y, gridDim.y, !p.in_place, [&](const LoraGroup &g) {
        f32x4 acc[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        const int rank = g.adapter < 0 ? 0 : lora_rank(p, g.adapter);
        const bool member = g.members >> (lane & 15) & 1;
        float scale = 0.0f, down = 1.0f;
        if (rank > 0) {
            scale = p.scales ? p.scales[g.adapter] : 1.0f;
            const float *h = p.h + (int64_t)(member ? t : blockIdx.x * 16) * p.ldh;
            const int64_t part = (int64_t)p.T * p.ldh;
            auto load_h = [&](int c, float (&v)[8]) {
                f32x4 a = {0.0f, 0.0f, 0.0f, 0.0f}, b = a;
                if (member) {
                    for (int s = 0; s < p.splits; ++s) {
                        a += *reinterpret_cast<const f32x4 *>(h + s * part + 8 * c);
                        b += *reinterpret_cast<const f32x4 *>(h + s * part + 8 * c + 4);
                    }
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = a[e], v[4 + e] = b[e];
            };
            float up = 1.0f;
            if constexpr (IT == IT_F16) {
                float m = 0.0f;
                for (int c = lg; c < chunks; c += 4) {
                    float v[8];
                    load_h(c, v);
#pragma unroll
                    for (int e = 0; e < 8; ++e) m = fmaxf(m, __builtin_fabsf(v[e]));
                }
                m = fmaxf(m, __shfl_xor(m, 16));
                m = fmaxf(m, __shfl_xor(m, 32));
                // (a largest value below 2^-118 is taken as that; Inf and NaN stay so)
                const int e = (int)(__float_as_uint(m) >> 23) - 127;
                const int by = min(max(8 - e, -119), 126);
                up = lora_pow2(by);
                down = lora_pow2(-by);
            }
            const uint8_t *b[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t col = n0 + 16 * ((lane & 15) >> 2) + 4 * j + (lane & 3);
                b[j] = p.B + ((int64_t)g.adapter * p.N + (col < p.N ? col : p.N - 1)) * p.ldb * 2;
            }
            for (int c0 = 0; c0 < PARTS * chunks; c0 += 4) {
                const int c = c0 + lg;
                const int which = c / chunks, rc = c - which * chunks;
                const bool used = which < PARTS;
                float v[8];
                u32x4 hv = {0u, 0u, 0u, 0u};
                if (used) {
                    load_h(rc, v);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        float x = v[e] * up;
                        uint32_t w = to_out16<DT>(x, false);
#pragma unroll
                        for (int q = 1; q < PARTS; ++q) {
                            if (q <= which) {
                                x -= from_out16<DT>(w);
                                w = to_out16<DT>(x, false);
                            }
                        }
                        // (a value that is not finite has no rest)
                        if (which > 0 && x != x) w = 0u;
                        hv[e / 2] |= w << (16 * (e % 2));
                    }
                }
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[j] = mfma16_1<IT>(stream_chunk<2, VEC>(b[j], used ? 8 * rc : rank, rank), hv,
                                          acc[j]);
            }
        }
        if (!member || left == 0) return;
        float y[16];
        const int64_t co = (int64_t)t * p.ldc + n, d_o = (int64_t)t * p.ldd + n;
        if (!p.C) {
#pragma unroll
            for (int e = 0; e < 16; ++e) y[e] = 0.0f;
        } else if (p.vec_cd && left == 16) {
            const u32x4 *c = reinterpret_cast<const u32x4 *>(p.C + co * OSZ);
#pragma unroll
            for (int q = 0; q < 2 * OSZ / 2; ++q) {
                const u32x4 w = c[q];
                if constexpr (OUT == DT_F32) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) y[4 * q + e] = __uint_as_float(w[e]);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[8 * q + e] = from_out16<OUT>(half_of(w, e));
                }
            }
        } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                y[e] = 0.0f;
                if (e < left) {
                    if constexpr (OUT == DT_F32)
                        y[e] = reinterpret_cast<const float *>(p.C)[co + e];
                    else
                        y[e] = from_out16<OUT>(reinterpret_cast<const uint16_t *>(p.C)[co + e]);
                }
            }
        }
        if (rank > 0) {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const float v = acc[e / 4][e % 4];
                y[e] += scale * (IT == IT_F16 ? v * down : v);
            }
        }
        if constexpr (OUT == DT_F32) {
            float *d = reinterpret_cast<float *>(p.D) + d_o;
            if (p.vec_cd && left == 16) {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    reinterpret_cast<f32x4 *>(d)[q] =
                        f32x4{y[4 * q], y[4 * q + 1], y[4 * q + 2], y[4 * q + 3]};
            } else {
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (e < left) d[e] = y[e];
            }
        } else {
            uint16_t *d = reinterpret_cast<uint16_t *>(p.D) + d_o;
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) w[e] = to_out16<OUT>(y[e], false);
            if (p.vec_cd && left == 16) {
#pragma unroll
                for (int q = 0; q < 2; ++q)
                    reinterpret_cast<u32x4 *>(d)[q] =
                        u32x4{w[8 * q] | (w[8 * q + 1] << 16), w[8 * q + 2] | (w[8 * q + 3] << 16),
                              w[8 * q + 4] | (w[8 * q + 5] << 16), w[8 * q + 6] | (w[8 * q + 7] << 16)};
            } else {
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (e < left) d[e] = (uint16_t)w[e];
            }
        }
    });
}

}  // namespace libgemm
