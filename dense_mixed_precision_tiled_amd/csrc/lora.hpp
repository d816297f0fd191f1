// Low-rank adapters of many requests at once: D(t) = C(t) + s_a (x_t A_a^T) B_a^T with
// a = ids[t].
//
//   down: h_t = x_t A_a^T, fp32, into the workspace (parts of K by different workgroups
//     each their own sums);
//   parts (many tokens): h's parts of K added up, and split into values of 16 bits;
//   up: D = C + s_a h_t B_a^T.
//
// Which adapters the tokens of a tile use is found by every wave from their ids: a round
// of the loop takes the first token left, its adapter and all the tokens that share it.
// Packed prompts have one round almost everywhere, and a decoding batch one for each
// request; no sort, no list in memory.  A row (or column) of an MFMA holds one token, so
// nothing of an adapter reaches another's tokens, which take no part in the round's stores.
//
// Up to kLoraFew tokens (a decoding batch) what counts is latency: weights straight from
// memory to the registers, for a few tokens in one kernel (lora_one_kernel), for more in two,
// the first 16 tokens and an adapter for each workgroup, the second a token for each wave.
// More tokens (prompts) are taken 64 at a time by the first product and 32 by the second, and
// what counts is the data: X and A go through LDS (read in the MFMA's own shape, a lane's 16
// bytes are a request of their own, 64 cycles of a CU's address path for each KiB), and a wave of
// the second kernel keeps B's part in registers for its 32 tokens.
//
// Kernels on 4096 x 4096 in bf16, us: one token, rank 16, 5.1; 64 tokens of 64 adapters 6.6
// and 5.2 (16.8 MB of weights, from memory); 4096 tokens, rank 64, 8 adapters 17.2, 4.8 and 29.4
// (2.0 and 2.3 TB/s).
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
    float *h;        // [splits][T][ldh]
    uint16_t *parts; // many tokens: the values of 16 bits whose sum is h, as lora_part() lays them out
    float *down;     // many tokens, fp16: [T], the power of two that the sum is multiplied with
    int ldh, splits, k_per_split;  // k_per_split: a multiple of 128
};

// h is held as two 16-bit values for 16-bit outputs, three for fp32 ones.
template <int OUT>
constexpr int kLoraParts = OUT == DT_F32 ? 3 : 2;

// Ranks 8 c .. 8 c + 7 of value q of token t in LoraParams::parts, in chunks of 8: by 16
// tokens, value and 32 ranks, and there in the order of the MFMA's lanes, so that a wave
// reads a KiB in a row.  (Read by rows of h, a lane's 16 bytes are a request of their own.)
template <int PARTS>
__device__ __forceinline__ int64_t lora_part(const LoraParams &p, int64_t t, int q, int c) {
    const int wide = (p.ldh + 31) / 32;
    return (((t / 16) * PARTS + q) * wide + c / 4) * 64 + c % 4 * 16 + t % 16;
}

// Tokens of a tile that share an adapter.
struct LoraGroup {
    int adapter;       // -1: tokens without one
    uint64_t members;  // bit t: token t of the tile
};

// The id of lane l's token, t0 + l: -1 for none, -2 past the tile's tokens or the last one.
__device__ __forceinline__ int lora_id(const LoraParams &p, int t0, int tokens, int lane) {
    const int t = t0 + lane;
    if (lane >= tokens || t >= p.T) return -2;
    const int id = p.ids[t];
    return id < 0 || id >= p.adapters ? -1 : id;
}

// The groups of a tile, one for each adapter in the order of their first tokens, then
// the tokens without one: calls f(group) for groups first, first + step, ...
template <class F>
__device__ __forceinline__ void lora_groups(int id, int first, int step, bool none, F &&f) {
    uint64_t left = __ballot(id >= 0), rest = none ? __ballot(id == -1) : 0;
    for (int g = 0; left | rest; ++g) {
        const int a = left ? __builtin_amdgcn_readlane(id, __builtin_ctzll(left)) : -1;
        const uint64_t members = __ballot(id == a);
        if (left) left &= ~members;
        else rest = 0;
        if (g != first) continue;
        first += step;
        f(LoraGroup{a, members});
    }
}

// An adapter's own rank.
__device__ __forceinline__ int lora_rank(const LoraParams &p, int a) {
    return p.ranks ? min(max(uniform(p.ranks[a]), 0), p.rank) : p.rank;
}

// Few tokens: h of one tile and adapter at a time; a workgroup of four waves, which take
// consecutive parts of its part of K.  RT row tiles of 16 ranks at once.  Latency: 64 tokens
// of 64 adapters, rank 16, K = 4096 take 5.9 us (8.9 MB, 1.5 TB/s).
// Grid: x tiles, y groups of a tile, z parts of K times chunks of 16 RT ranks.
template <int IT, int RT, bool VEC>
__global__ void __launch_bounds__(256) lora_down_kernel(LoraParams p) {
    __shared__ f32x4 part[3][RT][64];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int split = blockIdx.z % p.splits, r0 = blockIdx.z / p.splits * 16 * RT;
    const int id = lora_id(p, blockIdx.x * 16, 16, lane);
    const int t = blockIdx.x * 16 + (lane & 15), chunk = 8 * (lane >> 4);
    const uint8_t *x = p.X + (int64_t)min(t, p.T - 1) * p.ldx * 2;
    const int k_end = min(p.K, (split + 1) * p.k_per_split);
    const int per = p.k_per_split / 4, kb = split * p.k_per_split + wave * per;
    const int ke = min(k_end, kb + per);
    lora_groups(id, blockIdx.y, gridDim.y, false, [&](const LoraGroup &g) {
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

// Many tokens: h of 64 tokens and 16 RT ranks.  64 values of k at a time through four LDS
// stages, three of them on their way; a wave takes 16 of the tokens.  Bound by the loads in
// flight: 4096 tokens, K = 4096, rank 64 take 17.2 us (X at 2.0 TB/s) in 256 workgroups, one
// on a CU, each waiting for its own stages.
// Grid: x tiles, y chunks of 16 RT ranks, z parts of K.
template <int IT, int RT>
__global__ void __launch_bounds__(256) lora_down_tile_kernel(LoraParams p) {
    constexpr int ROWS = 64 + 16 * RT, STAGES = 4, NL = ROWS * 8 / 256;  // 8 chunks of 16 bytes a row
    static_assert(ROWS * 8 % 256 == 0, "whole loads of 64 chunks for each wave");
    __shared__ u32x4 smem[STAGES * ROWS * 8];
    char *const lds = reinterpret_cast<char *>(smem);
    const uint32_t lds_base = (uint32_t)(uintptr_t)(LIBGEMM_LDS char *)lds;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int t0 = blockIdx.x * 64, r0 = blockIdx.y * 16 * RT;
    const int kb = blockIdx.z * p.k_per_split, ke = min(p.K, kb + p.k_per_split);
    const int steps = ke > kb ? (ke - kb) / 64 : 0;  // whole ones; the rest straight from memory
    const int id = lora_id(p, t0, 64, lane);
    const int mine = t0 + 16 * wave + (lane & 15);  // this lane's token
    const uint8_t *const x = p.X + (int64_t)min(mine, p.T - 1) * p.ldx * 2;
    lora_groups(id, 0, 1, false, [&](const LoraGroup &g) {
        const int rank = lora_rank(p, g.adapter);
        const uint8_t *const a0 = p.A + (int64_t)g.adapter * p.rank * p.lda * 2;
        f32x4 acc[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i) acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if (r0 < rank) {
            // load i of the wave: rows 0 to 63 of a stage are tokens, the others ranks.  Rows
            // past the last token read it, rows past the rank read rank 0: columns that are
            // not kept
            const uint8_t *src[NL];
#pragma unroll
            for (int i = 0; i < NL; ++i) {
                const int q = (wave * NL + i) * 64 + lane, row = q / 8, c = (q % 8) ^ swz_kc(row);
                const int r = r0 + row - 64;
                const uint8_t *line = row < 64 ? p.X + (int64_t)min(t0 + row, p.T - 1) * p.ldx * 2
                                               : a0 + (int64_t)(r < rank ? r : 0) * p.lda * 2;
                src[i] = line + (kb + 8 * c) * 2;
            }
            // Step n of k into stage s.  (Written out: the compiler would let every LDS read
            // behind the builtin wait for it.  Nothing else here uses m0.)
            auto load = [&](int n, int s) {
#pragma unroll
                for (int i = 0; i < NL; ++i) {
                    const uint32_t dst = lds_base + ((s % STAGES) * ROWS * 8 + (wave * NL + i) * 64) * 16;
                    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
                                 :
                                 : "s"(uniform((int)dst)), "v"(src[i] + n * 128)
                                 : "memory");
                }
            };
            // (past the last step the loads go on, so that the waits' counts hold)
            const int last = steps - 1;
            if (steps > 0) {
#pragma unroll
                for (int s = 0; s < STAGES - 1; ++s) load(min(s, last), s);
            }
            const int lg = kc_group16(lane >> 4);
            for (int s = 0; s < steps; ++s) {
                wait_vmcnt<(STAGES - 2) * NL>();  // step s is there
                __syncthreads();                  // everywhere, and stage s - 1 is read
                load(min(s + STAGES - 1, last), s + STAGES - 1);
                const char *const st = lds + (s % STAGES) * ROWS * 128;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    auto frag = [&](int row) {
                        return *reinterpret_cast<const u32x4 *>(st + (row * 8 + ((4 * h + lg) ^ swz_kc(row))) * 16);
                    };
                    const u32x4 xv = frag(16 * wave + (lane & 15));
#pragma unroll
                    for (int i = 0; i < RT; ++i)
                        acc[i] = mfma16_1<IT>(frag(64 + 16 * i + (lane & 15)), xv, acc[i]);
                }
            }
            wait_vmcnt<0>();
            for (int k = kb + 64 * steps + 8 * (lane >> 4); k - 8 * (lane >> 4) < ke; k += 32) {
                const u32x4 xv = stream_chunk<2, true>(x, k, ke);
#pragma unroll
                for (int i = 0; i < RT; ++i) {
                    const int r = r0 + 16 * i + (lane & 15);
                    acc[i] = mfma16_1<IT>(
                        stream_chunk<2, true>(a0 + (int64_t)(r < rank ? r : 0) * p.lda * 2, k, ke), xv, acc[i]);
                }
            }
            __syncthreads();  // the stages are read
        }
        if (g.members >> (16 * wave + (lane & 15)) & 1) {
            float *h = p.h + ((int64_t)blockIdx.z * p.T + mine) * p.ldh;
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                const int r = r0 + 16 * i + 4 * (lane >> 4);
                f32x4 v = acc[i];
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = r + e < rank ? v[e] : 0.0f;
                if (r < p.ldh) *reinterpret_cast<f32x4 *>(h + r) = v;
            }
        }
    });
}

// 2^e for e in [-126, 127].
__device__ __forceinline__ float lora_pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// fp16: the exponent that brings a token's largest |h| to [2^13, 2^14).  fp16's least step,
// 2^-24, is then 2^-37 of it at most, half of which is lost, and the second product's sums (rank
// 256, B below 2^16) stay below 2^38.  (A largest value below 2^-113 is taken as that; Inf and NaN
// stay so.)
__device__ __forceinline__ int lora_exponent(float m) {
    const int e = (int)(__float_as_uint(m) >> 23) - 127;
    return min(13 - e, 126);
}

// Eight values (times a power of two) as PARTS 16-bit values each whose sum they are.  A
// value that is not finite has no rest.  A finite one past bf16's largest keeps that as its
// first part (rounded, it would be Inf, and its rest -Inf).
template <int IT, int PARTS>
__device__ __forceinline__ void lora_split(const float (&v)[8], float up, u32x4 (&w)[PARTS]) {
    constexpr int DT = IT == IT_F16 ? DT_F16 : DT_BF16;
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        float a = IT == IT_F16 ? v[e] * up : v[e], b = IT == IT_F16 ? v[e + 1] * up : v[e + 1];
#pragma unroll
        for (int q = 0; q < PARTS; ++q) {
            const bool bf = IT == IT_BF16 && q == 0;
            uint32_t x = to_out16<DT>(a, bf && __builtin_isfinite(a));
            uint32_t y = to_out16<DT>(b, bf && __builtin_isfinite(b));
            if (q > 0) {
                x = a != a ? 0u : x;
                y = b != b ? 0u : y;
            }
            w[q][e / 2] = x | (y << 16);
            a -= from_out16<DT>(x);
            b -= from_out16<DT>(y);
        }
    }
}

// The sum of h's parts of K (four at most), ranks 8c .. 8c + 7 of token t; all loads
// before the first addition.
__device__ __forceinline__ void lora_load_h(const LoraParams &p, int64_t t, int c, float (&v)[8]) {
    const int64_t part = (int64_t)p.T * p.ldh;
    const float *h = p.h + t * p.ldh + 8 * c;
    f32x4 w[4][2];
#pragma unroll
    for (int s = 0; s < 4; ++s)
        if (s < p.splits) {
            w[s][0] = *reinterpret_cast<const f32x4 *>(h + s * part);
            w[s][1] = *reinterpret_cast<const f32x4 *>(h + s * part + 4);
        }
    f32x4 a = w[0][0], b = w[0][1];
#pragma unroll
    for (int s = 1; s < 4; ++s)
        if (s < p.splits) a += w[s][0], b += w[s][1];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = a[e], v[4 + e] = b[e];
}

// Many tokens: a thread takes 8 ranks of a token (0 past the last, up to a multiple of 32), 32
// (or fewer) threads a token.  Once here instead of in each of the second product's column
// blocks: 4096 tokens of rank 64 in four parts of K (4 MB) take 4.8 us.
template <int IT, int PARTS>
__global__ void __launch_bounds__(256) lora_parts_kernel(LoraParams p, int lanes) {
    const int64_t t = (int64_t)blockIdx.x * (256 / lanes) + threadIdx.x / lanes;
    const int c = threadIdx.x % lanes;
    const bool in = t < p.T && 8 * c < p.ldh;
    float v[8] = {}, m = 0.0f, up = 1.0f;
    // (a token without an adapter has no h: what is there is split, and not used)
    if (in) lora_load_h(p, t, c, v);
    if constexpr (IT == IT_F16) {
#pragma unroll
        for (int e = 0; e < 8; ++e) m = fmaxf(m, __builtin_fabsf(v[e]));
        for (int s = 1; s < lanes; s *= 2) m = fmaxf(m, __shfl_xor(m, s));
        const int by = lora_exponent(m);
        up = lora_pow2(by);
        if (in && c == 0) p.down[t] = lora_pow2(-by);
    }
    if (t >= p.T || c >= (p.ldh + 31) / 32 * 4) return;
    u32x4 w[PARTS];
    lora_split<IT, PARTS>(v, up, w);
#pragma unroll
    for (int q = 0; q < PARTS; ++q)
        reinterpret_cast<u32x4 *>(p.parts)[lora_part<PARTS>(p, t, q, c)] = w[q];
}

// Four values of a row of C or D: from one load, or as many as n.
template <int OUT>
using LoraQuad = typename std::conditional<OUT == DT_F32, u32x4, u32x2>::type;
template <int OUT>
__device__ __forceinline__ f32x4 lora_values(const LoraQuad<OUT> &w) {
    if constexpr (OUT == DT_F32)
        return f32x4{__uint_as_float(w[0]), __uint_as_float(w[1]), __uint_as_float(w[2]), __uint_as_float(w[3])};
    else
        return f32x4{from_out16<OUT>(w[0] & 0xffffu), from_out16<OUT>(w[0] >> 16),
                     from_out16<OUT>(w[1] & 0xffffu), from_out16<OUT>(w[1] >> 16)};
}
template <int OUT>
__device__ __forceinline__ f32x4 lora_load_some(__amdgpu_buffer_rsrc_t rows, uint32_t voff, uint32_t soff, int n) {
    f32x4 y = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (e < n) {
            if constexpr (OUT == DT_F32)
                y[e] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rows, voff + 4 * e, soff, 0));
            else
                y[e] = from_out16<OUT>(__builtin_amdgcn_raw_buffer_load_b16(rows, voff + 2 * e, soff, 0));
        }
    return y;
}
template <int OUT>
__device__ __forceinline__ void lora_store_some(__amdgpu_buffer_rsrc_t rows, uint32_t voff, uint32_t soff, int n,
                                                const f32x4 &y) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (e < n) {
            if constexpr (OUT == DT_F32)
                __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(y[e]), rows, voff + 4 * e, soff, 0);
            else
                __builtin_amdgcn_raw_buffer_store_b16((unsigned short)to_out16<OUT>(y[e], false), rows, voff + 2 * e,
                                                      soff, 0);
        }
}

// Few tokens: D of one token, 64 columns for a wave.  A column is a lane's dot product of
// rank terms, in fp32 with h as it is: with a token an adapter, a column of the MFMA would
// be all that it uses of one (64 tokens of 64 adapters, 4096 columns: 10.0 us so, and 4.5
// with a token for each wave).
// Grid: x blocks of 256 columns, y tokens.
template <int IT, int OUT, bool VEC>
__global__ void __launch_bounds__(256) lora_up_few_kernel(LoraParams p) {
    const int lane = threadIdx.x & 63, t = blockIdx.y;
    const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x, row = min(n, (int64_t)p.N - 1);
    const int id = uniform(p.ids[t]);
    const bool has = id >= 0 && id < p.adapters;
    if (!has && p.in_place) return;
    auto c_at = [&](int64_t at) {
        if constexpr (OUT == DT_F32) return reinterpret_cast<const float *>(p.C)[at];
        else return from_out16<OUT>(reinterpret_cast<const uint16_t *>(p.C)[at]);
    };
    const float c = p.C ? c_at((int64_t)t * p.ldc + row) : 0.0f;
    float y = c;
    const int rank = has ? lora_rank(p, id) : 0;
    if (rank > 0) {
        const float scale = p.scales ? p.scales[id] : 1.0f;
        const uint8_t *b = p.B + ((int64_t)id * p.N + row) * p.ldb * 2;
        const float *h = p.h + (int64_t)t * p.ldh;
        const int64_t part = (int64_t)p.T * p.ldh;
        float dot = 0.0f;
        for (int r0 = 0; r0 < rank; r0 += 64) {
            // lane l holds rank r0 + l, 0 past the adapter's (where B is masked too)
            float mine = 0.0f;
            if (r0 + lane < p.ldh) {
                float w[4];
#pragma unroll
                for (int s = 0; s < 4; ++s) w[s] = s < p.splits ? h[s * part + r0 + lane] : 0.0f;
                mine = w[0];
#pragma unroll
                for (int s = 1; s < 4; ++s)
                    if (s < p.splits) mine += w[s];
            }
            const int chunks = min(8, (rank - r0 + 7) / 8);
            for (int k = 0; k < chunks; k += 2) {
                // (past the last chunk: the row's first, masked)
                u32x4 v[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) v[e] = stream_chunk<2, VEC>(b, r0 + 8 * (k + e), rank);
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float x = from_out16<IT == IT_F16 ? DT_F16 : DT_BF16>(half_of(v[e / 8], e % 8));
                    const float g = __uint_as_float((uint32_t)__builtin_amdgcn_readlane(
                        (int)__float_as_uint(mine), min(8 * k + e, 63)));
                    // (a masked term is 0 * 0, also where h is not finite)
                    dot = __builtin_fmaf(x, r0 + 8 * k + e < rank ? g : 0.0f, dot);
                }
            }
        }
        y = __builtin_fmaf(scale, dot, c);
    }
    if (n >= p.N) return;
    const int64_t at = (int64_t)t * p.ldd + n;
    if constexpr (OUT == DT_F32) reinterpret_cast<float *>(p.D)[at] = y;
    else reinterpret_cast<uint16_t *>(p.D)[at] = (uint16_t)to_out16<OUT>(y, false);
}

// A few tokens and small adapters: both products in one launch.  Each workgroup makes the
// token's h for itself (A comes from the caches after the first), a wave the dot products of
// ranks wave, wave + 16, ..., whose rows it reads a KiB at a time, and then 256 columns of D,
// whose part of B it has asked for before.
// Grid: x blocks of 256 columns, y tokens.
template <int IT, int OUT, int RT>
__global__ void __launch_bounds__(1024) lora_one_kernel(LoraParams p) {
    constexpr int RANKS = 16 * RT, DT = IT == IT_F16 ? DT_F16 : DT_BF16;
    __shared__ float h[RANKS];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), t = blockIdx.y;
    const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x, row = min(n, (int64_t)p.N - 1);
    const int id = uniform(p.ids[t]);
    const bool has = id >= 0 && id < p.adapters;
    if (!has && p.in_place) return;
    const int rank = has ? lora_rank(p, id) : 0;
    float c = 0.0f, scale = 1.0f;
    u32x4 bv[2 * RT];
    if (wave < 4) {
        if (rank > 0) {
            const uint8_t *b = p.B + ((int64_t)id * p.N + row) * p.ldb * 2;
#pragma unroll
            for (int q = 0; q < 2 * RT; ++q) bv[q] = stream_chunk<2, true>(b, 8 * q, rank);
            if (p.scales) scale = p.scales[id];
        }
        if (p.C) {
            const int64_t at = (int64_t)t * p.ldc + row;
            if constexpr (OUT == DT_F32) c = reinterpret_cast<const float *>(p.C)[at];
            else c = from_out16<OUT>(reinterpret_cast<const uint16_t *>(p.C)[at]);
        }
    }
    float y = c;
    if (rank > 0) {
        const uint8_t *x = p.X + (int64_t)t * p.ldx * 2, *a[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            const int r = 16 * i + wave;  // (past the rank: its first, not kept)
            a[i] = p.A + ((int64_t)id * p.rank + (r < rank ? r : 0)) * p.lda * 2;
        }
        float dot[RT][4] = {};
        auto add = [&](float &to, const u32x4 &u, const u32x4 &v) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                to = __builtin_fmaf(from_out16<DT>(half_of(u, e)), from_out16<DT>(half_of(v, e)), to);
        };
        int k = 0;
        for (; k + 2048 <= p.K; k += 2048) {
            u32x4 xv[4], av[RT][4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int64_t at = (int64_t)(k + 512 * q + 8 * lane) * 2;
                xv[q] = *reinterpret_cast<const u32x4 *>(x + at);
#pragma unroll
                for (int i = 0; i < RT; ++i) av[i][q] = *reinterpret_cast<const u32x4 *>(a[i] + at);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int i = 0; i < RT; ++i) add(dot[i][q], av[i][q], xv[q]);
        }
        for (; k < p.K; k += 512) {
            const u32x4 xv = stream_chunk<2, true>(x, k + 8 * lane, p.K);
#pragma unroll
            for (int i = 0; i < RT; ++i) add(dot[i][0], stream_chunk<2, true>(a[i], k + 8 * lane, p.K), xv);
        }
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            float sum = (dot[i][0] + dot[i][1]) + (dot[i][2] + dot[i][3]);
#pragma unroll
            for (int s = 1; s < 64; s *= 2) sum += __shfl_xor(sum, s);
            // (a masked term of the second product is 0 * 0, also where h is not finite)
            if (lane == 0) h[16 * i + wave] = 16 * i + wave < rank ? sum : 0.0f;
        }
        __syncthreads();
        if (wave < 4) {
            float d = 0.0f;
#pragma unroll
            for (int e = 0; e < RANKS; ++e) d = __builtin_fmaf(from_out16<DT>(half_of(bv[e / 8], e % 8)), h[e], d);
            y = __builtin_fmaf(scale, d, c);
        }
    }
    if (wave >= 4 || n >= p.N) return;
    const int64_t at = (int64_t)t * p.ldd + n;
    if constexpr (OUT == DT_F32) reinterpret_cast<float *>(p.D)[at] = y;
    else reinterpret_cast<uint16_t *>(p.D)[at] = (uint16_t)to_out16<OUT>(y, false);
}

// One value of D from h as it is, in fp32.  The second product of many tokens meets an Inf of B
// with h's parts one by one, 0 among them, and has NaN where h and the Inf make an Inf: sums that
// are NaN are left out of its stores and made here.  (That they are looked for takes 0.3 us of 512
// tokens' 15.2, 0.8 of 4096 tokens' 42.3 at rank 64.)
template <int IT, int OUT>
__device__ __forceinline__ void lora_again(const LoraParams &p, int64_t t, int64_t n) {
    const int id = p.ids[t], rank = p.ranks ? min(p.ranks[id], p.rank) : p.rank;
    const int64_t part = (int64_t)p.T * p.ldh;
    const float *h = p.h + t * p.ldh;
    const uint16_t *b = reinterpret_cast<const uint16_t *>(p.B) + ((int64_t)id * p.N + n) * p.ldb;
    float dot = 0.0f;
#pragma unroll 1
    for (int r = 0; r < rank && dot == dot; ++r) {
        float v = h[r];
        for (int s = 1; s < p.splits; ++s) v += h[s * part + r];
        dot = __builtin_fmaf(from_out16<IT == IT_F16 ? DT_F16 : DT_BF16>(b[r]), v, dot);
    }
    float y = 0.0f;
    if constexpr (OUT == DT_F32) {
        if (p.C) y = reinterpret_cast<const float *>(p.C)[t * p.ldc + n];
    } else {
        if (p.C) y = from_out16<OUT>(reinterpret_cast<const uint16_t *>(p.C)[t * p.ldc + n]);
    }
    y = __builtin_fmaf(p.scales ? p.scales[id] : 1.0f, dot, y);
    if constexpr (OUT == DT_F32) reinterpret_cast<float *>(p.D)[t * p.ldd + n] = y;
    else reinterpret_cast<uint16_t *>(p.D)[t * p.ldd + n] = (uint16_t)to_out16<OUT>(y, false);
}

// Tokens of a tile of the second product: with 64, the registers leave two waves a SIMD
// instead of four (three past rank 32), whose loads, products and stores then follow one
// another.  us, 64 and 32 tokens, N = 4096 in bf16 (both without the search for NaN sums, which
// adds 0.3 to 0.8): 512 tokens 9 and 6, 2048 of rank 32 11.6 and 10.2, 8192 of rank 16 37 and 33
// (4.1 TB/s), 4096 of rank 64 28 and 28.
constexpr int kLoraUpTokens = 32;

// Many tokens: D of a tile and an adapter at a time; a wave takes 64 columns.  Its four
// column tiles interleave the columns by ones, column i of tile j being 4 i + j, so that a
// lane ends up with four consecutive columns of four tokens, and 16 lanes with 128 bytes (of
// a 16-bit type) of a row.
//
// h goes into the MFMA as its 16-bit values, one MFMA after the other on the same part of
// B.  B's 32 RS ranks stay in registers for the tile's tokens (larger ranks read B for
// every 16 tokens).  C, which no id decides, is asked for first.  A row of the MFMA holds one
// token: those of other groups are computed on what is there, and not kept.
// What bounds it at rank 64 is B, read by rows of 16 bytes for each tile (half of the address
// path's time, and as many bytes from L2 as C and D have).
// Grid: x blocks of 256 columns (so that an XCD's L2 holds few blocks of B: 27.4 us, tiles
// first 29.3), z tiles.
template <int IT, int OUT, int RS, bool VEC>
__global__ void __launch_bounds__(256, OUT == DT_F32 ? 2 : RS == 2 || !VEC ? 3 : 4) lora_up_kernel(LoraParams p) {
    static_assert(kLoraUpTokens <= 32, "a lane's values of a tile are the bits of `again`");
    constexpr int SUBS = kLoraUpTokens / 16, PARTS = kLoraParts<OUT>, OSZ = OUT == DT_F32 ? 4 : 2;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int64_t n0 = (int64_t)blockIdx.x * 256 + wave * 64;
    if (n0 >= p.N) return;
    const int t0 = blockIdx.z * 16 * SUBS, lg = lane >> 4;
    const int id = lora_id(p, t0, 16 * SUBS, lane);
    const int64_t n = n0 + 4 * (lane & 15);  // this lane's four columns
    const int left = (int)min(max(p.N - n, (int64_t)0), (int64_t)4);
    const bool whole = p.vec_cd && left == 4;
    const int wide = (p.ldh + 31) / 32;      // of 32 ranks
    // Offsets in the tile's rows of C and D: 31 lines of 2^24 fp32 and a row of 2^19 stay
    // below 2^32.  (64-bit addresses for each of them take the registers of B.)
    auto rows = [&](const uint8_t *base, int64_t ld) {
        return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(base) + (int64_t)t0 * ld * OSZ, (short)0,
                                                 -1, 0x00020000);
    };
    const __amdgpu_buffer_rsrc_t c_rows = rows(p.C, p.ldc), d_rows = rows(p.D, p.ldd);
    const uint32_t c_at = (4u * lg * (uint32_t)p.ldc + (uint32_t)n) * OSZ;
    const uint32_t d_at = (4u * lg * (uint32_t)p.ldd + (uint32_t)n) * OSZ;
    const int tokens = p.T - t0 - 4 * lg;    // from this lane's first on
    const __amdgpu_buffer_rsrc_t downs = __builtin_amdgcn_make_buffer_rsrc(p.down + t0, (short)0, -1, 0x00020000);
    LoraQuad<OUT> cv[SUBS][4];
#pragma unroll
    for (int s = 0; s < SUBS; ++s)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (p.C && whole && 16 * s + e < tokens) {
                const uint32_t at = (16u * s + e) * (uint32_t)p.ldc * OSZ;
                if constexpr (OUT == DT_F32) cv[s][e] = __builtin_amdgcn_raw_buffer_load_b128(c_rows, c_at, at, 0);
                else cv[s][e] = __builtin_amdgcn_raw_buffer_load_b64(c_rows, c_at, at, 0);
            }
        }
    uint32_t again = 0;  // bit 16 s + 4 e + j: not stored, the sum being NaN
    lora_groups(id, 0, 1, !p.in_place, [&](const LoraGroup &g) {
        const int rank = g.adapter < 0 ? 0 : lora_rank(p, g.adapter);
        const float scale = rank > 0 && p.scales ? p.scales[g.adapter] : 1.0f;
        const uint8_t *b[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            b[j] = p.B + ((int64_t)max(g.adapter, 0) * p.N + min(n + j, (int64_t)p.N - 1)) * p.ldb * 2;
        const uint64_t mine = g.members >> (4 * lg);  // bit 16 s + e: this lane's token
        u32x4 bv[RS][4];
        auto load_b = [&](int r0) {
#pragma unroll
            for (int q = 0; q < RS; ++q)
#pragma unroll
                for (int j = 0; j < 4; ++j) bv[q][j] = stream_chunk<2, VEC>(b[j], r0 + 32 * q + 8 * lg, rank);
        };
        if (rank > 0) load_b(0);
#pragma unroll
        for (int s = 0; s < SUBS; ++s) {
            if (!(g.members >> (16 * s) & 0xffff)) continue;
            f32x4 acc[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            for (int r0 = 0; r0 < rank; r0 += 32 * RS) {
                if (rank > 32 * RS) load_b(r0);
                u32x4 hv[RS][PARTS];
#pragma unroll
                for (int q = 0; q < RS; ++q)
#pragma unroll
                    for (int k = 0; k < PARTS; ++k) {
                        hv[q][k] = u32x4{0u, 0u, 0u, 0u};
                        if (r0 / 32 + q < wide)
                            hv[q][k] = reinterpret_cast<const u32x4 *>(
                                p.parts)[lora_part<PARTS>(p, t0 + 16 * s, k, r0 / 8 + 4 * q) + lane];
                    }
#pragma unroll
                for (int q = 0; q < RS; ++q)
#pragma unroll
                    for (int k = 0; k < PARTS; ++k)
#pragma unroll
                        for (int j = 0; j < 4; ++j) acc[j] = mfma16_1<IT>(hv[q][k], bv[q][j], acc[j]);
            }
            // (the group's sums that are not finite, or whose own sum is not)
            const f32x4 all = (acc[0] + acc[1]) + (acc[2] + acc[3]);
            float sum = 0.0f;
#pragma unroll
            for (int e = 0; e < 4; ++e) sum += mine >> (16 * s + e) & 1 ? all[e] : 0.0f;
            const bool bad = __ballot(!__builtin_isfinite(sum)) != 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (!(mine >> (16 * s + e) & 1) || left == 0) continue;
                const uint32_t c_row = (16u * s + e) * (uint32_t)p.ldc * OSZ;
                const uint32_t d_row = (16u * s + e) * (uint32_t)p.ldd * OSZ;
                f32x4 y = {0.0f, 0.0f, 0.0f, 0.0f};
                if (p.C) y = whole ? lora_values<OUT>(cv[s][e]) : lora_load_some<OUT>(c_rows, c_at, c_row, left);
                if (rank > 0) {
                    const float down =
                        IT == IT_F16 ? __uint_as_float(buf_load4(downs, 16u * lg, (16u * s + e) * 4u)) : 1.0f;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float v = acc[j][e];
                        y[j] += scale * (IT == IT_F16 ? v * down : v);
                    }
                }
                if (bad) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (j >= left) continue;
                        if (acc[j][e] != acc[j][e]) again |= 1u << (16 * s + 4 * e + j);
                        else lora_store_some<OUT>(d_rows, d_at + j * OSZ, d_row, 1, f32x4{y[j], 0.0f, 0.0f, 0.0f});
                    }
                } else if (!whole)
                    lora_store_some<OUT>(d_rows, d_at, d_row, left, y);
                else if constexpr (OUT == DT_F32)
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, y), d_rows, d_at, d_row, 0);
                else
                    __builtin_amdgcn_raw_buffer_store_b64(
                        u32x2{pack_out16<OUT>(y[0], y[1]), pack_out16<OUT>(y[2], y[3])}, d_rows, d_at, d_row, 0);
            }
        }
    });
    for (; again; again &= again - 1) {
        const int bit = __builtin_ctz(again);
        lora_again<IT, OUT>(p, t0 + 16 * (bit / 16) + 4 * lg + bit / 4 % 4, n + bit % 4);
    }
}

}  // namespace libgemm
