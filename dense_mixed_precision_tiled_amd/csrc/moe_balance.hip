// gemm_moe_balance and gemm_moe_balance_grad: the balance loss of a router, the
// tokens of each expert, and the loss's gradient with respect to the logits.
//
//   p = softmax(l_t);  c_e = tokens whose topk largest l hold e;  f = c / (n topk);
//   loss = balance E sum_e f_e mean_t(p_te) + z mean_t(lse_t^2)
//   dl_te = g/n p_te (balance E (f_e - sum_j f_j p_tj) + 2 z lse_t)
//
// A group of G lanes takes a token, V experts each (V consecutive ones for a lane: 16-byte
// loads), so that a row is read once and stays in registers: its maximum is the first
// round of the selection, the others take the largest value left.  Sums over tokens stay
// in registers over a thread's tokens; then the groups of a wave, the waves of a workgroup
// and, in the second kernel, the workgroups are added up in a fixed order.
//
// In the gradient f is the same for every token and stays in registers.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/libgemm.h"
#include "gemm_host.hpp"
#include "gemm_kernels.hpp"
#include "gemm_validate.hpp"

namespace libgemm {

struct BalanceParams {
    const float *logits;
    const uint8_t *mask;
    int64_t ldl, ldd;
    int T, E, topk;
    float balance, z;
    float *loss;
    int *counts;
    float *lse;
    uint8_t *D;
    const float *dloss;
    int vec_out;  // rows of D allow a lane's V outputs in one store
    // workspace: by expert and workgroup, then by workgroup
    int parts;
    double *psum;  // [E + 1][parts]: sums of p, then of lse^2
    int *csum;     // [E + 1][parts]: tokens of e, then tokens that count
};

// exp(x) for x <= 0 or so: x log2(e) in two parts, so that a large argument's rounding
// does not show.
__device__ __forceinline__ float balance_exp(float x) {
    const float h = x * 1.44269504f;
    // (an infinite x: no rest)
    const float l = __builtin_fmaf(x, 1.44269504f, -h) + x * 1.92596299e-8f;
    const float y = __builtin_amdgcn_exp2f(h);
    return __builtin_isinf(h) ? y : __builtin_fmaf(y, l * 0.69314718f, y);
}

// Lane l reads lane l ^ X of its row of 16 (X = 1, 2), its mirror in the half row (which
// holds the other quad's result) or in the row (the other half's); past rows, LDS exchanges.
template <int STEP>
__device__ __forceinline__ float group_other(float v) {
    if constexpr (STEP <= 8) {
        constexpr int ctrl = STEP == 1 ? 0xb1 : STEP == 2 ? 0x4e : STEP == 4 ? 0x141 : 0x140;
        return __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp((int)__float_as_uint(v), ctrl, 0xf, 0xf, true));
    } else {
        return __shfl_xor(v, STEP);
    }
}
// Over the lanes of a group, the same in all of them.
template <int G, int STEP = 1>
__device__ __forceinline__ float group_max(float v) {
    if constexpr (STEP < G) return group_max<G, 2 * STEP>(fmaxf(v, group_other<STEP>(v)));
    else return v;
}
template <int G, int STEP = 1>
__device__ __forceinline__ float group_sum(float v) {
    if constexpr (STEP < G) return group_sum<G, 2 * STEP>(v + group_other<STEP>(v));
    else return v;
}

// V logits from expert e0 on; experts past E are -Inf.
template <int V, bool VEC>
__device__ __forceinline__ void balance_load(const float *row, int e0, int E, float (&l)[V]) {
    const float none = -__builtin_inff();
#pragma unroll
    for (int q = 0; q < V; q += 4) {
        if constexpr (VEC) {
            f32x4 v = {none, none, none, none};
            if (e0 + q < E) v = *reinterpret_cast<const f32x4 *>(row + e0 + q);
#pragma unroll
            for (int e = 0; e < 4; ++e) l[q + e] = e0 + q + e < E ? v[e] : none;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) l[q + e] = e0 + q + e < E ? row[e0 + q + e] : none;
        }
    }
}

template <int G, int V, bool VEC>
__global__ void __launch_bounds__(1024) balance_kernel(BalanceParams p) {
    const float none = -__builtin_inff();
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    const int in_group = lane % G, e0 = in_group * V;
    // lanes of the group below this one
    const uint64_t group_bits = G == 64 ? ~0ull : ((1ull << G) - 1ull) << (lane / G * G);
    const uint64_t below = group_bits & ((1ull << lane) - 1ull);
    const int64_t step = (int64_t)gridDim.x * (blockDim.x / G);
    double psum[V], zsum = 0.0;
    int csum[V], live_count = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) psum[i] = 0.0, csum[i] = 0;
    for (int64_t t = (int64_t)blockIdx.x * (blockDim.x / G) + threadIdx.x / G; t < p.T; t += step) {
        const bool masked = p.mask && p.mask[t] == 0;
        float l[V], left[V];
        if (masked) {
#pragma unroll
            for (int i = 0; i < V; ++i) l[i] = none;
        } else {
            balance_load<V, VEC>(p.logits + t * p.ldl, e0, p.E, l);
        }
        // NaN is never chosen
#pragma unroll
        for (int i = 0; i < V; ++i) left[i] = l[i] == l[i] ? l[i] : none;
        float top = none;
        for (int r = 0; r < p.topk; ++r) {
            float m = left[0];
#pragma unroll
            for (int i = 1; i < V; ++i) m = fmaxf(m, left[i]);
            m = group_max<G>(m);
            if (r == 0) top = m;
            // the lowest expert that holds it: the group's first lane, its first value
            bool mine = false;
#pragma unroll
            for (int i = 0; i < V; ++i) mine |= left[i] == m;
            const uint64_t has = __ballot(mine);
            bool take = mine && (has & below) == 0 && m > none;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const bool here = take && left[i] == m;
                csum[i] += here ? 1 : 0;
                left[i] = here ? none : left[i];
                take = take && !here;
            }
        }
        const float shift = top > none ? top : 0.0f;
        float e[V], sum = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            e[i] = balance_exp(l[i] - shift);
            sum += e[i];
        }
        sum = group_sum<G>(sum);
        const bool live = !masked && sum != 0.0f;  // (NaN counts)
        const float lse = masked ? 0.0f : (sum == 0.0f ? none : logf(sum) + shift);
        const float inv = 1.0f / sum;
        if (live) {
#pragma unroll
            for (int i = 0; i < V; ++i) psum[i] += (double)(e[i] * inv);
        }
        if (in_group == 0) {
            p.lse[t] = lse;
            if (live) zsum += (double)lse * (double)lse, ++live_count;
        }
    }
    // the groups of the wave
#pragma unroll
    for (int s = G; s < 64; s *= 2) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            psum[i] += __shfl_xor(psum[i], s);
            csum[i] += __shfl_xor(csum[i], s);
        }
        zsum += __shfl_xor(zsum, s);
        live_count += __shfl_xor(live_count, s);
    }
    // the waves
    extern __shared__ double smem[];  // [waves][E + 1], then the counts alike
    int *const cmem = reinterpret_cast<int *>(smem + waves * (p.E + 1));
    if (lane < G) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (e0 + i < p.E) {
                smem[wave * (p.E + 1) + e0 + i] = psum[i];
                cmem[wave * (p.E + 1) + e0 + i] = csum[i];
            }
        }
        if (lane == 0) {
            smem[wave * (p.E + 1) + p.E] = zsum;
            cmem[wave * (p.E + 1) + p.E] = live_count;
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e <= p.E; e += blockDim.x) {
        double s = 0.0;
        int c = 0;
        for (int w = 0; w < waves; ++w) s += smem[w * (p.E + 1) + e], c += cmem[w * (p.E + 1) + e];
        p.psum[(int64_t)e * p.parts + blockIdx.x] = s;
        p.csum[(int64_t)e * p.parts + blockIdx.x] = c;
    }
}

// One workgroup of 16 waves: a wave adds up the parts of an expert.
__global__ void __launch_bounds__(1024) balance_join_kernel(BalanceParams p) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    __shared__ double terms[16], zsum;
    __shared__ int live;
    double term = 0.0;
    for (int e = wave; e <= p.E; e += 16) {
        double s = 0.0;
        int c = 0;
        for (int i = lane; i < p.parts; i += 64)
            s += p.psum[(int64_t)e * p.parts + i], c += p.csum[(int64_t)e * p.parts + i];
#pragma unroll
        for (int o = 32; o; o >>= 1) s += __shfl_xor(s, o), c += __shfl_xor(c, o);
        if (e < p.E) term += s * (double)c;
        if (lane == 0) {
            p.counts[e] = c;
            if (e == p.E) zsum = s, live = c;
        }
    }
    if (lane == 0) terms[wave] = term;
    __syncthreads();
    if (threadIdx.x == 0) {
        double s = 0.0;
        for (int w = 0; w < 16; ++w) s += terms[w];
        const double n = (double)live;
        const double b = live ? (double)p.E * s / (n * n * (double)p.topk) : 0.0;
        const double z = live ? zsum / n : 0.0;
        p.loss[0] = (float)((double)p.balance * b + (double)p.z * z);
        p.loss[1] = (float)b;
        p.loss[2] = (float)z;
    }
}

template <int G, int V, int OUT, bool VEC>
__global__ void __launch_bounds__(256) balance_grad_kernel(BalanceParams p) {
    const int in_group = (threadIdx.x & 63) % G, e0 = in_group * V;
    const int64_t step = (int64_t)gridDim.x * (256 / G);
    const int n = p.counts[p.E];
    const float per = 1.0f / ((float)n * (float)p.topk);  // (n > 2^24: rounded, as f is)
    const float g = (p.dloss ? *p.dloss : 1.0f) / (float)n;
    const float a = p.balance * (float)p.E, b = 2.0f * p.z;
    float f[V];
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = e0 + i < p.E ? (float)p.counts[e0 + i] * per : 0.0f;
    for (int64_t t = (int64_t)blockIdx.x * (256 / G) + threadIdx.x / G; t < p.T; t += step) {
        const float lse = p.lse[t];
        const bool dead = (p.mask && p.mask[t] == 0) || lse == -__builtin_inff() || n == 0;
        float y[V];
        if (dead) {
#pragma unroll
            for (int i = 0; i < V; ++i) y[i] = 0.0f;
        } else {
            float l[V], dot = 0.0f;
            balance_load<V, VEC>(p.logits + t * p.ldl, e0, p.E, l);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                // (an expert at -Inf, and those past E, have none; NaN - lse is NaN)
                l[i] = balance_exp(l[i] - lse);
                dot = __builtin_fmaf(f[i], l[i], dot);
            }
            dot = group_sum<G>(dot);
#pragma unroll
            for (int i = 0; i < V; ++i) y[i] = g * l[i] * __builtin_fmaf(a, f[i] - dot, b * lse);
        }
#pragma unroll
        for (int q = 0; q < V; q += 4) {
            const int nv = p.E - e0 - q;
            const int64_t at = t * p.ldd + e0 + q;
            if constexpr (OUT == DT_F32) {
                float *d = reinterpret_cast<float *>(p.D) + at;
                if (p.vec_out && nv >= 4) {
                    *reinterpret_cast<f32x4 *>(d) = f32x4{y[q], y[q + 1], y[q + 2], y[q + 3]};
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (e < nv) d[e] = y[q + e];
                }
            } else {
                uint16_t *d = reinterpret_cast<uint16_t *>(p.D) + at;
                uint32_t h[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) h[e] = to_out16<OUT>(y[q + e], false);
                if (p.vec_out && nv >= 4) {
                    *reinterpret_cast<u32x2 *>(d) = u32x2{h[0] | (h[1] << 16), h[2] | (h[3] << 16)};
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (e < nv) d[e] = (uint16_t)h[e];
                }
            }
        }
    }
}

}  // namespace libgemm

using namespace libgemm;
using namespace libgemm_host;

namespace {

// Runs f<G, V>() for the least group that holds E experts at four for a lane, sixteen
// for a lane past 256.
template <class F>
auto balance_group(int64_t E, F &&f) {
    using std::integral_constant;
    auto at = [&](auto g, auto v) { return f(g, v); };
    integral_constant<int, 4> four;
    if (E <= 4) return at(integral_constant<int, 1>{}, four);
    if (E <= 8) return at(integral_constant<int, 2>{}, four);
    if (E <= 16) return at(integral_constant<int, 4>{}, four);
    if (E <= 32) return at(integral_constant<int, 8>{}, four);
    if (E <= 64) return at(integral_constant<int, 16>{}, four);
    if (E <= 128) return at(integral_constant<int, 32>{}, four);
    if (E <= 256) return at(integral_constant<int, 64>{}, four);
    return at(integral_constant<int, 64>{}, integral_constant<int, 16>{});
}

bool balance_vec(const float *logits, int64_t ldl) {
    return (uintptr_t)logits % 16 == 0 && ldl % 4 == 0;
}

}  // namespace

extern "C" {

int gemm_validate_moe_balance(int64_t T, int64_t E, int64_t topk, const float *logits, int64_t ldl,
                              const uint8_t *mask, float balance, float z, const float *loss,
                              const int32_t *counts, const float *lse, const void *workspace,
                              int64_t workspace_bytes) {
    return validate_moe_balance(T, E, topk, logits, ldl, mask, balance, z, loss, counts, lse,
                                workspace, workspace_bytes);
}

int gemm_validate_moe_balance_grad(int64_t T, int64_t E, int64_t topk, const float *logits,
                                   int64_t ldl, const uint8_t *mask, float balance, float z,
                                   const int32_t *counts, const float *lse, const float *dloss,
                                   const void *D, int64_t ldd, int out_dtype) {
    return validate_moe_balance_grad(T, E, topk, logits, ldl, mask, balance, z, counts, lse, dloss,
                                     D, ldd, out_dtype);
}

int64_t gemm_moe_balance_workspace(int64_t T, int64_t E, int64_t topk) {
    const int st = validate_moe_balance_dims(T, E, topk);
    return st == GEMM_OK ? moe_balance_workspace(E) : st;
}

int gemm_moe_balance(int64_t T, int64_t E, int64_t topk, const float *logits, int64_t ldl,
                     const uint8_t *mask, float balance, float z, float *loss, int32_t *counts,
                     float *lse, void *workspace, int64_t workspace_bytes, void *stream) {
    const int st = validate_moe_balance(T, E, topk, logits, ldl, mask, balance, z, loss, counts,
                                        lse, workspace, workspace_bytes);
    if (st != GEMM_OK) return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    BalanceParams p{};
    p.logits = logits;
    p.mask = mask;
    p.ldl = ldl;
    p.T = (int)T;
    p.E = (int)E;
    p.topk = (int)topk;
    p.balance = balance;
    p.z = z;
    p.loss = loss;
    p.counts = counts;
    p.lse = lse;
    char *ws = reinterpret_cast<char *>(((uintptr_t)workspace + 255) & ~(uintptr_t)255);
    void *args[] = {&p};
    hipError_t e = balance_group(E, [&](auto g, auto v) {
        constexpr int G = decltype(g)::value, V = decltype(v)::value;
        // 256 threads until every CU has four waves, then 1024 (a part for each workgroup);
        // past 256 experts 16 waves' sums would not fit in LDS
        const int threads = T * G <= 256 * kBalanceParts || V > 4 ? 256 : 1024;
        const int64_t blocks = cdiv(T * G, threads);
        p.parts = (int)(blocks < kBalanceParts ? (blocks > 0 ? blocks : 1) : kBalanceParts);
        p.psum = reinterpret_cast<double *>(ws);
        p.csum = reinterpret_cast<int *>(p.psum + p.parts * (E + 1));
        const size_t lds = (size_t)(threads / 64) * (E + 1) * 12;
        const void *k = balance_vec(logits, ldl) ? (const void *)balance_kernel<G, V, true>
                                                 : (const void *)balance_kernel<G, V, false>;
        return hipLaunchKernel(k, dim3((unsigned)p.parts), dim3(threads), args, lds, s);
    });
    if (e == hipSuccess)
        e = hipLaunchKernel((const void *)balance_join_kernel, dim3(1), dim3(1024), args, 0, s);
    return e == hipSuccess ? GEMM_OK : GEMM_ERR_HIP;
}

int gemm_moe_balance_grad(int64_t T, int64_t E, int64_t topk, const float *logits, int64_t ldl,
                          const uint8_t *mask, float balance, float z, const int32_t *counts,
                          const float *lse, const float *dloss, void *D, int64_t ldd,
                          int out_dtype, void *stream) {
    const int st = validate_moe_balance_grad(T, E, topk, logits, ldl, mask, balance, z, counts,
                                             lse, dloss, D, ldd, out_dtype);
    if (st != GEMM_OK) return st;
    if (T == 0) return GEMM_OK;
    hipStream_t s = static_cast<hipStream_t>(stream);
    BalanceParams p{};
    p.logits = logits;
    p.mask = mask;
    p.ldl = ldl;
    p.ldd = ldd;
    p.T = (int)T;
    p.E = (int)E;
    p.topk = (int)topk;
    p.balance = balance;
    p.z = z;
    p.counts = const_cast<int32_t *>(counts);
    p.lse = const_cast<float *>(lse);
    p.dloss = dloss;
    p.D = static_cast<uint8_t *>(D);
    const int osz = out_size(out_dtype);
    p.vec_out = (uintptr_t)D % (4 * osz) == 0 && ldd % 4 == 0;
    void *args[] = {&p};
    const bool vec = balance_vec(logits, ldl);
    const hipError_t e = balance_group(E, [&](auto g, auto v) {
        constexpr int G = decltype(g)::value, V = decltype(v)::value;
        const void *k;
        if (out_dtype == GEMM_F32)
            k = vec ? (const void *)balance_grad_kernel<G, V, DT_F32, true>
                    : (const void *)balance_grad_kernel<G, V, DT_F32, false>;
        else if (out_dtype == GEMM_F16)
            k = vec ? (const void *)balance_grad_kernel<G, V, DT_F16, true>
                    : (const void *)balance_grad_kernel<G, V, DT_F16, false>;
        else
            k = vec ? (const void *)balance_grad_kernel<G, V, DT_BF16, true>
                    : (const void *)balance_grad_kernel<G, V, DT_BF16, false>;
        int64_t blocks = cdiv(T, 256 / G);
        if (blocks > 2048) blocks = 2048;
        return hipLaunchKernel(k, dim3((unsigned)blocks), dim3(256), args, 0, s);
    });
    return e == hipSuccess ? GEMM_OK : GEMM_ERR_HIP;
}

}  // extern "C"
