// gemm_moe_balance and gemm_moe_balance_grad: the balance loss of a router, the
// tokens of each expert, and the loss's gradient with respect to the logits.
//
//   p = softmax(l_t);  c_e = tokens whose topk largest l hold e;  f = c / (n topk);
//   loss = balance E sum_e f_e mean_t(p_te) + z mean_t(lse_t^2)
//   dl_te = g/n p_te (balance E (f_e - sum_j f_j p_tj) + 2 z lse_t)
//
// A group of G lanes takes a token, V experts each (consecutive ones for a lane: 16-byte
// loads), so that a row is read once and stays in registers.  Sums over tokens stay in
// registers over a thread's tokens; then the groups of a wave, the waves of a workgroup
// and, in the second kernel, the workgroups are added up in a fixed order.
//
// In the gradient f is the same for every token and stays in registers; p is made from lse and
// brought to the sum 1.
//
// The first kernel is bound by its vector instructions (about 230 for four tokens of 64
// experts, top 8, most of them the choice), the gradient by latency: counts, lse and logits are
// read one after the other.  65536 tokens of 64 experts, top 8, us: 12.0 to 13.4 (1.4 TB/s), 4.6
// for the sums over the workgroups, and 8.9 to 9.7 for a gradient in bf16 (2.8 TB/s, half of a
// copy's rate); 1024 tokens of 8 experts 4.9, 2.8 and 3.2.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/libgemm.h"
#include "gemm_host.hpp"
#include "gemm_validate.hpp"
#include "moe.hpp"

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
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
    if constexpr (STEP < G) {
        const uint32_t o = __float_as_uint(group_other<STEP>(__uint_as_float(v)));
        return group_max<G, 2 * STEP>(max(v, o));
    } else {
        return v;
    }
}
template <int G, int STEP = 1>
__device__ __forceinline__ float group_sum(float v) {
    if constexpr (STEP < G) return group_sum<G, 2 * STEP>(v + group_other<STEP>(v));
    else return v;
}

// The topk largest of a group's keys (moe_key; ties to the lower expert, none at -Inf or
// NaN): adds 1 to csum of each of a lane's V experts among them.  Returns the largest key.
//
// A lane's keys are sorted, four at a time, so that a round looks at one key of each lane
// (of each four): the group's largest, whose lane's others move up.  Rounds know no ties; where
// two equal keys go in one round, or there are fewer than topk above -Inf, the keys that are
// not below the last round's do not number topk, which is counted, and the choice is made
// again with a round for each single key.
template <int G, int V>
__device__ __forceinline__ uint32_t balance_choose(const uint32_t (&key)[V], int topk, uint64_t below,
                                                   int (&csum)[V]) {
    constexpr int Q = V / 4;
    uint32_t x[Q][4];  // descending
    auto order = [](uint32_t &a, uint32_t &b) {
        const uint32_t hi = max(a, b);
        b = min(a, b);
        a = hi;
    };
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        uint32_t(&y)[4] = x[q];
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = key[4 * q + i];
        order(y[0], y[1]);
        order(y[2], y[3]);
        order(y[0], y[2]);
        order(y[1], y[3]);
        order(y[1], y[2]);
    }
    uint32_t top = 0, m = 0;
    for (int r = 0; r < topk; ++r) {
        m = x[0][0];
#pragma unroll
        for (int q = 1; q < Q; ++q) m = max(m, x[q][0]);
        m = group_max<G>(m);
        if (r == 0) top = m;
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            uint32_t(&y)[4] = x[q];
            const bool take = y[0] == m;
            y[0] = take ? y[1] : y[0];
            y[1] = take ? y[2] : y[1];
            y[2] = take ? y[3] : y[2];
            y[3] = take ? 0u : y[3];
        }
    }
    const bool full = m > kMoeNone;  // topk keys above -Inf; or else none at all
    int chosen = 0;                  // of the wave
#pragma unroll
    for (int i = 0; i < V; ++i) chosen += (int)__popcll(__ballot(full && key[i] >= m));
    const bool plain = chosen * G == topk * (int)__popcll(__ballot(full)) && __ballot(!full && top > kMoeNone) == 0;
    if (plain) {
#pragma unroll
        for (int i = 0; i < V; ++i) csum[i] += full && key[i] >= m ? 1 : 0;
        return top;
    }
    uint32_t left[V];
#pragma unroll
    for (int i = 0; i < V; ++i) left[i] = key[i];
#pragma unroll 1
    for (int r = 0; r < topk; ++r) {
        uint32_t k = left[0];
#pragma unroll
        for (int i = 1; i < V; ++i) k = max(k, left[i]);
        k = group_max<G>(k);
        bool mine = false;
#pragma unroll
        for (int i = 0; i < V; ++i) mine |= left[i] == k;
        // the group's first lane that holds it, whose experts are lower, and its first value
        const uint64_t has = __ballot(mine);
        bool take = mine && (has & below) == 0 && k > kMoeNone;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const bool here = take && left[i] == k;
            csum[i] += here ? 1 : 0;
            left[i] = here ? 0u : left[i];
            take = take && !here;
        }
    }
    return top;
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
__global__ void __launch_bounds__(V > 4 ? 256 : 1024) balance_kernel(BalanceParams p) {
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
    int64_t t = (int64_t)blockIdx.x * (blockDim.x / G) + threadIdx.x / G;
    while (t < p.T) {
        // 32 tokens in fp32, then on to fp64 (whose conversions take four times as long)
        float part[V];
#pragma unroll
        for (int i = 0; i < V; ++i) part[i] = 0.0f;
        for (int k = 0; k < 32 && t < p.T; ++k, t += step) {
            const bool masked = p.mask && p.mask[t] == 0;
            float l[V];
            uint32_t key[V];
            if (masked) {
#pragma unroll
                for (int i = 0; i < V; ++i) l[i] = none;
            } else {
                balance_load<V, VEC>(p.logits + t * p.ldl, e0, p.E, l);
            }
#pragma unroll
            for (int i = 0; i < V; ++i) key[i] = moe_key(l[i]);
            const uint32_t m = balance_choose<G, V>(key, p.topk, below, csum);
            // (the largest logit's value, 0 where there is none above -Inf)
            const float top = m > kMoeNone ? __uint_as_float(m >> 31 ? m & 0x7fffffffu : ~m) : 0.0f;
            float e[V], sum = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                e[i] = __expf(l[i] - top);
                sum += e[i];
            }
            sum = group_sum<G>(sum);
            const bool live = !masked && sum != 0.0f;  // (NaN counts)
            const float lse = masked ? 0.0f : (sum == 0.0f ? none : __logf(sum) + top);
            const float inv = __builtin_amdgcn_rcpf(sum);
            if (live) {
#pragma unroll
                for (int i = 0; i < V; ++i) part[i] = __builtin_fmaf(e[i], inv, part[i]);
                // (in fp64 at once: a square may lie past fp32's range)
                zsum = __builtin_fma((double)lse, (double)lse, zsum);
                ++live_count;
            }
            if (in_group == 0) p.lse[t] = lse;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) psum[i] += (double)part[i];
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

// Sum over the 16 lanes of a row, in all of them.
__device__ __forceinline__ double row_sum(double v) {
    auto other = [](double x, auto ctrl) {
        const uint64_t b = __builtin_bit_cast(uint64_t, x);
        const int lo = __builtin_amdgcn_mov_dpp((int)(uint32_t)b, decltype(ctrl)::value, 0xf, 0xf, true);
        const int hi = __builtin_amdgcn_mov_dpp((int)(b >> 32), decltype(ctrl)::value, 0xf, 0xf, true);
        return __builtin_bit_cast(double, (uint64_t)(uint32_t)hi << 32 | (uint32_t)lo);
    };
    v += other(v, std::integral_constant<int, 0xb1>{});   // lane ^ 1
    v += other(v, std::integral_constant<int, 0x4e>{});   // lane ^ 2
    v += other(v, std::integral_constant<int, 0x141>{});  // the other quad of the half row
    return v + other(v, std::integral_constant<int, 0x140>{});
}

// One workgroup: 16 lanes add up the parts (256 at most) of an expert, all of their loads
// on their way together: latency, 2.7 us for 8 experts and 4.5 for 64.  (Counts as doubles,
// which hold them exactly.)
__global__ void __launch_bounds__(1024) balance_join_kernel(BalanceParams p) {
    const int lane = threadIdx.x & 15, rows = blockDim.x / 16;
    __shared__ double terms[64], zsum, live;
    double term = 0.0;
    for (int e = threadIdx.x / 16; e <= p.E; e += rows) {
        double s[16];
        int c[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int64_t at = (int64_t)e * p.parts + min(lane + 16 * i, p.parts - 1);
            s[i] = p.psum[at];
            c[i] = p.csum[at];
        }
        double sum = 0.0, count = 0.0;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (lane + 16 * i < p.parts) sum += s[i], count += (double)c[i];
        sum = row_sum(sum);
        count = row_sum(count);
        if (e < p.E) term += sum * count;
        if (lane == 0) {
            p.counts[e] = (int)count;
            if (e == p.E) zsum = sum, live = count;
        }
    }
    if (lane == 0) terms[threadIdx.x / 16] = term;
    __syncthreads();
    if (threadIdx.x >= 16) return;
    double s = 0.0;
    for (int i = lane; i < rows; i += 16) s += terms[i];
    s = row_sum(s);
    if (lane != 0) return;
    const double n = live;
    const double b = n > 0.0 ? (double)p.E * s / (n * n * (double)p.topk) : 0.0;
    const double z = n > 0.0 ? zsum / n : 0.0;
    p.loss[0] = (float)((double)p.balance * b + (double)p.z * z);
    p.loss[1] = (float)b;
    p.loss[2] = (float)z;
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
            // p = exp(l - lse) over its sum: lse is rounded, and where it is large beside log E its
            // rounding is a factor that all of a row's p share (E, for logits alike past 2^27 or so)
            bool bad = false;
            float l[V], dot = 0.0f, sum = 0.0f;
            balance_load<V, VEC>(p.logits + t * p.ldl, e0, p.E, l);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                // (an expert at -Inf, and those past E, have none; NaN - lse is NaN)
                l[i] = balance_exp(l[i] - lse);
                sum += l[i];
                dot = __builtin_fmaf(f[i], l[i], dot);
            }
            sum = group_sum<G>(sum);
            dot = group_sum<G>(dot);
            const float inv = __builtin_amdgcn_rcpf(sum);
            dot *= inv;
#pragma unroll
            for (int i = 0; i < V; ++i) l[i] *= inv;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                y[i] = g * l[i] * __builtin_fmaf(a, f[i] - dot, b * lse);
                bad |= !__builtin_isfinite(y[i]);
            }
            // a factor may have left fp32's range (a weight times E, lse times a weight) where the
            // result has not: once more in fp64
            if (__ballot(bad)) {
                const double gd = (double)(p.dloss ? *p.dloss : 1.0f) / (double)n;
                const double ad = (double)p.balance * (double)p.E, bd = 2.0 * (double)p.z * (double)lse;
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (!__builtin_isfinite(y[i]))
                        y[i] = (float)(gd * (double)l[i] * __builtin_fma(ad, (double)(f[i] - dot), bd));
            }
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
        e = hipLaunchKernel((const void *)balance_join_kernel, dim3(1),
                            dim3(E < 16 ? 256 : E < 32 ? 512 : 1024), args, 0, s);
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
