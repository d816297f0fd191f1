// A mixture-of-experts layer for a few tokens, in two kernels.
//
//   p = softmax(l_t);  the topk experts of largest l_t (ties: lower index);
//   h = act(x_t G_e^T) * (x_t U_e^T);   y_t = sum_e w_te (h D_e^T)
//
// moe_up_kernel finds the routing and computes h for every (token, expert) pair
// into the workspace; moe_down_kernel computes y.  Both stream the chosen experts'
// weights once (stream.hpp), whatever the number of tokens that chose them: the
// tokens of one expert are gathered into the 16 rows of the matrix unit's second
// operand.  What bounds both is the weights' bytes; the routing is latency.
//
// No expert is known on the host, so the grid holds min(E, T * topk) slots of
// experts.  With E <= T * topk a slot is an expert.  Otherwise slot s is the
// expert that token s / topk ranks s % topk, if no earlier token chose it too.
// A slot without tokens ends at once.  Every workgroup finds its own expert
// and tokens by counting the logits above one (the rank of an expert is how
// many are larger, or equal with a lower index), which needs no sorting and no
// pass of its own: E / 64 loads and ballots for each token.
#pragma once

#include "stream.hpp"

namespace libgemm {

constexpr int kMoeMaxTokens = 64, kMoeMaxExperts = 1024, kMoeMaxTopk = 32;

struct MoeParams {
    const uint8_t *X, *W1, *W2;
    const float *logits, *s1, *s2;  // s1, s2: scales of int8 weights by row, or nullptr
    uint8_t *D;
    int64_t ldx, ldl, ld1, ld2, ldd;  // elements
    int T, H, I, E, topk, slots;
    int act, renorm;
    // workspace
    int *count;     // [slots] tokens of the slot's expert (0: no expert)
    int *expert;    // [slots]
    int *pairs;     // [slots][T] token * topk + rank, ascending
    float *weight;  // [T * topk] weight of each pair
    uint8_t *h;     // [T * topk][ldh] in the type of x
    int ldh;
};

enum { MOE_SILU = 3 };  // beside ACT_*

// silu(x) = x / (1 + exp(-x))
__device__ __forceinline__ float moe_activate(float x, int act) {
    return act == MOE_SILU ? x / (1.0f + __expf(-x)) : activate(x, act);
}

// Integers in the order of the logits (-0 equals +0); NaN below everything.
__device__ __forceinline__ uint32_t moe_key(float l) {
    const uint32_t u = __float_as_uint(l + 0.0f);
    if (l != l) return 0u;
    return (u >> 31) ? ~u : (u | 0x80000000u);
}
constexpr uint32_t kMoeNone = 0x007fffffu;  // key of -Inf: such an expert is not chosen

// Rank of expert e among the logits of one token: the whole wave counts.
__device__ __forceinline__ int moe_rank(const float *l, int E, int e, uint32_t mine, int lane) {
    int rank = 0;
    for (int j0 = 0; j0 < E; j0 += 64) {
        const int j = j0 + lane;
        const uint32_t k = j < E ? moe_key(l[j]) : 0u;
        rank += __popcll(__ballot(j < E && (k > mine || (k == mine && j < e))));
    }
    return rank;
}

template <int IT>
__device__ __forceinline__ uint16_t moe_round(float v) {
    constexpr int OUT = IT == IT_F16 ? DT_F16 : DT_BF16;
    return (uint16_t)to_out16<OUT>(v, false);
}

// Four values of 16 bits, as many of them as n.
template <int IT>
__device__ __forceinline__ void moe_store4(uint8_t *row, int64_t j, int n, bool vec, f32x4 v) {
    uint16_t *d = reinterpret_cast<uint16_t *>(row) + j;
    if (vec && n >= 4) {
        *reinterpret_cast<u32x2 *>(d) =
            u32x2{(uint32_t)moe_round<IT>(v[0]) | ((uint32_t)moe_round<IT>(v[1]) << 16),
                  (uint32_t)moe_round<IT>(v[2]) | ((uint32_t)moe_round<IT>(v[3]) << 16)};
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e < n) d[e] = moe_round<IT>(v[e]);
    }
}

// The weights of token t's pairs: exp(l - max) / sum, the sum over all experts
// or over the chosen ones.  A row with a NaN or +Inf gives NaN, a row of -Inf
// zeros; an expert at -Inf has weight 0.  The 256 threads of the workgroup.
__device__ inline void moe_weights(const MoeParams &p, int t, uint32_t *keys, float *part) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const float *l = p.logits + (int64_t)t * p.ldl;
    __syncthreads();  // keys and part of the token before
    float top = -__builtin_inff();
    for (int j = tid; j < p.E; j += 256) {
        const float x = l[j];
        keys[j] = moe_key(x);
        top = fmaxf(top, x);
    }
    for (int m = 32; m; m >>= 1) top = fmaxf(top, __shfl_xor(top, m));
    if (lane == 0) part[wave] = top;
    __syncthreads();
    top = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
    auto share = [&](float x) { return x == -__builtin_inff() ? 0.0f : expf(x - top); };
    auto rank_of = [&](int j) {
        const uint32_t mine = keys[j];
        int rank = 0;
        for (int i = 0; i < p.E; ++i) rank += keys[i] > mine || (keys[i] == mine && i < j);
        return rank;
    };
    float all = 0.0f, chosen = 0.0f;
    for (int j = tid; j < p.E; j += 256) {
        const float e = share(l[j]);
        all += e;
        if (rank_of(j) < p.topk) chosen += e;
    }
    for (int m = 32; m; m >>= 1) {
        all += __shfl_xor(all, m);
        chosen += __shfl_xor(chosen, m);
    }
    __syncthreads();
    if (lane == 0) part[wave] = all, part[4 + wave] = chosen;
    __syncthreads();
    all = (part[0] + part[1]) + (part[2] + part[3]);
    chosen = (part[4] + part[5]) + (part[6] + part[7]);
    // all is NaN where a logit is NaN or +Inf, and 0 only where every one is -Inf
    for (int j = tid; j < p.E; j += 256) {
        const int rank = rank_of(j);
        if (rank >= p.topk) continue;
        float w = share(l[j]) / (p.renorm ? chosen : all);
        if (all == 0.0f) w = 0.0f;
        p.weight[t * p.topk + rank] = all != all ? __builtin_nanf("") : w;
    }
}

// Slot blockIdx.y, columns of h in blocks of 16, one for each workgroup in
// turn; the last workgroup of a slot (blockIdx.x == gridDim.x - 1) writes the
// slot's tokens and the weights of token blockIdx.y, blockIdx.y + slots, ...
// instead.  MT: row groups of 16 tokens; four waves split H.
template <int IT, bool W8, int MT, bool VEC>
__global__ void __launch_bounds__(256) moe_up_kernel(MoeParams p) {
    using S = StreamTypes<IT, W8>;
    constexpr int U = MT == 4 ? 1 : (MT == 2 ? 2 : (W8 ? 2 : 4));
    __shared__ uint32_t keys[kMoeMaxExperts];
    __shared__ float part[8];
    __shared__ int ranks[kMoeMaxTokens], list[kMoeMaxTokens], found[2];
    __shared__ f32x4 sums[4][2 * MT][64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int slot = blockIdx.y;

    // the slot's expert
    int e = slot, t0 = 0;
    if (p.slots != p.E) {
        t0 = slot / p.topk;
        const int r0 = slot % p.topk;
        const float *l = p.logits + (int64_t)t0 * p.ldl;
        for (int j = tid; j < p.E; j += 256) keys[j] = moe_key(l[j]);
        __syncthreads();
        for (int j = tid; j < p.E; j += 256) {
            const uint32_t mine = keys[j];
            int rank = 0;
            for (int i = 0; i < p.E; ++i) rank += keys[i] > mine || (keys[i] == mine && i < j);
            if (rank == r0) found[0] = j;  // ranks are 0 .. E - 1, each once
        }
        __syncthreads();
        e = found[0];
    }
    // its tokens
    for (int t = wave; t < p.T; t += 4) {
        const float *l = p.logits + (int64_t)t * p.ldl;
        const uint32_t mine = moe_key(l[e]);
        const int rank = moe_rank(l, p.E, e, mine, lane);
        if (lane == 0) ranks[t] = rank < p.topk && mine > kMoeNone ? rank : -1;
    }
    __syncthreads();
    if (wave == 0) {
        const int rank = lane < p.T ? ranks[lane] : -1;
        const uint64_t m = __ballot(rank >= 0);
        if (rank >= 0) list[__popcll(m & ((1ull << lane) - 1))] = lane * p.topk + rank;
        // an expert that an earlier token chose is that token's slot
        if (lane == 0) found[1] = (m & ((1ull << t0) - 1)) ? 0 : (int)__popcll(m);
    }
    __syncthreads();
    const int n = found[1];
    if (blockIdx.x == gridDim.x - 1) {
        if (tid == 0) p.count[slot] = n, p.expert[slot] = e;
        if (tid < n) p.pairs[slot * p.T + tid] = list[tid];
        for (int t = slot; t < p.T; t += p.slots) moe_weights(p, t, keys, part);
        return;
    }
    if (n == 0) return;

    const int r = lane & 15;
    const uint8_t *xr[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t)  // rows past the last token repeat it; not stored
        xr[t] = p.X + (int64_t)(list[min(16 * t + r, n - 1)] / p.topk) * p.ldx * 2;
    const int blocks = (p.H + S::KB - 1) / S::KB, per = (blocks + 3) / 4;
    const int bbeg = min(wave * per, blocks), bend = min((wave + 1) * per, blocks);
    const int64_t first = (int64_t)e * 2 * p.I;
    for (int jb = blockIdx.x; jb * 16 < p.I; jb += gridDim.x - 1) {
        const int j = min(jb * 16 + r, p.I - 1);
        const uint8_t *wr[2] = {p.W1 + (first + j) * p.ld1 * S::WES,
                                p.W1 + (first + p.I + j) * p.ld1 * S::WES};
        f32x4 acc[MT][2] = {};
        Stream<IT, W8, MT, 2, U, VEC, VEC> stream;
        stream.run(wr, xr, lane, bbeg, bend, p.H, acc);
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            sums[wave][2 * t][lane] = acc[t][0];
            sums[wave][2 * t + 1][lane] = acc[t][1];
        }
        __syncthreads();
        // lane: row 16 t + lane % 16, four columns from 4 (lane / 16)
        if (wave < MT) {
            const int t = wave, row = 16 * t + r, c = jb * 16 + 4 * (lane >> 4);
            f32x4 g = sums[0][2 * t][lane], u = sums[0][2 * t + 1][lane];
#pragma unroll
            for (int z = 1; z < 4; ++z) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    g[q] += sums[z][2 * t][lane][q];
                    u[q] += sums[z][2 * t + 1][lane][q];
                }
            }
            if (row < n && c < p.I) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if constexpr (W8) {
                        const int cq = min(c + q, p.I - 1);
                        g[q] *= p.s1[first + cq];
                        u[q] *= p.s1[first + p.I + cq];
                    }
                    g[q] = moe_activate(g[q], p.act) * u[q];
                }
                // h is rounded to x's type: the second product's operand has
                // to be of that type, and its rounding errors, of independent
                // signs, come to about as much as y's own
                moe_store4<IT>(p.h + (int64_t)list[row] * p.ldh * 2, c, p.I - c, true, g);
            }
        }
        __syncthreads();
    }
}

// Workgroup b computes columns [16 b, 16 b + 16) of y.  Eight waves share the
// (expert, part of I) units; each adds w * (h D_e^T) to its own copy of y in LDS
// (16 columns of every token), and the copies are added in order.
template <int IT, bool W8, int MT, bool VEC>
__global__ void __launch_bounds__(512) moe_down_kernel(MoeParams p) {
    using S = StreamTypes<IT, W8>;
    constexpr int W = 8;
    constexpr int U = MT == 4 ? 2 : (W8 ? 2 : 4);
    __shared__ f32x4 y[W][16 * MT][4];
    __shared__ int slot_of[kMoeMaxExperts], begin[kMoeMaxExperts + 1], active;
    __shared__ int pairs[kMoeMaxTokens * kMoeMaxTopk];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int n0 = blockIdx.x * 16, r = lane & 15, lg = lane >> 4;

    for (int i = tid; i < W * 16 * MT * 4; i += 64 * W)
        (&y[0][0][0])[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    // the slots that have tokens, and where their pairs start
    if (wave == 0) {
        int a = 0, at = 0;
        for (int s0 = 0; s0 < p.slots; s0 += 64) {
            const int s = s0 + lane, c = s < p.slots ? p.count[s] : 0;
            const uint64_t m = __ballot(c > 0);
            int sum = c;  // inclusive prefix sum over the wave
            for (int d = 1; d < 64; d <<= 1) {
                const int o = __shfl_up(sum, d);
                if (lane >= d) sum += o;
            }
            if (c > 0) {
                const int pos = a + __popcll(m & ((1ull << lane) - 1));
                slot_of[pos] = s;
                begin[pos] = at + sum - c;
            }
            a += __popcll(m);
            at += __shfl(sum, 63);
        }
        if (lane == 0) active = a, begin[a] = at;
    }
    __syncthreads();
    const int A = active;
    for (int a = wave; a < A; a += W) {
        const int b0 = begin[a], c = begin[a + 1] - b0;
        if (lane < c) pairs[b0 + lane] = p.pairs[slot_of[a] * p.T + lane];
    }
    __syncthreads();

    // parts of I for each expert: enough units for every wave, evenly
    const int blocks = (p.I + S::KB - 1) / S::KB;
    int parts = 1;
    while (parts < W && (A * parts) % W != 0 && A * parts < 4 * W) ++parts;
    const int per = (blocks + parts - 1) / parts;
    for (int unit = wave; unit < A * parts; unit += W) {
        const int a = unit / parts, z = unit % parts;
        const int b0 = begin[a], n = begin[a + 1] - b0, e = p.expert[slot_of[a]];
        const int j = min(n0 + r, p.H - 1);
        const uint8_t *wr[1] = {p.W2 + ((int64_t)e * p.H + j) * p.ld2 * S::WES};
        const uint8_t *xr[MT];
#pragma unroll
        for (int t = 0; t < MT; ++t)
            xr[t] = p.h + (int64_t)pairs[b0 + min(16 * t + r, n - 1)] * p.ldh * 2;
        f32x4 acc[MT][1] = {};
        Stream<IT, W8, MT, 1, U, true, VEC> stream;
        stream.run(wr, xr, lane, min(z * per, blocks), min((z + 1) * per, blocks), p.I, acc);
        f32x4 s = {1.0f, 1.0f, 1.0f, 1.0f};
        if constexpr (W8) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                s[q] = p.s2[(int64_t)e * p.H + min(n0 + 4 * lg + q, p.H - 1)];
        }
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            const int row = 16 * t + r;
            if (row < n) {
                const int pair = pairs[b0 + row];
                const float w = p.weight[pair];
                f32x4 *dst = &y[wave][pair / p.topk][lg];
                f32x4 v = *dst;
#pragma unroll
                for (int q = 0; q < 4; ++q) v[q] += w * (acc[t][0][q] * s[q]);
                *dst = v;
            }
        }
    }
    __syncthreads();
    for (int i = tid; i < p.T * 4; i += 64 * W) {
        const int t = i >> 2, g = i & 3, c = n0 + 4 * g;
        if (c >= p.H) continue;
        f32x4 v = y[0][t][g];
#pragma unroll
        for (int z = 1; z < W; ++z) {
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] += y[z][t][g][q];
        }
        // a token whose weights are NaN has a NaN row, also where no expert was
        // chosen
        for (int k = 0; k < p.topk; ++k) {
            const float w = p.weight[t * p.topk + k];
            if (w != w) v = f32x4{w, w, w, w};
        }
        uint8_t *row = p.D + (int64_t)t * p.ldd * 2;
        const bool vec = (reinterpret_cast<uintptr_t>(p.D) % 8 == 0) && p.ldd % 4 == 0;
        moe_store4<IT>(row, c, p.H - c, vec, v);
    }
}

template <int IT, bool W8, bool VEC>
hipError_t moe_launch(const MoeParams &p, int up_blocks, hipStream_t s) {
    MoeParams arg = p;
    void *args[] = {&arg};
    const dim3 up((unsigned)up_blocks + 1, (unsigned)p.slots), down((unsigned)((p.H + 15) / 16));
    const void *k1, *k2;
    if (p.T <= 16) {
        k1 = (const void *)moe_up_kernel<IT, W8, 1, VEC>;
        k2 = (const void *)moe_down_kernel<IT, W8, 1, VEC>;
    } else if (p.T <= 32) {
        k1 = (const void *)moe_up_kernel<IT, W8, 2, VEC>;
        k2 = (const void *)moe_down_kernel<IT, W8, 2, VEC>;
    } else {
        k1 = (const void *)moe_up_kernel<IT, W8, 4, VEC>;
        k2 = (const void *)moe_down_kernel<IT, W8, 4, VEC>;
    }
    const hipError_t st = hipLaunchKernel(k1, up, dim3(256), args, 0, s);
    if (st != hipSuccess) return st;
    return hipLaunchKernel(k2, down, dim3(512), args, 0, s);
}

// One translation unit for each type of x and w: moe_<x>.hip, moe_<x>_i8.hip.
// vec: x and the weights allow 16-byte loads.
hipError_t launch_moe_f16(const MoeParams &, int up_blocks, bool vec, hipStream_t);
hipError_t launch_moe_bf16(const MoeParams &, int up_blocks, bool vec, hipStream_t);
hipError_t launch_moe_f16_i8(const MoeParams &, int up_blocks, bool vec, hipStream_t);
hipError_t launch_moe_bf16_i8(const MoeParams &, int up_blocks, bool vec, hipStream_t);

}  // namespace libgemm
