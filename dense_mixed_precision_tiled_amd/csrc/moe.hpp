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
// pass of its own: E / 64 loads and ballots for each token.  The expert of a slot that
// is not one is the largest logit left after r were taken out, up to 256 experts.
//
// One token's layer is mostly latency: the chain from the launch to the first
// weights (logits, expert, tokens) is kept to one load from memory in each kernel,
// with what follows from registers and LDS.
//
// Past 256 experts with fewer pairs than experts that does not hold: a workgroup ranks
// all experts of a token, E * E / 256 comparisons for a thread, from LDS up to 4096
// logits and from memory past that, before its first weight.  Top 8 of int8 experts of
// 512 x 256, one token: 35 us with 256 experts, 88 with 257, 167 with 512, 638 with
// 1024; eight tokens 48, 109, 190, 1204.
#pragma once

#include "stream.hpp"

namespace libgemm {

constexpr int kMoeMaxTokens = 64, kMoeMaxExperts = 1024, kMoeMaxTopk = 32;

struct MoeParams {
    const uint8_t *X, *W1, *W2;
    const float *logits, *s1, *s2;  // s1, s2: scales of int8 weights by row, or nullptr
    uint8_t *D;
    int64_t ldx, ldl, ld1, ld2, ldd;  // elements, at most 2^24: row offsets are 32 bits
    int T, H, I, E, topk, slots;
    int act, renorm;
    // workspace
    int *count;     // [slots] tokens of the slot's expert (0: no expert)
    int *expert;    // [slots]
    int *pairs;     // [slots][T] token * topk + rank, ascending
    float *weight;  // [T * topk] weight of each pair
    uint8_t *h;     // bf16: [2][T * topk][ldh], the values, and what is left of them;
                    // fp16: [T * topk][ldh] in fp32
    int ldh;
    __host__ __device__ int64_t h_low() const { return (int64_t)T * topk * ldh * 2; }
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

// Rank of expert e among the keys of one token (key(j) of expert j): the whole
// wave counts.
template <class Key>
__device__ __forceinline__ int moe_rank(Key &&key, int E, int e, int lane) {
    const uint32_t mine = key(e);
    int rank = 0;
    for (int j0 = 0; j0 < E; j0 += 64) {
        const int j = j0 + lane;
        const uint32_t k = j < E ? key(j) : 0u;
        rank += __popcll(__ballot(j < E && (k > mine || (k == mine && j < e))));
    }
    return mine > kMoeNone ? rank : kMoeMaxExperts;
}

// Largest value of the wave, in every lane.
__device__ __forceinline__ uint32_t moe_wave_max(uint32_t v) {
    auto step = [&](auto ctrl, auto rows) {
        v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, decltype(ctrl)::value,
                                                         decltype(rows)::value, 0xf, false));
    };
    using All = std::integral_constant<int, 0xf>;
    step(std::integral_constant<int, 0x111>{}, All{});  // row_shr 1, 2, 4, 8
    step(std::integral_constant<int, 0x112>{}, All{});
    step(std::integral_constant<int, 0x114>{}, All{});
    step(std::integral_constant<int, 0x118>{}, All{});
    step(std::integral_constant<int, 0x142>{}, std::integral_constant<int, 0xa>{});  // row_bcast 15
    step(std::integral_constant<int, 0x143>{}, std::integral_constant<int, 0xc>{});  // row_bcast 31
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// The expert of rank r among at most 256, or -1 (r experts or fewer above -Inf):
// the largest is taken out r times.  The whole wave, no LDS.
__device__ __forceinline__ int moe_expert_of_rank(const float *l, int E, int r, int lane) {
    uint32_t k[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) k[i] = lane + 64 * i < E ? moe_key(l[lane + 64 * i]) : 0u;
    for (;; --r) {
        const uint32_t m = moe_wave_max(max(max(k[0], k[1]), max(k[2], k[3])));
        if (m <= kMoeNone) return -1;
        int e = -1;
#pragma unroll
        for (int i = 3; i >= 0; --i) {
            const uint64_t b = __ballot(k[i] == m);
            if (b) e = 64 * i + (int)__builtin_ctzll(b);
        }
        if (r == 0) return e;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (e == lane + 64 * i) k[i] = 0u;
    }
}

template <int IT>
__device__ __forceinline__ uint16_t moe_round(float v) {
    constexpr int OUT = IT == IT_F16 ? DT_F16 : DT_BF16;
    return (uint16_t)to_out16<OUT>(v, false);
}

// What rounding v leaves of it; 0 where the rounded value is not finite.
template <int IT>
__device__ __forceinline__ float moe_rest(float v) {
    const float r = from_out16<IT == IT_F16 ? DT_F16 : DT_BF16>(moe_round<IT>(v));
    return fabsf(r) < __builtin_inff() ? v - r : 0.0f;
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
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
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

// Slot blockIdx.y, columns of h in blocks of 16, one in turn for each workgroup
// (KW = 4: its four waves split H) or for each wave (KW = 1: no exchange between
// waves); the last workgroup of a slot (blockIdx.x == gridDim.x - 1) writes the
// slot's tokens and the weights of token blockIdx.y, blockIdx.y + slots, ...
// instead.  MT = 1 takes the expert's tokens 16 at a time (the last four or eight
// without exchanges), MT = 0 (T <= 4) four.  One token and 8 experts of 2048 x 1024 in
// bf16: 16 us (4.2 TB/s); 16 tokens that reach 55 of them: 93 us (4.9 TB/s).
constexpr int kMoeStaged = 4096;  // logits (or pairs) that are held in LDS

template <int IT, bool W8, int MT, int KW, bool VEC>
__global__ void __launch_bounds__(256, 2) moe_up_kernel(MoeParams p) {
    using S = StreamTypes<IT, W8>;
    __shared__ uint32_t keys[kMoeStaged];
    __shared__ float part[8];
    __shared__ int ranks[kMoeMaxTokens], list[kMoeMaxTokens], found[2];
    constexpr int ROWS = MT == 0 ? 4 : 16;  // tokens of a pass
    __shared__ f32x4 sums[KW][KW > 1 ? 2 : 1][KW > 1 ? 64 : 1];
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int slot = blockIdx.y, t0 = slot / p.topk, r0 = slot % p.topk;
    const bool own = p.slots != p.E;  // the slot is token t0's expert of rank r0
    const bool staged = p.T * p.E <= kMoeStaged;

    int e = slot, n;
    if (own && p.T == 1 && p.E <= 256) {
        e = moe_expert_of_rank(p.logits, p.E, r0, lane);
        n = e >= 0 ? 1 : 0;
        if (tid == 0) list[0] = r0;
        __syncthreads();
    } else {
        auto key = [&](int t, int j) {
            return staged ? keys[t * p.E + j] : moe_key(p.logits[(int64_t)t * p.ldl + j]);
        };
        if (staged) {
            for (int i = tid; i < p.T * p.E; i += 256)
                keys[i] = moe_key(p.logits[(int64_t)(i / p.E) * p.ldl + i % p.E]);
            __syncthreads();
        }
        if (own) {
            if (p.E <= 256) {
                e = moe_expert_of_rank(p.logits + (int64_t)t0 * p.ldl, p.E, r0, lane);
            } else {
                if (tid == 0) found[0] = -1;
                __syncthreads();
                for (int j = tid; j < p.E; j += 256) {
                    const uint32_t mine = key(t0, j);
                    int rank = 0;
                    for (int i = 0; i < p.E; ++i) {
                        const uint32_t k = key(t0, i);
                        rank += k > mine || (k == mine && i < j);
                    }
                    if (rank == r0 && mine > kMoeNone) found[0] = j;
                }
                __syncthreads();
                e = found[0];
            }
        }
        // the tokens that chose it
        for (int t = wave; t < p.T; t += 4) {
            const int rank = e < 0 ? kMoeMaxExperts
                                   : moe_rank([&](int j) { return key(t, j); }, p.E, e, lane);
            if (lane == 0) ranks[t] = rank < p.topk ? rank : -1;
        }
        __syncthreads();
        if (wave == 0) {
            const int rank = lane < p.T ? ranks[lane] : -1;
            const uint64_t m = __ballot(rank >= 0);
            if (rank >= 0) list[__popcll(m & ((1ull << lane) - 1))] = lane * p.topk + rank;
            // an expert that an earlier token chose is that token's slot
            if (lane == 0)
                found[1] = own && (m & ((1ull << t0) - 1)) ? 0 : (int)__popcll(m);
        }
        __syncthreads();
        n = uniform(found[1]);
        e = uniform(e);
    }
    if (blockIdx.x == gridDim.x - 1) {
        if (tid == 0) p.count[slot] = n, p.expert[slot] = e;
        if (tid < n) p.pairs[slot * p.T + tid] = list[tid];
        for (int t = slot; t < p.T; t += p.slots) moe_weights(p, t, keys, part);
        return;
    }
    if (n == 0) return;

    const int groups = (p.H + S::KG - 1) / S::KG, per = (groups + KW - 1) / KW;
    const int kw = KW > 1 ? wave : 0;
    const int gbeg = min(kw * per, groups), gend = min((kw + 1) * per, groups);
    const int64_t first = (int64_t)e * 2 * p.I;
    auto token = [&](int i) {  // rows past the last token repeat it; not stored
        return (uint32_t)(list[min(i, n - 1)] / p.topk) * (uint32_t)p.ldx * 2u;
    };
    // h of row `row` of the list and columns c .. c + 3, from the gate's and up's sums
    auto finish = [&](int row, int c, f32x4 g, f32x4 u) {
        if (row >= n || c >= p.I) return;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if constexpr (W8) {
                const int cq = min(c + q, p.I - 1);
                g[q] *= p.s1[first + cq];
                u[q] *= p.s1[first + p.I + cq];
            }
            g[q] = moe_activate(g[q], p.act) * u[q];
        }
        // h as the sum of two values of x's type, which the second product's operand
        // has to be of.  Rounded to one value, its errors come to as much as y's own
        // rounding (1.41 times that together: 0.0024 against 0.0017 of y's norm for
        // bf16); 16 bits of h, or 22, leave them out.  It costs the second kernel the
        // reads of h twice (57 -> 71 us for 64 tokens and int8 experts of 4096 x 2048).
        // fp16's range is too small for h and for what is left of it, so there h
        // stays fp32 until the second kernel splits scaled rows of it (stream.hpp; two
        // unscaled parts: 64.4 us instead of 65.2 for 7 tokens and 16 experts of 4096 x
        // 1000, 192 instead of 205 for 64 tokens and 32 int8 experts of 4096 x 2048).
        uint8_t *const to = p.h + (int64_t)list[row] * p.ldh * (IT == IT_F16 ? 4 : 2);
        if constexpr (IT == IT_F16) {
            float *const d = reinterpret_cast<float *>(to) + c;
            if (p.I - c >= 4) {
                *reinterpret_cast<f32x4 *>(d) = g;
            } else {
#pragma unroll
                for (int q = 0; q < 3; ++q)
                    if (q < p.I - c) d[q] = g[q];
            }
        } else {
            moe_store4<IT>(to, c, p.I - c, true, g);
#pragma unroll
            for (int q = 0; q < 4; ++q) g[q] = moe_rest<IT>(g[q]);
            moe_store4<IT>(to + p.h_low(), c, p.I - c, true, g);
        }
    };
    const int step = (4 / KW) * (gridDim.x - 1);
#pragma nounroll
    for (int jb = (4 / KW) * blockIdx.x + (KW > 1 ? 0 : wave); jb * 16 < p.I; jb += step) {
        const int lane = opaque(tid & 63);
        StreamRows w[2];
#pragma unroll
        for (int f = 0; f < 2; ++f)
            w[f].set(lane, p.W1 + (first + f * p.I + jb * 16) * p.ld1 * S::WES, [&](int i) {
                return (uint32_t)min(i, p.I - 1 - jb * 16) * (uint32_t)p.ld1 * S::WES;
            });
#pragma nounroll
        for (int n0 = 0; n0 < n; n0 += ROWS) {
            const int lane = opaque(tid & 63);
            const int c = jb * 16 + 4 * (lane >> 4);
            // sums of the gate and up products, and the lane's row of this pass
            f32x4 g, u;
            int row;
            auto quads = [&](auto sets) {
                constexpr int SETS = decltype(sets)::value;
                StreamX<SETS> x;
                x.set(lane, p.X, [&](int i) { return token(n0 + i); });
                // (a second group in flight: 149 -> 142 us for a layer of 16 tokens, 214 ->
                // 198 with eight tokens for each of 32 int8 experts of 4096 x 2048; with
                // MT = 0 its registers cost more than it gives, 26.9 -> 27.3 at one token)
                StreamQuads<IT, W8, SETS, 2, (MT > 0), VEC, VEC> stream;
                stream.run(w, x, lane, gbeg, gend, p.H);
                g = stream.template own_sums<0>(lane);
                u = stream.template own_sums<1>(lane);
                row = stream_row<SETS>(lane);
            };
            if (MT == 0 || n - n0 <= 4) {
                quads(std::integral_constant<int, 1>{});
            } else if constexpr (MT > 0) {
                if (n - n0 <= 8) {
                    quads(std::integral_constant<int, 2>{});
                } else {
                    StreamRows x[1];
                    x[0].set(lane, p.X, [&](int i) { return token(n0 + i); });
                    f32x4 acc[1][2] = {};
                    StreamTiles<IT, W8, 1, 2, false, VEC, VEC> stream;
                    stream.run(w, x, lane, gbeg, gend, p.H, acc);
                    g = acc[0][0];
                    u = acc[0][1];
                    row = lane & 15;
                }
            }
            if constexpr (KW == 1) {
                finish(n0 + row, c, g, u);
            } else {
                sums[wave][0][lane] = g;
                sums[wave][1][lane] = u;
            }
            if constexpr (KW > 1) {
                __syncthreads();
                if (wave == 0) {
#pragma unroll
                    for (int z = 1; z < KW; ++z) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            g[q] += sums[z][0][lane][q];
                            u[q] += sums[z][1][lane][q];
                        }
                    }
                    finish(n0 + row, c, g, u);
                }
                __syncthreads();
            }
        }
    }
}

// Workgroup b computes columns [16 b, 16 b + 16) of y, or with NM = 2 columns [8 b,
// 8 b + 8).  W waves share the (expert, part of I) units; each adds w * (h D_e^T) to
// its own copy of y in LDS (the columns of every token), and the copies are added in
// order.  TM: the most tokens.  Passes of at most two tokens hold both parts of h in one set of rows,
// longer ones take a second operand for each of w's; those of up to 12 tokens (with
// blocks of 8 columns, 16) need no exchanges.  64 tokens and 32 int8 experts of 4096 x
// 2048: 71 us (3.8 TB/s).  Every workgroup reads all of h, twice the bytes of its
// weights there: 58 us with a single row of h; the conversion of the weights to bf16 is
// hidden (69 without it).
template <int IT, bool W8, int TM, int W, int NM, bool VEC>
__global__ void __launch_bounds__(64 * W) moe_down_kernel(MoeParams p) {
    using S = StreamTypes<IT, W8>;
    constexpr int MT = TM <= 4 ? 0 : 1, ROWS = MT == 0 ? 4 : 16;
    constexpr bool XF = IT == IT_F16;  // h is fp32
    typedef float Cols __attribute__((ext_vector_type(NM)));
    __shared__ Cols y[W][TM][4];
    __shared__ int active[kMoeMaxExperts], count[kMoeMaxExperts], expert[kMoeMaxExperts], found;
    __shared__ int pairs[kMoeStaged];
    __shared__ float weight[kMoeMaxTokens * kMoeMaxTopk];
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int n0 = blockIdx.x * (4 * NM);
    const bool staged = p.slots * p.T <= kMoeStaged;

    // everything that the first kernel found, in one go
    for (int i = tid; i < p.slots; i += 64 * W) {
        count[i] = p.count[i];
        expert[i] = p.expert[i];
    }
    if (staged)
        for (int i = tid; i < p.slots * p.T; i += 64 * W) pairs[i] = p.pairs[i];
    for (int i = tid; i < p.T * p.topk; i += 64 * W) weight[i] = p.weight[i];
    if (wave == 0) {  // the slots that have tokens
        int a = 0;
        for (int s0 = 0; s0 < p.slots; s0 += 64) {
            const int s = s0 + lane;
            const bool any = s < p.slots && p.count[s] > 0;
            const uint64_t m = __ballot(any);
            if (any) active[a + __popcll(m & ((1ull << lane) - 1))] = s;
            a += __popcll(m);
        }
        if (lane == 0) found = a;
    }
    for (int i = tid; i < W * TM * 4; i += 64 * W)
        (&y[0][0][0])[i] = Cols(0.0f);
    __syncthreads();

    // parts of I for each expert: enough units for every wave, evenly
    const int A = uniform(found);
    const int groups = (p.I + S::KG - 1) / S::KG;
    int parts = 1;
    while (parts < W && (A * parts) % W != 0 && A * parts < 4 * W) ++parts;
    const int per = (groups + parts - 1) / parts;
    for (int unit = wave; unit < A * parts; unit += W) {
        const int lane = opaque(tid & 63), lg = lane >> 4;
        const int slot = uniform(active[unit / parts]), z = unit % parts;
        const int n = uniform(count[slot]), e = uniform(expert[slot]);
        const int gbeg = min(z * per, groups), gend = min((z + 1) * per, groups);
        auto pair = [&](int i) {
            const int at = slot * p.T + min(i, n - 1);
            if (staged) return pairs[at];
            return p.pairs[at];
        };
        auto hrow = [&](int i) { return (uint32_t)pair(i) * (uint32_t)p.ldh * (XF ? 4u : 2u); };
        StreamRows w[1];
        w[0].template set<NM>(lane, p.W2 + ((int64_t)e * p.H + n0) * p.ld2 * S::WES, [&](int i) {
            return (uint32_t)min(i, p.H - 1 - n0) * (uint32_t)p.ld2 * S::WES;
        });
        f32x4 s = {1.0f, 1.0f, 1.0f, 1.0f};
        if constexpr (W8) {
#pragma unroll
            for (int q = 0; q < NM; ++q)
                s[q] = p.s2[(int64_t)e * p.H + min(n0 + NM * lg + q, p.H - 1)];
        }
        // add row i's sums v of columns NM lg + 0 .. NM - 1
        auto add = [&](int i, const f32x4 &v) {
            const int at = pair(i);
            const float wt = weight[at];
            Cols *dst = &y[wave][at / p.topk][lg];
            Cols o = *dst;
#pragma unroll
            for (int q = 0; q < NM; ++q) o[q] += wt * (v[q] * s[q]);
            *dst = o;
        };
#pragma nounroll
        for (int i0 = 0; i0 < n; i0 += ROWS) {
            const int lane = opaque(tid & 63);
            f32x4 v;
            int row;
            auto quads = [&](auto sets) {
                constexpr int SETS = decltype(sets)::value;
                StreamX<SETS> x;
                x.set(lane, p.h, [&](int i) { return hrow(i0 + i); }, p.h_low());
                StreamQuads<IT, W8, SETS, 1, SETS == 1, true, VEC, 2, NM, XF> stream;
                stream.run(w, x, lane, gbeg, gend, p.I);
                v = stream.template own_sums<0>(lane);
                row = stream_row<SETS>(lane);
            };
            if (n - i0 <= 2) {
                // both parts of h in one set: rows 0 and 1 the values, 2 and 3 the rests
                StreamX<1> x;
                x.set(lane, p.h, [&](int i) {
                    return hrow(i0 + (i & 1)) + (!XF && (i & 2) ? (uint32_t)p.h_low() : 0u);
                });
                StreamQuads<IT, W8, 1, 1, true, true, VEC, 1, NM, XF> stream;
                stream.run(w, x, lane, gbeg, gend, p.I);
                v = stream.template own_sums<0>(lane);
#pragma unroll
                for (int q = 0; q < NM; ++q)  // row_ror 8: lane l's neighbour at l ^ 8
                    v[q] += __int_as_float(
                        __builtin_amdgcn_mov_dpp(__float_as_int(v[q]), 0x128, 0xf, 0xf, true));
                row = stream_row<1>(lane);
            } else if (MT == 0 || n - i0 <= 4) {
                quads(std::integral_constant<int, 1>{});
            } else if constexpr (MT > 0) {
                if (n - i0 <= 8) {
                    quads(std::integral_constant<int, 2>{});
                } else if (n - i0 <= 12) {
                    quads(std::integral_constant<int, 3>{});
                } else if constexpr (NM == 2) {
                    quads(std::integral_constant<int, 4>{});
                } else {
                    StreamRows x[1];
                    x[0].set(lane, p.h, [&](int i) { return hrow(i0 + i); }, p.h_low());
                    f32x4 acc[1][1] = {};
                    StreamTiles<IT, W8, 1, 1, false, true, VEC, 2, XF> stream;
                    stream.run(w, x, lane, gbeg, gend, p.I, acc);
                    v = acc[0][0];
                    row = lane & 15;
                }
            }
            if (i0 + row < n) add(i0 + row, v);
        }
    }
    __syncthreads();
    for (int i = tid; i < p.T * 4; i += 64 * W) {
        const int t = i >> 2, g = i & 3, c = n0 + NM * g;
        if (c >= p.H) continue;
        f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int z = 0; z < W; ++z) {
#pragma unroll
            for (int q = 0; q < NM; ++q) v[q] += y[z][t][g][q];
        }
        // a token whose weights are NaN has a NaN row, also where no expert was
        // chosen
        for (int k = 0; k < p.topk; ++k) {
            const float wt = weight[t * p.topk + k];
            if (wt != wt) v = f32x4{wt, wt, wt, wt};
        }
        uint8_t *row = p.D + (int64_t)t * p.ldd * 2;
        const bool vec = (reinterpret_cast<uintptr_t>(p.D) % 8 == 0) && p.ldd % 4 == 0;
        moe_store4<IT>(row, c, min(p.H - c, NM), vec, v);
    }
}

template <int IT, bool W8, bool VEC>
hipError_t moe_launch(const MoeParams &p, int cus, hipStream_t s) {
    MoeParams arg = p;
    void *args[] = {&arg};
    // Blocks of 16 columns of every slot: one for each wave where that gives every
    // CU eight waves, otherwise one for each workgroup (7 tokens, 16 experts top 4 of
    // 4096 x 1000: 64 us with a block for each workgroup, 76 for each wave; 64 tokens,
    // 32 top 4 of 4096 x 2048 in int8: 211 and 198).  Then about four workgroups for each
    // CU; one takes several blocks where there are more (198; with two 213, eight 198).
    const int64_t blocks = (p.I + 15) / 16;
    const bool alone = blocks * p.slots >= 8 * (int64_t)cus;
    const int64_t parts = alone ? (blocks + 3) / 4 : blocks;
    const int64_t want = (4 * (int64_t)cus + p.slots - 1) / p.slots;
    const dim3 up((unsigned)(parts < want ? parts : want) + 1, (unsigned)p.slots);
    // Columns of y in blocks of 16, or of 8 where those of 16 leave half of the CUs idle
    // (H = 2048, 64 experts top 8: both kernels 147.7 -> 136.6 us at 16 tokens, 27.3 ->
    // 26.1 at one).  Every block reads all of h, so at H = 4096 those of 8 lose: 7 tokens
    // 64.2 -> 65.9 us, 64 tokens 198 -> 229.
    const bool narrow = 2 * ((p.H + 15) / 16) <= cus;
    const dim3 down((unsigned)(narrow ? (p.H + 7) / 8 : (p.H + 15) / 16));
    const void *k1, *k2;
    if (p.T <= 4)
        k1 = alone ? (const void *)moe_up_kernel<IT, W8, 0, 1, VEC>
                   : (const void *)moe_up_kernel<IT, W8, 0, 4, VEC>;
    else
        k1 = alone ? (const void *)moe_up_kernel<IT, W8, 1, 1, VEC>
                   : (const void *)moe_up_kernel<IT, W8, 1, 4, VEC>;
    if (narrow)
        k2 = p.T <= 4    ? (const void *)moe_down_kernel<IT, W8, 4, 8, 2, VEC>
             : p.T <= 16 ? (const void *)moe_down_kernel<IT, W8, 16, 8, 2, VEC>
                         : (const void *)moe_down_kernel<IT, W8, 64, 8, 2, VEC>;
    else
        k2 = p.T <= 4    ? (const void *)moe_down_kernel<IT, W8, 4, 8, 4, VEC>
             : p.T <= 16 ? (const void *)moe_down_kernel<IT, W8, 16, 8, 4, VEC>
                         : (const void *)moe_down_kernel<IT, W8, 64, 8, 4, VEC>;
    const hipError_t st = hipLaunchKernel(k1, up, dim3(256), args, 0, s);
    if (st != hipSuccess) return st;
    return hipLaunchKernel(k2, down, dim3(512), args, 0, s);
}

// One translation unit for each type of x and w: moe_<x>.hip, moe_<x>_i8.hip.
// vec: x and the weights allow 16-byte loads.
hipError_t launch_moe_f16(const MoeParams &, int cus, bool vec, hipStream_t);
hipError_t launch_moe_bf16(const MoeParams &, int cus, bool vec, hipStream_t);
hipError_t launch_moe_f16_i8(const MoeParams &, int cus, bool vec, hipStream_t);
hipError_t launch_moe_bf16_i8(const MoeParams &, int cus, bool vec, hipStream_t);

}  // namespace libgemm
