// gemm_checkpoint_wgrad: D = G^T X^ + C, a linear layer's weight gradient from packed
// activations (checkpoint.hpp).
//
//   D(n,k) = sum_m G(m,n) X^(m,k),   X^(m,k) = 2^(S(m,k/32) - 133) Q(m,k)
//
// A product whose reduction runs over the tokens m.  The scales belong to a token and a
// block of columns, so they cannot be applied to finished sums: Q is widened to the
// matrix units' 16-bit type on its way into LDS, where a 16-byte load holds 16 values of
// one block.  That is exact (seven bits and a power of two), and so are the products.
// Few outputs leave CUs idle, so their tokens are taken in parts by different workgroups,
// whose fp32 sums go to the workspace and are added up, in order, by a second kernel.
//
// Three kernels: tiles for 16-byte aligned lines (wgrad.hpp), thin ones for up to 64 outputs
// (wgrad_thin.hpp), and one for any alignment.  us: 16 x 4096 of 8192 tokens 13.2 and 2.4 for
// the sums (2.7 TB/s: latency); 1001 x 2056 of 3999 39 and 6 (420 TFLOP/s: 408 workgroups on
// 512 places, edge tiles); 4096 x 4096 of 4096 with C 152 (900 TFLOP/s), without 142 (bf16
// operands of the same layout 131, without Q to widen).  Any alignment: 117, 199 and 1196 without C.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/libgemm.h"
#include "gemm_configs.hpp"
#include "gemm_host.hpp"
#include "gemm_validate.hpp"
#include "wgrad_thin.hpp"

namespace libgemm {

// Any alignment, line length and number of tokens: the same product with one stage and
// element-wise loads.  128 x 128 tiles of D, four waves, 64 tokens at a time.
constexpr int kWgAnyBM = 128, kWgAnyBN = 128;

template <int IT, int OUT>
__global__ void __launch_bounds__(256) wgrad_any_kernel(WgradParams p) {
    using CF = TileCfg<kWgAnyBM, kWgAnyBN, 64, 2, 2, 32>;
    constexpr int BK = 64, CA = CF::BM / 8, CB = CF::BN / 8, TM = CF::TM, TN = CF::TN;
    constexpr int NA = BK * CA / 256, NB = BK * (CF::BN / 16) / 256;
    __shared__ u32x4 smem[BK * (CA + CB)];
    u32x4 *const sA = smem, *const sB = smem + BK * CA;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wm = wave / CF::WAVES_N, wn = wave % CF::WAVES_N;
    int tile_n, tile_k;
    map_tile(p.g, blockIdx.x, tile_n, tile_k);
    const int n0 = tile_n * CF::BM, k0 = tile_k * CF::BN, N = p.g.M, K = p.g.N;
    // (64 bits: a last step may end past 2^31)
    const int64_t m_beg = (int64_t)blockIdx.z * p.g.k_per_split;
    const int64_t m_end = m_beg + p.g.k_per_split < p.g.K ? m_beg + p.g.k_per_split : p.g.K;
    f32x16 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = f32x16{};

    for (int64_t m0 = m_beg; m0 < m_end; m0 += BK) {
        __syncthreads();  // the last step's reads are done
#pragma unroll
        for (int i = 0; i < NA; ++i) {
            const int at = i * 256 + tid, r = at / CA, c = at % CA, n = n0 + c * 8;
            const int64_t m = m0 + r;
            u32x4 a = {0u, 0u, 0u, 0u};
            if (m < m_end) {
                const uint16_t *row = p.g.A + m * p.g.lda;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (n + e < N) a[e / 2] |= (uint32_t)row[n + e] << (16 * (e % 2));
            }
            sA[r * CA + (c ^ wgrad_slot<CA>(r, c))] = a;
        }
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int at = i * 256 + tid, r = at / (CF::BN / 16), k = k0 + at % (CF::BN / 16) * 16;
            const int64_t m = m0 + r;
            float x[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = 0.0f;
            if (m < m_end && k < K) {
                const uint8_t *row = p.Q + m * p.ldq;
                const float unit = ck_unit(p.S[m * p.lds + k / kCkBlock]);
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (k + e < K) x[e] = (float)(int8_t)row[k + e] * unit;
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int c = at % (CF::BN / 16) * 2 + h;
                u32x4 w;
#pragma unroll
                for (int d = 0; d < 4; ++d) w[d] = ck_pair<IT>(x[8 * h + 2 * d], x[8 * h + 2 * d + 1]);
                sB[r * CB + (c ^ wgrad_slot<CB>(r, c))] = w;
            }
        }
        __syncthreads();
        const char *const bA = reinterpret_cast<const char *>(sA);
        const char *const bB = reinterpret_cast<const char *>(sB);
#pragma unroll
        for (int ks = 0; ks < BK / 16; ++ks) {
            u32x4 fa[TM], fb[TN];
#pragma unroll
            for (int i = 0; i < TM; ++i) {
                const char *at = bA + ks * 16 * CA * 16;
                const u32x2 lo = ds_read_tr16(at + wgrad_tr_offset<CA>(lane, 0, wm * CF::WTM + 32 * i));
                const u32x2 hi = ds_read_tr16(at + wgrad_tr_offset<CA>(lane, 1, wm * CF::WTM + 32 * i));
                fa[i] = u32x4{lo[0], lo[1], hi[0], hi[1]};
            }
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const char *at = bB + ks * 16 * CB * 16;
                const u32x2 lo = ds_read_tr16(at + wgrad_tr_offset<CB>(lane, 0, wn * CF::WTN + 32 * j));
                const u32x2 hi = ds_read_tr16(at + wgrad_tr_offset<CB>(lane, 1, wn * CF::WTN + 32 * j));
                fb[j] = u32x4{lo[0], lo[1], hi[0], hi[1]};
            }
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j) acc[i][j] = mfma32_1<IT>(fb[j], fa[i], acc[i][j]);
        }
    }
    if constexpr (OUT < 0) wgrad_store_part<CF>(p.g, acc, n0, k0, tid);
    else wgrad_store<CF, OUT>(p.g, acc, n0, k0, tid);
}

// D = the parts' sums + C: four columns of a row for each thread.
template <int OUT>
__global__ void __launch_bounds__(256) wgrad_join_kernel(Params p) {
    const int64_t quads = (p.N + 3) / 4, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= p.M * quads) return;
    const int64_t size = p.M * quads * 4;
    const int row = (int)(i / quads), col = (int)(i - row * quads) * 4;
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    int s = 0;
    for (; s + 8 <= p.splits; s += 8) {
        f32x4 w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = *reinterpret_cast<const f32x4 *>(p.ws + (s + e) * size + 4 * i);
#pragma unroll
        for (int e = 0; e < 8; ++e) v += w[e];
    }
#pragma unroll 4
    for (; s < p.splits; ++s) v += *reinterpret_cast<const f32x4 *>(p.ws + s * size + 4 * i);
    if (p.cd_vec && col + 4 <= p.N) finish4<OUT, true, false>(p, row, col, v);
    else finish4<OUT, false, false>(p, row, col, v);
}

}  // namespace libgemm

using namespace libgemm;
using namespace libgemm_host;

namespace {

// Inputs' type, D's type (or a part's sums), tile -> kernel.
template <int IT, int OUT>
const void *wgrad_of(const WgradPlan &plan, bool vec, unsigned *threads) {
    *threads = 256;
    if (!vec) return (const void *)wgrad_any_kernel<IT, OUT>;
    if (plan.bm == 128) return (const void *)wgrad_tile_kernel<CfgMedium, IT, OUT>;
    *threads = 512;
    static_assert(CfgMedium::THREADS == 256 && CfgLarge8::THREADS == 512 && 64 * kThinWaves == 512, "threads");
    if (plan.bm == 256) return (const void *)wgrad_tile_kernel<CfgLarge8, IT, OUT>;
    return plan.bm == 32 ? (const void *)wgrad_thin_kernel<IT, 1> : (const void *)wgrad_thin_kernel<IT, 2>;
}
template <int IT>
const void *wgrad_of(const WgradPlan &plan, bool vec, int out_dtype, unsigned *threads) {
    if (plan.splits > 1) return wgrad_of<IT, -1>(plan, vec, threads);
    return out_dtype == GEMM_F32   ? wgrad_of<IT, DT_F32>(plan, vec, threads)
           : out_dtype == GEMM_F16 ? wgrad_of<IT, DT_F16>(plan, vec, threads)
                                   : wgrad_of<IT, DT_BF16>(plan, vec, threads);
}

template <int OUT>
hipError_t launch_join(Params &p, hipStream_t s) {
    void *args[] = {&p};
    return hipLaunchKernel((const void *)wgrad_join_kernel<OUT>,
                           dim3((unsigned)cdiv(p.M * cdiv(p.N, 4), 256)), dim3(256), args, 0, s);
}

}  // namespace

extern "C" {

int gemm_validate_checkpoint_wgrad(int64_t M, int64_t N, int64_t K, const void *G, int64_t ldg,
                                   const void *Q, int64_t ldq, const uint8_t *S, int64_t lds,
                                   const void *C, int64_t ldc, const void *D, int64_t ldd,
                                   int in_dtype, int out_dtype, const void *workspace,
                                   int64_t workspace_bytes) {
    return validate_checkpoint_wgrad(M, N, K, G, ldg, Q, ldq, S, lds, C, ldc, D, ldd, in_dtype,
                                     out_dtype, workspace, workspace_bytes);
}

int64_t gemm_checkpoint_wgrad_workspace(int64_t M, int64_t N, int64_t K) {
    return checkpoint_wgrad_workspace(M, N, K);
}

int gemm_checkpoint_wgrad(int64_t M, int64_t N, int64_t K, const void *G, int64_t ldg,
                          const void *Q, int64_t ldq, const uint8_t *S, int64_t lds,
                          const void *C, int64_t ldc, void *D, int64_t ldd, int in_dtype,
                          int out_dtype, void *workspace, int64_t workspace_bytes, void *stream) {
    const int st = validate_checkpoint_wgrad(M, N, K, G, ldg, Q, ldq, S, lds, C, ldc, D, ldd,
                                             in_dtype, out_dtype, workspace, workspace_bytes);
    if (st != GEMM_OK) return st;
    if (N == 0 || K == 0) return GEMM_OK;
    WgradPlan plan = wgrad_plan(M, N, K);
    // 32-bit offsets in 64 lines; the tiles take 64 tokens at least
    const bool vec = M >= 64 && (uintptr_t)G % 16 == 0 && (uintptr_t)Q % 16 == 0 && ldg % 8 == 0 &&
                     ldq % 16 == 0 && ldg <= (1 << 24) && ldq <= (1 << 25) && lds <= (1 << 25);
    if (!vec) plan.bm = kWgAnyBM, plan.bn = kWgAnyBN;
    const int osz = out_size(out_dtype);
    WgradParams p{};
    Params &g = p.g;
    g.lda = ldg;
    g.ldc = C ? ldc : 0;
    g.ldd = ldd;
    g.K = (int)M;
    g.out_dtype = out_dtype;
    g.splits = (int)plan.splits;
    g.k_per_split = (int)(plan.per < M ? plan.per : M);  // (per may be 2^31)
    // groups of four elements in C and D's rows
    g.cd_vec = (uintptr_t)D % (4 * osz) == 0 && ldd % 4 == 0 &&
               (!C || ((uintptr_t)C % (4 * osz) == 0 && ldc % 4 == 0));
    g.group_m = 4;
    g.xcds = topology().xcds;
    if (g.splits > 1)
        g.ws = reinterpret_cast<float *>(((uintptr_t)workspace + 255) & ~(uintptr_t)255);
    p.ldq = ldq;
    p.lds = lds;
    hipStream_t s = static_cast<hipStream_t>(stream);
    unsigned threads = 256;
    const void *k = in_dtype == GEMM_BF16 ? wgrad_of<IT_BF16>(plan, vec, out_dtype, &threads)
                                          : wgrad_of<IT_F16>(plan, vec, out_dtype, &threads);
    // a grid holds fewer than 2^32 threads: at most 2^27 rows and columns of D for each launch
    const int64_t most = (int64_t)1 << 27;
    for (int64_t i = 0; i < N; i += most) {
        for (int64_t j = 0; j < K; j += most) {
            g.M = (int)(N - i < most ? N - i : most);
            g.N = (int)(K - j < most ? K - j : most);
            g.A = static_cast<const uint16_t *>(G) + i;
            g.C = C ? static_cast<const char *>(C) + (i * ldc + j) * osz : nullptr;
            g.D = static_cast<char *>(D) + (i * ldd + j) * osz;
            p.Q = static_cast<const uint8_t *>(Q) + j;
            p.S = S + j / kCkBlock;
            g.tiles_m = (int)cdiv(g.M, plan.bm);
            g.tiles_n = (int)cdiv(g.N, plan.bn);
            void *args[] = {&p};
            hipError_t e = hipLaunchKernel(k, dim3((unsigned)(g.tiles_m * g.tiles_n), 1, (unsigned)g.splits),
                                           dim3(threads), args, 0, s);
            if (e == hipSuccess && g.splits > 1)
                e = out_dtype == GEMM_F32   ? launch_join<DT_F32>(g, s)
                    : out_dtype == GEMM_F16 ? launch_join<DT_F16>(g, s)
                                            : launch_join<DT_BF16>(g, s);
            if (e != hipSuccess) return GEMM_ERR_HIP;
        }
    }
    return GEMM_OK;
}

}  // extern "C"
