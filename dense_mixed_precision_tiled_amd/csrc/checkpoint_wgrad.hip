// gemm_checkpoint_wgrad: D = G^T X^ + C, a linear layer's weight gradient from packed
// activations (checkpoint.hpp).
//
//   D(n,k) = sum_m G(m,n) X^(m,k),   X^(m,k) = 2^(S(m,k/32) - 133) Q(m,k)
//
// A product whose reduction runs over the tokens m.  The scales belong to a token and a
// block of columns, so they cannot be applied to finished sums: Q is widened to the
// matrix units' 16-bit type on its way into LDS, where a 16-byte load holds 16 values of
// one block.  That is exact (seven bits and a power of two), and so are the products.
//
// Both operands are contiguous along the output (n, k), not along m; LDS keeps them as
// they are, one row for each token, and the transposing LDS reads hand the MFMA its
// values along m.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/libgemm.h"
#include "checkpoint.hpp"
#include "gemm_host.hpp"
#include "gemm_validate.hpp"

namespace libgemm {

struct WgradParams {
    const uint16_t *G;
    const uint8_t *Q, *S;
    const uint8_t *C;
    uint8_t *D;
    float *parts;  // [splits][N][K] sums of the parts, or nullptr
    int64_t ldg, ldq, lds, ldc, ldd;
    int M, N, K;
    int per;       // tokens of a part, a multiple of 64
    int splits;
    int tiles_n, tiles_k;
    int64_t first;  // tile of workgroup 0
};

// Position of 16-byte chunk c of row m in an LDS tile of CH chunks (8 values each) for a
// row: the transposing reads of half a wave touch four rows at 64 bytes, which then lie
// in distinct banks.
template <int CH>
__device__ __forceinline__ int wg_swz(int m) {
    if constexpr (CH >= 16) return swz_rc(m, 32);
    else if constexpr (CH == 8) return ((m >> 1) & 1) << 2;
    else return 0;
}
template <int CH>
__device__ __forceinline__ int wg_tr_offset(int lane, int half, int r0) {
    const int g = lane / 16, f = (lane % 16) / 4, q = lane % 4;
    const int m = 8 * (g / 2) + 4 * half + f, r = r0 + 16 * (g % 2) + 4 * q;
    return (m * CH + ((r / 8) ^ wg_swz<CH>(m))) * 16 + (r % 8) * 2;
}

template <int OUT>
__device__ __forceinline__ float wg_load(const uint8_t *p, int64_t at) {
    if constexpr (OUT == DT_F32) return reinterpret_cast<const float *>(p)[at];
    else return from_out16<OUT>(reinterpret_cast<const uint16_t *>(p)[at]);
}
template <int OUT>
__device__ __forceinline__ void wg_store(uint8_t *p, int64_t at, float v) {
    if constexpr (OUT == DT_F32) reinterpret_cast<float *>(p)[at] = v;
    else reinterpret_cast<uint16_t *>(p)[at] = (uint16_t)to_out16<OUT>(v, false);
}

// BM x BN tile of D (n x k), four waves, 64 tokens at a time.  OUT < 0: the sums of a part.
template <int IT, int OUT, int BM, int BN, int WM, bool VEC>
__global__ void __launch_bounds__(256) wgrad_kernel(WgradParams p) {
    constexpr int BK = 64, CA = BM / 8, CB = BN / 8;
    constexpr int WN = 4 / WM, TM = BM / WM / 32, TN = BN / WN / 32;
    constexpr int NA = BK * CA / 256, NB = BK * (BN / 16) / 256;
    __shared__ u32x4 smem[BK * (CA + CB)];
    u32x4 *const sA = smem, *const sB = smem + BK * CA;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wm = wave / WN, wn = wave % WN;
    const int64_t tile = p.first + blockIdx.x;
    const int n0 = (int)(tile / p.tiles_k) * BM, k0 = (int)(tile % p.tiles_k) * BN;
    // (64 bits: a last step may end past 2^31)
    const int64_t m_beg = (int64_t)blockIdx.z * p.per;
    const int64_t m_end = m_beg + p.per < p.M ? m_beg + p.per : p.M;
    f32x16 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = f32x16{};

    for (int64_t m0 = m_beg; m0 < m_end; m0 += BK) {
        u32x4 a[NA], q[NB];
        float unit[NB];
#pragma unroll
        for (int i = 0; i < NA; ++i) {
            const int at = i * 256 + tid, n = n0 + at % CA * 8;
            const int64_t m = m0 + at / CA;
            const uint16_t *row = p.G + m * p.ldg;
            a[i] = u32x4{0u, 0u, 0u, 0u};
            if (m < m_end) {
                if constexpr (VEC) {
                    if (n < p.N) a[i] = *reinterpret_cast<const u32x4 *>(row + n);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (n + e < p.N) a[i][e / 2] |= (uint32_t)row[n + e] << (16 * (e % 2));
                }
            }
        }
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int at = i * 256 + tid, k = k0 + at % (BN / 16) * 16;
            const int64_t m = m0 + at / (BN / 16);
            const uint8_t *row = p.Q + m * p.ldq;
            q[i] = u32x4{0u, 0u, 0u, 0u};
            unit[i] = 0.0f;
            if (m < m_end && k < p.K) {
                unit[i] = ck_unit(p.S[m * p.lds + k / kCkBlock]);
                if constexpr (VEC) {
                    q[i] = *reinterpret_cast<const u32x4 *>(row + k);
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        if (k + e < p.K) q[i][e / 4] |= (uint32_t)row[k + e] << (8 * (e % 4));
                }
            }
        }
        __syncthreads();  // the last step's reads are done
#pragma unroll
        for (int i = 0; i < NA; ++i) {
            const int at = i * 256 + tid, m = at / CA;
            sA[m * CA + ((at % CA) ^ wg_swz<CA>(m))] = a[i];
        }
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int at = i * 256 + tid, m = at / (BN / 16), c = at % (BN / 16) * 2;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                u32x4 w;
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                    const int e = 8 * h + 2 * d;
                    w[d] = ck_pair<IT>(ck_int(q[i][e / 4], e % 4) * unit[i],
                                       ck_int(q[i][e / 4], e % 4 + 1) * unit[i]);
                }
                sB[m * CB + ((c + h) ^ wg_swz<CB>(m))] = w;
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
                const int r = wm * (BM / WM) + 32 * i;
                const u32x2 lo = ds_read_tr16(bA + wg_tr_offset<CA>(lane, 0, r) + ks * 16 * CA * 16);
                const u32x2 hi = ds_read_tr16(bA + wg_tr_offset<CA>(lane, 1, r) + ks * 16 * CA * 16);
                fa[i] = u32x4{lo[0], lo[1], hi[0], hi[1]};
            }
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const int r = wn * (BN / WN) + 32 * j;
                const u32x2 lo = ds_read_tr16(bB + wg_tr_offset<CB>(lane, 0, r) + ks * 16 * CB * 16);
                const u32x2 hi = ds_read_tr16(bB + wg_tr_offset<CB>(lane, 1, r) + ks * 16 * CB * 16);
                fb[j] = u32x4{lo[0], lo[1], hi[0], hi[1]};
            }
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j) acc[i][j] = mfma32_1<IT>(fa[i], fb[j], acc[i][j]);
        }
    }
    // lane l holds column l % 32, rows 8 (r / 4) + 4 (l / 32) + r % 4 of a 32 x 32 tile
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int n = n0 + wm * (BM / WM) + 32 * i + 8 * (r / 4) + 4 * (lane / 32) + r % 4;
                const int k = k0 + wn * (BN / WN) + 32 * j + lane % 32;
                if (n >= p.N || k >= p.K) continue;
                const float v = acc[i][j][r];
                if constexpr (OUT < 0)
                    p.parts[((int64_t)blockIdx.z * p.N + n) * p.K + k] = v;
                else
                    wg_store<OUT>(p.D, n * p.ldd + k,
                                  p.C ? v + wg_load<OUT>(p.C, n * p.ldc + k) : v);
            }
}

// D = the sum of the parts + C, one element for each thread.
template <int OUT>
__global__ void __launch_bounds__(256) wgrad_join_kernel(WgradParams p) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, size = (int64_t)p.N * p.K;
    if (i >= size) return;
    float v = 0.0f;
    for (int s = 0; s < p.splits; ++s) v += p.parts[s * size + i];
    const int64_t n = i / p.K, k = i - n * p.K;
    wg_store<OUT>(p.D, n * p.ldd + k, p.C ? v + wg_load<OUT>(p.C, n * p.ldc + k) : v);
}

}  // namespace libgemm

using namespace libgemm;
using namespace libgemm_host;

namespace {

template <int IT, int OUT, int BM, int BN, int WM>
const void *wgrad_of(bool vec) {
    return vec ? (const void *)wgrad_kernel<IT, OUT, BM, BN, WM, true>
               : (const void *)wgrad_kernel<IT, OUT, BM, BN, WM, false>;
}

template <int OUT>
hipError_t launch_wgrad(WgradParams p, const WgradPlan &plan, bool bf16, bool vec, hipStream_t s) {
    const int64_t tiles = (int64_t)p.tiles_n * p.tiles_k, most = (int64_t)1 << 22;
    const bool small = plan.bm == 32;
    for (int64_t t = 0; t < tiles; t += most) {
        p.first = t;
        void *args[] = {&p};
        const unsigned n = (unsigned)(tiles - t < most ? tiles - t : most);
        const void *k;
        if (p.splits > 1)
            k = small ? (bf16 ? wgrad_of<IT_BF16, -1, 32, 128, 1>(vec) : wgrad_of<IT_F16, -1, 32, 128, 1>(vec))
                      : (bf16 ? wgrad_of<IT_BF16, -1, 128, 128, 2>(vec) : wgrad_of<IT_F16, -1, 128, 128, 2>(vec));
        else
            k = small ? (bf16 ? wgrad_of<IT_BF16, OUT, 32, 128, 1>(vec) : wgrad_of<IT_F16, OUT, 32, 128, 1>(vec))
                      : (bf16 ? wgrad_of<IT_BF16, OUT, 128, 128, 2>(vec) : wgrad_of<IT_F16, OUT, 128, 128, 2>(vec));
        const hipError_t e = hipLaunchKernel(k, dim3(n, 1, (unsigned)p.splits), dim3(256), args, 0, s);
        if (e != hipSuccess) return e;
    }
    if (p.splits > 1) {
        void *args[] = {&p};
        return hipLaunchKernel((const void *)wgrad_join_kernel<OUT>,
                               dim3((unsigned)cdiv((int64_t)p.N * p.K, 256)), dim3(256), args, 0, s);
    }
    return hipSuccess;
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
    const WgradPlan plan = wgrad_plan(M, N, K);
    WgradParams p{};
    p.G = static_cast<const uint16_t *>(G);
    p.Q = static_cast<const uint8_t *>(Q);
    p.S = S;
    p.C = static_cast<const uint8_t *>(C);
    p.D = static_cast<uint8_t *>(D);
    p.ldg = ldg;
    p.ldq = ldq;
    p.lds = lds;
    p.ldc = ldc;
    p.ldd = ldd;
    p.M = (int)M;
    p.N = (int)N;
    p.K = (int)K;
    p.per = (int)plan.per;
    p.splits = (int)plan.splits;
    p.tiles_n = (int)cdiv(N, plan.bm);
    p.tiles_k = (int)cdiv(K, plan.bn);
    if (p.splits > 1)
        p.parts = reinterpret_cast<float *>(((uintptr_t)workspace + 255) & ~(uintptr_t)255);
    const bool vec = (uintptr_t)G % 16 == 0 && (uintptr_t)Q % 16 == 0 && ldg % 8 == 0 && ldq % 16 == 0;
    const bool bf16 = in_dtype == GEMM_BF16;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const hipError_t e = out_dtype == GEMM_F32   ? launch_wgrad<DT_F32>(p, plan, bf16, vec, s)
                         : out_dtype == GEMM_F16 ? launch_wgrad<DT_F16>(p, plan, bf16, vec, s)
                                                 : launch_wgrad<DT_BF16>(p, plan, bf16, vec, s);
    return e == hipSuccess ? GEMM_OK : GEMM_ERR_HIP;
}

}  // extern "C"
