// gemm_run_scaled: int8 products with a scale for each row and column.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <utility>

#include "../../include/libgemm.h"
#include "gemm_configs.hpp"
#include "gemm_host.hpp"
#include "gemm_validate.hpp"

using namespace libgemm;
using namespace libgemm_host;

namespace {

constexpr int64_t range = ((int64_t)1 << 32) - 256;  // of a buffer

int flip(int layout) { return layout == GEMM_ROW_MAJOR ? GEMM_COL_MAJOR : GEMM_ROW_MAJOR; }

// One launch.  aligned: the operands' lines allow 16-byte loads.
int run_part(Params &p, bool aligned, int akc, int bkc, int cus, int osz, hipStream_t stream) {
    const int64_t M = p.M, N = p.N, K = p.K;
    auto status = [](hipError_t e) { return e == hipSuccess ? GEMM_OK : GEMM_ERR_HIP; };
    // vector loads: extents, rounded up to 16 bytes, that fit a 32-bit buffer range (so
    // do the 127 bytes that a last K-tile may reach past them)
    const int64_t a_ext = akc ? (M - 1) * p.lda + K : (K - 1) * p.lda + M;
    const int64_t b_ext = bkc ? (N - 1) * p.ldb + K : (K - 1) * p.ldb + N;
    const int64_t a_rng = (a_ext + 15) & ~(int64_t)15, b_rng = (b_ext + 15) & ~(int64_t)15;
    p.vec_ok = aligned && a_rng < range && b_rng < range;
    p.a_bytes = p.vec_ok ? (uint32_t)a_rng : 0u;
    p.b_bytes = p.vec_ok ? (uint32_t)b_rng : 0u;
    // four outputs of a row in one store
    p.cd_vec = (uintptr_t)p.D % (4 * osz) == 0 && p.ldd % 4 == 0;
    p.group_m = 4;
    if (akc && bkc && aligned) {
        // (row offsets of the streaming kernels are 32 bits: 32 rows of A and B)
        if (M <= 32 && p.lda <= (1 << 26) && p.ldb <= (1 << 26))
            return status(launch_scaled_stream(p, cus, stream));
        hipError_t e;
        if (launch_scaled_pipe(p, cus, stream, &e)) return status(e);
    }
    // the int8 shape classes of gemm_run (without its split along K)
    int bm, bk;
    launch_fn launch;
    if (cdiv(M, 256) * cdiv(N, 256) >= 3 * cus / 4) {
        bm = 256, bk = CfgLarge8I8::BK;
        // (a ragged K on the four-wave tile: 77.5 us at 3999 x 4001 x 4104 against 75.7)
        launch = p.vec_ok && akc && bkc && K % CfgLargeDmaI8_16::BK == 0 ? launch_large_dma16_i8s
                                                                         : launch_large8_i8s;
    } else if (cdiv(M, 128) * cdiv(N, 128) >= cus / 2) {
        bm = 128, bk = CfgMediumI8::BK;
        launch = launch_medium_i8s;
    } else {
        bm = 64, bk = CfgSmallI8::BK;
        launch = launch_small_i8s;
    }
    p.tiles_m = (int)cdiv(M, bm);
    p.tiles_n = (int)cdiv(N, bm);
    const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n;
    if (tiles > 0x7fffffff) return GEMM_ERR_INVALID_DIM;
    // the raster of gemm_run: groups of 4 tile-rows, or 2 staggered ones where
    // each CU runs several large tiles with a short K loop
    const bool short_multi = bm == 256 && tiles > cus && K <= 2048;
    p.group_m = short_multi ? 2 : 4;
    p.skew = short_multi ? 1 : 0;
    p.k_per_split = (int)(cdiv(K > 0 ? K : 1, bk) * bk);
    return status(launch(p, 0, akc, bkc, dim3((unsigned)tiles), stream));
}

}  // namespace

extern "C" {

int gemm_validate_scaled(int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, int layoutA,
                         const void *B, int64_t ldb, int layoutB, const float *scaleA,
                         const float *scaleB, const void *C, int64_t ldc, const void *D,
                         int64_t ldd, int in_dtype, int acc_dtype, int out_dtype,
                         const gemm_epilogue_t *epi) {
    return validate_scaled(M, N, K, A, lda, layoutA, B, ldb, layoutB, scaleA, scaleB, C, ldc, D,
                           ldd, in_dtype, acc_dtype, out_dtype, epi);
}

int gemm_run_scaled(int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, int layoutA,
                    const void *B, int64_t ldb, int layoutB, const float *scaleA,
                    const float *scaleB, const void *C, int64_t ldc, void *D, int64_t ldd,
                    int in_dtype, int acc_dtype, int out_dtype, int satf,
                    const gemm_epilogue_t *epi_arg, void *stream_handle) {
    const int st = validate_scaled(M, N, K, A, lda, layoutA, B, ldb, layoutB, scaleA, scaleB, C,
                                   ldc, D, ldd, in_dtype, acc_dtype, out_dtype, epi_arg);
    if (st != GEMM_OK) return st;
    if (M == 0 || N == 0) return GEMM_OK;
    const gemm_epilogue_t epi = epi_arg ? *epi_arg : kPlainEpilogue;
    if (epi.beta == 0.0f) C = nullptr;  // beta == 0: C is not read
    if (K == 0) scaleA = scaleB = nullptr;  // no product: nothing to scale
    int layoutC = epi.layoutC;
    const bool swap = epi.layoutD == GEMM_COL_MAJOR;
    if (swap) {
        // a column-major D is the row-major N x M matrix D^T = B^T x A^T
        std::swap(A, B);
        std::swap(lda, ldb);
        std::swap(layoutA, layoutB);
        layoutA = flip(layoutA);
        layoutB = flip(layoutB);
        std::swap(M, N);
        std::swap(scaleA, scaleB);
        layoutC = flip(layoutC);
    }
    const Topology topo = topology();
    hipStream_t stream = static_cast<hipStream_t>(stream_handle);

    Params p{};
    p.C = C;
    p.lda = lda;
    p.ldb = ldb;
    p.ldc = C ? ldc : 0;
    p.ldd = ldd;
    p.K = (int)K;
    p.out_dtype = out_dtype;
    p.satf = satf ? 1 : 0;
    p.c_col = (C && layoutC == GEMM_COL_MAJOR) ? 1 : 0;
    p.epi = 1;
    p.alpha = epi.alpha;
    p.beta = epi.beta;
    p.bias = epi.bias;
    p.bias_rows = swap ? 1 : 0;
    p.act = epi.activation;
    p.row_scale = scaleA;
    p.col_scale = scaleB;
    p.splits = 1;
    p.xcds = topo.xcds;
    const int akc = layoutA == GEMM_ROW_MAJOR, bkc = layoutB == GEMM_COL_MAJOR;
    const bool aligned = K > 0 && (uintptr_t)A % 16 == 0 && (uintptr_t)B % 16 == 0 &&
                         lda % 16 == 0 && ldb % 16 == 0;
    // Buffer loads reach 4 GiB: K-contiguous operands past that are taken in
    // parts, rows of D by the extent of A and columns by that of B.  A part has at
    // most 2^27 rows and columns (a grid holds fewer than 2^32 threads, a tile's
    // last row an int).
    const bool parts = aligned && akc && bkc && lda <= range / 512 && ldb <= range / 512;
    const int64_t most = (int64_t)1 << 27;
    int64_t rows = M < most ? M : most, cols = N < most ? N : most;
    if (parts && (rows - 1) * lda + K > range) rows = (range - K) / lda / 256 * 256;
    if (parts && (cols - 1) * ldb + K > range) cols = (range - K) / ldb / 256 * 256;
    const int64_t a_row = akc ? lda : 1, b_col = bkc ? ldb : 1;
    const int osz = out_size(out_dtype);
    for (int64_t i = 0; i < M; i += rows) {
        for (int64_t j = 0; j < N; j += cols) {
            Params q = p;
            q.M = (int)(M - i < rows ? M - i : rows);
            q.N = (int)(N - j < cols ? N - j : cols);
            q.A = reinterpret_cast<const uint16_t *>(static_cast<const char *>(A) + i * a_row);
            q.B = reinterpret_cast<const uint16_t *>(static_cast<const char *>(B) + j * b_col);
            if (C)
                q.C = static_cast<const char *>(C) +
                      (p.c_col ? j * p.ldc + i : i * p.ldc + j) * osz;
            q.D = static_cast<char *>(D) + (i * ldd + j) * osz;
            if (p.bias) q.bias = p.bias + (p.bias_rows ? i : j);
            if (p.row_scale) q.row_scale = p.row_scale + i;
            if (p.col_scale) q.col_scale = p.col_scale + j;
            const int r = run_part(q, aligned, akc, bkc, topo.cus, osz, stream);
            if (r != GEMM_OK) return r;
        }
    }
    return GEMM_OK;
}

}  // extern "C"
