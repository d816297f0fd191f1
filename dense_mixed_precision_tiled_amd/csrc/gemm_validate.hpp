// Host-side argument validation of the C ABI (no HIP: the same code builds
// with a plain C++ compiler for the sanitizer test).  The checks follow the
// boundary's contract in include/libgemm.h: dimensions, leading dimensions,
// layouts, dtype combinations, null pointers and aliasing between D and the
// other operands.
#pragma once

#include <stdint.h>

#include "../../include/libgemm.h"

namespace libgemm_host {

inline bool is_fp8(int in_dtype) { return in_dtype == GEMM_FP8_E4M3 || in_dtype == GEMM_FP8_E5M2; }
inline int input_class(int in_dtype) { return in_dtype == GEMM_I8 ? 1 : (is_fp8(in_dtype) ? 2 : 0); }
inline int in_size(int in_dtype) { return (in_dtype == GEMM_I8 || is_fp8(in_dtype)) ? 1 : 2; }

inline int out_size(int dt) { return (dt == GEMM_F32 || dt == GEMM_I32) ? 4 : 2; }

// Byte range [lo, hi) of a matrix with `outer` lines of `inner` elements at
// stride ld; empty when either count is zero.
struct Range {
    unsigned __int128 lo, hi;
    bool empty() const { return hi <= lo; }
};

inline Range extent(const void *p, int64_t outer, int64_t inner, int64_t ld, int esize) {
    Range r;
    r.lo = (unsigned __int128)(uintptr_t)p;
    if (outer <= 0 || inner <= 0) {
        r.hi = r.lo;
        return r;
    }
    r.hi = r.lo + ((unsigned __int128)(outer - 1) * (unsigned __int128)ld +
                   (unsigned __int128)inner) * (unsigned __int128)esize;
    return r;
}

inline bool overlap(const Range &a, const Range &b) {
    return !a.empty() && !b.empty() && a.lo < b.hi && b.lo < a.hi;
}

inline const gemm_epilogue_t kPlainEpilogue = {1.0f, 1.0f, nullptr, GEMM_ACT_NONE, GEMM_ROW_MAJOR,
                                         GEMM_ROW_MAJOR};

inline int validate(int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, int layoutA,
             const void *B, int64_t ldb, int layoutB, const void *C, int64_t ldc, const void *D,
             int64_t ldd, int in_dtype, int acc_dtype, int out_dtype,
             const gemm_epilogue_t *epi, int satf_arg) {
    if (!epi) epi = &kPlainEpilogue;
    const int64_t kMaxDim = 0x7fffffff;
    if (M < 0 || N < 0 || K < 0 || M > kMaxDim || N > kMaxDim || K > kMaxDim)
        return GEMM_ERR_INVALID_DIM;
    if (in_dtype == GEMM_I8 && acc_dtype == GEMM_I32 && out_dtype == GEMM_I32 && satf_arg &&
        K >= ((int64_t)1 << 17))
        return GEMM_ERR_UNSUPPORTED;
    auto layout_ok = [](int l) { return l == GEMM_ROW_MAJOR || l == GEMM_COL_MAJOR; };
    if (!layout_ok(layoutA) || !layout_ok(layoutB) || !layout_ok(epi->layoutC) ||
        !layout_ok(epi->layoutD))
        return GEMM_ERR_INVALID_LAYOUT;
    if (in_dtype != GEMM_F16 && in_dtype != GEMM_BF16 && in_dtype != GEMM_I8 && !is_fp8(in_dtype))
        return GEMM_ERR_UNSUPPORTED;
    if (in_dtype == GEMM_I8) {
        // int8 x int8 -> int32: the plain epilogue only (C/D layouts allowed);
        // satf clamps the exact sum, which the int32 accumulator holds only
        // for K < 2^17 (|a*b| <= 2^14)
        if (acc_dtype != GEMM_I32 || out_dtype != GEMM_I32) return GEMM_ERR_UNSUPPORTED;
        if (epi->alpha != 1.0f || (C && epi->beta != 1.0f && epi->beta != 0.0f) || epi->bias ||
            epi->activation != GEMM_ACT_NONE)
            return GEMM_ERR_UNSUPPORTED;
    } else if (acc_dtype == GEMM_F32) {
        if (out_dtype != GEMM_F32 && out_dtype != GEMM_F16 && out_dtype != GEMM_BF16)
            return GEMM_ERR_UNSUPPORTED;
    } else if (acc_dtype == GEMM_F16) {
        if (in_dtype != GEMM_F16 || out_dtype != GEMM_F16) return GEMM_ERR_UNSUPPORTED;
    } else {
        return GEMM_ERR_UNSUPPORTED;
    }
    if (epi->activation != GEMM_ACT_NONE && epi->activation != GEMM_ACT_RELU &&
        epi->activation != GEMM_ACT_GELU)
        return GEMM_ERR_UNSUPPORTED;
    const int64_t a_inner = layoutA == GEMM_ROW_MAJOR ? K : M;
    const int64_t a_outer = layoutA == GEMM_ROW_MAJOR ? M : K;
    const int64_t b_inner = layoutB == GEMM_ROW_MAJOR ? N : K;
    const int64_t b_outer = layoutB == GEMM_ROW_MAJOR ? K : N;
    const int64_t c_inner = epi->layoutC == GEMM_ROW_MAJOR ? N : M;
    const int64_t c_outer = epi->layoutC == GEMM_ROW_MAJOR ? M : N;
    const int64_t d_inner = epi->layoutD == GEMM_ROW_MAJOR ? N : M;
    const int64_t d_outer = epi->layoutD == GEMM_ROW_MAJOR ? M : N;
    // C is read only when present and beta != 0
    const bool reads_c = C && epi->beta != 0.0f;
    // leading dimensions: at least one line's worth, and small enough that
    // every element offset fits in 62 bits
    const int64_t kMaxLd = (int64_t)1 << 40;
    if (lda < 1 || lda < a_inner || lda > kMaxLd) return GEMM_ERR_INVALID_LD;
    if (ldb < 1 || ldb < b_inner || ldb > kMaxLd) return GEMM_ERR_INVALID_LD;
    if (ldd < 1 || ldd < d_inner || ldd > kMaxLd) return GEMM_ERR_INVALID_LD;
    if (reads_c && (ldc < 1 || ldc < c_inner || ldc > kMaxLd)) return GEMM_ERR_INVALID_LD;
    if (M == 0 || N == 0) return GEMM_OK;
    if (!D) return GEMM_ERR_NULL_PTR;
    if (K > 0 && (!A || !B)) return GEMM_ERR_NULL_PTR;

    const int osz = out_size(out_dtype);
    const Range rd = extent(D, d_outer, d_inner, ldd, osz);
    const int isz = in_size(in_dtype);
    const Range ra = K > 0 ? extent(A, a_outer, a_inner, lda, isz) : extent(A, 0, 0, 1, isz);
    const Range rb = K > 0 ? extent(B, b_outer, b_inner, ldb, isz) : extent(B, 0, 0, 1, isz);
    if (overlap(rd, ra) || overlap(rd, rb)) return GEMM_ERR_ALIASING;
    if (epi->bias && overlap(extent(epi->bias, 1, N, N, 4), rd)) return GEMM_ERR_ALIASING;
    if (reads_c) {
        const bool in_place = (C == D) && (ldc == ldd) && (epi->layoutC == epi->layoutD);
        if (!in_place && overlap(extent(C, c_outer, c_inner, ldc, osz), rd))
            return GEMM_ERR_ALIASING;
    }
    return GEMM_OK;
}

// gemm_run_scaled: the dtypes and K first, then the checks of a product of
// 8-bit values with float outputs (those of an fp8 product of these sizes),
// then the scales.
inline int validate_scaled(int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, int layoutA,
                           const void *B, int64_t ldb, int layoutB, const float *scaleA,
                           const float *scaleB, const void *C, int64_t ldc, const void *D,
                           int64_t ldd, int in_dtype, int acc_dtype, int out_dtype,
                           const gemm_epilogue_t *epi) {
    if (in_dtype != GEMM_I8 || acc_dtype != GEMM_I32) return GEMM_ERR_UNSUPPORTED;
    const int st = validate(M, N, K, A, lda, layoutA, B, ldb, layoutB, C, ldc, D, ldd,
                            GEMM_FP8_E4M3, GEMM_F32, out_dtype, epi, 0);
    if (st != GEMM_OK) return st;
    if (K >= ((int64_t)1 << 17)) return GEMM_ERR_UNSUPPORTED;
    if (M == 0 || N == 0) return GEMM_OK;
    if (!epi) epi = &kPlainEpilogue;
    const bool row = epi->layoutD == GEMM_ROW_MAJOR;
    const Range rd = extent(D, row ? M : N, row ? N : M, ldd, out_size(out_dtype));
    if (scaleA && overlap(extent(scaleA, 1, M, M, 4), rd)) return GEMM_ERR_ALIASING;
    if (scaleB && overlap(extent(scaleB, 1, N, N, 4), rd)) return GEMM_ERR_ALIASING;
    return GEMM_OK;
}

inline int validate_quantize_rows(int64_t M, int64_t K, const void *X, int64_t ldx, int in_dtype,
                                  const void *Q, int64_t ldq, const float *scales) {
    const int64_t kMaxDim = 0x7fffffff, kMaxLd = (int64_t)1 << 40;
    if (M < 0 || K < 0 || M > kMaxDim || K > kMaxDim) return GEMM_ERR_INVALID_DIM;
    if (in_dtype != GEMM_F16 && in_dtype != GEMM_BF16 && in_dtype != GEMM_F32)
        return GEMM_ERR_UNSUPPORTED;
    if (ldx < 1 || ldx < K || ldx > kMaxLd) return GEMM_ERR_INVALID_LD;
    if (ldq < 1 || ldq < K || ldq > kMaxLd) return GEMM_ERR_INVALID_LD;
    if (M == 0) return GEMM_OK;
    if (!scales || (K > 0 && (!X || !Q))) return GEMM_ERR_NULL_PTR;
    const Range rx = extent(X, K > 0 ? M : 0, K, ldx, in_dtype == GEMM_F32 ? 4 : 2);
    const Range rq = extent(Q, K > 0 ? M : 0, K, ldq, 1);
    const Range rs = extent(scales, 1, M, M, 4);
    if (overlap(rx, rq) || overlap(rx, rs) || overlap(rq, rs)) return GEMM_ERR_ALIASING;
    return GEMM_OK;
}

// The layer's dimensions, and the workspace they need.
inline int validate_moe_dims(int64_t T, const gemm_moe_t *m) {
    if (!m) return GEMM_ERR_NULL_PTR;
    const int64_t kMaxWidth = (int64_t)1 << 19;
    if (T < 0 || m->H < 1 || m->I < 1 || m->H > kMaxWidth || m->I > kMaxWidth || m->E < 1 ||
        m->topk < 1 || m->topk > m->E)
        return GEMM_ERR_INVALID_DIM;
    if (T > 64 || m->E > 1024 || m->topk > 32) return GEMM_ERR_UNSUPPORTED;
    return GEMM_OK;
}

// Offsets of the parts of the workspace, from its start rounded up to 256 bytes.
struct MoeWorkspace {
    int64_t slots, ldh;
    int64_t count, expert, pairs, weight, h, bytes;
};

inline MoeWorkspace moe_workspace(int64_t T, const gemm_moe_t *m) {
    MoeWorkspace w;
    const int64_t npairs = T * m->topk;
    w.slots = m->E < npairs ? m->E : npairs;
    w.ldh = (m->I + 7) / 8 * 8;  // rows of whole 16 bytes
    w.count = 0;
    w.expert = w.count + 4 * w.slots;
    w.pairs = w.expert + 4 * w.slots;
    w.weight = w.pairs + 4 * w.slots * T;
    w.h = (w.weight + 4 * npairs + 255) / 256 * 256;
    w.bytes = w.h + 2 * 2 * npairs * w.ldh + 255;  // two parts of 16-bit values
    return w;
}

inline int validate_moe(int64_t T, const gemm_moe_t *m, const void *X, int64_t ldx,
                        const float *logits, int64_t ldl, const void *D, int64_t ldd, int in_dtype,
                        const void *workspace, int64_t workspace_bytes) {
    const int st = validate_moe_dims(T, m);
    if (st != GEMM_OK) return st;
    if (in_dtype != GEMM_F16 && in_dtype != GEMM_BF16) return GEMM_ERR_UNSUPPORTED;
    if (m->w_dtype != in_dtype && m->w_dtype != GEMM_I8) return GEMM_ERR_UNSUPPORTED;
    if (m->activation != GEMM_ACT_SILU && m->activation != GEMM_ACT_GELU &&
        m->activation != GEMM_ACT_RELU)
        return GEMM_ERR_UNSUPPORTED;
    // (the kernels' row offsets are 32 bits: 64 rows of X, 2048 of h)
    const int64_t kMaxLd = (int64_t)1 << 24;
    auto ld_bad = [&](int64_t ld, int64_t inner) { return ld < inner || ld > kMaxLd; };
    if (ld_bad(ldx, m->H) || ld_bad(ldl, m->E) || ld_bad(ldd, m->H) || ld_bad(m->ld1, m->H) ||
        ld_bad(m->ld2, m->I))
        return GEMM_ERR_INVALID_LD;
    if (T == 0) return GEMM_OK;
    const bool i8 = m->w_dtype == GEMM_I8;
    if (!X || !logits || !D || !workspace || !m->W1 || !m->W2 ||
        (i8 && (!m->scale1 || !m->scale2)))
        return GEMM_ERR_NULL_PTR;
    const int64_t need = moe_workspace(T, m).bytes;
    if (workspace_bytes < need) return GEMM_ERR_SCRATCH_TOO_SMALL;
    const int wsz = i8 ? 1 : 2;
    const int64_t r1 = m->E * 2 * m->I, r2 = m->E * m->H;
    const Range rd = extent(D, T, m->H, ldd, 2);
    const Range rw = extent(workspace, 1, need, need, 1);
    const Range in[6] = {extent(X, T, m->H, ldx, 2),
                         extent(logits, T, m->E, ldl, 4),
                         extent(m->W1, r1, m->H, m->ld1, wsz),
                         extent(m->W2, r2, m->I, m->ld2, wsz),
                         extent(m->scale1, i8 ? 1 : 0, r1, r1, 4),
                         extent(m->scale2, i8 ? 1 : 0, r2, r2, 4)};
    if (overlap(rd, rw)) return GEMM_ERR_ALIASING;
    for (const Range &r : in)
        if (overlap(r, rd) || overlap(r, rw)) return GEMM_ERR_ALIASING;
    return GEMM_OK;
}

}  // namespace libgemm_host
