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

// The router's balance: dimensions, then what both directions read.
inline int validate_moe_balance_dims(int64_t T, int64_t E, int64_t topk) {
    if (T < 0 || T > 0x7fffffff || E < 1 || topk < 1 || topk > E) return GEMM_ERR_INVALID_DIM;
    if (E > 1024 || topk > 32) return GEMM_ERR_UNSUPPORTED;
    return GEMM_OK;
}

inline bool finite_weight(float w) { return w - w == 0.0f; }

// Parts of the workspace, from its start rounded up to 256 bytes: for each of up to
// kBalanceParts workgroups the sums of p and the counts of its tokens, by expert.
constexpr int64_t kBalanceParts = 256;
inline int64_t moe_balance_workspace(int64_t E) { return kBalanceParts * (E + 1) * 12 + 255; }

inline int validate_moe_balance(int64_t T, int64_t E, int64_t topk, const float *logits,
                                int64_t ldl, const uint8_t *mask, float balance, float z,
                                const float *loss, const int32_t *counts, const float *lse,
                                const void *workspace, int64_t workspace_bytes) {
    const int st = validate_moe_balance_dims(T, E, topk);
    if (st != GEMM_OK) return st;
    if (!finite_weight(balance) || !finite_weight(z)) return GEMM_ERR_UNSUPPORTED;
    const int64_t kMaxLd = (int64_t)1 << 40;
    if (ldl < E || ldl > kMaxLd) return GEMM_ERR_INVALID_LD;
    if (!loss || !counts || !workspace || (T > 0 && (!logits || !lse))) return GEMM_ERR_NULL_PTR;
    const int64_t need = moe_balance_workspace(E);
    if (workspace_bytes < need) return GEMM_ERR_SCRATCH_TOO_SMALL;
    const Range in[2] = {extent(logits, T, E, ldl, 4), extent(mask, mask ? 1 : 0, T, T, 1)};
    const Range out[4] = {extent(loss, 1, 3, 3, 4), extent(counts, 1, E + 1, E + 1, 4),
                          extent(lse, 1, T, T, 4), extent(workspace, 1, need, need, 1)};
    for (int i = 0; i < 4; ++i) {
        for (const Range &r : in)
            if (overlap(r, out[i])) return GEMM_ERR_ALIASING;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return GEMM_ERR_ALIASING;
    }
    return GEMM_OK;
}

inline int validate_moe_balance_grad(int64_t T, int64_t E, int64_t topk, const float *logits,
                                     int64_t ldl, const uint8_t *mask, float balance, float z,
                                     const int32_t *counts, const float *lse, const float *dloss,
                                     const void *D, int64_t ldd, int out_dtype) {
    const int st = validate_moe_balance_dims(T, E, topk);
    if (st != GEMM_OK) return st;
    if (!finite_weight(balance) || !finite_weight(z)) return GEMM_ERR_UNSUPPORTED;
    if (out_dtype != GEMM_F32 && out_dtype != GEMM_F16 && out_dtype != GEMM_BF16)
        return GEMM_ERR_UNSUPPORTED;
    const int64_t kMaxLd = (int64_t)1 << 40;
    if (ldl < E || ldl > kMaxLd || ldd < E || ldd > kMaxLd) return GEMM_ERR_INVALID_LD;
    if (T == 0) return GEMM_OK;
    if (!logits || !counts || !lse || !D) return GEMM_ERR_NULL_PTR;
    const Range rd = extent(D, T, E, ldd, out_size(out_dtype));
    const Range in[5] = {extent(logits, T, E, ldl, 4), extent(mask, mask ? 1 : 0, T, T, 1),
                         extent(counts, 1, E + 1, E + 1, 4), extent(lse, 1, T, T, 4),
                         extent(dloss, dloss ? 1 : 0, 1, 1, 4)};
    for (const Range &r : in)
        if (overlap(r, rd)) return GEMM_ERR_ALIASING;
    return GEMM_OK;
}

// Low-rank adapters: the dimensions, and the workspace they need (partial sums of
// x A^T: splits x T x rank rounded up to 8, fp32).
inline int validate_lora_dims(int64_t T, const gemm_lora_t *l) {
    if (!l) return GEMM_ERR_NULL_PTR;
    const int64_t kMaxWidth = (int64_t)1 << 19, kMaxTokens = (int64_t)1 << 20;
    if (T < 0 || l->K < 1 || l->N < 1 || l->K > kMaxWidth || l->N > kMaxWidth ||
        l->adapters < 1 || l->rank < 1)
        return GEMM_ERR_INVALID_DIM;
    if (T > kMaxTokens || l->adapters > kMaxTokens || l->rank > 256) return GEMM_ERR_UNSUPPORTED;
    return GEMM_OK;
}

// Up to this many tokens they are taken one by one and 16 at a time, else 64 and 32 (lora.hpp).
// us on 4096 x 4096 in bf16, first against second way: packed prompts of 4 adapters, 256
// tokens, rank 16 18.5 and 20.9 (257), rank 64 42 and 24; 512 tokens 24 and 15.5, 59 and 18.4.
// Tokens of 32 adapters in any order, as a decoding batch has them: 256 tokens 21 and 165, 55
// and 212; 512 tokens 33 and 164, 90 and 211.
constexpr int64_t kLoraFew = 256;
// Parts of K that different workgroups take: with few tiles of tokens there are CUs to
// spare, and an adapter's rows of A are long.
inline int64_t lora_splits(int64_t T, const gemm_lora_t *l) {
    const bool few = T <= kLoraFew;
    // (few: as many groups as tokens, at the most)
    const int64_t tiles = few ? T : (T + 63) / 64 * ((l->rank + 63) / 64);
    const int64_t most = (l->K + 511) / 512;
    int64_t s = 1;
    while (s < 4 && tiles * s < 256 && 2 * s <= most) s *= 2;
    return s;
}
// Parts of the workspace, from its start rounded up to 256 bytes: the sums of each part of
// K, and for many tokens their values of 16 bits and powers of two.
struct LoraWorkspace {
    int64_t splits, ldh;
    int64_t parts, down, bytes;
};
inline LoraWorkspace lora_workspace(int64_t T, const gemm_lora_t *l) {
    LoraWorkspace w;
    w.splits = lora_splits(T, l);
    w.ldh = (l->rank + 7) / 8 * 8;
    w.parts = (w.splits * T * w.ldh * 4 + 255) / 256 * 256;
    // (up to three values, whole 16 tokens by 32 ranks)
    w.down = w.parts + (T > kLoraFew ? 3 * ((T + 15) / 16 * 16) * ((w.ldh + 31) / 32 * 32) * 2 : 0);
    w.bytes = w.down + (T > kLoraFew ? 4 * T : 0) + 255;
    return w;
}

inline int validate_lora(int64_t T, const gemm_lora_t *l, const void *X, int64_t ldx,
                         const int32_t *ids, const void *C, int64_t ldc, const void *D,
                         int64_t ldd, int in_dtype, int out_dtype, const void *workspace,
                         int64_t workspace_bytes) {
    const int st = validate_lora_dims(T, l);
    if (st != GEMM_OK) return st;
    if (in_dtype != GEMM_F16 && in_dtype != GEMM_BF16) return GEMM_ERR_UNSUPPORTED;
    if (out_dtype != GEMM_F32 && out_dtype != GEMM_F16 && out_dtype != GEMM_BF16)
        return GEMM_ERR_UNSUPPORTED;
    const int64_t kMaxLd = (int64_t)1 << 24;
    auto ld_bad = [&](int64_t ld, int64_t inner) { return ld < inner || ld > kMaxLd; };
    if (ld_bad(ldx, l->K) || ld_bad(l->lda, l->K) || ld_bad(l->ldb, l->rank) || ld_bad(ldd, l->N) ||
        (C && ld_bad(ldc, l->N)))
        return GEMM_ERR_INVALID_LD;
    if (T == 0) return GEMM_OK;
    if (!X || !ids || !D || !workspace || !l->A || !l->B) return GEMM_ERR_NULL_PTR;
    const int64_t need = lora_workspace(T, l).bytes;
    if (workspace_bytes < need) return GEMM_ERR_SCRATCH_TOO_SMALL;
    const int osz = out_size(out_dtype);
    const int64_t n = l->adapters;
    const Range rd = extent(D, T, l->N, ldd, osz), rw = extent(workspace, 1, need, need, 1);
    const Range in[6] = {extent(X, T, l->K, ldx, 2),
                         extent(ids, 1, T, T, 4),
                         extent(l->A, n * l->rank, l->K, l->lda, 2),
                         extent(l->B, n * l->N, l->rank, l->ldb, 2),
                         extent(l->ranks, l->ranks ? 1 : 0, n, n, 4),
                         extent(l->scales, l->scales ? 1 : 0, n, n, 4)};
    if (overlap(rd, rw)) return GEMM_ERR_ALIASING;
    for (const Range &r : in)
        if (overlap(r, rd) || overlap(r, rw)) return GEMM_ERR_ALIASING;
    if (C) {
        const Range rc = extent(C, T, l->N, ldc, osz);
        if (overlap(rc, rw) || (!(C == D && ldc == ldd) && overlap(rc, rd)))
            return GEMM_ERR_ALIASING;
    }
    return GEMM_OK;
}

// Activation checkpoints: M x K values in blocks of 32 along K.
constexpr int64_t kCheckpointBlock = 32;
inline int64_t checkpoint_blocks(int64_t K) {
    return (K + kCheckpointBlock - 1) / kCheckpointBlock;
}
inline bool is_float(int dt) { return dt == GEMM_F32 || dt == GEMM_F16 || dt == GEMM_BF16; }

inline int validate_checkpoint_dims(int64_t M, int64_t K, int64_t ldq, int64_t lds) {
    const int64_t kMaxDim = 0x7fffffff, kMaxLd = (int64_t)1 << 40;
    if (M < 0 || K < 0 || M > kMaxDim || K > kMaxDim) return GEMM_ERR_INVALID_DIM;
    if (ldq < 1 || ldq < K || ldq > kMaxLd) return GEMM_ERR_INVALID_LD;
    if (lds < 1 || lds < checkpoint_blocks(K) || lds > kMaxLd) return GEMM_ERR_INVALID_LD;
    return GEMM_OK;
}
inline bool line_bad(int64_t ld, int64_t inner) {
    return ld < 1 || ld < inner || ld > ((int64_t)1 << 40);
}

inline int validate_checkpoint_pack(int64_t M, int64_t K, const void *X, int64_t ldx, int in_dtype,
                                    const void *Q, int64_t ldq, const uint8_t *S, int64_t lds) {
    const int st = validate_checkpoint_dims(M, K, ldq, lds);
    if (st != GEMM_OK) return st;
    if (!is_float(in_dtype)) return GEMM_ERR_UNSUPPORTED;
    if (line_bad(ldx, K)) return GEMM_ERR_INVALID_LD;
    if (M == 0 || K == 0) return GEMM_OK;
    if (!X || !Q || !S) return GEMM_ERR_NULL_PTR;
    const Range rx = extent(X, M, K, ldx, out_size(in_dtype)), rq = extent(Q, M, K, ldq, 1);
    const Range rs = extent(S, M, checkpoint_blocks(K), lds, 1);
    if (overlap(rx, rq) || overlap(rx, rs) || overlap(rq, rs)) return GEMM_ERR_ALIASING;
    return GEMM_OK;
}

inline int validate_checkpoint_unpack(int64_t M, int64_t K, const void *Q, int64_t ldq,
                                      const uint8_t *S, int64_t lds, const void *D, int64_t ldd,
                                      int out_dtype) {
    const int st = validate_checkpoint_dims(M, K, ldq, lds);
    if (st != GEMM_OK) return st;
    if (!is_float(out_dtype)) return GEMM_ERR_UNSUPPORTED;
    if (line_bad(ldd, K)) return GEMM_ERR_INVALID_LD;
    if (M == 0 || K == 0) return GEMM_OK;
    if (!Q || !S || !D) return GEMM_ERR_NULL_PTR;
    const Range rd = extent(D, M, K, ldd, out_size(out_dtype));
    if (overlap(rd, extent(Q, M, K, ldq, 1)) ||
        overlap(rd, extent(S, M, checkpoint_blocks(K), lds, 1)))
        return GEMM_ERR_ALIASING;
    return GEMM_OK;
}

inline int validate_checkpoint_act_grad(int64_t M, int64_t K, const void *Q, int64_t ldq,
                                        const uint8_t *S, int64_t lds, const void *G, int64_t ldg,
                                        int activation, const void *D, int64_t ldd, int dtype) {
    if (activation != GEMM_ACT_RELU && activation != GEMM_ACT_GELU && activation != GEMM_ACT_SILU)
        return GEMM_ERR_UNSUPPORTED;
    const int st = validate_checkpoint_unpack(M, K, Q, ldq, S, lds, D, ldd, dtype);
    if (st != GEMM_OK) return st;
    if (line_bad(ldg, K)) return GEMM_ERR_INVALID_LD;
    if (M == 0 || K == 0) return GEMM_OK;
    if (!G) return GEMM_ERR_NULL_PTR;
    const int sz = out_size(dtype);
    if (!(G == D && ldg == ldd) && overlap(extent(G, M, K, ldg, sz), extent(D, M, K, ldd, sz)))
        return GEMM_ERR_ALIASING;
    return GEMM_OK;
}

// The weight gradient's tiles and the parts of its tokens that different workgroups
// take, from the sizes alone (for the 256 CUs of a whole device), so that the workspace
// a program reserves fits whatever the device.
//
// Up to 64 outputs the thin kernel (bm 32, 64) streams Q: parts of at least 256 tokens
// while there is less than a workgroup for each CU (16 x 4096 of 8192 tokens, us of the
// kernel and the join: 8 parts 15.0, 4 18.1, 16 18.5).  Past that, the tile and the number
// of parts with the least modelled time, in us: a workgroup's start and end (128 x 128: 5.9,
// 256 x 256: 8.2), its steps of 64 tokens (128: 0.73 alone on the GPU, 0.83 on every CU, 1.18
// with two on each; 256: 1.34 to 1.6), and the parts' sums written and read.  The constants
// are fitted to 290 measured (shape, tile, parts) of 24 shapes, 7% off in the mean, and the
// plan takes 0.8% longer than the best measured one.  Measured (best of the other tile
// beside it): 1001 x 2056 of 3999 128 in 3 40.4 (256 in 6 41.2; 128 whole 55); 512 x 512 of
// 8192 128 in 16 19.9 (26.8); 4096 x 4096 of 4096 256 134.7, the least of its times (184);
// 1024 x 4096 of 2048 128 whole 36.8 (43.6; 128 in 2 41.1); 2048 x 2048 of 4096 128 in 2 59.1
// (256 in 3 58.6).
struct WgradPlan {
    int64_t bm, bn, splits, per;  // per: tokens of a part, a multiple of 64
};
inline WgradPlan wgrad_plan(int64_t M, int64_t N, int64_t K) {
    WgradPlan w;
    const int64_t steps = (M + 63) / 64;
    int64_t s = 1;
    if (N <= 64) {
        w.bm = N <= 32 ? 32 : 64;
        w.bn = 128;
        const int64_t columns = (K + 127) / 128;
        s = columns < 256 ? 256 / columns : 1;
        if (s > steps / 4) s = steps / 4;
        if (s > 64) s = 64;
    } else {
        double best = 0;
        for (int64_t tile = 128; tile <= 256; tile += 128) {
            const double tiles = (double)((N + tile - 1) / tile) * (double)((K + tile - 1) / tile);
            for (int64_t i = 1; i <= 64 && i <= (steps > 1 ? steps / 2 : 1) && (i == 1 || tiles * i <= 1024);
                 ++i) {
                const double groups = tiles * i, per = (double)((steps + i - 1) / i);
                const auto rounds = [&](double at_once) { return (double)(int64_t)((groups + at_once - 1) / at_once); };
                const double busy = groups < 256 ? groups / 256 : 1;
                double t = tile == 256    ? 8.2 + per * (1.34 + 0.26 * busy) * rounds(256)
                           : groups <= 256 ? 5.9 + per * (0.73 + 0.1 * busy)
                                           : 5.9 + per * 1.18 * (0.6 * rounds(512) + 0.4 * groups / 512);
                if (i > 1) t += 2.1 + (double)i * (double)N * (double)K * 8 / 6e6;
                if (best == 0 || t < best) best = t, w.bm = w.bn = tile, s = i;
            }
        }
    }
    if (s < 1) s = 1;
    w.per = steps > 0 ? (steps + s - 1) / s * 64 : 64;
    w.splits = steps > 0 ? (steps * 64 + w.per - 1) / w.per : 1;
    return w;
}

inline int64_t checkpoint_wgrad_workspace(int64_t M, int64_t N, int64_t K) {
    const int64_t kMaxDim = 0x7fffffff;
    if (M < 0 || N < 0 || K < 0 || M > kMaxDim || N > kMaxDim || K > kMaxDim)
        return GEMM_ERR_INVALID_DIM;
    if (M == 0 || N == 0 || K == 0) return 0;
    const WgradPlan w = wgrad_plan(M, N, K);
    return w.splits > 1 ? w.splits * N * ((K + 3) / 4 * 4) * 4 + 255 : 0;
}

inline int validate_checkpoint_wgrad(int64_t M, int64_t N, int64_t K, const void *G, int64_t ldg,
                                     const void *Q, int64_t ldq, const uint8_t *S, int64_t lds,
                                     const void *C, int64_t ldc, const void *D, int64_t ldd,
                                     int in_dtype, int out_dtype, const void *workspace,
                                     int64_t workspace_bytes) {
    const int64_t need = checkpoint_wgrad_workspace(M, N, K);
    if (need < 0) return (int)need;
    const int st = validate_checkpoint_dims(M, K, ldq, lds);
    if (st != GEMM_OK) return st;
    if ((in_dtype != GEMM_F16 && in_dtype != GEMM_BF16) || !is_float(out_dtype))
        return GEMM_ERR_UNSUPPORTED;
    if (line_bad(ldg, N) || line_bad(ldd, K) || (C && line_bad(ldc, K))) return GEMM_ERR_INVALID_LD;
    if (N == 0 || K == 0) return GEMM_OK;
    if (!D || (M > 0 && (!G || !Q || !S)) || (need > 0 && !workspace)) return GEMM_ERR_NULL_PTR;
    if (workspace_bytes < need) return GEMM_ERR_SCRATCH_TOO_SMALL;
    const int osz = out_size(out_dtype);
    const Range rd = extent(D, N, K, ldd, osz), rw = extent(workspace, need > 0 ? 1 : 0, need, need, 1);
    const Range in[3] = {extent(G, M, N, ldg, 2), extent(Q, M, K, ldq, 1),
                         extent(S, M, checkpoint_blocks(K), lds, 1)};
    if (overlap(rd, rw)) return GEMM_ERR_ALIASING;
    for (const Range &r : in)
        if (overlap(r, rd) || overlap(r, rw)) return GEMM_ERR_ALIASING;
    if (C) {
        const Range rc = extent(C, N, K, ldc, osz);
        if (overlap(rc, rw) || (!(C == D && ldc == ldd) && overlap(rc, rd)))
            return GEMM_ERR_ALIASING;
    }
    return GEMM_OK;
}

}  // namespace libgemm_host
