// gemm_moe_run: a mixture-of-experts layer for a few tokens.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/libgemm.h"
#include "gemm_host.hpp"
#include "gemm_validate.hpp"
#include "moe.hpp"

using namespace libgemm;
using namespace libgemm_host;

extern "C" {

int gemm_validate_moe(int64_t T, const gemm_moe_t *layer, const void *X, int64_t ldx,
                      const float *logits, int64_t ldl, const void *D, int64_t ldd, int in_dtype,
                      const void *workspace, int64_t workspace_bytes) {
    return validate_moe(T, layer, X, ldx, logits, ldl, D, ldd, in_dtype, workspace,
                        workspace_bytes);
}

int64_t gemm_moe_workspace(int64_t T, const gemm_moe_t *layer) {
    const int st = validate_moe_dims(T, layer);
    return st == GEMM_OK ? moe_workspace(T, layer).bytes : st;
}

int gemm_moe_run(int64_t T, const gemm_moe_t *layer, const void *X, int64_t ldx,
                 const float *logits, int64_t ldl, void *D, int64_t ldd, int in_dtype,
                 void *workspace, int64_t workspace_bytes, void *stream) {
    const int st = validate_moe(T, layer, X, ldx, logits, ldl, D, ldd, in_dtype, workspace,
                                workspace_bytes);
    if (st != GEMM_OK) return st;
    if (T == 0) return GEMM_OK;
    const gemm_moe_t &m = *layer;
    const MoeWorkspace w = moe_workspace(T, layer);
    char *ws = reinterpret_cast<char *>(((uintptr_t)workspace + 255) & ~(uintptr_t)255);
    const bool i8 = m.w_dtype == GEMM_I8;
    MoeParams p{};
    p.X = static_cast<const uint8_t *>(X);
    p.W1 = static_cast<const uint8_t *>(m.W1);
    p.W2 = static_cast<const uint8_t *>(m.W2);
    p.logits = logits;
    p.s1 = i8 ? m.scale1 : nullptr;
    p.s2 = i8 ? m.scale2 : nullptr;
    p.D = static_cast<uint8_t *>(D);
    p.ldx = ldx;
    p.ldl = ldl;
    p.ld1 = m.ld1;
    p.ld2 = m.ld2;
    p.ldd = ldd;
    p.T = (int)T;
    p.H = (int)m.H;
    p.I = (int)m.I;
    p.E = (int)m.E;
    p.topk = (int)m.topk;
    p.slots = (int)w.slots;
    p.act = m.activation;
    p.renorm = m.renormalize ? 1 : 0;
    p.count = reinterpret_cast<int *>(ws + w.count);
    p.expert = reinterpret_cast<int *>(ws + w.expert);
    p.pairs = reinterpret_cast<int *>(ws + w.pairs);
    p.weight = reinterpret_cast<float *>(ws + w.weight);
    p.h = reinterpret_cast<uint8_t *>(ws + w.h);
    p.ldh = (int)w.ldh;
    const int wsz = i8 ? 1 : 2;
    const bool vec = (uintptr_t)X % 16 == 0 && (uintptr_t)m.W1 % 16 == 0 &&
                     (uintptr_t)m.W2 % 16 == 0 && ldx % 8 == 0 && (m.ld1 * wsz) % 16 == 0 &&
                     (m.ld2 * wsz) % 16 == 0;
    const int cus = topology().cus;
    hipStream_t s = static_cast<hipStream_t>(stream);
    hipError_t e;
    if (in_dtype == GEMM_F16)
        e = i8 ? launch_moe_f16_i8(p, cus, vec, s) : launch_moe_f16(p, cus, vec, s);
    else
        e = i8 ? launch_moe_bf16_i8(p, cus, vec, s) : launch_moe_bf16(p, cus, vec, s);
    return e == hipSuccess ? GEMM_OK : GEMM_ERR_HIP;
}

}  // extern "C"
