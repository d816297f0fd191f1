// gemm_lora_run: low-rank adapters of many requests at once.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/libgemm.h"
#include "gemm_host.hpp"
#include "gemm_validate.hpp"
#include "lora_launch.hpp"

using namespace libgemm;
using namespace libgemm_host;

extern "C" {

int gemm_validate_lora(int64_t T, const gemm_lora_t *lora, const void *X, int64_t ldx,
                       const int32_t *ids, const void *C, int64_t ldc, const void *D, int64_t ldd,
                       int in_dtype, int out_dtype, const void *workspace,
                       int64_t workspace_bytes) {
    return validate_lora(T, lora, X, ldx, ids, C, ldc, D, ldd, in_dtype, out_dtype, workspace,
                         workspace_bytes);
}

int64_t gemm_lora_workspace(int64_t T, const gemm_lora_t *lora) {
    const int st = validate_lora_dims(T, lora);
    return st == GEMM_OK ? lora_workspace(T, lora).bytes : st;
}

int gemm_lora_run(int64_t T, const gemm_lora_t *lora, const void *X, int64_t ldx,
                  const int32_t *ids, const void *C, int64_t ldc, void *D, int64_t ldd,
                  int in_dtype, int out_dtype, void *workspace, int64_t workspace_bytes,
                  void *stream) {
    const int st = validate_lora(T, lora, X, ldx, ids, C, ldc, D, ldd, in_dtype, out_dtype,
                                 workspace, workspace_bytes);
    if (st != GEMM_OK) return st;
    if (T == 0) return GEMM_OK;
    const gemm_lora_t &l = *lora;
    LoraParams p{};
    p.X = static_cast<const uint8_t *>(X);
    p.A = static_cast<const uint8_t *>(l.A);
    p.B = static_cast<const uint8_t *>(l.B);
    p.ids = ids;
    p.ranks = l.ranks;
    p.scales = l.scales;
    p.C = static_cast<const uint8_t *>(C);
    p.D = static_cast<uint8_t *>(D);
    p.ldx = ldx;
    p.lda = l.lda;
    p.ldb = l.ldb;
    p.ldc = ldc;
    p.ldd = ldd;
    p.T = (int)T;
    p.K = (int)l.K;
    p.N = (int)l.N;
    p.adapters = (int)l.adapters;
    p.rank = (int)l.rank;
    p.in_place = C == D;
    const LoraWorkspace w = lora_workspace(T, lora);
    char *ws = reinterpret_cast<char *>(((uintptr_t)workspace + 255) & ~(uintptr_t)255);
    p.h = reinterpret_cast<float *>(ws);
    p.parts = reinterpret_cast<uint16_t *>(ws + w.parts);
    p.down = reinterpret_cast<float *>(ws + w.down);
    p.ldh = (int)w.ldh;
    p.splits = (int)w.splits;
    p.k_per_split = (int)(cdiv(cdiv(l.K, p.splits), 128) * 128);
    const bool few = T <= kLoraFew;
    const int osz = out_size(out_dtype);
    p.vec_cd = (uintptr_t)D % 16 == 0 && ldd * osz % 16 == 0 &&
               (!C || ((uintptr_t)C % 16 == 0 && ldc * osz % 16 == 0));
    const bool vec_xa = (uintptr_t)X % 16 == 0 && (uintptr_t)l.A % 16 == 0 && ldx % 8 == 0 &&
                        l.lda % 8 == 0;
    const bool vec_b = (uintptr_t)l.B % 16 == 0 && l.ldb % 8 == 0;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const hipError_t e = in_dtype == GEMM_F16
                             ? launch_lora_f16(p, out_dtype, few, vec_xa, vec_b, s)
                             : launch_lora_bf16(p, out_dtype, few, vec_xa, vec_b, s);
    return e == hipSuccess ? GEMM_OK : GEMM_ERR_HIP;
}

}  // extern "C"
