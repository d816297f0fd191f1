// gemm_lora_run: low-rank adapters of many requests at once.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/libgemm.h"
#include "gemm_host.hpp"
#include "gemm_validate.hpp"
#include "lora.hpp"

using namespace libgemm;
using namespace libgemm_host;

namespace {

template <int IT, int RT>
const void *down_kernel(bool vec) {
    return vec ? (const void *)lora_down_kernel<IT, RT, true>
               : (const void *)lora_down_kernel<IT, RT, false>;
}

template <int IT, int OUT>
const void *up_kernel(bool vec) {
    return vec ? (const void *)lora_up_kernel<IT, OUT, true>
               : (const void *)lora_up_kernel<IT, OUT, false>;
}

template <int IT>
hipError_t launch_lora(const LoraParams &p, int out_dtype, bool vec_xa, bool vec_b, hipStream_t s) {
    LoraParams arg = p;
    void *args[] = {&arg};
    const unsigned tiles = (unsigned)cdiv(p.T, 16);
    // a workgroup for each group that a tile may hold while tiles are few
    const unsigned groups = p.T <= 256 ? (unsigned)(p.T < 16 ? p.T : 16) : 1;
    // ranks taken at once: 16, 32 or 64
    const int rt = p.rank <= 16 ? 1 : p.rank <= 32 ? 2 : 4;
    const unsigned chunks = (unsigned)cdiv(p.rank, 16 * rt);
    const void *down = rt == 1   ? down_kernel<IT, 1>(vec_xa)
                       : rt == 2 ? down_kernel<IT, 2>(vec_xa)
                                 : down_kernel<IT, 4>(vec_xa);
    hipError_t e = hipLaunchKernel(down, dim3(tiles, groups, (unsigned)p.splits * chunks),
                                   dim3(256), args, 0, s);
    if (e != hipSuccess) return e;
    const void *up = out_dtype == GEMM_F32   ? up_kernel<IT, DT_F32>(vec_b)
                     : out_dtype == GEMM_F16 ? up_kernel<IT, DT_F16>(vec_b)
                                             : up_kernel<IT, DT_BF16>(vec_b);
    return hipLaunchKernel(up, dim3(tiles, groups, (unsigned)cdiv(p.N, 256)), dim3(256), args, 0, s);
}

}  // namespace

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
    return st == GEMM_OK ? lora_workspace(T, lora) : st;
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
    p.h = reinterpret_cast<float *>(((uintptr_t)workspace + 255) & ~(uintptr_t)255);
    p.ldh = (int)lora_ldh(l.rank);
    p.splits = (int)lora_splits(T, l.K);
    p.k_per_split = (int)(cdiv(cdiv(l.K, p.splits), 128) * 128);
    const int osz = out_size(out_dtype);
    p.vec_cd = (uintptr_t)D % 16 == 0 && ldd * osz % 16 == 0 &&
               (!C || ((uintptr_t)C % 16 == 0 && ldc * osz % 16 == 0));
    const bool vec_xa = (uintptr_t)X % 16 == 0 && (uintptr_t)l.A % 16 == 0 && ldx % 8 == 0 &&
                        l.lda % 8 == 0;
    const bool vec_b = (uintptr_t)l.B % 16 == 0 && l.ldb % 8 == 0;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const hipError_t e = in_dtype == GEMM_F16
                             ? launch_lora<IT_F16>(p, out_dtype, vec_xa, vec_b, s)
                             : launch_lora<IT_BF16>(p, out_dtype, vec_xa, vec_b, s);
    return e == hipSuccess ? GEMM_OK : GEMM_ERR_HIP;
}

}  // extern "C"
