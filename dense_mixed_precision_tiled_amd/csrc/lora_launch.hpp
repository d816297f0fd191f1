// The launches of gemm_lora_run, instantiated for each type of its inputs.
#pragma once

#include "gemm_host.hpp"
#include "lora.hpp"

namespace libgemm {

template <int IT, int OUT, bool VEC>
const void *lora_up_of(bool few, int rank) {
    if (few) return (const void *)lora_up_few_kernel<IT, OUT, VEC>;
    return rank <= 32 ? (const void *)lora_up_kernel<IT, OUT, 1, VEC>
                      : (const void *)lora_up_kernel<IT, OUT, 2, VEC>;
}
template <int IT, bool VEC>
const void *lora_up_of(bool few, int out_dtype, int rank) {
    return out_dtype == DT_F32   ? lora_up_of<IT, DT_F32, VEC>(few, rank)
           : out_dtype == DT_F16 ? lora_up_of<IT, DT_F16, VEC>(few, rank)
                                 : lora_up_of<IT, DT_BF16, VEC>(few, rank);
}
template <int IT, int RT>
const void *lora_down_of(bool vec) {
    return vec ? (const void *)lora_down_kernel<IT, RT, true> : (const void *)lora_down_kernel<IT, RT, false>;
}

template <int IT, int OUT>
const void *lora_one_of(int rank) {
    return rank <= 16 ? (const void *)lora_one_kernel<IT, OUT, 1> : (const void *)lora_one_kernel<IT, OUT, 2>;
}

// Both products in one launch: while the workgroups, of which each reads its adapter's A, are
// at most one for each CU of a whole device, and that A is at most 512 KiB.  us, two launches
// and one, of 4096 x 4096: rank 16, 1 token 5.9 and 4.1, 16 6.9 and 4.7, 32 (512 workgroups)
// 7.4 and 7.7; rank 32, 1 token 7.4 and 6.0; rank 64 and 16 tokens 11.6 and 14.2.  16384 x 4096:
// rank 16 and 1 token 9.8 and 9.2, rank 32 (A of 1 MiB) 12.9 and 15.2.
inline bool lora_one(const LoraParams &p) {
    return p.rank <= 32 && (int64_t)p.T * libgemm_host::cdiv(p.N, 256) <= 256 &&
           (int64_t)p.K * (p.rank <= 16 ? 16 : 32) <= 1 << 18;
}

// few: 16 tokens at a time in the first product, one in the second.  vec_xa, vec_b: 16-byte
// loads of X and A, and of B.  Many tokens without vec_xa take the first kernel of the few: its
// loads know any alignment.
template <int IT>
hipError_t launch_lora(const LoraParams &p, int out_dtype, bool few, bool vec_xa, bool vec_b,
                       hipStream_t s) {
    using libgemm_host::cdiv;
    LoraParams arg = p;
    void *args[] = {&arg};
    // ranks taken at once: 16, 32 or 64
    const int rt = p.rank <= 16 ? 1 : p.rank <= 32 ? 2 : 4;
    const unsigned chunks = (unsigned)cdiv(p.rank, 16 * rt);
    const unsigned tiles16 = (unsigned)cdiv(p.T, 16), tiles64 = (unsigned)cdiv(p.T, 64);
    // a workgroup for each group that a tile may hold while tiles are few
    const unsigned groups = few ? (unsigned)(p.T < 16 ? p.T : 16) : 1;
    const unsigned columns = (unsigned)cdiv(p.N, 256);
    hipError_t e;
    if (few && vec_xa && vec_b && lora_one(p)) {
        const void *k = out_dtype == DT_F32   ? lora_one_of<IT, DT_F32>(p.rank)
                        : out_dtype == DT_F16 ? lora_one_of<IT, DT_F16>(p.rank)
                                              : lora_one_of<IT, DT_BF16>(p.rank);
        return hipLaunchKernel(k, dim3(columns, (unsigned)p.T), dim3(1024), args, 0, s);
    }
    if (few || !vec_xa) {
        const void *k = rt == 1   ? lora_down_of<IT, 1>(vec_xa)
                        : rt == 2 ? lora_down_of<IT, 2>(vec_xa)
                                  : lora_down_of<IT, 4>(vec_xa);
        e = hipLaunchKernel(k, dim3(tiles16, groups, (unsigned)p.splits * chunks), dim3(256), args, 0, s);
    } else {
        const void *k = rt < 4 ? (const void *)lora_down_tile_kernel<IT, 2>
                               : (const void *)lora_down_tile_kernel<IT, 4>;
        e = hipLaunchKernel(k, dim3(tiles64, chunks, (unsigned)p.splits), dim3(256), args, 0, s);
    }
    if (e != hipSuccess) return e;
    if (!few) {
        int lanes = 1;  // threads of a token, 8 ranks each
        while (lanes < (p.ldh + 31) / 32 * 4) lanes *= 2;
        void *with_lanes[] = {&arg, &lanes};
        const void *k = out_dtype == DT_F32 ? (const void *)lora_parts_kernel<IT, 3>
                                            : (const void *)lora_parts_kernel<IT, 2>;
        e = hipLaunchKernel(k, dim3((unsigned)cdiv(p.T, 256 / lanes)), dim3(256), with_lanes, 0, s);
        if (e != hipSuccess) return e;
    }
    const void *k = vec_b ? lora_up_of<IT, true>(few, out_dtype, p.rank)
                          : lora_up_of<IT, false>(few, out_dtype, p.rank);
    return hipLaunchKernel(k, few ? dim3(columns, (unsigned)p.T) : dim3(columns, 1, (unsigned)cdiv(p.T, kLoraUpTokens)), dim3(256),
                           args, 0, s);
}

hipError_t launch_lora_f16(const LoraParams &, int out_dtype, bool few, bool vec_xa, bool vec_b, hipStream_t);
hipError_t launch_lora_bf16(const LoraParams &, int out_dtype, bool few, bool vec_xa, bool vec_b, hipStream_t);

}  // namespace libgemm
