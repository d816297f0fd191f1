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

// few: 16 tokens at a time.  vec_xa, vec_b: 16-byte loads of X and A, and of B.  Many
// tokens without vec_xa take the first kernel of the few: its loads know any alignment.
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
    hipError_t e;
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
        while (8 * lanes < p.ldh) lanes *= 2;
        void *with_lanes[] = {&arg, &lanes};
        const void *k = out_dtype == DT_F32 ? (const void *)lora_parts_kernel<IT, 3>
                                            : (const void *)lora_parts_kernel<IT, 2>;
        e = hipLaunchKernel(k, dim3((unsigned)cdiv(p.T, 256 / lanes)), dim3(256), with_lanes, 0, s);
        if (e != hipSuccess) return e;
    }
    const void *k = vec_b ? lora_up_of<IT, true>(few, out_dtype, p.rank)
                          : lora_up_of<IT, false>(few, out_dtype, p.rank);
    const unsigned columns = (unsigned)cdiv(p.N, 256);
    return hipLaunchKernel(k, few ? dim3(columns, (unsigned)p.T) : dim3(columns, 1, tiles64), dim3(256),
                           args, 0, s);
}

hipError_t launch_lora_f16(const LoraParams &, int out_dtype, bool few, bool vec_xa, bool vec_b, hipStream_t);
hipError_t launch_lora_bf16(const LoraParams &, int out_dtype, bool few, bool vec_xa, bool vec_b, hipStream_t);

}  // namespace libgemm
