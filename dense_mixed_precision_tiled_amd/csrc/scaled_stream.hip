// The scaled int8 product for few rows (M <= 32): B streamed once.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gemm_configs.hpp"
#include "stream.hpp"

namespace libgemm {

// Workgroup b computes columns [16 NF b, 16 NF (b + 1)) of D for all rows; its
// W waves split K.  MT: groups of 16 rows, or 0 for at most four rows.
template <int MT, int NF, int W, bool DB>
__global__ void __launch_bounds__(64 * W) scaled_stream_kernel(Params p) {
    using S = StreamTypes<IT_I8, false>;
    constexpr int TILES = MT == 0 ? 1 : MT;
    __shared__ f32x4 part[W][TILES * NF][64];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int n0 = blockIdx.x * 16 * NF, r = lane & 15;
    const uint8_t *A = reinterpret_cast<const uint8_t *>(p.A);
    const uint8_t *B = reinterpret_cast<const uint8_t *>(p.B);
    // rows past M and channels past N repeat the last one: their sums are not
    // stored
    StreamRows w[NF];
#pragma unroll
    for (int f = 0; f < NF; ++f)
        w[f].set(lane, B + (int64_t)n0 * p.ldb,
                 [&](int i) { return (uint32_t)(min(16 * f + i, p.N - 1 - n0) * (int)p.ldb); });
    const int groups = (p.K + S::KG - 1) / S::KG, per = (groups + W - 1) / W;
    const int gbeg = min(wave * per, groups), gend = min((wave + 1) * per, groups);
    if constexpr (MT == 0) {  // at most four rows
        StreamFew<IT_I8, false, NF, true, true> stream;
        stream.run(w, A, (uint32_t)(min(r >> 2, p.M - 1) * (int)p.lda), lane, gbeg, gend, p.K);
        Unroll<0, NF>::run([&](auto ff) {
            constexpr int f = decltype(ff)::value;
            const f32x4 v = stream.template sums<f>(lane);
            if ((lane & 3) == 0) part[wave][f][(lane & 48) | (r >> 2)] = v;
        });
    } else {
        StreamRows x[TILES];
        f32x4 acc[TILES][NF] = {};  // int32 sums
#pragma unroll
        for (int t = 0; t < TILES; ++t)
            x[t].set(lane, A, [&](int i) {
                return (uint32_t)min(16 * t + i, p.M - 1) * (uint32_t)p.lda;
            });
        Stream<IT_I8, false, TILES, NF, DB, true, true> stream;
        stream.run(w, x, lane, gbeg, gend, p.K, acc);
#pragma unroll
        for (int t = 0; t < TILES; ++t)
#pragma unroll
            for (int f = 0; f < NF; ++f) part[wave][t * NF + f][lane] = acc[t][f];
    }
    __syncthreads();
    // tile (t, f): lane holds row 16 t + lane % 16, four columns from 4 (lane / 16)
    for (int tile = wave; tile < TILES * NF; tile += W) {
        i32x4 n = {0, 0, 0, 0};
#pragma unroll
        for (int z = 0; z < W; ++z) n += __builtin_bit_cast(i32x4, part[z][tile][lane]);
        const int i = 16 * (tile / NF) + r, j = n0 + 16 * (tile % NF) + 4 * (lane >> 4);
        if (i >= p.M || j >= p.N) continue;
        const float srow = p.row_scale ? p.row_scale[i] : 1.0f;
        f32x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int c = min(j + e, p.N - 1);
            v[e] = (float)n[e] * srow * (p.col_scale ? p.col_scale[c] : 1.0f) * p.alpha;
            if (p.C) v[e] += p.beta * load_c(p, i, c);
            if (p.bias) v[e] += p.bias[p.bias_rows ? i : c];
        }
        const bool full = p.cd_vec && j + 4 <= p.N;
        if (p.out_dtype == DT_F32) {
            if (full) finish4<DT_F32, true, true, true>(p, i, j, v);
            else finish4<DT_F32, false, true, true>(p, i, j, v);
        } else if (p.out_dtype == DT_F16) {
            if (full) finish4<DT_F16, true, true, true>(p, i, j, v);
            else finish4<DT_F16, false, true, true>(p, i, j, v);
        } else {
            if (full) finish4<DT_BF16, true, true, true>(p, i, j, v);
            else finish4<DT_BF16, false, true, true>(p, i, j, v);
        }
    }
}

template <int MT, int NF, int W, bool DB>
static hipError_t launch_stream(const Params &p, hipStream_t s) {
    const dim3 grid((unsigned)((p.N + 16 * NF - 1) / (16 * NF)));
    return launch_params(scaled_stream_kernel<MT, NF, W, DB>, grid, dim3(64 * W), p, s);
}

// Variants, measured with the weights in memory (us), by the channels and waves
// of a workgroup:
//   M x N x K            16, 8   16, 4   32, 4
//   1 x 4096 x 4096       6.1     6.2     6.7    at most four rows
//   1 x 4096 x 16384     14.0    16.1    17.5
//   1 x 16384 x 4096     14.9    14.4    14.6
//   16 x 16384 x 16384   49.1    53.5    56.1    one group of 16 rows
//   1 x 16384 x 4096     16.7    14.6    14.5    (the same for one row)
//   32 x 4096 x 4096      7.9     7.8    10.8    two groups
//   32 x 16384 x 4096    21.0    21.2    17.5
// Eight waves where each has a few groups of K to load ahead, or there are few
// workgroups; with two row groups the reads of x weigh as much as those of the
// weights, and 32 channels halve them once that leaves a workgroup for every CU.
hipError_t launch_scaled_stream(const Params &p, int cus, hipStream_t s) {
    if (p.M > 32 || p.K <= 0) return hipErrorInvalidValue;
    const bool many = p.N >= 32 * cus;
    if (p.M <= 4) return launch_stream<0, 1, 8, true>(p, s);
    if (p.M <= 16)
        return many && p.K < 8192 ? launch_stream<1, 1, 4, true>(p, s)
                                  : launch_stream<1, 1, 8, true>(p, s);
    return many ? launch_stream<2, 2, 4, false>(p, s) : launch_stream<2, 1, 4, true>(p, s);
}

}  // namespace libgemm
