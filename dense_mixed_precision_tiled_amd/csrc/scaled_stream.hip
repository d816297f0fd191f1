// The scaled int8 product for few rows (M <= 32): B streamed once.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gemm_configs.hpp"
#include "stream.hpp"

namespace libgemm {

// Workgroup b computes columns [16 NF b, 16 NF (b + 1)) of D for all rows; its
// W waves split K.  Up to 4 SETS rows, or with SETS = 0 up to 16 MT.
template <int SETS, int MT, int NF, int W, bool DB>
__global__ void __launch_bounds__(64 * W) scaled_stream_kernel(Params p) {
    using S = StreamTypes<IT_I8, false>;
    __shared__ f32x4 part[W][MT * NF][64];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int n0 = blockIdx.x * 16 * NF;
    const uint8_t *A = reinterpret_cast<const uint8_t *>(p.A);
    const uint8_t *B = reinterpret_cast<const uint8_t *>(p.B);
    // rows past M and channels past N repeat the last one: their sums are not
    // stored
    StreamRows w[NF];
#pragma unroll
    for (int f = 0; f < NF; ++f)
        w[f].set(lane, B + (int64_t)n0 * p.ldb,
                 [&](int i) { return (uint32_t)(min(16 * f + i, p.N - 1 - n0) * (int)p.ldb); });
    auto row = [&](int i) { return (uint32_t)min(i, p.M - 1) * (uint32_t)p.lda; };
    const int groups = (p.K + S::KG - 1) / S::KG, per = (groups + W - 1) / W;
    const int gbeg = min(wave * per, groups), gend = min((wave + 1) * per, groups);
    // (the accumulators hold int32 sums)
    if constexpr (SETS > 0) {
        static_assert(MT == 1 && SETS <= 4, "16 rows");
        StreamX<SETS> x;
        x.set(lane, A, row);
        StreamQuads<IT_I8, false, SETS, NF, DB, true, true> stream;
        stream.run(w, x, lane, gbeg, gend, p.K);
        Unroll<0, NF>::run([&](auto ff) {
            constexpr int f = decltype(ff)::value;
            part[wave][f][lane] = stream.template own_sums<f>(lane);
        });
    } else {
        StreamRows x[MT];
#pragma unroll
        for (int t = 0; t < MT; ++t) x[t].set(lane, A, [&](int i) { return row(16 * t + i); });
        f32x4 acc[MT][NF] = {};
        StreamTiles<IT_I8, false, MT, NF, DB, true, true> stream;
        stream.run(w, x, lane, gbeg, gend, p.K, acc);
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int f = 0; f < NF; ++f) part[wave][t * NF + f][lane] = acc[t][f];
    }
    __syncthreads();
    for (int tile = wave; tile < MT * NF; tile += W) {
        i32x4 n = {0, 0, 0, 0};
#pragma unroll
        for (int z = 0; z < W; ++z) n += __builtin_bit_cast(i32x4, part[z][tile][lane]);
        const int i = SETS > 0 ? stream_row<SETS>(lane) : 16 * (tile / NF) + (lane & 15);
        const int j = n0 + 16 * (tile % NF) + 4 * (lane >> 4);
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

template <int SETS, int MT, int NF, int W, bool DB>
static hipError_t launch_stream(const Params &p, hipStream_t s) {
    const dim3 grid((unsigned)((p.N + 16 * NF - 1) / (16 * NF)));
    return launch_params(scaled_stream_kernel<SETS, MT, NF, W, DB>, grid, dim3(64 * W), p, s);
}

// Variants, measured with the weights in memory (us), by the channels and waves
// of a workgroup:
//   M x N x K            16, 8   16, 4   32, 4
//   1 x 4096 x 4096       6.0     6.0     6.7    up to four rows
//   1 x 4096 x 16384     14.0    16.1    17.5
//   1 x 16384 x 4096     14.7    14.3    14.3
//   8 x 4096 x 4096       6.5     6.1     7.3    up to eight
//   8 x 16384 x 4096     16.4    14.1    14.4
//   16 x 16384 x 16384   49.1    53.5    56.1    sixteen
//   16 x 16384 x 4096    16.7    15.0    14.5
//   32 x 4096 x 4096      7.9     7.8    10.8    two groups of 16
//   32 x 16384 x 4096    21.0    21.2    17.5
// Eight waves where each has a few groups of K to load ahead; with two row groups
// the reads of x weigh as much as those of the weights, and 32 channels halve them
// once that leaves a workgroup for every CU.
hipError_t launch_scaled_stream(const Params &p, int cus, hipStream_t s) {
    if (p.M > 32 || p.K <= 0) return hipErrorInvalidValue;
    const bool deep = p.K >= 8192;
    if (p.M <= 4)
        return deep ? launch_stream<1, 1, 1, 8, true>(p, s) : launch_stream<1, 1, 1, 4, true>(p, s);
    if (p.M <= 8)
        return deep ? launch_stream<2, 1, 1, 8, true>(p, s) : launch_stream<2, 1, 1, 4, true>(p, s);
    if (p.M <= 16)
        return deep ? launch_stream<0, 1, 1, 8, true>(p, s) : launch_stream<0, 1, 1, 4, true>(p, s);
    return p.N >= 32 * cus ? launch_stream<0, 2, 2, 4, false>(p, s)
                           : launch_stream<0, 2, 1, 4, true>(p, s);
}

}  // namespace libgemm
