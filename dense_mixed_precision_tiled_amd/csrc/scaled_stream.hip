// The scaled int8 product for few rows (M <= 64): B streamed once.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gemm_configs.hpp"
#include "stream.hpp"

namespace libgemm {

// Workgroup b computes columns [16 NF b, 16 NF (b + 1)) of D for all rows; its
// W waves split K.
template <int MT, int NF, int W, int U>
__global__ void __launch_bounds__(64 * W) scaled_stream_kernel(Params p) {
    using S = StreamTypes<IT_I8, false>;
    __shared__ f32x4 part[W][MT * NF][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int n0 = blockIdx.x * 16 * NF, r = lane & 15;
    const uint8_t *A = reinterpret_cast<const uint8_t *>(p.A);
    const uint8_t *B = reinterpret_cast<const uint8_t *>(p.B);
    // rows past M and channels past N repeat the last one: their sums are not
    // stored
    const uint8_t *wr[NF], *xr[MT];
#pragma unroll
    for (int f = 0; f < NF; ++f) wr[f] = B + (int64_t)min(n0 + 16 * f + r, p.N - 1) * p.ldb;
#pragma unroll
    for (int t = 0; t < MT; ++t) xr[t] = A + (int64_t)min(16 * t + r, p.M - 1) * p.lda;
    f32x4 acc[MT][NF] = {};  // int32 sums
    const int blocks = (p.K + S::KB - 1) / S::KB, per = (blocks + W - 1) / W;
    Stream<IT_I8, false, MT, NF, U, true, true> stream;
    stream.run(wr, xr, lane, min(wave * per, blocks), min((wave + 1) * per, blocks), p.K, acc);
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int f = 0; f < NF; ++f) part[wave][t * NF + f][lane] = acc[t][f];
    __syncthreads();
    // tile (t, f): lane holds row 16 t + lane % 16, four columns from 4 (lane / 16)
    for (int tile = wave; tile < MT * NF; tile += W) {
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

template <int MT, int NF, int W, int U>
static hipError_t launch_stream(const Params &p, hipStream_t s) {
    const dim3 grid((unsigned)((p.N + 16 * NF - 1) / (16 * NF)));
    return launch_params(scaled_stream_kernel<MT, NF, W, U>, grid, dim3(64 * W), p, s);
}

// Variants, measured with the weights in memory (us; M x N x K):
//                    1x4096x4096  1x4096x16384  1x16384x4096  16x16384x16384
//   NF 1, 8 waves, U 2    6.3         14.3          15.2          65.4
//   NF 1, 4 waves, U 4    6.2         16.3          13.9          63.4
//   NF 2, 4 waves, U 4    7.6         19.8          14.5          60.1
// One workgroup for 16 channels; eight waves where that leaves few workgroups
// (more loads in flight on each CU); two channel groups for each wave where
// x is long enough that reading it for every 16 channels counts.  With more row
// groups x's reads count for more: at 32 rows NF 4 takes 17.5 us for
// 32x16384x4096 where NF 1 takes 25.7, but 15.4 against 9.0 for 32x4096x4096,
// where it leaves 64 workgroups.
hipError_t launch_scaled_stream(const Params &p, int cus, hipStream_t s) {
    if (p.M > 64 || p.K <= 0) return hipErrorInvalidValue;
    const bool few = p.N <= 32 * cus;
    if (p.M <= 16) {
        if (few) return launch_stream<1, 1, 8, 2>(p, s);
        if ((int64_t)p.M * p.K >= 131072) return launch_stream<1, 2, 4, 4>(p, s);
        return launch_stream<1, 1, 4, 4>(p, s);
    }
    if (p.M <= 32) return few ? launch_stream<2, 1, 4, 4>(p, s) : launch_stream<2, 4, 4, 2>(p, s);
    return few ? launch_stream<4, 1, 4, 2>(p, s) : launch_stream<4, 4, 8, 1>(p, s);
}

}  // namespace libgemm
