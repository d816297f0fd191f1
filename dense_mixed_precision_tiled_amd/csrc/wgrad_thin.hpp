// The weight gradient of a layer with few outputs (a router, an adapter's first matrix):
// D = G^T X^ + C with up to 64 rows of D.
//
// Q is all there is to read, and each of its values meets few of G, so Q goes from memory
// straight to the registers that feed the MFMA, with no barrier in the loop.  The MFMA
// wants a lane to hold eight tokens of one column.  A lane loads four consecutive columns
// of eight tokens, a dword each (32 lanes read 128 bytes of a row), and byte j of the eight
// dwords is its part of an MFMA whose columns are j, 4 + j, 8 + j, ...: four MFMAs for 128
// columns, and a lane ends up with four consecutive columns of D.
//
// The eight waves of a workgroup take consecutive tokens of the same 128 columns and add
// their sums up in LDS.  G's rows and the blocks' units (fp32) of a stretch of tokens are
// laid out in LDS before it: the loop reads them from there, G with the transposing reads.
//
// Bound by latency: 16 x 4096 of 8192 tokens, 256 workgroups, takes 13.2 us, 35 MB at 2.7 TB/s,
// half of a copy's rate, with one workgroup on a CU and nothing to cover its first loads of G, S
// and Q.
#pragma once

#include "wgrad.hpp"

namespace libgemm {

constexpr int kThinWaves = 8, kThinColumns = 128;

// Tokens of a stretch: G's rows of 32 TM values and four units take 80 KiB at most.
template <int TM>
constexpr int kThinTokens = TM == 1 ? 1024 : 512;

template <int IT, int TM>
__global__ void __launch_bounds__(64 * kThinWaves, 2) wgrad_thin_kernel(WgradParams p) {
    constexpr int P = kThinTokens<TM>, CA = 4 * TM, THREADS = 64 * kThinWaves;
    static_assert(THREADS == 16 * 32, "a thread for each four columns of 16 rows");
    constexpr int PW = P / kThinWaves, STEPS = PW / 16;  // of a wave
    constexpr int G_BYTES = P * CA * 16, SUM_BYTES = kThinWaves * 8 * 64 * 16;
    constexpr int BYTES = G_BYTES + 4 * P * 4;
    __shared__ u32x4 smem[(BYTES > SUM_BYTES ? BYTES : SUM_BYTES) / 16];
    // [4][P], token m of block b at m ^ 8 b: the blocks in banks of their own
    float *const units = reinterpret_cast<float *>(smem + P * CA);
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int N = p.g.M, K = p.g.N, k0 = blockIdx.x * kThinColumns;
    const int64_t m_beg = (int64_t)blockIdx.z * p.g.k_per_split;
    const int64_t m_end = m_beg + p.g.k_per_split < p.g.K ? m_beg + p.g.k_per_split : p.g.K;
    const int half = lane / 32, l = lane % 32;
    // columns past the last read the dword that holds the last
    const uint32_t col = (uint32_t)min(k0 + 4 * l, (K - 1) & ~3);
    const uint32_t voff = 8u * half * (uint32_t)p.ldq + col;
    uint32_t a_off[TM];
#pragma unroll
    for (int i = 0; i < TM; ++i) a_off[i] = wgrad_tr_offset<CA>(lane, 0, 32 * i);
    const char *const g_lds = reinterpret_cast<const char *>(smem);
    const float *const u_lane = units + (l / 8) * P;

    f32x16 acc[TM][4];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = f32x16{};

    // the eight dwords of the 16 tokens from m on; rows past the last read the last
    auto load = [&](int64_t m, uint32_t (&q)[8]) {
        const int left = (int)(m_end - m < 16 ? m_end - m : 16);
        const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<uint8_t *>(p.Q + (left > 0 ? m : m_end - 1) * p.ldq), (short)0, -1, 0x00020000);
        if (left == 16) {
#pragma unroll
            for (int e = 0; e < 8; ++e) q[e] = buf_load4(r, voff, (uint32_t)e * (uint32_t)p.ldq);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                q[e] = buf_load4(r, (uint32_t)min(8 * half + e, max(left - 1, 0)) * (uint32_t)p.ldq + col, 0u);
        }
    };
    // the MFMAs of step s of the stretch's tokens
    auto multiply = [&](int at, const uint32_t (&q)[8]) {
        u32x4 g[TM];
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            const u32x2 lo = ds_read_tr16(g_lds + a_off[i] + at * CA * 16);
            const u32x2 hi = ds_read_tr16(g_lds + a_off[i] + (at + 4) * CA * 16);
            g[i] = u32x4{lo[0], lo[1], hi[0], hi[1]};
        }
        const float *const u = u_lane + ((at + 8 * half) ^ (8 * (l / 8)));
        const f32x4 u0 = *reinterpret_cast<const f32x4 *>(u), u1 = *reinterpret_cast<const f32x4 *>(u + 4);
        Unroll<0, 4>::run([&](auto jj) {
            constexpr int j = decltype(jj)::value;
            u32x4 x;
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                const float a = d < 2 ? u0[2 * d] : u1[2 * d - 4], b = d < 2 ? u0[2 * d + 1] : u1[2 * d - 3];
                x[d] = ck_pair<IT>(ck_int(q[2 * d], j) * a, ck_int(q[2 * d + 1], j) * b);
            }
            Unroll<0, TM>::run([&](auto ii) {
                constexpr int i = decltype(ii)::value;
                acc[i][j] = mfma32_1<IT>(g[i], x, acc[i][j]);
            });
        });
    };

    const int blocks = (K + kCkBlock - 1) / kCkBlock;
    for (int64_t m0 = m_beg; m0 < m_end; m0 += P) {
        const int64_t mw = m0 + wave * PW;
        const int steps = (int)min((int64_t)STEPS, (m_end - mw + 15) / 16);  // (none: 0 or less)
        // four steps of Q on their way (a wave's 8 KiB), then the stretch of G and S
        uint32_t q[4][8];
#pragma unroll
        for (int s = 0; s < 4; ++s)
            if (s < steps) load(mw + 16 * s, q[s]);
        constexpr int NG = P * CA / THREADS, NS = 4 * P / THREADS;
        u32x4 g[NG];
        uint32_t u[NS];
        const int last = (int)min((int64_t)P, m_end - m0) - 1;
#pragma unroll
        for (int i = 0; i < NG; ++i) {
            const int at = i * THREADS + tid, m = min(at / CA, last), c = min(at % CA, (N - 1) / 8);
            g[i] = *reinterpret_cast<const u32x4 *>(p.g.A + (m0 + m) * p.g.lda + 8 * c);
        }
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            const int at = i * THREADS + tid, m = min(at / 4, last);
            u[i] = p.S[(m0 + m) * p.lds + min(k0 / kCkBlock + at % 4, blocks - 1)];
        }
        if (m0 > m_beg) __syncthreads();  // the last stretch's reads are done
#pragma unroll
        for (int i = 0; i < NG; ++i) {
            // rows past the last: 0
            const int at = i * THREADS + tid, m = at / CA, c = at % CA;
            smem[m * CA + (c ^ wgrad_slot<CA>(m, c))] = m <= last ? g[i] : u32x4{0u, 0u, 0u, 0u};
        }
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            const int at = i * THREADS + tid, m = at / 4, b = at % 4;
            // (tokens past the last, for which the last one's Q is read, are 0 on this side too: an
            // X^ that is Inf, as fp16 has it past 65504, would make 0 * Inf = NaN of them)
            units[b * P + (m ^ (8 * b))] = m <= last ? ck_unit(u[i]) : 0.0f;
        }
        __syncthreads();
        for (int s0 = 0; s0 < steps; s0 += 4) {
            Unroll<0, 4>::run([&](auto ss) {
                constexpr int s = decltype(ss)::value;
                if (s0 + s >= steps) return;
                multiply(wave * PW + 16 * (s0 + s), q[s]);
                if (s0 + s + 4 < steps) load(mw + 16 * (s0 + s + 4), q[s]);
            });
        }
    }

    // the eight waves' sums, in order, 16 rows of D at a time: register r of a half holds
    // row 8 (r / 4) + 4 half + r % 4, so eight registers make 16 rows, a thread four columns
    f32x4 *const sums = reinterpret_cast<f32x4 *>(smem);  // [waves][8][64]
    const int64_t ld = (K + 3) & ~3;
    float *const ws = p.g.ws + (int64_t)blockIdx.z * N * ld;
    const int row = tid / 32, k = k0 + 4 * (tid % 32);
    const int from = (row / 8 * 4 + row % 4) * 64 + row / 4 % 2 * 32 + tid % 32;
    Unroll<0, 2 * TM>::run([&](auto hh) {
        constexpr int i = decltype(hh)::value / 2, r0 = decltype(hh)::value % 2 * 8;
        if (32 * i + 2 * r0 >= N) return;
        __syncthreads();
#pragma unroll
        for (int r = 0; r < 8; ++r)
            sums[(wave * 8 + r) * 64 + lane] =
                f32x4{acc[i][0][r0 + r], acc[i][1][r0 + r], acc[i][2][r0 + r], acc[i][3][r0 + r]};
        __syncthreads();
        const int n = 32 * i + 2 * r0 + row;
        if (n >= N || k >= K) return;
        f32x4 v = sums[from];
#pragma unroll
        for (int w = 1; w < kThinWaves; ++w) v += sums[w * 8 * 64 + from];
        if (p.g.splits > 1) {
            *reinterpret_cast<f32x4 *>(ws + n * ld + k) = v;
        } else if (p.g.cd_vec && k + 4 <= K) {
            if (p.g.out_dtype == DT_F32) finish4<DT_F32, true, false>(p.g, n, k, v);
            else if (p.g.out_dtype == DT_F16) finish4<DT_F16, true, false>(p.g, n, k, v);
            else finish4<DT_BF16, true, false>(p.g, n, k, v);
        } else {
            if (p.g.out_dtype == DT_F32) finish4<DT_F32, false, false>(p.g, n, k, v);
            else if (p.g.out_dtype == DT_F16) finish4<DT_F16, false, false>(p.g, n, k, v);
            else finish4<DT_BF16, false, false>(p.g, n, k, v);
        }
    });
}

}  // namespace libgemm
