// The scaled int8 product for middle sizes: K-contiguous, 16-byte aligned
// operands and too few output tiles to hide a load behind another workgroup.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gemm_configs.hpp"

namespace libgemm {

// One BM x BN tile of D, its K-tiles loaded straight into LDS STAGES - 1 tiles
// ahead.  With one or two workgroups on a CU nothing else hides what a K-tile
// waits for: two stages (the tiles of gemm_run) leave about 0.6 us for every 128
// values of K, the latency of a load.
//
// WM x WN x WK waves: a K-tile's four MFMA steps (32 values of K each) are shared
// by WK waves, each over BM / WM x BN / WN outputs, and their sums added up in LDS
// at the end.  Waves that split a tile's outputs read its operands once for
// each row or column of waves, so splitting K instead halves the LDS reads of a
// 64 x 64 tile (32 -> 16 KiB for a K-tile), and the MFMAs of a step do not wait
// for each other.
//
// Iteration over G tiles from t on: wait until this wave's loads of them have landed
// (those of the STAGES - 2 G tiles after them may still be in flight; loads complete
// in order), barrier (so have the other waves', and all have read the G tiles
// before), load G tiles into the stages of those, multiply.  G = 2 where a wave has a
// single MFMA for each tile: barrier and LDS latency are paid half as often (40 x 4096 x
// 16384: 24.6 -> 20.6 us; 64 rows 23.5 -> 23.1).  More stages than these change
// nothing (18 of 32 x 32: 23.2).
template <int BM, int BN, int WM, int WN, int WK, int STAGES, int G, bool RAGGED>
__global__ void __launch_bounds__(64 * WM * WN * WK) scaled_pipe_kernel(Params p) {
    constexpr int BK = 128, MF = 32, KS = 4, NW = WM * WN * WK;
    constexpr int TM = BM / WM / MF, TN = BN / WN / MF;
    // A ragged last K-tile is loaded like any other: what lies past K are bytes of the
    // operand's own lines, or zeros past its end, and as no int8 value is Inf or NaN,
    // zeros in A's tile alone take them out of the sums.
    using DA = DmaOperand<BM, BK, NW, MF, true, false, 1>;
    using DB = DmaOperand<BN, BK, NW, MF, true, false, 1>;
    constexpr int SA = DA::BYTES, SB = DB::BYTES, NI = DA::NI + DB::NI;
    static_assert((STAGES - 2 * G) * NI < 64, "the wait counter holds 63 loads");
    static_assert(STAGES % G == 0 && STAGES >= 3 * G, "whole groups of stages");
    static_assert(KS % WK == 0, "MFMA steps of a K-tile");

    // the end: the TM x TN MFMA tiles that WK waves hold partial sums of are
    // finished by RM x RN of them, EM x EN tiles each
    constexpr int RM = TM < WK ? TM : WK, RN = TN < WK / RM ? TN : WK / RM;
    static_assert(TM % RM == 0 && TN % RN == 0, "tiles for each wave");
    constexpr int EM = TM / RM, EN = TN / RN;
    using CE = TileCfg<BM, BN, BK, WM * RM, WN * RN, MF, 1>;
    constexpr int PART = WK > 1 ? NW * TM * TN * 64 * 64 : 0;  // bytes of partial sums
    constexpr int EPI = 4 * (CE::WAVES_M * CE::WAVES_N * (MF * (CE::WTN + 8) + 2 * CE::WTM));
    constexpr int LOOP = STAGES * (SA + SB);
    constexpr int SMEM = LOOP > PART ? (LOOP > EPI ? LOOP : EPI) : (PART > EPI ? PART : EPI);

    __shared__ u32x4 smem[(SMEM + 15) / 16];
    char *const lds = reinterpret_cast<char *>(smem);
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wk = wave % WK, wn = wave / WK % WN, wm = wave / WK / WN;
    int tile_m, tile_n;
    map_tile(p, blockIdx.x, tile_m, tile_n);
    const int m0 = tile_m * BM, n0 = tile_n * BN;

    DA da;
    DB db;
    da.init(lane, wave, m0, p.M, p.lda);
    db.init(lane, wave, n0, p.N, p.ldb);
    const __amdgpu_buffer_rsrc_t ra =
        __builtin_amdgcn_make_buffer_rsrc((void *)p.A, (short)0, (int)p.a_bytes, 0x00020000);
    const __amdgpu_buffer_rsrc_t rb =
        __builtin_amdgcn_make_buffer_rsrc((void *)p.B, (short)0, (int)p.b_bytes, 0x00020000);
    auto fetch = [&](int t, int stage) {
        char *const a = lds + stage * (SA + SB), *const b = a + SA;
#pragma unroll
        for (int i = 0; i < DA::NI; ++i)
            da.issue(ra, a, nullptr, true, wave, i, t * BK, p.lda, p.K);
#pragma unroll
        for (int i = 0; i < DB::NI; ++i)
            db.issue(rb, b, nullptr, true, wave, i, t * BK, p.ldb, p.K);
    };
    // the lane's fragment offsets at this wave's first step (two chunks a step), as
    // in dma_k_loop; its step s moves by 2 WK s chunks
    const int lg = 2 * wk + lane / MF;
    uint32_t a_off[TM], b_off[TN];
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        const int r = wm * (BM / WM) + i * MF + (lane & (MF - 1));
        a_off[i] = (uint32_t)(r * DA::CH + (lg ^ swz_kc(r))) * 16u;
    }
#pragma unroll
    for (int j = 0; j < TN; ++j) {
        const int r = wn * (BN / WN) + j * MF + (lane & (MF - 1));
        b_off[j] = (uint32_t)(r * DB::CH + (lg ^ swz_kc(r))) * 16u + (uint32_t)SA;
    }

    f32x16 acc[TM][TN];  // int32 sums
    Unroll<0, TM>::run([&](auto ii) {
        Unroll<0, TN>::run([&](auto jj) {
            acc[decltype(ii)::value][decltype(jj)::value] = f32x16{};
        });
    });
    const int nk = (p.K + BK - 1) / BK;
#pragma nounroll
    for (int t = 0; t < STAGES - G && t < nk; ++t) fetch(t, t);
    int stage = 0;
#pragma nounroll
    for (int t = 0; t < nk; t += G) {
        if (t + STAGES - G <= nk) wait_vmcnt<(STAGES - 2 * G) * NI>();
        else wait_vmcnt<0>();
        // this wave's reads of the tiles before, whose stages are loaded next, are done
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        char *const at = lds + stage * (SA + SB);
        if constexpr (RAGGED) {
            if (t + G >= nk) {
                DA::zero_tail(at + (nk - 1 - t) * (SA + SB), p.K - (nk - 1) * BK, tid, 64 * NW);
                __syncthreads();
            }
        }
        u32x4 fa[G * KS / WK][TM], fb[G * KS / WK][TN];
        Unroll<0, G * KS / WK>::run([&](auto ss) {
            constexpr int s = decltype(ss)::value;
            constexpr uint32_t kx = (uint32_t)(s % (KS / WK) * WK * 2 * 16);
            char *const from = at + s / (KS / WK) * (SA + SB);
            Unroll<0, TM>::run([&](auto ii) {
                constexpr int i = decltype(ii)::value;
                fa[s][i] = *reinterpret_cast<const u32x4 *>(from + (a_off[i] ^ kx));
            });
            Unroll<0, TN>::run([&](auto jj) {
                constexpr int j = decltype(jj)::value;
                fb[s][j] = *reinterpret_cast<const u32x4 *>(from + (b_off[j] ^ kx));
            });
        });
        const int behind = stage == 0 ? STAGES - G : stage - G;
        Unroll<0, G>::run([&](auto uu) {
            constexpr int u = decltype(uu)::value;
            if (t + STAGES - G + u < nk) fetch(t + STAGES - G + u, behind + u);
        });
        Unroll<0, G * KS / WK>::run([&](auto ss) {
            constexpr int s = decltype(ss)::value;
            // (past the last tile a stage holds anything)
            if (s / (KS / WK) > 0 && t + s / (KS / WK) >= nk) return;
            Unroll<0, TM>::run([&](auto ii) {
                Unroll<0, TN>::run([&](auto jj) {
                    constexpr int i = decltype(ii)::value, j = decltype(jj)::value;
                    acc[i][j] = mfma32_1<IT_I8S>(fb[s][j], fa[s][i], acc[i][j]);
                });
            });
        });
        stage = stage == STAGES - G ? 0 : stage + G;
    }
    __syncthreads();  // every wave has read the last tile: LDS is free

    f32x16 sum[EM][EN];
    const int rm = wk / RN % RM, rn = wk % RN;
    if constexpr (WK == 1) {
        Unroll<0, TM>::run([&](auto ii) {
            Unroll<0, TN>::run([&](auto jj) {
                sum[decltype(ii)::value][decltype(jj)::value] =
                    acc[decltype(ii)::value][decltype(jj)::value];
            });
        });
    } else {
        // [wave][tile][group of four registers][lane]
        f32x4 *const part = reinterpret_cast<f32x4 *>(smem);
        auto at = [&](int w, int tile, int g) {
            return part + ((w * TM * TN + tile) * 4 + g) * 64 + lane;
        };
        Unroll<0, TM>::run([&](auto ii) {
            Unroll<0, TN>::run([&](auto jj) {
                Unroll<0, 4>::run([&](auto gg) {
                    constexpr int i = decltype(ii)::value, j = decltype(jj)::value;
                    constexpr int g = decltype(gg)::value;
                    *at(wave, i * TN + j, g) = acc_group<false>(acc[i][j], g);
                });
            });
        });
        __syncthreads();
        Unroll<0, EM>::run([&](auto ii) {
            Unroll<0, EN>::run([&](auto jj) {
                constexpr int i = decltype(ii)::value, j = decltype(jj)::value;
                const int tile = (rm * EM + i) * TN + rn * EN + j;
                Unroll<0, 4>::run([&](auto gg) {
                    constexpr int g = decltype(gg)::value;
                    i32x4 n = {0, 0, 0, 0};
#pragma unroll
                    for (int z = 0; z < WK; ++z)
                        n += __builtin_bit_cast(i32x4, *at(wave - wk + z, tile, g));
#pragma unroll
                    for (int e = 0; e < 4; ++e) sum[i][j][4 * g + e] = __int_as_float(n[e]);
                });
            });
        });
        __syncthreads();
        if (wk >= RM * RN) return;
    }
    const int etid = ((wm * RM + rm) * (WN * RN) + wn * RN + rn) * 64 + lane;
    ScaledEpilogue<CE, (int)sizeof(smem), false>(p, m0, n0, smem, etid).run(sum);
}

template <int BM, int BN, int WM, int WN, int WK, int STAGES, int G>
static hipError_t launch_pipe(const Params &p, hipStream_t s) {
    Params q = p;
    q.tiles_m = (p.M + BM - 1) / BM;
    q.tiles_n = (p.N + BN - 1) / BN;
    const dim3 grid((unsigned)((int64_t)q.tiles_m * q.tiles_n)), block(64 * WM * WN * WK);
    return p.K % 128
               ? launch_params(scaled_pipe_kernel<BM, BN, WM, WN, WK, STAGES, G, true>, grid, block,
                               q, s)
               : launch_params(scaled_pipe_kernel<BM, BN, WM, WN, WK, STAGES, G, false>, grid, block,
                               q, s);
}

// The tile: what a K-tile costs a CU is its loads, 128 (BM + BN) bytes at about
// 35 bytes a cycle from L2, and 140 cycles between barriers; larger tiles load
// less for each output but leave CUs idle.  Measured (us, one K-tile's cost in
// cycles, tiles for M x N x K):
//             cycles   128x4096x4096   256x4096x4096   512x4096x4096   1024x4096x16384
//   32 x 32    372         12.2 (2/CU)     21.3            39.7            213
//   64 x 32    488         11.6            16.5 (2/CU)     28.4            153
//   64 x 64    604         13.5            13.4            19.5 (2/CU)     108
//   64 x 128   836         17.9            17.5            17.5             91 (2/CU)
//   128 x 128  1068        23.4            22.8            23.2             65
// (the two-stage tiles of gemm_run: 20.3, 20.2, 25.6 and 85.6).  So the tile of the
// least cost is taken, a CU's rounds over its tiles times the tile's cycles.
// Returns false where even 128 x 128 leaves more than one for each CU: there the
// two-stage tiles, two workgroups on a CU, are faster (512x16384x4096: 47 against
// 51 us).
bool launch_scaled_pipe(const Params &p, int cus, hipStream_t s, hipError_t *status) {
    auto tiles = [&](int bm, int bn) {
        return (int64_t)((p.M + bm - 1) / bm) * ((p.N + bn - 1) / bn);
    };
    if (!p.vec_ok || p.K <= 0 || tiles(128, 128) > cus) return false;
    typedef hipError_t (*launch_t)(const Params &, hipStream_t);
    const struct {
        int bm, bn, cycles;
        launch_t launch;
    } kTiles[] = {{32, 32, 372, launch_pipe<32, 32, 1, 1, 4, 12, 2>},
                  {64, 32, 488, launch_pipe<64, 32, 1, 1, 4, 8, 2>},
                  {64, 64, 604, launch_pipe<64, 64, 1, 1, 4, 4, 1>},
                  {64, 128, 836, launch_pipe<64, 128, 1, 2, 4, 4, 1>},
                  {128, 128, 1068, launch_pipe<128, 128, 2, 2, 2, 4, 1>}};
    launch_t best = nullptr;
    int64_t least = 0;
    for (const auto &t : kTiles) {
        const int64_t cost = (tiles(t.bm, t.bn) + cus - 1) / cus * t.cycles;
        if (!best || cost < least) {
            best = t.launch;
            least = cost;
        }
    }
    *status = best(p, s);
    return true;
}

}  // namespace libgemm
