// The weight gradient's tiles: D = G^T X^ + C with X^ in the 8-bit format of
// checkpoint.hpp, for 16-byte aligned lines.
//
// The reduction runs over the tokens m, 64 at a time in two LDS stages.  G arrives by
// loads straight into LDS, one row for each token.  Q comes through registers: a thread
// holds 16 values of one block for each of its loads, widens them to 16 bits (a
// conversion, a multiplication with the block's unit, half a byte permutation for each
// value) between the MFMAs of the tile before, and writes them to the stage of the next.
// Both operands are read by the transposing LDS reads, which hand a lane 8 values along m.
//
// In LDS, chunk c (8 values) of row m sits at slot c ^ wgrad_slot(m, c).  The part that
// depends on m moves whole 64-byte groups, so that half a wave's transposing reads, four
// rows at 64 bytes, touch distinct banks; bit 0 keeps the widened values' writes apart,
// whose lanes write every second chunk.
//
// What bounds it: the matrix units are busy 45% of the time at 4096^3.  In 64 tokens a wave
// of the 256 x 256 tile issues 32 MFMAs and some 130 vector instructions, most of them
// widening Q (sixteen times over, once for each tile row that reads it); the stages' barrier
// leaves nothing else on the CU.  us, bf16 into fp32: 4096^3 142 without C (970 TFLOP/s; 131
// for a product of bf16 operands of these layouts) and 152 with it; 128 x 128 tiles 184 there,
// but 37 against 59 for 1024 x 4096 of 2048 tokens, where they fill the CUs.
#pragma once

#include "checkpoint.hpp"
#include "stream.hpp"

namespace libgemm {

// The product's own arguments are a Params with the names of D = A x B: M x N of D are the
// layer's outputs x inputs, K its tokens, A = G, and B unused.
struct WgradParams {
    Params g;
    const uint8_t *Q, *S;
    int64_t ldq, lds;
};

template <int CH>  // chunks of a row
__device__ __forceinline__ int wgrad_slot(int m, int c) {
    if constexpr (CH >= 32) return swz_rc(m, 32) | ((c >> 4) & 1);
    else if constexpr (CH == 16) return swz_rc(m, 32) | (m & 1);
    else if constexpr (CH == 8) return (((m >> 1) & 1) << 2) | (m & 1);
    else return m & 1;
}

// Byte offset of what lane `lane` reads for the MFMA operand of rows r0 .. r0 + 31 (of D or
// of D^T) at the first step, half h: as tr_read_offset, in this layout.
template <int CH>
__device__ __forceinline__ uint32_t wgrad_tr_offset(int lane, int h, int r0) {
    const int g = lane / 16, f = (lane % 16) / 4, q = lane % 4;
    const int m = 8 * (g / 2) + 4 * h + f, r = r0 + 16 * (g % 2) + 4 * q, c = r / 8;
    return (uint32_t)((m * CH + (c ^ wgrad_slot<CH>(m, c))) * 16 + (r % 8) * 2);
}

template <class CF, int IT>
struct WgradLoop {
    static constexpr int BM = CF::BM, BN = CF::BN, BK = 64;
    static constexpr int TM = CF::TM, TN = CF::TN, NM = TM * TN;
    static constexpr int NW = CF::WAVES_M * CF::WAVES_N, THREADS = CF::THREADS;
    static constexpr int CA = BM / 8, CB = BN / 8, QC = BN / 16;
    static constexpr int SA = BK * CA, SB = BK * CB;      // chunks of a stage
    static constexpr int NA = SA / 64 / NW;               // loads into LDS of a wave and tile
    static constexpr int NB = BK * QC / THREADS;          // 16-byte loads of Q of a thread and tile
    static constexpr int LDS_BYTES = 2 * (SA + SB) * 16;
    static_assert(SA % (64 * NW) == 0 && BK * QC % THREADS == 0 && THREADS % QC == 0, "shares");
    static_assert(CF::MF == 32 && CF::BK == BK, "32x32 MFMAs, 64 tokens");

    const WgradParams &p;
    char *const lds;
    const uint32_t lds_base;  // its address in LDS
    const int tid, lane, wave;
    const int64_t m_beg, m_end;
    const int nk;
    const uint16_t *a_base;
    const uint8_t *q_base, *s_base;
    uint32_t a_voff[NA], q_voff[NB], s_voff[NB];  // byte offsets in a tile
    u32x4 q[NB], qn[NB];  // of the next tile, and of the one after, on its way
    uint32_t s[NB], sn[NB];

    __device__ __forceinline__ int q_row(int i) const { return (i * THREADS + tid) / QC; }

    __device__ __forceinline__ WgradLoop(const WgradParams &p_, char *lds_, int tid_, int n0, int k0,
                                         int64_t beg, int64_t end)
        : p(p_), lds(lds_), lds_base((uint32_t)(uintptr_t)(LIBGEMM_LDS char *)lds_), tid(tid_), lane(tid_ & 63), wave(__builtin_amdgcn_readfirstlane(tid_ >> 6)),
          m_beg(beg), m_end(end), nk((int)((end - beg + BK - 1) / BK)) {
        a_base = p.g.A;
        q_base = p.Q;
        s_base = p.S;
        // columns past the last read the chunk that holds the last; they feed outputs
        // that are not stored
#pragma unroll
        for (int i = 0; i < NA; ++i) {
            const int at = (wave * NA + i) * 64 + lane, m = at / CA, slot = at % CA;
            const int c = CA >= 32 ? slot ^ swz_rc(m, 32) ^ (((slot ^ swz_rc(m, 32)) >> 4) & 1)
                                   : slot ^ wgrad_slot<CA>(m, 0);
            a_voff[i] = ((uint32_t)m * (uint32_t)p.g.lda + (uint32_t)min(n0 + 8 * c, (p.g.M - 1) & ~7)) * 2u;
        }
        const uint32_t k = (uint32_t)min(k0 + 16 * (tid % QC), (p.g.N - 1) & ~15);
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            q_voff[i] = (uint32_t)q_row(i) * (uint32_t)p.ldq + k;
            s_voff[i] = (uint32_t)q_row(i) * (uint32_t)p.lds + k / kCkBlock;
        }
    }

    // First token of tile t.  A ragged last tile starts where it ends with the part's last
    // token (M is at least 64), so that no lane's offset depends on the tile: its first
    // rows, `again` of them, were in the tile before, and become 0 in both stages (in G's alone,
    // an X^ that is Inf, as fp16 has it past 65504, would make 0 * Inf = NaN of them).
    __device__ __forceinline__ int64_t first(int t) const {
        return min(m_beg + (int64_t)t * BK, m_end - BK);
    }
    __device__ __forceinline__ int again(int t) const { return (int)(m_beg + (int64_t)t * BK - first(t)); }
    // 16 bytes of each lane from base + voff to the wave's next KiB of LDS at dst.  Written
    // out because the compiler lets every LDS read after the builtin of this load wait for
    // it (vmcnt(0), the memory's latency in each tile); here the one wait before the
    // tile's barrier orders them.
    __device__ __forceinline__ static void load_to_lds(const void *base, uint32_t dst, uint32_t voff) {
        const uint64_t a = (uint64_t)base;
        const u32x4 r = {(uint32_t)uniform((int)a), (uint32_t)uniform((int)(a >> 32)) & 0xffffu, 0xffffffffu,
                         0x00020000u};
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                     :
                     : "s"(uniform((int)dst)), "v"(voff), "s"(r)
                     : "memory");  // (m0: nothing else here uses it, and it is set each time)
    }
    __device__ __forceinline__ static __amdgpu_buffer_rsrc_t rsrc(const void *base) {
        return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, -1, 0x00020000);
    }

    __device__ __forceinline__ void load_a(int i, int t, int stage) const {
        load_to_lds(a_base + first(t) * p.g.lda, lds_base + (stage * SA + (wave * NA + i) * 64) * 16, a_voff[i]);
    }
    __device__ __forceinline__ void load_b(int t) {
        const int64_t m = first(t);
        const __amdgpu_buffer_rsrc_t rq = rsrc(q_base + m * p.ldq);
        // the aligned dword that holds the scale.  (A loaded byte is extended where it is
        // carried into the next tile, which waits for it.)
        const uintptr_t at = (uintptr_t)(s_base + m * p.lds);
        const __amdgpu_buffer_rsrc_t rs = rsrc(reinterpret_cast<const void *>(at & ~(uintptr_t)3));
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            qn[i] = buf_load16(rq, q_voff[i], 0u);
            sn[i] = buf_load4(rs, (((uint32_t)at & 3u) + s_voff[i]) & ~3u, 0u);
        }
    }
    // (moves of their own: left to the compiler, they end up behind the next loads, which
    // they then wait for)
    __device__ __forceinline__ static uint32_t taken(uint32_t v) {
        uint32_t d;
        asm volatile("v_mov_b32 %0, %1" : "=v"(d) : "v"(v));
        return d;
    }
    __device__ __forceinline__ void take_b(int t) {
        const uint32_t at = (uint32_t)(uintptr_t)(s_base + first(t) * p.lds);
#pragma unroll
        for (int i = 0; i < NB; ++i) {
#pragma unroll
            for (int e = 0; e < 4; ++e) q[i][e] = taken(qn[i][e]);
            s[i] = taken(sn[i]) >> (8 * ((at + s_voff[i]) & 3)) & 0xffu;
        }
    }
    // Q as taken, widened: dword d (values 2d, 2d + 1) of load i
    template <int i, int d>
    __device__ __forceinline__ uint32_t widen(float unit) const {
        return ck_pair<IT>(ck_int(q[i][d / 2], 2 * (d % 2)) * unit,
                           ck_int(q[i][d / 2], 2 * (d % 2) + 1) * unit);
    }
    template <int i, int h>
    __device__ __forceinline__ void store_b(int stage, const u32x4 &w) const {
        const int m = q_row(i), c = 2 * (tid % QC) + h;
        reinterpret_cast<u32x4 *>(lds)[2 * SA + stage * SB + m * CB + (c ^ wgrad_slot<CB>(m, c))] = w;
    }
    // the first rows of a stage become 0
    __device__ __forceinline__ void zero(int stage, int rows) const {
        u32x4 *const a = reinterpret_cast<u32x4 *>(lds) + stage * SA;
        u32x4 *const b = reinterpret_cast<u32x4 *>(lds) + 2 * SA + stage * SB;
        for (int i = tid; i < rows * CA; i += THREADS) a[i] = u32x4{0u, 0u, 0u, 0u};
        for (int i = tid; i < rows * CB; i += THREADS) b[i] = u32x4{0u, 0u, 0u, 0u};
    }

    __device__ __forceinline__ void run(f32x16 (&acc)[TM][TN]) {
        const int wm = wave / CF::WAVES_N, wn = wave % CF::WAVES_N;
        // (half 1 is four rows on, where the slots are the same)
        uint32_t a_off[TM], b_off[TN];
#pragma unroll
        for (int i = 0; i < TM; ++i) a_off[i] = wgrad_tr_offset<CA>(lane, 0, wm * CF::WTM + 32 * i);
#pragma unroll
        for (int j = 0; j < TN; ++j)
            b_off[j] = 2 * SA * 16 + wgrad_tr_offset<CB>(lane, 0, wn * CF::WTN + 32 * j);
        u32x4 fa[2][TM], fb[2][TN];
        auto read = [&](auto stage_tag, auto ks_tag, auto sl_tag, auto f_tag) {
            constexpr int ks = decltype(ks_tag)::value, sl = decltype(sl_tag)::value;
            constexpr int f = decltype(f_tag)::value, stage = decltype(stage_tag)::value;
            u32x2 v[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if constexpr (f < TM)
                    v[h] = ds_read_tr16(lds + a_off[f] + stage * SA * 16 + (16 * ks + 4 * h) * CA * 16);
                else
                    v[h] = ds_read_tr16(lds + b_off[f - TM] + stage * SB * 16 + (16 * ks + 4 * h) * CB * 16);
            }
            const u32x4 w = {v[0][0], v[0][1], v[1][0], v[1][1]};
            if constexpr (f < TM) fa[sl][f] = w;
            else fb[sl][f - TM] = w;
        };
        using Zero = std::integral_constant<int, 0>;
        // tile 0 in its stage, G of tile 1 on its way, Q of tiles 1 and 2 in registers
        const int last = nk - 1;
#pragma unroll
        for (int i = 0; i < NA; ++i) load_a(i, 0, 0);
        load_b(0);
        wait_vmcnt<0>();
        take_b(0);
        load_b(min(1, last));
        Unroll<0, NB>::run([&](auto ii) {
            constexpr int i = decltype(ii)::value;
            const float u = ck_unit(s[i]);
            Unroll<0, 2>::run([&](auto hh) {
                constexpr int h = decltype(hh)::value;
                store_b<i, h>(0, u32x4{widen<i, 4 * h>(u), widen<i, 4 * h + 1>(u), widen<i, 4 * h + 2>(u),
                                       widen<i, 4 * h + 3>(u)});
            });
        });
        __syncthreads();
        if (again(0) > 0) {
            zero(0, again(0));
            __syncthreads();
        }
        Unroll<0, TM + TN>::run([&](auto f) { read(Zero{}, Zero{}, Zero{}, f); });
        wait_vmcnt<0>();
        take_b(min(1, last));
        __builtin_amdgcn_sched_barrier(0);
        load_b(min(2, last));
#pragma unroll
        for (int i = 0; i < NA; ++i) load_a(i, min(1, last), 1);

        constexpr int KS = BK / 16, NR = TM + TN;
        constexpr int WORDS = 8 * NB, PER = (WORDS + 2 * NM - 1) / (2 * NM);  // dwords of a slot
        // tile t from stage CUR.  Past the last tile the loads and stores go on, into the stage
        // that is not read any more, so that there are no branches.
        auto tile = [&](int t, auto cur_tag) {
            constexpr int CUR = decltype(cur_tag)::value;
            using Cur = std::integral_constant<int, CUR>;
            using Other = std::integral_constant<int, CUR ^ 1>;
            const int after = min(t + 2, last);
            float u[NB];
            Unroll<0, NB>::run([&](auto i) { u[decltype(i)::value] = ck_unit(s[decltype(i)::value]); });
            __builtin_amdgcn_sched_barrier(0);
            u32x4 w;
            Unroll<0, KS>::run([&](auto ks_tag) {
                constexpr int ks = decltype(ks_tag)::value, sl = ks & 1;
                if constexpr (ks == KS - 1) {
                    // what was asked for a tile ago is there, G of tile t + 1 in its stage and Q
                    // of tile t + 2 in registers, and no wave reads stage CUR any more
                    wait_vmcnt<0>();
                    __syncthreads();
                    take_b(after);
                    __builtin_amdgcn_sched_barrier(0);
                    load_b(min(t + 3, last));
                    if (t + 1 == last && again(last) > 0) {
                        zero(CUR ^ 1, again(last));
                        __syncthreads();
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
                Unroll<0, NM>::run([&](auto m_tag) {
                    constexpr int m = decltype(m_tag)::value, i = m / TN, j = m % TN;
                    // (B first: a lane then holds four consecutive columns of a row)
                    acc[i][j] = mfma32_1<IT>(fb[sl][j], fa[sl][i], acc[i][j]);
                    if constexpr (ks < 2) {
                        constexpr int slot = ks * NM + m;
                        Unroll<0, PER>::run([&](auto d_tag) {
                            constexpr int at = slot * PER + decltype(d_tag)::value;
                            if constexpr (at < WORDS) {
                                w[at % 4] = widen<at / 8, at % 8>(u[at / 8]);
                                if constexpr (at % 4 == 3) store_b<at / 8, at / 4 % 2>(CUR ^ 1, w);
                            }
                        });
                    } else if constexpr (ks == KS - 1) {
                        Unroll<0, NA>::run([&](auto g_tag) {
                            constexpr int g = decltype(g_tag)::value;
                            if constexpr (g * NM / NA == m) load_a(g, after, CUR);
                        });
                    }
                    constexpr int lo = NR <= NM ? (m < NR ? m : NR) : m * NR / NM;
                    constexpr int hi = NR <= NM ? (m < NR ? m + 1 : NR) : (m + 1) * NR / NM;
                    Unroll<lo, hi>::run([&](auto q_tag) {
                        constexpr int qq = decltype(q_tag)::value;
                        using F = std::integral_constant<int, (qq == 0) ? 0 : (qq <= TN ? TM + qq - 1 : qq - TN)>;
                        using Sl = std::integral_constant<int, sl ^ 1>;
                        if constexpr (ks + 1 < KS)
                            read(Cur{}, std::integral_constant<int, ks + 1>{}, Sl{}, F{});
                        else
                            read(Other{}, Zero{}, Sl{}, F{});
                    });
                    __builtin_amdgcn_sched_barrier(0);
                });
            });
        };
        int t = 0;
        for (; t + 2 <= nk; t += 2) {
            tile(t, Zero{});
            tile(t + 1, std::integral_constant<int, 1>{});
        }
        if (t < nk) tile(t, Zero{});
    }
};

// The sums of a part, in rows of the workspace that are padded to four columns.
template <class CF>
__device__ __forceinline__ void wgrad_store_part(const Params &p, const f32x16 (&acc)[CF::TM][CF::TN],
                                                 int m0, int n0, int tid) {
    const int lane = tid & 63, wave = tid >> 6;
    const int64_t ld = (p.N + 3) & ~3;
    float *const ws = p.ws + (int64_t)blockIdx.z * p.M * ld;
    Unroll<0, CF::TM>::run([&](auto ii) {
        constexpr int i = decltype(ii)::value;
        const int row = m0 + wave / CF::WAVES_N * CF::WTM + 32 * i + acc_row<32>(lane);
        if (row >= p.M) return;
        Unroll<0, CF::TN * 4>::run([&](auto jg) {
            constexpr int j = decltype(jg)::value / 4, g = decltype(jg)::value % 4;
            const int col = n0 + wave % CF::WAVES_N * CF::WTN + 32 * j + acc_col<32>(lane, g);
            if (col < p.N)
                *reinterpret_cast<f32x4 *>(ws + row * ld + col) =
                    f32x4{acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]};
        });
    });
}

// D's rows straight from the accumulators, four columns for each store, one rounding.  All of
// C is added to the accumulators before the first store: a wait for a load waits for every
// store issued before it.  (tile_epilogue, which can do more, takes 5 us more for a tile of
// 128 x 128.)
template <class CF, int OUT>
__device__ __forceinline__ void wgrad_store(const Params &p, f32x16 (&acc)[CF::TM][CF::TN],
                                            int m0, int n0, int tid) {
    const int lane = tid & 63, wave = tid >> 6;
    constexpr int NG = CF::TN * 4;
    using Raw = typename std::conditional<OUT == DT_F32, u32x4, u32x2>::type;
    const int row0 = m0 + wave / CF::WAVES_N * CF::WTM + acc_row<32>(lane);
    const int col0 = n0 + wave % CF::WAVES_N * CF::WTN + acc_col<32>(lane, 0);
    auto col_of = [&](int g) { return col0 + 32 * (g / 4) + 8 * (g % 4); };
    if (p.C && p.cd_vec)
        Unroll<0, CF::TM>::run([&](auto ii) {
            constexpr int i = decltype(ii)::value;
            const int row = row0 + 32 * i;
            Raw c[NG];
            Unroll<0, NG>::run([&](auto gg) {
                constexpr int g = decltype(gg)::value;
                c[g] = Raw{};
                if (row < p.M && col_of(g) + 4 <= p.N) c[g] = load_c_raw<OUT>(p, row, col_of(g));
            });
            Unroll<0, NG>::run([&](auto gg) {
                constexpr int g = decltype(gg)::value, j = g / 4, r = g % 4 * 4;
                const f32x4 v = c_from_raw<OUT>(c[g]);
                acc[i][j][r] += v[0], acc[i][j][r + 1] += v[1];
                acc[i][j][r + 2] += v[2], acc[i][j][r + 3] += v[3];
            });
        });
    Unroll<0, CF::TM>::run([&](auto ii) {
        constexpr int i = decltype(ii)::value;
        const int row = row0 + 32 * i;
        if (row >= p.M) return;
        Unroll<0, NG>::run([&](auto gg) {
            constexpr int g = decltype(gg)::value, j = g / 4, r = g % 4 * 4;
            const f32x4 v = {acc[i][j][r], acc[i][j][r + 1], acc[i][j][r + 2], acc[i][j][r + 3]};
            if (p.cd_vec && col_of(g) + 4 <= p.N) finish4<OUT, true, false, true>(p, row, col_of(g), v);
            else if (col_of(g) < p.N) finish4<OUT, false, false>(p, row, col_of(g), v);
        });
    });
}

// OUT: the type of D, or less than 0 for the sums of a part.
template <class CF, int IT, int OUT>
__global__ void __launch_bounds__(CF::THREADS, 2) wgrad_tile_kernel(WgradParams p) {
    using L = WgradLoop<CF, IT>;
    __shared__ u32x4 smem[L::LDS_BYTES / 16];
    const int tid = threadIdx.x;
    int tile_n, tile_k;
    map_tile(p.g, blockIdx.x, tile_n, tile_k);
    const int n0 = tile_n * CF::BM, k0 = tile_k * CF::BN;
    const int64_t beg = (int64_t)blockIdx.z * p.g.k_per_split;
    const int64_t end = beg + p.g.k_per_split < p.g.K ? beg + p.g.k_per_split : p.g.K;
    f32x16 acc[CF::TM][CF::TN];
    Unroll<0, CF::TM>::run([&](auto i) {
        Unroll<0, CF::TN>::run([&](auto j) { acc[decltype(i)::value][decltype(j)::value] = f32x16{}; });
    });
    L(p, reinterpret_cast<char *>(smem), tid, n0, k0, beg, end).run(acc);
    if constexpr (OUT < 0) wgrad_store_part<CF>(p.g, acc, n0, k0, tid);
    else wgrad_store<CF, OUT>(p.g, acc, n0, k0, tid);
    wait_vmcnt<0>();  // the loads past the last tile land before the workgroup's LDS is released
}

}  // namespace libgemm
