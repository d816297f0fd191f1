// Products of a few rows with a weight matrix that is read once.
//
// y(r, j) = sum_k x(r, k) w(j, k) for up to 32 rows of x: the arithmetic for
// each byte of w is so little that the rate at which w arrives from memory
// is all that counts.  So w goes from memory straight to the matrix units'
// operand registers: a wave takes 16 rows of w (output channels) as the MFMA's
// first operand and rows of x as its second.  Staging w in LDS would add a
// write, a read and a wait to every byte without saving a load: no two waves
// share a byte of w.  x is small and comes from the caches, once for every
// 16 * NF channels.
//
// The MFMA wants lane l to hold row l % 16, a part of k by l / 16.  Loaded in that
// shape, neighbouring lanes are in different rows and every lane's 16 bytes are a
// request of their own: 64 cycles of a CU's address path for each KiB, of w and of
// x alike (16 x 16384 x 16384 ran at 4.1 TB/s).  So the four lanes of a quad read
// 64 consecutive bytes of one row, and the four quads with the same rows take
// consecutive 64 bytes: a load reads 256 bytes of four rows, and four loads the
// sixteen rows.
//
// The lanes of a quad then hold four different parts of k of one row of w.  With
// x loaded alike (lane 4 t + d of a quad row: part d of row t), the MFMA forms,
// for operand rows 4 j + c and columns 4 t + d, the product of part c of w with
// part d of x: those with c == d are terms of the sums, the others are left
// alone, and the sum over c is taken once, at the end (StreamQuads).  One MFMA
// then serves four rows of x instead of sixteen, of which there is plenty for up
// to eight rows.  For more, the parts are exchanged inside the quads (StreamTiles):
// 64 vector instructions for every four loads, but sixteen rows for each MFMA and
// accumulator (16 x 16384 x 4096: 15.0 us against 17.4; eight rows 15.0 against
// 14.1).
//
// The waves of a workgroup that share a product take consecutive parts of K and
// add their sums up in LDS, in a fixed order: the same call gives the same bits.
#pragma once

#include "gemm_kernels.hpp"

namespace libgemm {

// x of type XT (IT_F16, IT_BF16 or IT_I8); w of the same type, or int8 (W8)
// under 16-bit x, converted on the way (exact: |w| <= 128 fits fp16 and bf16).
template <int XT, bool W8>
struct StreamTypes {
    static constexpr int XES = XT == IT_I8 ? 1 : 2;
    static constexpr int WES = (W8 || XT == IT_I8) ? 1 : 2;
    static constexpr int EPC = 16 / WES;       // k values of one 16-byte chunk of w
    static constexpr int KB = 4 * EPC;         // k values of a block (64 bytes of a row of w)
    static constexpr int KG = 4 * KB;          // k values of a group (256 bytes of a row of w)
    static constexpr int XC = EPC * XES / 16;  // 16-byte chunks of x that go with it
};

// The 16 bytes of `row` that hold elements k, k+1, ... of ES bytes, those at
// and past K zero.  VEC: one load (the row is 16-byte aligned and k a multiple
// of a chunk; a chunk wholly past K reads the row's first instead, so every
// chunk read holds an element of the row).  Otherwise one load per element.
template <int ES, bool VEC>
__device__ __forceinline__ u32x4 stream_chunk(const uint8_t *row, int k, int K) {
    constexpr int EPC = 16 / ES;
    static_assert(VEC || ES <= 2, "rows of fp32 are aligned");
    const int n = min(max(K - k, 0), EPC);
    if constexpr (VEC) {
        const u32x4 v = *reinterpret_cast<const u32x4 *>(row + (int64_t)(n > 0 ? k : 0) * ES);
        return ES == 2 ? keep_first(v, n) : keep_first_bytes(v, n * ES);
    } else {
        u32x4 v = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int e = 0; e < EPC; ++e) {
            if (e < n) {
                const uint32_t h = ES == 2 ? (uint32_t)reinterpret_cast<const uint16_t *>(row)[k + e]
                                           : (uint32_t)row[k + e];
                v[e * ES / 4] |= h << (8 * ES * (e % (4 / ES)));
            }
        }
        return v;
    }
}

// Eight int8 values (two dwords) as eight fp16 or bf16 values, exactly.
template <int XT>
__device__ __forceinline__ u32x4 stream_widen(uint32_t lo, uint32_t hi) {
    u32x4 v;
    if constexpr (XT == IT_F16) {
        // the byte plus 128 in the low mantissa bits of 1024.0 is 1152 + the value
        typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
        const f16x2 off = {(_Float16)1152.0f, (_Float16)1152.0f};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t u = (h ? hi : lo) ^ 0x80808080u;
            const uint32_t a = __builtin_amdgcn_perm(0x64646464u, u, 0x04010400u);
            const uint32_t b = __builtin_amdgcn_perm(0x64646464u, u, 0x04030402u);
            v[2 * h] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, a) - off);
            v[2 * h + 1] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, b) - off);
        }
    } else {
        // through fp32, whose upper half is the bf16 value: an integer of at
        // most 8 bits has no bits below it
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t d = h ? hi : lo;
            uint32_t f[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                f[e] = __float_as_uint((float)(int8_t)(uint8_t)(d >> (8 * e)));
            v[2 * h] = __builtin_amdgcn_perm(f[1], f[0], 0x07060302u);
            v[2 * h + 1] = __builtin_amdgcn_perm(f[3], f[2], 0x07060302u);
        }
    }
    return v;
}

// A value that every lane of the wave holds, as a scalar: loop bounds and row
// numbers kept in vector registers make every branch a masked one and cost two
// registers for each address.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// The same value, computed anew as far as the compiler knows: what is derived from
// it stays inside its loop.  (Row offsets and addresses moved out of a loop over
// several streams, for all of them at once, took 100 registers.)
__device__ __forceinline__ int opaque(int v) {
    asm volatile("" : "+v"(v));
    return v;
}

// A loaded value, used from here on: conversions of it stay behind this point.
// (Moved up to the load, into the loop's previous round, they waited for it there
// and held three registers for each of its dwords.)
__device__ __forceinline__ void arrive(u32x4 &v) { asm volatile("" : "+v"(v)); }

// Lane l reads lane l ^ X of its quad (X = 1, 2).
template <int X>
__device__ __forceinline__ uint32_t quad_xor(uint32_t v) {
    constexpr int perm = X == 1 ? 0xb1 : 0x4e;  // quad_perm 1, 0, 3, 2 and 2, 3, 0, 1
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, perm, 0xf, 0xf, true);
}

// Element m of lane c of every quad becomes element c of lane m: exchanges with
// the neighbours at lane ^ 1 and lane ^ 2.  (64 vector instructions for four
// 16-byte values.  One v_cndmask with its source read across the quad, written as
// assembly, halves that, but ties the loads of a group together: 33 us against 24
// at 64 x 4096 x 16384.)
__device__ __forceinline__ void stream_transpose(u32x4 (&v)[4], int lane) {
    const bool b0 = lane & 1, b1 = lane & 2;
    auto swap1 = [&](uint32_t &lo, uint32_t &hi) {
        const uint32_t l = quad_xor<1>(lo), h = quad_xor<1>(hi);
        lo = b0 ? h : lo;
        hi = b0 ? hi : l;
    };
    auto swap2 = [&](uint32_t &lo, uint32_t &hi) {
        const uint32_t l = quad_xor<2>(lo), h = quad_xor<2>(hi);
        lo = b1 ? h : lo;
        hi = b1 ? hi : l;
    };
    Unroll<0, 4>::run([&](auto dd) {
        constexpr int d = decltype(dd)::value;
        uint32_t a0 = v[0][d], a1 = v[1][d], a2 = v[2][d], a3 = v[3][d];
        swap1(a0, a1);
        swap1(a2, a3);
        swap2(a0, a2);
        swap2(a1, a3);
        v[0][d] = a0, v[1][d] = a1, v[2][d] = a2, v[3][d] = a3;
    });
}

// 16 rows of an operand (NM = 2: 8 rows) as a lane reads them: the byte offsets of the
// four (two) rows of its quad from a common start.  The start is a scalar that moves along K, so the
// loads need no vector arithmetic for their addresses.
struct StreamRows {
    const uint8_t *base;
    int64_t low;  // of x in two parts: bytes from the first one to the second
    uint32_t o0, o1, o2, o3;
    // row(i): byte offset of row i
    template <int NM = 4, class F>
    __device__ __forceinline__ void set(int lane, const uint8_t *start, F &&row,
                                        int64_t second = 0) {
        const int i = (lane & 12) / (4 / NM);
        base = start;
        low = second;
        o0 = row(i), o1 = row(i + 1);
        if constexpr (NM == 4) o2 = row(i + 2), o3 = row(i + 3);
    }
    template <int M>
    __device__ __forceinline__ uint32_t quad() const {
        return M == 0 ? o0 : (M == 1 ? o1 : (M == 2 ? o2 : o3));
    }
};

// Rows 4 s + (lane % 16) / 4 of x, s < SETS: byte offsets from a common start.
template <int SETS>
struct StreamX {
    const uint8_t *base;
    int64_t low;  // x in two parts: bytes from the first one to the second
    uint32_t o[SETS];
    // row(i): byte offset of row i
    template <class F>
    __device__ __forceinline__ void set(int lane, const uint8_t *start, F &&row,
                                        int64_t second = 0) {
        base = start;
        low = second;
        Unroll<0, SETS>::run([&](auto ss) {
            o[decltype(ss)::value] = row(4 * decltype(ss)::value + ((lane & 15) >> 2));
        });
    }
};

// 16 bytes at a scalar start and a vector offset.
__device__ __forceinline__ u32x4 stream_load(const uint8_t *base, uint32_t offset) {
    return *reinterpret_cast<const u32x4 *>(base + (uint64_t)offset);
}

// Rows of x held in fp32 under fp16 weights (XF in what follows): a value times its
// row's scale, a power of two, is the sum of two fp16 values to 22 significant bits,
// wherever in fp32's range the row lies.  (Unscaled, the second one would end at
// 2^-24: 11 bits are left of a value of 1e-4, and one past 65504 is Inf.)  The largest
// value of a row is not known before its last one is read, so the scale follows the
// largest so far: where a scaled value would reach 2^15, the row is scaled down to
// [2^9, 2^10) and its sums with it, which is exact.  What is lost is then below 2^-34
// of the row's largest value so far.  Scales start at 2^126, which the first values
// above 2^-111 bring down.
constexpr float kStreamScale0 = 0x1p126f;

// Magnitudes (as bits) from which a scale of these bits gives 2^15 and more: an exponent
// field of 269 less the scale's, but never past that of Inf.
__device__ __forceinline__ uint32_t stream_limit(float scale) {
    return min((269u << 23) - __float_as_uint(scale), 0x7f800000u);
}
// 1 / scale
__device__ __forceinline__ float stream_unscale(float scale) {
    return __uint_as_float((254u << 23) - __float_as_uint(scale));
}
// The largest magnitude of a lane's N chunks of fp32 values, as bits.
template <int N>
__device__ __forceinline__ uint32_t stream_largest(const u32x4 (&v)[N], uint32_t below) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4 * N; ++i) {
        const uint32_t b = v[i / 4][i % 4] & 0x7fffffffu;
        m = max(m, b < below ? b : 0u);
    }
    return m;
}
// A row's new scale after values of largest finite magnitude m (of this lane; the
// lanes of a row are those that differ in the bits of LANES).  Returns the step of its
// exponent, 0 where it stays.
template <int LANES>
__device__ __forceinline__ int stream_rescale(float &scale, uint32_t m) {
#pragma unroll
    for (int b = 1; b < 64; b <<= 1)
        if (LANES & b) m = max(m, (uint32_t)__shfl_xor((int)m, b));
    if (m < stream_limit(scale)) return 0;
    const uint32_t old = __float_as_uint(scale) >> 23, e = 263 - (m >> 23);
    scale = __uint_as_float(e << 23);
    return (int)e - (int)old;
}
__device__ __forceinline__ void stream_shift(f32x4 &v, int step) {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = __builtin_ldexpf(v[e], step);
}
// Eight fp32 values times scale as two fp16 parts.  finite: all of them are; otherwise the
// second parts are 0 (Inf less Inf would be NaN).
__device__ __forceinline__ void stream_split(const u32x4 &a, const u32x4 &b, float scale,
                                             bool finite, u32x4 &hi, u32x4 &lo) {
    typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const u32x4 &v = i < 2 ? a : b;
        const float x = __uint_as_float(v[2 * (i & 1)]) * scale;
        const float y = __uint_as_float(v[2 * (i & 1) + 1]) * scale;
        const uint32_t both = pack_out16<DT_F16>(x, y);
        const f16x2 h = __builtin_bit_cast(f16x2, both);
        hi[i] = both;
        const uint32_t rest = pack_out16<DT_F16>(x - (float)h[0], y - (float)h[1]);
        lo[i] = finite ? rest : 0u;
    }
}

// The sums over groups [gbeg, gend) of K (KG values each) of NF times 16 rows of w
// and 4 SETS rows of x.  XV, WV: the rows allow 16-byte loads.  DB: a group is in
// flight while the one before it is multiplied.  XP = 2: x is the sum of two matrices
// of its type (a value and what its rounding left), or with XF of fp32 rows.  With XF and
// XP = 1 rows i and i + 2 of a set are the two parts of the same one.  NM = 2: 8 rows
// of w for each of NF instead of 16.
template <int XT, bool W8, int SETS, int NF, bool DB, bool XV, bool WV, int XP = 1, int NM = 4,
          bool XF = false>
struct StreamQuads {
    using S = StreamTypes<XT, W8>;
    static constexpr int XC = S::XC;
    static constexpr int XES = XF ? 4 : S::XES;
    static constexpr int XM = XF ? 2 * XC : XC;  // 16-byte chunks that are next to each other
    static constexpr int NX = XF ? XM : XP * XC;
    static_assert(!XF || (XT == IT_F16 && XV), "fp32 rows go with fp16 weights");
    u32x4 wv[DB ? 2 : 1][NF][NM], xv[DB ? 2 : 1][SETS][NX];
    f32x4 acc[NF][NM][SETS];  // [channel group][row of the quad][row set]
    float scale[XF ? SETS : 1];

    // a group that lies below K
    template <int SL>
    __device__ __forceinline__ void load(const StreamRows (&w)[NF], const StreamX<SETS> &x,
                                         int lane, int g) {
        const uint32_t o = (lane >> 4) * 64 + (lane & 3) * 16;
        Unroll<0, NM>::run([&](auto mm) {
            constexpr int m = decltype(mm)::value;
            Unroll<0, NF>::run([&](auto ff) {
                constexpr int f = decltype(ff)::value;
                wv[SL][f][m] =
                    stream_load(w[f].base + (int64_t)g * 256, w[f].template quad<m>() + o);
            });
        });
        Unroll<0, SETS>::run([&](auto ss) {
            Unroll<0, NX>::run([&](auto hh) {
                constexpr int s = decltype(ss)::value, h = decltype(hh)::value;
                const uint8_t *from = h < XM ? x.base : x.base + x.low;
                xv[SL][s][h] =
                    stream_load(from + (int64_t)g * 256 * XM + 16 * (h % XM), x.o[s] + o * XM);
            });
        });
    }
    // any group, values at and past K zero
    __device__ __forceinline__ void load_some(const StreamRows (&w)[NF], const StreamX<SETS> &x,
                                              int lane, int g, int K) {
        const int k = g * S::KG + (lane >> 4) * S::KB + (lane & 3) * S::EPC;
        Unroll<0, NM>::run([&](auto mm) {
            constexpr int m = decltype(mm)::value;
            Unroll<0, NF>::run([&](auto ff) {
                constexpr int f = decltype(ff)::value;
                wv[0][f][m] =
                    stream_chunk<S::WES, WV>(w[f].base + w[f].template quad<m>(), k, K);
            });
        });
        Unroll<0, SETS>::run([&](auto ss) {
            Unroll<0, NX>::run([&](auto hh) {
                constexpr int s = decltype(ss)::value, h = decltype(hh)::value;
                const uint8_t *from = h < XM ? x.base : x.base + x.low;
                xv[0][s][h] = stream_chunk<XES, XV>(from + x.o[s], k + h % XM * (16 / XES), K);
            });
        });
    }
    // the fp32 values of set s as fp16 parts, in their place
    template <int SL, int s>
    __device__ __forceinline__ void split(int lane) {
        const uint32_t m = stream_largest(xv[SL][s], ~0u);
        if (__ballot(m >= stream_limit(scale[s]))) {
            const int step =
                stream_rescale<1 + 2 + 16 + 32>(scale[s], stream_largest(xv[SL][s], 0x7f800000u));
            Unroll<0, NF * NM>::run([&](auto ii) {
                constexpr int i = decltype(ii)::value;
                stream_shift(acc[i / NM][i % NM][s], step);
            });
        }
        u32x4 hi[XC], lo[XC];
        Unroll<0, XC>::run([&](auto cc) {
            constexpr int c = decltype(cc)::value;
            stream_split(xv[SL][s][2 * c], xv[SL][s][2 * c + 1], scale[s], m < 0x7f800000u, hi[c],
                         lo[c]);
        });
        Unroll<0, XC>::run([&](auto cc) {
            constexpr int c = decltype(cc)::value;
            if constexpr (XP == 2) {
                xv[SL][s][c] = hi[c];
                xv[SL][s][XC + c] = lo[c];
            } else {
#pragma unroll
                for (int d = 0; d < 4; ++d) xv[SL][s][c][d] = lane & 8 ? lo[c][d] : hi[c][d];
            }
        });
    }
    template <int SL>
    __device__ __forceinline__ void multiply(int lane) {
        Unroll<0, SETS>::run([&](auto ss) {
            Unroll<0, NX>::run(
                [&](auto hh) { arrive(xv[SL][decltype(ss)::value][decltype(hh)::value]); });
        });
        if constexpr (XF)
            Unroll<0, SETS>::run([&](auto ss) { split<SL, decltype(ss)::value>(lane); });
        Unroll<0, NF>::run([&](auto ff) {
            Unroll<0, NM>::run([&](auto mm) {
                constexpr int f = decltype(ff)::value, m = decltype(mm)::value;
                arrive(wv[SL][f][m]);
                const u32x4 v = wv[SL][f][m];
                if constexpr (W8) {
                    const u32x4 a = stream_widen<XT>(v[0], v[1]), b = stream_widen<XT>(v[2], v[3]);
                    Unroll<0, XP * XC * SETS>::run([&](auto ss) {
                        constexpr int s = decltype(ss)::value % SETS, h = decltype(ss)::value / SETS;
                        acc[f][m][s] =
                            mfma16_1<XT>(h % XC == 0 ? a : b, xv[SL][s][h], acc[f][m][s]);
                    });
                    // (chunk by chunk: all of a group's widened at once take 64 registers)
                    __builtin_amdgcn_sched_barrier(0);
                } else {
                    Unroll<0, XP * SETS>::run([&](auto ss) {
                        constexpr int s = decltype(ss)::value % SETS, h = decltype(ss)::value / SETS;
                        acc[f][m][s] = mfma16_1<XT>(v, xv[SL][s][h], acc[f][m][s]);
                    });
                }
            });
        });
    }
    __device__ __forceinline__ void run(const StreamRows (&w)[NF], const StreamX<SETS> &x,
                                        int lane, int gbeg, int gend, int K) {
        Unroll<0, NF * NM * SETS>::run([&](auto ii) {
            constexpr int i = decltype(ii)::value;
            acc[i / SETS / NM][i / SETS % NM][i % SETS] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        });
        if constexpr (XF)
            Unroll<0, SETS>::run([&](auto ss) { scale[decltype(ss)::value] = kStreamScale0; });
        int g = gbeg;
        if constexpr (XV && WV) {
            const int whole = min(gend, K / S::KG);  // groups that lie below K
            if constexpr (DB) {
                if (g < whole) load<0>(w, x, lane, g);
#pragma nounroll
                for (; g + 2 <= whole; g += 2) {
                    load<1>(w, x, lane, g + 1);
                    __builtin_amdgcn_sched_barrier(0);
                    multiply<0>(lane);
                    __builtin_amdgcn_sched_barrier(0);
                    if (g + 2 < whole) load<0>(w, x, lane, g + 2);
                    __builtin_amdgcn_sched_barrier(0);
                    multiply<DB ? 1 : 0>(lane);
                    __builtin_amdgcn_sched_barrier(0);
                }
                if (g < whole) {
                    multiply<0>(lane);
                    ++g;
                }
            } else {
#pragma nounroll
                for (; g < whole; ++g) {
                    load<0>(w, x, lane, g);
                    multiply<0>(lane);
                }
            }
        }
#pragma nounroll
        for (; g < gend; ++g) {
            load_some(w, x, lane, g, K);
            multiply<0>(lane);
        }
    }
    // The sums of channel group f and row set s: row 4 s + (lane % 16) / 4 of x,
    // channels NM (lane / 16) + 0 .. NM - 1 (the lanes of a quad hold the same).
    template <int f, int s>
    __device__ __forceinline__ f32x4 sums(int lane) const {
        f32x4 out = {0.0f, 0.0f, 0.0f, 0.0f};
        Unroll<0, NM>::run([&](auto mm) {
            constexpr int m = decltype(mm)::value;
            const f32x4 a = acc[f][m][s];
            const float v01 = lane & 1 ? a[1] : a[0], v23 = lane & 1 ? a[3] : a[2];
            const uint32_t v = __float_as_uint(lane & 2 ? v23 : v01);
            if constexpr (XT == IT_I8) {
                const uint32_t p = v + quad_xor<1>(v);
                out[m] = __uint_as_float(p + quad_xor<2>(p));
            } else {
                const float p = __uint_as_float(v) + __uint_as_float(quad_xor<1>(v));
                out[m] = p + __uint_as_float(quad_xor<2>(__float_as_uint(p)));
                if constexpr (XF) out[m] *= stream_unscale(scale[s]);
            }
        });
        return out;
    }
    // The sums of channel group f and row stream_row<SETS>(lane) + 16 R: up to four
    // row sets at once, lane d of a quad taking set 4 R + d.
    template <int f, int R = 0>
    __device__ __forceinline__ f32x4 own_sums(int lane) const {
        f32x4 out = sums<f, 4 * R>(lane);
        Unroll<1, (SETS - 4 * R < 4 ? SETS - 4 * R : 4)>::run([&](auto dd) {
            constexpr int d = decltype(dd)::value;
            const f32x4 v = sums<f, 4 * R + d>(lane);
#pragma unroll
            for (int e = 0; e < 4; ++e) out[e] = (lane & 3) == d ? v[e] : out[e];
        });
        return out;
    }
};

// The row whose sums own_sums gives a lane: 4 d + (lane % 16) / 4 for lane d of its
// quad, or none (a row past every count) where d is not below SETS.
template <int SETS>
__device__ __forceinline__ int stream_row(int lane) {
    const int d = lane & 3;
    return d < SETS ? 4 * d + ((lane & 15) >> 2) : 1 << 20;
}

// The same for MT times 16 rows of x, exchanged inside the quads (x and w alike) so
// that one MFMA serves 16 rows: acc[t][f] += the products of w[f] and x[t].  Lane l
// of acc holds row l % 16 of x, channels 4 (l / 16) + 0 .. 3.
template <int XT, bool W8, int MT, int NF, bool DB, bool XV, bool WV, int XP = 1,
          bool XF = false>
struct StreamTiles {
    using S = StreamTypes<XT, W8>;
    static constexpr int XC = S::XC;
    static constexpr int XES = XF ? 4 : S::XES;
    static constexpr int XM = XF ? 2 * XC : XC;  // runs of 64 bytes that are next to each other
    static constexpr int NX = XF ? XM : XP * XC;
    static_assert(!XF || (XT == IT_F16 && XV && XP == 2), "fp32 rows as two fp16 parts");
    u32x4 wv[DB ? 2 : 1][NF][4], xv[DB ? 2 : 1][MT][NX][4];
    float scale[XF ? MT : 1];

    template <int SL>
    __device__ __forceinline__ void load(const StreamRows (&w)[NF], const StreamRows (&x)[MT],
                                         int lane, int g) {
        const uint32_t wo = (lane >> 4) * 64 + (lane & 3) * 16;
        const uint32_t xo = (lane >> 4) * 64 * XM + (lane & 3) * 16;
        Unroll<0, 4>::run([&](auto mm) {
            constexpr int m = decltype(mm)::value;
            Unroll<0, NF>::run([&](auto ff) {
                constexpr int f = decltype(ff)::value;
                wv[SL][f][m] =
                    stream_load(w[f].base + (int64_t)g * 256, w[f].template quad<m>() + wo);
            });
        });
        Unroll<0, 4 * NX>::run([&](auto mm) {
            constexpr int h = decltype(mm)::value / 4, m = decltype(mm)::value % 4;
            Unroll<0, MT>::run([&](auto tt) {
                constexpr int t = decltype(tt)::value;
                const uint8_t *from = h < XM ? x[t].base : x[t].base + x[t].low;
                xv[SL][t][h][m] = stream_load(from + (int64_t)g * 256 * XM + 64 * (h % XM),
                                              x[t].template quad<m>() + xo);
            });
        });
    }
    // any group, values at and past K zero
    __device__ __forceinline__ void load_some(const StreamRows (&w)[NF], const StreamRows (&x)[MT],
                                              int lane, int g, int K) {
        const int kw = g * S::KG + (lane >> 4) * S::KB + (lane & 3) * S::EPC;
        const int kx = g * S::KG + (lane >> 4) * S::KB + (lane & 3) * (16 / XES);
        Unroll<0, 4>::run([&](auto mm) {
            constexpr int m = decltype(mm)::value;
            Unroll<0, NF>::run([&](auto ff) {
                constexpr int f = decltype(ff)::value;
                wv[0][f][m] =
                    stream_chunk<S::WES, WV>(w[f].base + w[f].template quad<m>(), kw, K);
            });
        });
        Unroll<0, 4 * NX>::run([&](auto mm) {
            constexpr int h = decltype(mm)::value / 4, m = decltype(mm)::value % 4;
            Unroll<0, MT>::run([&](auto tt) {
                constexpr int t = decltype(tt)::value;
                const uint8_t *from = h < XM ? x[t].base : x[t].base + x[t].low;
                xv[0][t][h][m] = stream_chunk<XES, XV>(from + x[t].template quad<m>(),
                                                       kx + 64 / XES * (h % XM), K);
            });
        });
    }
    // the fp32 values of row group t (pieces of four, in the order of k) as fp16 parts, in
    // their place
    template <int SL, int t>
    __device__ __forceinline__ void split(f32x4 (&acc)[MT][NF]) {
        u32x4 v[4 * NX];
        Unroll<0, 4 * NX>::run([&](auto ii) {
            v[decltype(ii)::value] = xv[SL][t][decltype(ii)::value / 4][decltype(ii)::value % 4];
        });
        const uint32_t m = stream_largest(v, ~0u);
        if (__ballot(m >= stream_limit(scale[t]))) {
            const int step = stream_rescale<16 + 32>(scale[t], stream_largest(v, 0x7f800000u));
            Unroll<0, NF>::run(
                [&](auto ff) { stream_shift(acc[t][decltype(ff)::value], step); });
        }
        Unroll<0, 4 * XC>::run([&](auto cc) {
            constexpr int c = decltype(cc)::value;
            stream_split(v[2 * c], v[2 * c + 1], scale[t], m < 0x7f800000u, xv[SL][t][c / 4][c % 4],
                         xv[SL][t][XC + c / 4][c % 4]);
        });
    }
    template <int SL>
    __device__ __forceinline__ void multiply(f32x4 (&acc)[MT][NF], int lane) {
        Unroll<0, MT>::run([&](auto tt) {
            Unroll<0, NX>::run([&](auto hh) {
                constexpr int t = decltype(tt)::value, h = decltype(hh)::value;
                Unroll<0, 4>::run([&](auto mm) { arrive(xv[SL][t][h][decltype(mm)::value]); });
                stream_transpose(xv[SL][t][h], lane);
            });
            if constexpr (XF) split<SL, decltype(tt)::value>(acc);
        });
        Unroll<0, NF>::run([&](auto ff) {
            constexpr int f = decltype(ff)::value;
            Unroll<0, 4>::run([&](auto mm) { arrive(wv[SL][f][decltype(mm)::value]); });
            stream_transpose(wv[SL][f], lane);
            Unroll<0, 4>::run([&](auto mm) {
                // the lane's chunk m of w goes with x's chunk m, or with two chunks of
                // x for each of w's with its chunks 2 m and 2 m + 1 of 128 bytes
                constexpr int m = decltype(mm)::value;
                const u32x4 v = wv[SL][f][m];
                if constexpr (W8) {
                    const u32x4 a = stream_widen<XT>(v[0], v[1]), b = stream_widen<XT>(v[2], v[3]);
                    Unroll<0, MT * XP>::run([&](auto tt) {
                        constexpr int t = decltype(tt)::value % MT, c = 2 * m;
                        constexpr int h = decltype(tt)::value / MT * XC + c / 4 % XC;
                        acc[t][f] = mfma16_1<XT>(a, xv[SL][t][h][c % 4], acc[t][f]);
                        acc[t][f] = mfma16_1<XT>(b, xv[SL][t][h][c % 4 + 1], acc[t][f]);
                    });
                    __builtin_amdgcn_sched_barrier(0);
                } else {
                    Unroll<0, MT * XP>::run([&](auto tt) {
                        constexpr int t = decltype(tt)::value % MT, h = decltype(tt)::value / MT;
                        acc[t][f] = mfma16_1<XT>(v, xv[SL][t][h][m], acc[t][f]);
                    });
                }
            });
        });
    }
    __device__ __forceinline__ void run(const StreamRows (&w)[NF], const StreamRows (&x)[MT],
                                        int lane, int gbeg, int gend, int K,
                                        f32x4 (&acc)[MT][NF]) {
        if constexpr (XF)
            Unroll<0, MT>::run([&](auto tt) { scale[decltype(tt)::value] = kStreamScale0; });
        int g = gbeg;
        if constexpr (XV && WV) {
            const int whole = min(gend, K / S::KG);  // groups that lie below K
            if constexpr (DB) {
                if (g < whole) load<0>(w, x, lane, g);
#pragma nounroll
                for (; g + 2 <= whole; g += 2) {
                    load<1>(w, x, lane, g + 1);
                    __builtin_amdgcn_sched_barrier(0);
                    multiply<0>(acc, lane);
                    __builtin_amdgcn_sched_barrier(0);
                    if (g + 2 < whole) load<0>(w, x, lane, g + 2);
                    __builtin_amdgcn_sched_barrier(0);
                    multiply<DB ? 1 : 0>(acc, lane);
                    __builtin_amdgcn_sched_barrier(0);
                }
                if (g < whole) {
                    multiply<0>(acc, lane);
                    ++g;
                }
            } else {
#pragma nounroll
                for (; g < whole; ++g) {
                    load<0>(w, x, lane, g);
                    multiply<0>(acc, lane);
                }
            }
        }
#pragma nounroll
        for (; g < gend; ++g) {
            load_some(w, x, lane, g, K);
            multiply<0>(acc, lane);
        }
        if constexpr (XF)
            Unroll<0, MT * NF>::run([&](auto ii) {
                constexpr int i = decltype(ii)::value;
                const float f = stream_unscale(scale[i / NF]);
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i / NF][i % NF][e] *= f;
            });
    }
};

}  // namespace libgemm
