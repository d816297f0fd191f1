// Products of a few rows with a weight matrix that is read once.
//
// y(r, j) = sum_k x(r, k) w(j, k) for up to 16 * MT rows of x: the arithmetic
// for each byte of w is so little that the rate at which w arrives from memory
// is all that counts.  So w goes from memory straight to the matrix units'
// operand registers: a wave takes 16 rows of w (output channels) as the MFMA's
// first operand and 16 rows of x as its second.  Staging w in LDS would add a
// write, a read and a wait to every byte without saving a load: no two waves
// share a byte of w.  x is small and comes from the caches, once for every
// 16 * NF channels.
//
// The MFMA wants lane l to hold row l % 16, a part of k by l / 16.  Loaded in that
// shape, neighbouring lanes are in different rows and every lane's 16 bytes are a
// request of their own: 64 cycles of a CU's address path for each KiB, of w and of
// x alike (16 x 16384 x 16384: 4.1 TB/s; 64 x 4096 x 16384: 1.7 TB/s).  So the four
// lanes of a quad read 64 consecutive bytes of one row, four loads cover the
// quad's four rows, and a 4 x 4 transpose inside the quad (DPP) gives each
// lane 64 bytes of its own row.  The four quads with the same rows take
// consecutive 64 bytes, so a load reads 256 consecutive bytes of four rows.
//
// Any order of k is right as long as x and w take the same one.  The waves of a
// workgroup take consecutive parts of K and add their sums up in LDS, in a fixed
// order: the same call gives the same bits.
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
    const int n = min(max(K - k, 0), EPC);
    if constexpr (VEC) {
        const u32x4 v = *reinterpret_cast<const u32x4 *>(row + (int64_t)(n > 0 ? k : 0) * ES);
        return ES == 2 ? keep_first(v, n) : keep_first_bytes(v, n);
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
// assembly, halves that, but ties the loads of a group together: 64 x 4096 x 16384
// 33 us against 24.)
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

// The 16 rows of one operand tile as a lane reads them: the byte offsets of the
// four rows of its quad and of its own row from a common start.  The start is a
// scalar that moves along K, so the loads need no vector arithmetic for their
// addresses.
struct StreamRows {
    const uint8_t *base;
    uint32_t o0, o1, o2, o3, own;
    // row(i): byte offset of the tile's row i
    template <class F>
    __device__ __forceinline__ void set(int lane, const uint8_t *start, F &&row) {
        const int i = lane & 12;
        base = start;
        o0 = row(i), o1 = row(i + 1), o2 = row(i + 2), o3 = row(i + 3);
        own = row(lane & 15);
    }
    template <int M>
    __device__ __forceinline__ uint32_t quad() const {
        return M == 0 ? o0 : (M == 1 ? o1 : (M == 2 ? o2 : o3));
    }
};

// 16 bytes at a scalar start and a vector offset.
__device__ __forceinline__ u32x4 stream_load(const uint8_t *base, uint32_t offset) {
    return *reinterpret_cast<const u32x4 *>(base + (uint64_t)offset);
}

// acc[t][f] += the products of groups [gbeg, gend) of K (KG values each) of the
// weight rows w[f] and the rows x[t].  XV, WV: the rows allow 16-byte loads.  DB:
// a group is in flight while the one before it is multiplied.
template <int XT, bool W8, int MT, int NF, bool DB, bool XV, bool WV>
struct Stream {
    using S = StreamTypes<XT, W8>;
    static constexpr int XC = S::XC;
    u32x4 wv[DB ? 2 : 1][NF][4], xv[DB ? 2 : 1][MT][XC][4];

    template <int SL>
    __device__ __forceinline__ void load(const StreamRows (&w)[NF], const StreamRows (&x)[MT],
                                         int lane, int g) {
        const uint32_t wo = (lane >> 4) * 64 + (lane & 3) * 16;
        const uint32_t xo = (lane >> 4) * 64 * XC + (lane & 3) * 16;
        Unroll<0, 4>::run([&](auto mm) {
            constexpr int m = decltype(mm)::value;
            Unroll<0, NF>::run([&](auto ff) {
                constexpr int f = decltype(ff)::value;
                wv[SL][f][m] =
                    stream_load(w[f].base + (int64_t)g * 256, w[f].template quad<m>() + wo);
            });
        });
        Unroll<0, 4 * XC>::run([&](auto mm) {
            constexpr int h = decltype(mm)::value / 4, m = decltype(mm)::value % 4;
            Unroll<0, MT>::run([&](auto tt) {
                constexpr int t = decltype(tt)::value;
                xv[SL][t][h][m] = stream_load(x[t].base + (int64_t)g * 256 * XC + 64 * h,
                                              x[t].template quad<m>() + xo);
            });
        });
    }
    // chunk w of channel group f with the one or two chunks of x that go with it
    template <int f>
    __device__ __forceinline__ static void mac(const u32x4 &w, const u32x4 (&x)[MT][XC],
                                               f32x4 (&acc)[MT][NF]) {
        if constexpr (W8) {
            const u32x4 a = stream_widen<XT>(w[0], w[1]), b = stream_widen<XT>(w[2], w[3]);
            Unroll<0, MT>::run([&](auto tt) {
                constexpr int t = decltype(tt)::value;
                acc[t][f] = mfma16_1<XT>(a, x[t][0], acc[t][f]);
                acc[t][f] = mfma16_1<XT>(b, x[t][XC - 1], acc[t][f]);
            });
        } else {
            Unroll<0, MT>::run([&](auto tt) {
                constexpr int t = decltype(tt)::value;
                acc[t][f] = mfma16_1<XT>(w, x[t][0], acc[t][f]);
            });
        }
    }
    template <int SL>
    __device__ __forceinline__ void multiply(f32x4 (&acc)[MT][NF], int lane) {
        Unroll<0, MT>::run([&](auto tt) {
            Unroll<0, XC>::run([&](auto hh) {
                Unroll<0, 4>::run([&](auto mm) {
                    arrive(xv[SL][decltype(tt)::value][decltype(hh)::value][decltype(mm)::value]);
                });
                stream_transpose(xv[SL][decltype(tt)::value][decltype(hh)::value], lane);
            });
        });
        Unroll<0, NF>::run([&](auto ff) {
            constexpr int f = decltype(ff)::value;
            Unroll<0, 4>::run([&](auto mm) { arrive(wv[SL][f][decltype(mm)::value]); });
            stream_transpose(wv[SL][f], lane);
            Unroll<0, 4>::run([&](auto mm) {
                // the lane's chunk m of w: x's chunk m, or with two chunks of x for
                // each of w's its chunks 2m and 2m + 1 of 128 bytes
                constexpr int m = decltype(mm)::value;
                u32x4 xm[MT][XC];
                Unroll<0, MT>::run([&](auto tt) {
                    constexpr int t = decltype(tt)::value;
                    Unroll<0, XC>::run([&](auto hh) {
                        constexpr int c = m * XC + decltype(hh)::value;
                        xm[t][decltype(hh)::value] = xv[SL][t][c / 4][c % 4];
                    });
                });
                mac<f>(wv[SL][f][m], xm, acc);
            });
        });
    }
    __device__ __forceinline__ void run(const StreamRows (&w)[NF], const StreamRows (&x)[MT],
                                        int lane, int gbeg, int gend, int K,
                                        f32x4 (&acc)[MT][NF]) {
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
        // what is left: blocks of 64 bytes of a row, in the MFMA's own shape,
        // values at and past K zero
        if (g >= gend) return;
        const uint8_t *wr[NF], *xr[MT];
#pragma unroll
        for (int f = 0; f < NF; ++f) wr[f] = w[f].base + w[f].own;
#pragma unroll
        for (int t = 0; t < MT; ++t) xr[t] = x[t].base + x[t].own;
        const int bend = min(4 * gend, (K + S::KB - 1) / S::KB);
#pragma nounroll
        for (int b = 4 * g; b < bend; ++b) {
            const int k = b * S::KB + (lane >> 4) * S::EPC;
            u32x4 xm[MT][XC];
            Unroll<0, MT>::run([&](auto tt) {
                constexpr int t = decltype(tt)::value;
                Unroll<0, XC>::run([&](auto hh) {
                    constexpr int h = decltype(hh)::value;
                    xm[t][h] = stream_chunk<S::XES, XV>(xr[t], k + h * (16 / S::XES), K);
                });
            });
            Unroll<0, NF>::run([&](auto ff) {
                constexpr int f = decltype(ff)::value;
                mac<f>(stream_chunk<S::WES, WV>(wr[f], k, K), xm, acc);
            });
        }
    }
};

// The same for at most four rows of x, without the transposes.  A quad's lanes
// hold four different parts of k of one row of w, so the MFMA forms, for operand
// rows 4 j + c and columns 4 t + d, the product of part c of w with part d of x:
// those with c == d are terms of the sum, the others are left alone.  The sum
// over c is taken once, at the end.  One MFMA then serves four rows of x instead
// of sixteen, which costs nothing here, and x takes one load for every four of w.
template <int XT, bool W8, int NF, bool XV, bool WV>
struct StreamFew {
    using S = StreamTypes<XT, W8>;
    static constexpr int XC = S::XC;
    u32x4 wv[2][NF][4], xv[2][XC];
    f32x4 acc[NF][4], rest[NF];

    template <int SL>
    __device__ __forceinline__ void load(const StreamRows (&w)[NF], const uint8_t *x,
                                         uint32_t xrow, int lane, int g) {
        const uint32_t o = (lane >> 4) * 64 + (lane & 3) * 16;
        Unroll<0, 4>::run([&](auto mm) {
            constexpr int m = decltype(mm)::value;
            Unroll<0, NF>::run([&](auto ff) {
                constexpr int f = decltype(ff)::value;
                wv[SL][f][m] =
                    stream_load(w[f].base + (int64_t)g * 256, w[f].template quad<m>() + o);
            });
        });
        Unroll<0, XC>::run([&](auto hh) {
            constexpr int h = decltype(hh)::value;
            xv[SL][h] = stream_load(x + (int64_t)g * 256 * XC + 16 * h, xrow + o * XC);
        });
    }
    __device__ __forceinline__ static f32x4 mac(const u32x4 &w, const u32x4 (&x)[XC], f32x4 a) {
        if constexpr (W8) {
            a = mfma16_1<XT>(stream_widen<XT>(w[0], w[1]), x[0], a);
            return mfma16_1<XT>(stream_widen<XT>(w[2], w[3]), x[XC - 1], a);
        } else {
            return mfma16_1<XT>(w, x[0], a);
        }
    }
    template <int SL>
    __device__ __forceinline__ void multiply() {
        Unroll<0, XC>::run([&](auto hh) { arrive(xv[SL][decltype(hh)::value]); });
        Unroll<0, NF>::run([&](auto ff) {
            Unroll<0, 4>::run([&](auto mm) {
                constexpr int f = decltype(ff)::value, m = decltype(mm)::value;
                arrive(wv[SL][f][m]);
                acc[f][m] = mac(wv[SL][f][m], xv[SL], acc[f][m]);
            });
        });
    }
    // x + xrow: start of row (lane % 16) / 4 of x
    __device__ __forceinline__ void run(const StreamRows (&w)[NF], const uint8_t *x, uint32_t xrow,
                                        int lane, int gbeg, int gend, int K) {
        Unroll<0, NF>::run([&](auto ff) {
            constexpr int f = decltype(ff)::value;
            rest[f] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            Unroll<0, 4>::run([&](auto mm) { acc[f][decltype(mm)::value] = rest[f]; });
        });
        int g = gbeg;
        if constexpr (XV && WV) {
            const int whole = min(gend, K / S::KG);
            if (g < whole) load<0>(w, x, xrow, lane, g);
#pragma nounroll
            for (; g + 2 <= whole; g += 2) {
                load<1>(w, x, xrow, lane, g + 1);
                __builtin_amdgcn_sched_barrier(0);
                multiply<0>();
                __builtin_amdgcn_sched_barrier(0);
                if (g + 2 < whole) load<0>(w, x, xrow, lane, g + 2);
                __builtin_amdgcn_sched_barrier(0);
                multiply<1>();
                __builtin_amdgcn_sched_barrier(0);
            }
            if (g < whole) {
                multiply<0>();
                ++g;
            }
        }
        if (g >= gend) return;
        // what is left in the MFMA's own shape: the four columns of a quad are alike
        const int bend = min(4 * gend, (K + S::KB - 1) / S::KB);
#pragma nounroll
        for (int b = 4 * g; b < bend; ++b) {
            const int k = b * S::KB + (lane >> 4) * S::EPC;
            u32x4 xm[XC];
            Unroll<0, XC>::run([&](auto hh) {
                constexpr int h = decltype(hh)::value;
                xm[h] = stream_chunk<S::XES, XV>(x + xrow, k + h * (16 / S::XES), K);
            });
            Unroll<0, NF>::run([&](auto ff) {
                constexpr int f = decltype(ff)::value;
                rest[f] = mac(stream_chunk<S::WES, WV>(w[f].base + w[f].own, k, K), xm, rest[f]);
            });
        }
    }
    // The sums of channel group f: row (lane % 16) / 4 of x, channels
    // 4 (lane / 16) + 0 .. 3 (the lanes of a quad hold the same).
    template <int f>
    __device__ __forceinline__ f32x4 sums(int lane) const {
        f32x4 out;
        Unroll<0, 4>::run([&](auto mm) {
            constexpr int m = decltype(mm)::value;
            const f32x4 a = acc[f][m];
            const float v01 = lane & 1 ? a[1] : a[0], v23 = lane & 1 ? a[3] : a[2];
            const uint32_t v = __float_as_uint(lane & 2 ? v23 : v01);
            if constexpr (XT == IT_I8) {
                const uint32_t p = v + quad_xor<1>(v);
                out[m] = __uint_as_float(p + quad_xor<2>(p) + __float_as_uint(rest[f][m]));
            } else {
                const float p = __uint_as_float(v) + __uint_as_float(quad_xor<1>(v));
                out[m] = p + __uint_as_float(quad_xor<2>(__float_as_uint(p))) + rest[f][m];
            }
        });
        return out;
    }
};

}  // namespace libgemm
