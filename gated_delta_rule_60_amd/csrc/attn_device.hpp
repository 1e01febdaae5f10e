// attn_device.hpp -- device-side pieces shared by the softmax-attention
// kernels: LDS tiles of key/value/query rows, their MFMA fragments, and the
// map from workgroups to pieces of packed sequences.
//
// The products use the 32x32 MFMA shapes.  A 32x32 fp32 accumulator is 16
// floats per lane: lane l holds column (l & 31), and register i holds row
// 8 (i >> 2) + 4 (l >> 5) + (i & 3).  Scores are formed with the contracted
// tile's rows (keys, or queries in the dK/dV pass) as the 32 rows, so a lane
// owns one column: its softmax statistics are plain per-lane scalars, joined
// with the other half-wave by one v_permlane32_swap.  The same registers,
// rounded to the storage type, are the B operand of the second product with
// the reduction slots of a half-wave h being rows {4h .. 4h+3} and
// {8 + 4h .. 8 + 4h + 3} of every 16; its A operand is read from the tile
// column-wise in that order (ds_read_b64_tr_b16 hands a lane four rows of
// one column), so nothing is shuffled between the two products.
#pragma once

#include "kda_device.hpp"

namespace kda {

typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef unsigned short u16x4_t __attribute__((ext_vector_type(4)));

constexpr float kLn2 = 0.6931471805599453f;

#define KDA_LDS __attribute__((address_space(3)))

// max / sum over the two half-waves (lanes l and l ^ 32)
__device__ __forceinline__ float half_max(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float half_sum(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// 16 (4) bytes a lane from a buffer range to LDS at `lds` (the wave's base) + 16 (4) lane.  Written
// out, because the compiler waits for every load into LDS it knows of before each column read
// (ds_read_b64_tr_b16), the next tile's among them.  The load has no output register; whoever
// reads the tile waits for it with lds_ready().  m0 holds the LDS base, one wait state ahead.
__device__ __forceinline__ unsigned lds_offset(const char* p) {
    return __builtin_amdgcn_readfirstlane(static_cast<unsigned>(reinterpret_cast<uintptr_t>((KDA_LDS const char*)p)));
}
__device__ __forceinline__ void load_lds16(__amdgpu_buffer_rsrc_t r, char* lds, int voff, int soff) {
#if defined(__HIP_DEVICE_COMPILE__)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 :: "s"(lds_offset(lds)), "v"(voff), "s"(r), "s"(soff) : "memory", "m0");
#endif
}
__device__ __forceinline__ void load_lds4(__amdgpu_buffer_rsrc_t r, char* lds, int voff, int soff) {
#if defined(__HIP_DEVICE_COMPILE__)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, %3 offen lds"
                 :: "s"(lds_offset(lds)), "v"(voff), "s"(r), "s"(soff) : "memory", "m0");
#endif
}

// Column quads at LDS offsets p[0 .. N - 1] (each lane's own), and the wait for them in the same
// block: for kernels whose loads into LDS the compiler knows (see load_lds16).
template <int N>
__device__ __forceinline__ void read_quads(bf16x4_t (&x)[N], const unsigned (&p)[N]) {
#if defined(__HIP_DEVICE_COMPILE__)
    static_assert(N == 4, "one block of four reads");
    u32x2_t y[4];
    asm volatile("ds_read_b64_tr_b16 %0, %4\n\tds_read_b64_tr_b16 %1, %5\n\t"
                 "ds_read_b64_tr_b16 %2, %6\n\tds_read_b64_tr_b16 %3, %7\n\ts_waitcnt lgkmcnt(0)"
                 : "=&v"(y[0]), "=&v"(y[1]), "=&v"(y[2]), "=&v"(y[3])
                 : "v"(p[0]), "v"(p[1]), "v"(p[2]), "v"(p[3]) : "memory");
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = __builtin_bit_cast(bf16x4_t, y[i]);
#endif
}

// Sum over the wave, in every lane's scalar register.
__device__ __forceinline__ int wave_sum(int x) {
    x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xF, 0xF, true);  // row_shr:1
    x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xF, 0xF, true);  // row_shr:2
    x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xF, 0xF, true);  // row_shr:4
    x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xF, 0xF, true);  // row_shr:8
    x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xA, 0xF, false);  // row_bcast:15
    x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xC, 0xF, false);  // row_bcast:31
    return __builtin_amdgcn_readlane(x, 63);
}
// Inclusive prefix sum over the wave.
__device__ __forceinline__ int wave_scan(int x) {
    x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xF, 0xF, true);
    x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xF, 0xF, true);
    x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xF, 0xF, true);
    x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xF, 0xF, true);
    x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xA, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xC, 0xF, false);
    return x;
}

// ---------------------------------------------------------------------------
// A piece of a packed sequence: rows [beg + tile * BM, ...) of the sequence
// [beg, beg + len).
// ---------------------------------------------------------------------------
struct SeqTile {
    int beg, len, tile, n;  // n: the sequence
};

__device__ __forceinline__ int2 seq_bounds(const int32_t* cu, int n, int T_tot) {
    int a = cu[n], b = cu[n + 1];
    a = a < 0 ? 0 : (a > T_tot ? T_tot : a);
    b = b < a ? a : (b > T_tot ? T_tot : b);
    return make_int2(a, b - a);
}

// Piece number p of the batch; false if there are fewer.  Every lane of the
// wave gets the same answer.
//
// Up to 64 sequences: pieces in the order of falling work.  Piece t of a
// sequence (counted from its first row, or from its last with `from_end`)
// has t + 1 units of causal work, so all pieces with the largest t come
// first; the launch then ends with the short ones and the compute units
// finish together.  Piece p lies at the level L with C(L + 1) <= p < C(L),
// C(L) = sum_n max(0, tiles_n - L), found by bisection with one lane per
// sequence.  More sequences: in their own order, 64 at a time.
template <int BM>
__device__ __forceinline__ bool find_tile(const int32_t* cu, int N, int T_tot, int p, bool from_end, SeqTile& s) {
    const int lane = threadIdx.x & 63;
    if (N <= 64) {
        int2 bl = make_int2(0, 0);
        if (lane < N) bl = seq_bounds(cu, lane, T_tot);
        const int nt = (bl.y + BM - 1) / BM;
        if (p >= wave_sum(nt)) return false;
        int lo = 0, hi = (T_tot + BM - 1) / BM;  // C(lo) > p >= C(hi)
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            const int c = wave_sum(nt > mid ? nt - mid : 0);
            if (c > p) lo = mid; else hi = mid;
        }
        const int r = p - wave_sum(nt > lo + 1 ? nt - lo - 1 : 0);
        // the r-th sequence with more than lo pieces
        unsigned long long m = __ballot(nt > lo);
        for (int i = 0; i < r; ++i) m &= m - 1;
        const int n = __builtin_ctzll(m);
        s.beg = __builtin_amdgcn_readlane(bl.x, n);
        s.len = __builtin_amdgcn_readlane(bl.y, n);
        s.tile = from_end ? (s.len + BM - 1) / BM - 1 - lo : lo;
        s.n = n;
        return true;
    }
    for (int n0 = 0; n0 < N; n0 += 64) {
        int2 bl = make_int2(0, 0);
        if (n0 + lane < N) bl = seq_bounds(cu, n0 + lane, T_tot);
        const int nt = (bl.y + BM - 1) / BM;
        const int incl = wave_scan(nt);
        const int total = __builtin_amdgcn_readlane(incl, 63);
        if (p < total) {
            const int n = __builtin_ctzll(__ballot(incl > p));
            s.beg = __builtin_amdgcn_readlane(bl.x, n);
            s.len = __builtin_amdgcn_readlane(bl.y, n);
            s.tile = p - (__builtin_amdgcn_readlane(incl, n) - __builtin_amdgcn_readlane(nt, n));
            s.n = n0 + n;
            return true;
        }
        p -= total;
    }
    return false;
}

// ---------------------------------------------------------------------------
// Operand types of one product step.  Row fragments hold 16 bytes of a row:
// 8 bf16 (one 32x32x16 MFMA) or 4 floats (four 32x32x2 MFMAs).
// ---------------------------------------------------------------------------
template <bool BF16>
struct AttnOp;
template <>
struct AttnOp<true> {
    using G = uint16_t;
    using Row = bf16x8_t;
    static constexpr int ES = 2;
    static constexpr int BN = 64;  // rows of a streamed tile
    static __device__ __forceinline__ f32x16_t mma(const Row& a, const Row& b, const f32x16_t& c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ float dot(const Row& a, const Row& b) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s = fmaf(static_cast<float>(a[i]), static_cast<float>(b[i]), s);
        return s;
    }
};
template <>
struct AttnOp<false> {
    using G = float;
    using Row = f32x4_t;
    static constexpr int ES = 4;
    static constexpr int BN = 32;
    static __device__ __forceinline__ f32x16_t mma(const Row& a, const Row& b, f32x16_t c) {
#pragma unroll
        for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[i], b[i], c, 0, 0, 0);
        return c;
    }
    static __device__ __forceinline__ float dot(const Row& a, const Row& b) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) s = fmaf(a[i], b[i], s);
        return s;
    }
};

// A 32x32 accumulator as the B operand of a product over its rows.
template <bool BF16>
struct ColOp;
template <>
struct ColOp<true> {
    bf16x8_t x[2];  // rows 0..15 and 16..31
    __device__ __forceinline__ void set(const f32x16_t& a) {
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i >> 3][i & 7] = static_cast<__bf16>(a[i]);  // round to nearest even
    }
};
template <>
struct ColOp<false> {
    f32x16_t x;
    __device__ __forceinline__ void set(const f32x16_t& a) { x = a; }
};

// ---------------------------------------------------------------------------
// R rows of D elements in LDS, unpadded, written by the loads themselves
// (buffer_load ... lds, 16 bytes a lane, 1 KB a wave: lane l lands at the
// wave's base + 16 l).  Slot x of row r holds the row's 16-byte unit
// x ^ swz(r); the permutation is applied to the global address.  swz makes
// both kinds of read touch every LDS bank equally: row fragments (32 rows,
// one unit each) and column quads (four consecutive rows of 64 bytes).
// ---------------------------------------------------------------------------
template <bool BF16, int D>
struct AttnTile {
    using Op = AttnOp<BF16>;
    static constexpr int ROWB = D * Op::ES;
    static constexpr int U = ROWB / 16;    // 16-byte units a row
    static constexpr int RPI = 64 / U;     // rows one wave-wide load brings
    static constexpr int NF = U / 2;       // row fragments (one unit per half-wave) of a row
    static constexpr int ND = D / 32;      // 32-column blocks

    static __device__ __forceinline__ int swz(int r) {
        if constexpr (BF16) {
            if constexpr (U == 16) return ((r & 3) << 2) | ((r >> 2) & 3);
            if constexpr (U == 8) return (((r >> 1) & 1) << 2) | ((r >> 2) & 3);
            return (r >> 2) & 3;
        } else {
            if constexpr (U >= 16) return ((r & 7) << 1) | ((r >> 3) & 1);
            return (r >> 1) & 7;
        }
    }

    // Per-lane byte offsets of a wave's loads: even and odd passes (the swizzle
    // repeats every 16 rows; a pass of all waves may bring only 8).
    struct Src {
        int v[2];
    };
    template <int NW>
    static __device__ __forceinline__ Src src(int wave, int lane, int stride_bytes) {
        Src s;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int row = wave * RPI + lane / U;
            s.v[j] = row * stride_bytes + (((lane % U) ^ swz(row + j * RPI * NW)) << 4);
        }
        return s;
    }
    // rows [0, rows_left) of the tile at `base`; the rest of the R rows reads as zero
    template <int NW, int R>
    static __device__ __forceinline__ void stage(char* lds, const char* base, int rows_left, int stride_bytes,
                                                 const Src& s, int wave) {
        constexpr int PASS = RPI * NW;
        static_assert(R % PASS == 0 || PASS % R == 0, "whole passes, or one by some of the waves");
        if (R < PASS && wave * RPI >= R) return;
        const int rows = rows_left < R ? rows_left : R;
        const __amdgpu_buffer_rsrc_t rsrc = buffer_rsrc(base, rows > 0 ? (rows - 1) * stride_bytes + ROWB : 0);
#pragma unroll
        for (int j = 0; j < (R + PASS - 1) / PASS; ++j)
            load_lds16(rsrc, lds + (j * NW + wave) * 1024, s.v[j & 1], j * PASS * stride_bytes);
    }

    // byte offset of the lane's part of row fragment 0 of rows r0 .. r0 + 31 (r0 a multiple of 32)
    static __device__ __forceinline__ int row_at(int lane) {
        const int r = lane & 31;
        return r * ROWB + (((lane >> 5) ^ swz(r)) << 4);
    }
    static __device__ __forceinline__ typename Op::Row row(const char* t, int at, int r0, int kk) {
        return *reinterpret_cast<const typename Op::Row*>(t + r0 * ROWB + (at ^ (kk << 5)));
    }
    // acc += (rows r0 .. r0 + 31 of the tile) x (B given as its row fragments)
    static __device__ __forceinline__ f32x16_t rows_times(f32x16_t acc, const char* t, int at, int r0,
                                                          const typename Op::Row (&b)[NF]) {
#pragma unroll
        for (int kk = 0; kk < NF; ++kk) acc = Op::mma(row(t, at, r0, kk), b[kk], acc);
        return acc;
    }

    // column reads: byte offsets of the lane's two quads of column block 0, rows 0..15
    struct ColAt {
        int v[2];
    };
    static __device__ __forceinline__ ColAt col_at(int lane) {
        ColAt c;
        if constexpr (BF16) {
            const int i = lane & 15;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int r = 8 * j + 4 * (lane >> 5) + (i >> 2);
                const int u = 2 * ((lane >> 4) & 1) + ((i & 3) >> 1);
                c.v[j] = r * ROWB + ((u ^ swz(r)) << 4) + (i & 1) * 8;
            }
        } else {
            c.v[0] = (lane & 31) >> 2;
            c.v[1] = lane;
        }
        return c;
    }
    // acc += (columns 32 dt .. 32 dt + 31 of rows r0 .. r0 + 31)^T x (B over those rows); with
    // FINITE, non-finite elements of the tile count as zero
    template <bool FINITE = false>
    static __device__ __forceinline__ f32x16_t cols_times(f32x16_t acc, const char* t, const ColAt& at, int r0, int dt,
                                                          const ColOp<BF16>& b) {
        if constexpr (BF16) {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                bf16x8_t a;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const char* p = t + (r0 + 16 * s) * ROWB + (at.v[j] ^ (dt << 6));
                    const auto x = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((KDA_LDS bf16x4_t*)p);
#pragma unroll
                    for (int e = 0; e < 4; ++e) a[4 * j + e] = FINITE && !finite(x[e]) ? static_cast<__bf16>(0.f) : x[e];
                }
                acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b.x[s], acc, 0, 0, 0);
            }
        } else {
            const int lane = at.v[1];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int r = 8 * (i >> 2) + 4 * (lane >> 5) + (i & 3);
                float a = *reinterpret_cast<const float*>(t + (r0 + r) * ROWB + (((8 * dt + at.v[0]) ^ swz(r)) << 4) +
                                                          (lane & 3) * 4);
                if (FINITE && !finite(a)) a = 0.f;
                acc = __builtin_amdgcn_mfma_f32_32x32x2f32(a, b.x[i], acc, 0, 0, 0);
            }
        }
        return acc;
    }

    static __device__ __forceinline__ bool finite(__bf16 x) {
        return (__builtin_bit_cast(uint16_t, x) & 0x7F80) != 0x7F80;
    }
    static __device__ __forceinline__ bool finite(float x) { return (__float_as_uint(x) & 0x7F800000u) != 0x7F800000u; }

    // Whether any element of the tile's R rows is infinite or NaN (the same answer in every lane).
    template <int R>
    static __device__ __forceinline__ bool any_nonfinite(const char* t, int lane) {
        typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
        u16x2 m2 = {0, 0};
        unsigned m1 = 0;
#pragma unroll
        for (int i = 0; i < R * ROWB / 1024; ++i) {
            const u32x4_t x = *reinterpret_cast<const u32x4_t*>(t + i * 1024 + lane * 16);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if constexpr (BF16)
                    m2 = __builtin_elementwise_max(m2, __builtin_bit_cast(u16x2, x[e] & 0x7FFF7FFFu));
                else
                    m1 = __builtin_elementwise_max(m1, x[e] & 0x7FFFFFFFu);
            }
        }
        return __any(m2[0] >= 0x7F80 || m2[1] >= 0x7F80 || m1 >= 0x7F800000u);
    }

    // Adds the non-finite elements of tile row r to the accumulators of the columns (lanes) with `sees`.
    // A weight is positive, so its product with an infinity or NaN is that value.
    static __device__ __forceinline__ void add_nonfinite(f32x16_t (&acc)[ND], const char* t, int r, int half, bool sees) {
#pragma unroll
        for (int dt = 0; dt < ND; ++dt)
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
                const int byte = (32 * dt + 2 * i + 4 * half) * Op::ES;  // of four consecutive elements
                const char* p = t + r * ROWB + (((byte >> 4) ^ swz(r)) << 4) + (byte & 15);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float x;
                    bool bad;
                    if constexpr (BF16) {
                        const __bf16 y = (*reinterpret_cast<const bf16x4_t*>(p))[e];
                        x = static_cast<float>(y);
                        bad = !finite(y);
                    } else {
                        x = (*reinterpret_cast<const f32x4_t*>(p))[e];
                        bad = !finite(x);
                    }
                    if (bad && sees) acc[dt][i + e] += x;
                }
            }
    }
};

template <bool BF16, int D>
using RowFrags = typename AttnOp<BF16>::Row[AttnTile<BF16, D>::NF];

// The lane's row fragments of one row in global memory (zero if !live).
template <bool BF16, int D>
__device__ __forceinline__ void load_row_frags(RowFrags<BF16, D>& f,
                                               const typename AttnOp<BF16>::G* p, int half, bool live) {
    using Row = typename AttnOp<BF16>::Row;
    constexpr int E = 16 / AttnOp<BF16>::ES;
#pragma unroll
    for (int kk = 0; kk < AttnTile<BF16, D>::NF; ++kk) {
        Row x = {};
        if (live) x = *reinterpret_cast<const Row*>(p + (2 * kk + half) * E);
        f[kk] = x;
    }
}

// Rows of a [D x 32 columns] accumulator set (column = lane & 31) to global
// memory as the row `p` of its column: 16 contiguous bytes a lane for bf16.
template <bool BF16, int D>
__device__ __forceinline__ void store_col_as_row(typename AttnOp<BF16>::G* p, const f32x16_t (&acc)[D / 32], float mul,
                                                 int half, bool live) {
#pragma unroll
    for (int dt = 0; dt < D / 32; ++dt) {
        if constexpr (BF16) {
#pragma unroll
            for (int i = 0; i < 16; i += 8) {
                // quads i (columns 2i + 4 half ..) and i + 4: after the swaps the lower half-wave
                // holds 8 consecutive elements of the first, the upper of the second
                unsigned w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    bf16x4_t x;
                    x[0] = static_cast<__bf16>(acc[dt][i + 2 * e] * mul);
                    x[1] = static_cast<__bf16>(acc[dt][i + 2 * e + 1] * mul);
                    w[e] = __builtin_bit_cast(u32x2_t, x)[0];
                }
                const auto s0 = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
                const auto s1 = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
                const u32x4_t y = {s0[0], s1[0], s0[1], s1[1]};
                if (live) *reinterpret_cast<u32x4_t*>(p + 32 * dt + 2 * i + 8 * half) = y;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
                const f32x4_t y = {acc[dt][i] * mul, acc[dt][i + 1] * mul, acc[dt][i + 2] * mul, acc[dt][i + 3] * mul};
                if (live) *reinterpret_cast<f32x4_t*>(p + 32 * dt + 2 * i + 4 * half) = y;
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Four waves with accumulators of the same 32 columns and different shares of
// the reduction: their sum in wave 0, in a fixed order.  `lds`: 2 NA 4 KB.
// ---------------------------------------------------------------------------
template <int NA>
__device__ __forceinline__ void join_waves(f32x16_t (&acc)[NA], char* lds, int wave, int lane) {
#pragma unroll
    for (int w = 2; w >= 1; --w) {
        f32x4_t* p = reinterpret_cast<f32x4_t*>(lds) + (wave & (w - 1)) * NA * 256;
        __syncthreads();
        if (wave >= w && wave < 2 * w) {
#pragma unroll
            for (int n = 0; n < NA; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    p[(n * 4 + i) * 64 + lane] = f32x4_t{acc[n][4 * i], acc[n][4 * i + 1], acc[n][4 * i + 2], acc[n][4 * i + 3]};
        }
        __syncthreads();
        if (wave < w) {
#pragma unroll
            for (int n = 0; n < NA; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const f32x4_t y = p[(n * 4 + i) * 64 + lane];
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[n][4 * i + e] += y[e];
                }
        }
    }
}

// Every load so far has arrived, as the compiler knows too: without it the waits for the loads
// before a loop would be repeated inside it, where they hold up the loads into LDS.
__device__ __forceinline__ void loads_done() { __builtin_amdgcn_s_waitcnt(0x0F70); }

// All loads into LDS this wave issued have landed and its LDS reads are done;
// then every wave's.
__device__ __forceinline__ void lds_ready() {
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

}  // namespace kda
