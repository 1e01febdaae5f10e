// attn_backward.hip -- gradients of the causal softmax attention of
// attn_prefill.hip, gfx950.
//
// With p_ij = exp(s_ij - lse_i) and dp_ij = do_i . v_j,
//     D_i = do_i . o_i,           ds_ij = p_ij (dp_ij - D_i),
//     dq_i = scale sum_j ds_ij k_j,
//     dk_j = scale sum_h sum_i ds_ij q_i,   dv_j = sum_h sum_i p_ij do_i
// (h over the query heads of the key head).  Two launches: one walks the
// keys of a block of query rows (dq, and D_i on the way), the other the
// query rows of a block of keys (dk, dv).  Scores are formed in both, 7
// products instead of 5, and in return every sum has one owner and one
// order: no atomics, the same bits every time.  Both are laid out as the
// forward kernel, and bound by what feeds the matrix cores (16k tokens in 4
// sequences, 32/8 heads of 128, bf16: dq 1.0 ms for 3 products, 56 % busy;
// dk/dv 1.7 ms for 4, 43 % busy: two accumulators leave two waves a SIMD and
// no registers for a second tile's scores, so reads from LDS are waited for).
//
// D_i = do_i . o_i takes o as stored.  In bf16 its rounding matters where a
// row has few keys (o is then as large as v, and ds is too): the first 128
// rows of a sequence take D_i = sum_j p_ij dp_ij instead, the same number
// from unrounded weights (77 tokens, 128/64 channels: d_q 2.4e-3 from its
// value instead of 2.8e-3; 1.7e-3 is its own rounding).
#include <hip/hip_runtime.h>

#include "attn_device.hpp"
#include "attn_launch.hpp"

namespace kda {

namespace {

constexpr int kWaves = 4;
constexpr int kBM = 32 * kWaves;  // query rows (dq) or keys (dk, dv) of a workgroup

// Row statistics the dq pass leaves for the dk/dv pass, head-major:
// [H_q][T_tot] each of lse log2(e) and D.
struct Stats {
    float* lse2;
    float* D;
};

}  // namespace

template <bool BF16, int DK, int DV>
__global__ __launch_bounds__(256, BF16 || DK < 128 ? 2 : 1) void attn_bwd_dq_kernel(AttnBwdArgs b, float c, Stats stats) {
    using Op = AttnOp<BF16>;
    using KT = AttnTile<BF16, DK>;
    using VT = AttnTile<BF16, DV>;
    using G = typename Op::G;
    constexpr int BN = Op::BN;
    constexpr int KB = BN * KT::ROWB, VB = BN * VT::ROWB;
    __shared__ __attribute__((aligned(1024))) char lds[2][KB + VB];

    const AttnArgs& a = b.f;
    const int lane = threadIdx.x & 63, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int hp = blockIdx.x % a.Hq;
    const int group = a.Hq / a.Hkv;
    const int g = hp % a.Hkv, h = g * group + hp / a.Hkv;
    SeqTile st;
    if (!find_tile<kBM>(a.cu_seqlens, a.N, a.T_tot, blockIdx.x / a.Hq, false, st)) return;

    const int row0 = st.tile * kBM;
    const int wrow = row0 + 32 * wave;
    const int qi = wrow + (lane & 31);
    const bool live = qi < st.len;
    const size_t tok = static_cast<size_t>(st.beg) + (live ? qi : 0);

    RowFrags<BF16, DK> q;
    RowFrags<BF16, DV> d_o;
    load_row_frags<BF16, DK>(q, static_cast<const G*>(a.q) + tok * a.q_stride + static_cast<size_t>(h) * DK, half, live);
    load_row_frags<BF16, DV>(d_o, static_cast<const G*>(b.d_o) + (tok * a.Hq + h) * DV, half, live);
    float lse2 = 0.f, D = 0.f;
    {
        RowFrags<BF16, DV> o;
        load_row_frags<BF16, DV>(o, static_cast<const G*>(a.o) + (tok * a.Hq + h) * DV, half, live);
#pragma unroll
        for (int kk = 0; kk < VT::NF; ++kk) D += Op::dot(o[kk], d_o[kk]);
        D = half_sum(D);
        if (live) lse2 = a.lse[tok * a.Hq + h] * kLog2e;
    }
    const int ks = a.k_stride * Op::ES, vs = a.v_stride * Op::ES;
    const char* kb = static_cast<const char*>(a.k) + (static_cast<size_t>(st.beg) * a.k_stride + static_cast<size_t>(g) * DK) * Op::ES;
    const char* vb = static_cast<const char*>(a.v) + (static_cast<size_t>(st.beg) * a.v_stride + static_cast<size_t>(g) * DV) * Op::ES;
    const auto ksrc = KT::template src<kWaves>(wave, lane, ks);
    const auto vsrc = VT::template src<kWaves>(wave, lane, vs);
    const int kat = KT::row_at(lane), vat = VT::row_at(lane);
    const auto kct = KT::col_at(lane);

    const int last = st.len < row0 + kBM ? st.len : row0 + kBM;
    const int tiles = (last + BN - 1) / BN;
    const int wtiles = wrow < st.len ? (wrow + 31) / BN + 1 : 0;

    auto stage_tile = [&](int t) __attribute__((always_inline)) {
        char* l = lds[t & 1];
        KT::template stage<kWaves, BN>(l, kb + static_cast<size_t>(t) * BN * ks, st.len - t * BN, ks, ksrc, wave);
        VT::template stage<kWaves, BN>(l + KB, vb + static_cast<size_t>(t) * BN * vs, st.len - t * BN, vs, vsrc, wave);
    };

    if (BF16 && st.tile == 0) {  // D from the weights: the same walk over the keys, two or three tiles
        float sum = 0.f;
        stage_tile(0);
        loads_done();
        for (int t = 0; t < tiles; ++t) {
            lds_ready();
            if (t + 1 < tiles) stage_tile(t + 1);
            if (t >= wtiles) continue;
            const char* kt = lds[t & 1];
#pragma unroll 1
            for (int n = 0; n < BN / 32; ++n) {
                const f32x16_t s = KT::rows_times(f32x16_t{}, kt, kat, 32 * n, q);
                const f32x16_t dp = VT::rows_times(f32x16_t{}, kt + KB, vat, 32 * n, d_o);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float x = __builtin_amdgcn_exp2f(fmaf(s[i], c, -lse2)) * dp[i];
                    sum += t * BN + 32 * n + 8 * (i >> 2) + 4 * half + (i & 3) <= qi ? x : 0.f;
                }
            }
        }
        D = half_sum(sum);
        lds_ready();  // the tiles are read: they are filled again from the first
    }
    if (live && half == 0) {
        stats.lse2[static_cast<size_t>(h) * a.T_tot + tok] = lse2;
        stats.D[static_cast<size_t>(h) * a.T_tot + tok] = D;
    }

    f32x16_t dq[KT::ND];
#pragma unroll
    for (int dt = 0; dt < KT::ND; ++dt) dq[dt] = f32x16_t{};

    stage_tile(0);
    loads_done();
    for (int t = 0; t < tiles; ++t) {
        lds_ready();
        if (t + 1 < tiles) stage_tile(t + 1);
        if (t >= wtiles) continue;
        const char* kt = lds[t & 1];
        const char* vt = kt + KB;
        const bool diagonal = t * BN + BN - 1 > wrow;
#pragma unroll
        for (int n = 0; n < BN / 32; ++n) {
            f32x16_t s = KT::rows_times(f32x16_t{}, kt, kat, 32 * n, q);
            const f32x16_t dp = VT::rows_times(f32x16_t{}, vt, vat, 32 * n, d_o);
#pragma unroll
            for (int i = 0; i < 16; ++i) s[i] = __builtin_amdgcn_exp2f(fmaf(s[i], c, -lse2)) * (dp[i] - D);
            if (diagonal) {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int key = t * BN + 32 * n + 8 * (i >> 2) + 4 * half + (i & 3);
                    s[i] = key <= qi ? s[i] : 0.f;
                }
            }
            ColOp<BF16> ds;
            ds.set(s);
#pragma unroll
            for (int dt = 0; dt < KT::ND; ++dt) dq[dt] = KT::cols_times(dq[dt], kt, kct, 32 * n, dt, ds);
        }
    }
    store_col_as_row<BF16, DK>(static_cast<G*>(b.d_q) + (tok * a.Hq + h) * DK, dq, a.scale, half, live);
}

template <bool BF16, int DK, int DV>
__global__ __launch_bounds__(256, BF16 || DK + DV <= 128 ? 2 : 1) void attn_bwd_dkv_kernel(AttnBwdArgs b, float c, Stats stats) {
    using Op = AttnOp<BF16>;
    using QT = AttnTile<BF16, DK>;
    using OT = AttnTile<BF16, DV>;
    using G = typename Op::G;
    constexpr int BN = 32;
    // The values' fragments of bf16 are read from LDS each time: with both accumulators and the
    // keys' fragments in registers they would leave one wave a SIMD (128 + 128 channels, 16k packed
    // tokens: 2.35 ms, against 1.91 ms with two, either before the loads were written out).
    constexpr bool V_LDS = BF16;
    constexpr int QB = BN * QT::ROWB, OB = BN * OT::ROWB;
    constexpr int SB = 256;  // bytes of one statistic of a tile: a wave-wide load brings 64 floats
    __shared__ __attribute__((aligned(1024))) char lds[2][QB + OB + 2 * SB];
    __shared__ __attribute__((aligned(1024))) char ldsv[V_LDS ? kBM * OT::ROWB : 16];

    const AttnArgs& a = b.f;
    const int lane = threadIdx.x & 63, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int g = blockIdx.x % a.Hkv;
    const int group = a.Hq / a.Hkv;
    SeqTile st;
    if (!find_tile<kBM>(a.cu_seqlens, a.N, a.T_tot, blockIdx.x / a.Hkv, true, st)) return;

    const int key0 = st.tile * kBM;
    const int wkey = key0 + 32 * wave;
    const int kj = wkey + (lane & 31);  // the lane's key in its sequence
    const bool live = kj < st.len;
    const size_t tok = static_cast<size_t>(st.beg) + (live ? kj : 0);

    RowFrags<BF16, DK> k;
    RowFrags<BF16, DV> v;
    load_row_frags<BF16, DK>(k, static_cast<const G*>(a.k) + tok * a.k_stride + static_cast<size_t>(g) * DK, half, live);
    if constexpr (V_LDS) {
        const int vs = a.v_stride * Op::ES;
        OT::template stage<kWaves, kBM>(ldsv, static_cast<const char*>(a.v) + ((static_cast<size_t>(st.beg) + key0) * a.v_stride +
                                                                               static_cast<size_t>(g) * DV) * Op::ES,
                                        st.len - key0, vs, OT::template src<kWaves>(wave, lane, vs), wave);
    } else {
        load_row_frags<BF16, DV>(v, static_cast<const G*>(a.v) + tok * a.v_stride + static_cast<size_t>(g) * DV, half, live);
    }

    const int qs = a.q_stride * Op::ES, os = a.Hq * DV * Op::ES;
    const auto qsrc = QT::template src<kWaves>(wave, lane, qs);
    const auto osrc = OT::template src<kWaves>(wave, lane, os);
    const int qat = QT::row_at(lane), oat = OT::row_at(lane);
    const auto qct = QT::col_at(lane);
    const auto oct = OT::col_at(lane);

    // query tiles t0 .. t1 - 1 of every head of the group, one after another
    const int t0 = key0 / BN, t1 = (st.len + BN - 1) / BN;
    const int wt0 = wkey / BN;  // the wave's first

    auto stage_tile = [&](int slot, int hh, int t) __attribute__((always_inline)) {
        char* l = lds[slot];
        const int h = g * group + hh;
        const size_t r = static_cast<size_t>(st.beg) + static_cast<size_t>(t) * BN;
        const int left = st.len - t * BN;
        QT::template stage<kWaves, BN>(l, static_cast<const char*>(a.q) + (r * a.q_stride + static_cast<size_t>(h) * DK) * Op::ES,
                                       left, qs, qsrc, wave);
        OT::template stage<kWaves, BN>(l + QB, static_cast<const char*>(b.d_o) + (r * a.Hq + h) * DV * Op::ES, left, os, osrc, wave);
        if (wave < 2) {
            const float* p = (wave == 0 ? stats.lse2 : stats.D) + static_cast<size_t>(h) * a.T_tot + r;
            load_lds4(buffer_rsrc(p, (left < BN ? left : BN) * 4), l + QB + OB + wave * SB, lane * 4, 0);
        }
    };

    f32x16_t dk[QT::ND], dv[OT::ND];
#pragma unroll
    for (int dt = 0; dt < QT::ND; ++dt) dk[dt] = f32x16_t{};
#pragma unroll
    for (int dt = 0; dt < OT::ND; ++dt) dv[dt] = f32x16_t{};

    int hh = 0, t = t0, slot = 0;
    stage_tile(0, 0, t0);
    loads_done();
    while (hh < group) {
        int nh = hh, nt = t + 1;
        if (nt == t1) {
            nt = t0;
            ++nh;
        }
        lds_ready();
        if (nh < group) stage_tile(slot ^ 1, nh, nt);
        if (t >= wt0 && wkey < st.len) {
            const char* qt = lds[slot];
            const char* ot = qt + QB;
            const float* sl = reinterpret_cast<const float*>(ot + OB);
            const float* sd = sl + SB / 4;
            const bool diagonal = t * BN < wkey + 31;
#pragma unroll
            for (int n = 0; n < BN / 32; ++n) {
                f32x16_t s = QT::rows_times(f32x16_t{}, qt, qat, 32 * n, k);
                f32x16_t dp = {};
#pragma unroll
                for (int kk = 0; kk < OT::NF; ++kk)
                    dp = Op::mma(OT::row(ot, oat, 32 * n, kk), V_LDS ? OT::row(ldsv, oat, 32 * wave, kk) : v[kk], dp);
#pragma unroll
                for (int i4 = 0; i4 < 4; ++i4) {
                    const f32x4_t l2 = *reinterpret_cast<const f32x4_t*>(sl + 32 * n + 8 * i4 + 4 * half);
                    const f32x4_t dd = *reinterpret_cast<const f32x4_t*>(sd + 32 * n + 8 * i4 + 4 * half);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int i = 4 * i4 + e;
                        s[i] = __builtin_amdgcn_exp2f(fmaf(s[i], c, -l2[e]));
                        dp[i] = s[i] * (dp[i] - dd[e]);
                    }
                }
                if (diagonal) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int row = t * BN + 32 * n + 8 * (i >> 2) + 4 * half + (i & 3);
                        s[i] = kj <= row ? s[i] : 0.f;
                        dp[i] = kj <= row ? dp[i] : 0.f;
                    }
                }
                ColOp<BF16> p, ds;
                p.set(s);
                ds.set(dp);
#pragma unroll
                for (int dt = 0; dt < OT::ND; ++dt) dv[dt] = OT::cols_times(dv[dt], ot, oct, 32 * n, dt, p);
#pragma unroll
                for (int dt = 0; dt < QT::ND; ++dt) dk[dt] = QT::cols_times(dk[dt], qt, qct, 32 * n, dt, ds);
            }
        }
        hh = nh;
        t = nt;
        slot ^= 1;
    }
    store_col_as_row<BF16, DK>(static_cast<G*>(b.d_k) + (tok * a.Hkv + g) * DK, dk, a.scale, half, live);
    store_col_as_row<BF16, DV>(static_cast<G*>(b.d_v) + (tok * a.Hkv + g) * DV, dv, 1.f, half, live);
}

// The same two for batches that leave compute units idle: 32 rows (or keys) a
// workgroup, its four waves on every fourth 32-key (or 32-row) tile, their
// sums joined at the end.  Bound by the chain of the longest sequence (513
// tokens of 924 in 5 sequences, 8/2 fp32 heads of 64: dq 25 us, dk/dv 34 us;
// an fp32 MFMA of this shape takes 64 cycles and carries 2 channels).
template <bool BF16, int DK, int DV>
__global__ __launch_bounds__(256, 1) void attn_bwd_dq_split_kernel(AttnBwdArgs b, float c, Stats stats) {
    using Op = AttnOp<BF16>;
    using KT = AttnTile<BF16, DK>;
    using VT = AttnTile<BF16, DV>;
    using G = typename Op::G;
    constexpr int TG = 32 * kWaves;
    constexpr int KB = TG * KT::ROWB, VB = TG * VT::ROWB;
    constexpr int NBUF = 2 * (KB + VB) <= 128 * 1024 ? 2 : 1;
    constexpr int JOIN = 2 * KT::ND * 4096;
    __shared__ __attribute__((aligned(1024))) char lds[NBUF * (KB + VB) > JOIN ? NBUF * (KB + VB) : JOIN];
    __shared__ float s_D[kWaves][32];

    const AttnArgs& a = b.f;
    const int lane = threadIdx.x & 63, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int hp = blockIdx.x % a.Hq;
    const int group = a.Hq / a.Hkv;
    const int g = hp % a.Hkv, h = g * group + hp / a.Hkv;
    SeqTile st;
    if (!find_tile<32>(a.cu_seqlens, a.N, a.T_tot, blockIdx.x / a.Hq, false, st)) return;

    const int row0 = st.tile * 32;
    const int qi = row0 + (lane & 31);
    const bool live = qi < st.len;
    const size_t tok = static_cast<size_t>(st.beg) + (live ? qi : 0);
    const int ks = a.k_stride * Op::ES, vs = a.v_stride * Op::ES;
    const char* kb = static_cast<const char*>(a.k) + (static_cast<size_t>(st.beg) * a.k_stride + static_cast<size_t>(g) * DK) * Op::ES;
    const char* vb = static_cast<const char*>(a.v) + (static_cast<size_t>(st.beg) * a.v_stride + static_cast<size_t>(g) * DV) * Op::ES;
    const auto ksrc = KT::template src<kWaves>(wave, lane, ks);
    const auto vsrc = VT::template src<kWaves>(wave, lane, vs);
    const int kat = KT::row_at(lane), vat = VT::row_at(lane);
    const auto kct = KT::col_at(lane);
    auto stage_group = [&](int t) __attribute__((always_inline)) {
        char* l = lds + (NBUF == 2 ? t & 1 : 0) * (KB + VB);
        KT::template stage<kWaves, TG>(l, kb + static_cast<size_t>(t) * TG * ks, st.len - t * TG, ks, ksrc, wave);
        VT::template stage<kWaves, TG>(l + KB, vb + static_cast<size_t>(t) * TG * vs, st.len - t * TG, vs, vsrc, wave);
    };
    stage_group(0);

    RowFrags<BF16, DK> q;
    RowFrags<BF16, DV> d_o;
    load_row_frags<BF16, DK>(q, static_cast<const G*>(a.q) + tok * a.q_stride + static_cast<size_t>(h) * DK, half, live);
    load_row_frags<BF16, DV>(d_o, static_cast<const G*>(b.d_o) + (tok * a.Hq + h) * DV, half, live);
    float lse2 = 0.f, D = 0.f;
    {
        RowFrags<BF16, DV> o;
        load_row_frags<BF16, DV>(o, static_cast<const G*>(a.o) + (tok * a.Hq + h) * DV, half, live);
#pragma unroll
        for (int kk = 0; kk < VT::NF; ++kk) D += Op::dot(o[kk], d_o[kk]);
        D = half_sum(D);
        if (live) lse2 = a.lse[tok * a.Hq + h] * kLog2e;
    }
    f32x16_t dq[KT::ND];
#pragma unroll
    for (int dt = 0; dt < KT::ND; ++dt) dq[dt] = f32x16_t{};
    const int groups = (row0 + TG) / TG;
    auto put_stats = [&]() __attribute__((always_inline)) {
        if (live && half == 0 && wave == 0) {
            stats.lse2[static_cast<size_t>(h) * a.T_tot + tok] = lse2;
            stats.D[static_cast<size_t>(h) * a.T_tot + tok] = D;
        }
    };
    const bool few = BF16 && row0 < TG;  // one group of keys: D from the weights, which are all here
    if (!few) put_stats();
    loads_done();
    for (int t = 0; t < groups; ++t) {
        lds_ready();
        if (NBUF == 2 && t + 1 < groups) stage_group(t + 1);
        const int key0 = t * TG + 32 * wave;
        const bool mine = key0 <= row0;
        const char* kt = lds + (NBUF == 2 ? t & 1 : 0) * (KB + VB);
        f32x16_t s = {}, dp = {};
        if (mine) {
            s = KT::rows_times(s, kt, kat, 32 * wave, q);
            dp = VT::rows_times(dp, kt + KB, vat, 32 * wave, d_o);
#pragma unroll
            for (int i = 0; i < 16; ++i) s[i] = __builtin_amdgcn_exp2f(fmaf(s[i], c, -lse2));
            if (key0 == row0) {
#pragma unroll
                for (int i = 0; i < 16; ++i) s[i] = key0 + 8 * (i >> 2) + 4 * half + (i & 3) <= qi ? s[i] : 0.f;
            }
        }
        if (few) {  // the same for every wave
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) sum += s[i] != 0.f ? s[i] * dp[i] : 0.f;
            sum = half_sum(sum);
            if (half == 0) s_D[wave][lane] = sum;
            __syncthreads();
            D = 0.f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) D += s_D[w][lane & 31];
            put_stats();
        }
        if (mine) {
            // a weight of zero: what stands behind the mask may be anything
#pragma unroll
            for (int i = 0; i < 16; ++i) s[i] = s[i] != 0.f ? s[i] * (dp[i] - D) : 0.f;
            ColOp<BF16> ds;
            ds.set(s);
#pragma unroll
            for (int dt = 0; dt < KT::ND; ++dt) dq[dt] = KT::cols_times(dq[dt], kt, kct, 32 * wave, dt, ds);
        }
        if (NBUF == 1 && t + 1 < groups) {
            lds_ready();
            stage_group(t + 1);
        }
    }
    join_waves(dq, lds, wave, lane);
    if (wave == 0) store_col_as_row<BF16, DK>(static_cast<G*>(b.d_q) + (tok * a.Hq + h) * DK, dq, a.scale, half, live);
}

template <bool BF16, int DK, int DV>
__global__ __launch_bounds__(256, 1) void attn_bwd_dkv_split_kernel(AttnBwdArgs b, float c, Stats stats) {
    using Op = AttnOp<BF16>;
    using QT = AttnTile<BF16, DK>;
    using OT = AttnTile<BF16, DV>;
    using G = typename Op::G;
    constexpr int TG = 32 * kWaves;  // query rows the waves take together
    constexpr int QB = TG * QT::ROWB, OB = TG * OT::ROWB, SB = TG * 4;
    constexpr int NBUF = 2 * (QB + OB + 2 * SB) <= 144 * 1024 ? 2 : 1;
    constexpr int SLOT = (QB + OB + 2 * SB + 1023) / 1024 * 1024;
    constexpr int JOIN = 2 * 4096 * (QT::ND > OT::ND ? QT::ND : OT::ND);
    __shared__ __attribute__((aligned(1024))) char lds[NBUF * SLOT > JOIN ? NBUF * SLOT : JOIN];

    const AttnArgs& a = b.f;
    const int lane = threadIdx.x & 63, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int g = blockIdx.x % a.Hkv;
    const int group = a.Hq / a.Hkv;
    // the query heads of this workgroup, of those of the key head
    const int h0 = group * blockIdx.y / b.head_parts, heads = group * (blockIdx.y + 1) / b.head_parts - h0;
    SeqTile st;
    if (!find_tile<32>(a.cu_seqlens, a.N, a.T_tot, blockIdx.x / a.Hkv, true, st)) return;

    const int key0 = st.tile * 32;
    const int kj = key0 + (lane & 31);
    const bool live = kj < st.len;
    const size_t tok = static_cast<size_t>(st.beg) + (live ? kj : 0);
    const int qs = a.q_stride * Op::ES, os = a.Hq * DV * Op::ES;
    const auto qsrc = QT::template src<kWaves>(wave, lane, qs);
    const auto osrc = OT::template src<kWaves>(wave, lane, os);
    const int qat = QT::row_at(lane), oat = OT::row_at(lane);
    const auto qct = QT::col_at(lane);
    const auto oct = OT::col_at(lane);

    const int first = key0 / TG, groups = (st.len + TG - 1) / TG - first;  // row groups of a head
    auto stage_group = [&](int slot, int hh, int t) __attribute__((always_inline)) {
        char* l = lds + slot * SLOT;
        const int h = g * group + h0 + hh;
        const size_t r = static_cast<size_t>(st.beg) + static_cast<size_t>(t) * TG;
        const int left = st.len - t * TG;
        QT::template stage<kWaves, TG>(l, static_cast<const char*>(a.q) + (r * a.q_stride + static_cast<size_t>(h) * DK) * Op::ES, left,
                                       qs, qsrc, wave);
        OT::template stage<kWaves, TG>(l + QB, static_cast<const char*>(b.d_o) + (r * a.Hq + h) * DV * Op::ES, left, os, osrc, wave);
        // two waves a statistic, 64 rows each
        const float* p = (wave < 2 ? stats.lse2 : stats.D) + static_cast<size_t>(h) * a.T_tot + r;
        load_lds4(buffer_rsrc(p, (left < TG ? left : TG) * 4), l + QB + OB + wave * 256, ((wave & 1) * 64 + lane) * 4, 0);
    };
    stage_group(0, 0, first);

    RowFrags<BF16, DK> k;
    RowFrags<BF16, DV> v;
    load_row_frags<BF16, DK>(k, static_cast<const G*>(a.k) + tok * a.k_stride + static_cast<size_t>(g) * DK, half, live);
    load_row_frags<BF16, DV>(v, static_cast<const G*>(a.v) + tok * a.v_stride + static_cast<size_t>(g) * DV, half, live);
    f32x16_t dk[QT::ND], dv[OT::ND];
#pragma unroll
    for (int dt = 0; dt < QT::ND; ++dt) dk[dt] = f32x16_t{};
#pragma unroll
    for (int dt = 0; dt < OT::ND; ++dt) dv[dt] = f32x16_t{};

    const int steps = groups * heads;
    int hh = 0, t = first, slot = 0;
    loads_done();
    for (int n = 0; n < steps; ++n) {
        int nh = hh, nt = t + 1;
        if (nt == first + groups) {
            nt = first;
            ++nh;
        }
        lds_ready();
        if (NBUF == 2 && n + 1 < steps) stage_group(slot ^ 1, nh, nt);
        const int r0 = t * TG + 32 * wave;  // the wave's first row
        if (r0 >= key0 && r0 < st.len) {
            const char* qt = lds + slot * SLOT;
            const char* ot = qt + QB;
            const float* sl = reinterpret_cast<const float*>(ot + OB) + 32 * wave;
            const float* sd = sl + TG;
            f32x16_t s = QT::rows_times(f32x16_t{}, qt, qat, 32 * wave, k);
            f32x16_t dp = OT::rows_times(f32x16_t{}, ot, oat, 32 * wave, v);
#pragma unroll
            for (int i4 = 0; i4 < 4; ++i4) {
                const f32x4_t l2 = *reinterpret_cast<const f32x4_t*>(sl + 8 * i4 + 4 * half);
                const f32x4_t dd = *reinterpret_cast<const f32x4_t*>(sd + 8 * i4 + 4 * half);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int i = 4 * i4 + e;
                    s[i] = __builtin_amdgcn_exp2f(fmaf(s[i], c, -l2[e]));
                    dp[i] = s[i] * (dp[i] - dd[e]);
                }
            }
            if (r0 == key0) {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const bool sees = kj <= r0 + 8 * (i >> 2) + 4 * half + (i & 3);
                    s[i] = sees ? s[i] : 0.f;
                    dp[i] = sees ? dp[i] : 0.f;
                }
            }
            ColOp<BF16> p, ds;
            p.set(s);
            ds.set(dp);
#pragma unroll
            for (int dt = 0; dt < OT::ND; ++dt) dv[dt] = OT::cols_times(dv[dt], ot, oct, 32 * wave, dt, p);
#pragma unroll
            for (int dt = 0; dt < QT::ND; ++dt) dk[dt] = QT::cols_times(dk[dt], qt, qct, 32 * wave, dt, ds);
        }
        if (NBUF == 1 && n + 1 < steps) {
            lds_ready();
            stage_group(0, nh, nt);
        }
        hh = nh;
        t = nt;
        if (NBUF == 2) slot ^= 1;
    }
    join_waves(dk, lds, wave, lane);
    join_waves(dv, lds, wave, lane);
    if (wave != 0) return;
    if (b.head_parts > 1) {
        float* p = b.parts + ((static_cast<size_t>(blockIdx.y) * a.T_tot + tok) * a.Hkv + g) * (DK + DV);
        store_col_as_row<false, DK>(p, dk, a.scale, half, live);
        store_col_as_row<false, DV>(p + DK, dv, 1.f, half, live);
        return;
    }
    store_col_as_row<BF16, DK>(static_cast<G*>(b.d_k) + (tok * a.Hkv + g) * DK, dk, a.scale, half, live);
    store_col_as_row<BF16, DV>(static_cast<G*>(b.d_v) + (tok * a.Hkv + g) * DV, dv, 1.f, half, live);
}

// Sums the parts of dk and dv that the workgroups of different query heads left, in their order.
template <bool BF16, int DK, int DV>
__global__ __launch_bounds__(256) void attn_bwd_join_kernel(AttnBwdArgs b) {
    using T = Elem<BF16>;
    const AttnArgs& a = b.f;
    const int g = blockIdx.x % a.Hkv;
    SeqTile st;
    if (!find_tile<32>(a.cu_seqlens, a.N, a.T_tot, blockIdx.x / a.Hkv, true, st)) return;
    constexpr int Q = (DK + DV) / 4;
    for (int x = threadIdx.x; x < 32 * Q; x += 256) {
        const int row = st.tile * 32 + x / Q, e = 4 * (x % Q);
        if (row >= st.len) return;
        const size_t at = (static_cast<size_t>(st.beg) + row) * a.Hkv + g;
        const float* p = b.parts + at * (DK + DV) + e;
        float y[4] = {0.f, 0.f, 0.f, 0.f};
        for (int s = 0; s < b.head_parts; ++s) {
            const f32x4_t z = *reinterpret_cast<const f32x4_t*>(p + static_cast<size_t>(s) * a.T_tot * a.Hkv * (DK + DV));
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] += z[i];
        }
        T::store4(e < DK ? static_cast<typename T::G*>(b.d_k) + at * DK + e : static_cast<typename T::G*>(b.d_v) + at * DV + e - DK, y);
    }
}

namespace {

template <bool BF16, int DK, int DV>
hipError_t launch(const AttnBwdArgs& b) {
    const AttnArgs& a = b.f;
    const int64_t units = (static_cast<int64_t>(a.T_tot) + kBM - 1) / kBM + a.N;
    const size_t n = static_cast<size_t>(a.T_tot) * a.Hq;
    const Stats stats{static_cast<float*>(b.workspace), static_cast<float*>(b.workspace) + n};
    const hipStream_t st = static_cast<hipStream_t>(a.stream);
    const float c = a.scale * kLog2e;
    const int64_t units32 = (static_cast<int64_t>(a.T_tot) + 31) / 32 + a.N;
    const dim3 threads(64 * kWaves);
    if (a.split)
        hipLaunchKernelGGL((attn_bwd_dq_split_kernel<BF16, DK, DV>), dim3(static_cast<unsigned>(units32 * a.Hq)), threads, 0, st, b, c, stats);
    else
        hipLaunchKernelGGL((attn_bwd_dq_kernel<BF16, DK, DV>), dim3(static_cast<unsigned>(units * a.Hq)), threads, 0, st, b, c, stats);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (b.head_parts > 1) {
        hipLaunchKernelGGL((attn_bwd_dkv_split_kernel<BF16, DK, DV>), dim3(static_cast<unsigned>(units32 * a.Hkv), b.head_parts), threads,
                           0, st, b, c, stats);
        const hipError_t e2 = hipGetLastError();
        if (e2 != hipSuccess) return e2;
        hipLaunchKernelGGL((attn_bwd_join_kernel<BF16, DK, DV>), dim3(static_cast<unsigned>(units32 * a.Hkv)), dim3(256), 0, st, b);
    } else if (b.head_parts == 1)
        hipLaunchKernelGGL((attn_bwd_dkv_split_kernel<BF16, DK, DV>), dim3(static_cast<unsigned>(units32 * a.Hkv)), threads, 0, st, b, c, stats);
    else
        hipLaunchKernelGGL((attn_bwd_dkv_kernel<BF16, DK, DV>), dim3(static_cast<unsigned>(units * a.Hkv)), threads, 0, st, b, c, stats);
    return hipGetLastError();
}

template <bool BF16, int DK>
hipError_t launch_dv(const AttnBwdArgs& b) {
    switch (b.f.d_v) {
        case 32: return launch<BF16, DK, 32>(b);
        case 64: return launch<BF16, DK, 64>(b);
        default: return launch<BF16, DK, 128>(b);
    }
}

template <bool BF16>
hipError_t launch_dk(const AttnBwdArgs& b) {
    switch (b.f.d_k) {
        case 32: return launch_dv<BF16, 32>(b);
        case 64: return launch_dv<BF16, 64>(b);
        default: return launch_dv<BF16, 128>(b);
    }
}

}  // namespace

// Where even the split blocks of the key heads leave compute units idle, the query heads of a key
// head go to several workgroups and their sums are joined (5 ragged fp32 sequences of 924 tokens,
// 8/2 heads of 64: dk/dv 107 us in one part, 34 us and 7 to join in four).
BwdPlan attn_bwd_plan(int32_t N, int64_t T_tot, int32_t Hq, int32_t Hkv, int32_t d_k, int32_t d_v, bool bf16, int cus) {
    BwdPlan p;
    p.stats_bytes = (static_cast<size_t>(T_tot) * Hq * 2 * sizeof(float) + 255) / 256 * 256;
    p.head_parts = 0;
    p.bytes = p.stats_bytes;
    if (T_tot > 0 && attn_split(N, T_tot, Hkv, bf16, cus)) {
        const int64_t blocks = ((T_tot + 31) / 32 + N) * Hkv;
        const int64_t parts = 2 * static_cast<int64_t>(cus) / blocks, group = Hq / Hkv;
        p.head_parts = static_cast<int32_t>(parts < 1 ? 1 : parts > group ? group : parts);
        if (p.head_parts > 1) p.bytes += static_cast<size_t>(p.head_parts) * T_tot * Hkv * (d_k + d_v) * sizeof(float);
    }
    return p;
}

hipError_t launch_attn_bwd(const AttnBwdArgs& b) {
    if (b.f.T_tot == 0) return hipSuccess;
    return b.f.bf16 ? launch_dk<true>(b) : launch_dk<false>(b);
}

}  // namespace kda
