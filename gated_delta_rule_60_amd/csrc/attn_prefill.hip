// attn_prefill.hip -- causal softmax attention over packed prompts, gfx950.
//
// For row i of a sequence and query head h (key head g = h / (Hq / Hkv)):
//     s_ij = scale q_i . k_j (j <= i),  lse_i = ln sum_j exp(s_ij),
//     o_i = sum_j exp(s_ij - lse_i) v_j.
// One pass over the keys: with m the running maximum, l = sum exp(s - m) and
// O = sum exp(s - m) v_j, a new tile adds to l and O, and both are rescaled
// only when m rises.
//
// Long prompts are bound by the matrix cores: 2 (d_k + d_v) products a (row,
// key) pair against bytes that grow with the rows only.  A workgroup has 128
// rows of one head, 32 a wave, so that K and V tiles are read from LDS once
// for 32 rows; S^T = K Q^T gives a lane one query row, whose statistics need
// no shuffles, and P^T is the next product's operand as it stands.  The two
// products of a step depend on each other through the exponentials; the next
// tile's scores are formed in between (32k tokens in 8 prompts, 32/8 heads of
// 128, bf16: 1.45 ms, 1030 TFLOP/s; one prompt of 16k, 16 heads: 1.0 ms, 1100
// TFLOP/s, the matrix cores busy 61 % of the time at the 1.63 GHz that they
// leave the chip).
#include <hip/hip_runtime.h>

#include <type_traits>

#include "attn_device.hpp"
#include "attn_launch.hpp"

namespace kda {

namespace {

constexpr int kWaves = 4;
constexpr int kBM = 32 * kWaves;  // query rows of a workgroup
// The running maximum is moved (and O, l rescaled) only when a row's scores
// exceed it by more than this many powers of two: p then stays below 2^8,
// where bf16 and fp32 hold it as exactly as below 1.
constexpr float kLazyLog2 = 8.f;
// Where it starts: below every score but -infinity, which a product past the range of fp32 gives and
// which weighs nothing (2^(-inf - kLowest) = 0, where -inf - -inf would be NaN for the whole row).
constexpr float kLowest = -3.402823466e38f;

}  // namespace

template <bool BF16, int DK, int DV>
__global__ __launch_bounds__(256, 2) void attn_prefill_kernel(AttnArgs a, float c /* scale log2(e) */) {
    using Op = AttnOp<BF16>;
    using KT = AttnTile<BF16, DK>;
    using VT = AttnTile<BF16, DV>;
    using G = typename Op::G;
    constexpr int BN = Op::BN, NS = BN / 32;
    constexpr int KB = BN * KT::ROWB, VB = BN * VT::ROWB;
    __shared__ __attribute__((aligned(1024))) char lds[2][KB + VB];

    const int lane = threadIdx.x & 63, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // consecutive workgroups take consecutive key heads: a key head's workgroups share an XCD's
    // L2 when Hkv is a multiple of the 8 XCDs they are dealt to
    const int hp = blockIdx.x % a.Hq;
    const int group = a.Hq / a.Hkv;
    const int g = hp % a.Hkv, h = g * group + hp / a.Hkv;
    SeqTile st;
    if (!find_tile<kBM>(a.cu_seqlens, a.N, a.T_tot, blockIdx.x / a.Hq, false, st)) return;

    const int row0 = st.tile * kBM;
    const int qi = row0 + 32 * wave + (lane & 31);  // the lane's query row in its sequence
    const bool live = qi < st.len;
    const size_t tok = static_cast<size_t>(st.beg) + (live ? qi : 0);

    typename Op::Row q[KT::NF];
    load_row_frags<BF16, DK>(q, static_cast<const G*>(a.q) + tok * a.q_stride + static_cast<size_t>(h) * DK, half, live);

    const int ks = a.k_stride * Op::ES, vs = a.v_stride * Op::ES;
    const char* kb = static_cast<const char*>(a.k) + (static_cast<size_t>(st.beg) * a.k_stride + static_cast<size_t>(g) * DK) * Op::ES;
    const char* vb = static_cast<const char*>(a.v) + (static_cast<size_t>(st.beg) * a.v_stride + static_cast<size_t>(g) * DV) * Op::ES;
    const auto ksrc = KT::template src<kWaves>(wave, lane, ks);
    const auto vsrc = VT::template src<kWaves>(wave, lane, vs);
    const int kat = KT::row_at(lane);
    const auto vat = VT::col_at(lane);

    const int last = st.len < row0 + kBM ? st.len : row0 + kBM;
    const int tiles = (last + BN - 1) / BN;
    const int wrow = row0 + 32 * wave;               // the wave's first row
    const int wtiles = wrow < st.len ? (wrow + 31) / BN + 1 : 0;  // tiles it needs

    // Keys go two tiles ahead, values one: while a tile's weights are formed, the next tile's scores
    // are (below), so its keys are needed a step earlier.
    auto stage_k = [&](int t) __attribute__((always_inline)) {
        KT::template stage<kWaves, BN>(lds[t & 1], kb + static_cast<size_t>(t) * BN * ks, st.len - t * BN, ks, ksrc, wave);
    };
    auto stage_v = [&](int t) __attribute__((always_inline)) {
        VT::template stage<kWaves, BN>(lds[t & 1] + KB, vb + static_cast<size_t>(t) * BN * vs, st.len - t * BN, vs, vsrc, wave);
    };

    f32x16_t o[VT::ND];
#pragma unroll
    for (int dt = 0; dt < VT::ND; ++dt) o[dt] = f32x16_t{};
    float mc = kLowest;  // running maximum of c s
    float l = 0.f;         // this half-wave's part of the row's sum

    auto scores = [&](int t, f32x16_t (&s)[NS]) __attribute__((always_inline)) {
#pragma unroll
        for (int n = 0; n < NS; ++n) s[n] = KT::rows_times(f32x16_t{}, lds[t & 1], kat, 32 * n, q);
    };
    // One tile's scores into the row's statistics and O.  LAST: the wave's last tile, which holds the
    // diagonal; otherwise the next tile's scores go to `s1`, between the two dependent halves of the
    // step: their products run while the weights are formed.
    auto step = [&](int t, f32x16_t (&s)[NS], f32x16_t (&s1)[NS], auto LAST) __attribute__((always_inline)) {
        const char* vt = lds[t & 1] + KB;
        if constexpr (LAST) {
#pragma unroll
            for (int n = 0; n < NS; ++n)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int key = t * BN + 32 * n + 8 * (i >> 2) + 4 * half + (i & 3);
                    s[n][i] = key <= qi ? s[n][i] : -INFINITY;
                }
        }
        float mx = s[0][0];
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
            for (int i = 0; i < 16; ++i) mx = fmaxf(mx, s[n][i]);
        mx = half_max(mx) * c;
        if (__any(mx > mc + kLazyLog2)) {
            // by row: what a row gives does not depend on the rows beside it
            const float m1 = mx > mc + kLazyLog2 ? mx : mc;
            const float r = exp2f(mc - m1);
            mc = m1;
            l *= r;
#pragma unroll
            for (int dt = 0; dt < VT::ND; ++dt)
#pragma unroll
                for (int i = 0; i < 16; ++i) o[dt][i] *= r;
        }
        if constexpr (!LAST) scores(t + 1, s1);
        ColOp<BF16> p[NS];
#pragma unroll
        for (int n = 0; n < NS; ++n) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                s[n][i] = __builtin_amdgcn_exp2f(fmaf(s[n][i], c, -mc));
                l += s[n][i];
            }
            p[n].set(s[n]);
        }
        // a weight of zero does not keep out an infinity or NaN behind the mask
        if (LAST && VT::template any_nonfinite<BN>(vt, lane)) {
#pragma unroll
            for (int dt = 0; dt < VT::ND; ++dt)
#pragma unroll
                for (int n = 0; n < NS; ++n) o[dt] = VT::template cols_times<true>(o[dt], vt, vat, 32 * n, dt, p[n]);
#pragma unroll 1
            for (int j = 0; j < BN; ++j) VT::add_nonfinite(o, vt, j, half, t * BN + j <= qi);
        } else {
#pragma unroll
            for (int dt = 0; dt < VT::ND; ++dt)
#pragma unroll
                for (int n = 0; n < NS; ++n) o[dt] = VT::cols_times(o[dt], vt, vat, 32 * n, dt, p[n]);
        }
    };

    // Every wave passes every tile's barrier; each works on its own tiles.  Past it, tile t's values
    // and tile t + 1's keys are there, and nobody reads tile t's keys or tile t - 1's values any more.
    auto next = [&](int t) __attribute__((always_inline)) {
        lds_ready();
        if (t + 2 < tiles) stage_k(t + 2);
        if (t + 1 < tiles) stage_v(t + 1);
    };
    stage_k(0);
    stage_v(0);
    loads_done();
    lds_ready();
    if (1 < tiles) stage_k(1);
    f32x16_t sa[NS], sb[NS];
    if (wtiles > 0) scores(0, sa);
    int t = 0;
    for (; t + 2 < wtiles; t += 2) {
        next(t);
        step(t, sa, sb, std::false_type{});
        next(t + 1);
        step(t + 1, sb, sa, std::false_type{});
    }
    if (t + 1 < wtiles) {
        next(t);
        step(t, sa, sb, std::false_type{});
        ++t;
#pragma unroll
        for (int n = 0; n < NS; ++n) sa[n] = sb[n];
    }
    if (t < wtiles) {
        next(t);
        step(t, sa, sb, std::true_type{});
        ++t;
    }
    for (; t < tiles; ++t) next(t);

    l = half_sum(l);
    if (a.lse && live && half == 0) a.lse[tok * a.Hq + h] = (mc + log2f(l)) * kLn2;
    store_col_as_row<BF16, DV>(static_cast<G*>(a.o) + (tok * a.Hq + h) * DV, o, 1.f / l, half, live);
}

// The same for batches that leave compute units idle: 32 query rows a
// workgroup, its four waves on every fourth 32-key tile, joined at the end.
// Four times the workgroups and a quarter of the steps one after another:
// what bounds it is that chain (256 tokens, 2 fp32 heads of 32: 8 us, of which
// two steps of 16 dependent fp32 MFMAs and the join).
template <bool BF16, int DK, int DV>
__global__ __launch_bounds__(256, 1) void attn_prefill_split_kernel(AttnArgs a, float c) {
    using Op = AttnOp<BF16>;
    using KT = AttnTile<BF16, DK>;
    using VT = AttnTile<BF16, DV>;
    using G = typename Op::G;
    constexpr int TG = 32 * kWaves;  // keys the waves take together
    constexpr int KB = TG * KT::ROWB, VB = TG * VT::ROWB;
    constexpr int NBUF = 2 * (KB + VB) <= 128 * 1024 ? 2 : 1;
    constexpr int JOIN = 2 * VT::ND * 4096 + kWaves * 32 * 8;
    __shared__ __attribute__((aligned(1024))) char lds[NBUF * (KB + VB) > JOIN ? NBUF * (KB + VB) : JOIN];

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
    RowFrags<BF16, DK> q;
    load_row_frags<BF16, DK>(q, static_cast<const G*>(a.q) + tok * a.q_stride + static_cast<size_t>(h) * DK, half, live);

    const int ks = a.k_stride * Op::ES, vs = a.v_stride * Op::ES;
    const char* kb = static_cast<const char*>(a.k) + (static_cast<size_t>(st.beg) * a.k_stride + static_cast<size_t>(g) * DK) * Op::ES;
    const char* vb = static_cast<const char*>(a.v) + (static_cast<size_t>(st.beg) * a.v_stride + static_cast<size_t>(g) * DV) * Op::ES;
    const auto ksrc = KT::template src<kWaves>(wave, lane, ks);
    const auto vsrc = VT::template src<kWaves>(wave, lane, vs);
    const int kat = KT::row_at(lane);
    const auto vat = VT::col_at(lane);
    auto stage_group = [&](int t) __attribute__((always_inline)) {
        char* b = lds + (NBUF == 2 ? t & 1 : 0) * (KB + VB);
        KT::template stage<kWaves, TG>(b, kb + static_cast<size_t>(t) * TG * ks, st.len - t * TG, ks, ksrc, wave);
        VT::template stage<kWaves, TG>(b + KB, vb + static_cast<size_t>(t) * TG * vs, st.len - t * TG, vs, vsrc, wave);
    };

    f32x16_t o[VT::ND];
#pragma unroll
    for (int dt = 0; dt < VT::ND; ++dt) o[dt] = f32x16_t{};
    float mc = kLowest, l = 0.f;

    const int groups = (row0 + TG) / TG;  // row0 is a multiple of 32: up to the diagonal
    stage_group(0);
    loads_done();
    for (int t = 0; t < groups; ++t) {
        lds_ready();
        if (NBUF == 2 && t + 1 < groups) stage_group(t + 1);
        const int key0 = t * TG + 32 * wave;
        if (key0 <= row0) {
            const char* kt = lds + (NBUF == 2 ? t & 1 : 0) * (KB + VB);
            const char* vt = kt + KB + 32 * wave * VT::ROWB;
            f32x16_t s = KT::rows_times(f32x16_t{}, kt, kat, 32 * wave, q);
            const bool diagonal = key0 == row0;
            if (diagonal) {
#pragma unroll
                for (int i = 0; i < 16; ++i) s[i] = key0 + 8 * (i >> 2) + 4 * half + (i & 3) <= qi ? s[i] : -INFINITY;
            }
            float mx = s[0];
#pragma unroll
            for (int i = 1; i < 16; ++i) mx = fmaxf(mx, s[i]);
            mx = half_max(mx) * c;
            if (__any(mx > mc + kLazyLog2)) {
                const float m1 = mx > mc + kLazyLog2 ? mx : mc;
                const float r = m1 > mc ? exp2f(mc - m1) : 1.f;
                mc = m1;
                l *= r;
#pragma unroll
                for (int dt = 0; dt < VT::ND; ++dt)
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[dt][i] *= r;
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                s[i] = __builtin_amdgcn_exp2f(fmaf(s[i], c, -mc));
                l += s[i];
            }
            ColOp<BF16> p;
            p.set(s);
            if (diagonal && VT::template any_nonfinite<32>(vt, lane)) {
#pragma unroll
                for (int dt = 0; dt < VT::ND; ++dt) o[dt] = VT::template cols_times<true>(o[dt], vt, vat, 0, dt, p);
#pragma unroll 1
                for (int j = 0; j < 32; ++j) VT::add_nonfinite(o, vt, j, half, key0 + j <= qi);
            } else {
#pragma unroll
                for (int dt = 0; dt < VT::ND; ++dt) o[dt] = VT::cols_times(o[dt], vt, vat, 0, dt, p);
            }
        }
        if (NBUF == 1 && t + 1 < groups) {
            lds_ready();
            stage_group(t + 1);
        }
    }

    // the row's maximum and sum over the waves; each scales its part to them
    l = half_sum(l);
    float* sm = reinterpret_cast<float*>(lds + 2 * VT::ND * 4096);  // [kWaves][32][2]
    __syncthreads();
    if (half == 0) {
        sm[(wave * 32 + lane) * 2] = mc;
        sm[(wave * 32 + lane) * 2 + 1] = l;
    }
    __syncthreads();
    float m = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) m = fmaxf(m, sm[(w * 32 + (lane & 31)) * 2]);
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        const float mw = sm[(w * 32 + (lane & 31)) * 2];
        sum = fmaf(sm[(w * 32 + (lane & 31)) * 2 + 1], mw == m ? 1.f : exp2f(mw - m), sum);
    }
    const float r = mc == m ? 1.f : exp2f(mc - m);
#pragma unroll
    for (int dt = 0; dt < VT::ND; ++dt)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[dt][i] *= r;
    join_waves(o, lds, wave, lane);
    if (wave != 0) return;
    if (a.lse && live && half == 0) a.lse[tok * a.Hq + h] = (m + log2f(sum)) * kLn2;
    store_col_as_row<BF16, DV>(static_cast<G*>(a.o) + (tok * a.Hq + h) * DV, o, 1.f / sum, half, live);
}

namespace {

template <bool BF16, int DK, int DV>
hipError_t launch(const AttnArgs& a) {
    if (a.split) {
        const int64_t units = (static_cast<int64_t>(a.T_tot) + 31) / 32 + a.N;
        hipLaunchKernelGGL((attn_prefill_split_kernel<BF16, DK, DV>), dim3(static_cast<unsigned>(units * a.Hq)), dim3(64 * kWaves), 0,
                           static_cast<hipStream_t>(a.stream), a, a.scale * kLog2e);
        return hipGetLastError();
    }
    const int64_t units = (static_cast<int64_t>(a.T_tot) + kBM - 1) / kBM + a.N;
    hipLaunchKernelGGL((attn_prefill_kernel<BF16, DK, DV>), dim3(static_cast<unsigned>(units * a.Hq)), dim3(64 * kWaves), 0,
                       static_cast<hipStream_t>(a.stream), a, a.scale * kLog2e);
    return hipGetLastError();
}

template <bool BF16, int DK>
hipError_t launch_dv(const AttnArgs& a) {
    switch (a.d_v) {
        case 32: return launch<BF16, DK, 32>(a);
        case 64: return launch<BF16, DK, 64>(a);
        default: return launch<BF16, DK, 128>(a);
    }
}

template <bool BF16>
hipError_t launch_dk(const AttnArgs& a) {
    switch (a.d_k) {
        case 32: return launch_dv<BF16, 32>(a);
        case 64: return launch_dv<BF16, 64>(a);
        default: return launch_dv<BF16, 128>(a);
    }
}

}  // namespace

// Measured for one sequence (whole blocks against split ones): the split is the faster up to a block
// for every compute unit in bf16 (forward, 8 heads of 128: 2048 tokens 43 against 37 us; 16 heads: 45
// against 69), and up to one and a half in fp32 (8 heads of 64: 4096 tokens 298 against 212 us; 32
// heads: 2048 tokens 204 against 236).
bool attn_split(int32_t N, int64_t T_tot, int32_t heads, bool bf16, int cus) {
    return (T_tot / kBM + N) * heads <= (bf16 ? cus : cus + cus / 2);
}

hipError_t launch_attn_prefill(const AttnArgs& a) {
    if (a.T_tot == 0) return hipSuccess;
    return a.bf16 ? launch_dk<true>(a) : launch_dk<false>(a);
}

}  // namespace kda
