// attn_window.hip -- causal softmax attention with a sliding window and sinks
// over packed prompts, gfx950.
//
// Row i of a sequence sees key j <= i if j > i - window or j < sinks:
//     s_ij = scale q_i . k_j,  lse_i = ln sum_j exp(s_ij),
//     o_i = sum_j exp(s_ij - lse_i) v_j   over the j it sees.
//
// Laid out as attn_prefill.hip: 32 query rows of a head a wave, one pass over
// the keys with a running maximum and sum, the next tile's scores between a
// tile's statistics and its weights.  What differs is the list of key tiles a
// workgroup walks: the tiles of the sinks, then those from its first row's
// window to its diagonal.  Where query heads share a key head the four waves
// are four (or two) of them over the same rows: the list is then as short as
// one wave's, and no wave waits for tiles that only others see (together with
// taking the masked tiles into the pipeline: 32k tokens in 8 prompts, 32/8 heads
// of 128, window 1024: 635 to 609 us; not measured apart).  Three kinds of tile are masked, by at most two comparisons
// a score: the last of the sinks, the ones where a row's window begins, the
// diagonal.  Values are not looked through for infinities and NaN, which a
// weight of zero would let through the mask: they turn a column of the result
// NaN, and a workgroup that finds one walks again, looking.
//
// Bound, as the plain attention, by what feeds the matrix cores: 610 to 645 us,
// 745 to 790 TFLOP/s on those 32k tokens; on 16k in 4 sequences the matrix cores
// are busy 36 % and the vector units 41 % of the time.  A workgroup walks some 18
// tiles: its look-up, first loads and last steps are a fifth of its time (read
// from the clock: 9 of 87 thousand cycles before the first pair of tiles, 10
// after the last), where a long causal row has them
// once for hundreds of tiles.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "attn_window.hpp"

namespace kda {

namespace {

constexpr int kWaves = 4;
constexpr int kBM = 32 * kWaves;  // query rows of a workgroup
constexpr float kLazyLog2 = 8.f;  // as in attn_prefill.hip
constexpr float kLowest = -3.402823466e38f;

}  // namespace

template <bool BF16, int DK, int DV>
__global__ __launch_bounds__(256, 2) void attn_window_kernel(WindowArgs w, float c /* scale log2(e) */) {
    using Op = AttnOp<BF16>;
    using KT = AttnTile<BF16, DK>;
    using VT = AttnTile<BF16, DV>;
    using G = typename Op::G;
    constexpr int BN = Op::BN, NS = BN / 32;
    constexpr int KB = BN * KT::ROWB, VB = BN * VT::ROWB;
    __shared__ __attribute__((aligned(1024))) char lds[2][KB + VB];

    const AttnArgs& a = w.f;
    const int lane = threadIdx.x & 63, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // The waves are w.heads query heads of one key head by 4 / w.heads blocks of 32 rows.  Consecutive
    // workgroups take consecutive key heads: as in attn_prefill.hip.
    const int sets = a.Hq / w.heads, hp = blockIdx.x % sets;
    const int g = hp % a.Hkv, h = g * (a.Hq / a.Hkv) + hp / a.Hkv * w.heads + wave % w.heads;
    const int span = kBM / w.heads;  // rows of the workgroup
    SeqTile st;
    if (!find_window_tile(a.cu_seqlens, a.N, a.T_tot, span, blockIdx.x / sets, st)) return;

    const int row0 = st.tile * span;
    const int wrow = row0 + 32 * (wave / w.heads);   // the wave's first row
    const int qi = wrow + (lane & 31);   // the lane's query row in its sequence
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

    const WindowTiles<BN> list(w, row0, st.len - row0 < span ? st.len : row0 + span);
    const WindowRows<BN> rows(w, wrow, 32);
    // the wave's last tile in the list, and whether it works on tile u of it
    const int upto = wrow < st.len ? list.number(wrow / BN) : -1;
    auto active = [&](int u) __attribute__((always_inline)) { return u <= upto && rows.sees(list.tile(u)); };

    auto stage_k = [&](int u) __attribute__((always_inline)) {
        const int t = list.tile(u);
        KT::template stage<kWaves, BN>(lds[u & 1], kb + static_cast<size_t>(t) * BN * ks, st.len - t * BN, ks, ksrc, wave);
    };
    auto stage_v = [&](int u) __attribute__((always_inline)) {
        const int t = list.tile(u);
        VT::template stage<kWaves, BN>(lds[u & 1] + KB, vb + static_cast<size_t>(t) * BN * vs, st.len - t * BN, vs, vsrc, wave);
    };

    f32x16_t o[VT::ND];
    float mc, l;  // running maximum of c s, and this half-wave's part of the row's sum

    auto scores = [&](int u, f32x16_t (&s)[NS]) __attribute__((always_inline)) {
#pragma unroll
        for (int n = 0; n < NS; ++n) s[n] = KT::rows_times(f32x16_t{}, lds[u & 1], kat, 32 * n, q);
    };
    // One tile's scores into the row's statistics and O.  kAhead: the next tile's scores go to `s1`,
    // between the two dependent halves of the step.  kCareful: values behind the mask may be infinite or
    // NaN, which a weight of zero does not keep out.
    enum { kAhead, kAlone, kCareful };
    auto step = [&](int u, f32x16_t (&s)[NS], f32x16_t (&s1)[NS], auto kind) __attribute__((always_inline)) {
        const char* vt = lds[u & 1] + KB;
        const int key0 = list.tile(u) * BN;
        auto cols = vat;
        // what is worked out from them stays in here: kept over the loop it would be spilled
        if constexpr (kind != kAhead) asm volatile("" : "+v"(cols.v[0]), "+v"(cols.v[1]));
        if (!rows.sees_all(list.tile(u))) {
            int at = key0 + 4 * half;  // of the lane's first score
            asm volatile("" : "+v"(at));
            if (key0 + BN - 1 > wrow) {
#pragma unroll
                for (int n = 0; n < NS; ++n)
#pragma unroll
                    for (int i = 0; i < 16; ++i) s[n][i] = 32 * n + 8 * (i >> 2) + (i & 3) <= qi - at ? s[n][i] : -INFINITY;
            }
            if (key0 < rows.all_lo) {
#pragma unroll
                for (int n = 0; n < NS; ++n)
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int x = 32 * n + 8 * (i >> 2) + (i & 3);
                        s[n][i] = x > qi - w.window - at || x < w.sinks - at ? s[n][i] : -INFINITY;
                    }
            }
        }
        float mx = s[0][0];
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
            for (int i = 0; i < 16; ++i) mx = fmaxf(mx, s[n][i]);
        mx = half_max(mx) * c;
        if (__any(mx > mc + kLazyLog2)) {
            const float m1 = mx > mc + kLazyLog2 ? mx : mc;
            const float r = exp2f(mc - m1);
            mc = m1;
            l *= r;
#pragma unroll
            for (int dt = 0; dt < VT::ND; ++dt)
#pragma unroll
                for (int i = 0; i < 16; ++i) o[dt][i] *= r;
        }
        if constexpr (kind == kAhead) scores(u + 1, s1);
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
        if (kind == kCareful && VT::template any_nonfinite<BN>(vt, lane)) {
#pragma unroll
            for (int dt = 0; dt < VT::ND; ++dt)
#pragma unroll
                for (int n = 0; n < NS; ++n) o[dt] = VT::template cols_times<true>(o[dt], vt, cols, 32 * n, dt, p[n]);
#pragma unroll 1
            for (int j = 0; j < BN; ++j) VT::add_nonfinite(o, vt, j, half, window_sees(w, qi, key0 + j));
        } else {
#pragma unroll
            for (int dt = 0; dt < VT::ND; ++dt)
#pragma unroll
                for (int n = 0; n < NS; ++n) o[dt] = VT::cols_times(o[dt], vt, cols, 32 * n, dt, p[n]);
        }
    };

    // Every wave passes every tile's barrier.  Past it, tile u's values and tile u + 1's keys are there,
    // and nobody reads tile u's keys or tile u - 1's values any more.
    const int tiles = list.count;
    auto next = [&](int u) __attribute__((always_inline)) {
        lds_ready();
        if (u + 2 < tiles) stage_k(u + 2);
        if (u + 1 < tiles) stage_v(u + 1);
    };
    f32x16_t sa[NS], sb[NS];
    // The walk over the tiles.  sa holds the scores of tile u, if the wave works on it.  Tiles before two
    // others that it works on go in pairs, the last ones and those before a gap one by one.
    auto walk = [&](auto careful) __attribute__((always_inline)) {
#pragma unroll
        for (int dt = 0; dt < VT::ND; ++dt) o[dt] = f32x16_t{};
        mc = kLowest;
        l = 0.f;
        auto alone = [&](int u) __attribute__((always_inline)) {
            next(u);
            if (active(u)) step(u, sa, sb, std::integral_constant<int, careful ? kCareful : kAlone>{});
            if (active(u + 1)) scores(u + 1, sa);
        };
        auto paired = [&](int u) __attribute__((always_inline)) { return active(u) && active(u + 1) && active(u + 2); };
        stage_k(0);
        stage_v(0);
        loads_done();
        lds_ready();
        if (1 < tiles) stage_k(1);
        if (active(0)) scores(0, sa);
        int u = 0;
        if constexpr (!careful) {
            for (; u < tiles && !paired(u); ++u) alone(u);
            for (; paired(u); u += 2) {
                next(u);
                step(u, sa, sb, std::integral_constant<int, kAhead>{});
                next(u + 1);
                step(u + 1, sb, sa, std::integral_constant<int, kAhead>{});
            }
        }
        for (; u < tiles; ++u) alone(u);
    };
    walk(std::false_type{});
    // An infinity or NaN behind the mask has made its column NaN: the walk once more, looking through the
    // values.  (Looked through at every masked tile they cost a third of the vector work.)
    float zero = 0.f;
#pragma unroll
    for (int dt = 0; dt < VT::ND; ++dt)
#pragma unroll
        for (int i = 0; i < 16; ++i) zero = fmaf(o[dt][i], 0.f, zero);
    if (__syncthreads_or(zero != 0.f)) walk(std::true_type{});

    l = half_sum(l);
    if (a.lse && live && half == 0) a.lse[tok * a.Hq + h] = (mc + log2f(l)) * kLn2;
    store_col_as_row<BF16, DV>(static_cast<G*>(a.o) + (tok * a.Hq + h) * DV, o, 1.f / l, half, live);
}

// The same for batches that leave compute units idle (attn_split): 32 query
// rows a workgroup, its four waves on every fourth 32-key tile of the list,
// joined at the end.  Bound by that chain (256 tokens, 2 fp32 heads of 32,
// window 50: 7 us; 5 ragged fp32 sequences of 924 tokens, 8/2 heads of 64: 16).
template <bool BF16, int DK, int DV>
__global__ __launch_bounds__(256, 1) void attn_window_split_kernel(WindowArgs w, float c) {
    using Op = AttnOp<BF16>;
    using KT = AttnTile<BF16, DK>;
    using VT = AttnTile<BF16, DV>;
    using G = typename Op::G;
    constexpr int KB = 32 * KT::ROWB, VB = 32 * VT::ROWB;  // of a wave's tile
    constexpr int SLOT = kWaves * (KB + VB);
    constexpr int NBUF = 2 * SLOT <= 128 * 1024 ? 2 : 1;
    constexpr int JOIN = 2 * VT::ND * 4096 + kWaves * 32 * 8;
    __shared__ __attribute__((aligned(1024))) char lds[NBUF * SLOT > JOIN ? NBUF * SLOT : JOIN];

    const AttnArgs& a = w.f;
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

    // the list's tiles, four at a time; all waves load all four
    const WindowTiles<32> list(w, row0, st.len < row0 + 32 ? st.len : row0 + 32);
    const WindowRows<32> rows(w, row0, 32);
    auto stage_group = [&](int t) __attribute__((always_inline)) {
        char* b = lds + (NBUF == 2 ? t & 1 : 0) * SLOT;
#pragma unroll
        for (int x = 0; x < kWaves; ++x) {
            const int u = kWaves * t + x, tile = list.tile(u);
            const int left = u < list.count ? st.len - 32 * tile : 0;  // past the list: nothing, read as zero
            KT::template stage<kWaves, 32>(b + x * KB, kb + static_cast<size_t>(tile) * 32 * ks, left, ks, ksrc, wave);
            VT::template stage<kWaves, 32>(b + kWaves * KB + x * VB, vb + static_cast<size_t>(tile) * 32 * vs, left, vs, vsrc, wave);
        }
    };

    f32x16_t o[VT::ND];
#pragma unroll
    for (int dt = 0; dt < VT::ND; ++dt) o[dt] = f32x16_t{};
    float mc = kLowest, l = 0.f;

    const int groups = (list.count + kWaves - 1) / kWaves;
    stage_group(0);
    loads_done();
    for (int t = 0; t < groups; ++t) {
        lds_ready();
        if (NBUF == 2 && t + 1 < groups) stage_group(t + 1);
        const int u = kWaves * t + wave;
        if (u < list.count) {
            const int key0 = 32 * list.tile(u);
            const char* kt = lds + (NBUF == 2 ? t & 1 : 0) * SLOT + wave * KB;
            const char* vt = lds + (NBUF == 2 ? t & 1 : 0) * SLOT + kWaves * KB + wave * VB;
            f32x16_t s = KT::rows_times(f32x16_t{}, kt, kat, 0, q);
            const bool masked = !rows.sees_all(list.tile(u));
            if (masked) {
#pragma unroll
                for (int i = 0; i < 16; ++i) s[i] = window_sees(w, qi, key0 + 8 * (i >> 2) + 4 * half + (i & 3)) ? s[i] : -INFINITY;
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
            if (masked && VT::template any_nonfinite<32>(vt, lane)) {
#pragma unroll
                for (int dt = 0; dt < VT::ND; ++dt) o[dt] = VT::template cols_times<true>(o[dt], vt, vat, 0, dt, p);
#pragma unroll 1
                for (int j = 0; j < 32; ++j) VT::add_nonfinite(o, vt, j, half, window_sees(w, qi, key0 + j));
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
    for (int x = 0; x < kWaves; ++x) m = fmaxf(m, sm[(x * 32 + (lane & 31)) * 2]);
    float sum = 0.f;
#pragma unroll
    for (int x = 0; x < kWaves; ++x) {
        const float mw = sm[(x * 32 + (lane & 31)) * 2];
        sum = fmaf(sm[(x * 32 + (lane & 31)) * 2 + 1], mw == m ? 1.f : exp2f(mw - m), sum);
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
hipError_t launch(const WindowArgs& w) {
    const AttnArgs& a = w.f;
    const hipStream_t st = static_cast<hipStream_t>(a.stream);
    if (a.split) {
        const int64_t units = (static_cast<int64_t>(a.T_tot) + 31) / 32 + a.N;
        hipLaunchKernelGGL((attn_window_split_kernel<BF16, DK, DV>), dim3(static_cast<unsigned>(units * a.Hq)), dim3(64 * kWaves), 0,
                           st, w, a.scale * kLog2e);
        return hipGetLastError();
    }
    const int64_t span = kBM / w.heads, units = (static_cast<int64_t>(a.T_tot) + span - 1) / span + a.N;
    hipLaunchKernelGGL((attn_window_kernel<BF16, DK, DV>), dim3(static_cast<unsigned>(units * (a.Hq / w.heads))), dim3(64 * kWaves), 0,
                       st, w, a.scale * kLog2e);
    return hipGetLastError();
}

template <bool BF16, int DK>
hipError_t launch_dv(const WindowArgs& w) {
    switch (w.f.d_v) {
        case 32: return launch<BF16, DK, 32>(w);
        case 64: return launch<BF16, DK, 64>(w);
        default: return launch<BF16, DK, 128>(w);
    }
}

template <bool BF16>
hipError_t launch_dk(const WindowArgs& w) {
    switch (w.f.d_k) {
        case 32: return launch_dv<BF16, 32>(w);
        case 64: return launch_dv<BF16, 64>(w);
        default: return launch_dv<BF16, 128>(w);
    }
}

}  // namespace

hipError_t launch_attn_window(const WindowArgs& w) {
    if (w.f.T_tot == 0) return hipSuccess;
    return w.f.bf16 ? launch_dk<true>(w) : launch_dk<false>(w);
}

}  // namespace kda
