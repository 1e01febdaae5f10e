// attn_window_backward.hip -- gradients of the windowed attention of
// attn_window.hip, gfx950.
//
// Over the pairs that row i sees (j <= i, and i - j < window or j < sinks),
// with p_ij = exp(s_ij - lse_i) and dp_ij = do_i . v_j:
//     D_i = do_i . o_i,           ds_ij = p_ij (dp_ij - D_i),
//     dq_i = scale sum_j ds_ij k_j,
//     dk_j = scale sum_h sum_i ds_ij q_i,   dv_j = sum_h sum_i p_ij do_i.
//
// Laid out as attn_backward.hip: a pass over the keys of a block of rows (dq,
// and D; its waves on the heads of a group as in attn_window.hip), one over the
// rows of a block of keys (dk, dv); no atomics, one order of every sum.  The
// rows that see a key are those of its window; the few sinks are seen by all
// rows behind them too.  Left to the workgroup of their block those would be a
// chain as long as the sequence, so the rows past the window go in pieces to
// workgroups of their own (32 keys each), and a last launch adds what the
// pieces give the sinks to what their window gave.
//
// Bound by what feeds the matrix cores (16k tokens in 4 sequences, 32/8 heads
// of 128, bf16, window 1024: forward and backward 1.30 to 1.35 ms; one by one
// under the profiler forward 0.31, dq 0.40, 44 % busy, dk/dv 0.52, 41 % busy,
// its waves waiting half of their time, the sinks' pieces 0.06, the join 0.006).
#include <hip/hip_runtime.h>

#include "attn_window.hpp"

namespace kda {

namespace {

constexpr int kWaves = 4;
constexpr int kBM = 32 * kWaves;  // query rows (dq) or keys (dk, dv) of a workgroup

// Row statistics the dq pass leaves for the dk/dv pass, head-major: [H_q][T_tot] each.
struct Stats {
    float* lse2;  // lse log2(e)
    float* D;
};

__device__ __forceinline__ WindowArgs window_of(const WindowBwdArgs& w) { return {w.b.f, w.window, w.sinks, w.heads}; }

// Rows past the first key's window of a sequence, in pieces of w.rows: the number of pieces.
__device__ __forceinline__ int sink_pieces(const WindowBwdArgs& w, int len) {
    return len > w.window ? (len - w.window - 1) / w.rows + 1 : 0;
}

// Where the band parts of sequence n stand, if it is longer than the window: at n if there are places for
// all, else by its beginning (two such sequences begin more than a window apart).  Below w.bands.
__device__ __forceinline__ int band_place(const WindowBwdArgs& w, int n, int beg) {
    return w.b.f.N <= w.bands ? n : beg / (w.window + 1);
}

}  // namespace

template <bool BF16, int DK, int DV>
__global__ __launch_bounds__(256, BF16 || DK < 128 ? 2 : 1) void attn_window_dq_kernel(WindowBwdArgs wb, float c, Stats stats) {
    using Op = AttnOp<BF16>;
    using KT = AttnTile<BF16, DK>;
    using VT = AttnTile<BF16, DV>;
    using G = typename Op::G;
    constexpr int BN = Op::BN;
    constexpr int KB = BN * KT::ROWB, VB = BN * VT::ROWB;
    __shared__ __attribute__((aligned(1024))) char lds[2][KB + VB];

    const AttnBwdArgs& b = wb.b;
    const AttnArgs& a = b.f;
    const WindowArgs w = window_of(wb);
    const int lane = threadIdx.x & 63, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // waves on heads and blocks of rows as in attn_window.hip
    const int sets = a.Hq / w.heads, hp = blockIdx.x % sets;
    const int g = hp % a.Hkv, h = g * (a.Hq / a.Hkv) + hp / a.Hkv * w.heads + wave % w.heads;
    const int span = kBM / w.heads;
    SeqTile st;
    if (!find_window_tile(a.cu_seqlens, a.N, a.T_tot, span, blockIdx.x / sets, st)) return;

    const int row0 = st.tile * span;
    const int wrow = row0 + 32 * (wave / w.heads);
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

    const WindowTiles<BN> list(w, row0, st.len - row0 < span ? st.len : row0 + span);
    const WindowRows<BN> rows(w, wrow, 32);
    const int upto = wrow < st.len ? list.number(wrow / BN) : -1;  // the wave's last tile in the list

    auto stage_tile = [&](int u) __attribute__((always_inline)) {
        char* l = lds[u & 1];
        const int t = list.tile(u);
        KT::template stage<kWaves, BN>(l, kb + static_cast<size_t>(t) * BN * ks, st.len - t * BN, ks, ksrc, wave);
        VT::template stage<kWaves, BN>(l + KB, vb + static_cast<size_t>(t) * BN * vs, st.len - t * BN, vs, vsrc, wave);
    };

    // Rows with few keys take D from their weights, not from the rounded o (attn_backward.hip): the
    // same walk over the keys, a few tiles.
    if (BF16 && (row0 < kBM || w.window + w.sinks <= kBM)) {
        float sum = 0.f;
        stage_tile(0);
        loads_done();
        for (int u = 0; u < list.count; ++u) {
            lds_ready();
            if (u + 1 < list.count) stage_tile(u + 1);
            const int t = list.tile(u);
            if (u > upto || !rows.sees(t)) continue;
            const char* kt = lds[u & 1];
#pragma unroll 1
            for (int n = 0; n < BN / 32; ++n) {
                const f32x16_t s = KT::rows_times(f32x16_t{}, kt, kat, 32 * n, q);
                const f32x16_t dp = VT::rows_times(f32x16_t{}, kt + KB, vat, 32 * n, d_o);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float x = __builtin_amdgcn_exp2f(fmaf(s[i], c, -lse2)) * dp[i];
                    sum += window_sees(w, qi, t * BN + 32 * n + 8 * (i >> 2) + 4 * half + (i & 3)) ? x : 0.f;
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
    for (int u = 0; u < list.count; ++u) {
        lds_ready();
        if (u + 1 < list.count) stage_tile(u + 1);
        const int t = list.tile(u);
        if (u > upto || !rows.sees(t)) continue;
        const char* kt = lds[u & 1];
        const char* vt = kt + KB;
        const bool masked = !rows.sees_all(t);
#pragma unroll
        for (int n = 0; n < BN / 32; ++n) {
            f32x16_t s = KT::rows_times(f32x16_t{}, kt, kat, 32 * n, q);
            const f32x16_t dp = VT::rows_times(f32x16_t{}, vt, vat, 32 * n, d_o);
#pragma unroll
            for (int i = 0; i < 16; ++i) s[i] = __builtin_amdgcn_exp2f(fmaf(s[i], c, -lse2)) * (dp[i] - D);
            if (masked) {
                const int at = t * BN + 32 * n + 4 * half;  // of the lane's first key
                if (t * BN + BN - 1 > wrow) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) s[i] = 8 * (i >> 2) + (i & 3) <= qi - at ? s[i] : 0.f;
                }
                if (t * BN < rows.all_lo) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int x = 8 * (i >> 2) + (i & 3);
                        s[i] = x > qi - w.window - at || x < w.sinks - at ? s[i] : 0.f;
                    }
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
__global__ __launch_bounds__(256, BF16 || DK + DV <= 128 ? 2 : 1) void attn_window_dkv_kernel(WindowBwdArgs wb, float c, Stats stats) {
    using Op = AttnOp<BF16>;
    using QT = AttnTile<BF16, DK>;
    using OT = AttnTile<BF16, DV>;
    using G = typename Op::G;
    constexpr int BN = 32;
    constexpr bool V_LDS = BF16;  // as in attn_backward.hip: registers for two waves a SIMD
    constexpr int QB = BN * QT::ROWB, OB = BN * OT::ROWB;
    constexpr int SB = 256;  // bytes of one statistic of a tile: a wave-wide load brings 64 floats
    __shared__ __attribute__((aligned(1024))) char lds[2][QB + OB + 2 * SB];
    __shared__ __attribute__((aligned(1024))) char ldsv[V_LDS ? kBM * OT::ROWB : 16];

    const AttnBwdArgs& b = wb.b;
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

    // query tiles t0 .. t1 - 1, up to the end of the last key's window, of every head of the group
    const int end = st.len - key0 < kBM - 1 + wb.window ? st.len : key0 + kBM - 1 + wb.window;
    const int t0 = key0 / BN, t1 = (end + BN - 1) / BN;
    const int wt0 = wkey / BN, wt1 = static_cast<int>((wkey + 30u + wb.window) / BN + 1);  // the wave's

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
        if (t >= wt0 && t < wt1 && wkey < st.len) {
            const char* qt = lds[slot];
            const char* ot = qt + QB;
            const float* sl = reinterpret_cast<const float*>(ot + OB);
            const float* sd = sl + SB / 4;
            const bool masked = t * BN < wkey + 31 || t * BN + BN - 1 - wkey >= wb.window;
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
                if (masked) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int back = t * BN + 32 * n + 8 * (i >> 2) + 4 * half + (i & 3) - kj;
                        const bool sees = back >= 0 && back < wb.window;
                        s[i] = sees ? s[i] : 0.f;
                        dp[i] = sees ? dp[i] : 0.f;
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
    if (wkey < 32 * wb.blocks && st.len > wb.window) {  // the sinks' rows past the window are added later
        float* p = wb.band_parts + ((static_cast<size_t>(band_place(wb, st.n, st.beg)) * 32 * wb.blocks + kj) * a.Hkv + g) * (DK + DV);
        store_col_as_row<false, DK>(p, dk, a.scale, half, live);
        store_col_as_row<false, DV>(p + DK, dv, 1.f, half, live);
        return;
    }
    store_col_as_row<BF16, DK>(static_cast<G*>(b.d_k) + (tok * a.Hkv + g) * DK, dk, a.scale, half, live);
    store_col_as_row<BF16, DV>(static_cast<G*>(b.d_v) + (tok * a.Hkv + g) * DV, dv, 1.f, half, live);
}

// dq for batches that leave compute units idle: 32 rows a workgroup, its four
// waves on every fourth 32-key tile, their sums joined at the end.
template <bool BF16, int DK, int DV>
__global__ __launch_bounds__(256, 1) void attn_window_dq_split_kernel(WindowBwdArgs wb, float c, Stats stats) {
    using Op = AttnOp<BF16>;
    using KT = AttnTile<BF16, DK>;
    using VT = AttnTile<BF16, DV>;
    using G = typename Op::G;
    constexpr int KB = 32 * KT::ROWB, VB = 32 * VT::ROWB;  // of a wave's tile
    constexpr int SLOT = kWaves * (KB + VB);
    // two slots only where two workgroups a compute unit still fit (2048 tokens, 8/2 bf16 heads of 128, window
    // 1024, backward: 99 us, 111 with two slots and one workgroup)
    constexpr int NBUF = 2 * SLOT <= 64 * 1024 ? 2 : 1;
    constexpr int JOIN = 2 * KT::ND * 4096;
    __shared__ __attribute__((aligned(1024))) char lds[NBUF * SLOT > JOIN ? NBUF * SLOT : JOIN];
    __shared__ float s_D[kWaves][32];

    const AttnBwdArgs& b = wb.b;
    const AttnArgs& a = b.f;
    const WindowArgs w = window_of(wb);
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
    const WindowTiles<32> list(w, row0, st.len < row0 + 32 ? st.len : row0 + 32);
    const WindowRows<32> rows(w, row0, 32);
    auto stage_group = [&](int t) __attribute__((always_inline)) {
        char* l = lds + (NBUF == 2 ? t & 1 : 0) * SLOT;
#pragma unroll
        for (int x = 0; x < kWaves; ++x) {
            const int u = kWaves * t + x, tile = list.tile(u);
            const int left = u < list.count ? st.len - 32 * tile : 0;
            KT::template stage<kWaves, 32>(l + x * KB, kb + static_cast<size_t>(tile) * 32 * ks, left, ks, ksrc, wave);
            VT::template stage<kWaves, 32>(l + kWaves * KB + x * VB, vb + static_cast<size_t>(tile) * 32 * vs, left, vs, vsrc, wave);
        }
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
    const int groups = (list.count + kWaves - 1) / kWaves;
    auto put_stats = [&]() __attribute__((always_inline)) {
        if (live && half == 0 && wave == 0) {
            stats.lse2[static_cast<size_t>(h) * a.T_tot + tok] = lse2;
            stats.D[static_cast<size_t>(h) * a.T_tot + tok] = D;
        }
    };
    const bool few = BF16 && groups == 1;  // D from the weights, which are all here
    if (!few) put_stats();
    loads_done();
    for (int t = 0; t < groups; ++t) {
        lds_ready();
        if (NBUF == 2 && t + 1 < groups) stage_group(t + 1);
        const int u = kWaves * t + wave, key0 = 32 * list.tile(u);
        const bool mine = u < list.count;
        const char* kt = lds + (NBUF == 2 ? t & 1 : 0) * SLOT + wave * KB;
        const char* vt = lds + (NBUF == 2 ? t & 1 : 0) * SLOT + kWaves * KB + wave * VB;
        f32x16_t s = {}, dp = {};
        if (mine) {
            s = KT::rows_times(s, kt, kat, 0, q);
            dp = VT::rows_times(dp, vt, vat, 0, d_o);
#pragma unroll
            for (int i = 0; i < 16; ++i) s[i] = __builtin_amdgcn_exp2f(fmaf(s[i], c, -lse2));
            if (!rows.sees_all(list.tile(u))) {
#pragma unroll
                for (int i = 0; i < 16; ++i) s[i] = window_sees(w, qi, key0 + 8 * (i >> 2) + 4 * half + (i & 3)) ? s[i] : 0.f;
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
            for (int x = 0; x < kWaves; ++x) D += s_D[x][lane & 31];
            put_stats();
        }
        if (mine) {
            // a weight of zero: what stands behind the mask may be anything
#pragma unroll
            for (int i = 0; i < 16; ++i) s[i] = s[i] != 0.f ? s[i] * (dp[i] - D) : 0.f;
            ColOp<BF16> ds;
            ds.set(s);
#pragma unroll
            for (int dt = 0; dt < KT::ND; ++dt) dq[dt] = KT::cols_times(dq[dt], kt, kct, 0, dt, ds);
        }
        if (NBUF == 1 && t + 1 < groups) {
            lds_ready();
            stage_group(t + 1);
        }
    }
    join_waves(dq, lds, wave, lane);
    if (wave == 0) store_col_as_row<BF16, DK>(static_cast<G*>(b.d_q) + (tok * a.Hq + h) * DK, dq, a.scale, half, live);
}

// dk and dv of 32 keys a workgroup, its four waves on every fourth 32-row tile,
// for a part of the query heads: one piece of the rows past the window of the
// sinks' keys, or the rows of the keys' window (for batches that leave compute
// units idle).  Both in one launch, the sinks' first.
template <bool BF16, int DK, int DV>
__global__ __launch_bounds__(256, 1) void attn_window_dkv_split_kernel(WindowBwdArgs wb, float c, Stats stats) {
    using Op = AttnOp<BF16>;
    using QT = AttnTile<BF16, DK>;
    using OT = AttnTile<BF16, DV>;
    using G = typename Op::G;
    constexpr int TG = 32 * kWaves;  // query rows the waves take together
    constexpr int QB = TG * QT::ROWB, OB = TG * OT::ROWB, SB = TG * 4;
    // fp32: as in the dq kernel (4096 tokens, 8/2 heads of 64, window 512, backward: 229 us, 238 with two slots);
    // bf16, whose steps are shorter than its loads: two (2048 tokens as above: 99 us, 107 with one)
    constexpr int NBUF = 2 * (QB + OB + 2 * SB) <= (BF16 ? 144 : 80) * 1024 ? 2 : 1;
    constexpr int SLOT = (QB + OB + 2 * SB + 1023) / 1024 * 1024;
    constexpr int JOIN = 2 * 4096 * (QT::ND > OT::ND ? QT::ND : OT::ND);
    __shared__ __attribute__((aligned(1024))) char lds[NBUF * SLOT > JOIN ? NBUF * SLOT : JOIN];

    const AttnBwdArgs& b = wb.b;
    const AttnArgs& a = b.f;
    const int lane = threadIdx.x & 63, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int g = blockIdx.x % a.Hkv;
    const int group = a.Hq / a.Hkv;
    // the query heads of this workgroup, of those of the key head
    const int head_parts = gridDim.y;
    const int h0 = group * blockIdx.y / head_parts, heads = group * (blockIdx.y + 1) / head_parts - h0;
    const int unit = blockIdx.x / a.Hkv, sink_units = wb.pieces * wb.blocks;
    const bool sinks = unit < sink_units;
    SeqTile st;
    int key0, base, end;  // rows [base, end)
    if (sinks) {
        int p = unit / wb.blocks;
        key0 = 32 * (unit % wb.blocks);
        st.n = -1;
        for (int n0 = 0; n0 < a.N; n0 += 64) {
            int2 bl = make_int2(0, 0);
            if (n0 + lane < a.N) bl = seq_bounds(a.cu_seqlens, n0 + lane, a.T_tot);
            const int nt = sink_pieces(wb, bl.y);
            const int incl = wave_scan(nt);
            const int total = __builtin_amdgcn_readlane(incl, 63);
            if (p < total) {
                const int n = __builtin_ctzll(__ballot(incl > p));
                st.n = n0 + n;
                st.beg = __builtin_amdgcn_readlane(bl.x, n);
                st.len = __builtin_amdgcn_readlane(bl.y, n);
                st.tile = p - (__builtin_amdgcn_readlane(incl, n) - __builtin_amdgcn_readlane(nt, n));
                break;
            }
            p -= total;
        }
        if (st.n < 0) return;
        base = wb.window + st.tile * wb.rows;
        end = st.len - base < wb.rows ? st.len : base + wb.rows;
    } else {
        if (!find_tile<32>(a.cu_seqlens, a.N, a.T_tot, unit - sink_units, true, st)) return;
        key0 = st.tile * 32;
        base = key0;
        end = st.len - key0 < 31 + wb.window ? st.len : key0 + 31 + wb.window;
    }

    const int kj = key0 + (lane & 31);
    const bool live = kj < st.len;
    const size_t tok = static_cast<size_t>(st.beg) + (live ? kj : 0);
    const int qs = a.q_stride * Op::ES, os = a.Hq * DV * Op::ES;
    const auto qsrc = QT::template src<kWaves>(wave, lane, qs);
    const auto osrc = OT::template src<kWaves>(wave, lane, os);
    const int qat = QT::row_at(lane), oat = OT::row_at(lane);
    const auto qct = QT::col_at(lane);
    const auto oct = OT::col_at(lane);

    const int groups = (end - base + TG - 1) / TG;  // row groups of a head
    auto stage_group = [&](int slot, int hh, int t) __attribute__((always_inline)) {
        char* l = lds + slot * SLOT;
        const int h = g * group + h0 + hh;
        const size_t r = static_cast<size_t>(st.beg) + base + static_cast<size_t>(t) * TG;
        const int left = end - base - t * TG;
        QT::template stage<kWaves, TG>(l, static_cast<const char*>(a.q) + (r * a.q_stride + static_cast<size_t>(h) * DK) * Op::ES, left,
                                       qs, qsrc, wave);
        OT::template stage<kWaves, TG>(l + QB, static_cast<const char*>(b.d_o) + (r * a.Hq + h) * DV * Op::ES, left, os, osrc, wave);
        // two waves a statistic, 64 rows each
        const float* p = (wave < 2 ? stats.lse2 : stats.D) + static_cast<size_t>(h) * a.T_tot + r;
        load_lds4(buffer_rsrc(p, (left < TG ? left : TG) * 4), l + QB + OB + wave * 256, ((wave & 1) * 64 + lane) * 4, 0);
    };
    stage_group(0, 0, 0);

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
    int hh = 0, t = 0, slot = 0;
    loads_done();
    for (int n = 0; n < steps; ++n) {
        int nh = hh, nt = t + 1;
        if (nt == groups) {
            nt = 0;
            ++nh;
        }
        lds_ready();
        if (NBUF == 2 && n + 1 < steps) stage_group(slot ^ 1, nh, nt);
        const int r0 = base + t * TG + 32 * wave;  // the wave's first row
        if (r0 < end) {
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
            // rows past the window of every sink of the block see it whole
            const bool masked = sinks ? r0 - key0 - 31 < wb.window || key0 + 32 > wb.sinks
                                      : r0 < key0 + 31 || r0 + 31 - key0 >= wb.window;
            if (masked) {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int back = r0 + 8 * (i >> 2) + 4 * half + (i & 3) - kj;
                    const bool sees = sinks ? back >= wb.window && kj < wb.sinks : back >= 0 && back < wb.window;
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
    if (sinks || head_parts > 1 || wb.blocks > 0) {
        const size_t row = sinks ? (static_cast<size_t>(unit / wb.blocks) * head_parts + blockIdx.y) * 32 * wb.blocks + kj
                                 : static_cast<size_t>(blockIdx.y) * a.T_tot + tok;
        float* p = (sinks ? wb.sink_parts : b.parts) + (row * a.Hkv + g) * (DK + DV);
        store_col_as_row<false, DK>(p, dk, a.scale, half, live);
        store_col_as_row<false, DV>(p + DK, dv, 1.f, half, live);
        return;
    }
    store_col_as_row<BF16, DK>(static_cast<G*>(b.d_k) + (tok * a.Hkv + g) * DK, dk, a.scale, half, live);
    store_col_as_row<BF16, DV>(static_cast<G*>(b.d_v) + (tok * a.Hkv + g) * DV, dv, 1.f, half, live);
}

// Sums the parts of dk and dv in their order: those of the window (WHOLE: the
// sinks' one part; else the parts of all keys by query heads), then those of
// the pieces of rows past it.
template <bool BF16, int DK, int DV, bool WHOLE>
__global__ __launch_bounds__(256) void attn_window_join_kernel(WindowBwdArgs wb) {
    using T = Elem<BF16>;
    const AttnBwdArgs& b = wb.b;
    const AttnArgs& a = b.f;
    const int lane = threadIdx.x & 63;
    const int g = blockIdx.x % a.Hkv;
    SeqTile st;
    const int place = blockIdx.x / a.Hkv / (WHOLE ? wb.blocks : 1);
    if constexpr (WHOLE) {  // the sequence whose band parts stand at `place`
        st.n = -1;
        st.tile = blockIdx.x / a.Hkv % wb.blocks;
        for (int n0 = 0; n0 < a.N && st.n < 0; n0 += 64) {
            int2 bl = make_int2(0, 0);
            if (n0 + lane < a.N) bl = seq_bounds(a.cu_seqlens, n0 + lane, a.T_tot);
            const unsigned long long m = __ballot(bl.y > wb.window && band_place(wb, n0 + lane, bl.x) == place);
            if (m) {
                const int n = __builtin_ctzll(m);
                st.n = n0 + n;
                st.beg = __builtin_amdgcn_readlane(bl.x, n);
                st.len = __builtin_amdgcn_readlane(bl.y, n);
            }
        }
        if (st.n < 0) return;
    } else {
        if (!find_tile<32>(a.cu_seqlens, a.N, a.T_tot, place, true, st)) return;
    }
    int first = 0, pieces = 0;  // of the sequence, among all
    if (st.tile < wb.blocks) {
        for (int n0 = 0; n0 < st.n; n0 += 64)
            first += wave_sum(n0 + lane < st.n ? sink_pieces(wb, seq_bounds(a.cu_seqlens, n0 + lane, a.T_tot).y) : 0);
        pieces = sink_pieces(wb, st.len);
        if (first + pieces > wb.pieces) pieces = first < wb.pieces ? wb.pieces - first : 0;  // offsets that overlap: no more
    }
    constexpr int W = DK + DV, Q = W / 4;  // a thread has four elements of a row
    const size_t keys = 32 * static_cast<size_t>(wb.blocks);
    const int x = blockIdx.y * 256 + threadIdx.x, row = st.tile * 32 + x / Q, e = 4 * (x % Q);
    if (row >= st.len) return;
    const size_t at = (static_cast<size_t>(st.beg) + row) * a.Hkv + g;
    float y[4] = {0.f, 0.f, 0.f, 0.f};
    auto add = [&](const float* p, int n, size_t step) __attribute__((always_inline)) {
#pragma unroll 8
        for (int s = 0; s < n; ++s) {
            const f32x4_t z = *reinterpret_cast<const f32x4_t*>(p + s * step);
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] += z[i];
        }
    };
    if constexpr (WHOLE)
        add(wb.band_parts + ((place * keys + row) * a.Hkv + g) * W + e, 1, 0);
    else
        add(b.parts + at * W + e, b.head_parts, static_cast<size_t>(a.T_tot) * a.Hkv * W);
    const int head_parts = WHOLE ? 1 : b.head_parts;  // of every piece
    add(wb.sink_parts + ((first * head_parts * keys + row) * a.Hkv + g) * W + e, pieces * head_parts, keys * a.Hkv * W);
    T::store4(e < DK ? static_cast<typename T::G*>(b.d_k) + at * DK + e : static_cast<typename T::G*>(b.d_v) + at * DV + e - DK, y);
}

namespace {

template <bool BF16, int DK, int DV>
hipError_t launch(const WindowBwdArgs& w, const WindowBwdPlan& plan) {
    const AttnBwdArgs& b = w.b;
    const AttnArgs& a = b.f;
    const int64_t units = (static_cast<int64_t>(a.T_tot) + kBM - 1) / kBM + a.N;
    const int64_t units32 = (static_cast<int64_t>(a.T_tot) + 31) / 32 + a.N;
    const size_t n = static_cast<size_t>(a.T_tot) * a.Hq;
    const Stats stats{static_cast<float*>(b.workspace), static_cast<float*>(b.workspace) + n};
    const hipStream_t st = static_cast<hipStream_t>(a.stream);
    const float c = a.scale * kLog2e;
    const dim3 threads(64 * kWaves);
    if (a.split)
        hipLaunchKernelGGL((attn_window_dq_split_kernel<BF16, DK, DV>), dim3(static_cast<unsigned>(units32 * a.Hq)), threads, 0, st, w, c, stats);
    else {
        const int64_t span = kBM / w.heads, pieces = (static_cast<int64_t>(a.T_tot) + span - 1) / span + a.N;
        hipLaunchKernelGGL((attn_window_dq_kernel<BF16, DK, DV>), dim3(static_cast<unsigned>(pieces * (a.Hq / w.heads))), threads, 0, st, w, c,
                           stats);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const bool whole = b.head_parts == 0;
    if (whole) {
        hipLaunchKernelGGL((attn_window_dkv_kernel<BF16, DK, DV>), dim3(static_cast<unsigned>(units * a.Hkv)), threads, 0, st, w, c, stats);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const int64_t small = plan.pieces * w.blocks + (whole ? 0 : units32);
    if (small > 0) {
        hipLaunchKernelGGL((attn_window_dkv_split_kernel<BF16, DK, DV>), dim3(static_cast<unsigned>(small * a.Hkv), whole ? 1 : b.head_parts),
                           threads, 0, st, w, c, stats);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (whole && w.blocks > 0)
        hipLaunchKernelGGL((attn_window_join_kernel<BF16, DK, DV, true>),
                           dim3(static_cast<unsigned>(static_cast<int64_t>(w.bands) * w.blocks * a.Hkv), (DK + DV) / 32), dim3(256), 0, st, w);
    else if (!whole && (b.head_parts > 1 || w.blocks > 0))
        hipLaunchKernelGGL((attn_window_join_kernel<BF16, DK, DV, false>), dim3(static_cast<unsigned>(units32 * a.Hkv), (DK + DV) / 32),
                           dim3(256), 0, st, w);
    return hipGetLastError();
}

template <bool BF16, int DK>
hipError_t launch_dv(const WindowBwdArgs& w, const WindowBwdPlan& p) {
    switch (w.b.f.d_v) {
        case 32: return launch<BF16, DK, 32>(w, p);
        case 64: return launch<BF16, DK, 64>(w, p);
        default: return launch<BF16, DK, 128>(w, p);
    }
}

template <bool BF16>
hipError_t launch_dk(const WindowBwdArgs& w, const WindowBwdPlan& p) {
    switch (w.b.f.d_k) {
        case 32: return launch_dv<BF16, 32>(w, p);
        case 64: return launch_dv<BF16, 64>(w, p);
        default: return launch_dv<BF16, 128>(w, p);
    }
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

// Pieces of rows: of one length, a workgroup for every compute unit (it holds no second one) if one sequence had
// all the rows, and at least one group of 128 rows.  The length does not depend on the number of sequences, most of
// which may have no row past their window; a short last piece of each is a small matter.  Without the forward pass,
// 32/8 heads of 128, window 1024: 16k tokens in 4 sequences with 4 sinks 989 us, 996 with two workgroups a unit, 1015
// with four, 990 with so many fewer pieces that the short ones fit the round too; with 256 sinks 1237, 1222 and
// 1221, 1354 in one piece a sequence; 8192 tokens beside 31 sequences of 256, 4 sinks, 682, 670 and 674, 1163 in one
// piece (644 without sinks).
WindowBwdPlan attn_window_bwd_plan(int32_t N, int64_t T_tot, int32_t Hq, int32_t Hkv, int32_t d_k, int32_t d_v, int32_t window,
                                   int32_t sinks, bool bf16, int cus) {
    const BwdPlan plain = attn_bwd_plan(N, T_tot, Hq, Hkv, d_k, d_v, bf16, cus);
    WindowBwdPlan p{};
    p.head_parts = plain.head_parts;
    p.stats_bytes = plain.stats_bytes;
    const size_t row = static_cast<size_t>(Hkv) * (d_k + d_v) * sizeof(float);
    if (sinks > 0 && window < T_tot) {
        const int64_t keys = sinks < T_tot ? sinks : T_tot;
        p.blocks = static_cast<int32_t>((keys + 31) / 32);
        // k sequences longer than the window have at most (T_tot - k (window + 1)) / rows + k pieces: the most with
        // one of them or with all
        p.bands = static_cast<int32_t>(N < T_tot / (window + 1) ? N : T_tot / (window + 1));
        const int64_t wgs = static_cast<int64_t>(p.blocks) * Hkv, left = T_tot - window;  // workgroups of a piece
        const int64_t share = left * wgs / cus, rows = share < left ? share : left;
        p.rows = static_cast<int32_t>(rows < 1 ? 128 : (rows + 127) / 128 * 128);
        const int64_t one = (left - 1) / p.rows + 1, all = (T_tot - p.bands * (int64_t{window} + 1)) / p.rows + p.bands;
        p.pieces = one > all ? one : all;
        p.parts_bytes = up256(static_cast<size_t>(p.pieces) * (p.head_parts > 1 ? p.head_parts : 1) * 32 * p.blocks * row);
        if (p.head_parts == 0) p.band_bytes = up256(static_cast<size_t>(p.bands) * 32 * p.blocks * row);
    }
    size_t heads = 0;
    if (p.head_parts > 1 || (p.head_parts == 1 && p.blocks > 0)) heads = up256(static_cast<size_t>(p.head_parts) * T_tot * row);
    p.bytes = p.stats_bytes + p.parts_bytes + p.band_bytes + heads;
    return p;
}

hipError_t launch_attn_window_bwd(const WindowBwdArgs& w, const WindowBwdPlan& p) {
    if (w.b.f.T_tot == 0) return hipSuccess;
    return w.b.f.bf16 ? launch_dk<true>(w, p) : launch_dk<false>(w, p);
}

}  // namespace kda
