// attn_weights.hip -- how much attention the positions of a prompt have drawn
// from its (last) rows, gfx950.
//
// For sequence n, key head g and position j, over the last `rows` rows i:
//     w[n, g, j] = sum_{h of g} sum_{i >= j} exp(s_ij - lse_i).
//
// The scores of the forward pass once more, with the keys kept and the rows
// walked: a wave has 64 keys of a key head in registers, the tiles of 64 query
// rows of its heads come through LDS, and S = Q K^T in 32x32 MFMAs leaves a
// lane the scores of 16 rows against one key, whose weights it adds into one
// number.  So there is one product a pair and no second one to feed; 64 keys
// a wave and not 32, because a row read from LDS then serves two products.
// Each sum is one lane's, in one order, joined with the other half-wave's at
// the end.
//
// A long sequence's first keys have all of its rows; a block's rows (of all the
// query heads of its key head, one after another) are therefore given to several
// workgroups, and a second launch adds their sums in order (32k tokens in 8
// prompts, 32/8 heads of 128, every row: 1156 us in one part, 915 in six, 936 and
// 941 in three and twelve; with a sequence's blocks following one another 850 in
// six; with the statistics of rows without a score seen to 880, and 852 where the
// parts look their blocks of keys up, in turn; 811 to 850 among calls, 880 to 920
// TFLOP/s).  What bounds it there is open: the matrix cores are busy 41 % and the
// vector units 55 % of the time, which hardly overlap, with 2.4 waves a SIMD
// of the three that fit.  Taking turns by hand (products of the next rows between
// the exponentials) took 877 to 928 us beside 846 to 870, workgroups that stay 943
// to 996 beside 849 to 856.
#include <hip/hip_runtime.h>

#include <cfloat>
#include <type_traits>

#include "attn_window.hpp"

namespace kda {

namespace {

constexpr int kWaves = 4;
constexpr int kKeys = 64;             // of a wave
constexpr int kBK = kKeys * kWaves;   // of a workgroup
constexpr int kStrip = 4096;          // positions that a workgroup clears

// The blocks of keys that workgroups are launched for.
enum class KeyBlocks {
    kWidth,         // of the width, in one part or several
    kThere,         // those that there are, looked up, in one part; a second row of the grid clears what lies behind
    kThereInParts,  // the same in several parts (the join writes what lies behind)
};

}  // namespace

// In parts and looked up, the compiler is held to the registers of three waves a SIMD, which it takes by itself by
// the width (32k tokens, every row: 847 us, 882 with two waves).  Not in one part, where a chain is short and its
// first loads count (the last 64 rows of 4000: 22 us, 25 with three).
template <bool BF16, int DK, KeyBlocks B>
__global__ __launch_bounds__(256, B == KeyBlocks::kThereInParts && DK * (BF16 ? 2 : 4) <= 256 ? 3 : 2) void attn_weights_kernel(WeightsArgs wa, float c /* scale log2(e) */) {
    using Op = AttnOp<BF16>;
    using QT = AttnTile<BF16, DK>;
    using G = typename Op::G;
    constexpr int BN = 64;                 // query rows of a tile
    constexpr int QB = BN * QT::ROWB, SLOT = QB + 1024;
    constexpr int NK = kKeys / 32;
    __shared__ __attribute__((aligned(1024))) char lds[2][SLOT];

    const AttnArgs& a = wa.f;
    const int lane = threadIdx.x & 63, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int group = a.Hq / a.Hkv;
    const int g = blockIdx.x % a.Hkv;
    if (B == KeyBlocks::kThere && blockIdx.y == 1) {  // the zeros behind a sequence's last block of keys
        const int strips = (wa.width + kStrip - 1) / kStrip, n = blockIdx.x / a.Hkv / strips;
        if (n >= a.N) return;
        const int len = seq_bounds(a.cu_seqlens, n, a.T_tot).y, there = (len + kBK - 1) / kBK * kBK;
        float* w = wa.weights + (static_cast<size_t>(n) * a.Hkv + g) * wa.width;
        const int j0 = static_cast<int>(blockIdx.x / a.Hkv % strips) * kStrip;
#pragma unroll 1
        for (int j = (j0 > there ? j0 : there) + threadIdx.x; j < wa.width && j < j0 + kStrip; j += 64 * kWaves) w[j] = 0.f;
        return;
    }
    // a sequence's blocks of keys follow one another, the key heads of a block side by side
    SeqTile st;
    if constexpr (B != KeyBlocks::kWidth) {
        if (!find_window_tile(a.cu_seqlens, a.N, a.T_tot, kBK, blockIdx.x / a.Hkv, st) || st.tile * kBK >= wa.width) return;
    } else {
        const int KBn = (wa.width + kBK - 1) / kBK;
        st.n = blockIdx.x / a.Hkv / KBn;
        st.tile = static_cast<int>(blockIdx.x / a.Hkv % KBn);
        const int2 bl = seq_bounds(a.cu_seqlens, st.n, a.T_tot);
        st.beg = bl.x;
        st.len = bl.y;
    }
    const int key0 = st.tile * kBK, wkey = key0 + kKeys * wave;
    const int n = st.n, beg = st.beg, len = st.len;
    const int parts = B == KeyBlocks::kThere ? 1 : wa.parts, part = B == KeyBlocks::kThere ? 0 : blockIdx.y;
    if (B == KeyBlocks::kWidth && parts > 1 && key0 >= len) return;

    // A tile's weights are summed by themselves and added with what the sum before has lost to rounding
    // (compensated): one number takes thousands of rows of every head.
    float sum[NK] = {}, lost[NK] = {};
    if (B != KeyBlocks::kWidth || key0 < len) {
        typename Op::Row k[NK][QT::NF];
#pragma unroll
        for (int x = 0; x < NK; ++x) {
            const int kj = wkey + 32 * x + (lane & 31);
            const size_t tok = static_cast<size_t>(beg) + (kj < len ? kj : 0);
            load_row_frags<BF16, DK>(k[x], static_cast<const G*>(a.k) + tok * a.k_stride + static_cast<size_t>(g) * DK, half, kj < len);
        }
        const int qs = a.q_stride * Op::ES;
        const auto qsrc = QT::template src<kWaves>(wave, lane, qs);
        const int qat = QT::row_at(lane);
        // row tiles t0 .. t1 - 1 of every head of the group, one after another
        const int first = len > wa.rows ? len - wa.rows : 0;  // the first row that counts
        const int t0 = (first > key0 ? first : key0) / BN, t1 = (len + BN - 1) / BN;
        auto stage_tile = [&](int slot, int hh, int t) __attribute__((always_inline)) {
            const int h = g * group + hh, left = len - t * BN;
            const size_t r = static_cast<size_t>(beg) + static_cast<size_t>(t) * BN;
            QT::template stage<kWaves, BN>(lds[slot], static_cast<const char*>(a.q) + (r * a.q_stride + static_cast<size_t>(h) * DK) * Op::ES,
                                           left, qs, qsrc, wave);
        };
        // the rows' statistics, one a lane of the first wave; rows past the last are masked
        auto statistic = [&](int hh, int t) __attribute__((always_inline)) {
            const int row = t * BN + lane < len ? t * BN + lane : len - 1;
            return a.lse[(static_cast<size_t>(beg) + row) * a.Hq + g * group + hh];
        };
        // As powers of two, once for all waves and keys.  A row whose scores are all below the range of fp32
        // has -infinity: from the lowest finite number they weigh nothing (-infinity less -infinity is NaN).
        // NaN stays NaN, and so do the weights of that row (fmaxf would take the number).
        auto keep_statistic = [&](int slot, float lse) __attribute__((always_inline)) {
            const float l2 = lse * kLog2e;
            reinterpret_cast<float*>(lds[slot] + QB)[lane] = l2 == -INFINITY ? -FLT_MAX : l2;
        };
        // this workgroup's part of them
        const int64_t all = static_cast<int64_t>(group) * (t1 - t0);
        const int begin = static_cast<int>(all * part / parts), end = static_cast<int>(all * (part + 1) / parts);
        int hh = begin / (t1 - t0), t = t0 + begin % (t1 - t0), slot = 0;
        if (begin < end) {
            if (wave == 0) keep_statistic(0, statistic(hh, t));
            stage_tile(0, hh, t);
        }
        loads_done();
        for (int step = begin; step < end; ++step) {
            int nh = hh, nt = t + 1;
            if (nt == t1) {
                nt = t0;
                ++nh;
            }
            lds_ready();
            float next = 0.f;
            if (step + 1 < end) {
                if (wave == 0) next = statistic(nh, nt);
                stage_tile(slot ^ 1, nh, nt);
            }
            if (t * BN + BN > wkey && wkey < len) {
                const char* qt = lds[slot];
                const float* sl = reinterpret_cast<const float*>(qt + QB);
                auto scores = [&](int r0, f32x16_t (&s)[NK]) __attribute__((always_inline)) {
#pragma unroll
                    for (int x = 0; x < NK; ++x) s[x] = f32x16_t{};
#pragma unroll
                    for (int kk = 0; kk < QT::NF; ++kk) {
                        const typename Op::Row q = QT::row(qt, qat, r0, kk);
#pragma unroll
                        for (int x = 0; x < NK; ++x) s[x] = Op::mma(q, k[x][kk], s[x]);
                    }
                };
                auto add = [&](int r0, const f32x16_t (&s)[NK], auto MASKED) __attribute__((always_inline)) {
                    f32x4_t l2[4];
#pragma unroll
                    for (int i4 = 0; i4 < 4; ++i4) l2[i4] = *reinterpret_cast<const f32x4_t*>(sl + r0 + 8 * i4 + 4 * half);
#pragma unroll
                    for (int x = 0; x < NK; ++x) {
                        float p[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const int row = t * BN + r0 + 8 * (i >> 2) + 4 * half + (i & 3);
                            p[i] = __builtin_amdgcn_exp2f(fmaf(s[x][i], c, -l2[i >> 2][i & 3]));
                            if (MASKED && !(row >= wkey + 32 * x + (lane & 31) && row >= first && row < len)) p[i] = 0.f;
                        }
#pragma unroll
                        for (int d = 8; d >= 1; d /= 2)
#pragma unroll
                            for (int i = 0; i < d; ++i) p[i] += p[i + d];
                        const float y = p[0] - lost[x], z = sum[x] + y;
                        lost[x] = (z - sum[x]) - y;
                        sum[x] = z;
                    }
                };
                if (t * BN < wkey + kKeys - 1 || t * BN < first || t * BN + BN > len) {
#pragma unroll 1
                    for (int r0 = 0; r0 < BN; r0 += 32) {
                        f32x16_t s[NK];
                        scores(r0, s);
                        add(r0, s, std::true_type{});
                    }
                } else {
                    f32x16_t s0[NK], s1[NK];
                    scores(0, s0);
                    scores(32, s1);
                    add(0, s0, std::false_type{});
                    add(32, s1, std::false_type{});
                }
            }
            if (step + 1 < end && wave == 0) keep_statistic(slot ^ 1, next);
            hh = nh;
            t = nt;
            slot ^= 1;
        }
    }
#pragma unroll
    for (int x = 0; x < NK; ++x) {
        const int kj = wkey + 32 * x + (lane & 31);
        const float y = half_sum(sum[x]);
        if (half != 0) continue;
        if (parts > 1) {
            if (kj < len) wa.part[(static_cast<size_t>(part) * a.Hkv + g) * a.T_tot + beg + kj] = y;
        } else if (kj < wa.width) {
            wa.weights[(static_cast<size_t>(n) * a.Hkv + g) * wa.width + kj] = kj < len ? y : 0.f;
        }
    }
}

// The parts' sums, in their order; zero behind a sequence.
__global__ __launch_bounds__(256) void attn_weights_join_kernel(WeightsArgs wa) {
    const AttnArgs& a = wa.f;
    const int g = blockIdx.x % a.Hkv, n = blockIdx.x / a.Hkv % a.N;
    const int j = static_cast<int>(blockIdx.x / a.Hkv / a.N) * kBK + threadIdx.x;
    if (j >= wa.width) return;
    const int2 bl = seq_bounds(a.cu_seqlens, n, a.T_tot);
    float y = 0.f;
    if (j < bl.y) {
        const float* p = wa.part + static_cast<size_t>(g) * a.T_tot + bl.x + j;
        const size_t step = static_cast<size_t>(a.Hkv) * a.T_tot;
#pragma unroll 4
        for (int x = 0; x < wa.parts; ++x) y += p[x * step];
    }
    wa.weights[(static_cast<size_t>(n) * a.Hkv + g) * wa.width + j] = y;
}

namespace {

template <bool BF16, int DK>
hipError_t launch(const WeightsArgs& w) {
    const AttnArgs& a = w.f;
    const hipStream_t st = static_cast<hipStream_t>(a.stream);
    const unsigned blocks = static_cast<unsigned>((w.width + kBK - 1) / kBK) * a.N * a.Hkv;
    const int64_t there = (static_cast<int64_t>(a.T_tot) / kBK + a.N) * a.Hkv;
    const int64_t strips = (static_cast<int64_t>(w.width) + kStrip - 1) / kStrip * a.N * a.Hkv;
    // A workgroup for every block of keys that there can be, or for every block of the width, most of them empty where
    // a table has room to grow (and the full ones then on few of the XCDs).  A look-up costs a round of loads for 64
    // sequences, which many short ones pay, and in one part a kernel of more registers.  Parts, looked up and by the
    // width, us: 32k tokens in 8 prompts, 32/8 heads of 128, in a table of 8192 positions 816 and 849, of 131072 826
    // and 920; 4000 tokens in one of 4096 108 and 106, of 65536 103 and 125; 16 prompts of 500 in one of 32768 72 and
    // 244; 1000 of 100, 8/1 heads, in one of 256 105 and 71, of 1024 106 and 249.  One part: the last 64 rows of the
    // 32k tokens in a table of 16384 72 and 66, of 131072 75 and 97; of 128 prompts of 500 in one of 1536 116 and 108,
    // of 32768 150 and 341; 4096 of 64, 8/2 heads, in one of 512 292 and 228, of 16384 777 and 2319.
    const bool look_up = static_cast<int64_t>(blocks) * 2048 > (w.parts > 1 ? 1 : 4) * there * (2048 + a.N);
    const float c = a.scale * kLog2e;
    if (!look_up)
        hipLaunchKernelGGL((attn_weights_kernel<BF16, DK, KeyBlocks::kWidth>), dim3(blocks, w.parts), dim3(64 * kWaves), 0, st, w, c);
    else if (w.parts > 1)
        hipLaunchKernelGGL((attn_weights_kernel<BF16, DK, KeyBlocks::kThereInParts>), dim3(static_cast<unsigned>(there), w.parts),
                           dim3(64 * kWaves), 0, st, w, c);
    else
        hipLaunchKernelGGL((attn_weights_kernel<BF16, DK, KeyBlocks::kThere>), dim3(static_cast<unsigned>(there > strips ? there : strips), 2),
                           dim3(64 * kWaves), 0, st, w, c);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || w.parts == 1) return e;
    hipLaunchKernelGGL(attn_weights_join_kernel, dim3(blocks), dim3(256), 0, st, w);
    return hipGetLastError();
}

template <bool BF16>
hipError_t launch_dk(const WeightsArgs& w) {
    switch (w.f.d_k) {
        case 32: return launch<BF16, 32>(w);
        case 64: return launch<BF16, 64>(w);
        default: return launch<BF16, 128>(w);
    }
}

}  // namespace

// Parts that the rows of a block of keys go to.  The first keys of a long sequence have all its rows: one
// workgroup's chain of them is longer than the whole launch should take, and few blocks leave compute
// units idle.  24 workgroups a unit, whose chains differ (32/8 heads of 128, 32k tokens in 8 prompts: 825 us, 889
// with 12, 836 with 48; one of 4000: 99.6, 95.9, 99.2; 4 of 4096, 16/16 heads of 64: 130, 125, 153), in parts of
// eight tiles at least (32k tokens, the last 256 rows: 111 us, 119 with two, 123 with 16; one of 4000: 99.5, 108,
// 96; one of 2000, 4/4 heads: 17, 14, 25), and 64 parts at most (8000 tokens, 8/1 heads: 121 us, 131 with 32 and
// with 128, 124 with 16).
int32_t attn_weights_parts(int32_t N, int64_t T_tot, int32_t Hq, int32_t Hkv, int32_t rows, int cus) {
    const int64_t blocks = (T_tot / kBK + N) * Hkv;
    const int64_t steps = (Hq / Hkv) * (((rows < T_tot ? rows : T_tot) + 63) / 64);  // of the longest chain, at most
    int64_t parts = (24 * static_cast<int64_t>(cus) + blocks - 1) / blocks;
    if (parts > steps / 8) parts = steps / 8;
    return static_cast<int32_t>(parts < 1 ? 1 : parts > 64 ? 64 : parts);
}

hipError_t launch_attn_weights(const WeightsArgs& w) { return w.f.bf16 ? launch_dk<true>(w) : launch_dk<false>(w); }

}  // namespace kda
