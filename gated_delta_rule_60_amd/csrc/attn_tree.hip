// attn_tree.hip -- softmax attention of drafted tokens over a paged cache,
// gfx950.  One drafted token per sequence is the plain decode step.
//
// Sequence n holds ctx_n committed positions and, behind them, the keys and
// values of its drafted tokens; position p lies in page
// block_table[n][p / page_size] at row p % page_size.  A drafted token sees
// every committed position and the drafted ones its mask names.
//
// The step reads every visible key and value once per key head and does
// little with them (2 H_q / H_kv products a value), so it is bound by HBM
// (256 sequences of 300 to 4000 positions, 32/8 heads of 128, bf16: 0.34 ms,
// 4.7 TB/s of keys and values, and 0.01 ms to join); at 128 rows a pass by the
// softmax's vector work (329 drafted tokens of 12 trees over up to 32k
// positions: 0.17 ms and 0.01 ms to join, the matrix cores busy 10 %).
// The query rows of a key head (drafted tokens x grouped heads) are the
// columns of 16x16 MFMAs, 16 to 128 of them per pass over the keys.  The keys
// of a sequence are cut into chunks of equal work over the whole batch, a
// workgroup each.  A wave holds up to 32 rows.  With no more rows than that
// its waves take 32-key tiles in turn, each with its own running maximum, sum
// and output and its own two tiles in LDS, which the loads fill directly: a
// wave always has a tile in flight and never waits for another.  With more
// rows, four waves share a tile, and all waves load it.  (One wave with 64
// rows spilled: 0.69 ms for the 12 trees, against 0.29 ms with 32 a pass.)
// The waves' results are joined in LDS, the chunks' by a second launch, in a
// fixed order.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "attn_device.hpp"
#include "attn_launch.hpp"
#include "kda_launch.hpp"

namespace kda {

namespace {

constexpr int kTK = 32;      // keys of a wave's tile
constexpr int kBlock = 128;  // chunks are multiples of this many keys
constexpr float kLazyLog2 = 8.f;  // as in attn_prefill.hip

// what the loads of rows outside the cache read instead
__device__ const float kZeroRow[128] = {};

// NQ 16-row groups a wave, RW waves to a tile (KW tiles at a time, TT in a slot of LDS).
template <bool BF16, int DK, int DV, int NQ, int RW>
struct TreeShape {
    static constexpr int ES = BF16 ? 2 : 4;
    static constexpr int KB = kTK * DK * ES, VB = kTK * DV * ES;  // tile bytes
    // two waves a SIMD where the tiles have a load for each (329 drafted tokens of 12 trees: 241 us with one)
    static constexpr int NW = RW == 1 ? (8 * (KB + VB) <= 128 * 1024 ? 4 : 2) : BF16 && DK >= 64 && DV >= 64 ? 8 : 4;
    static constexpr int KW = NW / RW;
    static constexpr int R = 16 * NQ * RW;  // query rows
    // slots: of one wave's tile (RW = 1), or of two tiles that all waves load
    static constexpr int TT = RW == 1 ? 1 : 2;
    static constexpr int SLOT = TT * (KB + VB);
    static constexpr int NS = RW == 1 ? 2 : 4 * SLOT <= 128 * 1024 ? 4 : 2;
    static constexpr int JOIN = KW / 2 * R * (DV + 2) * 4 + NW * 4;
    static constexpr int TILES = (RW == 1 ? NW : 1) * NS * SLOT;
    static constexpr int LDS = TILES > JOIN ? TILES : JOIN;
    static constexpr int WPS = NW == 8 || (LDS <= 80 * 1024 && NW == 4) ? 2 : 1;  // waves a SIMD
};

}  // namespace

// One workgroup's share: query rows [rt R, ...) of sequence n against keys
// [k0, k1); part `item` of the partial results if the sequence has several
// chunks.
struct TreeItem {
    int n, tok0, lq, ctx, rt, chunks, item, k0, k1;
};

struct SeqWork {
    int tok0, lq, ctx, tiles, blocks;
};

__device__ __forceinline__ SeqWork seq_work(const TreeArgs& a, int n, int rows) {
    SeqWork s = {0, 0, 0, 0, 0};
    if (n < a.N) {
        const int2 bl = seq_bounds(a.cu_q, n, a.T_q);
        const int room = a.max_pages * a.page_size;
        int ctx = a.ctx_lens[n];
        ctx = ctx < 0 ? 0 : (ctx > room ? room : ctx);
        const int total = ctx + (bl.y < room - ctx ? bl.y : room - ctx);
        s.tok0 = bl.x;
        s.lq = bl.y;
        s.ctx = ctx;
        s.tiles = (bl.y * (a.Hq / a.Hkv) + rows - 1) / rows;
        s.blocks = (total + kBlock - 1) / kBlock;
    }
    return s;
}

// The work of the first 64 SETS sequences, kept: their loads are in flight together (one decode row:
// 12.8 us, 13.4 with one load after another).  Not in the kernel of 64 and 128 rows, whose loop got slower
// by it (329 tokens of 12 trees: 171 us without, 180 with).
template <int SETS>
struct FirstWork {
    SeqWork s[SETS + 1];
};

template <int SETS>
__device__ __forceinline__ FirstWork<SETS> first_work(const TreeArgs& a, int lane, int rows) {
    FirstWork<SETS> f = {};
#pragma unroll
    for (int b = 0; b < SETS; ++b) f.s[b] = 64 * b < a.N ? seq_work(a, 64 * b + lane, rows) : SeqWork{};
    return f;
}

// Blocks a chunk: the whole batch's (row tile, key block) pairs over a.chunks_target chunks.  Every row
// tile's last chunk is cut short, which makes more chunks than that; with few sequences the chunks are
// made larger until their number fits, so that no compute unit is left with one more than the others.
template <int SETS>
__device__ __forceinline__ int chunk_blocks(const TreeArgs& a, const FirstWork<SETS>& f, int lane, int rows) {
    int sum = 0;
#pragma unroll
    for (int b = 0; b < SETS; ++b) sum += f.s[b].tiles * f.s[b].blocks;
    int tiles = f.s[0].tiles, blocks = f.s[0].blocks;  // of 64 sequences, if there are no more
    for (int n0 = 64 * SETS; n0 < a.N; n0 += 64) {
        const SeqWork s = seq_work(a, n0 + lane, rows);
        sum += s.tiles * s.blocks;
        tiles = s.tiles;
        blocks = s.blocks;
    }
    sum = wave_sum(sum);
    int per = sum / a.chunks_target + (sum % a.chunks_target != 0);
    per = per < 1 ? 1 : per;
    if (a.N <= 64 && 2 * static_cast<int64_t>(wave_sum(tiles)) <= a.chunks_target) {
        // ends: at twice the size they fit
        while (wave_sum(tiles * ((blocks + per - 1) / per)) > a.chunks_target) per += (per + 7) / 8;
    }
    return per;
}

// Row tile `p` of the batch (by_chunk: chunk p, counting every row tile's chunks).
template <int SETS>
__device__ __forceinline__ bool find_item(const TreeArgs& a, int p, int rows, bool by_chunk, TreeItem& t) {
    const int lane = threadIdx.x & 63;
    const FirstWork<SETS> f = first_work<SETS>(a, lane, rows);
    const int per = chunk_blocks<SETS>(a, f, lane, rows);
    int base = 0;  // chunks before
    // whether it is among these 64 sequences, and then whether it is sound
    bool sound = false;
    auto among = [&](const SeqWork& s, int n0) __attribute__((always_inline)) {
        const int chunks = s.blocks > per ? (s.blocks + per - 1) / per : 1;
        const int all = s.tiles * chunks, mine = by_chunk ? all : s.tiles;
        const int upto = wave_scan(mine), upto_chunks = wave_scan(all);
        const int total = __builtin_amdgcn_readlane(upto, 63);
        if (p < total) {
            const int l = __builtin_ctzll(__ballot(upto > p));
            const int r = p - (__builtin_amdgcn_readlane(upto, l) - __builtin_amdgcn_readlane(mine, l));
            if (r < 0) return true;  // offsets that overlap so far that the counts wrap
            t.chunks = __builtin_amdgcn_readlane(chunks, l);
            t.n = n0 + l;
            t.tok0 = __builtin_amdgcn_readlane(s.tok0, l);
            t.lq = __builtin_amdgcn_readlane(s.lq, l);
            t.ctx = __builtin_amdgcn_readlane(s.ctx, l);
            t.rt = by_chunk ? r / t.chunks : r;
            const int c = by_chunk ? r % t.chunks : 0;
            t.item = base + __builtin_amdgcn_readlane(upto_chunks, l) - __builtin_amdgcn_readlane(all, l) + t.rt * t.chunks + c;
            const int blocks = __builtin_amdgcn_readlane(s.blocks, l);
            // even chunks, in blocks
            t.k0 = static_cast<int>(static_cast<int64_t>(blocks) * c / t.chunks) * kBlock;
            t.k1 = static_cast<int>(static_cast<int64_t>(blocks) * (c + 1) / t.chunks) * kBlock;
            sound = true;
            return true;
        }
        p -= total;
        base += __builtin_amdgcn_readlane(upto_chunks, 63);
        return false;
    };
#pragma unroll
    for (int b = 0; b < SETS; ++b)
        if (64 * b < a.N && among(f.s[b], 64 * b)) return sound;
    for (int n0 = 64 * SETS; n0 < a.N; n0 += 64)
        if (among(seq_work(a, n0 + lane, rows), n0)) return sound;
    return false;
}

__device__ __forceinline__ float quad_max(float x) {
    const unsigned u = __float_as_uint(x);
    const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    return half_max(fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
}
__device__ __forceinline__ float quad_sum(float x) {
    const unsigned u = __float_as_uint(x);
    const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    return half_sum(__uint_as_float(r[0]) + __uint_as_float(r[1]));
}

// An LDS address, and a read from one.
__device__ __forceinline__ unsigned lds_at(const char* p) { return static_cast<unsigned>(reinterpret_cast<uintptr_t>((KDA_LDS const char*)p)); }
template <class V>
__device__ __forceinline__ V lds_read(unsigned at) {
    return *reinterpret_cast<KDA_LDS const V*>(at);
}

// 16 bytes a lane from its own address to LDS at `lds` + 16 lane.
__device__ __forceinline__ void load_lds16_from(const char* p, char* lds) {
#if defined(__HIP_DEVICE_COMPILE__)
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)p, (KDA_LDS void*)lds, 16, 0, 0);
#endif
}

template <bool BF16, int DK, int DV, int NQ, int RW>
__global__ __launch_bounds__((64 * TreeShape<BF16, DK, DV, NQ, RW>::NW), (TreeShape<BF16, DK, DV, NQ, RW>::WPS)) void attn_tree_kernel(TreeArgs a, float c) {
    using Sh = TreeShape<BF16, DK, DV, NQ, RW>;
    using T = Elem<BF16>;
    using KT = AttnTile<BF16, DK>;
    using VT = AttnTile<BF16, DV>;
    constexpr int NW = Sh::NW, KW = Sh::KW, R = Sh::R, ES = Sh::ES, KB = Sh::KB, VB = Sh::VB, SLOT = Sh::SLOT, NS = Sh::NS, TT = Sh::TT;
    constexpr int NK = DK / 32, ND = DV / 16;
    constexpr int LW = RW == 1 ? 1 : NW;            // waves that load a slot
    constexpr int TK = TT * kTK;                    // its keys
    constexpr int KI = TT * KB / 1024 / LW, VI = TT * VB / 1024 / LW;  // wave-wide loads of each wave
    static_assert(KI >= 1 && VI >= 1, "every wave loads");
    __shared__ __attribute__((aligned(1024))) char lds[Sh::LDS];

    const int lane = threadIdx.x & 63, g4 = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int kw = wave / RW, rw = wave % RW;  // the wave's tile among KW, its rows among RW
    const int g = blockIdx.x % a.Hkv;
    const int group = a.Hq / a.Hkv;
    TreeItem it;
    if (!find_item<RW == 1 ? 4 : 0>(a, blockIdx.x / a.Hkv, R, true, it)) return;
    const int wrow = it.rt * R + rw * 16 * NQ;  // the wave's first row
    const bool working = wrow < it.lq * group;

    // the lane's query rows: column lane & 15 of each 16-row tile
    typename T::F8 q[NQ][NK];
    unsigned long long sees[NQ];  // drafted positions the row sees
    int own[NQ];                  // its token
#pragma unroll
    for (int x = 0; x < NQ; ++x) {
        const int r = wrow + 16 * x + (lane & 15);
        const int t = r / group, h = g * group + r % group;
        const bool live = t < it.lq;
        const typename T::G* p = static_cast<const typename T::G*>(a.q) + static_cast<size_t>(it.tok0 + (live ? t : 0)) * a.q_stride +
                                 static_cast<size_t>(live ? h : 0) * DK;
#pragma unroll
        for (int kk = 0; kk < NK; ++kk) {
            typename T::F8 f = {};
            if (live) f = *reinterpret_cast<const typename T::F8*>(p + 32 * kk + 8 * g4);
            q[x][kk] = f;
        }
        unsigned long long m = 0;
        if (live) {
            if (a.tree_mask) {
                m = a.tree_mask[it.tok0 + t];
                if (it.lq < 64) m &= (1ull << it.lq) - 1;
            }
        }
        sees[x] = m;
        own[x] = t;
    }

    // Which of the 32 keys from key0 on the row sees, a bit each.  Without a mask a token sees the
    // drafted ones up to itself, however many.
    auto visible = [&](int x, int key0) __attribute__((always_inline)) {
        const int past = key0 - it.ctx;  // committed keys come first: -past of them, or none
        const int upto = a.tree_mask ? -past : own[x] + 1 - past;  // leading keys seen for sure
        unsigned v = upto >= 32 ? ~0u : upto > 0 ? (1u << upto) - 1 : 0u;
        const unsigned long long up = past <= -32 ? 0ull : sees[x] << (past < 0 ? -past : 0);
        const unsigned long long down = past >= 64 ? 0ull : sees[x] >> (past > 0 ? past : 0);
        const unsigned drafted = static_cast<unsigned>(past < 0 ? up : down);
        return a.tree_mask ? v | drafted : v;
    };

    const int room = a.max_pages * a.page_size;
    const int total = it.ctx + (it.lq < room - it.ctx ? it.lq : room - it.ctx);
    const int k1 = it.k1 < total ? it.k1 : total;
    // slots of keys this wave sees go by: its own tiles, every NW-th, or all
    const int all = k1 > it.k0 ? (k1 - it.k0 + TK - 1) / TK : 0;
    const int slots = RW > 1 ? all : all > wave ? (all - wave + NW - 1) / NW : 0;
    char* const mine = lds + (RW == 1 ? wave * NS * SLOT : 0);
    const int32_t* table = a.block_table + static_cast<size_t>(it.n) * a.max_pages;

    auto slot_key = [&](int i) __attribute__((always_inline)) { return it.k0 + (RW == 1 ? wave + i * NW : i) * TK; };
    // token row in the cache of key `lane % TK` of slot i; negative if there is none
    auto lookup = [&](int i) __attribute__((always_inline)) {
        const int pos = slot_key(i) + lane % TK;
        int tok = -1;
        if (i < slots && pos < k1) {
            const int page = table[pos >> a.page_shift];
            if (page >= 0 && page < a.n_pages) tok = (page << a.page_shift) + (pos & (a.page_size - 1));
        }
        return tok;
    };
    const char* const kc = static_cast<const char*>(a.k_cache) + static_cast<size_t>(g) * DK * ES;
    const char* const vc = static_cast<const char*>(a.v_cache) + static_cast<size_t>(g) * DV * ES;
    const size_t krow = static_cast<size_t>(a.Hkv) * DK * ES, vrow = static_cast<size_t>(a.Hkv) * DV * ES;
    const char* const zeros = reinterpret_cast<const char*>(kZeroRow);
    // slot: TT tiles' keys, then their values
    auto stage = [&](int slot, int tok) __attribute__((always_inline)) {
        char* b = mine + slot * SLOT;
        const int w = RW == 1 ? 0 : wave;
#pragma unroll
        for (int i = 0; i < KI; ++i) {
            const int r = (i * LW + w) * KT::RPI + lane / KT::U, u = (lane % KT::U) ^ KT::swz(r);
            const int t = __shfl(tok, r);
            load_lds16_from(t >= 0 ? kc + t * krow + u * 16 : zeros, b + (i * LW + w) * 1024);
        }
#pragma unroll
        for (int i = 0; i < VI; ++i) {
            const int r = (i * LW + w) * VT::RPI + lane / VT::U, u = (lane % VT::U) ^ VT::swz(r);
            const int t = __shfl(tok, r);
            load_lds16_from(t >= 0 ? vc + t * vrow + u * 16 : zeros, b + TT * KB + (i * LW + w) * 1024);
        }
    };

    f32x4_t o[NQ][ND];
    float mc[NQ], l[NQ];
    int poisoned = 0;  // a drafted value of a tile was not finite
#pragma unroll
    for (int x = 0; x < NQ; ++x) {
        mc[x] = -INFINITY;
        l[x] = 0.f;
#pragma unroll
        for (int d = 0; d < ND; ++d) o[x][d] = f32x4_t{};
    }

    // The lane's places in a tile: row lane & 15 and its unit 0 for keys, the quads of columns 0..15
    // for values.  Others differ by bits of the unit alone; taken off the slot's address, which
    // changes, they cost an instruction each and no register.
    const int kat = (lane & 15) * KT::ROWB + (((BF16 ? g4 : 2 * g4) ^ KT::swz(lane & 15)) << 4);
    auto kfrag = [&](const char* kt, int y, int kk) __attribute__((always_inline)) {
        const unsigned p = lds_at(kt) + kat + 16 * y * KT::ROWB;
        if constexpr (BF16) {
            return lds_read<typename T::F8>(p ^ (kk << 6));
        } else {
            const f32x4_t lo = lds_read<f32x4_t>(p ^ (kk << 7)), hi = lds_read<f32x4_t>(p ^ (kk << 7) ^ 16);
            return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        }
    };
    const int vrow0 = 4 * g4 + ((lane & 15) >> 2);
    const int vat0 = vrow0 * VT::ROWB + ((((lane & 3) >> 1) ^ VT::swz(vrow0)) << 4) + (lane & 1) * 8;
    // columns 16 d .. 16 d + 15 of the tile's rows, as the A operand over its 32 rows, for d = d0 and d0 + 1
    auto vfrags = [&](typename T::F8 (&f)[2], const char* vt, int d0) __attribute__((always_inline)) {
        if constexpr (BF16) {
            unsigned at[4];
            bf16x4_t x[4];
            // rows r and r + 16 have the same permutation
#pragma unroll
            for (int n = 0; n < 4; ++n) at[n] = (lds_at(vt) + vat0 + 16 * (n & 1) * VT::ROWB) ^ ((d0 + n / 2) << 5);
            read_quads<4>(x, at);
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) f[n / 2][4 * (n & 1) + e] = x[n][e];
        } else {
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int s = 0; s < 8; ++s) {
                    const int r = 16 * (s >> 2) + 4 * g4 + (s & 3), u = 4 * (d0 + n) + ((lane & 15) >> 2);
                    f[n][s] = *reinterpret_cast<const float*>(vt + r * VT::ROWB + ((u ^ VT::swz(r)) << 4) + (lane & 3) * 4);
                }
        }
    };

    // One tile into the rows' statistics and outputs.  MASKED: the tile holds drafted positions or
    // rows that are not in the cache.
    auto step = [&](auto MASKED, const char* kt, char* vt, int key0, unsigned there) __attribute__((always_inline)) {
        f32x4_t s[NQ][2];
#pragma unroll
        for (int x = 0; x < NQ; ++x)
#pragma unroll
            for (int y = 0; y < 2; ++y) s[x][y] = f32x4_t{};
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int kk = 0; kk < NK; ++kk) {
                const typename T::F8 k = kfrag(kt, y, kk);
#pragma unroll
                for (int x = 0; x < NQ; ++x) s[x][y] = mma8<BF16>(s[x][y], k, q[x][kk]);
            }
        if constexpr (MASKED) {
#pragma unroll
            for (int x = 0; x < NQ; ++x) {
                const unsigned w = (visible(x, key0) & there) >> (4 * g4);
#pragma unroll
                for (int y = 0; y < 2; ++y)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[x][y][e] = (w >> (16 * y + e)) & 1 ? s[x][y][e] : -INFINITY;
            }
        }
        typename T::F8 p[NQ];
#pragma unroll
        for (int x = 0; x < NQ; ++x) {
            float mx = s[x][0][0];
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
                for (int e = 0; e < 4; ++e) mx = fmaxf(mx, s[x][y][e]);
            mx = quad_max(mx) * c;
            if (__any(mx > mc[x] + kLazyLog2)) {
                const float m1 = mx > mc[x] + kLazyLog2 ? mx : mc[x];
                const float r = m1 > mc[x] ? exp2f(mc[x] - m1) : 1.f;
                mc[x] = m1;
                l[x] *= r;
#pragma unroll
                for (int d = 0; d < ND; ++d)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[x][d][e] *= r;
            }
            const float m = mc[x] == -INFINITY ? 0.f : mc[x];  // nothing seen yet: weights are 2^-inf
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s[x][y][e] = __builtin_amdgcn_exp2f(fmaf(s[x][y][e], c, -m));
                    l[x] += s[x][y][e];
                }
            p[x] = acc_frag8<BF16>(s[x][0], s[x][1]);
        }
        // A weight of zero does not keep out an infinity or NaN behind the mask: where the tile has
        // any, drafted positions' are cleared, and added at the end to the rows that see them.
        // (Committed positions are seen by all rows.)
        if (MASKED && VT::template any_nonfinite<kTK>(vt, lane)) {
            poisoned = 1;
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            // not unrolled: its registers would be spilled ones of the loop around (12 trees: 168 us, 171 unrolled)
#pragma unroll 1
            for (int r = 0; r < kTK; ++r)
                if (key0 + r >= it.ctx)
#pragma unroll 1
                    for (int e = lane; e < DV; e += 64) {  // in any order of the row's units
                        typename T::E* y = reinterpret_cast<typename T::E*>(vt + r * VT::ROWB) + e;
                        if (!VT::finite(*y)) *y = static_cast<typename T::E>(0.f);
                    }
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        }
#pragma unroll
        for (int d = 0; d < ND; d += 2) {
            typename T::F8 v[2];
            vfrags(v, vt, d);
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int x = 0; x < NQ; ++x) o[x][d + n] = mma8<BF16>(o[x][d + n], v[n], p[x]);
        }
    };

    // tokens of slots i .. i + NS: one more than are loaded or in flight
    int tok[NS + 1];
#pragma unroll
    for (int n = 0; n < NS; ++n) tok[n] = lookup(n);
    loads_done();
#pragma unroll
    for (int n = 0; n < NS - 1; ++n)
        if (n < slots) stage(n, tok[n]);
    for (int i = 0, slot = 0; i < slots; ++i, slot = slot + 1 == NS ? 0 : slot + 1) {
        tok[NS] = lookup(i + NS);
        // slot i has landed: at most the loads of the NS - 2 after it are still on the way
        const int after = slots - 1 - i;
        if (NS > 2 && after >= NS - 2)
            asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(NS > 2 ? (NS - 2) * (KI + VI) : 0) : "memory");
        else if (RW > 1 || NS > 2)
            asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
        else
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        if constexpr (RW > 1) {  // and every wave's part; all are done with the slot before
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
        }
        if (i + NS - 1 < slots) {
            stage(slot == 0 ? NS - 1 : slot - 1, tok[NS - 1]);
            if constexpr (RW == 1) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(KI + VI) : "memory");
        } else if constexpr (RW == 1) {
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        }
        for (int tt = RW == 1 ? 0 : kw; tt < TT; tt += KW) {
            const char* kt = mine + slot * SLOT + tt * KB;
            char* vt = mine + slot * SLOT + TT * KB + tt * VB;
            const int key0 = slot_key(i) + tt * kTK;
            if (!working || key0 >= k1) break;
            // keys of the tile that exist; drafted ones need a look at the masks
            const unsigned there = static_cast<unsigned>(__ballot(tok[0] >= 0) >> (tt * kTK));
            const bool masked = there != 0xFFFFFFFFu || key0 + kTK > it.ctx;
            if (masked) step(std::true_type{}, kt, vt, key0, there); else step(std::false_type{}, kt, vt, key0, there);
        }
#pragma unroll
        for (int n = 0; n < NS; ++n) tok[n] = tok[n + 1];
    }

    // join the waves, the upper half into the lower until one is left
#pragma unroll
    for (int x = 0; x < NQ; ++x) l[x] = quad_sum(l[x]);
    float* const so = reinterpret_cast<float*>(lds);                  // [KW / 2][RW][NQ][ND][64 lanes][4]
    float* const sm = so + KW / 2 * R * DV;                           // [KW / 2][RW][NQ][16][2]
    int* const sp = reinterpret_cast<int*>(sm + KW / 2 * R * 2);      // [NW]
    __syncthreads();
    if (lane == 0) sp[wave] = poisoned;
    if constexpr (KW > 1) {
        for (int w = KW / 2; w >= 1; w /= 2) {
            if (w < KW / 2) __syncthreads();
            if (kw >= w && kw < 2 * w) {
#pragma unroll
                for (int x = 0; x < NQ; ++x) {
                    const int y = ((kw - w) * RW + rw) * NQ + x;
                    if (g4 == 0) {
                        sm[2 * (y * 16 + lane)] = mc[x];
                        sm[2 * (y * 16 + lane) + 1] = l[x];
                    }
#pragma unroll
                    for (int d = 0; d < ND; ++d) *reinterpret_cast<f32x4_t*>(so + ((y * ND + d) * 64 + lane) * 4) = o[x][d];
                }
            }
            __syncthreads();
            if (kw < w) {
#pragma unroll
                for (int x = 0; x < NQ; ++x) {
                    const int z = (kw * RW + rw) * NQ + x, b = z * 16 + (lane & 15);
                    const float m2 = sm[2 * b], l2 = sm[2 * b + 1];
                    const float m1 = fmaxf(mc[x], m2);
                    const float r1 = mc[x] == m1 ? 1.f : exp2f(mc[x] - m1), r2 = m2 == m1 ? 1.f : exp2f(m2 - m1);
                    mc[x] = m1;
                    l[x] = l[x] * r1 + l2 * r2;
#pragma unroll
                    for (int d = 0; d < ND; ++d) {
                        const f32x4_t y = *reinterpret_cast<const f32x4_t*>(so + ((z * ND + d) * 64 + lane) * 4);
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[x][d][e] = o[x][d][e] * r1 + y[e] * r2;
                    }
                }
            }
        }
    } else {
        __syncthreads();
    }
    if (kw != 0 || !working) return;
#pragma unroll
    for (int w = 0; w < NW; ++w) poisoned |= sp[w];
    if (poisoned) {
#pragma unroll 1
        for (int pos = it.k0 > it.ctx ? it.k0 : it.ctx; pos < k1; ++pos) {
            const int page = table[pos >> a.page_shift];
            if (page < 0 || page >= a.n_pages) continue;
            const size_t t = (static_cast<size_t>(page) << a.page_shift) + (pos & (a.page_size - 1));
            unsigned v1[NQ];
#pragma unroll
            for (int x = 0; x < NQ; ++x) v1[x] = visible(x, pos) & 1;
#pragma unroll
            for (int d = 0; d < ND; ++d) {
                float v[4];
                T::load4(reinterpret_cast<const typename T::G*>(vc + t * vrow) + 16 * d + 4 * g4, v);
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int x = 0; x < NQ; ++x)
                        if (!VT::finite(v[e]) && v1[x]) o[x][d][e] += v[e];
            }
        }
    }
#pragma unroll
    for (int x = 0; x < NQ; ++x) {
        const int rr = (rw * NQ + x) * 16 + (lane & 15), r = it.rt * R + rr;
        const int t = r / group, h = g * group + r % group;
        if (t >= it.lq) continue;
        if (it.chunks == 1) {
            const size_t row = static_cast<size_t>(it.tok0 + t) * a.Hq + h;
            const float inv = l[x] > 0.f ? 1.f / l[x] : (l[x] == 0.f ? 0.f : l[x]);
            typename T::G* p = static_cast<typename T::G*>(a.o) + row * DV + 4 * g4;
#pragma unroll
            for (int d = 0; d < ND; ++d) {
                const float y[4] = {o[x][d][0] * inv, o[x][d][1] * inv, o[x][d][2] * inv, o[x][d][3] * inv};
                T::store4(p + 16 * d, y);
            }
            if (a.lse && g4 == 0) a.lse[row] = (mc[x] + log2f(l[x])) * kLn2;
        } else {
            const size_t row = (static_cast<size_t>(it.item) * a.Hkv + g) * R + rr;
            float* p = a.part_o + row * DV + 4 * g4;
#pragma unroll
            for (int d = 0; d < ND; ++d) *reinterpret_cast<f32x4_t*>(p + 16 * d) = o[x][d];
            if (g4 == 0) {
                a.part_ml[2 * row] = mc[x];
                a.part_ml[2 * row + 1] = l[x];
            }
        }
    }
}

// Joins the chunks of a row tile: o = sum_c 2^(m_c - m) o_c / sum_c 2^(m_c - m) l_c, with a running
// maximum.  CG groups of threads share a row's chunks, and their sums are joined in the groups' order.
// The chunks are a chain of loads, eight of each group in flight, bound by its latency where they are
// many: one sequence of 32k positions and one key head, 16 rows in 250 chunks, 80 us in all with one
// group and 23 with eight; eight are taken where a row tile has 16 chunks and more.
template <bool BF16, int DV, int CG>
__global__ __launch_bounds__(256) void attn_tree_join_kernel(TreeArgs a, int R) {
    using T = Elem<BF16>;
    constexpr int TPR = DV / 4;             // threads of a row's group
    constexpr int ROWS = 256 / TPR / CG;    // rows a workgroup
    __shared__ __attribute__((aligned(16))) float s_o[CG][ROWS][DV];
    __shared__ float s_ml[CG][ROWS][2];
    const int g = blockIdx.x % a.Hkv;
    const int group = a.Hq / a.Hkv;
    TreeItem it;
    if (!find_item<4>(a, blockIdx.x / a.Hkv, R, false, it) || it.chunks == 1) return;
    if (it.item + it.chunks > a.items) return;  // offsets that overlap: no such partial results
    const int x = threadIdx.x / TPR, row = x % ROWS, cg = x / ROWS;
    const int rr = blockIdx.y * ROWS + row;
    const int r = it.rt * R + rr, t = r / group, h = g * group + r % group;
    const bool live = rr < R && t < it.lq;
    if (CG == 1 && !live) return;
    const int d = 4 * (threadIdx.x % TPR);
    const size_t step = static_cast<size_t>(a.Hkv) * R;
    const size_t row0 = (static_cast<size_t>(it.item) * a.Hkv + g) * R + (live ? rr : 0);
    float m = -INFINITY, l = 0.f;
    f32x4_t o = {};
    // a group's next B chunks of those there are; past the last, the last again without weight
    auto add = [&](int c, auto Bc) __attribute__((always_inline)) {
        constexpr int B = Bc;
        float m2[B], l2[B];
        f32x4_t y[B];
#pragma unroll
        for (int b = 0; b < B; ++b) {
            const int cb = c + b * CG;
            const size_t at = row0 + (cb < it.chunks ? cb : it.chunks - 1) * step;
            m2[b] = a.part_ml[2 * at];
            l2[b] = a.part_ml[2 * at + 1];
            y[b] = *reinterpret_cast<const f32x4_t*>(a.part_o + at * DV + d);
        }
        float m1 = m;
#pragma unroll
        for (int b = 0; b < B; ++b) m1 = fmaxf(m1, m2[b]);
        const float w0 = m == m1 ? 1.f : exp2f(m - m1);
        m = m1;
        l *= w0;
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] *= w0;
#pragma unroll
        for (int b = 0; b < B; ++b) {
            if (c + b * CG >= it.chunks) break;
            const float w = m2[b] == m ? 1.f : exp2f(m2[b] - m);
            l = fmaf(l2[b], w, l);
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = fmaf(y[b][e], w, o[e]);
        }
    };
    int c = cg;
    for (; c + 4 * CG < it.chunks; c += 8 * CG) add(c, std::integral_constant<int, 8>{});
    if (c < it.chunks) add(c, std::integral_constant<int, 4>{});
    if constexpr (CG > 1) {
        *reinterpret_cast<f32x4_t*>(&s_o[cg][row][d]) = o;
        if (d == 0) {
            s_ml[cg][row][0] = m;
            s_ml[cg][row][1] = l;
        }
        __syncthreads();
        if (cg > 0 || !live) return;
        // a group without a chunk left -infinity and zeros
        float m1 = m;
#pragma unroll
        for (int k = 1; k < CG; ++k) m1 = fmaxf(m1, s_ml[k][row][0]);
        const float w0 = m == m1 ? 1.f : exp2f(m - m1);
        m = m1;
        l *= w0;
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] *= w0;
#pragma unroll
        for (int k = 1; k < CG; ++k) {
            const float m2 = s_ml[k][row][0], w = m2 == m ? 1.f : exp2f(m2 - m);
            const f32x4_t y = *reinterpret_cast<const f32x4_t*>(&s_o[k][row][d]);
            l = fmaf(s_ml[k][row][1], w, l);
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = fmaf(y[e], w, o[e]);
        }
    }
    const size_t out = static_cast<size_t>(it.tok0 + t) * a.Hq + h;
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
    const float y[4] = {o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv};
    T::store4(static_cast<typename T::G*>(a.o) + out * DV + d, y);
    if (a.lse && d == 0) a.lse[out] = (m + log2f(l)) * kLn2;
}

namespace {

template <bool BF16, int DV, int CG>
hipError_t launch_join(const TreeArgs& a, const TreePlan& p) {
    constexpr int rows = 256 / (DV / 4) / CG;  // of a workgroup
    hipLaunchKernelGGL((attn_tree_join_kernel<BF16, DV, CG>), dim3(static_cast<unsigned>(p.tiles * a.Hkv), (p.rows + rows - 1) / rows),
                       dim3(256), 0, static_cast<hipStream_t>(a.stream), a, p.rows);
    return hipGetLastError();
}

template <bool BF16, int DK, int DV, int NQ, int RW>
hipError_t launch(const TreeArgs& a, const TreePlan& p) {
    using Sh = TreeShape<BF16, DK, DV, NQ, RW>;
    const hipStream_t st = static_cast<hipStream_t>(a.stream);
    hipLaunchKernelGGL((attn_tree_kernel<BF16, DK, DV, NQ, RW>), dim3(static_cast<unsigned>(p.items * a.Hkv)), dim3(64 * Sh::NW), 0,
                       st, a, a.scale * kLog2e);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !p.split) return e;
    return p.chunky ? launch_join<BF16, DV, 8>(a, p) : launch_join<BF16, DV, 1>(a, p);
}

template <bool BF16, int DK, int DV>
hipError_t launch_rows(const TreeArgs& a, const TreePlan& p) {
    switch (p.rows) {
        case 16: return launch<BF16, DK, DV, 1, 1>(a, p);
        case 32: return launch<BF16, DK, DV, 2, 1>(a, p);
        case 64: return launch<BF16, DK, DV, 1, 4>(a, p);
        default: return launch<BF16, DK, DV, 2, 4>(a, p);
    }
}

template <bool BF16, int DK>
hipError_t launch_dv(const TreeArgs& a, const TreePlan& p) {
    switch (a.d_v) {
        case 32: return launch_rows<BF16, DK, 32>(a, p);
        case 64: return launch_rows<BF16, DK, 64>(a, p);
        default: return launch_rows<BF16, DK, 128>(a, p);
    }
}

template <bool BF16>
hipError_t launch_dk(const TreeArgs& a, const TreePlan& p) {
    switch (a.d_k) {
        case 32: return launch_dv<BF16, 32>(a, p);
        case 64: return launch_dv<BF16, 64>(a, p);
        default: return launch_dv<BF16, 128>(a, p);
    }
}

}  // namespace

// Query rows a pass: the smallest of 16, 32, 64 and 128 that holds an average
// sequence's rows (64 sequences of 2000 positions, 32/8 heads of 128: 16 rows
// 107 us, 112 in passes of 32; 32 rows 116 us, 161 in passes of 16, 119 of 64;
// 64 rows 128 us, 196 in passes of 32, 151 of 128; 96 rows 159 us, 219 in
// passes of 64).  One width for the batch: a sequence with more rows than the
// average walks its positions once a pass (255 decode rows at 2000 positions
// 402 us; a tree of 64 tokens beside them at 2000 too: 430, at 32000: 638,
// which alone takes 80).
//
// Chunks: as many as compute units where the row tiles are few, so that each
// has one (one sequence of 32k positions: 31 us, 37 with two a unit, 48 with
// four: every chunk writes and joins its rows' sums).  Else two a unit, which
// evens out ragged sequences (32 of up to 8000 positions: 121 us, 137 with
// one, 132 with four; 329 tokens of 12 trees: 169 us, 202 and 186); four where
// the sequences alone are four a unit and more, and only the longest are cut
// (256 decode rows: 349 us, 359 with two).  Never more than the blocks.
TreePlan tree_plan(int32_t N, int64_t T_q, int32_t Hq, int32_t Hkv, int32_t d_v, int64_t room, int cus) {
    TreePlan p;
    const int64_t rows = T_q * (Hq / Hkv);
    const int64_t avg = (rows + N - 1) / N;
    p.rows = avg <= 16 ? 16 : avg <= 32 ? 32 : avg <= 64 ? 64 : 128;
    p.tiles = rows / p.rows + N;
    if (p.tiles > rows) p.tiles = rows;
    const int64_t blocks = (room + kBlock - 1) / kBlock;
    const int64_t least = N > rows / p.rows ? N : rows / p.rows;  // row tiles
    const int64_t rounds = 4 * least * Hkv <= cus ? 1 : least * Hkv < 4 * static_cast<int64_t>(cus) ? 2 : 4;
    int64_t target = rounds * cus / Hkv;
    if (target < 1) target = 1;
    p.target = static_cast<int32_t>(target);
    p.chunky = target >= 16 * least && blocks >= 16;
    p.split = blocks > 1 && T_q > 0;
    p.items = p.split ? p.tiles + p.target : p.tiles;
    if (p.items > p.tiles * blocks) p.items = p.tiles * (blocks > 0 ? blocks : 1);
    p.part_rows = p.split ? p.items * Hkv * p.rows : 0;
    p.bytes = p.split ? static_cast<size_t>(p.part_rows) * (d_v + 2) * sizeof(float) : 0;
    return p;
}

hipError_t launch_attn_tree(TreeArgs a, const TreePlan& p) {
    if (a.T_q == 0) return hipSuccess;
    a.chunks_target = p.target;
    a.items = static_cast<int32_t>(p.items);
    a.part_o = static_cast<float*>(a.workspace);
    a.part_ml = a.part_o + static_cast<size_t>(p.part_rows) * a.d_v;
    return a.bf16 ? launch_dk<true>(a, p) : launch_dk<false>(a, p);
}

}  // namespace kda
