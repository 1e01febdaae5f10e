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
#include "attn_tree.hpp"

namespace kda {

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
TreePlan tree_plan(int32_t N, int64_t T_q, int32_t Hq, int32_t Hkv, int32_t d_v, int64_t room, int cus, int32_t most_rows) {
    TreePlan p;
    p.cus = cus;
    const int64_t rows = T_q * (Hq / Hkv);
    const int64_t avg = (rows + N - 1) / N;
    p.rows = avg <= 16 ? 16 : avg <= 32 ? 32 : avg <= 64 ? 64 : 128;
    if (p.rows > most_rows) p.rows = most_rows;
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

hipError_t launch_attn_tree(const TreeArgs& a, const TreePlan& p) {
    return a.T_q == 0 ? hipSuccess : launch_tree<TreeMode::kTree>(a, p);
}

}  // namespace kda
