// attn_launch.hpp -- internal host interface between the C ABI layer and the
// launchers of the softmax-attention and cache-page kernels.  Arguments
// arrive here already validated.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace kda {

// Prompt attention over a packed batch (strides in elements between tokens).
struct AttnArgs {
    const void* q;
    const void* k;
    const void* v;
    const int32_t* cu_seqlens;
    int32_t N;
    int32_t T_tot;
    int32_t Hq, Hkv, d_k, d_v;
    int32_t q_stride, k_stride, v_stride;
    float scale;
    bool bf16;
    void* o;     // [T_tot, Hq, d_v]
    float* lse;  // [T_tot, Hq], natural log
    void* stream;
    bool split;  // attn_split
};

// Whether a batch leaves so many compute units idle that its pieces are split
// over the waves of four times as many workgroups.
bool attn_split(int32_t N, int64_t T_tot, int32_t heads, bool bf16, int cus);

struct AttnBwdArgs {
    AttnArgs f;        // o and lse are read
    const void* d_o;   // [T_tot, Hq, d_v]
    void* d_q;         // [T_tot, Hq, d_k]
    void* d_k;         // [T_tot, Hkv, d_k]
    void* d_v;         // [T_tot, Hkv, d_v]
    void* workspace;   // attn_bwd_plan's bytes
    float* parts;      // [head_parts][T_tot][Hkv][d_k + d_v], if head_parts > 1
    int32_t head_parts;  // 0: whole blocks of 128 keys; else blocks of 32, the query heads in so many parts
};

// Launch shape of the dk/dv pass, and what the backward needs: the row statistics, then the parts.
struct BwdPlan {
    size_t stats_bytes, bytes;
    int32_t head_parts;
};
BwdPlan attn_bwd_plan(int32_t N, int64_t T_tot, int32_t Hq, int32_t Hkv, int32_t d_k, int32_t d_v, bool bf16, int cus);

// The same with a sliding window and sinks: row i sees key j <= i if i - j < window or j < sinks.
struct WindowArgs {
    AttnArgs f;
    int32_t window;  // in [1, 2^30]
    int32_t sinks;   // in [0, kMaxSinks]
    int32_t heads;   // query heads of one key head in a workgroup's four waves: 1, 2 or 4
};
constexpr int32_t kMaxSinks = 256;

// Its backward pass.  The rows past the window of the sinks' keys go to pieces of `rows` rows, each
// with a sum of its own for those keys.
struct WindowBwdArgs {
    AttnBwdArgs b;
    int32_t window;     // at most T_tot
    int32_t sinks;
    int32_t rows;
    int32_t blocks;     // of 32 keys that hold the sinks; 0: no row is past their window
    int32_t pieces;     // at most
    int32_t heads;      // as WindowArgs'
    int32_t bands;      // sequences longer than the window, at most
    float* sink_parts;  // [pieces][head parts][32 blocks][Hkv][d_k + d_v]
    float* band_parts;  // [bands][32 blocks][Hkv][d_k + d_v]: what the window gives those keys (whole blocks only)
};

struct WindowBwdPlan {
    size_t stats_bytes, parts_bytes, band_bytes, bytes;
    int32_t head_parts;  // as BwdPlan's
    int32_t rows, blocks, bands;
    int64_t pieces;
};
WindowBwdPlan attn_window_bwd_plan(int32_t N, int64_t T_tot, int32_t Hq, int32_t Hkv, int32_t d_k, int32_t d_v, int32_t window,
                                   int32_t sinks, bool bf16, int cus);

// Attention of drafted tokens over a paged cache.
struct TreeArgs {
    const void* q;        // [T_q, Hq, d_k], q_stride elements between tokens
    const void* k_cache;  // [n_pages, page_size, Hkv, d_k]
    const void* v_cache;  // [n_pages, page_size, Hkv, d_v]
    const int32_t* block_table;  // [N, max_pages]
    const int32_t* ctx_lens;     // [N]
    const int32_t* cu_q;         // [N + 1]
    const unsigned long long* tree_mask;  // [T_q] or null
    int32_t N, T_q, Hq, Hkv, d_k, d_v;
    int32_t n_pages, page_size, page_shift, max_pages;
    int32_t q_stride;
    float scale;
    bool bf16;
    void* o;
    float* lse;  // may be null
    void* workspace;
    void* stream;
    // set by the launcher
    int32_t chunks_target = 0;
    int32_t items = 0;
    float* part_o = nullptr;
    float* part_ml = nullptr;
    int32_t join_heads = 1;
    // of a window
    int32_t window = 0, sinks = 0;
    // of a weighed step
    float* scores = nullptr;    // [N, Hq, score_pitch]: q . k of every position
    int32_t score_pitch = 0;    // at least the sequence's room, a multiple of 32
    float* weights = nullptr;   // [N, Hkv, room], added to
};

// Launch shape: query rows a pass, row tiles and chunk items at most, and the
// partial results' rows and bytes.
struct TreePlan {
    int32_t rows, target;
    int64_t tiles, items, part_rows;
    size_t bytes;
    bool split;   // sequences may have several chunks
    bool chunky;  // they have many
    int32_t cus;
};

// most_rows: of a pass, 32 (a weighed step's kernels) or 128.
TreePlan tree_plan(int32_t N, int64_t T_q, int32_t Hq, int32_t Hkv, int32_t d_v, int64_t room, int cus, int32_t most_rows = 128);
hipError_t launch_attn_tree(const TreeArgs& a, const TreePlan& p);
hipError_t launch_attn_window_decode(const TreeArgs& a, const TreePlan& p);
hipError_t launch_attn_weighed(const TreeArgs& a, const TreePlan& p);

// The pages of a cache: block table rows and what is kept about them.  Calls
// that only read the table and the lengths leave the rest null.
struct PageArgs {
    int32_t* table;   // [n_rows, max_pages]
    int32_t* lens;    // [n_rows]
    int32_t* held;    // [n_rows] pages of a row
    int32_t* refs;    // [n_pages] rows that hold a page
    int32_t* free;    // [n_pages] free pages, n_free of them
    int32_t* n_free;  // [1]
    int32_t n_rows, n_pages, page_size, page_shift, max_pages;
    void* stream;
};

// The cache [n_layers, n_pages, page_size, row] and new tokens [n_layers, tokens, row]; rows in
// 16-byte units.
struct CacheArgs {
    void* k_cache;
    void* v_cache;
    const void* k_new;
    const void* v_new;
    int32_t n_layers;
    int64_t k_row, v_row;
};

// What kv_evict keeps, and by which weights.
struct EvictArgs {
    float* weights;  // [n_layers, n_rows, Hkv, max_pages page_size], or null: no position between sinks and recent ones is kept
    int32_t Hkv, budget, recent, sinks;
};

// How much attention the positions of prompts have drawn from their last `rows` rows (o and v are not used, lse is read).
struct WeightsArgs {
    AttnArgs f;
    int32_t rows;
    int32_t width;
    float* weights;  // [N, Hkv, width]
    int32_t parts;   // attn_weights_parts
    float* part;     // [parts, Hkv, T_tot], if parts > 1
};

int32_t attn_weights_parts(int32_t N, int64_t T_tot, int32_t Hq, int32_t Hkv, int32_t rows, int cus);

hipError_t launch_attn_weights(const WeightsArgs& w);

hipError_t launch_kv_evict(const PageArgs& a, const CacheArgs& c, const EvictArgs& e, const int32_t* rows, int n, int32_t* status);
hipError_t launch_kv_reserve(const PageArgs& a, const int32_t* rows, const int32_t* n_tokens, int n, int32_t* status);
hipError_t launch_kv_free(const PageArgs& a, const int32_t* rows, int n);
hipError_t launch_kv_fork(const PageArgs& a, const CacheArgs& c, const int32_t* src, const int32_t* dst, int n, int32_t* status);
hipError_t launch_kv_append(const PageArgs& a, const CacheArgs& c, const int32_t* cu_new, int N, int T_new);
hipError_t launch_kv_compact(const PageArgs& a, const CacheArgs& c, const int32_t* accepted, const int32_t* cu_accepted, int N,
                             int A_tot, int32_t* new_lens);

hipError_t launch_attn_prefill(const AttnArgs& a);
hipError_t launch_attn_bwd(const AttnBwdArgs& a);
hipError_t launch_attn_window(const WindowArgs& a);
hipError_t launch_attn_window_bwd(const WindowBwdArgs& a, const WindowBwdPlan& p);

}  // namespace kda
