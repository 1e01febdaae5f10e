// attn_api.cpp -- the softmax-attention part of the C ABI in include/kda.h:
// host-side argument validation before any HIP call.
#include "kda.h"

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <string>

#include "attn_launch.hpp"
#include "kda_launch.hpp"

namespace {

kda_status fail(kda_status s, const std::string& msg) {
    kda::set_last_error(msg.c_str());
    return s;
}

kda_status hip_fail(hipError_t e, const char* what) {
    return fail(KDA_ERR_HIP, std::string(what) + ": " + hipGetErrorString(e));
}

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// Whether int32 arrays of na and nb entries share memory.
bool overlap(const int32_t* a, int64_t na, const int32_t* b, int64_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return na > 0 && nb > 0 && x < y + 4 * static_cast<uintptr_t>(nb) && y < x + 4 * static_cast<uintptr_t>(na);
}

// A launch counts its work items along x in 32 bits.
constexpr int64_t kMaxItems = int64_t{1} << 32;

bool supported_dim(int32_t d) { return d == 32 || d == 64 || d == 128; }

// Head counts, head sizes and type, common to every entry point.
kda_status check_heads(int32_t H_q, int32_t H_kv, int32_t d_k, int32_t d_v, kda_dtype dtype) {
    if (dtype != KDA_DTYPE_BF16 && dtype != KDA_DTYPE_F32)
        return fail(KDA_ERR_UNSUPPORTED, "dtype must be KDA_DTYPE_BF16 or KDA_DTYPE_F32");
    if (!supported_dim(d_k) || !supported_dim(d_v))
        return fail(KDA_ERR_UNSUPPORTED, "d_k and d_v must each be 32, 64 or 128 (got " + std::to_string(d_k) + ", " +
                                             std::to_string(d_v) + ")");
    if (H_kv < 1 || H_q < 1 || H_q % H_kv != 0)
        return fail(KDA_ERR_INVALID_ARG, "need H_kv >= 1 and H_q a positive multiple of H_kv");
    if (H_q > 4096) return fail(KDA_ERR_INVALID_ARG, "H_q must not exceed 4096");
    return KDA_OK;
}

kda_status check_scale(float scale) {
    if (!(scale > 0.f) || !std::isfinite(scale * 1.4427f))  // the kernels work in powers of two
        return fail(KDA_ERR_INVALID_ARG, "scale must be positive, and scale log2(e) finite");
    return KDA_OK;
}

// Elements between tokens: at least one token, 16-byte steps, and small
// enough that the rows of one tile span less than 2^31 bytes.
kda_status check_stride(int64_t stride, int64_t row, kda_dtype dtype, const char* name) {
    const int64_t unit = dtype == KDA_DTYPE_BF16 ? 8 : 4;
    if (stride < row || stride % unit != 0 || stride > (int64_t{1} << 22))
        return fail(KDA_ERR_INVALID_ARG, std::string(name) + " must be at least heads * head size, a multiple of 16 bytes "
                                                             "and at most 2^22 elements");
    return KDA_OK;
}

kda_status check_prefill(const void* q, const void* k, const void* v, const int32_t* cu_seqlens, int32_t N, int64_t T_tot,
                         int32_t H_q, int32_t H_kv, int32_t d_k, int32_t d_v, int64_t q_stride, int64_t k_stride,
                         int64_t v_stride, float scale, kda_dtype dtype, const void* o, const float* lse) {
    kda::set_last_error("");
    if (N < 1 || T_tot < 0) return fail(KDA_ERR_INVALID_ARG, "need N >= 1 and T_tot >= 0");
    kda_status s = check_heads(H_q, H_kv, d_k, d_v, dtype);
    if (s != KDA_OK) return s;
    if ((s = check_scale(scale)) != KDA_OK) return s;
    if ((s = check_stride(q_stride, static_cast<int64_t>(H_q) * d_k, dtype, "q_stride")) != KDA_OK) return s;
    if ((s = check_stride(k_stride, static_cast<int64_t>(H_kv) * d_k, dtype, "k_stride")) != KDA_OK) return s;
    if ((s = check_stride(v_stride, static_cast<int64_t>(H_kv) * d_v, dtype, "v_stride")) != KDA_OK) return s;
    if (!cu_seqlens) return fail(KDA_ERR_INVALID_ARG, "cu_seqlens must not be NULL");
    if (T_tot > 0 && (!q || !k || !v || !o)) return fail(KDA_ERR_INVALID_ARG, "q, k, v and o must not be NULL when T_tot > 0");
    if (T_tot > (int64_t{1} << 30)) return fail(KDA_ERR_INVALID_ARG, "T_tot must not exceed 2^30");
    for (const void* p : {q, k, v, o})
        if (!aligned(p, 16)) return fail(KDA_ERR_INVALID_ARG, "tensor pointers must be 16-byte aligned");
    if (!aligned(lse, 4) || !aligned(cu_seqlens, 4))
        return fail(KDA_ERR_INVALID_ARG, "lse and cu_seqlens must be 4-byte aligned");
    // workgroups of the launches: one of 256 work items per (piece of 128 rows, head)
    if (((T_tot + 127) / 128 + N) * H_q * 256 >= kMaxItems)
        return fail(KDA_ERR_INVALID_ARG, "(ceil(T_tot / 128) + N) * H_q too large");
    return KDA_OK;
}

}  // namespace

extern "C" {

kda_status attn_prefill(const void* q, const void* k, const void* v, const int32_t* cu_seqlens, int32_t N, int64_t T_tot,
                        int32_t H_q, int32_t H_kv, int32_t d_k, int32_t d_v, int64_t q_stride, int64_t k_stride,
                        int64_t v_stride, float scale, kda_dtype dtype, void* o, float* lse, void* stream) {
    const kda_status s = check_prefill(q, k, v, cu_seqlens, N, T_tot, H_q, H_kv, d_k, d_v, q_stride, k_stride, v_stride,
                                       scale, dtype, o, lse);
    if (s != KDA_OK) return s;
    if (T_tot == 0) return KDA_OK;
    const kda::AttnArgs a{q, k, v, cu_seqlens, N, static_cast<int32_t>(T_tot), H_q, H_kv, d_k, d_v,
                          static_cast<int32_t>(q_stride), static_cast<int32_t>(k_stride), static_cast<int32_t>(v_stride),
                          scale, dtype == KDA_DTYPE_BF16, o, lse, stream,
                          kda::attn_split(N, T_tot, H_q, dtype == KDA_DTYPE_BF16, kda::device_cus_or_default())};
    (void)hipGetLastError();  // report only this launch's status
    const hipError_t e = kda::launch_attn_prefill(a);
    return e == hipSuccess ? KDA_OK : hip_fail(e, "attention kernel launch");
}

size_t attn_prefill_backward_workspace_size(int32_t N, int64_t T_tot, int32_t H_q, int32_t H_kv, int32_t d_k, int32_t d_v,
                                            kda_dtype dtype) {
    if (N < 1 || T_tot < 0 || T_tot > (int64_t{1} << 30) || H_kv < 1 || H_q < 1 || H_q > 4096 || H_q % H_kv != 0 ||
        !supported_dim(d_k) || !supported_dim(d_v) || (dtype != KDA_DTYPE_BF16 && dtype != KDA_DTYPE_F32))
        return 0;
    return kda::attn_bwd_plan(N, T_tot, H_q, H_kv, d_k, d_v, dtype == KDA_DTYPE_BF16, kda::device_cus_or_default()).bytes;
}

kda_status attn_prefill_backward(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* d_o,
                                 const int32_t* cu_seqlens, int32_t N, int64_t T_tot, int32_t H_q, int32_t H_kv, int32_t d_k,
                                 int32_t d_v, int64_t q_stride, int64_t k_stride, int64_t v_stride, float scale,
                                 kda_dtype dtype, void* d_q, void* d_k_out, void* d_v_out, void* workspace,
                                 size_t workspace_bytes, void* stream) {
    const kda_status s = check_prefill(q, k, v, cu_seqlens, N, T_tot, H_q, H_kv, d_k, d_v, q_stride, k_stride, v_stride,
                                       scale, dtype, o, lse);
    if (s != KDA_OK) return s;
    if (T_tot > 0 && (!lse || !d_o || !d_q || !d_k_out || !d_v_out))
        return fail(KDA_ERR_INVALID_ARG, "lse, d_o, d_q, d_k and d_v must not be NULL when T_tot > 0");
    for (const void* p : {d_o, static_cast<const void*>(d_q), static_cast<const void*>(d_k_out), static_cast<const void*>(d_v_out)})
        if (!aligned(p, 16)) return fail(KDA_ERR_INVALID_ARG, "gradient pointers must be 16-byte aligned");
    const kda::BwdPlan plan =
        kda::attn_bwd_plan(N, T_tot, H_q, H_kv, d_k, d_v, dtype == KDA_DTYPE_BF16, kda::device_cus_or_default());
    if (workspace_bytes < plan.bytes)
        return fail(KDA_ERR_INVALID_ARG, "workspace smaller than attn_prefill_backward_workspace_size");
    if (T_tot > 0 && !workspace) return fail(KDA_ERR_INVALID_ARG, "workspace must not be NULL");
    if (!aligned(workspace, 256)) return fail(KDA_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
    if (T_tot == 0) return KDA_OK;
    const kda::AttnArgs a{q, k, v, cu_seqlens, N, static_cast<int32_t>(T_tot), H_q, H_kv, d_k, d_v,
                          static_cast<int32_t>(q_stride), static_cast<int32_t>(k_stride), static_cast<int32_t>(v_stride),
                          scale, dtype == KDA_DTYPE_BF16, const_cast<void*>(o), const_cast<float*>(lse), stream,
                          kda::attn_split(N, T_tot, H_q, dtype == KDA_DTYPE_BF16, kda::device_cus_or_default())};
    (void)hipGetLastError();  // report only this launch's status
    const hipError_t e = kda::launch_attn_bwd({a, d_o, d_q, d_k_out, d_v_out, workspace,
                                                reinterpret_cast<float*>(static_cast<char*>(workspace) + plan.stats_bytes),
                                                plan.head_parts});
    return e == hipSuccess ? KDA_OK : hip_fail(e, "attention backward kernel launch");
}

}  // extern "C"

namespace {

bool pow2(int32_t x) { return x > 0 && (x & (x - 1)) == 0; }

// The cache's shape, common to every entry point that reads or writes it.
kda_status check_cache(int32_t n_pages, int32_t page_size, int32_t max_pages) {
    if (!pow2(page_size) || page_size > 4096)
        return fail(KDA_ERR_INVALID_ARG, "page_size must be a power of two, at most 4096");
    if (n_pages < 1 || static_cast<int64_t>(n_pages) * page_size > INT32_MAX)
        return fail(KDA_ERR_INVALID_ARG, "need n_pages >= 1 and fewer than 2^31 positions in the cache");
    if (max_pages < 1 || static_cast<int64_t>(max_pages) * page_size > (int64_t{1} << 30))
        return fail(KDA_ERR_INVALID_ARG, "need max_pages >= 1 and at most 2^30 positions in a sequence");
    return KDA_OK;
}

// Query rows, row tiles times key blocks, and the work items of workgroups of up to 512, must stay
// countable in 32 bits.
bool tree_countable(const kda::TreePlan& p, int64_t T_q, int32_t max_pages, int32_t page_size, int32_t H_q, int32_t H_kv) {
    const int64_t blocks = static_cast<int64_t>(max_pages) * page_size / 128 + 1;
    return T_q * (H_q / H_kv) <= (int64_t{1} << 30) && p.tiles <= INT32_MAX / blocks && (p.items + p.tiles) * H_kv * 512 < kMaxItems;
}

}  // namespace

extern "C" {

size_t attn_tree_decode_workspace_size(int32_t N, int64_t T_q, int32_t H_q, int32_t H_kv, int32_t d_v, int32_t page_size,
                                       int32_t max_pages) {
    if (N < 1 || T_q < 0 || T_q > (int64_t{1} << 24) || H_kv < 1 || H_q < 1 || H_q > 4096 || H_q % H_kv != 0 ||
        !supported_dim(d_v) || !pow2(page_size) || page_size > 4096 || max_pages < 1 ||
        static_cast<int64_t>(max_pages) * page_size > (int64_t{1} << 30))
        return 0;
    return kda::tree_plan(N, T_q, H_q, H_kv, d_v, static_cast<int64_t>(max_pages) * page_size, kda::device_cus_or_default()).bytes;
}

kda_status attn_tree_decode(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_table,
                            const int32_t* ctx_lens, const int32_t* cu_q, const uint64_t* tree_mask, int32_t N, int64_t T_q,
                            int32_t H_q, int32_t H_kv, int32_t d_k, int32_t d_v, int32_t n_pages, int32_t page_size,
                            int32_t max_pages, int64_t q_stride, float scale, kda_dtype dtype, void* o, float* lse,
                            void* workspace, size_t workspace_bytes, void* stream) {
    kda::set_last_error("");
    if (N < 1 || T_q < 0 || T_q > (int64_t{1} << 24)) return fail(KDA_ERR_INVALID_ARG, "need N >= 1 and T_q in [0, 2^24]");
    kda_status s = check_heads(H_q, H_kv, d_k, d_v, dtype);
    if (s != KDA_OK) return s;
    if ((s = check_cache(n_pages, page_size, max_pages)) != KDA_OK) return s;
    if ((s = check_scale(scale)) != KDA_OK) return s;
    if ((s = check_stride(q_stride, static_cast<int64_t>(H_q) * d_k, dtype, "q_stride")) != KDA_OK) return s;
    if (!block_table || !ctx_lens || !cu_q) return fail(KDA_ERR_INVALID_ARG, "block_table, ctx_lens and cu_q must not be NULL");
    if (T_q > 0 && (!q || !k_cache || !v_cache || !o))
        return fail(KDA_ERR_INVALID_ARG, "q, k_cache, v_cache and o must not be NULL when T_q > 0");
    for (const void* p : {q, k_cache, v_cache, static_cast<const void*>(o)})
        if (!aligned(p, 16)) return fail(KDA_ERR_INVALID_ARG, "tensor pointers must be 16-byte aligned");
    if (!aligned(tree_mask, 8)) return fail(KDA_ERR_INVALID_ARG, "tree_mask must be 8-byte aligned");
    if (!aligned(lse, 4) || !aligned(block_table, 4) || !aligned(ctx_lens, 4) || !aligned(cu_q, 4))
        return fail(KDA_ERR_INVALID_ARG, "lse, block_table, ctx_lens and cu_q must be 4-byte aligned");
    const kda::TreePlan plan = kda::tree_plan(N, T_q, H_q, H_kv, d_v, static_cast<int64_t>(max_pages) * page_size,
                                              kda::device_cus_or_default());
    if (!tree_countable(plan, T_q, max_pages, page_size, H_q, H_kv))
        return fail(KDA_ERR_INVALID_ARG, "too many drafted tokens for sequences this long");
    if (workspace_bytes < plan.bytes) return fail(KDA_ERR_INVALID_ARG, "workspace smaller than attn_tree_decode_workspace_size");
    if (plan.bytes > 0 && !workspace) return fail(KDA_ERR_INVALID_ARG, "workspace must not be NULL");
    if (!aligned(workspace, 256)) return fail(KDA_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
    if (T_q == 0) return KDA_OK;
    kda::TreeArgs a{q, k_cache, v_cache, block_table, ctx_lens, cu_q, reinterpret_cast<const unsigned long long*>(tree_mask),
                    N, static_cast<int32_t>(T_q), H_q, H_kv, d_k, d_v, n_pages, page_size, __builtin_ctz(page_size), max_pages,
                    static_cast<int32_t>(q_stride), scale, dtype == KDA_DTYPE_BF16, o, lse, workspace, stream};
    (void)hipGetLastError();  // report only this launch's status
    const hipError_t e = kda::launch_attn_tree(a, plan);
    return e == hipSuccess ? KDA_OK : hip_fail(e, "tree attention kernel launch");
}

}  // extern "C"

namespace {

constexpr int32_t kMaxRequests = 1024;  // of one bookkeeping call

kda_status check_pages(const void* const* ptrs, int count, int32_t n_rows, int32_t n_pages, int32_t page_size, int32_t max_pages) {
    kda::set_last_error("");
    if (n_rows < 1) return fail(KDA_ERR_INVALID_ARG, "need n_rows >= 1");
    const kda_status s = check_cache(n_pages, page_size, max_pages);
    if (s != KDA_OK) return s;
    for (int i = 0; i < count; ++i) {
        if (!ptrs[i]) return fail(KDA_ERR_INVALID_ARG, "block_table, lens, held, refs, free_list, n_free and the requests must not be NULL");
        if (!aligned(ptrs[i], 4)) return fail(KDA_ERR_INVALID_ARG, "int32 pointers must be 4-byte aligned");
    }
    return KDA_OK;
}

kda_status check_requests(int32_t n) {
    if (n < 0 || n > kMaxRequests) return fail(KDA_ERR_INVALID_ARG, "n must lie in [0, 1024]");
    return KDA_OK;
}

// The cache of all layers, its rows in 16-byte units.
kda_status check_layers(const void* k_cache, const void* v_cache, int32_t n_layers, int32_t H_kv, int32_t d_k, int32_t d_v,
                        kda_dtype dtype, kda::CacheArgs& c) {
    const kda_status s = check_heads(H_kv, H_kv, d_k, d_v, dtype);
    if (s != KDA_OK) return s;
    if (n_layers < 1 || n_layers > 65535) return fail(KDA_ERR_INVALID_ARG, "n_layers must lie in [1, 65535]");
    if (!k_cache || !v_cache) return fail(KDA_ERR_INVALID_ARG, "k_cache and v_cache must not be NULL");
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16)) return fail(KDA_ERR_INVALID_ARG, "tensor pointers must be 16-byte aligned");
    const int64_t es = dtype == KDA_DTYPE_BF16 ? 2 : 4;
    c.k_cache = const_cast<void*>(k_cache);
    c.v_cache = const_cast<void*>(v_cache);
    c.n_layers = n_layers;
    c.k_row = H_kv * d_k * es / 16;
    c.v_row = H_kv * d_v * es / 16;
    return KDA_OK;
}

}  // namespace

extern "C" {

kda_status kv_reserve(int32_t* block_table, int32_t* lens, int32_t* held, int32_t* refs, int32_t* free_list, int32_t* n_free,
                      int32_t n_rows, int32_t n_pages, int32_t page_size, int32_t max_pages, const int32_t* rows,
                      const int32_t* n_tokens, int32_t n, int32_t* status, void* stream) {
    const void* ptrs[] = {block_table, lens, held, refs, free_list, n_free, rows, n_tokens, status};
    kda_status s = check_pages(ptrs, n > 0 ? 9 : 6, n_rows, n_pages, page_size, max_pages);
    if (s != KDA_OK || (s = check_requests(n)) != KDA_OK) return s;
    (void)hipGetLastError();
    const hipError_t e = kda::launch_kv_reserve({block_table, lens, held, refs, free_list, n_free, n_rows, n_pages, page_size,
                                                 __builtin_ctz(page_size), max_pages, stream}, rows, n_tokens, n, status);
    return e == hipSuccess ? KDA_OK : hip_fail(e, "page kernel launch");
}

kda_status kv_free(int32_t* block_table, int32_t* lens, int32_t* held, int32_t* refs, int32_t* free_list, int32_t* n_free,
                   int32_t n_rows, int32_t n_pages, int32_t page_size, int32_t max_pages, const int32_t* rows, int32_t n,
                   void* stream) {
    const void* ptrs[] = {block_table, lens, held, refs, free_list, n_free, rows};
    kda_status s = check_pages(ptrs, n > 0 ? 7 : 6, n_rows, n_pages, page_size, max_pages);
    if (s != KDA_OK || (s = check_requests(n)) != KDA_OK) return s;
    if (static_cast<int64_t>(n) * max_pages > (int64_t{1} << 29))
        return fail(KDA_ERR_INVALID_ARG, "n * max_pages must not exceed 2^29");
    (void)hipGetLastError();
    const hipError_t e = kda::launch_kv_free({block_table, lens, held, refs, free_list, n_free, n_rows, n_pages, page_size,
                                              __builtin_ctz(page_size), max_pages, stream}, rows, n);
    return e == hipSuccess ? KDA_OK : hip_fail(e, "page kernel launch");
}

kda_status kv_fork(int32_t* block_table, int32_t* lens, int32_t* held, int32_t* refs, int32_t* free_list, int32_t* n_free,
                   int32_t n_rows, int32_t n_pages, int32_t page_size, int32_t max_pages, const int32_t* src, const int32_t* dst,
                   int32_t n, void* k_cache, void* v_cache, int32_t n_layers, int32_t H_kv, int32_t d_k, int32_t d_v,
                   kda_dtype dtype, int32_t* status, void* stream) {
    const void* ptrs[] = {block_table, lens, held, refs, free_list, n_free, src, dst, status};
    kda_status s = check_pages(ptrs, n > 0 ? 9 : 6, n_rows, n_pages, page_size, max_pages);
    if (s != KDA_OK || (s = check_requests(n)) != KDA_OK) return s;
    kda::CacheArgs c{};
    if ((s = check_layers(k_cache, v_cache, n_layers, H_kv, d_k, d_v, dtype, c)) != KDA_OK) return s;
    if (overlap(status, n, src, n) || overlap(status, n, dst, n))
        return fail(KDA_ERR_INVALID_ARG, "status must not lie in src or dst: the copies read them after it is written");
    (void)hipGetLastError();
    const hipError_t e = kda::launch_kv_fork({block_table, lens, held, refs, free_list, n_free, n_rows, n_pages, page_size,
                                              __builtin_ctz(page_size), max_pages, stream}, c, src, dst, n, status);
    return e == hipSuccess ? KDA_OK : hip_fail(e, "page kernel launch");
}

kda_status kv_append(const void* k, const void* v, void* k_cache, void* v_cache, const int32_t* block_table, const int32_t* lens,
                     const int32_t* cu_new, int32_t N, int64_t T_new, int32_t n_layers, int32_t H_kv, int32_t d_k, int32_t d_v,
                     int32_t n_pages, int32_t page_size, int32_t max_pages, kda_dtype dtype, void* stream) {
    const void* ptrs[] = {block_table, lens, cu_new};
    kda_status s = check_pages(ptrs, 3, N, n_pages, page_size, max_pages);
    if (s != KDA_OK) return s;
    if (T_new < 0 || T_new * 256 >= kMaxItems) return fail(KDA_ERR_INVALID_ARG, "T_new must lie in [0, 2^24)");
    kda::CacheArgs c{};
    if ((s = check_layers(k_cache, v_cache, n_layers, H_kv, d_k, d_v, dtype, c)) != KDA_OK) return s;
    if (T_new > 0 && (!k || !v)) return fail(KDA_ERR_INVALID_ARG, "k and v must not be NULL when T_new > 0");
    if (!aligned(k, 16) || !aligned(v, 16)) return fail(KDA_ERR_INVALID_ARG, "tensor pointers must be 16-byte aligned");
    c.k_new = k;
    c.v_new = v;
    (void)hipGetLastError();
    const hipError_t e = kda::launch_kv_append({const_cast<int32_t*>(block_table), const_cast<int32_t*>(lens), nullptr, nullptr, nullptr,
                                                nullptr, N, n_pages, page_size, __builtin_ctz(page_size), max_pages, stream},
                                               c, cu_new, N, static_cast<int32_t>(T_new));
    return e == hipSuccess ? KDA_OK : hip_fail(e, "page kernel launch");
}

kda_status kv_compact(void* k_cache, void* v_cache, const int32_t* block_table, const int32_t* lens, const int32_t* accepted,
                      const int32_t* cu_accepted, int32_t N, int64_t A_tot, int32_t n_layers, int32_t H_kv, int32_t d_k, int32_t d_v,
                      int32_t n_pages, int32_t page_size, int32_t max_pages, kda_dtype dtype, int32_t* new_lens, void* stream) {
    const void* ptrs[] = {block_table, lens, cu_accepted, new_lens, accepted};
    kda_status s = check_pages(ptrs, A_tot > 0 ? 5 : 4, N, n_pages, page_size, max_pages);
    if (s != KDA_OK) return s;
    if (static_cast<int64_t>(N) * 256 >= kMaxItems) return fail(KDA_ERR_INVALID_ARG, "N must be less than 2^24");
    if (A_tot < 0 || A_tot > (int64_t{1} << 24)) return fail(KDA_ERR_INVALID_ARG, "A_tot must lie in [0, 2^24]");
    kda::CacheArgs c{};
    if ((s = check_layers(k_cache, v_cache, n_layers, H_kv, d_k, d_v, dtype, c)) != KDA_OK) return s;
    if (overlap(new_lens, N, lens, N)) return fail(KDA_ERR_INVALID_ARG, "new_lens must not be lens: every layer's work reads it");
    if (overlap(new_lens, N, accepted, A_tot) || overlap(new_lens, N, cu_accepted, static_cast<int64_t>(N) + 1) ||
        overlap(new_lens, N, block_table, static_cast<int64_t>(N) * max_pages))
        return fail(KDA_ERR_INVALID_ARG, "new_lens must not lie in block_table, accepted or cu_accepted: every layer's work reads them");
    (void)hipGetLastError();
    const hipError_t e = kda::launch_kv_compact({const_cast<int32_t*>(block_table), const_cast<int32_t*>(lens), nullptr, nullptr, nullptr,
                                                 nullptr, N, n_pages, page_size, __builtin_ctz(page_size), max_pages, stream},
                                                c, accepted, cu_accepted, N, static_cast<int32_t>(A_tot), new_lens);
    return e == hipSuccess ? KDA_OK : hip_fail(e, "page kernel launch");
}

}  // extern "C"
