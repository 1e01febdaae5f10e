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

// Window and sinks, common to the windowed entry points.
kda_status check_window(int32_t window, int32_t sinks) {
    if (window < 1 || window > (1 << 30)) return fail(KDA_ERR_INVALID_ARG, "window must lie in [1, 2^30]");
    if (sinks < 0 || sinks > kda::kMaxSinks) return fail(KDA_ERR_INVALID_ARG, "sinks must lie in [0, 256]");
    return KDA_OK;
}

int32_t window_heads(int32_t group) { return group % 4 == 0 ? 4 : group % 2 == 0 ? 2 : 1; }

}  // namespace

extern "C" {

kda_status attn_window_prefill(const void* q, const void* k, const void* v, const int32_t* cu_seqlens, int32_t N, int64_t T_tot,
                               int32_t H_q, int32_t H_kv, int32_t d_k, int32_t d_v, int64_t q_stride, int64_t k_stride,
                               int64_t v_stride, int32_t window, int32_t sinks, float scale, kda_dtype dtype, void* o, float* lse,
                               void* stream) {
    kda_status s = check_prefill(q, k, v, cu_seqlens, N, T_tot, H_q, H_kv, d_k, d_v, q_stride, k_stride, v_stride, scale, dtype, o, lse);
    if (s != KDA_OK || (s = check_window(window, sinks)) != KDA_OK) return s;
    if (T_tot == 0) return KDA_OK;
    const kda::AttnArgs a{q, k, v, cu_seqlens, N, static_cast<int32_t>(T_tot), H_q, H_kv, d_k, d_v,
                          static_cast<int32_t>(q_stride), static_cast<int32_t>(k_stride), static_cast<int32_t>(v_stride),
                          scale, dtype == KDA_DTYPE_BF16, o, lse, stream,
                          kda::attn_split(N, T_tot, H_q, dtype == KDA_DTYPE_BF16, kda::device_cus_or_default())};
    (void)hipGetLastError();  // report only this launch's status
    const hipError_t e = kda::launch_attn_window({a, window, sinks, window_heads(H_q / H_kv)});
    return e == hipSuccess ? KDA_OK : hip_fail(e, "windowed attention kernel launch");
}

size_t attn_window_prefill_backward_workspace_size(int32_t N, int64_t T_tot, int32_t H_q, int32_t H_kv, int32_t d_k, int32_t d_v,
                                                   int32_t window, int32_t sinks, kda_dtype dtype) {
    if (N < 1 || T_tot < 0 || T_tot > (int64_t{1} << 30) || H_kv < 1 || H_q < 1 || H_q > 4096 || H_q % H_kv != 0 ||
        !supported_dim(d_k) || !supported_dim(d_v) || (dtype != KDA_DTYPE_BF16 && dtype != KDA_DTYPE_F32) || window < 1 ||
        window > (1 << 30) || sinks < 0 || sinks > kda::kMaxSinks)
        return 0;
    return kda::attn_window_bwd_plan(N, T_tot, H_q, H_kv, d_k, d_v, window, sinks, dtype == KDA_DTYPE_BF16,
                                     kda::device_cus_or_default()).bytes;
}

kda_status attn_window_prefill_backward(const void* q, const void* k, const void* v, const void* o, const float* lse,
                                        const void* d_o, const int32_t* cu_seqlens, int32_t N, int64_t T_tot, int32_t H_q,
                                        int32_t H_kv, int32_t d_k, int32_t d_v, int64_t q_stride, int64_t k_stride,
                                        int64_t v_stride, int32_t window, int32_t sinks, float scale, kda_dtype dtype, void* d_q,
                                        void* d_k_out, void* d_v_out, void* workspace, size_t workspace_bytes, void* stream) {
    kda_status s = check_prefill(q, k, v, cu_seqlens, N, T_tot, H_q, H_kv, d_k, d_v, q_stride, k_stride, v_stride, scale, dtype, o, lse);
    if (s != KDA_OK || (s = check_window(window, sinks)) != KDA_OK) return s;
    if (T_tot > 0 && (!lse || !d_o || !d_q || !d_k_out || !d_v_out))
        return fail(KDA_ERR_INVALID_ARG, "lse, d_o, d_q, d_k and d_v must not be NULL when T_tot > 0");
    for (const void* p : {d_o, static_cast<const void*>(d_q), static_cast<const void*>(d_k_out), static_cast<const void*>(d_v_out)})
        if (!aligned(p, 16)) return fail(KDA_ERR_INVALID_ARG, "gradient pointers must be 16-byte aligned");
    const int cus = kda::device_cus_or_default();
    const kda::WindowBwdPlan plan =
        kda::attn_window_bwd_plan(N, T_tot, H_q, H_kv, d_k, d_v, window, sinks, dtype == KDA_DTYPE_BF16, cus);
    // the sinks' sums: one workgroup of 256 per (piece of rows, 32 sinks, key head), and some for every sequence
    if ((plan.pieces > N ? plan.pieces : N) * plan.blocks * H_kv * 256 >= kMaxItems)
        return fail(KDA_ERR_INVALID_ARG, "N * ceil(sinks / 32) * H_kv too large");
    if (workspace_bytes < plan.bytes)
        return fail(KDA_ERR_INVALID_ARG, "workspace smaller than attn_window_prefill_backward_workspace_size");
    if (T_tot > 0 && !workspace) return fail(KDA_ERR_INVALID_ARG, "workspace must not be NULL");
    if (!aligned(workspace, 256)) return fail(KDA_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
    if (T_tot == 0) return KDA_OK;
    const kda::AttnArgs a{q, k, v, cu_seqlens, N, static_cast<int32_t>(T_tot), H_q, H_kv, d_k, d_v,
                          static_cast<int32_t>(q_stride), static_cast<int32_t>(k_stride), static_cast<int32_t>(v_stride),
                          scale, dtype == KDA_DTYPE_BF16, const_cast<void*>(o), const_cast<float*>(lse), stream,
                          kda::attn_split(N, T_tot, H_q, dtype == KDA_DTYPE_BF16, cus)};
    char* const at = static_cast<char*>(workspace) + plan.stats_bytes;
    float* const sink_parts = reinterpret_cast<float*>(at);
    float* const band_parts = reinterpret_cast<float*>(at + plan.parts_bytes);
    float* const parts = reinterpret_cast<float*>(at + plan.parts_bytes + plan.band_bytes);
    (void)hipGetLastError();  // report only this launch's status
    const hipError_t e = kda::launch_attn_window_bwd({{a, d_o, d_q, d_k_out, d_v_out, workspace, parts, plan.head_parts},
                                                      static_cast<int32_t>(window < T_tot ? window : T_tot), sinks, plan.rows,
                                                      plan.blocks, static_cast<int32_t>(plan.pieces), window_heads(H_q / H_kv), plan.bands,
                                                      sink_parts, band_parts},
                                                     plan);
    return e == hipSuccess ? KDA_OK : hip_fail(e, "windowed attention backward kernel launch");
}

}  // extern "C"

extern "C" {

size_t attn_prefill_weights_workspace_size(int32_t N, int64_t T_tot, int32_t H_q, int32_t H_kv, int32_t rows) {
    if (N < 1 || T_tot < 0 || T_tot > (int64_t{1} << 30) || H_kv < 1 || H_q < 1 || H_q > 4096 || H_q % H_kv != 0 || rows < 1)
        return 0;
    const int32_t parts = kda::attn_weights_parts(N, T_tot, H_q, H_kv, rows, kda::device_cus_or_default());
    return parts > 1 ? static_cast<size_t>(parts) * H_kv * T_tot * sizeof(float) : 0;
}

kda_status attn_prefill_weights(const void* q, const void* k, const float* lse, const int32_t* cu_seqlens, int32_t N,
                                int64_t T_tot, int32_t H_q, int32_t H_kv, int32_t d_k, int64_t q_stride, int64_t k_stride,
                                int32_t rows, float scale, kda_dtype dtype, float* weights, int32_t width, void* workspace,
                                size_t workspace_bytes, void* stream) {
    // the checks of attn_prefill, with the keys in the place of values and the queries in that of outputs
    const kda_status s = check_prefill(q, k, k, cu_seqlens, N, T_tot, H_q, H_kv, d_k, d_k, q_stride, k_stride, k_stride, scale,
                                       dtype, q, lse);
    if (s != KDA_OK) return s;
    if (T_tot > 0 && !lse) return fail(KDA_ERR_INVALID_ARG, "lse must not be NULL when T_tot > 0");
    if (rows < 1) return fail(KDA_ERR_INVALID_ARG, "rows must be at least 1");
    if (width < 1 || width > (1 << 30)) return fail(KDA_ERR_INVALID_ARG, "width must lie in [1, 2^30]");
    if (!weights || !aligned(weights, 4)) return fail(KDA_ERR_INVALID_ARG, "weights must not be NULL, and 4-byte aligned");
    // one workgroup of 256 per (256 positions, sequence, key head)
    if ((static_cast<int64_t>(width) + 255) / 256 * N * H_kv * 256 >= kMaxItems)
        return fail(KDA_ERR_INVALID_ARG, "ceil(width / 256) * N * H_kv too large");
    const size_t need = attn_prefill_weights_workspace_size(N, T_tot, H_q, H_kv, rows);
    if (workspace_bytes < need) return fail(KDA_ERR_INVALID_ARG, "workspace smaller than attn_prefill_weights_workspace_size");
    if (need > 0 && !workspace) return fail(KDA_ERR_INVALID_ARG, "workspace must not be NULL");
    if (!aligned(workspace, 256)) return fail(KDA_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
    const kda::AttnArgs a{q, k, nullptr, cu_seqlens, N, static_cast<int32_t>(T_tot), H_q, H_kv, d_k, d_k,
                          static_cast<int32_t>(q_stride), static_cast<int32_t>(k_stride), 0, scale, dtype == KDA_DTYPE_BF16,
                          nullptr, const_cast<float*>(lse), stream, false};
    (void)hipGetLastError();  // report only this launch's status
    const hipError_t e = kda::launch_attn_weights({a, rows, width, weights,
                                                   kda::attn_weights_parts(N, T_tot, H_q, H_kv, rows, kda::device_cus_or_default()),
                                                   static_cast<float*>(workspace)});
    return e == hipSuccess ? KDA_OK : hip_fail(e, "attention weights kernel launch");
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
bool tree_countable(const kda::TreePlan& p, int64_t T_q, int64_t room, int32_t H_q, int32_t H_kv) {
    const int64_t blocks = room / 128 + 1;
    return T_q * (H_q / H_kv) <= (int64_t{1} << 30) && p.tiles <= INT32_MAX / blocks && (p.items + p.tiles) * H_kv * 512 < kMaxItems;
}

// Sizes that the workspace functions answer for.
bool decode_sizes(int32_t N, int64_t T_q, int32_t H_q, int32_t H_kv, int32_t d_v, int32_t page_size, int32_t max_pages) {
    return N >= 1 && T_q >= 0 && T_q <= (int64_t{1} << 24) && H_kv >= 1 && H_q >= 1 && H_q <= 4096 && H_q % H_kv == 0 &&
           supported_dim(d_v) && pow2(page_size) && page_size <= 4096 && max_pages >= 1 &&
           static_cast<int64_t>(max_pages) * page_size <= (int64_t{1} << 30);
}

// What the entry points over a paged cache have in common; sets page_shift.  `lists` is the last of the
// required lists, `names` what to say of them.
kda_status check_decode(kda::TreeArgs& a, int64_t T_q, int64_t q_stride, kda_dtype dtype, const char* names, const int32_t* lists) {
    kda::set_last_error("");
    if (a.N < 1 || T_q < 0 || T_q > (int64_t{1} << 24)) return fail(KDA_ERR_INVALID_ARG, "need N >= 1 and T_q in [0, 2^24]");
    kda_status s = check_heads(a.Hq, a.Hkv, a.d_k, a.d_v, dtype);
    if (s != KDA_OK) return s;
    if ((s = check_cache(a.n_pages, a.page_size, a.max_pages)) != KDA_OK) return s;
    if ((s = check_scale(a.scale)) != KDA_OK) return s;
    if ((s = check_stride(q_stride, static_cast<int64_t>(a.Hq) * a.d_k, dtype, "q_stride")) != KDA_OK) return s;
    if (!a.block_table || !a.ctx_lens || !lists) return fail(KDA_ERR_INVALID_ARG, names);
    if (T_q > 0 && (!a.q || !a.k_cache || !a.v_cache || !a.o))
        return fail(KDA_ERR_INVALID_ARG, "q, k_cache, v_cache and o must not be NULL when T_q > 0");
    for (const void* p : {a.q, a.k_cache, a.v_cache, static_cast<const void*>(a.o)})
        if (!aligned(p, 16)) return fail(KDA_ERR_INVALID_ARG, "tensor pointers must be 16-byte aligned");
    if (!aligned(a.lse, 4) || !aligned(a.block_table, 4) || !aligned(a.ctx_lens, 4) || !aligned(lists, 4))
        return fail(KDA_ERR_INVALID_ARG, "lse, block_table, ctx_lens and cu_q must be 4-byte aligned");
    a.page_shift = __builtin_ctz(a.page_size);
    return KDA_OK;
}

// The launch shape over at most `room` positions a row tile.
kda_status check_tree_plan(const kda::TreeArgs& a, int64_t room, kda::TreePlan& plan, int32_t most_rows = 128) {
    plan = kda::tree_plan(a.N, a.T_q, a.Hq, a.Hkv, a.d_v, room, kda::device_cus_or_default(), most_rows);
    if (!tree_countable(plan, a.T_q, room, a.Hq, a.Hkv))
        return fail(KDA_ERR_INVALID_ARG, "too many drafted tokens for sequences this long");
    return KDA_OK;
}

kda_status check_tree_workspace(const kda::TreeArgs& a, size_t need, size_t have, const char* size) {
    if (have < need) return fail(KDA_ERR_INVALID_ARG, std::string("workspace smaller than ") + size);
    if (need > 0 && !a.workspace) return fail(KDA_ERR_INVALID_ARG, "workspace must not be NULL");
    if (!aligned(a.workspace, 256)) return fail(KDA_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
    return KDA_OK;
}

// Positions a row tile of up to 128 tokens walks at most.
int64_t window_room(int32_t page_size, int32_t max_pages, int32_t window, int32_t sinks) {
    const int64_t room = static_cast<int64_t>(max_pages) * page_size, most = static_cast<int64_t>(window) + sinks + 128;
    return room < most ? room : most;
}

constexpr int32_t kWeighedRows = 32;  // of a pass

// A weighed step's workspace: the partial results, the scores, and lse if the caller wants none.
struct WeighedBytes {
    size_t scores, lse, all;
    int32_t pitch;
};
WeighedBytes weighed_bytes(int32_t N, int32_t H_q, int64_t room, const kda::TreePlan& plan) {
    WeighedBytes w;
    w.pitch = static_cast<int32_t>((room + 31) / 32 * 32);
    w.scores = (plan.bytes + 255) / 256 * 256;
    w.lse = w.scores + static_cast<size_t>(N) * H_q * w.pitch * sizeof(float);
    w.all = w.lse + static_cast<size_t>(N) * H_q * sizeof(float);
    return w;
}

}  // namespace

extern "C" {

size_t attn_tree_decode_workspace_size(int32_t N, int64_t T_q, int32_t H_q, int32_t H_kv, int32_t d_v, int32_t page_size,
                                       int32_t max_pages) {
    if (!decode_sizes(N, T_q, H_q, H_kv, d_v, page_size, max_pages)) return 0;
    return kda::tree_plan(N, T_q, H_q, H_kv, d_v, static_cast<int64_t>(max_pages) * page_size, kda::device_cus_or_default()).bytes;
}

kda_status attn_tree_decode(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_table,
                            const int32_t* ctx_lens, const int32_t* cu_q, const uint64_t* tree_mask, int32_t N, int64_t T_q,
                            int32_t H_q, int32_t H_kv, int32_t d_k, int32_t d_v, int32_t n_pages, int32_t page_size,
                            int32_t max_pages, int64_t q_stride, float scale, kda_dtype dtype, void* o, float* lse,
                            void* workspace, size_t workspace_bytes, void* stream) {
    kda::TreeArgs a{q, k_cache, v_cache, block_table, ctx_lens, cu_q, reinterpret_cast<const unsigned long long*>(tree_mask),
                    N, static_cast<int32_t>(T_q), H_q, H_kv, d_k, d_v, n_pages, page_size, 0, max_pages,
                    static_cast<int32_t>(q_stride), scale, dtype == KDA_DTYPE_BF16, o, lse, workspace, stream};
    kda_status s = check_decode(a, T_q, q_stride, dtype, "block_table, ctx_lens and cu_q must not be NULL", cu_q);
    if (s != KDA_OK) return s;
    if (!aligned(tree_mask, 8)) return fail(KDA_ERR_INVALID_ARG, "tree_mask must be 8-byte aligned");
    kda::TreePlan plan;
    if ((s = check_tree_plan(a, static_cast<int64_t>(max_pages) * page_size, plan)) != KDA_OK) return s;
    if ((s = check_tree_workspace(a, plan.bytes, workspace_bytes, "attn_tree_decode_workspace_size")) != KDA_OK) return s;
    if (T_q == 0) return KDA_OK;
    (void)hipGetLastError();  // report only this launch's status
    const hipError_t e = kda::launch_attn_tree(a, plan);
    return e == hipSuccess ? KDA_OK : hip_fail(e, "tree attention kernel launch");
}

size_t attn_window_decode_workspace_size(int32_t N, int64_t T_q, int32_t H_q, int32_t H_kv, int32_t d_v, int32_t page_size,
                                         int32_t max_pages, int32_t window, int32_t sinks) {
    if (!decode_sizes(N, T_q, H_q, H_kv, d_v, page_size, max_pages) || window < 1 || window > (1 << 30) || sinks < 0 ||
        sinks > kda::kMaxSinks)
        return 0;
    return kda::tree_plan(N, T_q, H_q, H_kv, d_v, window_room(page_size, max_pages, window, sinks), kda::device_cus_or_default()).bytes;
}

kda_status attn_window_decode(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_table,
                              const int32_t* ctx_lens, const int32_t* cu_q, int32_t N, int64_t T_q, int32_t H_q, int32_t H_kv,
                              int32_t d_k, int32_t d_v, int32_t n_pages, int32_t page_size, int32_t max_pages, int64_t q_stride,
                              int32_t window, int32_t sinks, float scale, kda_dtype dtype, void* o, float* lse, void* workspace,
                              size_t workspace_bytes, void* stream) {
    kda::TreeArgs a{q, k_cache, v_cache, block_table, ctx_lens, cu_q, nullptr,
                    N, static_cast<int32_t>(T_q), H_q, H_kv, d_k, d_v, n_pages, page_size, 0, max_pages,
                    static_cast<int32_t>(q_stride), scale, dtype == KDA_DTYPE_BF16, o, lse, workspace, stream};
    a.window = window;
    a.sinks = sinks;
    kda_status s = check_decode(a, T_q, q_stride, dtype, "block_table, ctx_lens and cu_q must not be NULL", cu_q);
    if (s != KDA_OK || (s = check_window(window, sinks)) != KDA_OK) return s;
    kda::TreePlan plan;
    if ((s = check_tree_plan(a, window_room(page_size, max_pages, window, sinks), plan)) != KDA_OK) return s;
    if ((s = check_tree_workspace(a, plan.bytes, workspace_bytes, "attn_window_decode_workspace_size")) != KDA_OK) return s;
    if (T_q == 0) return KDA_OK;
    (void)hipGetLastError();  // report only this launch's status
    const hipError_t e = kda::launch_attn_window_decode(a, plan);
    return e == hipSuccess ? KDA_OK : hip_fail(e, "windowed decode kernel launch");
}

size_t attn_weighed_decode_workspace_size(int32_t N, int32_t H_q, int32_t H_kv, int32_t d_v, int32_t page_size, int32_t max_pages) {
    if (!decode_sizes(N, N, H_q, H_kv, d_v, page_size, max_pages)) return 0;
    return weighed_bytes(N, H_q, static_cast<int64_t>(max_pages) * page_size,
                         kda::tree_plan(N, N, H_q, H_kv, d_v, static_cast<int64_t>(max_pages) * page_size,
                                        kda::device_cus_or_default(), kWeighedRows)).all;
}

kda_status attn_weighed_decode(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_table,
                               const int32_t* ctx_lens, int32_t N, int32_t H_q, int32_t H_kv, int32_t d_k, int32_t d_v,
                               int32_t n_pages, int32_t page_size, int32_t max_pages, int64_t q_stride, float scale,
                               kda_dtype dtype, void* o, float* lse, float* weights, void* workspace, size_t workspace_bytes,
                               void* stream) {
    kda::TreeArgs a{q, k_cache, v_cache, block_table, ctx_lens, nullptr, nullptr,
                    N, N, H_q, H_kv, d_k, d_v, n_pages, page_size, 0, max_pages,
                    static_cast<int32_t>(q_stride), scale, dtype == KDA_DTYPE_BF16, o, lse, workspace, stream};
    kda_status s = check_decode(a, N, q_stride, dtype, "block_table and ctx_lens must not be NULL", ctx_lens);
    if (s != KDA_OK) return s;
    if (!weights || !aligned(weights, 4)) return fail(KDA_ERR_INVALID_ARG, "weights must not be NULL, and 4-byte aligned");
    const int64_t room = static_cast<int64_t>(max_pages) * page_size;
    kda::TreePlan plan;
    if ((s = check_tree_plan(a, room, plan, kWeighedRows)) != KDA_OK) return s;
    // the weights: workgroups of 256, at most 4096 turns of 1024 positions each
    const int64_t turns = (room + 1023) / 1024 < 4096 ? (room + 1023) / 1024 : 4096;
    if (static_cast<int64_t>(N) * H_kv * turns * 256 >= kMaxItems)
        return fail(KDA_ERR_INVALID_ARG, "N * H_kv too large for sequences this long");
    const WeighedBytes bytes = weighed_bytes(N, H_q, room, plan);
    if ((s = check_tree_workspace(a, bytes.all, workspace_bytes, "attn_weighed_decode_workspace_size")) != KDA_OK) return s;
    a.scores = reinterpret_cast<float*>(static_cast<char*>(workspace) + bytes.scores);
    a.score_pitch = bytes.pitch;
    a.weights = weights;
    if (!a.lse) a.lse = reinterpret_cast<float*>(static_cast<char*>(workspace) + bytes.lse);
    (void)hipGetLastError();  // report only this launch's status
    const hipError_t e = kda::launch_attn_weighed(a, plan);
    return e == hipSuccess ? KDA_OK : hip_fail(e, "weighed decode kernel launch");
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

kda_status kv_evict(int32_t* block_table, int32_t* lens, int32_t* held, int32_t* refs, int32_t* free_list, int32_t* n_free,
                    int32_t n_rows, int32_t n_pages, int32_t page_size, int32_t max_pages, const int32_t* rows, int32_t n,
                    void* k_cache, void* v_cache, int32_t n_layers, int32_t H_kv, int32_t d_k, int32_t d_v, kda_dtype dtype,
                    float* weights, int32_t budget, int32_t recent, int32_t sinks, int32_t* status, void* stream) {
    const void* ptrs[] = {block_table, lens, held, refs, free_list, n_free, rows, status};
    kda_status s = check_pages(ptrs, n > 0 ? 8 : 6, n_rows, n_pages, page_size, max_pages);
    if (s != KDA_OK || (s = check_requests(n)) != KDA_OK) return s;
    kda::CacheArgs c{};
    if ((s = check_layers(k_cache, v_cache, n_layers, H_kv, d_k, d_v, dtype, c)) != KDA_OK) return s;
    if (budget < 1 || budget > (1 << 30) || recent < 0 || sinks < 0 || static_cast<int64_t>(recent) + sinks > budget)
        return fail(KDA_ERR_INVALID_ARG, "need budget in [1, 2^30], recent >= 0, sinks >= 0 and recent + sinks <= budget");
    if (!weights && recent + sinks != budget)
        return fail(KDA_ERR_INVALID_ARG, "without weights the budget must be recent + sinks: there is nothing to choose by");
    if (!aligned(weights, 4)) return fail(KDA_ERR_INVALID_ARG, "weights must be 4-byte aligned");
    if (static_cast<int64_t>(n) * n_layers * H_kv * 1024 >= kMaxItems)
        return fail(KDA_ERR_INVALID_ARG, "n * n_layers * H_kv too large");
    if (overlap(status, n, rows, n) || overlap(status, n, lens, n_rows) || overlap(status, n, held, n_rows) ||
        overlap(status, n, refs, n_pages) || overlap(status, n, block_table, static_cast<int64_t>(n_rows) * max_pages) ||
        overlap(status, n, free_list, n_pages) || overlap(status, n, n_free, 1))
        return fail(KDA_ERR_INVALID_ARG, "status must not lie in rows or the bookkeeping: they are read after it is written");
    (void)hipGetLastError();
    const hipError_t e = kda::launch_kv_evict({block_table, lens, held, refs, free_list, n_free, n_rows, n_pages, page_size,
                                               __builtin_ctz(page_size), max_pages, stream}, c,
                                              {weights, H_kv, budget, recent, sinks}, rows, n, status);
    return e == hipSuccess ? KDA_OK : hip_fail(e, "page kernel launch");
}

}  // extern "C"
