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
    if (!(scale > 0.f) || !std::isfinite(scale)) return fail(KDA_ERR_INVALID_ARG, "scale must be positive and finite");
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
    // workgroups of the launches: one per (piece of at least 64 rows, head)
    if ((T_tot / 64 + 1 + N) * H_q > INT32_MAX) return fail(KDA_ERR_INVALID_ARG, "(T_tot / 64 + N) * H_q too large");
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
                          scale, dtype == KDA_DTYPE_BF16, o, lse, stream};
    (void)hipGetLastError();  // report only this launch's status
    const hipError_t e = kda::launch_attn_prefill(a);
    return e == hipSuccess ? KDA_OK : hip_fail(e, "attention kernel launch");
}

size_t attn_prefill_backward_workspace_size(int64_t T_tot, int32_t H_q) {
    if (T_tot < 0 || T_tot > (int64_t{1} << 30) || H_q < 1 || H_q > 4096) return 0;
    return kda::attn_bwd_workspace_bytes(T_tot, H_q);
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
    if (workspace_bytes < kda::attn_bwd_workspace_bytes(T_tot, H_q))
        return fail(KDA_ERR_INVALID_ARG, "workspace smaller than attn_prefill_backward_workspace_size");
    if (T_tot > 0 && !workspace) return fail(KDA_ERR_INVALID_ARG, "workspace must not be NULL");
    if (!aligned(workspace, 256)) return fail(KDA_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
    if (T_tot == 0) return KDA_OK;
    const kda::AttnArgs a{q, k, v, cu_seqlens, N, static_cast<int32_t>(T_tot), H_q, H_kv, d_k, d_v,
                          static_cast<int32_t>(q_stride), static_cast<int32_t>(k_stride), static_cast<int32_t>(v_stride),
                          scale, dtype == KDA_DTYPE_BF16, const_cast<void*>(o), const_cast<float*>(lse), stream};
    (void)hipGetLastError();  // report only this launch's status
    const hipError_t e = kda::launch_attn_bwd({a, d_o, d_q, d_k_out, d_v_out, workspace});
    return e == hipSuccess ? KDA_OK : hip_fail(e, "attention backward kernel launch");
}

}  // extern "C"
