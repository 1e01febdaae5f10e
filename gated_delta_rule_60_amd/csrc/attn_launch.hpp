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
};

struct AttnBwdArgs {
    AttnArgs f;        // o and lse are read
    const void* d_o;   // [T_tot, Hq, d_v]
    void* d_q;         // [T_tot, Hq, d_k]
    void* d_k;         // [T_tot, Hkv, d_k]
    void* d_v;         // [T_tot, Hkv, d_v]
    void* workspace;   // attn_bwd_workspace_bytes
};

hipError_t launch_attn_prefill(const AttnArgs& a);
hipError_t launch_attn_bwd(const AttnBwdArgs& a);
size_t attn_bwd_workspace_bytes(int64_t T_tot, int32_t Hq);

}  // namespace kda
