// attn_weighed.hip -- a decode step over a paged cache that adds its attention
// weights to what every position has drawn so far, gfx950.
//
// For the one token of sequence n, key head g and position j:
//     w[n, g, j] += sum_{h of g} exp(s_hj - lse_h).
// The pass over the keys is attn_tree.hip's.  A weight needs the row's lse,
// which is known only when all chunks of the sequence are joined, so the pass
// also leaves its scores (4 bytes a query head and position, beside the
// 2 d 2 bytes of keys and values a key head that it reads in bf16), and a last
// launch turns them into weights: one read of the scores, one of w and one
// write, against a second pass over the keys (256 sequences of 300 to 4000
// positions, 32/8 heads of 128, bf16: 380 us; one by one under the profiler the
// pass 355, the join 9, the weights 18).  Bound by HBM: 3.9 TB/s of keys, values
// and weights.
#include <cfloat>

#include "attn_tree.hpp"

namespace kda {

namespace {

constexpr int kKeys = 1024;  // positions of a workgroup's turn

}  // namespace

__global__ __launch_bounds__(256) void attn_weigh_kernel(TreeArgs a, float c) {
    const int g = blockIdx.x % a.Hkv, n = blockIdx.x / a.Hkv, group = a.Hq / a.Hkv;
    const int room = a.max_pages * a.page_size;
    int ctx = a.ctx_lens[n];
    ctx = ctx < 0 ? 0 : (ctx > room ? room : ctx);
    const int total = ctx < room ? ctx + 1 : room;
    const float* lse = a.lse + static_cast<size_t>(n) * a.Hq + static_cast<size_t>(g) * group;
    const float* s = a.scores + (static_cast<size_t>(n) * a.Hkv + g) * group * a.score_pitch;
    float* w = a.weights + (static_cast<size_t>(n) * a.Hkv + g) * room;
    for (int k0 = blockIdx.y * kKeys; k0 < total; k0 += gridDim.y * kKeys) {
        float sum[kKeys / 256] = {};
        for (int r = 0; r < group; ++r) {
            // lse is -infinity where every score was below the range of fp32, by the product or by c: from the
            // lowest finite number such scores weigh nothing
            const float l2 = lse[r] == -INFINITY ? -FLT_MAX : lse[r] * kLog2e;
            const float* row = s + static_cast<size_t>(r) * a.score_pitch;
#pragma unroll
            for (int i = 0; i < kKeys / 256; ++i) {
                const int j = k0 + i * 256 + threadIdx.x;
                const float x = j < total ? row[j] : -INFINITY;
                // a position without a page is seen by no row
                sum[i] += x == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(fmaf(x, c, -l2));
            }
        }
#pragma unroll
        for (int i = 0; i < kKeys / 256; ++i) {
            const int j = k0 + i * 256 + threadIdx.x;
            if (j < total) w[j] += sum[i];
        }
    }
}

hipError_t launch_attn_weighed(const TreeArgs& a, const TreePlan& p) {
    const hipError_t e = launch_tree<TreeMode::kWeighed>(a, p);
    if (e != hipSuccess) return e;
    const int64_t rows = static_cast<int64_t>(a.N) * a.Hkv, turns = (static_cast<int64_t>(a.max_pages) * a.page_size + kKeys - 1) / kKeys;
    // Up to 64 workgroups a compute unit, which take a row's positions in turns: one for every 1024 positions of the
    // room are most of them empty where the rows are short (256 of 1000 positions, 32/8 heads, in a table of 131072:
    // 332 us, 279 with 64, 277 with 32 and with 8; one of 32000 beside 255 of 100, in the same: 199, 155, 164, 222).
    int64_t side = (64 * static_cast<int64_t>(p.cus) + rows - 1) / rows;
    if (side > turns) side = turns;
    hipLaunchKernelGGL(attn_weigh_kernel, dim3(static_cast<unsigned>(rows), static_cast<unsigned>(side < 4096 ? side : 4096)), dim3(256), 0,
                       static_cast<hipStream_t>(a.stream), a, a.scale * kLog2e);
    return hipGetLastError();
}

}  // namespace kda
