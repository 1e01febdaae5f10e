// kv_device.hpp -- pieces of the workgroups that keep a cache's pages.
#pragma once

#include "attn_device.hpp"
#include "attn_launch.hpp"

namespace kda {

namespace {

constexpr int kThreads = 1024;  // of the bookkeeping workgroup: one per request

// Inclusive prefix sum over the workgroup's NT threads; `total` in every thread.
template <int NT = kThreads>
__device__ __forceinline__ int64_t block_scan(int64_t x, int64_t* s_wave, int64_t& total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int64_t y = __shfl_up(x, d);
        if (lane >= d) x += y;
    }
    __syncthreads();  // the sums of an earlier scan have been read
    if (lane == 63) s_wave[wave] = x;
    __syncthreads();
    int64_t before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) {
        const int64_t y = s_wave[w];
        if (w < wave) before += y;
        total += y;
    }
    return before + x;
}

// The same for sums that fit 32 bits, by lane moves instead of shuffles.
template <int NT = kThreads>
__device__ __forceinline__ int block_scan(int x, int* s_wave, int& total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    x = wave_scan(x);
    __syncthreads();
    if (lane == 63) s_wave[wave] = x;
    __syncthreads();
    const int all = wave_scan(lane < NT / 64 ? s_wave[lane & (NT / 64 - 1)] : 0);
    total = __builtin_amdgcn_readlane(all, 63);
    return x + (wave ? __builtin_amdgcn_readlane(all, __builtin_amdgcn_readfirstlane(wave) - 1) : 0);
}

// The request that entry e belongs to: the first whose inclusive sum passes e.
template <class N>
__device__ __forceinline__ int request_of(const N* upto, int n, N e) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (upto[mid] > e) hi = mid; else lo = mid + 1;
    }
    return lo;
}

__device__ __forceinline__ int free_pages(const PageArgs& a) {
    const int n = *a.n_free;
    return n < 0 ? 0 : (n > a.n_pages ? a.n_pages : n);
}

}  // namespace

}  // namespace kda
