// kv_pages.hip -- the pages of a key/value cache, gfx950: room for new
// tokens, writing them, moving accepted ones together, sharing a sequence's
// pages with another, and giving pages back.
//
// A row of the block table holds a sequence's pages; refs counts the rows
// that hold a page, and free[0 .. n_free) are the pages nobody holds, taken
// from the end.  Everything lies on the device, so none of these calls waits
// for it.
//
// The bookkeeping of a call (reserve, fork, free) is one workgroup's: its
// requests are a few integers each, and one workgroup gives them one order.
// The results are those of the requests taken one after another, worked out
// for all at once by prefix sums.  What moves bytes (append, compact, fork's
// copy) is spread over the chip, 16 bytes a lane, and bound by HBM.
#include <hip/hip_runtime.h>

#include "attn_device.hpp"
#include "attn_launch.hpp"

namespace kda {

namespace {

constexpr int kThreads = 1024;  // of the bookkeeping workgroup: one per request
constexpr int kAppendLayers = 4;  // of a workgroup of append, its loads in flight together
constexpr int kBatch = 8;       // pages a thread handles at a time, their loads in flight together

enum { kOk = 0, kNoPage = 1, kBadRequest = 2 };

// Inclusive prefix sum over the workgroup's threads; `total` in every thread.
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
    for (int w = 0; w < kThreads / 64; ++w) {
        const int64_t y = s_wave[w];
        if (w < wave) before += y;
        total += y;
    }
    return before + x;
}

// The same for sums that fit 32 bits, by lane moves instead of shuffles.
__device__ __forceinline__ int block_scan(int x, int* s_wave, int& total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    x = wave_scan(x);
    __syncthreads();
    if (lane == 63) s_wave[wave] = x;
    __syncthreads();
    const int all = wave_scan(lane < kThreads / 64 ? s_wave[lane & (kThreads / 64 - 1)] : 0);
    total = __builtin_amdgcn_readlane(all, 63);
    return x + (wave ? __builtin_amdgcn_readlane(all, __builtin_amdgcn_readfirstlane(wave) - 1) : 0);
}

// Whether an earlier request of `list` (n of them, in LDS, the rest of it -1) names the same row;
// `among`: whether any request names `other`.
__device__ __forceinline__ bool repeated(const int* list, int n, int i, int row, int other, bool& among) {
    bool again = false;
    among = false;
    for (int j = 0; j < n; j += 8) {
        int x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = list[j + e];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            again |= x[e] == row && j + e < i;
            among |= x[e] == other;
        }
    }
    return again;
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

__device__ __forceinline__ int load_ref(int32_t* p) { return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }

__device__ __forceinline__ int free_pages(const PageArgs& a) {
    const int n = *a.n_free;
    return n < 0 ? 0 : (n > a.n_pages ? a.n_pages : n);
}

}  // namespace

// ---------------------------------------------------------------------------
// reserve: pages for n_tokens[i] more positions of row rows[i]
// (64 requests: 7 us, a chain of dependent loads and scans)
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(kThreads) void kv_reserve_kernel(PageArgs a, const int32_t* rows, const int32_t* n_tokens, int n,
                                                              int32_t* status) {
    __shared__ int s_row[kThreads], s_held[kThreads];
    __shared__ int64_t s_upto[kThreads], s_wave[kThreads / 64];
    const int i = threadIdx.x;
    const int row = i < n ? rows[i] : -1;
    s_row[i] = row;
    __syncthreads();
    bool among;
    bool good = !repeated(s_row, n, i, row, -2, among) && i < n && row >= 0 && row < a.n_rows;  // a row's first request counts
    int need = 0, held = 0;
    if (good) {
        const int64_t len = a.lens[row], more = n_tokens[i];
        held = a.held[row];
        const int64_t pages = (len + more + a.page_size - 1) >> a.page_shift;
        good = len >= 0 && more >= 0 && held >= 0 && held <= a.max_pages && pages <= a.max_pages;
        if (good && pages > held) need = static_cast<int>(pages - held);
    }
    const int have = free_pages(a);
    int64_t total;
    const int64_t upto = block_scan(need, s_wave, total);
    const bool got = good && (need == 0 || upto <= have);
    s_upto[i] = upto;
    s_held[i] = held;
    __syncthreads();
    if (i < n) status[i] = !good ? kBadRequest : got ? kOk : kNoPage;
    // pages of the requests that got theirs: the last sum that fits
    const int64_t granted_here = got && need > 0 ? upto : 0;
    int64_t granted;
    {
        __syncthreads();
        int64_t m = granted_here;
#pragma unroll
        for (int d = 32; d; d /= 2) {
            const int64_t y = __shfl_xor(m, d);
            m = y > m ? y : m;
        }
        if ((i & 63) == 0) s_wave[i >> 6] = m;
        __syncthreads();
        granted = 0;
        for (int w = 0; w < kThreads / 64; ++w) granted = s_wave[w] > granted ? s_wave[w] : granted;
    }
    for (int64_t e = i; e < granted; e += kThreads) {
        const int r = request_of(s_upto, n, e);
        const int64_t before = r ? s_upto[r - 1] : 0;
        const int page = a.free[have - 1 - e];
        a.table[static_cast<int64_t>(s_row[r]) * a.max_pages + s_held[r] + (e - before)] = page;
        if (page >= 0 && page < a.n_pages) a.refs[page] = 1;
    }
    if (got && need > 0) a.held[row] = held + need;
    if (i == 0 && granted > 0) *a.n_free = static_cast<int>(have - granted);
}

// ---------------------------------------------------------------------------
// free: row rows[i] gives back its pages
// (128 rows of 2900 pages: 16 us, three passes of one workgroup over them)
// ---------------------------------------------------------------------------
// Entry e is page j of request i, counted over all requests.  A page whose
// count falls to zero is freed once, at the first entry that holds it: the
// entries of such a page write e - kMark into its count, and the smallest
// stays.
__global__ __launch_bounds__(kThreads) void kv_free_kernel(PageArgs a, const int32_t* rows, int n) {
    constexpr int kMark = 1 << 30;  // n max_pages <= 2^29
    constexpr int kRound = kBatch * kThreads;
    __shared__ int s_row[kThreads], s_upto[kThreads], s_wave[kThreads / 64];
    const int i = threadIdx.x;
    const int row = i < n ? rows[i] : -1;
    s_row[i] = row;
    __syncthreads();
    bool among;
    const bool good = !repeated(s_row, n, i, row, -2, among) && i < n && row >= 0 && row < a.n_rows;
    int held = 0;
    if (good) {
        held = a.held[row];
        held = held < 0 ? 0 : (held > a.max_pages ? a.max_pages : held);
    }
    int total;
    s_upto[i] = block_scan(held, s_wave, total);
    __syncthreads();
    const int have = free_pages(a);

    // where the thread's entries e0 + b kThreads + i lie in the table, and their pages (-1: none);
    // one round of them stays in registers
    int64_t at[kBatch];
    int page[kBatch], ref[kBatch];
    auto entries = [&](int e0) __attribute__((always_inline)) {
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int e = e0 + b * kThreads + i;
            at[b] = -1;
            if (e0 + b * kThreads < total && e < total) {
                const int r = request_of(s_upto, n, e);
                at[b] = static_cast<int64_t>(s_row[r]) * a.max_pages + (e - (r ? s_upto[r - 1] : 0));
            }
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            page[b] = at[b] >= 0 ? a.table[at[b]] : -1;
            if (page[b] >= a.n_pages) page[b] = -1;
        }
    };
    // Every thread's changes to the counts are made.  They are atomics, made in the L2 that this
    // workgroup's compute unit shares, and are read there (load_ref): to wait for them is enough, and
    // a fence for the whole device, which writes that L2 back, is not needed.
    auto counted = [&]() __attribute__((always_inline)) {
        loads_done();
        __syncthreads();
    };
    auto counts = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int b = 0; b < kBatch; ++b) ref[b] = page[b] >= 0 ? load_ref(&a.refs[page[b]]) : 1;
    };

    for (int e0 = 0; e0 < total; e0 += kRound) {
        entries(e0);
#pragma unroll
        for (int b = 0; b < kBatch; ++b)
            if (page[b] >= 0) atomicSub(&a.refs[page[b]], 1);
    }
    counted();
    for (int e0 = 0; e0 < total; e0 += kRound) {
        if (total > kRound) entries(e0);
        counts();
#pragma unroll
        for (int b = 0; b < kBatch; ++b)
            if (ref[b] == 0 || ref[b] < -(kMark / 2)) atomicMin(&a.refs[page[b]], e0 + b * kThreads + i - kMark);
    }
    counted();
    int pushed = 0;
    for (int e0 = 0; e0 < total; e0 += kRound) {
        if (total > kRound) entries(e0);
        counts();
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            if (e0 + b * kThreads >= total) break;  // the same for every thread
            const bool first = ref[b] == e0 + b * kThreads + i - kMark;
            int all;
            const int upto = block_scan(first ? 1 : 0, s_wave, all);
            if (first) {
                const int to = have + pushed + upto - 1;
                if (to < a.n_pages) a.free[to] = page[b];
                a.refs[page[b]] = 0;
            }
            pushed += all;
            if (at[b] >= 0) a.table[at[b]] = -1;
        }
    }
    if (good) {
        a.held[row] = 0;
        a.lens[row] = 0;
    }
    if (i == 0 && pushed > 0) *a.n_free = have + pushed < a.n_pages ? have + pushed : a.n_pages;
}

// ---------------------------------------------------------------------------
// fork: row dst[i] becomes a copy of row src[i]
// (128 requests: 9 us, dependent loads and scans; the copies below)
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(kThreads) void kv_fork_kernel(PageArgs a, const int32_t* src, const int32_t* dst, int n, int32_t* status) {
    __shared__ int s_dst[kThreads], s_wave[kThreads / 64];
    const int i = threadIdx.x;
    const int from = i < n ? src[i] : -1, to = i < n ? dst[i] : -1;
    s_dst[i] = to;
    __syncthreads();
    // every request sees the rows as they were: nobody copies a row that this call writes, and a
    // row's first request counts
    bool written;
    bool good = !repeated(s_dst, n, i, to, from, written) && i < n && from >= 0 && from < a.n_rows && to >= 0 && to < a.n_rows;
    good = good && !written;
    int len = 0, full = 0, part = 0;
    if (good) {
        len = a.lens[from];
        const int held = a.held[from];
        full = len >> a.page_shift;
        part = (len & (a.page_size - 1)) != 0;
        good = len >= 0 && held <= a.max_pages && full + part <= held && a.held[to] == 0;
    }
    const int need = good ? part : 0;
    const int have = free_pages(a);
    int total;
    const int upto = block_scan(need, s_wave, total);
    const bool got = good && (need == 0 || upto <= have);
    if (i < n) status[i] = !good ? kBadRequest : got ? kOk : kNoPage;
    __syncthreads();  // every request has read the rows
    if (got) {
        if (part) {
            const int page = a.free[have - upto];
            a.table[static_cast<int64_t>(to) * a.max_pages + full] = page;
            if (page >= 0 && page < a.n_pages) a.refs[page] = 1;
        }
        a.lens[to] = len;
        a.held[to] = full + part;
    }
    if (i == 0) *a.n_free = have - (total < have ? total : have);
}

// The shared pages of request x (of one workgroup), and the rows of its last page that hold
// positions, for one layer's keys (z = 0) or values (z = 1).
__global__ __launch_bounds__(256) void kv_fork_copy_kernel(PageArgs a, CacheArgs c, const int32_t* src, const int32_t* dst,
                                                           const int32_t* status) {
    const int i = blockIdx.x;
    if (status[i] != kOk) return;
    const int64_t from = static_cast<int64_t>(src[i]) * a.max_pages, to = static_cast<int64_t>(dst[i]) * a.max_pages;
    const int len = a.lens[dst[i]];
    const int full = len >> a.page_shift, used = len & (a.page_size - 1);
    if (blockIdx.y == 0 && blockIdx.z == 0) {
        for (int p = threadIdx.x; p < full; p += 256) {
            const int page = a.table[from + p];
            a.table[to + p] = page;
            if (page >= 0 && page < a.n_pages) atomicAdd(&a.refs[page], 1);
        }
    }
    if (used == 0) return;
    const int p0 = a.table[from + full], p1 = a.table[to + full];
    if (p0 < 0 || p0 >= a.n_pages || p1 < 0 || p1 >= a.n_pages) return;
    const int64_t row = blockIdx.z ? c.v_row : c.k_row;  // 16-byte units of a position
    const int64_t page = row * a.page_size;
    u32x4_t* base = static_cast<u32x4_t*>(blockIdx.z ? c.v_cache : c.k_cache) + static_cast<int64_t>(blockIdx.y) * a.n_pages * page;
    const u32x4_t* x = base + p0 * page;
    u32x4_t* y = base + p1 * page;
    const int units = static_cast<int>(used * row);
    // cached loads and stores: a parent's page is read by each of its children, and the copies are the
    // next step's to read (128 children, 267 MB read and written: 43 us against 65 past the caches)
    constexpr int B = 8;
    for (int u0 = threadIdx.x; u0 < units; u0 += 256 * B) {
        u32x4_t w[B];
#pragma unroll
        for (int b = 0; b < B; ++b) w[b] = u0 + b * 256 < units ? x[u0 + b * 256] : u32x4_t{};
#pragma unroll
        for (int b = 0; b < B; ++b)
            if (u0 + b * 256 < units) y[u0 + b * 256] = w[b];
    }
}

// ---------------------------------------------------------------------------
// append: token x of the packed new ones to position lens[n] + its number
// (1920 tokens, 8 layers of 8 bf16 heads of 128, 126 MB read and written: 23 us)
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(256) void kv_append_kernel(PageArgs a, CacheArgs c, const int32_t* cu, int N, int T) {
    const int t = blockIdx.x;
    const int lane = threadIdx.x & 63;
    // its sequence: as many as end at or before it
    int n = 0;
    for (int n0 = 0; n0 < N; n0 += 64) {
        const bool before = n0 + lane < N && cu[n0 + lane + 1] <= t;
        const int m = __builtin_popcountll(__ballot(before));
        n += m;
        if (m < 64) break;
    }
    if (n >= N) return;
    const int j = t - cu[n];
    const int64_t pos = static_cast<int64_t>(a.lens[n]) + j;
    if (j < 0 || pos < j || (pos >> a.page_shift) >= a.max_pages) return;
    const int page = a.table[static_cast<int64_t>(n) * a.max_pages + (pos >> a.page_shift)];
    if (page < 0 || page >= a.n_pages) return;
    const int64_t at = (static_cast<int64_t>(page) << a.page_shift) + (pos & (a.page_size - 1));
    const int64_t positions = static_cast<int64_t>(a.n_pages) << a.page_shift;
    const int row = static_cast<int>(c.k_row + c.v_row);
    for (int u = threadIdx.x; u < row; u += 256) {
        const bool is_v = u >= c.k_row;
        const int64_t r = is_v ? c.v_row : c.k_row, w = is_v ? u - c.k_row : u;
        const u32x4_t* x = static_cast<const u32x4_t*>(is_v ? c.v_new : c.k_new) + t * r + w;
        u32x4_t* y = static_cast<u32x4_t*>(is_v ? c.v_cache : c.k_cache) + at * r + w;
        constexpr int B = kAppendLayers;
        const int l0 = blockIdx.y * B;
        u32x4_t z[B];
#pragma unroll
        for (int b = 0; b < B; ++b) z[b] = l0 + b < c.n_layers ? x[static_cast<int64_t>(l0 + b) * T * r] : u32x4_t{};
#pragma unroll
        for (int b = 0; b < B; ++b)
            if (l0 + b < c.n_layers) y[static_cast<int64_t>(l0 + b) * positions * r] = z[b];
    }
}

// ---------------------------------------------------------------------------
// compact: drafted position accepted[i] of sequence n to lens[n] + i
// (700 tokens of 64 sequences in 8 such layers, 46 MB: 15 us)
// ---------------------------------------------------------------------------
// One workgroup a sequence and layer.  A lane owns one 16-byte column of the positions and takes
// the accepted ones in order, a few at a time: it reads them all before it writes any, and a
// target is never behind a source still to come (accepted[i] >= i, rising).
__global__ __launch_bounds__(256) void kv_compact_kernel(PageArgs a, CacheArgs c, const int32_t* accepted, const int32_t* cu, int A_tot,
                                                         int32_t* new_lens) {
    constexpr int kRound = 256;
    __shared__ int64_t s_from[kRound], s_to[kRound];
    __shared__ int s_good;
    const int n = blockIdx.x;
    const int tid = threadIdx.x;
    const int2 bl = seq_bounds(cu, n, A_tot);
    const int64_t len = a.lens[n];
    const int64_t room = static_cast<int64_t>(a.max_pages) << a.page_shift;
    const int64_t positions = static_cast<int64_t>(a.n_pages) << a.page_shift;
    auto place = [&](int64_t pos) __attribute__((always_inline)) -> int64_t {
        if (len < 0 || pos >= room) return -1;
        const int page = a.table[static_cast<int64_t>(n) * a.max_pages + (pos >> a.page_shift)];
        if (page < 0 || page >= a.n_pages) return -1;
        return (static_cast<int64_t>(page) << a.page_shift) + (pos & (a.page_size - 1));
    };
    int done = 0;
    for (int i0 = 0; i0 < bl.y; i0 += kRound) {
        const int i = i0 + tid;
        __syncthreads();
        if (tid == 0) s_good = bl.y - i0 < kRound ? bl.y - i0 : kRound;
        __syncthreads();
        if (i < bl.y) {
            const int64_t x = accepted[bl.x + i];
            const int64_t before = i > 0 ? accepted[bl.x + i - 1] : -1;
            s_from[tid] = x >= i && x > before ? place(len + x) : -1;
            s_to[tid] = place(len + i);
            if (s_from[tid] < 0 || s_to[tid] < 0) atomicMin(&s_good, tid);  // what follows is not accepted either
        }
        __syncthreads();
        const int good = s_good;
        const int row = static_cast<int>(c.k_row + c.v_row);
        for (int u = tid; u < row; u += 256) {
            const bool is_v = u >= c.k_row;
            const int64_t r = is_v ? c.v_row : c.k_row, w = is_v ? u - c.k_row : u;
            u32x4_t* y = static_cast<u32x4_t*>(is_v ? c.v_cache : c.k_cache) + static_cast<int64_t>(blockIdx.y) * positions * r + w;
            constexpr int B = 8;
            for (int k0 = 0; k0 < good; k0 += B) {
                u32x4_t z[B];
#pragma unroll
                for (int b = 0; b < B; ++b) z[b] = k0 + b < good ? y[s_from[k0 + b] * r] : u32x4_t{};
#pragma unroll
                for (int b = 0; b < B; ++b)
                    if (k0 + b < good && s_to[k0 + b] != s_from[k0 + b]) y[s_to[k0 + b] * r] = z[b];
            }
        }
        done = i0 + good;
        if (good < (bl.y - i0 < kRound ? bl.y - i0 : kRound)) break;
    }
    if (blockIdx.y == 0 && tid == 0) new_lens[n] = static_cast<int>(len + done);
}

hipError_t launch_kv_reserve(const PageArgs& a, const int32_t* rows, const int32_t* n_tokens, int n, int32_t* status) {
    if (n == 0) return hipSuccess;
    hipLaunchKernelGGL(kv_reserve_kernel, dim3(1), dim3(kThreads), 0, static_cast<hipStream_t>(a.stream), a, rows, n_tokens, n, status);
    return hipGetLastError();
}

hipError_t launch_kv_free(const PageArgs& a, const int32_t* rows, int n) {
    if (n == 0) return hipSuccess;
    hipLaunchKernelGGL(kv_free_kernel, dim3(1), dim3(kThreads), 0, static_cast<hipStream_t>(a.stream), a, rows, n);
    return hipGetLastError();
}

hipError_t launch_kv_fork(const PageArgs& a, const CacheArgs& c, const int32_t* src, const int32_t* dst, int n, int32_t* status) {
    if (n == 0) return hipSuccess;
    const hipStream_t st = static_cast<hipStream_t>(a.stream);
    hipLaunchKernelGGL(kv_fork_kernel, dim3(1), dim3(kThreads), 0, st, a, src, dst, n, status);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kv_fork_copy_kernel, dim3(n, c.n_layers, 2), dim3(256), 0, st, a, c, src, dst, status);
    return hipGetLastError();
}

hipError_t launch_kv_append(const PageArgs& a, const CacheArgs& c, const int32_t* cu_new, int N, int T_new) {
    if (T_new == 0) return hipSuccess;
    hipLaunchKernelGGL(kv_append_kernel, dim3(T_new, (c.n_layers + kAppendLayers - 1) / kAppendLayers), dim3(256), 0, static_cast<hipStream_t>(a.stream), a, c, cu_new, N, T_new);
    return hipGetLastError();
}

hipError_t launch_kv_compact(const PageArgs& a, const CacheArgs& c, const int32_t* accepted, const int32_t* cu_accepted, int N, int A_tot,
                             int32_t* new_lens) {
    hipLaunchKernelGGL(kv_compact_kernel, dim3(N, c.n_layers), dim3(256), 0, static_cast<hipStream_t>(a.stream), a, c, accepted,
                       cu_accepted, A_tot, new_lens);
    return hipGetLastError();
}

}  // namespace kda
