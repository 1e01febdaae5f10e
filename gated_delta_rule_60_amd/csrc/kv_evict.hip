// kv_evict.hip -- sequences that outgrew their budget of a paged key/value
// cache keep the first `sinks` positions, the last `recent` ones and, of the
// others, those with the most accumulated weight, gfx950.
//
// The choice is each layer's and key head's own: without position encodings a
// cache is a set, so the heads of a page need not hold the same positions, only
// as many.  What is moved is little: with front = budget - recent,
//   - a chosen position before `front` stays where it is;
//   - one behind it goes to the place of a position before `front` that is
//     given up, both in rising order;
//   - the last `recent` positions move together to [front, budget), in order,
//     so that they are still the last ones.
// Against moving all survivors up in order that reads and writes only what
// must change places (a sequence one page over its budget: the page's worth of
// choices and the recent positions, not the whole budget).
//
// One workgroup does all of it for a request, layer and key head: it finds the
// weight that parts the chosen from the others digit by digit (three histograms
// of 2048 bins; the positions with exactly that weight are taken from the
// lowest on), lists both kinds of place, copies 16 bytes a lane, and clears the
// weights behind the budget.  A second launch, one workgroup, gives the pages
// behind the budget back.
//
// Bound by HBM where there are many rows (32 of 700 to 4000 positions down to
// 1024, 8 layers of 8 bf16 heads of 128: 290 us, 4.3 TB/s; 1088 to 1024: 165 us,
// 4.1 TB/s): workgroups of 512 threads, so that one's search overlaps others'
// copies (with places looked up once a move 367 to 324 us; not measured apart).
// A single long row is one workgroup a layer and head (32000 positions to 8192
// in 8 layers: 0.42 ms, 1 TB/s), and a small one a chain of dependent loads and
// scans (300 to 256: 13 us, and 5 for the pages).
#include <hip/hip_runtime.h>

#include <type_traits>

#include "attn_device.hpp"
#include "attn_launch.hpp"
#include "kv_device.hpp"

namespace kda {

namespace {

constexpr int kBins = 2048;
constexpr int kNT = 512;                 // threads of the workgroup that evicts
constexpr int kPer = 4;                  // candidates a thread looks at in a turn
constexpr int kTurn = kPer * kNT;
constexpr int kList = 2 * kTurn;         // places listed at a time: turns until one is full
constexpr int kMoves = 8;                // 16-byte units of a thread in flight

// Weights in rising order as unsigned numbers: -0 is 0, and NaN lies below everything.
__device__ __forceinline__ unsigned order_of(float w) {
    const unsigned u = __float_as_uint(w + 0.f);
    return w != w ? 0u : (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

}  // namespace

// Request i, the same for every thread: its row's length, 0 if nothing is to be done; `good` false if it
// is refused.  A row counts once, and holds its positions in pages that it shares with no other.
__device__ __forceinline__ int evict_request(const PageArgs& a, const int32_t* rows, int i, int& row, bool& good) {
    row = rows[i];
    int bad = 0;
    for (int j = threadIdx.x; j < i; j += kNT) bad |= rows[j] == row;
    good = row >= 0 && row < a.n_rows;
    int len = 0, held = 0;
    if (good) {
        len = a.lens[row];
        held = a.held[row];
        good = len >= 0 && held >= 0 && held <= a.max_pages && len <= static_cast<int64_t>(held) << a.page_shift;
    }
    if (good)
        for (int p = threadIdx.x; p < held; p += kNT) {
            const int page = a.table[static_cast<int64_t>(row) * a.max_pages + p];
            bad |= page < 0 || page >= a.n_pages || a.refs[page] != 1;
        }
    good = !__syncthreads_or(bad) && good;
    return good ? len : 0;
}

__global__ __launch_bounds__(kNT) void kv_evict_kernel(PageArgs a, CacheArgs c, EvictArgs e, const int32_t* rows, int32_t* status) {
    __shared__ int s_hist[kBins], s_wave[kNT / 64], s_pick[2];
    __shared__ int s_src[kList], s_dst[kList];  // the listed positions, from where to where; then their places in the cache
    const int tid = threadIdx.x;
    const int g = blockIdx.x % e.Hkv, layer = blockIdx.x / e.Hkv % c.n_layers, i = blockIdx.x / e.Hkv / c.n_layers;
    int row;
    bool good;
    const int len = evict_request(a, rows, i, row, good);
    if (g == 0 && layer == 0 && tid == 0) status[i] = good ? 0 : 2;
    if (len <= e.budget) return;

    const int32_t* table = a.table + static_cast<int64_t>(row) * a.max_pages;
    auto token = [&](int pos) __attribute__((always_inline)) {
        return (table[pos >> a.page_shift] << a.page_shift) + (pos & (a.page_size - 1));
    };
    float* w = e.weights ? e.weights + ((static_cast<int64_t>(layer) * a.n_rows + row) * e.Hkv + g) * (static_cast<int64_t>(a.max_pages) << a.page_shift)
                         : nullptr;
    const int front = e.budget - e.recent, choose = front - e.sinks;
    const int from = e.sinks, to = len - e.recent;  // the ones to choose from

    // this layer's and head's units of 16 bytes: of a token, and between tokens
    const int64_t positions = static_cast<int64_t>(a.n_pages) << a.page_shift;
    const int ku = static_cast<int>(c.k_row / e.Hkv), vu = static_cast<int>(c.v_row / e.Hkv);
    u32x4_t* const kc = static_cast<u32x4_t*>(c.k_cache) + layer * positions * c.k_row + g * ku;
    u32x4_t* const vc = static_cast<u32x4_t*>(c.v_cache) + layer * positions * c.v_row + g * vu;

    // The first n listed moves: the places of their positions, then 16 bytes a lane.  ORDERED: all of a
    // block is read before any of it is written.
    auto places = [&](int n) __attribute__((always_inline)) {
        for (int m = tid; m < n; m += kNT) {
            s_src[m] = token(s_src[m]);
            s_dst[m] = token(s_dst[m]);
        }
        __syncthreads();
    };
    auto move = [&](int n, auto ORDERED) __attribute__((always_inline)) {
        const int lk = __builtin_ctz(ku), lv = __builtin_ctz(vu), keys = n << lk, all = keys + (n << lv);
        for (int x0 = 0; x0 < all; x0 += kNT * kMoves) {
            u32x4_t y[kMoves];
            // unit x0 + b kNT + tid of the keys and then the values: its place, from the list of places
            auto at = [&](int b, const int* list) __attribute__((always_inline)) {
                const int x = x0 + b * kNT + tid;
                return x < keys ? kc + (list[x >> lk] * c.k_row + (x & (ku - 1))) : vc + (list[(x - keys) >> lv] * c.v_row + ((x - keys) & (vu - 1)));
            };
#pragma unroll
            for (int b = 0; b < kMoves; ++b)
                if (x0 + b * kNT + tid < all) y[b] = *at(b, s_src);
            if constexpr (ORDERED) {
                loads_done();
                __syncthreads();
            }
#pragma unroll
            for (int b = 0; b < kMoves; ++b)
                if (x0 + b * kNT + tid < all) *at(b, s_dst) = y[b];
        }
    };

    // Up to kFew candidates stay in registers, in the order of two turns.
    constexpr int kFew = 2 * kTurn;
    const bool few = to - from <= kFew;
    unsigned kept_keys[kFew / kNT];
    auto few_position = [&](int x) __attribute__((always_inline)) { return from + x / kPer * kTurn + kPer * tid + x % kPer; };
    if (choose > 0) {
        if (few) {
#pragma unroll
            for (int x = 0; x < kFew / kNT; ++x) kept_keys[x] = few_position(x) < to ? order_of(w[few_position(x)]) : 0u;
        }
        // the weight `least` that the choose-th heaviest has, and how many of exactly that are chosen
        unsigned least = 0, known = 0;  // digits found so far, and their bits
        int ties = choose;
        for (int shift = 21; shift >= 0; shift = shift == 21 ? 10 : shift == 10 ? 0 : -1) {
            const unsigned bins = shift == 0 ? 1024 : kBins;
            for (int b = tid; b < kBins; b += kNT) s_hist[b] = 0;
            __syncthreads();
            auto count = [&](unsigned x) __attribute__((always_inline)) {
                if ((x & known) == least) atomicAdd(&s_hist[(x >> shift) & (bins - 1)], 1);
            };
            if (few) {
#pragma unroll
                for (int x = 0; x < kFew / kNT; ++x)
                    if (few_position(x) < to) count(kept_keys[x]);
            } else {
                for (int p = from + tid; p < to; p += kNT) count(order_of(w[p]));
            }
            __syncthreads();
            // a thread has four bins, from the top down: the bin in which the count passes `ties`
            constexpr int B = kBins / kNT;
            const int top = kBins - 1 - B * tid;
            int n = 0, all;
#pragma unroll
            for (int x = 0; x < B; ++x) n += s_hist[top - x];
            int before = block_scan<kNT>(n, s_wave, all) - n;
#pragma unroll
            for (int x = 0; x < B; ++x) {
                const int m = s_hist[top - x];
                if (before < ties && before + m >= ties) {
                    s_pick[0] = top - x;
                    s_pick[1] = ties - before;
                }
                before += m;
            }
            __syncthreads();
            least |= static_cast<unsigned>(s_pick[0]) << shift;
            known |= (bins - 1) << shift;
            ties = s_pick[1];
        }

        // the listed moves, n of them: weights, keys and values
        auto carry_out = [&](int n) __attribute__((always_inline)) {
            for (int m = tid; m < n; m += kNT) w[s_dst[m]] = w[s_src[m]];
            places(n);
            move(n, std::false_type{});
        };
        if (few) {
            // counts of the two turns in the halves of one number
            int eq = 0, all;
#pragma unroll
            for (int x = 0; x < kFew / kNT; ++x) eq += (few_position(x) < to && kept_keys[x] == least) << (x / kPer * 16);
            int rank = block_scan<kNT>(eq, s_wave, all) - eq;
            rank += (all & 0xFFFF) << 16;  // the first turn's come before
            int gone = 0, come = 0;
            bool is_gone[kFew / kNT], is_come[kFew / kNT];
#pragma unroll
            for (int x = 0; x < kFew / kNT; ++x) {
                const int p = few_position(x), half = x / kPer * 16;
                const bool same = kept_keys[x] == least;
                const bool kept = kept_keys[x] > least || (same && ((rank >> half) & 0xFFFF) < ties);
                if (p < to && same) rank += 1 << half;
                is_gone[x] = p < front && !kept;
                is_come[x] = p >= front && p < to && kept;
                gone += is_gone[x] << half;
                come += is_come[x] << half;
            }
            int all_gone, all_come;
            int g0 = block_scan<kNT>(gone, s_wave, all_gone) - gone, c0 = block_scan<kNT>(come, s_wave, all_come) - come;
            g0 += (all_gone & 0xFFFF) << 16;
            c0 += (all_come & 0xFFFF) << 16;
#pragma unroll
            for (int x = 0; x < kFew / kNT; ++x) {
                const int half = x / kPer * 16;
                if (is_gone[x]) {
                    s_dst[(g0 >> half) & 0xFFFF] = few_position(x);
                    g0 += 1 << half;
                }
                if (is_come[x]) {
                    s_src[(c0 >> half) & 0xFFFF] = few_position(x);
                    c0 += 1 << half;
                }
            }
            __syncthreads();
            carry_out((all_gone & 0xFFFF) + (all_gone >> 16));
        } else {
            // chosen ones before `front`
            int over = 0, equal = 0;
            for (int p = from + tid; p < front; p += kNT) {
                const unsigned x = order_of(w[p]);
                over += x > least;
                equal += x == least;
            }
            int over_front, equal_front;
            block_scan<kNT>(over, s_wave, over_front);
            block_scan<kNT>(equal, s_wave, equal_front);
            const int moves = choose - over_front - (equal_front < ties ? equal_front : ties);

            // Two streams of places, each in rising order: given up before `front`, chosen behind it.  A turn is
            // looked at once: a place that has been filled has another weight.
            struct Stream {
                int pos, equal;  // where it goes on, and equal weights before
                int n;           // listed
            };
            Stream gone{from, 0, 0}, come{front, equal_front, 0};
            auto list = [&](Stream& s, int end, bool want, int* out) __attribute__((always_inline)) {
                while (s.pos < end && s.n <= kList - kTurn) {
                    bool over[kPer], same[kPer];
                    int eq = 0;
#pragma unroll
                    for (int x = 0; x < kPer; ++x) {
                        const int p = s.pos + kPer * tid + x;
                        const unsigned y = p < end ? order_of(w[p]) : 0u;
                        over[x] = p < end && y > least;
                        same[x] = p < end && y == least;
                        eq += same[x];
                    }
                    int all_equal, all_found;
                    int rank_equal = s.equal + block_scan<kNT>(eq, s_wave, all_equal) - eq;
                    bool found[kPer];
                    int n = 0;
#pragma unroll
                    for (int x = 0; x < kPer; ++x) {
                        const bool kept = over[x] || (same[x] && rank_equal < ties);
                        rank_equal += same[x];
                        found[x] = kept == want && s.pos + kPer * tid + x < end;
                        n += found[x];
                    }
                    int at = s.n + block_scan<kNT>(n, s_wave, all_found) - n;
#pragma unroll
                    for (int x = 0; x < kPer; ++x)
                        if (found[x]) out[at++] = s.pos + kPer * tid + x;
                    s.pos += kTurn;
                    s.equal += all_equal;
                    s.n += all_found;
                }
            };
            // the first n of a list are done: the others move up
            auto used = [&](Stream& s, int n, int* out) __attribute__((always_inline)) {
                int rest[kList / kNT];
#pragma unroll
                for (int x = 0; x < kList / kNT; ++x) {
                    const int at = x * kNT + tid;
                    rest[x] = at < s.n - n ? out[n + at] : 0;
                }
                __syncthreads();
#pragma unroll
                for (int x = 0; x < kList / kNT; ++x) {
                    const int at = x * kNT + tid;
                    if (at < s.n - n) out[at] = rest[x];
                }
                s.n -= n;
            };
            for (int done = 0; done < moves;) {
                list(gone, front, false, s_dst);
                list(come, to, true, s_src);
                __syncthreads();
                const int n = gone.n < come.n ? gone.n : come.n;  // at least one: each is listed until it is long or all there
                carry_out(n);
                done += n;
                __syncthreads();
                if (done < moves) {
                    used(gone, n, s_dst);
                    used(come, n, s_src);
                    __syncthreads();
                }
            }
        }
    }

    // The last ones, in order, each block of them read before it is written; its writes lie before every
    // later block's reads.
    const int back = len - e.budget;
    for (int m0 = 0; m0 < e.recent; m0 += kList) {
        const int n = e.recent - m0 < kList ? e.recent - m0 : kList;
        __syncthreads();  // what goes to places in front has been read, and the list used
        for (int m = tid; m < n; m += kNT) {
            s_src[m] = front + m0 + m + back;
            s_dst[m] = front + m0 + m;
        }
        places(n);
        move(n, std::true_type{});
    }
    __syncthreads();
    if (!w) return;
    for (int m0 = 0; m0 < e.recent; m0 += kNT) {
        const int m = m0 + tid;
        const float x = m < e.recent ? w[front + m + back] : 0.f;
        loads_done();
        __syncthreads();
        if (m < e.recent) w[front + m] = x;
    }
    __syncthreads();  // written before cleared, read before cleared
    for (int p = e.budget + tid; p < len; p += kNT) w[p] = 0.f;
}

// The pages behind the budget go back, in the order of the requests and of the rows' pages.
__global__ __launch_bounds__(kThreads) void kv_evict_pages_kernel(PageArgs a, int budget, const int32_t* rows, int n, const int32_t* status) {
    __shared__ int s_row[kThreads];
    __shared__ int64_t s_upto[kThreads], s_wave[kThreads / 64];
    const int i = threadIdx.x;
    int row = -1, give = 0;
    const int need = (budget + a.page_size - 1) >> a.page_shift;
    if (i < n && status[i] == 0) {
        row = rows[i];
        if (a.lens[row] > budget) {
            a.lens[row] = budget;
            give = a.held[row] - need;
            a.held[row] = need;
        }
    }
    s_row[i] = row;
    int64_t total;
    s_upto[i] = block_scan(static_cast<int64_t>(give), s_wave, total);
    const int have = free_pages(a);
    __syncthreads();
    for (int64_t e = i; e < total; e += kThreads) {
        const int r = request_of(s_upto, n, e);
        const int64_t at = static_cast<int64_t>(s_row[r]) * a.max_pages + need + (e - (r ? s_upto[r - 1] : 0));
        const int page = a.table[at];
        a.table[at] = -1;
        if (page < 0 || page >= a.n_pages) continue;
        a.refs[page] = 0;
        if (have + e < a.n_pages) a.free[have + e] = page;
    }
    if (i == 0 && total > 0) *a.n_free = static_cast<int>(have + total < a.n_pages ? have + total : a.n_pages);
}

hipError_t launch_kv_evict(const PageArgs& a, const CacheArgs& c, const EvictArgs& e, const int32_t* rows, int n, int32_t* status) {
    if (n == 0) return hipSuccess;
    const hipStream_t st = static_cast<hipStream_t>(a.stream);
    hipLaunchKernelGGL(kv_evict_kernel, dim3(static_cast<unsigned>(n) * c.n_layers * e.Hkv), dim3(kNT), 0, st, a, c, e, rows, status);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    hipLaunchKernelGGL(kv_evict_pages_kernel, dim3(1), dim3(kThreads), 0, st, a, e.budget, rows, n, status);
    return hipGetLastError();
}

}  // namespace kda
