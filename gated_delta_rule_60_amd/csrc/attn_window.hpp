// attn_window.hpp -- which keys a row of windowed attention sees, by row, by
// tile and by block of rows; shared by the forward and the backward kernels
// (the look-up of a piece also by attn_weights.hip).
#pragma once

#include "attn_device.hpp"
#include "attn_launch.hpp"

namespace kda {

__device__ __forceinline__ bool window_sees(const WindowArgs& w, int row, int key) {
    return key <= row && (row - key < w.window || key < w.sinks);
}

// Piece number p of the batch, in the sequences' order, as find_tile past 64 sequences: behind the first
// window's rows all pieces have the same work, and one round of sums is all it takes.
__device__ __forceinline__ bool find_window_tile(const int32_t* cu, int N, int T_tot, int BM, int p, SeqTile& s) {
    const int lane = threadIdx.x & 63;
    for (int n0 = 0; n0 < N; n0 += 64) {
        int2 bl = make_int2(0, 0);
        if (n0 + lane < N) bl = seq_bounds(cu, n0 + lane, T_tot);
        const int nt = (bl.y + BM - 1) / BM;
        const int incl = wave_scan(nt);
        const int total = __builtin_amdgcn_readlane(incl, 63);
        if (p < total) {
            const int n = __builtin_ctzll(__ballot(incl > p));
            s.beg = __builtin_amdgcn_readlane(bl.x, n);
            s.len = __builtin_amdgcn_readlane(bl.y, n);
            s.tile = p - (__builtin_amdgcn_readlane(incl, n) - __builtin_amdgcn_readlane(nt, n));
            s.n = n0 + n;
            return true;
        }
        p -= total;
    }
    return false;
}

// The tiles of BN keys that a block of rows [row0, end) walks: those of the
// sinks that lie before the first row's window, then from that window to the
// diagonal.
template <int BN>
struct WindowTiles {
    int head;   // tiles of the sinks before the window's
    int skip;   // tiles between them and the window's
    int count;
    __device__ __forceinline__ WindowTiles(const WindowArgs& w, int row0, int end) {
        const int lo = row0 - w.window + 1;
        const int first = lo > 0 ? lo / BN : 0;
        const int sinks = (w.sinks + BN - 1) / BN;
        head = sinks < first ? sinks : first;
        skip = first - head;
        count = (end + BN - 1) / BN - skip;
    }
    // tile number u of the list, and the number of a tile at or past the window's first
    __device__ __forceinline__ int tile(int u) const { return u < head ? u : u + skip; }
    __device__ __forceinline__ int number(int t) const { return t - skip; }
};

// Rows [row0, row0 + n) against tiles of BN keys at or before their diagonal.
template <int BN>
struct WindowRows {
    int lo;     // the first row's first key in its window
    int all_lo; // the last row's
    int row0, sinks;
    __device__ __forceinline__ WindowRows(const WindowArgs& w, int row0_, int n)
        : lo(row0_ - w.window + 1), all_lo(row0_ + n - w.window), row0(row0_), sinks(w.sinks) {}
    // some row may see some key of tile t (which begins at or before the last row)
    __device__ __forceinline__ bool sees(int t) const { return (t + 1) * BN > lo || t * BN < sinks; }
    // every row sees every key of it
    __device__ __forceinline__ bool sees_all(int t) const {
        return (t + 1) * BN - 1 <= row0 && (t * BN >= all_lo || (t + 1) * BN <= sinks);
    }
};

}  // namespace kda
