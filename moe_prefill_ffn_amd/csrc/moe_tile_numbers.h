// Which tiles of a product over a row table a persistent workgroup takes.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_tile.h"

namespace moe {

namespace {

// This workgroup's tiles: first, first + step, ... below end.  Each XCD has a run of as many tiles as
// the others, each of its workgroups as many of them.
struct TileRun {
    int64_t first, end;
    int step;
};
__device__ __forceinline__ TileRun tile_run(int64_t slots, int n_tiles)
{
    const int64_t total = slots * n_tiles, per = (total + 7) >> 3;
    const int64_t run0 = (int64_t)(blockIdx.x & 7) * per, run1 = run0 + per < total ? run0 + per : total;
    return {run0 + (blockIdx.x >> 3), run1, (int)(gridDim.x >> 3)};
}

// The tiles of BM rows that hold any, in the groups' order (args: bounds or null, M, G; n_slots: the
// most there can be).  Every wave of the workgroup takes part in each call.
template <int NW, int BM>
struct TileNumbers {
    static constexpr int kPer = 4, kWin = 64 * NW * kPer, kBytes = (kWin + NW) * 4;
    uint32_t* s_pre;          // LDS: how many tiles of a window lie before each of its groups'
    uint32_t* s_wave;
    int64_t slots;            // tiles in all
    uint32_t first_window;

    template <class Args>
    __device__ __forceinline__ TileNumbers(const Args& a, uint32_t* lds, int64_t n_slots) : s_pre(lds), s_wave(lds + kWin), slots(n_slots), first_window(0)
    {
        if (!a.bounds) return;
        int64_t n = 0;
        for (int base = 0; base < a.G; base += kWin) n += first_window = scan(a, base);
        slots = n < n_slots ? n : n_slots;                // bounds that do not ascend
    }

    template <class Args>
    __device__ __forceinline__ static int bound(const Args& a, int g) { return bound_of(a, g < a.G ? g : a.G); }

    // the tiles of the kWin groups from base on
    template <class Args>
    __device__ __forceinline__ uint32_t scan(const Args& a, int base)
    {
        const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
        int b[kPer + 1];
        uint32_t n[kPer], sum = 0;
#pragma unroll
        for (int i = 0; i <= kPer; ++i) b[i] = bound(a, base + tid * kPer + i);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            n[i] = b[i + 1] > b[i] ? (uint32_t)(b[i + 1] - b[i] + BM - 1) / BM : 0u;
            sum += n[i];                                  // at most 2^22 a group, 2^32 - 1 a window of 1024
        }
        uint32_t upto = sum;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const uint32_t y = (uint32_t)__shfl_up((int)upto, o);
            if (lane >= o) upto += y;
        }
        __syncthreads();                                  // the last scan's, or list's, readers are done
        if (lane == 63) s_wave[wave] = upto;
        __syncthreads();
        uint32_t before = upto - sum, all = 0;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            before += w < wave ? s_wave[w] : 0u;
            all += s_wave[w];
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            s_pre[tid * kPer + i] = before;
            before += n[i];
        }
        __syncthreads();
        return (uint32_t)__builtin_amdgcn_readfirstlane((int)all);
    }

    // Tile `in` of a group of `high` row tiles by n_tiles column tiles: bands of 8 row tiles, in a band one
    // column tile after the other.
    __device__ __forceinline__ static void place(uint32_t in, uint32_t high, int n_tiles, int* row, int* nt)
    {
        const uint32_t band = in / (uint32_t)(8 * n_tiles), first = band * 8, of = high - first < 8 ? high - first : 8;
        in -= first * n_tiles;
        *row = (int)(first + in % of);
        *nt = (int)(in / of);
    }

    // The run's tiles from number list0 on, into LDS: as many as there are, kListMost at most.  Tiles are
    // numbered group by group, so that what an XCD runs at once shares rows of A and of B in its L2 and a
    // group's B is read at one time.  n_tiles * slots <= 2^30.
    template <class Args>
    __device__ __forceinline__ int list(const Args& a, ListedTile* s_list, int64_t list0, const TileRun& run, int n_tiles)
    {
        static_assert(kListMost <= 64 * NW, "a listed tile a thread");
        const int tid = threadIdx.x;
        const int64_t id = list0 + (int64_t)tid * run.step;
        const bool want = tid < kListMost && id < run.end;
        int row, nt;
        __syncthreads();                                  // the previous list is done
        if (!a.bounds) {
            if (want) {
                place((uint32_t)id, (uint32_t)slots, n_tiles, &row, &nt);
                const int64_t m0 = (int64_t)row * BM;
                s_list[tid] = {0, (int)m0, (int)(m0 + BM < a.M ? m0 + BM : a.M), nt};
            }
        }
        const int64_t at = want ? (uint32_t)id / (uint32_t)n_tiles : 0;    // row tiles before it, whole groups' among them
        int64_t before = 0;                               // row tiles before the window's
        for (int base = 0; a.bounds && base < a.G; base += kWin) {
            const bool have = a.G <= kWin && list0 == run.first;           // scanned already, uniform
            const uint32_t n = have ? first_window : scan(a, base);
            const int64_t x = at - before;
            if (want && x >= 0 && x < n) {
                int lo = 0, hi = kWin - 1;                // the last group with s_pre <= x
                while (lo < hi) {
                    const int mid = (lo + hi + 1) >> 1;
                    if (s_pre[mid] <= (uint32_t)x)
                        lo = mid;
                    else
                        hi = mid - 1;
                }
                const int g = base + lo, m0 = bound(a, g), end = bound(a, g + 1);
                place((uint32_t)(id - (before + s_pre[lo]) * n_tiles), (uint32_t)(end - m0 + BM - 1) / BM, n_tiles, &row, &nt);
                const int r0 = m0 + row * BM;
                s_list[tid] = {g, r0, r0 + BM < end ? r0 + BM : end, nt};
            }
            before += n;
        }
        __syncthreads();
        const int64_t left = (run.end - list0 + run.step - 1) / run.step;
        return left < kListMost ? (int)left : kListMost;
    }
};

}  // namespace

}  // namespace moe
