// HIP kernels (CDNA4 / gfx950) around the products of a row table: the table itself from
// the experts that any router chose, and the weighted sum of the experts' rows per token.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_dtype.h"
#include "moe_rows.h"
#include "moe_tile.h"

namespace moe {

namespace {

// -------------------------------------------------------------------- group ---
// A stable counting sort: pair p of group e goes to row
//   bounds[e] + (pairs of e before p),
// the pairs before p being those of earlier workgroups, of earlier waves of its workgroup
// (each wave takes a run of the workgroup's pairs), and before it in its wave.  No order of
// execution enters: the same table on every run.
constexpr int kGroupThreads = 1024, kGroupWaves = kGroupThreads / 64;

// LDS: counters [waves][E], the groups' first rows [E], one sum a wave
constexpr int kGroupLds = (kGroupWaves * kGroupMostGroups + kGroupMostGroups + kGroupWaves) * 4;

// Pairs of each group among this workgroup's: one workgroup of the launch's share of the table.
__global__ __launch_bounds__(kGroupThreads) void k_group_count(GroupRows g, int64_t chunk)
{
    extern __shared__ int s_count[];
    const int64_t p0 = blockIdx.x * chunk, p1 = p0 + chunk < g.pairs ? p0 + chunk : g.pairs;
    for (int e = threadIdx.x; e < g.E; e += kGroupThreads) s_count[e] = 0;
    __syncthreads();
    for (int64_t p = p0 + threadIdx.x; p < p1; p += kGroupThreads) {
        const uint32_t e = (uint32_t)g.eidx[p];
        if (e < (uint32_t)g.E) atomicAdd(&s_count[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < g.E; e += kGroupThreads) g.ws[(int64_t)blockIdx.x * g.E + e] = s_count[e];
}

// What bounds it is latency: the counts' loads, the waves' prefixes and the scan over the groups
// follow each other.  65536 pairs in 256 groups 7.9 us and the count's 2.6 (18.6 where each thread summed its group's
// counts one workgroup after the other); 192 pairs, one workgroup, 3.5.
__global__ __launch_bounds__(kGroupThreads) void k_group_place(GroupRows g, int64_t chunk)
{
    extern __shared__ int lds[];
    __shared__ int s_sum[2][kGroupThreads];
    const int E = g.E, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int* s_count = lds;                                   // [waves][E]: pairs of the wave, then its next row
    int* s_first = lds + kGroupWaves * E;                 // [E]: pairs of earlier workgroups
    int* s_wave = s_first + E;
    // the other workgroups' counts: `parts` threads a group, each every so-many-th workgroup, eight loads out
    int ep = 64;
    while (ep < E) ep *= 2;
    const int parts = kGroupThreads / ep;
    if (gridDim.x > 1) {
        const int e = tid & (ep - 1), blocks = (int)gridDim.x;
        int all = 0, before = 0;
        for (int b0 = tid / ep; b0 < blocks; b0 += 8 * parts) {
            int n[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) n[i] = e < E && b0 + i * parts < blocks ? g.ws[(int64_t)(b0 + i * parts) * E + e] : 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                all += n[i];
                before += b0 + i * parts < (int)blockIdx.x ? n[i] : 0;
            }
        }
        s_sum[0][tid] = all;
        s_sum[1][tid] = before;
    }
    const int64_t p0 = blockIdx.x * chunk, p1 = p0 + chunk < g.pairs ? p0 + chunk : g.pairs;
    const int64_t share = ((p1 - p0 + kGroupWaves - 1) / kGroupWaves + 63) / 64 * 64;
    const int64_t w0 = p0 + wave * share < p1 ? p0 + wave * share : p1, w1 = w0 + share < p1 ? w0 + share : p1;
    for (int i = tid; i < kGroupWaves * E; i += kGroupThreads) s_count[i] = 0;
    __syncthreads();
    for (int64_t p = w0 + lane; p < w1; p += 64) {
        const uint32_t e = (uint32_t)g.eidx[p];
        if (e < (uint32_t)E) atomicAdd(&s_count[wave * E + e], 1);
    }
    __syncthreads();
    // thread e: the group's pairs in all, and before this workgroup's (E <= 1024 threads)
    int all = 0, before = 0;
    if (gridDim.x > 1) {
        for (int q = 0; tid < E && q < parts; ++q) {      // tid + q ep < 1024
            all += s_sum[0][tid + q * ep];
            before += s_sum[1][tid + q * ep];
        }
    } else if (tid < E) {
#pragma unroll
        for (int w = 0; w < kGroupWaves; ++w) all += s_count[w * E + tid];
    }
    int upto = all;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int y = __shfl_up(upto, o);
        if (lane >= o) upto += y;
    }
    if (lane == 63) s_wave[wave] = upto;
    __syncthreads();
    int first = upto - all;
    for (int w = 0; w < wave; ++w) first += s_wave[w];
    if (tid < E) {
        if (blockIdx.x == 0) {
            if (g.counts) g.counts[tid] = all;
            g.bounds[tid] = first;
            if (tid == E - 1) g.bounds[E] = first + all;
        }
        int at = first + before, n[kGroupWaves];
#pragma unroll
        for (int w = 0; w < kGroupWaves; ++w) n[w] = s_count[w * E + tid];
#pragma unroll
        for (int w = 0; w < kGroupWaves; ++w) {
            s_count[w * E + tid] = at;
            at += n[w];
        }
    }
    __syncthreads();
    int* next = s_count + wave * E;
    const int bits = 32 - __clz(E);                       // E itself stands for no group
    for (int64_t p = w0 + lane; p - lane < w1; p += 64) {
        const uint32_t raw = p < w1 ? (uint32_t)g.eidx[p] : ~0u;
        const int e = raw < (uint32_t)E ? (int)raw : E;
        uint64_t same = ~0ull;                            // lanes of the same group
        for (int i = 0; i < bits; ++i) {
            const uint64_t m = __ballot((e >> i) & 1);
            same &= ((e >> i) & 1) ? m : ~m;
        }
        const uint64_t below = same & ((1ull << lane) - 1);
        const int row = e < E ? next[e] + __popcll(below) : -1;
        __builtin_amdgcn_wave_barrier();                  // every lane has read its counter
        if (e < E && (same >> lane) == 1) next[e] = row + 1;   // the last lane of the group
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (p < w1) {
            if (g.pos) g.pos[p] = row;
            if (g.rows && row >= 0) g.rows[row] = (int)p;
        }
    }
}

// ------------------------------------------------------------------ combine ---
// One pass over the experts' rows, summed in slot order in fp32, rounded once: memory bounds it, 8192 tokens of 8
// rows of 4096 bf16 values beside a base (671 MB) 129 us, 5.2 TB/s.
// A thread takes kV consecutive columns of one token (16 bytes of d), its k rows kSlots at a time so
// that their loads are all out together.
constexpr int kCombineThreads = 256, kSlots = 8;

template <int n>
__device__ __forceinline__ void load_any(const void* p, int64_t at, int type, float (&v)[n])
{
    if (type == kF32) {
#pragma unroll
        for (int i = 0; i < n; i += 4) {
            if constexpr (n >= 4) {
                float t[4];
                load_n<kF32, 4>(static_cast<const float*>(p) + at + i, t);
#pragma unroll
                for (int q = 0; q < 4; ++q) v[i + q] = t[q];
            } else {
                v[i] = static_cast<const float*>(p)[at + i];
            }
        }
    } else if (type == kBF16) {
        load_n<kBF16, n>(static_cast<const __bf16*>(p) + at, v);
    } else {
        load_n<kF16, n>(static_cast<const _Float16*>(p) + at, v);
    }
}

template <int n>
__device__ __forceinline__ void store_any(void* p, int64_t at, int type, const float (&v)[n])
{
    if (type == kF32) {
#pragma unroll
        for (int i = 0; i < n; i += 4) {
            if constexpr (n >= 4) {
                const float t[4] = {v[i], v[i + 1], v[i + 2], v[i + 3]};
                store_n<kF32, 4>(static_cast<float*>(p) + at + i, t);
            } else {
                static_cast<float*>(p)[at + i] = v[i];
            }
        }
    } else if (type == kBF16) {
        store_n<kBF16, n>(static_cast<__bf16*>(p) + at, v);
    } else {
        store_n<kF16, n>(static_cast<_Float16*>(p) + at, v);
    }
}

// cols: threads of a workgroup along a row (a power of two), the rest are tokens.
template <int kT, int kV>
__global__ __launch_bounds__(kCombineThreads) void k_combine_rows(CombineRows c, int cols)
{
    typedef typename Elem<kT>::type T;
    typedef T Tv __attribute__((ext_vector_type(kV)));
    const int64_t t = (int64_t)blockIdx.x * (kCombineThreads / cols) + threadIdx.x / cols;
    const int64_t n0 = ((int64_t)blockIdx.y * cols + (threadIdx.x & (cols - 1))) * kV;
    if (t >= c.T || n0 >= c.n) return;
    float acc[kV];
#pragma unroll
    for (int i = 0; i < kV; ++i) acc[i] = 0.0f;
    if (c.base) load_any<kV>(c.base, t * c.base_stride + n0, c.base_type, acc);
    const T* d = static_cast<const T*>(c.d) + n0;
    for (int j0 = 0; j0 < c.k; j0 += kSlots) {
        int row[kSlots];
        float w[kSlots];
        Tv v[kSlots];
#pragma unroll
        for (int j = 0; j < kSlots; ++j) {
            const bool in = j0 + j < c.k;
            row[j] = in ? c.pos[t * c.k + j0 + j] : -1;
            w[j] = in ? c.weights[t * c.k + j0 + j] : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < kSlots; ++j)
            if (row[j] >= 0 && row[j] < c.d_rows) v[j] = *reinterpret_cast<const Tv*>(d + row[j] * c.d_stride);
#pragma unroll
        for (int j = 0; j < kSlots; ++j)
            if (row[j] >= 0 && row[j] < c.d_rows) {
#pragma unroll
                for (int i = 0; i < kV; ++i) acc[i] = __builtin_fmaf(w[j], (float)v[j][i], acc[i]);
            }
    }
    store_any<kV>(c.y, t * c.y_stride + n0, c.y_type, acc);
}

template <int kT>
void launch_combine(const CombineRows& c, hipStream_t st)
{
    constexpr int kV = kT == kF32 ? 4 : 8;
    // whole vectors at aligned addresses in every operand
    auto even = [&](const void* p, int64_t stride, int type) {
        const int64_t size = kV * dtype_bytes(type) < 16 ? kV * dtype_bytes(type) : 16;
        return reinterpret_cast<uintptr_t>(p) % size == 0 && stride * dtype_bytes(type) % size == 0;
    };
    const bool wide = c.n % kV == 0 && even(c.d, c.d_stride, kT) && even(c.y, c.y_stride, c.y_type) &&
                      (!c.base || even(c.base, c.base_stride, c.base_type));
    const int per = wide ? c.n / kV : c.n;                // threads a row needs
    int cols = 64;
    while (cols < kCombineThreads && cols < per) cols *= 2;
    const dim3 grid(nblk(c.T, kCombineThreads / cols), nblk(per, cols));
    if (wide)
        hipLaunchKernelGGL((k_combine_rows<kT, kV>), grid, dim3(kCombineThreads), 0, st, c, cols);
    else
        hipLaunchKernelGGL((k_combine_rows<kT, 1>), grid, dim3(kCombineThreads), 0, st, c, cols);
}

}  // namespace

// ----------------------------------------------------------------- launches ---
hipError_t launch_group_rows(const GroupRows& g, hipStream_t st)
{
    const int64_t chunk = group_chunk(g.pairs);
    const int blocks = g.pairs ? group_blocks(g.pairs) : 1;
    const int lds = (kGroupWaves * g.E + g.E + kGroupWaves) * 4;
    // more than the default limit of dynamic LDS
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&k_group_place), hipFuncAttributeMaxDynamicSharedMemorySize, kGroupLds);
    if (e != hipSuccess) return e;
    if (blocks > 1) hipLaunchKernelGGL(k_group_count, dim3(blocks), dim3(kGroupThreads), g.E * 4, st, g, chunk);
    hipLaunchKernelGGL(k_group_place, dim3(blocks), dim3(kGroupThreads), lds, st, g, chunk);
    return hipGetLastError();
}

hipError_t launch_combine_rows(const CombineRows& c, hipStream_t st)
{
    if (c.T == 0) return hipSuccess;
    if (c.d_type == kF32)
        launch_combine<kF32>(c, st);
    else if (c.d_type == kBF16)
        launch_combine<kBF16>(c, st);
    else
        launch_combine<kF16>(c, st);
    return hipGetLastError();
}

}  // namespace moe
