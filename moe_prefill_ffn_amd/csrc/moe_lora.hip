// HIP kernels (CDNA4 / gfx950) of the low-rank adapters of many requests beside a shared
// projection:
//   out[t] = base[t] + scale_i (x[t] A_i^T) B_i^T,  i = adapters[t] (none: out[t] = base[t]).
//
// Two launches: s = x A_i^T in fp32, K in parts; then the parts' sum times B_i^T onto base.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_dtype.h"
#include "moe_lora.h"
#include "moe_tile.h"

namespace moe {

namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));

// First operand: adapter rows, lane i = lane % 16 holds one; second: rows of x (or of s).  Lane
// group g = lane / 16 takes 8 values of the summed dimension and gets four consecutive results of
// row i of the second operand.
template <int kIn>
__device__ __forceinline__ v4f mfma16x16(v4i w, v4i x, v4f c)
{
    if constexpr (kIn == kBF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, w), __builtin_bit_cast(v8bf, x), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, w), __builtin_bit_cast(v8h, x), c, 0, 0, 0);
}

constexpr int kLoraWaves = 4, kLoraThreads = 64 * kLoraWaves;

// The adapter of row (lane & 31) of the tile of `rows` rows at m0, -1: none, or no such row.
__device__ __forceinline__ int adapter_of(const LoraAdd& l, int64_t m0, int rows)
{
    const int row = threadIdx.x & 31;
    const int id = row < rows && m0 + row < l.M ? l.adapters[m0 + row] : -1;
    return (uint32_t)id < (uint32_t)l.n ? id : -1;
}

// Calls f(adapter) for the tile's distinct adapters number way, way + ways, ... in the order in
// which rows first name them; uniform over the wave.
template <class F>
__device__ __forceinline__ void each_adapter(int id, int way, int ways, F f)
{
    uint32_t left = (uint32_t)__ballot(id >= 0);
    for (int at = 0; left; ++at) {
        const int cur = __builtin_amdgcn_readlane(id, __builtin_ctz(left));
        left &= ~(uint32_t)__ballot(id == cur);
        if (at % ways == way) f(cur);
    }
}

// --------------------------------------------------------------- s = x A^T ---
// A workgroup: 16 kR rows, one part of K shared out to its waves 64 values at a time, up to 16 kRT
// ranks.  Rows of another adapter are computed along and not stored.  A wave's next loads are out
// while it multiplies.
template <int kIn, int kRT, int kR>
__global__ __launch_bounds__(kLoraThreads) void k_lora_down(LoraAdd l, int parts)
{
    __shared__ float red[kLoraWaves][16 * kR][16 * kRT + 4];
    const int tid = threadIdx.x, lane = tid & 63, i = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t m0 = (int64_t)blockIdx.x * (16 * kR);
    const int part = (int)blockIdx.y % parts, r0 = (int)blockIdx.y / parts * 16 * kRT;
    const int chunks = l.K / 8, per = ((chunks + parts - 1) / parts + 7) / 8 * 8;    // 16-byte chunks a part
    const int c0 = part * per + wave * 8, c1 = (part + 1) * per < chunks ? (part + 1) * per : chunks;
    constexpr int kStep = 8 * kLoraWaves;
    const int id = adapter_of(l, m0, 16 * kR);
    const uint8_t* x[kR];
#pragma unroll
    for (int q = 0; q < kR; ++q) x[q] = l.x + (m0 + 16 * q + i < l.M ? m0 + 16 * q + i : l.M - 1) * l.x_stride + 32 * g;
    struct Frag {
        v4i x[2][kR], a[2][kRT];
    };
    each_adapter(id, blockIdx.z, gridDim.z, [&](int cur) {
        const uint8_t* a[kRT];
        v4f acc[kR][kRT];
#pragma unroll
        for (int t = 0; t < kRT; ++t) {
            const int q = r0 + 16 * t + i < l.r ? r0 + 16 * t + i : l.r - 1;
            a[t] = l.a + ((int64_t)cur * l.r + q) * l.K * 2 + 32 * g;
#pragma unroll
            for (int q2 = 0; q2 < kR; ++q2) acc[q2][t] = v4f{0, 0, 0, 0};
        }
        // lane group g: chunks u + 2 g, + 1; past the part's end 0
        auto load = [&](Frag& f, int u) {
            const bool whole = u + 8 <= c1;               // uniform
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const bool in = whole || u + 2 * g + s < c1;
                const int64_t at = (int64_t)(u + s) * 16;
#pragma unroll
                for (int q = 0; q < kR; ++q) f.x[s][q] = in ? *reinterpret_cast<const v4i*>(x[q] + at) : v4i{0, 0, 0, 0};
#pragma unroll
                for (int t = 0; t < kRT; ++t) f.a[s][t] = in ? *reinterpret_cast<const v4i*>(a[t] + at) : v4i{0, 0, 0, 0};
            }
        };
        auto multiply = [&](const Frag& f) {
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int t = 0; t < kRT; ++t)
#pragma unroll
                    for (int q = 0; q < kR; ++q) acc[q][t] = mfma16x16<kIn>(f.a[s][t], f.x[s][q], acc[q][t]);
        };
        Frag f0, f1;
        if (c0 < c1) load(f0, c0);
        for (int u = c0; u < c1; u += 2 * kStep) {
            if (u + kStep < c1) load(f1, u + kStep);
            multiply(f0);
            if (u + kStep >= c1) break;
            if (u + 2 * kStep < c1) load(f0, u + 2 * kStep);
            multiply(f1);
        }
        __syncthreads();                                  // the last adapter's sums are read
#pragma unroll
        for (int q = 0; q < kR; ++q)
#pragma unroll
            for (int t = 0; t < kRT; ++t) *reinterpret_cast<v4f*>(&red[wave][16 * q + i][16 * t + 4 * g]) = acc[q][t];
        __syncthreads();
        for (int e = tid; e < 256 * kR * kRT; e += kLoraThreads) {
            const int row = e / (16 * kRT), q = e % (16 * kRT);
            if (__shfl(id, row) != cur || r0 + q >= l.r) continue;
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < kLoraWaves; ++w) s += red[w][row][q];
            l.ws[((int64_t)part * l.M + m0 + row) * l.r + r0 + q] = s;
        }
    });
}

// ------------------------------------------------------- out = base + s B^T ---
// s enters the matrix instruction as a sum of 16-bit parts, so that little of its 24 bits is lost: bf16
// two parts, each the nearest to what the parts before it left (2^-16 of s lost at most), for fp32
// results three (2^-24).  fp16: the row of s times the power of two that brings its largest value to
// [2^14, 2^15), as two parts: 2^-22 of a value lost, or 2^-39 of the row's largest.
template <int kIn, int kP, int kKS>
struct Parts {
    v4i v[kKS][kP];
    float back;               // what the results are multiplied by
};

template <int kIn, int kP, int kKS>
__device__ __forceinline__ Parts<kIn, kP, kKS> split(const float (&s)[kKS][8])
{
    Parts<kIn, kP, kKS> p;
    float to = 1.0f;
    p.back = 1.0f;
    if constexpr (kIn == kF16) {
        float most = 0.0f;
#pragma unroll
        for (int k = 0; k < kKS; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float v = __builtin_fabsf(s[k][e]);
                most = v > most && v < __builtin_inff() ? v : most;
            }
#pragma unroll
        for (int o = 16; o < 64; o <<= 1) {               // the row's other lane groups
            const float v = __shfl_xor(most, o);
            most = v > most ? v : most;
        }
        int e = (int)(__float_as_uint(most) >> 23) - 127; // floor(log2 most)
        e = e < -100 ? -100 : e;
        to = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
        p.back = __uint_as_float((uint32_t)(127 - 14 + e) << 23);
    }
#pragma unroll
    for (int k = 0; k < kKS; ++k) {
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            float rest[2] = {s[k][e] * to, s[k][e + 1] * to};
#pragma unroll
            for (int q = 0; q < kP; ++q) {
                uint32_t w;
                float at[2];
                if constexpr (kIn == kBF16) {
                    uint32_t b[2];
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        b[z] = (uint32_t)__builtin_bit_cast(uint16_t, from_f32<kBF16>(rest[z]));
                        // a number that would round up to infinity: the largest one
                        if ((b[z] & 0x7fffu) == 0x7f80u && __builtin_fabsf(rest[z]) < __builtin_inff()) --b[z];
                        at[z] = __uint_as_float(b[z] << 16);
                    }
                    w = b[0] | b[1] << 16;
                } else {
                    typedef _Float16 v2h __attribute__((ext_vector_type(2)));
                    const v2h h = {(_Float16)rest[0], (_Float16)rest[1]};
                    at[0] = (float)h[0];
                    at[1] = (float)h[1];
                    w = __builtin_bit_cast(uint32_t, h);
                }
                p.v[k][q][e / 2] = (int)w;
#pragma unroll
                for (int z = 0; z < 2; ++z)               // an infinity or a NaN is in the first part alone
                    rest[z] = __builtin_fabsf(at[z]) < __builtin_inff() ? rest[z] - at[z] : 0.0f;
            }
        }
    }
    return p;
}

// Eight consecutive columns of a row, from and to memory: `wide` where they lie in aligned 16-byte
// vectors, else the n there are one by one.
__device__ __forceinline__ void load_row8(const void* p, int64_t at, int type, bool wide, int n, float (&v)[8])
{
    if (wide) {
        if (type == kF32) {
            float lo[4], hi[4];
            load_n<kF32, 4>(static_cast<const float*>(p) + at, lo);
            load_n<kF32, 4>(static_cast<const float*>(p) + at + 4, hi);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = lo[e], v[4 + e] = hi[e];
        } else if (type == kBF16) {
            load_n<kBF16, 8>(static_cast<const __bf16*>(p) + at, v);
        } else {
            load_n<kF16, 8>(static_cast<const _Float16*>(p) + at, v);
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        v[e] = 0.0f;
        if (e >= n) continue;
        v[e] = type == kF32 ? static_cast<const float*>(p)[at + e] : type == kBF16 ? (float)static_cast<const __bf16*>(p)[at + e]
                                                                                   : (float)static_cast<const _Float16*>(p)[at + e];
    }
}
__device__ __forceinline__ void store_row8(void* p, int64_t at, int type, bool wide, int n, const float (&v)[8])
{
    if (wide) {
        if (type == kF32) {
            const float lo[4] = {v[0], v[1], v[2], v[3]}, hi[4] = {v[4], v[5], v[6], v[7]};
            store_n<kF32, 4>(static_cast<float*>(p) + at, lo);
            store_n<kF32, 4>(static_cast<float*>(p) + at + 4, hi);
        } else if (type == kBF16) {
            store_n<kBF16, 8>(static_cast<__bf16*>(p) + at, v);
        } else {
            store_n<kF16, 8>(static_cast<_Float16*>(p) + at, v);
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        if (e >= n) continue;
        if (type == kF32)
            static_cast<float*>(p)[at + e] = v[e];
        else if (type == kBF16)
            static_cast<__bf16*>(p)[at + e] = (__bf16)v[e];
        else
            static_cast<_Float16*>(p)[at + e] = (_Float16)v[e];
    }
}

// A workgroup: 16 kR rows by cols columns (a multiple of 256), its waves 64 columns at a time as two
// pairs of products of 16 columns.  Product t of a pair has columns 8 (i / 4) + 4 t + i % 4 of its 32, so that
// lane group g gets 8 consecutive ones, 8 g on, of its row from the two.
template <int kIn, int kP, int kKS, int kR>
__global__ __launch_bounds__(kLoraThreads) void k_lora_up(LoraAdd l, int parts, int cols, int wide)
{
    const int tid = threadIdx.x, lane = tid & 63, i = lane & 15, g = lane >> 4, wave = tid >> 6;
    const int64_t m0 = (int64_t)blockIdx.x * (16 * kR);
    const int first = (int)blockIdx.y * cols + wave * 64, end = ((int)blockIdx.y + 1) * cols < l.N ? ((int)blockIdx.y + 1) * cols : l.N;
    const int id = adapter_of(l, m0, 16 * kR);
    int ids[kR];
#pragma unroll
    for (int q = 0; q < kR; ++q) ids[q] = __shfl(id, 16 * q + i);
    // eight columns from n on of this lane's row of row tile q
    auto finish = [&](int q, int n, float factor, float scale, const float (&z)[8]) {
        const int64_t m = m0 + 16 * q + i;
        if (n >= l.N) return;
        float v[8] = {};
        if (l.base) load_row8(l.base, m * l.base_stride + n, l.base_type, wide, l.N - n, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += z[e] * factor * scale;
        store_row8(l.out, m * l.out_stride + n, l.out_type, wide, l.N - n, v);
    };
    each_adapter(id, blockIdx.z, gridDim.z, [&](int cur) {
        Parts<kIn, kP, kKS> p[kR];
#pragma unroll
        for (int q = 0; q < kR; ++q) {
            float s[kKS][8];
#pragma unroll
            for (int k = 0; k < kKS; ++k) {
#pragma unroll
                for (int e = 0; e < 8; ++e) s[k][e] = 0.0f;
                const int at = 32 * k + 8 * g;
                if (ids[q] == cur && at < l.r) {
                    const float* w = l.ws + (m0 + 16 * q + i) * l.r + at;
                    for (int part = 0; part < parts; ++part, w += l.M * l.r) {
                        const v4f lo = *reinterpret_cast<const v4f*>(w), hi = *reinterpret_cast<const v4f*>(w + 4);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            s[k][e] += lo[e];
                            s[k][4 + e] += hi[e];
                        }
                    }
                }
            }
            p[q] = split<kIn, kP, kKS>(s);
        }
        const float scale = l.scales ? l.scales[cur] : 1.0f;
        for (int n0 = first; n0 < end; n0 += 64 * kLoraWaves) {
#pragma unroll
            for (int pair = 0; pair < 2; ++pair) {
                v4f acc[kR][2];
#pragma unroll
                for (int t = 0; t < 2; ++t) {
#pragma unroll
                    for (int q = 0; q < kR; ++q) acc[q][t] = v4f{0, 0, 0, 0};
                    const int col = n0 + 32 * pair + 8 * (i >> 2) + 4 * t + (i & 3), n = col < l.N ? col : l.N - 1;
                    const uint8_t* b = l.b + ((int64_t)cur * l.N + n) * l.r * 2;
#pragma unroll
                    for (int k = 0; k < kKS; ++k) {
                        const int at = 32 * k + 8 * g;
                        const v4i w = at < l.r ? *reinterpret_cast<const v4i*>(b + at * 2) : v4i{0, 0, 0, 0};
#pragma unroll
                        for (int z = kP - 1; z >= 0; --z)
#pragma unroll
                            for (int q = 0; q < kR; ++q) acc[q][t] = mfma16x16<kIn>(w, p[q].v[k][z], acc[q][t]);
                    }
                }
#pragma unroll
                for (int q = 0; q < kR; ++q) {
                    if (ids[q] != cur) continue;
                    const float z[8] = {acc[q][0][0], acc[q][0][1], acc[q][0][2], acc[q][0][3], acc[q][1][0], acc[q][1][1], acc[q][1][2], acc[q][1][3]};
                    finish(q, n0 + 32 * pair + 8 * g, p[q].back, scale, z);
                }
            }
        }
    });
    if (blockIdx.z != 0 || l.out == l.base) return;       // in place: rows of no adapter stay as they are
    const float none[8] = {};
    for (int n0 = first; n0 < end; n0 += 64 * kLoraWaves)
#pragma unroll
        for (int pair = 0; pair < 2; ++pair)
#pragma unroll
            for (int q = 0; q < kR; ++q)
                if (ids[q] < 0 && m0 + 16 * q + i < l.M) finish(q, n0 + 32 * pair + 8 * g, 0.0f, 0.0f, none);
}

template <int kIn, int kP, int kKS>
void launch_up_tile(const LoraAdd& l, int parts, int ways, hipStream_t st)
{
    // whole vectors of 8 columns at aligned addresses
    auto even = [&](const void* p, int64_t stride, int type) {
        return (reinterpret_cast<uintptr_t>(p) | (uint64_t)(stride * dtype_bytes(type))) % 16 == 0;
    };
    const int wide = l.N % 8 == 0 && even(l.out, l.out_stride, l.out_type) && (!l.base || even(l.base, l.base_stride, l.base_type));
    // a wave splits s into its parts once for its columns: as many columns as leave the chip full
    const unsigned tiles = nblk(l.M, lora_tile(l.M));
    const int64_t blocks = nblk(l.N, 64 * kLoraWaves), want = (1024 + tiles - 1) / tiles;
    const int cols = (int)((blocks + want - 1) / want) * 64 * kLoraWaves;
    const dim3 grid(tiles, nblk(l.N, cols), ways);
    if (lora_tile(l.M) == 32)
        hipLaunchKernelGGL((k_lora_up<kIn, kP, kKS, 2>), grid, dim3(kLoraThreads), 0, st, l, parts, cols, wide);
    else
        hipLaunchKernelGGL((k_lora_up<kIn, kP, kKS, 1>), grid, dim3(kLoraThreads), 0, st, l, parts, cols, wide);
}

template <int kIn, int kP>
void launch_up(const LoraAdd& l, int parts, int ways, hipStream_t st)
{
    if (l.r <= 32)
        launch_up_tile<kIn, kP, 1>(l, parts, ways, st);
    else if (l.r <= 64)
        launch_up_tile<kIn, kP, 2>(l, parts, ways, st);
    else if (l.r <= 128)
        launch_up_tile<kIn, kP, 4>(l, parts, ways, st);
    else
        launch_up_tile<kIn, kP, 8>(l, parts, ways, st);
}

template <int kIn, int kRT>
void launch_down(const LoraAdd& l, int parts, int ways, hipStream_t st)
{
    const dim3 grid(nblk(l.M, lora_tile(l.M)), parts * nblk(l.r, 16 * kRT), ways);
    if (lora_tile(l.M) == 32)
        hipLaunchKernelGGL((k_lora_down<kIn, kRT, 2>), grid, dim3(kLoraThreads), 0, st, l, parts);
    else
        hipLaunchKernelGGL((k_lora_down<kIn, kRT, 1>), grid, dim3(kLoraThreads), 0, st, l, parts);
}

template <int kIn>
void launch_typed(const LoraAdd& l, hipStream_t st)
{
    const int parts = lora_parts(l.M, l.K);
    // rows of a small batch mostly have an adapter each: its tiles' adapters go to workgroups of their own
    const int ways = l.M <= 512 ? (l.M < 16 ? (int)l.M : 16) : 1;
    if (l.r <= 16)
        launch_down<kIn, 1>(l, parts, ways, st);
    else if (l.r <= 32)
        launch_down<kIn, 2>(l, parts, ways, st);
    else
        launch_down<kIn, 4>(l, parts, ways, st);
    if constexpr (kIn == kBF16) {
        if (l.out_type == kF32) return launch_up<kIn, 3>(l, parts, ways, st);
    }
    launch_up<kIn, 2>(l, parts, ways, st);
}

}  // namespace

// ----------------------------------------------------------------- launches ---
hipError_t launch_lora_add(const LoraAdd& l, hipStream_t st)
{
    if (l.M == 0) return hipSuccess;
    if (l.in_type == kBF16)
        launch_typed<kBF16>(l, st);
    else
        launch_typed<kF16>(l, st);
    return hipGetLastError();
}

}  // namespace moe
