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

// The adapter of row (lane & 15) of the tile at m0, -1: none.
__device__ __forceinline__ int adapter_of(const LoraAdd& l, int64_t m0)
{
    const int64_t m = m0 + (threadIdx.x & 15);
    const int id = m < l.M ? l.adapters[m] : -1;
    return (uint32_t)id < (uint32_t)l.n ? id : -1;
}

// Calls f(adapter) for the tile's distinct adapters number way, way + ways, ... in the order in
// which rows first name them; uniform over the wave.
template <class F>
__device__ __forceinline__ void each_adapter(int id, int way, int ways, F f)
{
    uint32_t left = (uint32_t)__ballot(id >= 0) & 0xffffu;
    for (int at = 0; left; ++at) {
        const int cur = __builtin_amdgcn_readlane(id, __builtin_ctz(left));
        left &= ~((uint32_t)__ballot(id == cur) & 0xffffu);
        if (at % ways == way) f(cur);
    }
}

// --------------------------------------------------------------- s = x A^T ---
// A workgroup: 16 rows, one part of K shared out to its waves 64 values at a time, up to 16 kRT ranks.
// Rows of another adapter are computed along and not stored.
template <int kIn, int kRT>
__global__ __launch_bounds__(kLoraThreads) void k_lora_down(LoraAdd l, int parts)
{
    __shared__ float red[kLoraWaves][16][16 * kRT + 4];
    const int tid = threadIdx.x, lane = tid & 63, i = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t m0 = (int64_t)blockIdx.x * kLoraTile;
    const int part = (int)blockIdx.y % parts, r0 = (int)blockIdx.y / parts * 16 * kRT;
    const int chunks = l.K / 8, per = ((chunks + parts - 1) / parts + 7) / 8 * 8;    // 16-byte chunks a part
    const int c1 = (part + 1) * per < chunks ? (part + 1) * per : chunks;
    const int id = adapter_of(l, m0);
    const uint8_t* x = l.x + (m0 + i < l.M ? m0 + i : l.M - 1) * l.x_stride;
    each_adapter(id, blockIdx.z, gridDim.z, [&](int cur) {
        const uint8_t* a[kRT];
        v4f acc[kRT];
#pragma unroll
        for (int t = 0; t < kRT; ++t) {
            const int q = r0 + 16 * t + i < l.r ? r0 + 16 * t + i : l.r - 1;
            a[t] = l.a + ((int64_t)cur * l.r + q) * l.K * 2;
            acc[t] = v4f{0, 0, 0, 0};
        }
        for (int u = part * per + wave * 8; u < c1; u += 8 * kLoraWaves) {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int c = u + 2 * g + s;
                const bool in = c < c1;
                const v4i zero = {0, 0, 0, 0};
                const v4i vx = in ? *reinterpret_cast<const v4i*>(x + c * 16) : zero;
#pragma unroll
                for (int t = 0; t < kRT; ++t)
                    acc[t] = mfma16x16<kIn>(in ? *reinterpret_cast<const v4i*>(a[t] + c * 16) : zero, vx, acc[t]);
            }
        }
        __syncthreads();                                  // the last adapter's sums are read
#pragma unroll
        for (int t = 0; t < kRT; ++t)
            *reinterpret_cast<v4f*>(&red[wave][i][16 * t + 4 * g]) = acc[t];
        __syncthreads();
        for (int e = tid; e < 256 * kRT; e += kLoraThreads) {
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

__device__ __forceinline__ float load_one(const void* p, int64_t at, int type)
{
    return type == kF32 ? static_cast<const float*>(p)[at] : type == kBF16 ? (float)static_cast<const __bf16*>(p)[at]
                                                                           : (float)static_cast<const _Float16*>(p)[at];
}
__device__ __forceinline__ void store_one(void* p, int64_t at, int type, float v)
{
    if (type == kF32)
        static_cast<float*>(p)[at] = v;
    else if (type == kBF16)
        static_cast<__bf16*>(p)[at] = (__bf16)v;
    else
        static_cast<_Float16*>(p)[at] = (_Float16)v;
}

// A wave: 16 rows by 64 columns, in four products of 16 columns; lane group g gets columns
// 16 t + 4 g .. + 3 of its row from product t.
template <int kIn, int kP, int kKS>
__global__ __launch_bounds__(kLoraThreads) void k_lora_up(LoraAdd l, int parts)
{
    const int tid = threadIdx.x, lane = tid & 63, i = lane & 15, g = lane >> 4, wave = tid >> 6;
    const int64_t m0 = (int64_t)blockIdx.x * kLoraTile, m = m0 + i;
    const int n0 = ((int)blockIdx.y * kLoraWaves + wave) * 64;
    if (n0 >= l.N) return;
    const int id = adapter_of(l, m0);
    v4f res[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) res[t] = v4f{0, 0, 0, 0};
    bool mine = id < 0 && blockIdx.z == 0;                // this workgroup stores the lane's row
    each_adapter(id, blockIdx.z, gridDim.z, [&](int cur) {
        float s[kKS][8];
#pragma unroll
        for (int k = 0; k < kKS; ++k) {
#pragma unroll
            for (int e = 0; e < 8; ++e) s[k][e] = 0.0f;
            const int q = 32 * k + 8 * g;
            if (id == cur && q < l.r) {
                const float* p = l.ws + m * l.r + q;
                for (int part = 0; part < parts; ++part, p += l.M * l.r) {
                    const v4f lo = *reinterpret_cast<const v4f*>(p), hi = *reinterpret_cast<const v4f*>(p + 4);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        s[k][e] += lo[e];
                        s[k][4 + e] += hi[e];
                    }
                }
            }
        }
        const Parts<kIn, kP, kKS> p = split<kIn, kP, kKS>(s);
        const float scale = l.scales ? l.scales[cur] : 1.0f;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            v4f acc = {0, 0, 0, 0};
            const int n = n0 + 16 * t + i < l.N ? n0 + 16 * t + i : l.N - 1;
            const uint8_t* b = l.b + ((int64_t)cur * l.N + n) * l.r * 2;
#pragma unroll
            for (int k = 0; k < kKS; ++k) {
                const int q = 32 * k + 8 * g;
                const v4i w = q < l.r ? *reinterpret_cast<const v4i*>(b + q * 2) : v4i{0, 0, 0, 0};
#pragma unroll
                for (int z = kP - 1; z >= 0; --z) acc = mfma16x16<kIn>(w, p.v[k][z], acc);
            }
            if (id == cur) {
#pragma unroll
                for (int e = 0; e < 4; ++e) res[t][e] = acc[e] * p.back * scale;
            }
        }
        mine = mine || id == cur;
    });
    if (!mine || m >= l.M) return;
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int n = n0 + 16 * t + 4 * g + e;
            if (n >= l.N) continue;
            const float base = l.base ? load_one(l.base, m * l.base_stride + n, l.base_type) : 0.0f;
            store_one(l.out, m * l.out_stride + n, l.out_type, base + res[t][e]);
        }
}

template <int kIn, int kP>
void launch_up(const LoraAdd& l, int parts, dim3 grid, hipStream_t st)
{
    if (l.r <= 32)
        hipLaunchKernelGGL((k_lora_up<kIn, kP, 1>), grid, dim3(kLoraThreads), 0, st, l, parts);
    else if (l.r <= 64)
        hipLaunchKernelGGL((k_lora_up<kIn, kP, 2>), grid, dim3(kLoraThreads), 0, st, l, parts);
    else if (l.r <= 128)
        hipLaunchKernelGGL((k_lora_up<kIn, kP, 4>), grid, dim3(kLoraThreads), 0, st, l, parts);
    else
        hipLaunchKernelGGL((k_lora_up<kIn, kP, 8>), grid, dim3(kLoraThreads), 0, st, l, parts);
}

template <int kIn>
void launch_typed(const LoraAdd& l, hipStream_t st)
{
    const unsigned tiles = nblk(l.M, kLoraTile);
    const int parts = lora_parts(l.M, l.K);
    // rows of a small batch mostly have an adapter each: its tiles' adapters go to workgroups of their own
    const unsigned ways = l.M <= 512 ? (unsigned)(l.M < 16 ? l.M : 16) : 1;
    if (l.r <= 16)
        hipLaunchKernelGGL((k_lora_down<kIn, 1>), dim3(tiles, parts, ways), dim3(kLoraThreads), 0, st, l, parts);
    else if (l.r <= 32)
        hipLaunchKernelGGL((k_lora_down<kIn, 2>), dim3(tiles, parts, ways), dim3(kLoraThreads), 0, st, l, parts);
    else
        hipLaunchKernelGGL((k_lora_down<kIn, 4>), dim3(tiles, parts * nblk(l.r, 64), ways), dim3(kLoraThreads), 0, st, l, parts);
    const dim3 grid(tiles, nblk(l.N, 64 * kLoraWaves), ways);
    if (kIn == kBF16 && l.out_type == kF32)
        launch_up<kIn, 3>(l, parts, grid, st);
    else
        launch_up<kIn, 2>(l, parts, grid, st);
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
