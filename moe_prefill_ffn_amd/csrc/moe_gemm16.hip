// HIP kernels (CDNA4 / gfx950) of products of 16-bit matrices (bf16 or fp16), dense or over the
// groups of a row table:
//   out[r, n] = sum_k A[src(r), k] B[g(r), n, k]
// in fp32, with SwiGLU of gate and up rows of B where asked for, rounded once.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "moe_dtype.h"
#include "moe_gemm16.h"
#include "moe_tile.h"

namespace moe {

namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));

// The matrix instruction takes 8 values of K per lane half and operand.  Its first operand is the
// weights, the second the activations, so a lane holds four consecutive output columns of one row
// in consecutive result registers.  Which 8 values of K a lane half takes is free as long as both
// operands agree: half h takes chunk 4 h + s (16 bytes) in step s of 64 values (128 bytes, a cache
// line), so that a lane reads 64 consecutive bytes of a row.
template <int kIn>
__device__ __forceinline__ v16f mfma16(v4i w, v4i x, v16f c)
{
    if constexpr (kIn == kBF16)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, w), __builtin_bit_cast(v8bf, x), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v8h, w), __builtin_bit_cast(v8h, x), c, 0, 0, 0);
}

// A row of the product reads this row of A.
__device__ __forceinline__ int64_t a_row(const Gemm16& a, int64_t r)
{
    int src = a.rows ? a.rows[r] : (int)r;                // r < 2^27
    if (a.row_div > 1) src /= a.row_div;
    return src < 0 ? 0 : (src >= a.a_rows ? a.a_rows - 1 : src);
}

// ----------------------------------------------------------- few-row kernel ---
// Up to 32 rows of a group by 32 columns (SwiGLU: 32 gate and 32 up rows of B) per workgroup; its
// waves take every eighth 64 values of K, fed straight from memory, and add up through LDS in wave
// order.  A chunk past the end of K is 0 in both operands.
constexpr int kFewWaves = 8, kFewRows = 32;

template <int kIn, int kT, bool kSwiglu>
__global__ __launch_bounds__(64 * kFewWaves) void k_gemm16_few(Gemm16 a)
{
    constexpr int NT = kSwiglu ? 2 : 1;
    __shared__ float red[kFewWaves][NT][32][33];
    const Rows t = rows_of_slot<kFewRows>(a, blockIdx.x);
    if (t.m0 >= t.m1) return;                             // uniform
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, h = lane >> 5, j = lane & 31;
    const int chunks = a.K / 8;
    const int n0 = (int)blockIdx.y * 32;
    const uint8_t* x = a.a + a_row(a, t.m0 + j < t.m1 ? t.m0 + j : t.m1 - 1) * a.a_stride;
    const uint8_t* w[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i)
        w[i] = a.b + t.g * a.b_group + (int64_t)((n0 + j < a.N ? n0 + j : a.N - 1) + i * a.N) * a.b_stride;
    v16f acc[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][e] = 0.0f;
    for (int u = wave * 8; u < chunks; u += 8 * kFewWaves) {
        v4i vx[4], vw[NT][4];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int c = u + 4 * h + s;
            const bool in = c < chunks;
#pragma unroll
            for (int i = 0; i < NT; ++i) vw[i][s] = in ? *reinterpret_cast<const v4i*>(w[i] + c * 16) : v4i{0, 0, 0, 0};
            vx[s] = in ? *reinterpret_cast<const v4i*>(x + c * 16) : v4i{0, 0, 0, 0};
        }
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int i = 0; i < NT; ++i) acc[i] = mfma16<kIn>(vw[i][s], vx[s], acc[i]);
    }
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) red[wave][i][j][8 * (e >> 2) + 4 * h + (e & 3)] = acc[i][e];
    __syncthreads();
    typedef typename Elem<kT>::type T;
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        const int row = p * 16 + (tid >> 5), col = tid & 31;
        if (t.m0 + row >= t.m1 || n0 + col >= a.N) continue;
        float z[NT] = {};
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int v = 0; v < kFewWaves; ++v) z[i] += red[v][i][row][col];
        static_cast<T*>(a.out)[(t.m0 + row) * a.out_stride + n0 + col] =
            from_f32<kT>(kSwiglu ? silu_mul(z[0], z[NT - 1]) : z[0]);
    }
}

}  // namespace

// ----------------------------------------------------------------- launches ---
namespace {

// The most tiles of BM rows that the groups can have.
int64_t slots_of(const Gemm16& g, int BM) { return g.bounds ? g.M / BM + g.G : (g.M + BM - 1) / BM; }

template <int kIn, int kT, bool kSwiglu>
hipError_t launch_shape(const Gemm16& g, hipStream_t st)
{
    hipLaunchKernelGGL((k_gemm16_few<kIn, kT, kSwiglu>), dim3((unsigned)slots_of(g, kFewRows), nblk(g.N, 32)), dim3(64 * kFewWaves), 0, st, g);
    return hipGetLastError();
}

template <int kIn>
hipError_t launch_typed(const Gemm16& g, hipStream_t st)
{
    if (g.out_type == kF32) return g.swiglu ? launch_shape<kIn, kF32, true>(g, st) : launch_shape<kIn, kF32, false>(g, st);
    return g.swiglu ? launch_shape<kIn, kIn, true>(g, st) : launch_shape<kIn, kIn, false>(g, st);
}

}  // namespace

hipError_t launch_gemm16(const Gemm16& g, hipStream_t st)
{
    if (g.M == 0) return hipSuccess;
    return g.in_type == kBF16 ? launch_typed<kBF16>(g, st) : launch_typed<kF16>(g, st);
}

}  // namespace moe
