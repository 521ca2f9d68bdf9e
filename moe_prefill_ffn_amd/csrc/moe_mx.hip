// HIP kernels (CDNA4 / gfx950) of the MXFP4 operators: a matrix to blocks of 32 4-bit
// floating-point elements with one power-of-two scale each and back, and the product of
// two such matrices, dense or over the groups of a row table.
//
// A block's scale is 2^(s - 127) for its E8M0 byte s = max(0, floor(log2 amax) - 2 + 127)
// (2: the exponent of the largest element, 6 = 1.5 * 2^2); its elements are E2M1, the
// values 0, 0.5, 1, 1.5, 2, 3, 4, 6 with a sign, x / scale rounded to the nearest, ties to
// the even code, 6 beyond the largest.  Byte 255 marks a block that held an infinity or a
// NaN; such a block reads as NaN (OCP Microscaling Formats v1.0, sections 5 and 6.3).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_dtype.h"
#include "moe_math.h"
#include "moe_mx.h"

namespace moe {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v2f __attribute__((ext_vector_type(2)));
typedef float v16f __attribute__((ext_vector_type(16)));

namespace {

unsigned nblk(int64_t n, int per) { return (unsigned)((n + per - 1) / per); }

// 2^(s - 127); s = 0 is the fp32 subnormal 2^-127, s = 255 NaN
__device__ __forceinline__ float e8m0(uint32_t s)
{
    return s == 0 ? __uint_as_float(0x00400000u) : s == 255 ? __builtin_nanf("") : __uint_as_float(s << 23);
}

// ---------------------------------------------------- quantise, dequantise ---
// Four lanes per block, eight values each; a wave takes 16 consecutive blocks.
constexpr int kQuantThreads = 256;
constexpr int kQuantBlocks = kQuantThreads / 4;           // blocks per workgroup

struct BlockAt {
    int64_t row;
    int b;
};
__device__ __forceinline__ BlockAt block_at(int64_t blk, int nb)
{
    const uint32_t row = (uint32_t)blk / (uint32_t)nb;    // fewer than 2^31 blocks
    return {(int64_t)row, (int)((uint32_t)blk - row * (uint32_t)nb)};
}

template <int kT>
__device__ __forceinline__ void load8(const uint8_t* p, float (&v)[8])
{
    if constexpr (kT == kF32) {
        float a[4], b[4];
        load_n<kT, 4>(p, a);
        load_n<kT, 4>(p + 16, b);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = a[i];
            v[4 + i] = b[i];
        }
    } else {
        load_n<kT, 8>(p, v);
    }
}

template <int kT>
__device__ __forceinline__ void store8(uint8_t* p, const float (&v)[8])
{
    if constexpr (kT == kF32) {
        const float a[4] = {v[0], v[1], v[2], v[3]}, b[4] = {v[4], v[5], v[6], v[7]};
        store_n<kT, 4>(p, a);
        store_n<kT, 4>(p + 16, b);
    } else {
        store_n<kT, 8>(p, v);
    }
}

template <int kT>
__global__ __launch_bounds__(kQuantThreads) void k_mx_quantize(MxQuant q, int64_t n_blocks)
{
    const int nb = q.K / 32, sub = threadIdx.x & 3;
    const int64_t blk = (int64_t)blockIdx.x * kQuantBlocks + (threadIdx.x >> 2);
    if (blk >= n_blocks) return;                          // uniform over the 4-lane group
    const BlockAt at = block_at(blk, nb);
    float v[8];
    load8<kT>(static_cast<const uint8_t*>(q.x) + (at.row * q.stride + at.b * 32 + sub * 8) * dtype_bytes(kT), v);
    // the largest magnitude by its bits: an infinity, then a NaN, order above every number
    uint32_t u = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t a = __float_as_uint(v[i]) & 0x7fffffffu;
        u = a > u ? a : u;
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
        const uint32_t a = (uint32_t)__shfl_xor((int)u, o);
        u = a > u ? a : u;
    }
    const bool bad = u >= 0x7f800000u;
    const int e = (int)(u >> 23) - 2;
    const uint32_t s = bad ? 255u : (uint32_t)(e < 0 ? 0 : e);
    const float sc = e8m0(bad ? 127u : s);
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], sc, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], sc, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], sc, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], sc, 3);
    reinterpret_cast<uint32_t*>(q.codes)[blk * 4 + sub] = bad ? 0u : w;
    if (sub == 0) q.scales[blk] = (uint8_t)s;
}

template <int kT>
__global__ __launch_bounds__(kQuantThreads) void k_mx_dequantize(MxQuant q, int64_t n_blocks)
{
    const int nb = q.K / 32, sub = threadIdx.x & 3;
    const int64_t blk = (int64_t)blockIdx.x * kQuantBlocks + (threadIdx.x >> 2);
    if (blk >= n_blocks) return;
    const BlockAt at = block_at(blk, nb);
    const uint32_t w = reinterpret_cast<const uint32_t*>(q.codes)[blk * 4 + sub];
    const float sc = e8m0(q.scales[blk]);
    float v[8];
    const v2f p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0);
    const v2f p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
    const v2f p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2);
    const v2f p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
    v[0] = p0.x * sc;
    v[1] = p0.y * sc;
    v[2] = p1.x * sc;
    v[3] = p1.y * sc;
    v[4] = p2.x * sc;
    v[5] = p2.y * sc;
    v[6] = p3.x * sc;
    v[7] = p3.y * sc;
    store8<kT>(static_cast<uint8_t*>(q.y) + (at.row * q.stride + at.b * 32 + sub * 8) * dtype_bytes(kT), v);
}

// ------------------------------------------------------------------ product ---
// The scaled matrix instruction takes 32 codes of one block and the block's scale byte
// per lane and adds the scaled products into fp32.
//
// Groups of a row table: tile slot s belongs to the last group g whose first slot
// bounds[g] / BM + g is <= s (a group of c rows never needs more than the
// bounds[g + 1] / BM + 1 - bounds[g] / BM slots up to the next group's first), so a
// workgroup finds its rows from the bounds alone, without a list of tiles.
struct Tile {
    int g;
    int64_t m0, m1;           // rows [m0, m1) of the tile; m0 >= m1: nothing to do
};

template <int BM>
__device__ __forceinline__ Tile tile_of_slot(const MxGemm& a, int64_t slot)
{
    if (!a.bounds) {
        const int64_t m0 = slot * BM;
        return {0, m0, m0 + BM < a.M ? m0 + BM : a.M};
    }
    int lo = 0, hi = a.G - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if ((int64_t)(a.bounds[mid] / BM) + mid <= slot)
            lo = mid;
        else
            hi = mid - 1;
    }
    const int64_t b0 = a.bounds[lo], b1 = a.bounds[lo + 1];
    int64_t m0 = b0 + (slot - (b0 / BM + lo)) * BM, m1 = m0 + BM < b1 ? m0 + BM : b1;
    // sound bounds ascend within [0, M]; this only keeps others from reaching outside
    if (m0 < b0 || m0 < 0) m0 = m1;
    if (m1 > a.M) m1 = a.M;
    return {lo, m0, m1};
}

constexpr int kMxWaves = 4;
constexpr int kMxBM = 32, kMxBN = 32 * kMxWaves;          // columns per workgroup, per half

// Each wave: 32 rows x two 32-column tiles, fed straight from memory.  SwiGLU: the two
// tiles are the gate and the up rows of the same output columns.
template <int kT, bool kSwiglu>
__global__ __launch_bounds__(64 * kMxWaves) void k_mx_gemm(MxGemm a)
{
    const Tile t = tile_of_slot<kMxBM>(a, blockIdx.x);
    if (t.m0 >= t.m1) return;                             // uniform
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, h = lane >> 5, j = lane & 31;
    const int nb = a.K / 32, NB = kSwiglu ? 2 * a.N : a.N;
    const int n0 = ((int)blockIdx.y * kMxWaves + wave) * (kSwiglu ? 32 : 64);
    if (n0 >= a.N) return;
    const int64_t r = t.m0 + j < t.m1 ? t.m0 + j : t.m1 - 1;
    int64_t src = (a.rows ? (int64_t)a.rows[r] : r) / a.row_div;
    src = src < 0 ? 0 : (src >= a.a_rows ? a.a_rows - 1 : src);
    int bn[2];
    bn[0] = n0 + j < a.N ? n0 + j : a.N - 1;
    bn[1] = kSwiglu ? a.N + bn[0] : (n0 + 32 + j < a.N ? n0 + 32 + j : a.N - 1);
    const uint8_t* ac = a.a_codes + src * (a.K / 2);
    const uint8_t* as = a.a_scales + src * nb;
    const uint8_t* bc[2];
    const uint8_t* bs[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int64_t row = (int64_t)t.g * NB + bn[i];
        bc[i] = a.b_codes + row * (a.K / 2);
        bs[i] = a.b_scales + row * nb;
    }
    v16f acc[2];
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[0][i] = acc[1][i] = 0.0f;
    for (int b0 = 0; b0 < nb; b0 += 2) {
        const int b = b0 + h;
        v8i av = {0, 0, 0, 0, 0, 0, 0, 0}, bv[2] = {av, av};
        int sa = 127, sb[2] = {127, 127};
        if (b < nb) {                                     // past the end: zeros with scale 1
            const uint4 w = *reinterpret_cast<const uint4*>(ac + b * 16);
            av[0] = (int)w.x, av[1] = (int)w.y, av[2] = (int)w.z, av[3] = (int)w.w;
            sa = as[b];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint4 u = *reinterpret_cast<const uint4*>(bc[i] + b * 16);
                bv[i][0] = (int)u.x, bv[i][1] = (int)u.y, bv[i][2] = (int)u.z, bv[i][3] = (int)u.w;
                sb[i] = bs[i][b];
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
            acc[i] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, bv[i], acc[i], 4, 4, 0, sa, 0, sb[i]);
    }
    uint8_t* out = static_cast<uint8_t*>(a.out);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int64_t row = t.m0 + 8 * (i >> 2) + 4 * h + (i & 3);
        if (row >= t.m1) continue;
        typedef typename Elem<kT>::type T;
        T* o = reinterpret_cast<T*>(out) + row * a.out_stride;
        if (kSwiglu) {
            const float gt = acc[0][i];
            if (n0 + j < a.N) o[n0 + j] = from_f32<kT>(gt / (1.0f + exp_cw(-gt)) * acc[1][i]);
        } else {
            if (n0 + j < a.N) o[n0 + j] = from_f32<kT>(acc[0][i]);
            if (n0 + 32 + j < a.N) o[n0 + 32 + j] = from_f32<kT>(acc[1][i]);
        }
    }
}

}  // namespace

// ----------------------------------------------------------------- launches ---
hipError_t launch_mx_quantize(const MxQuant& q, hipStream_t st)
{
    const int64_t n = q.M * (q.K / 32);
    if (n == 0) return hipSuccess;
    const dim3 grid(nblk(n, kQuantBlocks)), block(kQuantThreads);
    if (q.dtype == kF32)
        hipLaunchKernelGGL(k_mx_quantize<kF32>, grid, block, 0, st, q, n);
    else if (q.dtype == kBF16)
        hipLaunchKernelGGL(k_mx_quantize<kBF16>, grid, block, 0, st, q, n);
    else
        hipLaunchKernelGGL(k_mx_quantize<kF16>, grid, block, 0, st, q, n);
    return hipGetLastError();
}

hipError_t launch_mx_dequantize(const MxQuant& q, hipStream_t st)
{
    const int64_t n = q.M * (q.K / 32);
    if (n == 0) return hipSuccess;
    const dim3 grid(nblk(n, kQuantBlocks)), block(kQuantThreads);
    if (q.dtype == kF32)
        hipLaunchKernelGGL(k_mx_dequantize<kF32>, grid, block, 0, st, q, n);
    else if (q.dtype == kBF16)
        hipLaunchKernelGGL(k_mx_dequantize<kBF16>, grid, block, 0, st, q, n);
    else
        hipLaunchKernelGGL(k_mx_dequantize<kF16>, grid, block, 0, st, q, n);
    return hipGetLastError();
}

template <int kT>
static void gemm_typed(const MxGemm& g, dim3 grid, hipStream_t st)
{
    if (g.swiglu)
        hipLaunchKernelGGL((k_mx_gemm<kT, true>), grid, dim3(64 * kMxWaves), 0, st, g);
    else
        hipLaunchKernelGGL((k_mx_gemm<kT, false>), grid, dim3(64 * kMxWaves), 0, st, g);
}

hipError_t launch_mx_gemm(const MxGemm& g, hipStream_t st)
{
    if (g.M == 0) return hipSuccess;
    const int64_t slots = g.bounds ? g.M / kMxBM + g.G : (int64_t)nblk(g.M, kMxBM);
    const dim3 grid((unsigned)slots, nblk(g.N, g.swiglu ? kMxBN : 2 * kMxBN));
    if (g.dtype == kF32)
        gemm_typed<kF32>(g, grid, st);
    else if (g.dtype == kBF16)
        gemm_typed<kBF16>(g, grid, st);
    else
        gemm_typed<kF16>(g, grid, st);
    return hipGetLastError();
}

}  // namespace moe
