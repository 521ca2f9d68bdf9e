// HIP kernels (CDNA4 / gfx950) of the MoE FFN layer for a few tokens: the layer of
// moe_kernels.hip on the same packed Q4 blob, for the one-token steps after a prompt.
//
//   route     top-k of the E logits (ties to the lower expert), w = softmax over the k;
//             a logit of -inf marks an expert that is not available: its slot has no
//             work and weight 0
//   gate/up   z = x [W_g | W_u]^T, h = z_g / (1 + exp(-z_g)) * z_u
//   down      dm = h W_d^T
//   combine   y[t] = sum_j w[t, j] dm[t, j], j ascending
//
// What bounds it: the bytes of the experts reached (0.5625 per weight); a token brings
// two operations per weight, far below the matrix cores' rate.  So the activations can
// be carried exactly enough to leave no rounding of their own: a block of 32 values is
// held as 24-bit integers times one power of two (error at most 2^-23 of the block's
// largest value), split into three signed bytes ("limbs"), and the
// int8 matrix instruction multiplies the limbs with the 4-bit codes exactly.  The three
// limbs of eight tokens fill the 32 rows of one instruction, which at these row counts
// would idle otherwise.  Per 32-block the limb sums are joined exactly in integers and
// scaled into an fp32 accumulator.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_decode.h"
#include "moe_dtype.h"
#include "moe_math.h"

namespace moe {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v16i __attribute__((ext_vector_type(16)));

namespace {

// -------------------------------------------------------------- fixed point ---
// Exponent field of the fixed-point scale of a block whose largest magnitude has the
// fp32 bits u: with E = that field, the value is q * 2^(E - 149), |q| <= 0x7F7F7F, so
// that three signed bytes hold q.  2^17 added to the mantissa moves the top 1/64 of a
// binade to the next one (q would pass 0x7F7F7F).  E >= 23 keeps 2^(E - 149) normal.
__device__ __forceinline__ int fix_exp(uint32_t u)
{
    const int e = (int)((u + (1u << 17)) >> 23);
    return e < 23 ? 23 : e;
}
// the block scale; NaN for a block that holds an infinity or a NaN
__device__ __forceinline__ float fix_scale(uint32_t u, int e)
{
    return u >= 0x7f800000u ? __builtin_nanf("") : __uint_as_float((uint32_t)(e - 22) << 23);
}
__device__ __forceinline__ int fix_code(float v, int e) { return (int)__builtin_rintf(ldexpf(v, 149 - e)); }

// q = l0 + 256 l1 + 65536 l2 with signed bytes
__device__ __forceinline__ void limbs(int q, int& l0, int& l1, int& l2)
{
    l0 = (int8_t)q;
    q = (q - l0) >> 8;
    l1 = (int8_t)q;
    l2 = (q - l1) >> 8;
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }
__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// ------------------------------------------------------------------ routing ---
// Keys order as (logit descending, expert ascending), -0 as +0: the order of the
// prompt path's routing.
__device__ __forceinline__ uint64_t route_key(float v, int e)
{
    uint32_t u = v == 0.0f ? 0u : __float_as_uint(v);
    u = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
    return ((uint64_t)u << 32) | (uint32_t)(0xFFFFFFFFu - (uint32_t)e);
}

__device__ __forceinline__ uint64_t wave_max_u64(uint64_t v)
{
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const uint64_t w = ((uint64_t)(uint32_t)__shfl_xor((int)(uint32_t)(v >> 32), o) << 32) |
                           (uint32_t)__shfl_xor((int)(uint32_t)v, o);
        v = v > w ? v : w;
    }
    return v;
}

// One token by one wave: the experts of its k slots (-1: not available) and their logits.
template <int NK>   // keys per lane: E <= 64 * NK
__device__ __forceinline__ void route_token(const float* __restrict__ lt, int E, int k,
                                            int* eidx, float* z)
{
    const int lane = threadIdx.x & 63;
    uint64_t key[NK];
#pragma unroll
    for (int i = 0; i < NK; ++i) {
        const int e = lane + 64 * i;
        key[i] = e < E ? route_key(lt[e], e) : 0ull;      // 0: below every real key
    }
    for (int j = 0; j < k; ++j) {
        uint64_t m = key[0];
#pragma unroll
        for (int i = 1; i < NK; ++i) m = key[i] > m ? key[i] : m;
        m = wave_max_u64(m);
#pragma unroll
        for (int i = 0; i < NK; ++i) key[i] = key[i] == m ? 0ull : key[i];
        if (lane == 0) {
            const int e = (int)(0xFFFFFFFFu - (uint32_t)m);
            const float l = lt[e];
            eidx[j] = l == -__builtin_inff() ? -1 : e;
            z[j] = l;
        }
    }
}

// Weights of one token's slots by one wave: softmax over the available ones, summed in
// slot order; 0 for the others (also where none is available).
__device__ __forceinline__ void route_weights(int k, const int* eidx, float* z)
{
    const int lane = threadIdx.x & 63;
    __builtin_amdgcn_wave_barrier();
    const float top = z[0];
    __builtin_amdgcn_wave_barrier();
    for (int j = lane; j < k; j += 64) z[j] = eidx[j] < 0 ? 0.0f : exp_cw(z[j] - top);
    __builtin_amdgcn_wave_barrier();
    float sum = 0.0f;
    for (int j = 0; j < k; ++j) sum += z[j];
    __builtin_amdgcn_wave_barrier();
    for (int j = lane; j < k; j += 64) z[j] = eidx[j] < 0 ? 0.0f : z[j] / sum;
}

constexpr int kRouteThreads = 1024;
constexpr int kRouteWaves = kRouteThreads / 64;
constexpr int kMaxE = 1024;

struct RouteArgs {
    const float* logits;
    int64_t logits_stride;
    int T, E, k;
    int32_t* eidx;
    float* wts;
    int32_t* counts;
    int32_t* nchunks;
    DecodeChunk* chunks;
    int max_chunks;
    int32_t* eidx_out;
    float* wts_out;
    const void* x;
    int64_t x_stride;
    int d;
    int8_t* xl;
    float* xs;
};

// Workgroup 0 routes every token (a token per wave at a time) and lists the chunks: per
// expert its pairs in groups of kChunkRows.  A pair's row inside its chunk depends on
// the order of LDS atomics; nothing else does, since every row is computed by itself.
__device__ __forceinline__ void route_all(const RouteArgs& a)
{
    __shared__ int s_eidx[kDecodeMaxPairs];
    __shared__ float s_z[kDecodeMaxPairs];
    __shared__ int s_cnt[kMaxE], s_first[kMaxE], s_fill[kMaxE];
    __shared__ int s_wave[kRouteWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int R = a.T * a.k;
    s_cnt[tid] = 0;
    s_fill[tid] = 0;
    for (int t = wave; t < a.T; t += kRouteWaves) {
        const float* lt = a.logits + (int64_t)t * a.logits_stride;
        if (a.E <= 256)
            route_token<4>(lt, a.E, a.k, s_eidx + t * a.k, s_z + t * a.k);
        else
            route_token<16>(lt, a.E, a.k, s_eidx + t * a.k, s_z + t * a.k);
        route_weights(a.k, s_eidx + t * a.k, s_z + t * a.k);
    }
    __syncthreads();
    const int e_of = tid < R ? s_eidx[tid] : -1;          // R <= kRouteThreads
    if (tid < R) {
        a.eidx[tid] = e_of;
        a.wts[tid] = s_z[tid];
        if (a.eidx_out) a.eidx_out[tid] = e_of;
        if (a.wts_out) a.wts_out[tid] = s_z[tid];
        if (e_of >= 0) atomicAdd(&s_cnt[e_of], 1);
    }
    __syncthreads();
    const int c = tid < a.E ? s_cnt[tid] : 0;
    const int nc = (c + kChunkRows - 1) / kChunkRows;
    int incl = nc;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int y = __shfl_up(incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 63) s_wave[wave] = incl;
    __syncthreads();
    int before = 0, total = 0;
    for (int i = 0; i < kRouteWaves; ++i) {
        before += i < wave ? s_wave[i] : 0;
        total += s_wave[i];
    }
    const int first = before + incl - nc;
    s_first[tid] = first;
    if (tid < a.E) {
        a.counts[tid] = c;
        for (int i = 0; i < nc; ++i) {
            a.chunks[first + i].expert = tid;
            a.chunks[first + i].n = c - i * kChunkRows < kChunkRows ? c - i * kChunkRows : kChunkRows;
        }
    }
    if (tid == 0) *a.nchunks = total;
    __syncthreads();
    if (e_of >= 0) {
        const int r = atomicAdd(&s_fill[e_of], 1);
        a.chunks[s_first[e_of] + r / kChunkRows].pair[r % kChunkRows] = tid;
    }
}

// x in fixed point: 8 lanes per block of 32, limb plane l of token t at xl[(3 t + l) d].
template <int kT>
__device__ __forceinline__ void x_to_fixed(const RouteArgs& a, int64_t first)
{
    const int nb = a.d / 32;
    const int64_t blk = first + (threadIdx.x >> 3);
    if (blk >= (int64_t)a.T * nb) return;                 // uniform over the 8-lane group
    const int sub = threadIdx.x & 7;
    const int t = (int)(blk / nb), b = (int)(blk - (int64_t)t * nb);
    float v[4];
    load_n<kT, 4>(static_cast<const uint8_t*>(a.x) +
                  ((int64_t)t * a.x_stride + b * 32 + sub * 4) * dtype_bytes(kT), v);
    uint32_t u = umax(umax(abs_bits(v[0]), abs_bits(v[1])), umax(abs_bits(v[2]), abs_bits(v[3])));
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) u = umax(u, (uint32_t)__shfl_xor((int)u, o));
    const int e = fix_exp(u);
    uint32_t w[3] = {0, 0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        int l[3];
        limbs(u >= 0x7f800000u ? 0 : fix_code(v[i], e), l[0], l[1], l[2]);
#pragma unroll
        for (int j = 0; j < 3; ++j) w[j] |= (uint32_t)(l[j] & 0xff) << (8 * i);
    }
#pragma unroll
    for (int j = 0; j < 3; ++j)
        *reinterpret_cast<uint32_t*>(a.xl + ((int64_t)t * 3 + j) * a.d + b * 32 + sub * 4) = w[j];
    if (sub == 0) a.xs[(int64_t)t * nb + b] = fix_scale(u, e);
}

template <int kT>
__global__ __launch_bounds__(kRouteThreads) void k_decode_route(RouteArgs a)
{
    if (blockIdx.x == 0) {
        route_all(a);
        return;
    }
    x_to_fixed<kT>(a, (int64_t)(blockIdx.x - 1) * (kRouteThreads / 8));
}

// ---------------------------------------------------------- expert products ---
struct ProductArgs {
    const int32_t* nchunks;
    const DecodeChunk* chunks;
    const uint8_t* blob;
    uint64_t expert_stride, q_off, s_off;
    const int8_t* al;         // fixed-point activations: limb plane l of row r at al[(3 r + l) K]
    const float* as;          // their block scales [rows][K / 32]
    int K, E;
    int pair_div;             // row of a pair: pair / pair_div (gate/up: top_k, down: 1)
    int max_rows;             // rows of al (bounds the pair list)
    int8_t* hl;               // gate/up: h in fixed point
    float* hs;
    int f;
    float* dm;                // down: [pairs][d]
    int d;
};

// Eight codes of a word as bytes holding 16 x the weight (see moe_kernels.hip's grouped
// GEMM: the code with its top bit flipped is the weight in 4-bit two's complement).
__device__ __forceinline__ v4i unpack16x(uint32_t w0, uint32_t w1)
{
    v4i b;
    b.x = (int)(((w0 << 4) & 0xF0F0F0F0u) ^ 0x80808080u);
    b.y = (int)((w0 & 0xF0F0F0F0u) ^ 0x80808080u);
    b.z = (int)(((w1 << 4) & 0xF0F0F0F0u) ^ 0x80808080u);
    b.w = (int)((w1 & 0xF0F0F0F0u) ^ 0x80808080u);
    return b;
}

constexpr int kProdWaves = 4;
constexpr int kMaxBlocks = 16384 / 32;

// One chunk of one expert times one 32-column tile of its matrix (gate/up: the gate tile
// and the up tile of the same columns).  The waves of a workgroup split K and add up
// through LDS in wave order.  Row 4 m + l of the instruction's 32 rows holds limb l of
// token m, so that a lane gets the three limb sums of a (token, column) in one quad of
// its result registers: token m is register quad m / 2 of lane half m % 2.
template <bool kGateUp>
__global__ __launch_bounds__(64 * kProdWaves) void k_decode_product(ProductArgs g)
{
    constexpr int NT = kGateUp ? 2 : 1;
    __shared__ float s_scale[kChunkRows * kMaxBlocks];
    __shared__ float s_red[kProdWaves][NT][kChunkRows][32];
    if ((int)blockIdx.y >= *g.nchunks) return;            // uniform
    const DecodeChunk& ch = g.chunks[blockIdx.y];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, h = lane >> 5, j32 = lane & 31;
    const int nb = g.K / 32, npairs = k_pairs(g.K), ngroups = scale_groups(g.K);
    int n = ch.n, e = ch.expert;
    n = n < 1 ? 1 : (n > kChunkRows ? kChunkRows : n);
    e = e < 0 ? 0 : (e >= g.E ? g.E - 1 : e);
    auto row_of = [&](int m) {
        int r = ch.pair[m] / g.pair_div;
        return r < 0 ? 0 : (r >= g.max_rows ? g.max_rows - 1 : r);
    };
    for (int i = tid; i < n * nb; i += 64 * kProdWaves) {
        const int m = i / nb;
        s_scale[i] = g.as[(int64_t)row_of(m) * nb + (i - m * nb)];
    }
    const int m_a = j32 >> 2, l_a = j32 & 3;              // the A row this lane feeds
    const bool a_on = m_a < n && l_a < 3;
    const int8_t* al = g.al + ((int64_t)row_of(a_on ? m_a : 0) * 3 + (a_on ? l_a : 0)) * g.K + 16 * h;
    const uint8_t* ex = g.blob + (uint64_t)e * g.expert_stride;
    const int nt0 = (int)blockIdx.x * NT;
    const uint8_t* wq = ex + g.q_off + (uint64_t)nt0 * npairs * 1024 + lane * 16;
    const uint8_t* wsc = ex + g.s_off + ((uint64_t)nt0 * ngroups * 32 + j32) * 16;
    __syncthreads();

    float acc[NT][4] = {};
    const v16i zero = {0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
    const int ng = (n + 1) >> 1;
    const int p0 = wave * npairs / kProdWaves, p1 = (wave + 1) * npairs / kProdWaves;
#pragma unroll 2
    for (int pr = p0; pr < p1; ++pr) {
        uint4 bq[NT];
        uint32_t bs[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            bq[t] = *reinterpret_cast<const uint4*>(wq + ((uint64_t)t * npairs + pr) * 1024);
            bs[t] = *reinterpret_cast<const uint32_t*>(wsc + ((uint64_t)t * ngroups + (pr >> 2)) * 512 + (pr & 3) * 4);
        }
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int b = 2 * pr + q;
            if (b >= nb) break;                           // uniform: the padded block of an odd count
            v4i a = {0, 0, 0, 0};
            if (a_on) a = *reinterpret_cast<const v4i*>(al + b * 32);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const v4i w = q ? unpack16x(bq[t].z, bq[t].w) : unpack16x(bq[t].x, bq[t].y);
                const uint16_t hb = (uint16_t)(q ? bs[t] >> 16 : bs[t] & 0xffffu);
                const float ws = (float)__builtin_bit_cast(_Float16, hb) * 0.0625f;
                const v16i s = __builtin_amdgcn_mfma_i32_32x32x32_i8(a, w, zero, 0, 0, 0);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    if (c < ng) {                         // uniform
                        // 16 x the limb sums; s0 + 256 s1 is a multiple of 16 below 2^28: exact in fp32
                        const float lo = (float)(s[4 * c] + (s[4 * c + 1] << 8));
                        const float v = __builtin_fmaf((float)s[4 * c + 2], 65536.0f, lo);
                        const int m = 2 * c + h < n ? 2 * c + h : n - 1;
                        acc[t][c] = __builtin_fmaf(v, ws * s_scale[m * nb + b], acc[t][c]);
                    }
                }
            }
        }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int c = 0; c < 4; ++c) s_red[wave][t][2 * c + h][j32] = acc[t][c];
    __syncthreads();
    const int m = tid >> 5, col = (int)blockIdx.x * 32 + j32;
    static_assert(64 * kProdWaves == 32 * kChunkRows, "one thread per (row, column)");
    if (m >= n) return;                                   // uniform over the 32-lane half
    float z[NT] = {};
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int w = 0; w < kProdWaves; ++w) z[t] += s_red[w][t][m][j32];
    int p = ch.pair[m];
    if (kGateUp) {
        const float hv = z[0] / (1.0f + exp_cw(-z[0])) * z[NT - 1];
        uint32_t u = abs_bits(hv);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) u = umax(u, (uint32_t)__shfl_xor((int)u, o));
        const int ex2 = fix_exp(u);
        int l0, l1, l2;
        limbs(u >= 0x7f800000u ? 0 : fix_code(hv, ex2), l0, l1, l2);
        int8_t* o = g.hl + (int64_t)p * 3 * g.f + col;
        o[0] = (int8_t)l0;
        o[g.f] = (int8_t)l1;
        o[2 * g.f] = (int8_t)l2;
        if (j32 == 0) g.hs[(int64_t)p * (g.f / 32) + blockIdx.x] = fix_scale(u, ex2);
    } else {
        g.dm[(int64_t)p * g.d + col] = z[0];
    }
}

// ------------------------------------------------------------------ combine ---
template <int kT>
__global__ __launch_bounds__(256) void k_decode_combine(const float* __restrict__ dm,
                                                        const float* __restrict__ wts,
                                                        const int32_t* __restrict__ eidx, int T, int k,
                                                        int d, void* __restrict__ y, int64_t y_stride)
{
    const int d4 = d >> 2;
    const int64_t gid = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (gid >= (int64_t)T * d4) return;
    const int t = (int)(gid / d4), c = (int)(gid - (int64_t)t * d4) * 4;
    float acc[4] = {};
    for (int j = 0; j < k; ++j) {
        const int p = t * k + j;
        if (eidx[p] < 0) continue;
        const float w = wts[p];
        const float4 v = *reinterpret_cast<const float4*>(dm + (int64_t)p * d + c);
        acc[0] = __builtin_fmaf(w, v.x, acc[0]);
        acc[1] = __builtin_fmaf(w, v.y, acc[1]);
        acc[2] = __builtin_fmaf(w, v.z, acc[2]);
        acc[3] = __builtin_fmaf(w, v.w, acc[3]);
    }
    store_n<kT, 4>(static_cast<uint8_t*>(y) + ((int64_t)t * y_stride + c) * dtype_bytes(kT), acc);
}

unsigned nblk(int64_t n, int per) { return (unsigned)((n + per - 1) / per); }

}  // namespace

// ----------------------------------------------------------------- launches ---
hipError_t launch_decode_route(const DecodeLaunch& D, hipStream_t st)
{
    RouteArgs a;
    a.logits = D.logits;
    a.logits_stride = D.logits_stride;
    a.T = D.T;
    a.E = D.E;
    a.k = D.k;
    a.eidx = reinterpret_cast<int32_t*>(D.ws + D.L.eidx);
    a.wts = reinterpret_cast<float*>(D.ws + D.L.wts);
    a.counts = reinterpret_cast<int32_t*>(D.ws + D.L.counts);
    a.nchunks = reinterpret_cast<int32_t*>(D.ws + D.L.nchunks);
    a.chunks = reinterpret_cast<DecodeChunk*>(D.ws + D.L.chunks);
    a.max_chunks = D.L.max_chunks;
    a.eidx_out = D.eidx_out;
    a.wts_out = D.wts_out;
    a.x = D.x;
    a.x_stride = D.x_stride;
    a.d = D.d;
    a.xl = reinterpret_cast<int8_t*>(D.ws + D.L.xl);
    a.xs = reinterpret_cast<float*>(D.ws + D.L.xs);
    const dim3 grid(1 + nblk((int64_t)D.T * (D.d / 32), kRouteThreads / 8)), block(kRouteThreads);
    if (D.dtype == kF32)
        hipLaunchKernelGGL(k_decode_route<kF32>, grid, block, 0, st, a);
    else if (D.dtype == kBF16)
        hipLaunchKernelGGL(k_decode_route<kBF16>, grid, block, 0, st, a);
    else
        hipLaunchKernelGGL(k_decode_route<kF16>, grid, block, 0, st, a);
    return hipGetLastError();
}

hipError_t launch_decode_products(const DecodeLaunch& D, hipStream_t st)
{
    ProductArgs g;
    g.nchunks = reinterpret_cast<const int32_t*>(D.ws + D.L.nchunks);
    g.chunks = reinterpret_cast<const DecodeChunk*>(D.ws + D.L.chunks);
    g.blob = D.blob;
    g.expert_stride = D.expert_stride;
    g.q_off = D.gu_q_off;
    g.s_off = D.gu_s_off;
    g.al = reinterpret_cast<const int8_t*>(D.ws + D.L.xl);
    g.as = reinterpret_cast<const float*>(D.ws + D.L.xs);
    g.K = D.d;
    g.E = D.E;
    g.pair_div = D.k;
    g.max_rows = D.T;
    g.hl = reinterpret_cast<int8_t*>(D.ws + D.L.hl);
    g.hs = reinterpret_cast<float*>(D.ws + D.L.hs);
    g.f = D.f;
    g.dm = reinterpret_cast<float*>(D.ws + D.L.dm);
    g.d = D.d;
    hipLaunchKernelGGL(k_decode_product<true>, dim3(D.f / 32, D.L.max_chunks), dim3(64 * kProdWaves), 0, st, g);
    g.q_off = D.d_q_off;
    g.s_off = D.d_s_off;
    g.al = g.hl;
    g.as = g.hs;
    g.K = D.f;
    g.pair_div = 1;
    g.max_rows = D.T * D.k;
    hipLaunchKernelGGL(k_decode_product<false>, dim3(D.d / 32, D.L.max_chunks), dim3(64 * kProdWaves), 0, st, g);
    return hipGetLastError();
}

hipError_t launch_decode_combine(const DecodeLaunch& D, hipStream_t st)
{
    const float* dm = reinterpret_cast<const float*>(D.ws + D.L.dm);
    const float* wts = reinterpret_cast<const float*>(D.ws + D.L.wts);
    const int32_t* eidx = reinterpret_cast<const int32_t*>(D.ws + D.L.eidx);
    const dim3 grid(nblk((int64_t)D.T * (D.d / 4), 256)), block(256);
    if (D.dtype == kF32)
        hipLaunchKernelGGL(k_decode_combine<kF32>, grid, block, 0, st, dm, wts, eidx, D.T, D.k, D.d, D.y, D.y_stride);
    else if (D.dtype == kBF16)
        hipLaunchKernelGGL(k_decode_combine<kBF16>, grid, block, 0, st, dm, wts, eidx, D.T, D.k, D.d, D.y, D.y_stride);
    else
        hipLaunchKernelGGL(k_decode_combine<kF16>, grid, block, 0, st, dm, wts, eidx, D.T, D.k, D.d, D.y, D.y_stride);
    return hipGetLastError();
}

}  // namespace moe
