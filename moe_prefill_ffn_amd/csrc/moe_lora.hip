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

// The adapter of row m, -1: none, or no such row.
__device__ __forceinline__ int adapter_of(const LoraAdd& l, int64_t m)
{
    const int id = m < l.M ? l.adapters[m] : -1;
    return (uint32_t)id < (uint32_t)l.n ? id : -1;
}

// Calls f(adapter) for the distinct adapters of a tile, number way, way + ways, ... in the order in which
// rows first name them; uniform over the wave.  id: of rows lane, lane + 64, ... of the tile (-1 beyond its rows).
template <int kI, class F>
__device__ __forceinline__ void each_adapter(const int (&id)[kI], int way, int ways, F f)
{
    uint64_t left[kI];
#pragma unroll
    for (int i = 0; i < kI; ++i) left[i] = __ballot(id[i] >= 0);
    for (int at = 0;; ++at) {
        int cur = -1;
#pragma unroll
        for (int i = kI - 1; i >= 0; --i)
            if (left[i]) cur = __builtin_amdgcn_readlane(id[i], __builtin_ctzll(left[i]));
        if (cur < 0) break;
#pragma unroll
        for (int i = 0; i < kI; ++i) left[i] &= ~__ballot(id[i] == cur);
        if (at % ways == way) f(cur);
    }
}

// --------------------------------------------------------------- s = x A^T ---
// Few rows.  A workgroup: 16 rows, one part of K shared out to its waves 64 values at a time, up to 16 kRT
// ranks, straight from memory.  Rows of another adapter are computed along and not stored.  A wave's next
// loads are out while it multiplies.
template <int kIn, int kRT>
__global__ __launch_bounds__(kLoraThreads) void k_lora_down_few(LoraAdd l, int parts)
{
    __shared__ float red[kLoraWaves][16][16 * kRT + 4];
    const int tid = threadIdx.x, lane = tid & 63, i = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t m0 = (int64_t)blockIdx.x * 16;
    const int part = (int)blockIdx.y % parts, r0 = (int)blockIdx.y / parts * 16 * kRT;
    const int chunks = l.K / 8, per = ((chunks + parts - 1) / parts + 7) / 8 * 8;    // 16-byte chunks a part
    const int c0 = part * per + wave * 8, c1 = (part + 1) * per < chunks ? (part + 1) * per : chunks;
    constexpr int kStep = 8 * kLoraWaves;
    const int id[1] = {lane < 16 ? adapter_of(l, m0 + lane) : -1};
    const uint8_t* x = l.x + (m0 + i < l.M ? m0 + i : l.M - 1) * l.x_stride + 32 * g;
    struct Frag {
        v4i x[2], a[2][kRT];
    };
    each_adapter(id, blockIdx.z, gridDim.z, [&](int cur) {
        const uint8_t* a[kRT];
        v4f acc[kRT];
#pragma unroll
        for (int t = 0; t < kRT; ++t) {
            const int q = r0 + 16 * t + i < l.r ? r0 + 16 * t + i : l.r - 1;
            a[t] = l.a + ((int64_t)cur * l.r + q) * l.K * 2 + 32 * g;
            acc[t] = v4f{0, 0, 0, 0};
        }
        // lane group g: chunks u + 2 g, + 1; past the part's end 0
        auto load = [&](Frag& f, int u) {
            const bool whole = u + 8 <= c1;               // uniform
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const bool in = whole || u + 2 * g + s < c1;
                const int64_t at = (int64_t)(u + s) * 16;
                f.x[s] = in ? *reinterpret_cast<const v4i*>(x + at) : v4i{0, 0, 0, 0};
#pragma unroll
                for (int t = 0; t < kRT; ++t) f.a[s][t] = in ? *reinterpret_cast<const v4i*>(a[t] + at) : v4i{0, 0, 0, 0};
            }
        };
        auto multiply = [&](const Frag& f) {
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int t = 0; t < kRT; ++t) acc[t] = mfma16x16<kIn>(f.a[s][t], f.x[s], acc[t]);
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
        for (int t = 0; t < kRT; ++t) *reinterpret_cast<v4f*>(&red[wave][i][16 * t + 4 * g]) = acc[t];
        __syncthreads();
        for (int e = tid; e < 256 * kRT; e += kLoraThreads) {
            const int row = e / (16 * kRT), q = e % (16 * kRT);
            const int who = __shfl(id[0], row);
            if (who != cur || r0 + q >= l.r) continue;
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < kLoraWaves; ++w) s += red[w][row][q];
            l.ws[((int64_t)part * l.M + m0 + row) * l.r + r0 + q] = s;
        }
    });
}

// What a chunk past the end of K is loaded from.
__device__ const uint4 kZeros = {0, 0, 0, 0};

// Many rows.  A workgroup: 32 WR rows by 16 WC ranks, a wave 32 by 16 of them; one part of K in stages
// of 64 values (128 bytes a row, a cache line) through four LDS slots, three stages' loads out at a
// time.  What bounds it is x, read once (and again for each further adapter of a tile's rows).
template <int WR, int WC>
struct DownShape {
    static_assert(WR * WC == kLoraWaves, "waves");
    static constexpr int BM = 32 * WR, BN = 16 * WC, NS = 4, kStage = (BM + BN) * 128, kLds = NS * kStage;
    // 1 KiB loads per wave and stage: of x's rows, of A's (WC = 1: two loads, by two waves each)
    static constexpr int NLA = WR, NLB = WC > 1 ? WC / 2 : 1, NL = NLA + NLB;
};

template <int kIn, int WR, int WC>
__global__ __launch_bounds__(kLoraThreads) void k_lora_down(LoraAdd l, int parts)
{
    using S = DownShape<WR, WC>;
    constexpr int kI = (S::BM + 63) / 64;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const int tid = threadIdx.x, lane = tid & 63, i = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), wr = wave / WC, wc = wave % WC;
    const int64_t m0 = (int64_t)blockIdx.x * S::BM;
    const int part = (int)blockIdx.y % parts, r0 = (int)blockIdx.y / parts * S::BN;
    const int chunks = l.K / 8, per = ((chunks + parts - 1) / parts + 7) / 8 * 8;    // 16-byte chunks a part
    const int c0 = part * per, c1 = (part + 1) * per < chunks ? (part + 1) * per : chunks, n = c1 > c0 ? (c1 - c0 + 7) / 8 : 0;
    const uint32_t lds0 = lds_addr(lds);
    int id[kI], mine[2];                                  // of the tile's rows; of this lane's two
#pragma unroll
    for (int k = 0; k < kI; ++k) id[k] = lane + 64 * k < S::BM ? adapter_of(l, m0 + lane + 64 * k) : -1;
#pragma unroll
    for (int q = 0; q < 2; ++q) mine[q] = adapter_of(l, m0 + 32 * wr + 16 * q + i);
    // a load's lane: row lane / 8 of 8, the chunk that belongs into slot lane % 8 of its row
    const uint8_t* x[S::NLA];
    int cx[S::NLA], ca[S::NLB];
#pragma unroll
    for (int k = 0; k < S::NLA; ++k) {
        const int q = (wave * S::NLA + k) * 8 + (lane >> 3);
        cx[k] = c0 + ((lane & 7) ^ swz(q));
        x[k] = l.x + (m0 + q < l.M ? m0 + q : l.M - 1) * l.x_stride + (int64_t)cx[k] * 16;
    }
    auto load_of = [&](int k) { return WC > 1 ? wave * S::NLB + k : wave & 1; };
    each_adapter(id, 0, 1, [&](int cur) {
        const uint8_t* a[S::NLB];
#pragma unroll
        for (int k = 0; k < S::NLB; ++k) {
            const int q = load_of(k) * 8 + (lane >> 3);
            ca[k] = c0 + ((lane & 7) ^ swz(q));
            a[k] = l.a + ((int64_t)cur * l.r + (r0 + q < l.r ? r0 + q : l.r - 1)) * l.K * 2 + (int64_t)ca[k] * 16;
        }
        auto issue = [&](int s) {
            const uint32_t to = lds0 + (s & 3) * S::kStage;
            static_assert(S::NS == 4, "slots");
#pragma unroll
            for (int k = 0; k < S::NLA; ++k)
                g2lds16(cx[k] + 8 * s < c1 ? x[k] + s * 128 : reinterpret_cast<const uint8_t*>(&kZeros), to + (wave * S::NLA + k) * 1024);
#pragma unroll
            for (int k = 0; k < S::NLB; ++k)
                g2lds16(ca[k] + 8 * s < c1 ? a[k] + s * 128 : reinterpret_cast<const uint8_t*>(&kZeros), to + S::BM * 128 + load_of(k) * 1024);
        };
        v4f acc[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
        __syncthreads();                                  // the last adapter's stages are read
#pragma unroll
        for (int s = 0; s < S::NS - 1; ++s)
            if (s < n) issue(s);
        for (int s = 0; s < n; ++s) {
            if (s + S::NS - 1 <= n)                       // the loads of the NS - 2 stages behind it may be out
                asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"((S::NS - 2) * S::NL) : "memory");
            else
                asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
            if (s + S::NS - 1 < n) issue(s + S::NS - 1);  // into the slot that every wave has read
            const uint8_t* at = lds + (s & 3) * S::kStage;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int c = ((2 * g + h) ^ swz(i)) << 4;
                const v4i va = *reinterpret_cast<const v4i*>(at + (S::BM + 16 * wc + i) * 128 + c);
#pragma unroll
                for (int q = 0; q < 2; ++q)
                    acc[q] = mfma16x16<kIn>(va, *reinterpret_cast<const v4i*>(at + (32 * wr + 16 * q + i) * 128 + c), acc[q]);
            }
        }
        const int q0 = r0 + 16 * wc + 4 * g;
#pragma unroll
        for (int q = 0; q < 2; ++q)
            if (mine[q] == cur && q0 < l.r)
                *reinterpret_cast<v4f*>(l.ws + ((int64_t)part * l.M + m0 + 32 * wr + 16 * q + i) * l.r + q0) = acc[q];
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

// Eight consecutive values of a row: from two 16-byte vectors (16-bit types: the first); the n there
// are one by one; and to memory, `wide` in aligned 16-byte vectors.
__device__ __forceinline__ void unpack8(const uint4 (&raw)[2], int type, float (&v)[8])
{
    const uint32_t w[8] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w, raw[1].x, raw[1].y, raw[1].z, raw[1].w};
    if (type == kF32) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(w[e]);
    } else if (type == kBF16) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(e & 1 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = (float)__builtin_bit_cast(_Float16, (uint16_t)(w[e / 2] >> (16 * (e & 1))));
    }
}
__device__ __forceinline__ void load_row8(const void* p, int64_t at, int type, int n, float (&v)[8])
{
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

// A workgroup: 16 kR rows by cols columns (a multiple of 128), its waves 32 columns at a time as two
// products of 16 columns.  Product t has columns 8 (i / 4) + 4 t + i % 4 of the 32, so that lane group g gets 8
// consecutive ones, 8 g on, of its row from the two.  The loads of B and base for the next 32 columns are out
// under the products (kKS > 4: registers are too few), those for the first under the sum of the parts, which
// the workgroup makes once, in LDS.
template <int kIn, int kP, int kKS, int kR>
__global__ __launch_bounds__(kLoraThreads) void k_lora_up(LoraAdd l, int parts, int cols, int wide)
{
    constexpr int kRanks = 32 * kKS;
    __shared__ float sum[16 * kR][kRanks + 4];
    const int tid = threadIdx.x, lane = tid & 63, i = lane & 15, g = lane >> 4, wave = tid >> 6;
    const int64_t m0 = (int64_t)blockIdx.x * (16 * kR);
    const int first = (int)blockIdx.y * cols + wave * 32, end = ((int)blockIdx.y + 1) * cols < l.N ? ((int)blockIdx.y + 1) * cols : l.N;
    constexpr int kStep = 32 * kLoraWaves;
    const int id[1] = {lane < 16 * kR ? adapter_of(l, m0 + lane) : -1};
    int ids[kR];
#pragma unroll
    for (int q = 0; q < kR; ++q) ids[q] = __shfl(id[0], 16 * q + i);
    const int base_size = dtype_bytes(l.base_type);
    struct Cols {                                         // 32 columns' operands
        v4i b[2][kKS];
        uint4 base[kR][2];                                // this lane's 8 of a row, 16 or 32 bytes
    };
    // eight columns from n on of this lane's row of row tile q
    auto finish = [&](int q, int n, float factor, float scale, const float (&z)[8], const uint4 (&raw)[2]) {
        const int64_t m = m0 + 16 * q + i;
        if (n >= l.N) return;
        float v[8] = {};
        if (l.base) {
            if (wide)
                unpack8(raw, l.base_type, v);
            else
                load_row8(l.base, m * l.base_stride + n, l.base_type, l.N - n, v);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += z[e] * factor * scale;
        store_row8(l.out, m * l.out_stride + n, l.out_type, wide, l.N - n, v);
    };
    auto load_base = [&](int cur, int n0, uint4 (&raw)[kR][2]) {
        if (!l.base || !wide || n0 + 8 * g >= l.N) return;
#pragma unroll
        for (int q = 0; q < kR; ++q) {
            const int64_t m = m0 + 16 * q + i;
            if (ids[q] != cur || m >= l.M) continue;
            const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(l.base) + (m * l.base_stride + n0 + 8 * g) * base_size);
            raw[q][0] = p[0];
            if (base_size == 4) raw[q][1] = p[1];
        }
    };
    each_adapter(id, blockIdx.z, gridDim.z, [&](int cur) {
        auto load = [&](Cols& c, int n0) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int col = n0 + 8 * (i >> 2) + 4 * t + (i & 3), n = col < l.N ? col : l.N - 1;
                const uint8_t* b = l.b + ((int64_t)cur * l.N + n) * l.r * 2 + 16 * g;
#pragma unroll
                for (int k = 0; k < kKS; ++k) c.b[t][k] = 32 * k + 8 * g < l.r ? *reinterpret_cast<const v4i*>(b + 64 * k) : v4i{0, 0, 0, 0};
            }
            load_base(cur, n0, c.base);
        };
        Cols c0, c1;
        if (first < end) load(c0, first);
        __syncthreads();                                  // the last adapter's sums are read
        for (int e = tid * 4; e < 16 * kR * kRanks; e += 4 * kLoraThreads) {
            const int row = e / kRanks, q = e % kRanks, who = __shfl(id[0], row);
            v4f s = {0, 0, 0, 0};
            if (q < l.r && who == cur) {
                const float* w = l.ws + (m0 + row) * l.r + q;
                const int64_t step = l.M * l.r;
                int part = 0;
                for (; part + 4 <= parts; part += 4, w += 4 * step) {
                    const v4f w0 = *reinterpret_cast<const v4f*>(w), w1 = *reinterpret_cast<const v4f*>(w + step),
                              w2 = *reinterpret_cast<const v4f*>(w + 2 * step), w3 = *reinterpret_cast<const v4f*>(w + 3 * step);
                    s += w0;
                    s += w1;
                    s += w2;
                    s += w3;
                }
                for (; part < parts; ++part, w += step) s += *reinterpret_cast<const v4f*>(w);
            }
            *reinterpret_cast<v4f*>(&sum[row][q]) = s;
        }
        __syncthreads();
        Parts<kIn, kP, kKS> p[kR];
#pragma unroll
        for (int q = 0; q < kR; ++q) {
            float s[kKS][8];
#pragma unroll
            for (int k = 0; k < kKS; ++k)
#pragma unroll
                for (int e = 0; e < 8; e += 4) {
                    const v4f v = *reinterpret_cast<const v4f*>(&sum[16 * q + i][32 * k + 8 * g + e]);
#pragma unroll
                    for (int z = 0; z < 4; ++z) s[k][e + z] = v[z];
                }
            p[q] = split<kIn, kP, kKS>(s);
        }
        const float scale = l.scales ? l.scales[cur] : 1.0f;
        auto compute = [&](const Cols& c, int n0) {
            v4f acc[kR][2];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
#pragma unroll
                for (int q = 0; q < kR; ++q) acc[q][t] = v4f{0, 0, 0, 0};
#pragma unroll
                for (int k = 0; k < kKS; ++k)
#pragma unroll
                    for (int z = kP - 1; z >= 0; --z)
#pragma unroll
                        for (int q = 0; q < kR; ++q) acc[q][t] = mfma16x16<kIn>(c.b[t][k], p[q].v[k][z], acc[q][t]);
            }
#pragma unroll
            for (int q = 0; q < kR; ++q) {
                if (ids[q] != cur) continue;
                const float z[8] = {acc[q][0][0], acc[q][0][1], acc[q][0][2], acc[q][0][3], acc[q][1][0], acc[q][1][1], acc[q][1][2], acc[q][1][3]};
                finish(q, n0 + 8 * g, p[q].back, scale, z, c.base[q]);
            }
        };
        for (int n0 = first; n0 < end; n0 += 2 * kStep) {
            if constexpr (kKS <= 4) {
                if (n0 + kStep < end) load(c1, n0 + kStep);
                compute(c0, n0);
                if (n0 + kStep >= end) break;
                if (n0 + 2 * kStep < end) load(c0, n0 + 2 * kStep);
                compute(c1, n0 + kStep);
            } else {
                compute(c0, n0);
                if (n0 + kStep >= end) break;
                load(c0, n0 + kStep);
                compute(c0, n0 + kStep);
                if (n0 + 2 * kStep < end) load(c0, n0 + 2 * kStep);
            }
        }
    });
    if (blockIdx.z != 0 || l.out == l.base) return;       // in place: rows of no adapter stay as they are
    const float none[8] = {};
    for (int n0 = first; n0 < end; n0 += kStep) {
        uint4 raw[kR][2];
        load_base(-1, n0, raw);
#pragma unroll
        for (int q = 0; q < kR; ++q)
            if (ids[q] < 0 && m0 + 16 * q + i < l.M) finish(q, n0 + 8 * g, 0.0f, 0.0f, none, raw[q]);
    }
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
    const int rows = lora_few(l.M) ? 16 : 32;
    const unsigned tiles = nblk(l.M, rows);
    const int64_t blocks = nblk(l.N, 32 * kLoraWaves), want = (1024 + tiles - 1) / tiles;
    const int cols = (int)((blocks + want - 1) / want) * 32 * kLoraWaves;
    const dim3 grid(tiles, nblk(l.N, cols), ways);
    if (rows == 16)
        hipLaunchKernelGGL((k_lora_up<kIn, kP, kKS, 1>), grid, dim3(kLoraThreads), 0, st, l, parts, cols, wide);
    else
        hipLaunchKernelGGL((k_lora_up<kIn, kP, kKS, 2>), grid, dim3(kLoraThreads), 0, st, l, parts, cols, wide);
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

template <int kIn, int WR, int WC>
hipError_t launch_down(const LoraAdd& l, int parts, int ways, hipStream_t st)
{
    using S = DownShape<WR, WC>;
    const unsigned y = (unsigned)parts * nblk(l.r, S::BN);
    if (lora_few(l.M)) {
        hipLaunchKernelGGL((k_lora_down_few<kIn, WC>), dim3(nblk(l.M, 16), y, ways), dim3(kLoraThreads), 0, st, l, parts);
        return hipSuccess;
    }
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&k_lora_down<kIn, WR, WC>), hipFuncAttributeMaxDynamicSharedMemorySize, S::kLds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((k_lora_down<kIn, WR, WC>), dim3(nblk(l.M, S::BM), y), dim3(kLoraThreads), S::kLds, st, l, parts);
    return hipSuccess;
}

template <int kIn>
hipError_t launch_typed(const LoraAdd& l, hipStream_t st)
{
    const int parts = lora_parts(l.M, l.K, l.r);
    // rows of a small batch mostly have an adapter each: its tiles' adapters go to workgroups of their own
    const int ways = l.M <= 512 ? (l.M < 16 ? (int)l.M : 16) : lora_few(l.M) ? 4 : 1;
    const hipError_t e = lora_ranks(l.r) == 16 ? launch_down<kIn, 4, 1>(l, parts, ways, st) : lora_ranks(l.r) == 32 ? launch_down<kIn, 2, 2>(l, parts, ways, st)
                                                                                                                    : launch_down<kIn, 1, 4>(l, parts, ways, st);
    if (e != hipSuccess) return e;
    bool three = false;
    if constexpr (kIn == kBF16) {
        three = l.out_type == kF32;
        if (three) launch_up<kIn, 3>(l, parts, ways, st);
    }
    if (!three) launch_up<kIn, 2>(l, parts, ways, st);
    return hipGetLastError();
}

}  // namespace

// ----------------------------------------------------------------- launches ---
hipError_t launch_lora_add(const LoraAdd& l, hipStream_t st)
{
    if (l.M == 0) return hipSuccess;
    return l.in_type == kBF16 ? launch_typed<kBF16>(l, st) : launch_typed<kF16>(l, st);
}

}  // namespace moe
