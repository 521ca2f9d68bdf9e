// HIP kernels (CDNA4 / gfx950) of the low-rank adapters of many requests beside a shared
// projection:
//   out[t] = base[t] + scale_i (x[t] A_i^T) B_i^T,  i = adapters[t] (none: out[t] = base[t]).
//
// Two launches: s = x A_i^T in fp32, K in parts; then the parts' sum times B_i^T onto base.  One for a few rows,
// see launch_typed.  Rows are taken in tiles, once for each adapter that the tile's rows name: runs of rows of
// one adapter (prompts) cost least, and tiles of a few rows share the adapters out to workgroups.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "moe_dtype.h"
#include "moe_lora.h"
#include "moe_mfma16.h"
#include "moe_tile.h"

namespace moe {

namespace {

constexpr int kLoraWaves = 4, kLoraThreads = 64 * kLoraWaves;
constexpr int kOneWaves = 8;              // of the launch that makes s itself

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

// Many rows.  A workgroup: 32 WR rows by 16 WC TC ranks, a wave 32 by 16 TC of them; one part of K in
// stages of 64 values (128 bytes a row, a cache line) through four LDS slots, three stages' loads out at a
// time.  What bounds it is x, read once (and again for each further adapter of a tile's rows), and A, read
// from the L2 for each tile: 8192 rows of rank 64, K = 4096 30 us in tiles of 32 rows, 27 in tiles of 64.
template <int WR, int WC, int TC>
struct DownShape {
    static_assert(WR * WC == kLoraWaves, "waves");
    static constexpr int BM = 32 * WR, BN = 16 * WC * TC, NS = 4, kStage = (BM + BN) * 128, kLds = NS * kStage;
    // 1 KiB loads per wave and stage: of x's rows, of A's (16 ranks: two loads, by two waves each)
    static constexpr int NLA = WR, NLB = BN > 16 ? BN / 32 : 1, NL = NLA + NLB;
};

template <int kIn, int WR, int WC, int TC>
__global__ __launch_bounds__(kLoraThreads) void k_lora_down(LoraAdd l, int parts)
{
    using S = DownShape<WR, WC, TC>;
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
    auto load_of = [&](int k) { return S::BN > 16 ? wave * S::NLB + k : wave & 1; };
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
        v4f acc[TC][2];
#pragma unroll
        for (int t = 0; t < TC; ++t) acc[t][0] = acc[t][1] = v4f{0, 0, 0, 0};
        __syncthreads();                                  // the last adapter's stages are read
#pragma unroll
        for (int s = 0; s < S::NS - 1; ++s)
            if (s < n) issue(s);
        for (int s = 0; s < n; ++s) {
            // this wave's reads of the stage before are done, by its own wait and not by where the compiler put one
            if (s + S::NS - 1 <= n)                       // the loads of the NS - 2 stages behind it may be out
                asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((S::NS - 2) * S::NL) : "memory");
            else
                asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
            if (s + S::NS - 1 < n) issue(s + S::NS - 1);  // into the slot that every wave has read
            const uint8_t* at = lds + (s & 3) * S::kStage;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int c = ((2 * g + h) ^ swz(i)) << 4;
                v4i vx[2];
#pragma unroll
                for (int q = 0; q < 2; ++q) vx[q] = *reinterpret_cast<const v4i*>(at + (32 * wr + 16 * q + i) * 128 + c);
#pragma unroll
                for (int t = 0; t < TC; ++t) {
                    const v4i va = *reinterpret_cast<const v4i*>(at + (S::BM + 16 * (TC * wc + t) + i) * 128 + c);
#pragma unroll
                    for (int q = 0; q < 2; ++q) acc[t][q] = mfma16x16<kIn>(va, vx[q], acc[t][q]);
                }
            }
        }
#pragma unroll
        for (int t = 0; t < TC; ++t) {
            const int q0 = r0 + 16 * (TC * wc + t) + 4 * g;
#pragma unroll
            for (int q = 0; q < 2; ++q)
                if (mine[q] == cur && q0 < l.r)
                    *reinterpret_cast<v4f*>(l.ws + ((int64_t)part * l.M + m0 + 32 * wr + 16 * q + i) * l.r + q0) = acc[t][q];
        }
    });
}

// ------------------------------------------------------- out = base + s B^T ---
// s enters the matrix instruction as a sum of 16-bit parts, so that little of its 24 bits is lost: bf16
// two parts, each the nearest to what the parts before it left (2^-16 of s lost at most), for fp32
// results three (2^-24).  fp16: the row of s times the power of two that brings its largest value to
// [2^14, 2^15), as two parts, the second, what the first left, times 2^12 and its products' sum times 2^-12: 2^-22 of a
// value lost, or 2^-16 where the output has 16 bits anyway, if the value is within `width` (29, or 35) powers of two of the
// largest.  A smaller one is multiplied by 2^width until it is, and belongs to the window of that number, whose product
// product_long makes apart (of normally distributed values some 2^-28, or 2^-34).  Sums of products of fp16 numbers span 100 powers of
// two, which four windows hold.
constexpr int fp16_width(bool out32) { return out32 ? 29 : 35; }
constexpr float kSecond = 0x1p12f;                        // fp16: what the second part is multiplied by

template <int kIn, int kP, int kKS>
struct Parts {
    v4i v[kKS][kP];
    float back;               // what the results are multiplied by
    uint32_t windows = 1;     // a bit for each that holds something in the wave (fp16), and the first
    uint32_t window[kKS];     // 4 bits a value
    int width;
};

template <int kIn, int kP, int kKS>
__device__ __forceinline__ Parts<kIn, kP, kKS> split(float (&s)[kKS][8], int width)
{
    Parts<kIn, kP, kKS> p;
    p.back = 1.0f;
    p.width = width;
#pragma unroll
    for (int k = 0; k < kKS; ++k) p.window[k] = 0;
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
        const float to = __uint_as_float((uint32_t)(127 + 14 - e) << 23), least = __uint_as_float((uint32_t)(127 + 15 - width) << 23);
        p.back = __uint_as_float((uint32_t)(127 - 14 + e) << 23);
        bool small = false;
#pragma unroll
        for (int k = 0; k < kKS; ++k)
#pragma unroll
            for (int z = 0; z < 8; ++z) {
                s[k][z] *= to;
                small |= __builtin_fabsf(s[k][z]) < least && s[k][z] != 0.0f;
            }
        if (__ballot(small)) {
            uint32_t mine = 1;
#pragma unroll
            for (int k = 0; k < kKS; ++k)
#pragma unroll
                for (int z = 0; z < 8; ++z) {
                    const int down = 14 + 127 - (int)(__float_as_uint(s[k][z]) >> 23 & 255);      // below 0: infinity, NaN
                    const int w = s[k][z] == 0.0f || down < width ? 0 : min(down / width, 112 / width);
                    s[k][z] *= __uint_as_float((uint32_t)(127 + width * w) << 23);
                    p.window[k] |= (uint32_t)w << (4 * z);
                    mine |= 1u << w;
                    asm volatile("" : "+v"(s[k][z]), "+v"(mine));    // one value after the other, not all in registers at once
                }
            p.windows = 0;
#pragma unroll 1
            for (int w = 0; w < 4; ++w) p.windows |= __ballot(mine >> w & 1) ? 1u << w : 0u;
        }
    }
#pragma unroll
    for (int k = 0; k < kKS; ++k) {
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            float rest[2] = {s[k][e], s[k][e + 1]};
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
                    rest[z] = __builtin_fabsf(at[z]) < __builtin_inff() ? (rest[z] - at[z]) * (kIn == kF16 ? kSecond : 1.0f) : 0.0f;
            }
        }
    }
    return p;
}

// acc = B s of kT tiles, the smaller parts first: of each step of ranks (bf16), or of all ranks (fp16).
template <int kIn, int kP, int kKS, int kT>
__device__ __forceinline__ void product(const v4i (*b)[kKS], const Parts<kIn, kP, kKS>& p, v4f* acc)
{
#pragma unroll
    for (int t = 0; t < kT; ++t) acc[t] = v4f{0, 0, 0, 0};
    if constexpr (kIn == kBF16) {
#pragma unroll
        for (int k = 0; k < kKS; ++k)
#pragma unroll
            for (int z = kP - 1; z >= 0; --z)
#pragma unroll
                for (int t = 0; t < kT; ++t) acc[t] = mfma16x16<kIn>(b[t][k], p.v[k][z], acc[t]);
    } else {
        static_assert(kP == 2, "parts of fp16");
#pragma unroll
        for (int z = 1; z >= 0; --z) {
#pragma unroll
            for (int k = 0; k < kKS; ++k)
#pragma unroll
                for (int t = 0; t < kT; ++t) acc[t] = mfma16x16<kIn>(b[t][k], p.v[k][z], acc[t]);
#pragma unroll
            for (int t = 0; t < (z ? kT : 0); ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[t][e] *= 1.0f / kSecond;
        }
    }
}

// The same product the long way, taken where a sum of the short way is not finite or s has several windows: each window's
// product by itself, the smallest first.  Where B holds infinities or NaN the sum of parts would make NaN (hi inf + lo inf,
// lo being 0 or of the other sign), so: sign(s) times those, 0 in place of B's numbers, plus the parts times B with a 1 of the
// same sign in their place.  What the ones add is finite, and lost beside an infinity.  read(k): b[k]; odd: B may hold some.
template <int kIn, int kP, int kKS, class F>
__device__ __forceinline__ v4f product_long(const Parts<kIn, kP, kKS>& p, bool odd, F read)
{
    constexpr uint32_t two = 0x10001u, inf = kIn == kBF16 ? 0x7f80u : 0x7c00u, one = (kIn == kBF16 ? 0x3f80u : 0x3c00u) * two;
    // all bits of a half where its magnitude and `add` reach 2^15
    auto reach = [](uint32_t w, uint32_t add) {
        const uint32_t m = (((w & 0x7fff7fffu) + add * 0x10001u) >> 15) & 0x10001u;
        return (m << 16) - m;
    };
    // what is made of a value is made here, not ahead of the loops in registers of its own
    auto here = [](uint32_t w) {
        asm volatile("" : "+v"(w));
        return w;
    };
    v4f z = {0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < kKS; ++k) {
        if (!odd) break;                                  // uniform
        const v4i b = read(k);
        v4i alone, sign;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const uint32_t w = here((uint32_t)b[q]), s = here((uint32_t)p.v[k][0][q]);
            alone[q] = (int)(w & reach(w, 0x8000u - inf));
            sign[q] = (int)((reach(s, 0x7fffu) & ((s & 0x80008000u) | one)) | (reach(s, 0x7fffu - inf) & 0x7fff7fffu));
        }
        z = mfma16x16<kIn>(alone, sign, z);
        __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll 1
    for (uint32_t left = p.windows; left;) {
        const int win = 31 - __builtin_clz(left);
        left &= ~(1u << win);
        v4f sum[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};        // of fp16's second parts, of the rest
#pragma unroll
        for (int k = 0; k < kKS; ++k) {
            asm volatile("" ::: "memory");                // b[k] is read here, for each window again
            const v4i b = read(k);
            v4i rest, part[kP];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint32_t w = here((uint32_t)b[q]), m = reach(w, 0x8000u - inf);
                rest[q] = (int)((w & ~m) | (m & ((w & 0x80008000u) | one)));
                uint32_t in = ~0u;
                if constexpr (kIn == kF16) {
                    const uint32_t of = here(p.window[k]) >> (8 * q);
                    in = ((of & 15) == (uint32_t)win ? 0xffffu : 0u) | ((of >> 4 & 15) == (uint32_t)win ? 0xffff0000u : 0u);
                }
#pragma unroll
                for (int y = 0; y < kP; ++y) part[y][q] = (int)((uint32_t)p.v[k][y][q] & in);
            }
#pragma unroll
            for (int y = kP - 1; y >= 0; --y) sum[kIn == kBF16 || !y] = mfma16x16<kIn>(rest, part[y], sum[kIn == kBF16 || !y]);
            __builtin_amdgcn_sched_barrier(0);
        }
        const float back = __uint_as_float((uint32_t)(127 - p.width * win) << 23);
#pragma unroll
        for (int e = 0; e < 4; ++e) z[e] = __builtin_fmaf(__builtin_fmaf(sum[0][e], 1.0f / kSecond, sum[1][e]), back, z[e]);
    }
    return z;
}
// The larger of `most` and z's magnitudes; NaN stays.
__device__ __forceinline__ float most_of(float most, const v4f& z)
{
#pragma unroll
    for (int e = 0; e < 4; ++e) most = __builtin_elementwise_maximum(most, __builtin_fabsf(z[e]));
    return most;
}

// n consecutive values, n * size <= 16 bytes, of a vector of that type; and to aligned memory.
template <int n>
__device__ __forceinline__ void unpack(const uint4& raw, int type, float (&v)[n])
{
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    if (type == kF32) {
        if constexpr (n == 4) {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = __uint_as_float(w[e]);
        }
    } else if (type == kBF16) {
#pragma unroll
        for (int e = 0; e < n; ++e) v[e] = __uint_as_float(e & 1 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
    } else {
#pragma unroll
        for (int e = 0; e < n; ++e) v[e] = (float)__builtin_bit_cast(_Float16, (uint16_t)(w[e / 2] >> (16 * (e & 1))));
    }
}
template <int n>
__device__ __forceinline__ void store_row(void* p, int64_t at, int type, const float (&v)[n])
{
    if (type == kF32) {
        if constexpr (n == 4) store_n<kF32, 4>(static_cast<float*>(p) + at, v);
    } else if (type == kBF16) {
        store_n<kBF16, n>(static_cast<__bf16*>(p) + at, v);
    } else {
        store_n<kF16, n>(static_cast<_Float16*>(p) + at, v);
    }
}
__device__ __forceinline__ float load1(const void* p, int64_t at, int type)
{
    return type == kF32 ? static_cast<const float*>(p)[at] : type == kBF16 ? (float)static_cast<const __bf16*>(p)[at]
                                                                           : (float)static_cast<const _Float16*>(p)[at];
}
__device__ __forceinline__ void store1(void* p, int64_t at, int type, float v)
{
    if (type == kF32)
        static_cast<float*>(p)[at] = v;
    else if (type == kBF16)
        static_cast<__bf16*>(p)[at] = (__bf16)v;
    else
        static_cast<_Float16*>(p)[at] = (_Float16)v;
}

// Few rows, or rows that are not aligned vectors.  A workgroup: 16 rows by cols columns, its waves 64 columns at a
// time, as products of 16.  s is summed once, in LDS: of the parts (kRT = 0), or it is made here from all of K, in
// kRT tiles of 16 ranks -- one launch and each workgroup reads A again, for a few rows (8.9 us against 11.1 of one
// row, rank 16, 4096 x 4096).  A wave's results go through LDS, so that base and out are read and written a whole
// line at a time: kV values a lane (8: both of x's type; 4: one is fp32; 1: rows that are not aligned vectors).
// Waves a SIMD that the registers leave, where the compiler would go a little past them: 48 rows of rank 64, fp16, 19 us with
// three and 23 with two; 1000 rows of rank 256 onto fp32 98 with two and 118 with one.
constexpr int up_few_waves(int in, int KS, int V, int RT) { return in != kF16 || RT ? 1 : KS == 8 ? 2 : V == 8 ? 3 : 1; }

template <int kIn, int kP, int kKS, int kV, int kRT, int kWaves>
__global__ __launch_bounds__(64 * kWaves, up_few_waves(kIn, kKS, kV, kRT)) void k_lora_up_few(LoraAdd l, int parts, int cols)
{
    constexpr int kRanks = 32 * kKS, kRows = 16;
    constexpr int kB = kKS <= 2 ? 4 : kKS == 4 ? 2 : 1;   // products of 16 columns whose B is in registers at once
    __shared__ float sum[kRows][kRanks + 4];
    __shared__ float tile[kWaves][kRows][68];
    const int tid = threadIdx.x, lane = tid & 63, i = lane & 15, g = lane >> 4, wave = tid >> 6;
    const int64_t m0 = (int64_t)blockIdx.x * kRows;
    const int first = (int)blockIdx.y * cols + wave * 64, end = ((int)blockIdx.y + 1) * cols < l.N ? ((int)blockIdx.y + 1) * cols : l.N;
    constexpr int kStep = 64 * kWaves;
    const int id[1] = {lane < kRows ? adapter_of(l, m0 + lane) : -1};
    const bool there = lane < kRows && m0 + lane < l.M;
    // of 16-bit types there is x's, where the rows are vectors: no branch between a block's loads
    const int base_type = kV == 8 ? kIn : kV == 4 && l.base_type != kF32 ? kIn : l.base_type;
    const int out_type = kV == 8 ? kIn : kV == 4 && l.out_type != kF32 ? kIn : l.out_type;
    const int base_size = dtype_bytes(base_type);
    // out = base + z (null: 0) of the rows in `rows` in columns n0 .. n0 + 63: lane's columns from `col` on, of every
    // kPer-th row
    constexpr int kLanes = 64 / kV, kPer = kV, kIt = kV > 1 ? kRows / kPer : 1;
    const int col = kV * (lane % kLanes), row0 = lane / kLanes;
    struct Base {
        uint4 v[kIt];
    };
    auto load_base = [&](uint64_t rows, int n0, Base& raw) {
        if constexpr (kV > 1) {
            if (!l.base || n0 + col >= l.N) return;
#pragma unroll
            for (int t = 0; t < kIt; ++t) {
                const int row = kPer * t + row0;
                if (!(rows >> row & 1)) continue;
                const uint8_t* p = static_cast<const uint8_t*>(l.base) + ((m0 + row) * l.base_stride + n0 + col) * base_size;
                if (kV * base_size == 16) {
                    raw.v[t] = *reinterpret_cast<const uint4*>(p);
                } else {
                    const uint2 half = *reinterpret_cast<const uint2*>(p);
                    raw.v[t].x = half.x;
                    raw.v[t].y = half.y;
                }
            }
        }
    };
    auto finish = [&](uint64_t rows, int n0, const Base& raw, const float (*z)[68]) {
        if constexpr (kV > 1) {
            if (n0 + col >= l.N) return;
#pragma unroll
            for (int t = 0; t < kIt; ++t) {
                const int row = kPer * t + row0;
                if (!(rows >> row & 1)) continue;
                float v[kV] = {};
                if (l.base) unpack<kV>(raw.v[t], base_type, v);
                if (z) {
#pragma unroll
                    for (int e = 0; e < kV; e += 4) {
                        const v4f add = *reinterpret_cast<const v4f*>(&z[row][col + e]);
#pragma unroll
                        for (int x = 0; x < 4; ++x) v[e + x] += add[x];
                    }
                }
                store_row<kV>(l.out, (m0 + row) * l.out_stride + n0 + col, out_type, v);
            }
        } else {
            const int n = n0 + lane;
            if (n >= l.N) return;
            for (int t = 0; t < kRows; t += 8) {
                if (!(rows >> t & 255)) continue;         // uniform
                float v[8] = {};
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (l.base && (rows >> (t + e) & 1)) v[e] = load1(l.base, (m0 + t + e) * l.base_stride + n, l.base_type);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (rows >> (t + e) & 1) store1(l.out, (m0 + t + e) * l.out_stride + n, l.out_type, v[e] + (z ? z[t + e][lane] : 0.0f));
            }
        }
    };
    each_adapter(id, blockIdx.z, gridDim.z, [&](int cur) {
        const uint64_t rows = __ballot(id[0] == cur);
        v4i b[kB][kKS];
        auto b_at = [&](int n0) {                         // of a product's columns from n0 on
            return l.b + ((int64_t)cur * l.N + (n0 + i < l.N ? n0 + i : l.N - 1)) * l.r * 2 + 16 * g;
        };
        auto load_one = [&](const uint8_t* p, int k) { return 32 * k + 8 * g < l.r ? *reinterpret_cast<const v4i*>(p + 64 * k) : v4i{0, 0, 0, 0}; };
        auto load_b = [&](int n0) {                       // of kB products
#pragma unroll
            for (int t = 0; t < kB; ++t) {
                const uint8_t* p = b_at(n0 + 16 * t);
#pragma unroll
                for (int k = 0; k < kKS; ++k) b[t][k] = load_one(p, k);
            }
        };
        Base raw;
        if (first < end) {
            load_b(first);
            load_base(rows, first, raw);
        }
        const float scale = l.scales ? l.scales[cur] : 1.0f;
        if constexpr (kRT > 0) {
            // the waves share K 64 values at a time: two of them a buffer, lane group g has chunks u + 2 g, + 1
            const int chunks = l.K / 8;
            constexpr int kUnit = 8 * kWaves;
            const uint8_t* x = l.x + (m0 + i < l.M ? m0 + i : l.M - 1) * l.x_stride + 32 * g;
            const uint8_t* a[kRT];
            v4f acc[kRT];
#pragma unroll
            for (int t = 0; t < kRT; ++t) {
                a[t] = l.a + ((int64_t)cur * l.r + (16 * t + i < l.r ? 16 * t + i : l.r - 1)) * l.K * 2 + 32 * g;
                acc[t] = v4f{0, 0, 0, 0};
            }
            struct Frag {
                v4i x[4], a[4][kRT];
            };
            auto load = [&](Frag& f, int u0) {
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const int u = u0 + (s >> 1) * kUnit;
                    const bool in = u + 8 <= chunks || u + 2 * g + (s & 1) < chunks;
                    const int64_t at = (int64_t)(u + (s & 1)) * 16;
                    f.x[s] = in ? *reinterpret_cast<const v4i*>(x + at) : v4i{0, 0, 0, 0};
#pragma unroll
                    for (int t = 0; t < kRT; ++t) f.a[s][t] = in ? *reinterpret_cast<const v4i*>(a[t] + at) : v4i{0, 0, 0, 0};
                }
            };
            auto multiply = [&](const Frag& f) {
#pragma unroll
                for (int s = 0; s < 4; ++s)
#pragma unroll
                    for (int t = 0; t < kRT; ++t) acc[t] = mfma16x16<kIn>(f.a[s][t], f.x[s], acc[t]);
            };
            Frag f0, f1;
            const int u0 = wave * 8;
            if (u0 < chunks) load(f0, u0);
            if (u0 + 2 * kUnit < chunks) load(f1, u0 + 2 * kUnit);
            for (int u = u0; u < chunks; u += 4 * kUnit) {
                multiply(f0);
                if (u + 4 * kUnit < chunks) load(f0, u + 4 * kUnit);
                if (u + 2 * kUnit >= chunks) break;
                multiply(f1);
                if (u + 6 * kUnit < chunks) load(f1, u + 6 * kUnit);
            }
            __syncthreads();                              // the last adapter's results are out of the tiles
            constexpr int kLine = 16 * kRT + 4;
            float* red = &tile[0][0][0];                  // [waves][16][kLine]
            static_assert(kLine <= 68, "inside the tiles");
#pragma unroll
            for (int t = 0; t < kRT; ++t) *reinterpret_cast<v4f*>(red + (wave * 16 + i) * kLine + 16 * t + 4 * g) = acc[t];
            __syncthreads();
            for (int e = tid; e < kRows * kRanks; e += 64 * kWaves) {
                const int row = e / kRanks, q = e % kRanks;
                float s = 0.0f;
                if (q < l.r && (rows >> row & 1))
#pragma unroll
                    for (int w = 0; w < kWaves; ++w) s += red[(w * 16 + row) * kLine + q];
                sum[row][q] = s;
            }
            __syncthreads();
        } else {
            __syncthreads();                              // the last adapter's sums are read
            for (int e = tid * 4; e < kRows * kRanks; e += 4 * 64 * kWaves) {
                const int row = e / kRanks, q = e % kRanks;
                v4f s = {0, 0, 0, 0};
                if (q < l.r && (rows >> row & 1)) {
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
        }
        float s[kKS][8];
#pragma unroll
        for (int k = 0; k < kKS; ++k)
#pragma unroll
            for (int e = 0; e < 8; e += 4) {
                const v4f v = *reinterpret_cast<const v4f*>(&sum[i][32 * k + 8 * g + e]);
#pragma unroll
                for (int z = 0; z < 4; ++z) s[k][e + z] = v[z];
            }
        const Parts<kIn, kP, kKS> p = split<kIn, kP, kKS>(s, fp16_width(l.out_type == kF32));
        auto put = [&](int t, const v4f& z) {
            v4f v;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = z[e] * p.back * scale;
            *reinterpret_cast<v4f*>(&tile[wave][i][16 * t + 4 * g]) = v;
        };
        for (int n0 = first; n0 < end; n0 += kStep) {
            float most = 0.0f;
#pragma unroll
            for (int t0 = 0; t0 < 4; t0 += kB) {
                v4f acc[kB];
#pragma unroll
                for (int t = 0; t < kB; ++t) {
                    product<kIn, kP, kKS, 1>(&b[t], p, &acc[t]);
                }
                if (t0 + kB < 4)
                    load_b(n0 + 16 * (t0 + kB));
                else if (n0 + kStep < end)
                    load_b(n0 + kStep);
#pragma unroll
                for (int t = 0; t < kB; ++t) {
                    put(t0 + t, acc[t]);
                    most = most_of(most, acc[t]);
                }
            }
            const bool odd = __ballot(!(most < __builtin_inff())) != 0;
            if (odd || p.windows > 1) {                   // seldom: B is read again
#pragma unroll 1
                for (int t = 0; t < 4; ++t) {
                    const uint8_t* from = b_at(n0 + 16 * t);
                    put(t, product_long(p, odd, [&](int k) { return load_one(from, k); }));
                }
            }
            // within a wave LDS works in order; the compiler must not move across
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            finish(rows, n0, raw, tile[wave]);
            if (n0 + kStep < end) load_base(rows, n0 + kStep, raw);
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        }
    });
    if (blockIdx.z != 0 || l.out == l.base) return;       // in place: rows of no adapter stay as they are
    const uint64_t none = __ballot(there && id[0] < 0);
    if (!none) return;
    for (int n0 = first; n0 < end; n0 += kStep) {
        Base raw;
        load_base(none, n0, raw);
        finish(none, n0, raw, nullptr);
    }
}

// Many rows.  A workgroup: 64 rows, 16 of each of four waves, by cols columns (a multiple of 64), 64 at a time as a
// stage in LDS: B's rows and base.  Four more waves issue the stages' loads, NS - 1 ahead, straight into LDS, and alone
// wait for them (one wave for all loads took 20 to 80% longer); the others' stores, which come back in order with a wave's loads, hold nothing up.  A wave adds its
// products to base, and writes 16 rows a line at a time through LDS.  8192 rows of rank 64 and 4096 columns, 128 MB of
// base and out: 42 to 48 us, 2.8 TB/s, where a copy in the same pattern takes 27; what bounds it is a stage's chain
// (barrier, LDS, products, LDS, stores), of which two workgroups a CU overlap two.  (Four waves that loaded for
// themselves: 69 us with stores from the result registers, 59 a line at a time.)
constexpr int kUpRows = 64, kUpCols = 64, kUpLoaders = 4, kUpThreads = kLoraThreads + 64 * kUpLoaders;

template <int kKS>
struct UpShape {
    static constexpr int kRow = 64 * kKS, kB = kUpCols * kRow;               // bytes of a row of B (r padded), of a stage's
    static constexpr int kChunks = 4 * kKS;
    // which chunk of 16 bytes is in slot c of row n: 16 rows' same chunk lies in 16 distinct bank groups of 256 bytes
    static __device__ __forceinline__ int swap(int n) { return (kKS == 1 ? n >> 2 : kKS == 2 ? n >> 1 : n) & (kChunks < 16 ? kChunks - 1 : 15); }
};
constexpr int up_slots(int KS, int base_size) { return KS == 8 && base_size == 4 ? 2 : KS == 8 || (KS == 4 && base_size == 4) ? 3 : 4; }
// rows of the waves' results, padded against bank conflicts
constexpr int up_out_row(int out_size) { return kUpCols * out_size + 16; }
constexpr int up_lds(int KS, int base_size, int out_size)
{
    return up_slots(KS, base_size) * kUpCols * (64 * KS + kUpRows * base_size) + kUpRows * up_out_row(out_size);
}

// kBase, kOut: bytes of an element of base (0: there is none) and of out; those of 2 bytes are of x's type, known
// here so that nothing branches between a stage's loads from LDS (2.1 us a stage where it did, of one wave a SIMD)
template <int kIn, int kP, int kKS, int kBase, int kOut>
__global__ __launch_bounds__(kUpThreads) void k_lora_up(LoraAdd l, int parts, int cols)
{
    using S = UpShape<kKS>;
    constexpr int NS = up_slots(kKS, kBase), kBaseRow = kUpCols * kBase, kStage = S::kB + kUpRows * kBaseRow;
    // 1 KiB loads a stage and loading wave
    constexpr int kLoadsB = S::kB / 1024 / kUpLoaders, kLoadsBase = kUpRows * kBaseRow / 1024 / kUpLoaders, NL = kLoadsB + kLoadsBase;
    static_assert((NS - 2) * NL <= 63, "vmcnt");
    constexpr int kBaseChunks = kBaseRow / 16, kOutRow = up_out_row(kOut);
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const int tid = threadIdx.x, lane = tid & 63, i = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t m0 = (int64_t)blockIdx.x * kUpRows;
    const int first = (int)blockIdx.y * cols, end = first + cols < l.N ? first + cols : l.N, n = (end - first + kUpCols - 1) / kUpCols;
    const int id[1] = {adapter_of(l, m0 + lane)};
    auto base_swap = [](int row) { return kBase == 2 ? (row >> 1) & 7 : row & 15; };
    each_adapter(id, 0, 1, [&](int cur) {
        const uint64_t rows = __ballot(id[0] == cur);
        if (wave >= kLoraWaves) {
            const int loader = wave - kLoraWaves;
            const uint32_t lds0 = lds_addr(lds);
            const uint8_t* b_at = l.b + ((int64_t)cur * l.N + first) * l.r * 2;
            const uint8_t* base_at = static_cast<const uint8_t*>(l.base) + (m0 * l.base_stride + first) * kBase;
            // What is not there (a column past the end, a rank past r, a row of another adapter) is read from what
            // is, and not used.  32 bits of offset: the host checked that 64 rows of base span less.
            const int one = __builtin_ctzll(rows);
            auto issue = [&](int s) {
                const uint32_t to = lds0 + s % NS * kStage;
                const int last = end - 1 - first - s * kUpCols;          // the last column's place in the stage
                const uint8_t* bs = b_at + (int64_t)s * kUpCols * l.r * 2;
#pragma unroll
                for (int q = 0; q < kLoadsB; ++q) {
                    const int k = loader * kLoadsB + q, at = k * 64 + lane, col = at / S::kChunks, c = at % S::kChunks ^ S::swap(col);
                    g2lds16_at(bs, (uint32_t)((col < last ? col : last) * l.r * 2 + (8 * c < l.r ? c : 0) * 16), to + k * 1024);
                }
                if constexpr (kBase) {
                    const uint8_t* from = base_at + s * kUpCols * kBase;
#pragma unroll
                    for (int q = 0; q < kLoadsBase; ++q) {
                        const int k = loader * kLoadsBase + q, at = k * 64 + lane, row = at / kBaseChunks, c = at % kBaseChunks ^ base_swap(row);
                        const uint32_t row_at = (uint32_t)((rows >> row & 1) ? row : one) * (uint32_t)(l.base_stride * kBase);
                        g2lds16_at(from, row_at + (c * (16 / kBase) <= last ? c : 0) * 16, to + S::kB + k * 1024);
                    }
                }
            };
#pragma unroll 1
            for (int s = 0; s < NS - 1 && s < n; ++s) issue(s);
#pragma unroll 1
            for (int s = 0; s < n; ++s) {
                if (s + NS - 1 <= n)                      // the loads of the NS - 2 stages behind it may be out
                    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((NS - 2) * NL) : "memory");
                else
                    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
                if (s + NS - 1 < n) issue(s + NS - 1);    // into the slot that every wave has read
            }
        } else {
            const int row = 16 * wave + i;                // of the tile
            const bool mine = rows >> row & 1;
            float sums[kKS][8];
#pragma unroll
            for (int k = 0; k < kKS; ++k) {
#pragma unroll
                for (int e = 0; e < 8; ++e) sums[k][e] = 0.0f;
                const int q = 32 * k + 8 * g;
                if (mine && q < l.r) {
                    const float* w = l.ws + (m0 + row) * l.r + q;
                    for (int part = 0; part < parts; ++part, w += l.M * l.r) {
                        const v4f lo = *reinterpret_cast<const v4f*>(w), hi = *reinterpret_cast<const v4f*>(w + 4);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            sums[k][e] += lo[e];
                            sums[k][4 + e] += hi[e];
                        }
                    }
                }
            }
            const Parts<kIn, kP, kKS> p = split<kIn, kP, kKS>(sums, fp16_width(kOut == 4));
            const float factor = (l.scales ? l.scales[cur] : 1.0f) * p.back;     // p.back: a power of two
            uint8_t* out_rows = lds + NS * kStage + 16 * wave * kOutRow;
            for (int s = 0; s < n; ++s) {
                // this wave's reads of the stage before are done; the loading waves admit this one
                asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
                const uint8_t* at = lds + s % NS * kStage;
                auto read_b = [&](int t, int k) {         // of product t's 16 columns
                    const int col = 16 * t + i;
                    const v4i b = *reinterpret_cast<const v4i*>(at + col * S::kRow + (((4 * k + g) ^ S::swap(col)) << 4));
                    return 32 * k + 8 * g < l.r ? b : v4i{0, 0, 0, 0};
                };
                // products t0 .. t0 + kT - 1 onto base, into the waves' rows
                auto columns = [&](int t0, auto n_c, auto product) {
                    constexpr int kT = decltype(n_c)::value;
                    uint4 raw[kT];
                    if constexpr (kBase) {
#pragma unroll
                        for (int t = 0; t < kT; ++t) {
                            const int byte = (16 * (t0 + t) + 4 * g) * kBase;
                            const uint8_t* from = at + S::kB + row * kBaseRow + (((byte >> 4) ^ base_swap(row)) << 4) + (byte & 15);
                            if constexpr (kBase == 4) {
                                raw[t] = *reinterpret_cast<const uint4*>(from);
                            } else {
                                const uint2 half = *reinterpret_cast<const uint2*>(from);
                                raw[t] = {half.x, half.y, 0, 0};
                            }
                        }
                    }
                    v4f acc[kT];
                    product(acc);
#pragma unroll
                    for (int t = 0; t < kT; ++t) {
                        float v[4] = {};                  // columns 16 (t0 + t) + 4 g .. + 3 of the row
                        if constexpr (kBase) unpack<4>(raw[t], kBase == 4 ? (int)kF32 : kIn, v);
#pragma unroll
                        for (int e = 0; e < 4; ++e) v[e] = __builtin_fmaf(acc[t][e], factor, v[e]);
                        store_row<4>(out_rows + i * kOutRow, 16 * (t0 + t) + 4 * g, kOut == 4 ? (int)kF32 : kIn, v);
                    }
                };
                constexpr int kT = kKS <= 2 ? 4 : 1;      // products whose operands are read together
                float most = 0.0f;
#pragma unroll
                for (int t0 = 0; t0 < 4; t0 += kT) {
                    v4i b[kT][kKS];
#pragma unroll
                    for (int t = 0; t < kT; ++t)
#pragma unroll
                        for (int k = 0; k < kKS; ++k) b[t][k] = read_b(t0 + t, k);
                    columns(t0, std::integral_constant<int, kT>{}, [&](v4f(&acc)[kT]) {
                        product<kIn, kP, kKS, kT>(b, p, acc);
#pragma unroll
                        for (int t = 0; t < kT; ++t) most = most_of(most, acc[t]);
                    });
                }
                const bool odd = __ballot(!(most < __builtin_inff())) != 0;
                if (odd || p.windows > 1) {               // seldom
#pragma unroll 1
                    for (int t = 0; t < 4; ++t)
                        columns(t, std::integral_constant<int, 1>{}, [&](v4f(&acc)[1]) { acc[0] = product_long(p, odd, [&](int k) { return read_b(t, k); }); });
                }
                // within a wave LDS works in order; the compiler must not move across
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                constexpr int kLanes = kUpCols * kOut / 16, kPer = 64 / kLanes;        // lanes a row, rows at a time
                const int out_col = first + s * kUpCols + lane % kLanes * (16 / kOut);
#pragma unroll
                for (int q = 0; q < 16; q += kPer) {
                    const int r = q + lane / kLanes;
                    const uint4 v = *reinterpret_cast<const uint4*>(out_rows + r * kOutRow + lane % kLanes * 16);
                    if (out_col < end && (rows >> (16 * wave + r) & 1))
                        *reinterpret_cast<uint4*>(static_cast<uint8_t*>(l.out) + ((m0 + 16 * wave + r) * l.out_stride + out_col) * kOut) = v;
                }
            }
        }
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");   // every wave has read the last stage
    });
    if (l.out == l.base || wave >= kLoraWaves) return;    // in place: rows of no adapter stay as they are
    const uint64_t none = __ballot(m0 + lane < l.M && id[0] < 0);
    constexpr int kV = 16 / (kOut > kBase ? kOut : kBase), kLanes = kUpCols / kV;
    for (int n0 = first; n0 < end; n0 += kUpCols) {
        const int col = n0 + kV * (lane % kLanes);
#pragma unroll
        for (int r = lane / kLanes; r < 16; r += 64 / kLanes) {
            const int64_t m = m0 + 16 * wave + r;
            if (col >= end || !(none >> (16 * wave + r) & 1)) continue;
            float v[kV] = {};
            if constexpr (kBase == 4)
                load_n<kF32, kV>(static_cast<const float*>(l.base) + m * l.base_stride + col, v);
            else if constexpr (kBase == 2)
                load_n<kIn, kV>(static_cast<const typename Elem<kIn>::type*>(l.base) + m * l.base_stride + col, v);
            store_row<kV>(l.out, m * l.out_stride + col, kOut == 4 ? (int)kF32 : kIn, v);
        }
    }
}

template <int kIn, int kP, int kKS, int kBase, int kOut>
hipError_t launch_up_ring(const LoraAdd& l, int parts, hipStream_t st)
{
    constexpr int lds = up_lds(kKS, kBase, kOut);
    static_assert(lds <= 163840, "a CU's LDS");
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&k_lora_up<kIn, kP, kKS, kBase, kOut>),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
    // as many columns a workgroup as leave the chip full
    const unsigned tiles = nblk(l.M, kUpRows);
    const int64_t blocks = nblk(l.N, kUpCols), want = (256 * (163840 / lds) + tiles - 1) / tiles;
    const int cols = (int)((blocks + want - 1) / want) * kUpCols;
    hipLaunchKernelGGL((k_lora_up<kIn, kP, kKS, kBase, kOut>), dim3(tiles, nblk(l.N, cols)), dim3(kUpThreads), lds, st, l, parts, cols);
    return hipSuccess;
}

// whole vectors of 8 columns at aligned addresses
bool wide_rows(const LoraAdd& l)
{
    auto even = [&](const void* p, int64_t stride, int type) {
        return (reinterpret_cast<uintptr_t>(p) | (uint64_t)(stride * dtype_bytes(type))) % 16 == 0;
    };
    return l.N % 8 == 0 && even(l.out, l.out_stride, l.out_type) && (!l.base || even(l.base, l.base_stride, l.base_type));
}
// values a lane of k_lora_up_few
int few_vector(const LoraAdd& l)
{
    const int base = l.base ? dtype_bytes(l.base_type) : 0, out = dtype_bytes(l.out_type);
    return !wide_rows(l) || (out == 2 && l.out_type != l.in_type) || (base == 2 && l.base_type != l.in_type) ? 1 : base == 4 || out == 4 ? 4 : 8;
}

template <int kIn, int kP, int kKS>
hipError_t launch_up_ranks(const LoraAdd& l, int parts, int ways, hipStream_t st)
{
    const bool wide = wide_rows(l);
    const int base = l.base ? dtype_bytes(l.base_type) : 0, out = dtype_bytes(l.out_type);
    const bool types = (out == 4 || l.out_type == kIn) && (base != 2 || l.base_type == kIn);
    if (!lora_few(l.M) && wide && types && (!l.base || l.base_stride * base <= 1 << 25)) {
        if constexpr (kIn == kF16 || kP == 3) {
            if (out == 4) return base == 0 ? launch_up_ring<kIn, kP, kKS, 0, 4>(l, parts, st) : base == 2 ? launch_up_ring<kIn, kP, kKS, 2, 4>(l, parts, st)
                                                                                                         : launch_up_ring<kIn, kP, kKS, 4, 4>(l, parts, st);
        }
        if constexpr (kP == 2)
            return base == 0 ? launch_up_ring<kIn, kP, kKS, 0, 2>(l, parts, st) : base == 2 ? launch_up_ring<kIn, kP, kKS, 2, 2>(l, parts, st)
                                                                                           : launch_up_ring<kIn, kP, kKS, 4, 2>(l, parts, st);
    }
    const int v = few_vector(l);
    const unsigned tiles = nblk(l.M, 16);
    const int64_t blocks = nblk(l.N, 64 * kLoraWaves), want = (1024 + tiles - 1) / tiles;
    int cols = (int)((blocks + want - 1) / want) * 64 * kLoraWaves, threads = kLoraThreads;
    auto launch = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3(tiles, nblk(l.N, cols), ways), dim3(threads), 0, st, l, parts, cols); };
    constexpr int k16 = kP == 3 ? 4 : 8;                  // three parts are of an fp32 out
    auto launch_v = [&](auto k1, auto k4, auto k8) { v == 1 ? launch(k1) : v == 4 ? launch(k4) : launch(k8); };
    if (parts == 0) {
        cols = threads = 64 * kOneWaves;
        if constexpr (kKS == 1) {
            if (l.r <= 16)
                launch_v(k_lora_up_few<kIn, kP, 1, 1, 1, kOneWaves>, k_lora_up_few<kIn, kP, 1, 4, 1, kOneWaves>, k_lora_up_few<kIn, kP, 1, k16, 1, kOneWaves>);
            else
                launch_v(k_lora_up_few<kIn, kP, 1, 1, 2, kOneWaves>, k_lora_up_few<kIn, kP, 1, 4, 2, kOneWaves>, k_lora_up_few<kIn, kP, 1, k16, 2, kOneWaves>);
        }
        return hipSuccess;
    }
    launch_v(k_lora_up_few<kIn, kP, kKS, 1, 0, kLoraWaves>, k_lora_up_few<kIn, kP, kKS, 4, 0, kLoraWaves>, k_lora_up_few<kIn, kP, kKS, k16, 0, kLoraWaves>);
    return hipSuccess;
}

template <int kIn, int kP>
hipError_t launch_up(const LoraAdd& l, int parts, int ways, hipStream_t st)
{
    return l.r <= 32 ? launch_up_ranks<kIn, kP, 1>(l, parts, ways, st) : l.r <= 64 ? launch_up_ranks<kIn, kP, 2>(l, parts, ways, st)
           : l.r <= 128 ? launch_up_ranks<kIn, kP, 4>(l, parts, ways, st) : launch_up_ranks<kIn, kP, 8>(l, parts, ways, st);
}

template <int kIn, int WR, int WC, int TC>
hipError_t launch_down(const LoraAdd& l, int parts, int ways, hipStream_t st)
{
    using S = DownShape<WR, WC, TC>;
    const unsigned y = (unsigned)parts * nblk(l.r, S::BN);
    if (lora_few(l.M)) {
        hipLaunchKernelGGL((k_lora_down_few<kIn, S::BN / 16>), dim3(nblk(l.M, 16), y, ways), dim3(kLoraThreads), 0, st, l, parts);
        return hipSuccess;
    }
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&k_lora_down<kIn, WR, WC, TC>), hipFuncAttributeMaxDynamicSharedMemorySize,
                                             S::kLds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((k_lora_down<kIn, WR, WC, TC>), dim3(nblk(l.M, S::BM), y), dim3(kLoraThreads), S::kLds, st, l, parts);
    return hipSuccess;
}

template <int kIn>
hipError_t launch_typed(const LoraAdd& l, hipStream_t st)
{
    // rows of a small batch mostly have an adapter each: its tiles' adapters go to workgroups of their own
    const int ways = l.M <= 512 ? (l.M < 16 ? (int)l.M : 16) : lora_few(l.M) ? 4 : 1;
    // One launch where its workgroups read A and x again for less than another launch takes (4096 x 4096, rank 16: 1 row
    // 8.9 us against 11.1 of two, 16 rows of 16 adapters 13.0, 13.7, 64 rows 24, 17; 2048 x 2048: 64 rows 10.9, 13.3); its
    // registers hold 32 ranks (of 64 31 us against 11 for one row).  Beside rows in fp32 vectors more than 16 ranks spill 10
    // to 20, and are worth one launch of short reads alone (rank 32, 1, 16 and 48 rows: K = 512 8.0, 8.5, 9.1 us against 10.7 of two,
    // 1184 8.0, 9.3, 10.9, 2048 10.6, 13.1, 14.4, 4096 14.6, 19.0, -; rank 24, 1 row, 2048 9.6).
    const int64_t reads = (l.r + (l.M < 16 ? l.M : 16)) * l.K * 2, again = (int64_t)nblk(l.M, 16) * ways * nblk(l.N, 64 * kOneWaves) * reads;
    const bool one = lora_few(l.M) && l.r <= 32 && again <= (int64_t)48 << 20 && (l.r <= 16 || few_vector(l) != 4 || reads <= 1 << 17);
    const int parts = one ? 0 : lora_parts(l.M, l.K, l.r);
    const hipError_t e = one ? hipSuccess : l.r <= 16 ? launch_down<kIn, 4, 1, 1>(l, parts, ways, st) : l.r <= 32 ? launch_down<kIn, 4, 1, 2>(l, parts, ways, st)
                                                                                                               : launch_down<kIn, 2, 2, 2>(l, parts, ways, st);
    if (e != hipSuccess) return e;
    hipError_t e2;
    if constexpr (kIn == kBF16)
        e2 = l.out_type == kF32 ? launch_up<kIn, 3>(l, parts, ways, st) : launch_up<kIn, 2>(l, parts, ways, st);
    else
        e2 = launch_up<kIn, 2>(l, parts, ways, st);
    return e2 != hipSuccess ? e2 : hipGetLastError();
}

}  // namespace

// ----------------------------------------------------------------- launches ---
hipError_t launch_lora_add(const LoraAdd& l, hipStream_t st)
{
    if (l.M == 0) return hipSuccess;
    return l.in_type == kBF16 ? launch_typed<kBF16>(l, st) : launch_typed<kF16>(l, st);
}

}  // namespace moe
