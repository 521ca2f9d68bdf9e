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

#include <type_traits>

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
// per lane and adds the scaled products into fp32.  Its first operand is the weights, the
// second the activations, so a lane holds four consecutive output columns of one row in
// consecutive result registers.
//
// Which K-block a lane's 32 codes are is free as long as both operands agree: lane half h
// takes block 4 h + s in step s of a 256-code stage (8 blocks a row), so that its four
// scale bytes are one word.
//
// A block past the end of K is read from the last block (in bounds, any finite codes) with
// scale byte 0 on both sides: 2^-254 of a product below 2^11 is 0 in fp32.
//
// Groups of a row table: tile slot s belongs to the last group g whose first slot
// bounds[g] / BM + g is <= s (a group of c rows never needs more than the
// bounds[g + 1] / BM + 1 - bounds[g] / BM slots up to the next group's first), so a
// workgroup finds its rows from the bounds alone, without a list of tiles.
typedef int v4i __attribute__((ext_vector_type(4)));

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
    // 64 groups are compared at a time, one per lane: two rounds of loads up to 4096 groups
    int g = 0, span = a.G;
    const int lane = threadIdx.x & 63;
    while (span > 1) {
        const int step = (span + 63) >> 6, at = g + lane * step;
        const bool le = lane * step < span && (int64_t)(a.bounds[at] / BM) + at <= slot;
        const int n = __popcll(__ballot(le));             // a run of lanes from 0 for sound bounds
        const int skip = (n > 0 ? n - 1 : 0) * step;
        g += skip;
        span = span - skip < step ? span - skip : step;
    }
    g = __builtin_amdgcn_readfirstlane(g);
    const int64_t b0 = a.bounds[g], b1 = a.bounds[g + 1];
    int64_t m0 = b0 + (slot - (b0 / BM + g)) * BM, m1 = m0 + BM < b1 ? m0 + BM : b1;
    // sound bounds ascend within [0, M]; this only keeps others from reaching outside
    if (m0 < b0 || m0 < 0) m0 = m1;
    if (m1 > a.M) m1 = a.M;
    return {g, m0, m1};
}

// A row of the product reads this row of A.
__device__ __forceinline__ int64_t a_row(const MxGemm& a, int64_t r)
{
    int src = a.rows ? a.rows[r] : (int)r;                // r < 2^31
    if (a.row_div > 1) src /= a.row_div;
    return src < 0 ? 0 : (src >= a.a_rows ? a.a_rows - 1 : src);
}

// step: which byte of the two registers holds the scale (the instruction's own selector)
template <int step>
__device__ __forceinline__ v16f mfma_fp4(v4i w, v4i x, v16f c, int sw, int sx)
{
    const v8i w8 = __builtin_shufflevector(w, w, 0, 1, 2, 3, -1, -1, -1, -1);
    const v8i x8 = __builtin_shufflevector(x, x, 0, 1, 2, 3, -1, -1, -1, -1);
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w8, x8, c, 4, 4, step, sw, step, sx);   // 4: E2M1
}

__device__ __forceinline__ float silu_mul(float g, float u) { return g / (1.0f + exp_cw(-g)) * u; }

// ------------------------------------------------------------- tiled kernel ---
// Direct global->LDS loads, lane i's bytes at wave_base + size * i; inline asm so that the
// compiler does not drain them (the ring waits for them itself).
__device__ __forceinline__ uint32_t lds_addr(const void* p)
{
    return __builtin_amdgcn_readfirstlane(
        (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p);
}
__device__ __forceinline__ void g2lds16(const void* g, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %1\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(g), "s"(lds) : "memory", "m0");
}
__device__ __forceinline__ void g2lds4(const void* g, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %1\n\tglobal_load_lds_dword %0, off" ::"v"(g), "s"(lds) : "memory", "m0");
}

// Chunk c (16 bytes, one block) of a 128-byte row r sits in slot c ^ swz(r): any 8
// consecutive rows touch 8 distinct 16-byte bank groups of 128 bytes, any 16 rows 16
// distinct ones of 256.
__device__ __forceinline__ int swz(int r) { return (r ^ ((r >> 3) & 1)) & 7; }

// WM x WN waves, each TM x TN tiles of 32 x 32: BM rows of A by BN rows of B, K in stages of
// 256 codes (128 bytes a row) through two LDS slots.
//
// A row's 128 bytes are one cache line: 64-byte rows (128-code stages) and scales loaded a
// word per row asked the L2 for 20 M lines at 8192 x 4096 x 4096, more than its channels
// serve in the products' time (97 us).
template <int WM_, int WN_, int TM_, int TN_>
struct MxShape {
    static constexpr int WM = WM_, WN = WN_, TM = TM_, TN = TN_;
    static constexpr int NW = WM * WN, BM = 32 * WM * TM, BN = 32 * WN * TN, kRows = BM + BN;
    static constexpr int NL = kRows / 8 / NW;             // 1 KiB data loads per wave and stage
    static_assert(NL * NW * 8 == kRows, "whole loads");
};

// How the scale bytes come in, by the alignment of the rows of both scale matrices: 16 bytes
// a row every second stage; two words a row and stage; three words a row and stage around
// bytes at any address.
enum ScaleMode { kScale16, kScale4, kScale1 };

template <class S, int kMode>
struct MxLds {
    static constexpr int kRowBytes = kMode == kScale16 ? 16 : kMode == kScale4 ? 8 : 12;
    static constexpr int kPerLoad = kMode == kScale16 ? 1024 : 256;         // bytes of a wave's scale load
    static constexpr int NS = (S::kRows * kRowBytes + kPerLoad * S::NW - 1) / (kPerLoad * S::NW);
    static constexpr int kDataBytes = S::kRows * 128;
    static constexpr int kScaleBytes = NS * S::NW * kPerLoad;
    static constexpr int kScaleOff = 2 * kDataBytes;
    static constexpr int kBytes = 2 * kDataBytes + 2 * kScaleBytes;
};

template <class S, int kT, bool kSwiglu, int kMode>
__global__ __launch_bounds__(64 * S::NW) void k_mx_tile(MxGemm a, int n_tiles, int64_t n_slots)
{
    using L = MxLds<S, kMode>;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5, j = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / S::WN, wn = wave % S::WN;

    // Workgroups go round-robin over the 8 XCDs: XCD x takes a contiguous run of tiles, and
    // inside a run bands of 8 slots by all column tiles, so that what an XCD runs at once
    // shares rows of A and of B in its L2.
    Tile t;
    int nt;
    {
        const int64_t total = n_slots * n_tiles, per = (total + 7) >> 3;
        const int64_t id = (int64_t)(blockIdx.x & 7) * per + (blockIdx.x >> 3);
        if ((blockIdx.x >> 3) >= per || id >= total) return;
        const uint32_t band = (uint32_t)id / (uint32_t)(8 * n_tiles), first = band * 8;   // total < 2^31
        const uint32_t high = n_slots - first < 8 ? (uint32_t)(n_slots - first) : 8;
        const uint32_t in = (uint32_t)id - first * n_tiles;
        nt = (int)(in / high);
        t = tile_of_slot<S::BM>(a, first + in % high);
    }
    if (t.m0 >= t.m1) return;                             // uniform
    const int nb = a.K / 32, nst = (nb + 7) >> 3;
    const int NB = kSwiglu ? 2 * a.N : a.N;
    constexpr int kOutCols = kSwiglu ? S::BN / 2 : S::BN;
    const int n0 = nt * kOutCols;

    // row q of the stage: rows of A, then rows of B (SwiGLU: 32 gate rows and their 32 up rows in turn)
    auto src_row = [&](int q, bool& is_a) -> int64_t {
        is_a = q < S::BM;
        if (is_a) {
            const int64_t r = t.m0 + q < t.m1 ? t.m0 + q : t.m1 - 1;
            return a_row(a, r);
        }
        q -= S::BM;
        int n = kSwiglu ? n0 + (q >> 6) * 32 + (q & 31) : n0 + q;
        n = n < a.N ? n : a.N - 1;
        if (kSwiglu && (q & 32)) n += a.N;
        return (int64_t)t.g * NB + n;
    };

    const uint8_t* dsrc[S::NL];                           // this lane's row, per load
    const int dchunk = lane & 7;                          // ... and slot in it
    int dswz[S::NL];
#pragma unroll
    for (int l = 0; l < S::NL; ++l) {
        const int q = (wave * S::NL + l) * 8 + (lane >> 3);
        bool is_a;
        const int64_t r = src_row(q, is_a);
        dswz[l] = dchunk ^ swz(q);
        dsrc[l] = (is_a ? a.a_codes : a.b_codes) + r * (a.K / 2);
        if (kMode == kScale16) dsrc[l] += dswz[l] * 16;   // K is a multiple of 512: no clamp below
    }
    const uint8_t* ssrc[L::NS];                           // where this lane's scale loads start
    const uint8_t* slast[L::NS];                          // kScale1: the last aligned word that holds one of the row's bytes
#pragma unroll
    for (int l = 0; l < L::NS; ++l) {
        int i = (wave * L::NS + l) * 64 + lane;
        constexpr int kParts = kMode == kScale16 ? 1 : L::kRowBytes / 4;
        i = i < S::kRows * kParts ? i : 0;
        const int q = i / kParts, part = i % kParts;
        bool is_a;
        const int64_t r = src_row(q, is_a);
        const uint8_t* p = (is_a ? a.a_scales : a.b_scales) + r * nb;
        if constexpr (kMode == kScale1) {
            // a word that holds a valid byte lies in that byte's page
            slast[l] = reinterpret_cast<const uint8_t*>(reinterpret_cast<uintptr_t>(p + nb - 1) & ~(uintptr_t)3);
            p = reinterpret_cast<const uint8_t*>(reinterpret_cast<uintptr_t>(p) & ~(uintptr_t)3);
        } else {
            slast[l] = p + nb - 4;
        }
        ssrc[l] = p + 4 * part;
    }
    constexpr int kOps = S::TM + S::TN, kProd = S::TM * S::TN;
    const int sa_base = wm * S::TM * 32 + j, sb_base = S::BM + wn * S::TN * 32 + j;
    auto op_row = [&](int i) { return i < S::TM ? sa_base + i * 32 : sb_base + (i - S::TM) * 32; };
    int mis[kOps];                                        // kScale1: where the row's first byte is in its word
    if constexpr (kMode == kScale1) {
#pragma unroll
        for (int i = 0; i < kOps; ++i) {
            bool is_a;
            const int64_t r = src_row(op_row(i), is_a);
            mis[i] = (int)(reinterpret_cast<uintptr_t>((is_a ? a.a_scales : a.b_scales) + r * nb) & 3);
        }
    }

    const uint32_t lds0 = lds_addr(lds);
    // data load l of stage s (clamped: a load past the last stage repeats it) into slot s % 2
    auto issue_data = [&](int l, int s) {
        const uint32_t to = lds0 + (s & 1) * L::kDataBytes + (wave * S::NL + l) * 1024;
        const int sc = s < nst ? s : nst - 1;
        if constexpr (kMode == kScale16) {
            g2lds16(dsrc[l] + sc * 128, to);
        } else {
            const int c = sc * 8 + dswz[l];
            g2lds16(dsrc[l] + (c < nb ? c : nb - 1) * 16, to);
        }
    };
    // scale load l of stage s (kScale16: of the stages s, s + 1 for an even s, buffer s / 2 % 2)
    auto issue_scales = [&](int l, int s) {
        const int sc = s < nst ? s : (kMode == kScale16 ? (nst - 1) & ~1 : nst - 1);
        const int buf = kMode == kScale16 ? (s >> 1) & 1 : s & 1;
        const uint32_t to = lds0 + L::kScaleOff + buf * L::kScaleBytes + (wave * L::NS + l) * L::kPerLoad;
        const uint8_t* p = ssrc[l] + sc * 8;
        if constexpr (kMode == kScale16) {
            g2lds16(p, to);
        } else {
            g2lds4(p < slast[l] ? p : slast[l], to);
        }
    };

    // Operands of one step: tiles of the activations, then of the weights.  Tile rows are 32
    // apart, so the swizzle is that of row j.
    struct Ops {
        v4i v[kOps];
    };
    struct Scales {
        int v[kOps];
    };
    auto read_op = [&](int i, int s, int step, Ops& o) {
        o.v[i] = *reinterpret_cast<const v4i*>(lds + (s & 1) * L::kDataBytes + op_row(i) * 128 +
                                               (((4 * h + step) ^ swz(j)) << 4));
    };
    // the scale bytes of this lane half's four blocks of stage s: 0 past the end of K
    auto read_scale = [&](int i, int s, Scales& o) {
        const uint8_t* base = lds + L::kScaleOff;
        if constexpr (kMode == kScale16) {
            o.v[i] = *reinterpret_cast<const int*>(base + ((s >> 1) & 1) * L::kScaleBytes + op_row(i) * 16 + (s & 1) * 8 + 4 * h);
        } else if constexpr (kMode == kScale4) {
            const int v = *reinterpret_cast<const int*>(base + (s & 1) * L::kScaleBytes + op_row(i) * 8 + 4 * h);
            o.v[i] = 8 * s + 4 * h < nb ? v : 0;
        } else {
            const uint32_t* p = reinterpret_cast<const uint32_t*>(base + (s & 1) * L::kScaleBytes + op_row(i) * 12 + 4 * h);
            const uint32_t v = __builtin_amdgcn_alignbyte(p[1], p[0], mis[i]);
            const int left = nb - (8 * s + 4 * h);
            o.v[i] = (int)(left >= 4 ? v : left <= 0 ? 0u : v & ((1u << (8 * left)) - 1u));
        }
    };

    v16f acc[S::TM][S::TN];
#pragma unroll
    for (int i = 0; i < S::TM; ++i)
#pragma unroll
        for (int n = 0; n < S::TN; ++n)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][n][e] = 0.0f;

    // Stage s, four steps of kProd products.  Steps 0 and 1 read the operands of steps 1 to 3;
    // then every wave has read its share of slot s % 2, and the barrier frees it for stage
    // s + 2 and admits stage s + 1 (its loads, the only ones out, have had a stage's time).
    // Step 2 issues the loads of stage s + 2, step 3 reads step 0 of stage s + 1.  Each memory
    // instruction is placed behind a product of its own, in whose 32 cycles it issues.
    auto products = [&](auto step_c, const Ops& o, const Scales& sc, auto between) {
#pragma unroll
        for (int i = 0; i < S::TM; ++i)
#pragma unroll
            for (int n = 0; n < S::TN; ++n) {
                acc[i][n] = mfma_fp4<decltype(step_c)::value>(o.v[S::TM + n], o.v[i], acc[i][n], sc.v[S::TM + n], sc.v[i]);
                between(i * S::TN + n);
                __builtin_amdgcn_sched_barrier(0);
            }
    };
    Ops o0, o1, o2, o3;
    Scales sc0, sc1;
    auto stage = [&](int s) {
        products(std::integral_constant<int, 0>{}, o0, sc0, [&](int at) {
#pragma unroll
            for (int i = at * 2 * kOps / kProd; i < (at + 1) * 2 * kOps / kProd; ++i) {
                if (i < kOps)
                    read_op(i, s, 1, o1);
                else
                    read_op(i - kOps, s, 2, o2);
            }
        });
        products(std::integral_constant<int, 1>{}, o1, sc0, [&](int at) {
#pragma unroll
            for (int i = at * kOps / kProd; i < (at + 1) * kOps / kProd; ++i) read_op(i, s, 3, o3);
        });
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
        products(std::integral_constant<int, 2>{}, o2, sc0, [&](int at) {
            if (kMode != kScale16 || (s & 1) == 0) {
#pragma unroll
                for (int l = at * L::NS / kProd; l < (at + 1) * L::NS / kProd; ++l) issue_scales(l, s + 2);
            }
#pragma unroll
            for (int l = at * S::NL / kProd; l < (at + 1) * S::NL / kProd; ++l) issue_data(l, s + 2);
        });
        products(std::integral_constant<int, 3>{}, o3, sc0, [&](int at) {
            // past the last stage: a repeated one, not used
#pragma unroll
            for (int i = at * kOps / kProd; i < (at + 1) * kOps / kProd; ++i) {
                read_op(i, s + 1, 0, o0);
                read_scale(i, s + 1, sc1);
            }
        });
    };
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        if (kMode != kScale16 || u == 0) {
#pragma unroll
            for (int l = 0; l < L::NS; ++l) issue_scales(l, u);
        }
#pragma unroll
        for (int l = 0; l < S::NL; ++l) issue_data(l, u);
    }
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(S::NL + (kMode == kScale16 ? 0 : L::NS)) : "memory");
#pragma unroll
    for (int i = 0; i < kOps; ++i) {
        read_op(i, 0, 0, o0);
        read_scale(i, 0, sc0);
    }
    for (int s = 0; s < nst; ++s) {
        stage(s);
        sc0 = sc1;
    }
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");   // the slots are dead: the epilogue takes them

    // Epilogue: each wave turns its tile, 32 rows at a time, through LDS of its own into
    // row-major order and writes 16 bytes a lane, whole runs of a row at a time.
    typedef typename Elem<kT>::type T;
    constexpr int kCols = (kSwiglu ? S::TN / 2 : S::TN) * 32;
    constexpr int kStride = kCols * (int)sizeof(T) + 16;
    constexpr int kVec = 16 / (int)sizeof(T), kLanes = kCols / kVec;   // lanes a row
    static_assert(32 * kStride * S::NW <= L::kBytes, "the waves' turning space fits the ring");
    static_assert(64 % kLanes == 0, "whole rows a pass");
    uint8_t* mine = lds + wave * 32 * kStride;
    const int c0 = n0 + wn * kCols;
    const bool vec = (reinterpret_cast<uintptr_t>(a.out) | (uint64_t)(a.out_stride * (int64_t)sizeof(T))) % 16 == 0;
#pragma unroll
    for (int i = 0; i < S::TM; ++i) {
#pragma unroll
        for (int n = 0; n < (kSwiglu ? S::TN / 2 : S::TN); ++n)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if constexpr (kSwiglu)
                        v[e] = silu_mul(acc[i][2 * n][4 * g + e], acc[i][2 * n + 1][4 * g + e]);
                    else
                        v[e] = acc[i][n][4 * g + e];
                }
                store_n<kT, 4>(mine + j * kStride + (n * 32 + 8 * g + 4 * h) * sizeof(T), v);
            }
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int p = 0; p < 32 * kLanes / 64; ++p) {
            const int row = p * (64 / kLanes) + lane / kLanes, col = (lane % kLanes) * kVec;
            const int64_t r = t.m0 + (wm * S::TM + i) * 32 + row;
            const uint8_t* from = mine + row * kStride + col * sizeof(T);
            if (r < t.m1 && c0 + col < a.N) {
                T* o = static_cast<T*>(a.out) + r * a.out_stride + c0 + col;
                if (vec && c0 + col + kVec <= a.N) {
                    *reinterpret_cast<uint4*>(o) = *reinterpret_cast<const uint4*>(from);
                } else {
                    const T* f = reinterpret_cast<const T*>(from);
                    for (int e = 0; e < kVec && c0 + col + e < a.N; ++e) o[e] = f[e];
                }
            }
        }
        __builtin_amdgcn_wave_barrier();
    }
}

// ----------------------------------------------------------- few-row kernel ---
// Up to 32 rows of a group by 32 columns (SwiGLU: 32 gate and 32 up rows of B) per
// workgroup; its waves take every eighth run of 256 codes of K, fed straight from memory,
// and add up through LDS in wave order.  What bounds it is B's bytes, read once: lane half
// h takes blocks 4 h + s of a run, 64 consecutive bytes of a row in four loads.
constexpr int kFewWaves = 8;

template <int kT, bool kSwiglu, bool kAligned>
__global__ __launch_bounds__(64 * kFewWaves) void k_mx_few(MxGemm a)
{
    constexpr int NT = kSwiglu ? 2 : 1;
    __shared__ float red[kFewWaves][NT][32][33];
    const Tile t = tile_of_slot<32>(a, blockIdx.x);
    if (t.m0 >= t.m1) return;                             // uniform
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, h = lane >> 5, j = lane & 31;
    const int nb = a.K / 32, NB = kSwiglu ? 2 * a.N : a.N;
    const int n0 = (int)blockIdx.y * 32;
    const int64_t ar = a_row(a, t.m0 + j < t.m1 ? t.m0 + j : t.m1 - 1);
    const int bn = n0 + j < a.N ? n0 + j : a.N - 1;
    const uint8_t* xc = a.a_codes + ar * (a.K / 2);
    const uint8_t* xs = a.a_scales + ar * nb;
    const uint8_t* wc[NT];
    const uint8_t* ws[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const int64_t r = (int64_t)t.g * NB + bn + i * a.N;
        wc[i] = a.b_codes + r * (a.K / 2);
        ws[i] = a.b_scales + r * nb;
    }
    v16f acc[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][e] = 0.0f;
    // four scale bytes from block b on: 0 past the end
    auto scales4 = [&](const uint8_t* p, int b) -> uint32_t {
        if (kAligned) return b < nb ? *reinterpret_cast<const uint32_t*>(p + b) : 0u;
        uint32_t v = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (b + i < nb) v |= (uint32_t)p[b + i] << (8 * i);
        return v;
    };
    const int runs = (nb + 7) >> 3;
#pragma unroll 2
    for (int u = wave; u < runs; u += kFewWaves) {
        const int b = u * 8 + 4 * h;
        v4i x[4], w[NT][4];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int c = b + s < nb ? b + s : nb - 1;
#pragma unroll
            for (int i = 0; i < NT; ++i) w[i][s] = *reinterpret_cast<const v4i*>(wc[i] + c * 16);
            x[s] = *reinterpret_cast<const v4i*>(xc + c * 16);
        }
        uint32_t sw[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) sw[i] = scales4(ws[i], b);
        const uint32_t sx = scales4(xs, b);
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int i = 0; i < NT; ++i)
                acc[i] = mfma_fp4<0>(w[i][s], x[s], acc[i], (int)(sw[i] >> (8 * s)), (int)(sx >> (8 * s)));
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
            for (int w = 0; w < kFewWaves; ++w) z[i] += red[w][i][row][col];
        static_cast<T*>(a.out)[(t.m0 + row) * a.out_stride + n0 + col] =
            from_f32<kT>(kSwiglu ? silu_mul(z[0], z[NT - 1]) : z[0]);
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

namespace {

using Tile256 = MxShape<2, 2, 4, 4>;      // 256 x 256
using Tile128 = MxShape<2, 2, 2, 2>;      // 128 x 128
using Tile64 = MxShape<2, 2, 1, 2>;       // 64 x 128

// Slots of BM rows: see tile_of_slot.
int64_t slots_of(const MxGemm& g, int BM) { return g.bounds ? g.M / BM + g.G : (g.M + BM - 1) / BM; }

template <class S, int kT, bool kSwiglu, int kMode>
hipError_t launch_tile(const MxGemm& g, hipStream_t st)
{
    constexpr int lds = MxLds<S, kMode>::kBytes;
    const int n_tiles = (int)nblk(g.N, kSwiglu ? S::BN / 2 : S::BN);
    const int64_t slots = slots_of(g, S::BM), total = slots * n_tiles;
    if (total > INT32_MAX - 8) return hipErrorInvalidValue;
    // more than the default limit of dynamic LDS
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&k_mx_tile<S, kT, kSwiglu, kMode>),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((k_mx_tile<S, kT, kSwiglu, kMode>), dim3(8 * nblk(total, 8)), dim3(64 * S::NW), lds, st, g,
                       n_tiles, slots);
    return hipGetLastError();
}

template <int kT, bool kSwiglu, int kMode>
hipError_t launch_shape(const MxGemm& g, hipStream_t st)
{
    const int64_t rows = g.M / g.G;       // rows a group has on average
    auto tiles = [&](int BM, int BN) { return (g.bounds ? g.M / BM + 1 : (g.M + BM - 1) / BM) * nblk(g.N, kSwiglu ? BN / 2 : BN); };
    if (rows <= 32) {
        hipLaunchKernelGGL((k_mx_few<kT, kSwiglu, kMode != kScale1>), dim3((unsigned)slots_of(g, 32), nblk(g.N, 32)),
                           dim3(64 * kFewWaves), 0, st, g);
        return hipGetLastError();
    }
    if (rows >= 192 && tiles(256, 256) >= 192) return launch_tile<Tile256, kT, kSwiglu, kMode>(g, st);
    if (rows >= 48 && tiles(128, 128) >= 192) return launch_tile<Tile128, kT, kSwiglu, kMode>(g, st);
    return launch_tile<Tile64, kT, kSwiglu, kMode>(g, st);
}

template <int kT, bool kSwiglu>
hipError_t launch_mode(const MxGemm& g, hipStream_t st)
{
    const uint64_t at = reinterpret_cast<uintptr_t>(g.a_scales) | reinterpret_cast<uintptr_t>(g.b_scales) | (uint64_t)(g.K / 32);
    if (at % 16 == 0) return launch_shape<kT, kSwiglu, kScale16>(g, st);
    if (at % 4 == 0) return launch_shape<kT, kSwiglu, kScale4>(g, st);
    return launch_shape<kT, kSwiglu, kScale1>(g, st);
}

template <int kT>
hipError_t launch_typed(const MxGemm& g, hipStream_t st)
{
    return g.swiglu ? launch_mode<kT, true>(g, st) : launch_mode<kT, false>(g, st);
}

}  // namespace

hipError_t launch_mx_gemm(const MxGemm& g, hipStream_t st)
{
    if (g.M == 0) return hipSuccess;
    if (g.dtype == kF32) return launch_typed<kF32>(g, st);
    if (g.dtype == kBF16) return launch_typed<kBF16>(g, st);
    return launch_typed<kF16>(g, st);
}

}  // namespace moe
