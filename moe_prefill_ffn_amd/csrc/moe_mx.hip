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
#include "moe_tile.h"

namespace moe {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v2f __attribute__((ext_vector_type(2)));

namespace {

// 2^(s - 127); s = 0 is the fp32 subnormal 2^-127, s = 255 NaN
__device__ __forceinline__ float e8m0(uint32_t s)
{
    return s == 0 ? __uint_as_float(0x00400000u) : s == 255 ? __builtin_nanf("") : __uint_as_float(s << 23);
}

// ---------------------------------------------------- quantise, dequantise ---
// Four lanes per block, eight values each; a wave takes 16 consecutive blocks.  One pass, one read
// and one write of everything, so memory bounds it: 8192 x 4096 fp32 (152 MB) 26.5 us, back
// 25.0, 5.7 and 6.1 TB/s, next to the 5.2 of a copy kernel over a gigabyte; one row 1.5 us, a launch's time.
constexpr int kQuantThreads = 256;
constexpr int kQuantBlocks = kQuantThreads / 4;           // blocks per workgroup
static_assert((kMxMostBlocks + kQuantBlocks - 1) / kQuantBlocks * kQuantThreads < (int64_t)1 << 32, "threads of a launch");

struct BlockAt {
    int64_t row;
    int b;
};
__device__ __forceinline__ BlockAt block_at(int64_t blk, int nb)
{
    const uint32_t row = (uint32_t)blk / (uint32_t)nb;    // fewer than 2^30 blocks
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
// A row of the product reads this row of A.
__device__ __forceinline__ int64_t a_row(const MxGemm& a, int64_t r)
{
    int src = a.rows ? a.rows[r] : (int)r;                // r < 2^27
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

// ------------------------------------------------------------- tiled kernel ---
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
    // 1 KiB data loads per wave and stage: of A's rows, of B's
    static constexpr int NLA = BM / 8 / NW, NLB = BN / 8 / NW, NL = NLA + NLB;
    static_assert(NLA * NW * 8 == BM && NLB * NW * 8 == BN, "whole loads");
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
    static constexpr int kRowsOff = kScaleOff + 2 * kScaleBytes;            // row indices of two tiles
    static constexpr int kListOff = kRowsOff + 2 * S::BM * 4;
    static constexpr int kBytes = kListOff + kListMost * (int)sizeof(ListedTile);
};

// Persistent workgroups: each takes every so-many-th tile of its XCD's run (workgroups go
// round-robin over the 8 XCDs), one after the other without a pause in its stages -- the last two
// stages of a tile issue the first two of the next, whose pointers are made under the products,
// and the epilogue's stores drain under them.  (A workgroup a tile spent 14 us of 43 a tile of
// 8192 x 4096 x 4096 on its start, its first loads and its stores.)
//
// What bounds it: large dense products the matrix cores -- 8192 x 4096 x 4096, bf16 out, 89 to 92 us or
// 3.0 PFLOP/s, 4.4 as K grows; the instruction alone on random codes reaches 5.6 to 6.7 on all CUs,
// where power holds the clock (10 on zeros).  Grouped ones memory -- 24576 rows in 256 groups
// (N = 4096, K = 1536, fp32 out) move 1.28 GB in 341 us, 3.8 TB/s.  Scale rows that are not 16-byte aligned cost
// more the more scales there are to an output: 8192 x 4096 x 2816 (words) takes 77 us and 2880
// (bytes at any address) 88, between 67 at K = 2560 and 83 at 3584 (16 bytes); gate and up of 128 groups of 64 rows (N = 768)
// 59 at K = 2560, 72 at 2816, 114 at 2880.
template <class S, int kT, bool kSwiglu, int kMode>
__global__ __launch_bounds__(64 * S::NW) void k_mx_tile(MxGemm a, int n_tiles, int64_t n_slots)
{
    using L = MxLds<S, kMode>;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5, j = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / S::WN, wn = wave % S::WN;
    const int nb = a.K / 32;
    // at least two stages (a stage past the end of K adds 0): a stage issues the one two further,
    // which is then in this tile or the next
    const int nst = nb > 8 ? (nb + 7) >> 3 : 2;
    const int NB = kSwiglu ? 2 * a.N : a.N;
    constexpr int kOutCols = kSwiglu ? S::BN / 2 : S::BN;
    int32_t* s_rows = reinterpret_cast<int32_t*>(lds + L::kRowsOff);
    ListedTile* s_list = reinterpret_cast<ListedTile*>(lds + L::kListOff);
    const uint32_t lds0 = lds_addr(lds);

    // Data: a base per operand and tile, an offset per lane and load (kScale16: to its chunk, else
    // to its row).  32 bits of offset: a tile's rows of B span at most BN K / 2 bytes, A's at most
    // what the host checked.
    const uint8_t* a_at;
    const uint8_t* b_at;
    uint32_t dofs[S::NL];
    const uint8_t* ssrc[L::NS];                           // where this lane's scale loads start
    const uint8_t* slast[L::NS];                          // the last word it may read there
    constexpr int kOps = S::TM + S::TN, kProd = S::TM * S::TN;
    const int sa_base = wm * S::TM * 32 + j, sb_base = S::BM + wn * S::TN * 32 + j;
    auto op_row = [&](int i) { return i < S::TM ? sa_base + i * 32 : sb_base + (i - S::TM) * 32; };
    int mis[kOps];                                        // kScale1: where an operand row's first byte is in its word

    // row q of tile t's rows of A, relative to a_at's row: from the row table (indices in
    // s_rows[buf]) relative to A, else to the tile's first
    const bool by_table = a.rows != nullptr || a.row_div > 1;
    auto a_ofs = [&](const ListedTile& t, int buf, int q) -> uint32_t {
        const int last = t.m1 - 1 - t.m0, at = q < last ? q : last;
        if (!by_table) return (uint32_t)at;
        int r = a.rows ? s_rows[buf * S::BM + at] : t.m0 + at;
        if (a.row_div > 1) r /= a.row_div;
        return (uint32_t)(r < 0 ? 0 : (r >= a.a_rows ? (int)(a.a_rows - 1) : r));
    };
    auto a_first = [&](const ListedTile& t) -> int64_t { return by_table ? 0 : t.m0; };
    // row q of its rows of B, relative to the tile's first (SwiGLU: 32 gate rows and their 32 up
    // rows in turn, the up rows relative to the first up row)
    auto b_ofs = [&](const ListedTile& t, int q) -> uint32_t {
        const int n = kSwiglu ? (q >> 6) * 32 + (q & 31) : q, last = a.N - 1 - t.nt * kOutCols;
        return (uint32_t)(n < last ? n : last);
    };
    auto b_first = [&](const ListedTile& t) -> int64_t { return (int64_t)t.g * NB + t.nt * kOutCols; };
    const int64_t up = kSwiglu ? (int64_t)a.N * (a.K / 2) : 0;      // bytes from a gate row to its up row
    auto point_data = [&](const ListedTile& t, int buf) {
        a_at = a.a_codes + a_first(t) * (a.K / 2);
        b_at = a.b_codes + b_first(t) * (a.K / 2);
        const uint32_t half = (uint32_t)(a.K / 2);
#pragma unroll
        for (int l = 0; l < S::NL; ++l) {
            const bool is_a = l < S::NLA;
            const int q = (is_a ? wave * S::NLA + l : wave * S::NLB + l - S::NLA) * 8 + (lane >> 3);
            dofs[l] = (is_a ? a_ofs(t, buf, q) : b_ofs(t, q)) * half;
            if (kMode == kScale16) dofs[l] += ((lane & 7) ^ swz(q)) * 16;   // K is a multiple of 512: no clamp below
        }
#pragma unroll
        for (int l = 0; l < L::NS; ++l) {
            int i = (wave * L::NS + l) * 64 + lane;
            constexpr int kParts = kMode == kScale16 ? 1 : L::kRowBytes / 4;
            i = i < S::kRows * kParts ? i : S::kRows * kParts - 1;     // the last rows are B's
            const int q = i / kParts, part = i % kParts, qb = q - S::BM;
            // uniform where a load's 64 or 32 rows lie on one side
            const bool is_a = kMode == kScale1 ? q < S::BM : (wave * L::NS + l) * 64 / kParts < S::BM;
            const uint8_t* p = is_a ? a.a_scales + (a_first(t) + a_ofs(t, buf, q)) * nb
                                    : a.b_scales + (b_first(t) + b_ofs(t, qb) + (kSwiglu && (qb & 32) ? a.N : 0)) * nb;
            if constexpr (kMode == kScale1) {
                // a word that holds a valid byte lies in that byte's page
                slast[l] = reinterpret_cast<const uint8_t*>(reinterpret_cast<uintptr_t>(p + nb - 1) & ~(uintptr_t)3);
                p = reinterpret_cast<const uint8_t*>(reinterpret_cast<uintptr_t>(p) & ~(uintptr_t)3);
            } else {
                slast[l] = p + nb - 4;
            }
            ssrc[l] = p + 4 * part;
        }
    };
    auto point_mis = [&](const ListedTile& t, int buf) {
        if constexpr (kMode == kScale1) {
#pragma unroll
            for (int i = 0; i < kOps; ++i) {
                const int q = op_row(i), qb = q - S::BM;
                const int64_t r = i < S::TM ? a_first(t) + a_ofs(t, buf, q) : b_first(t) + b_ofs(t, qb) + (kSwiglu && (qb & 32) ? a.N : 0);
                mis[i] = (int)((reinterpret_cast<uintptr_t>(i < S::TM ? a.a_scales : a.b_scales) + (uintptr_t)(r * nb)) & 3);
            }
        }
    };
    // Stages are counted through a list's tiles; a stage sits in slot gs % 2 (kScale16: scales of
    // the stages gs, gs + 1 of an even gs in buffer gs / 2 % 2; a tile then has an even number).
    auto issue_data = [&](int l, int gs, int s) {
        const bool is_a = l < S::NLA;
        const int ql = is_a ? wave * S::NLA + l : wave * S::NLB + l - S::NLA;       // load of the operand: 8 rows
        const uint32_t to = lds0 + (gs & 1) * L::kDataBytes + ((is_a ? 0 : S::BM / 8) + ql) * 1024;
        const uint8_t* base = (is_a ? a_at : b_at + (kSwiglu && (ql & 4) ? up : 0)) + s * 128;
        if constexpr (kMode == kScale16) {
            g2lds16_at(base, dofs[l], to);
        } else {
            const int q = ql * 8 + (lane >> 3), c = (lane & 7) ^ swz(q), left = nb - 1 - s * 8;
            // past the end of K: the last block again; a stage past it altogether starts before its base
            g2lds16(base + dofs[l] + (int64_t)(c < left ? c : left) * 16, to);
        }
    };
    auto issue_scales = [&](int l, int gs, int s) {
        const int buf = kMode == kScale16 ? (gs >> 1) & 1 : gs & 1;
        const uint32_t to = lds0 + L::kScaleOff + buf * L::kScaleBytes + (wave * L::NS + l) * L::kPerLoad;
        const uint8_t* p = ssrc[l] + s * 8;
        if constexpr (kMode == kScale16) {
            g2lds16(p, to);
        } else {
            g2lds4(p < slast[l] ? p : slast[l], to);
        }
    };
    // the row indices of tile t into s_rows[buf] (past its end: the last one again)
    auto issue_rows = [&](const ListedTile& t, int buf) {
        if (!a.rows || wave * 64 >= S::BM) return;
        static_assert(S::BM <= 64 * S::NW, "one index a thread");
        const int at = wave * 64 + lane, last = t.m1 - 1 - t.m0;
        g2lds4(a.rows + t.m0 + (at < last ? at : last), lds0 + L::kRowsOff + (buf * S::BM + wave * 64) * 4);
    };

    struct Ops {
        v4i v[kOps];
    };
    struct Scales {
        int v[kOps];
    };
    auto read_op = [&](int i, int gs, int step, Ops& o) {
        o.v[i] = *reinterpret_cast<const v4i*>(lds + (gs & 1) * L::kDataBytes + op_row(i) * 128 +
                                               (((4 * h + step) ^ swz(j)) << 4));
    };
    // the scale bytes of this lane half's four blocks of stage s: 0 past the end of K
    auto read_scale = [&](int i, int gs, int s, Scales& o) {
        const uint8_t* base = lds + L::kScaleOff;
        if constexpr (kMode == kScale16) {
            o.v[i] = *reinterpret_cast<const int*>(base + ((gs >> 1) & 1) * L::kScaleBytes + op_row(i) * 16 + (gs & 1) * 8 + 4 * h);
        } else if constexpr (kMode == kScale4) {
            const int v = *reinterpret_cast<const int*>(base + (gs & 1) * L::kScaleBytes + op_row(i) * 8 + 4 * h);
            o.v[i] = 8 * s + 4 * h < nb ? v : 0;
        } else {
            const uint32_t* p = reinterpret_cast<const uint32_t*>(base + (gs & 1) * L::kScaleBytes + op_row(i) * 12 + 4 * h);
            const uint32_t v = __builtin_amdgcn_alignbyte(p[1], p[0], mis[i]);
            const int left = nb - (8 * s + 4 * h);
            o.v[i] = (int)(left >= 4 ? v : left <= 0 ? 0u : v & ((1u << (8 * left)) - 1u));
        }
    };

    v16f acc[S::TM][S::TN];
    auto clear = [&] {
#pragma unroll
        for (int i = 0; i < S::TM; ++i)
#pragma unroll
            for (int n = 0; n < S::TN; ++n)
#pragma unroll
                for (int e = 0; e < 16; ++e) acc[i][n][e] = 0.0f;
    };
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

    // Stores straight from the result registers.  A lane holds 4 consecutive columns of row j per
    // register quad g: columns 8 g + 4 h.  Exchanges between lanes make 16 bytes a lane and 64
    // consecutive bytes a row of them (32 at a time took the L2 twice the requests): of 16-bit
    // types quads 2 p and 2 p + 1 between the lane halves (each then has 8 columns, of quad
    // 2 p + h), and of all types two such vectors between lanes 16 apart, so that the first store
    // takes rows 0-15 of the tile and the second rows 16-31, lane group j / 16 the first or the
    // second vector.
    typedef typename Elem<kT>::type T;
    constexpr int kVec = 16 / (int)sizeof(T), kTiles = kSwiglu ? S::TN / 2 : S::TN;
    constexpr int kStores = S::TM * kTiles * (sizeof(T) == 4 ? 4 : 2);
    const bool vec = (reinterpret_cast<uintptr_t>(a.out) | (uint64_t)(a.out_stride * (int64_t)sizeof(T))) % 16 == 0 &&
                     a.N % kVec == 0;
    auto value = [&](int i, int n, int x) -> float {
        if constexpr (kSwiglu)
            return silu_mul(acc[i][2 * n][x], acc[i][2 * n + 1][x]);
        else
            return acc[i][n][x];
    };
    // vector p of tile (i, n): fp32 quad p, 16-bit quads 2 p and 2 p + 1
    auto vector = [&](int i, int n, int p, uint32_t(&w)[4]) {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = __float_as_uint(value(i, n, 4 * p + e));
        } else {
            typedef T T2 __attribute__((ext_vector_type(2)));
            uint32_t q[2][2];
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const T2 v = {from_f32<kT>(value(i, n, 4 * (2 * p + b) + 2 * e)),
                                  from_f32<kT>(value(i, n, 4 * (2 * p + b) + 2 * e + 1))};
                    q[b][e] = __builtin_bit_cast(uint32_t, v);
                }
            const auto s0 = __builtin_amdgcn_permlane32_swap(q[0][0], q[1][0], false, false);
            const auto s1 = __builtin_amdgcn_permlane32_swap(q[0][1], q[1][1], false, false);
            w[0] = s0[0], w[1] = s1[0], w[2] = s0[1], w[3] = s1[1];
        }
    };
    auto store_tile = [&](const ListedTile& t, auto whole_c) {
        constexpr bool kWhole = decltype(whole_c)::value;  // every row and column of the tile exists
#pragma unroll
        for (int i = 0; i < S::TM; ++i) {
#pragma unroll
            for (int n = 0; n < kTiles; ++n) {
                const int64_t r0 = t.m0 + (wm * S::TM + i) * 32 + (j & 15);
                const int c0 = t.nt * kOutCols + (wn * kTiles + n) * 32 + kVec * h + (j >> 4) * 2 * kVec;
                T* o = static_cast<T*>(a.out) + r0 * a.out_stride + c0;
#pragma unroll
                for (int p = 0; p < (sizeof(T) == 4 ? 4 : 2); p += 2) {
                    uint32_t w[2][4];
                    vector(i, n, p, w[0]);
                    vector(i, n, p + 1, w[1]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const auto x = __builtin_amdgcn_permlane16_swap(w[0][e], w[1][e], false, false);
                        w[0][e] = x[0];
                        w[1][e] = x[1];
                    }
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const uint4 v = {w[q][0], w[q][1], w[q][2], w[q][3]};
                        const int c = c0 + 2 * kVec * p;
                        T* at = o + 16 * q * a.out_stride + 2 * kVec * p;
                        if (kWhole || (vec && r0 + 16 * q < t.m1 && c < a.N)) {
                            *reinterpret_cast<uint4*>(at) = v;
                        } else if (r0 + 16 * q < t.m1) {
#pragma unroll
                            for (int e = 0; e < kVec; ++e) {
                                if (c + e >= a.N) break;
                                if constexpr (sizeof(T) == 4)
                                    at[e] = __uint_as_float(w[q][e]);
                                else
                                    at[e] = __builtin_bit_cast(T, (uint16_t)(w[q][e >> 1] >> (16 * (e & 1))));
                            }
                        }
                    }
                    __builtin_amdgcn_sched_barrier(0);    // two vectors at a time in registers
                }
            }
        }
    };

    // The tiles of BM rows that hold any, in the groups' order.  scan: those of the kWin groups from
    // base on, and in s_pre how many of them lie before each group's.
    constexpr int kPer = 4, kWin = 64 * S::NW * kPer;
    uint32_t* s_pre = reinterpret_cast<uint32_t*>(lds);   // nothing else is in the stages' slots then
    uint32_t* s_wave = s_pre + kWin;
    static_assert((kWin + S::NW) * 4 <= 2 * L::kDataBytes, "inside the stages' slots");
    auto bound = [&](int g) -> int { return bound_of(a, g < a.G ? g : a.G); };
    auto scan = [&](int base) -> uint32_t {
        int b[kPer + 1];
        uint32_t n[kPer], sum = 0;
#pragma unroll
        for (int i = 0; i <= kPer; ++i) b[i] = bound(base + tid * kPer + i);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            n[i] = b[i + 1] > b[i] ? (uint32_t)(b[i + 1] - b[i] + S::BM - 1) / S::BM : 0u;
            sum += n[i];                                  // at most 2^21 a group, 2^31 a window
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
        for (int w = 0; w < S::NW; ++w) {
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
    };
    int64_t slots = n_slots;
    uint32_t first_window = 0;
    if (a.bounds) {
        slots = 0;
        for (int base = 0; base < a.G; base += kWin) slots += first_window = scan(base);
        if (slots > n_slots) slots = n_slots;             // bounds that do not ascend
    }

    // this workgroup's tiles: bands of 8 row tiles by all column tiles, so that what an XCD runs at
    // once shares rows of A and of B in its L2; each XCD a run of as many tiles as the others, each of
    // its workgroups as many of them.  (Empty tiles numbered along, at most one a group, left the
    // fullest workgroup of 24576 rows in 256 groups 28 tiles of 19 on average.)
    const int64_t total = slots * n_tiles, per = (total + 7) >> 3;
    const int64_t run0 = (int64_t)(blockIdx.x & 7) * per, run1 = run0 + per < total ? run0 + per : total;
    const int nq = gridDim.x >> 3;
    static_assert(kListMost == 64 * S::NW, "a listed tile a thread");
    for (int64_t list0 = run0 + (blockIdx.x >> 3); list0 < run1; list0 += (int64_t)nq * kListMost) {
        const int64_t id = list0 + (int64_t)tid * nq;
        const bool want = id < run1;
        const uint32_t band = (uint32_t)id / (uint32_t)(8 * n_tiles), first = band * 8;   // total <= 2^30
        const uint32_t high = slots - first < 8 ? (uint32_t)(slots - first) : 8;
        const uint32_t in = (uint32_t)id - first * n_tiles;
        const int64_t at = first + (want ? in % high : 0);
        const int nt = want ? (int)(in / high) : 0;
        __syncthreads();                                  // the previous list is done
        if (!a.bounds) {
            const int64_t end = (at + 1) * S::BM;
            if (want) s_list[tid] = {0, (int)(at * S::BM), (int)(end < a.M ? end : a.M), nt};
        }
        int64_t before = 0;                               // tiles before the window's
        for (int base = 0; a.bounds && base < a.G; base += kWin) {
            const bool have = a.G <= kWin && list0 < run0 + nq;          // scanned above, uniform
            const uint32_t n = have ? first_window : scan(base);
            const int64_t x = at - before;
            before += n;
            if (want && x >= 0 && x < n) {
                int lo = 0, hi = kWin - 1;                // the last group with s_pre <= x
                while (lo < hi) {
                    const int mid = (lo + hi + 1) >> 1;
                    if (s_pre[mid] <= (uint32_t)x)
                        lo = mid;
                    else
                        hi = mid - 1;
                }
                const int g = base + lo, m0 = bound(g) + (int)((uint32_t)x - s_pre[lo]) * S::BM, end = bound(g + 1);
                s_list[tid] = {g, m0, m0 + S::BM < end ? m0 + S::BM : end, nt};
            }
        }
        __syncthreads();
        const int64_t left = (run1 - list0 + nq - 1) / nq;
        const int count = left < kListMost ? (int)left : kListMost;
        auto listed = [&](int i) -> ListedTile {
            const ListedTile t = s_list[i < count ? i : count - 1];
            return {__builtin_amdgcn_readfirstlane(t.g), __builtin_amdgcn_readfirstlane(t.m0),
                    __builtin_amdgcn_readfirstlane(t.m1), __builtin_amdgcn_readfirstlane(t.nt)};
        };
        ListedTile cur = listed(0);
        issue_rows(cur, 0);
        issue_rows(listed(1), 1);
        asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
        point_data(cur, 0);
        point_mis(cur, 0);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            if (kMode != kScale16 || u == 0) {
#pragma unroll
                for (int l = 0; l < L::NS; ++l) issue_scales(l, u, u);
            }
#pragma unroll
            for (int l = 0; l < S::NL; ++l) issue_data(l, u, u);
        }
        asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
        Ops o0, o1, o2, o3;
        Scales sc0, sc1;
#pragma unroll
        for (int i = 0; i < kOps; ++i) {
            read_op(i, 0, 0, o0);
            read_scale(i, 0, 0, sc0);
        }
        clear();
        int gs = 0;
        bool stored = false;                              // the last tile's kStores stores are out, nothing else behind the loads
        for (int ti = 0; ti < count; ++ti) {
            ListedTile next = cur;
            for (int s = 0; s < nst; ++s, ++gs) {
                // Stage gs, four steps of kProd products.  Steps 0 and 1 read the operands of steps 1
                // to 3; then every wave has read its share of slot gs % 2, and the barrier frees it for
                // stage gs + 2 and admits stage gs + 1 (its loads, the only ones out but for stores,
                // have had a stage's time).  Step 2 issues the loads of stage gs + 2, step 3 reads step
                // 0 of stage gs + 1.  Each memory instruction is placed behind a product of its own, in
                // whose 32 cycles it issues.
                products(std::integral_constant<int, 0>{}, o0, sc0, [&](int at) {
#pragma unroll
                    for (int i = at * 2 * kOps / kProd; i < (at + 1) * 2 * kOps / kProd; ++i) {
                        if (i < kOps)
                            read_op(i, gs, 1, o1);
                        else
                            read_op(i - kOps, gs, 2, o2);
                    }
                });
                products(std::integral_constant<int, 1>{}, o1, sc0, [&](int at) {
#pragma unroll
                    for (int i = at * kOps / kProd; i < (at + 1) * kOps / kProd; ++i) read_op(i, gs, 3, o3);
                });
                if (stored) {
                    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(kStores < 63 ? kStores : 63) : "memory");
                    stored = false;
                } else {
                    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
                }
                // past the list's last tile: its first stages again, not used
                const int s2 = s + 2 < nst ? s + 2 : s + 2 - nst;
                if (s + 2 == nst && ti + 1 < count) {     // this tile's loads are all issued: on to the next
                    next = listed(ti + 1);
                    point_data(next, (ti + 1) & 1);
                    if (ti + 2 < count) issue_rows(listed(ti + 2), ti & 1);   // its buffer: this tile's, pointed long ago
                }
                products(std::integral_constant<int, 2>{}, o2, sc0, [&](int at) {
                    if (at == 0 && (kMode != kScale16 || (s & 1) == 0)) {
#pragma unroll
                        for (int l = 0; l < L::NS; ++l) issue_scales(l, gs + 2, s2);
                    }
#pragma unroll
                    for (int l = at * S::NL / kProd; l < (at + 1) * S::NL / kProd; ++l) issue_data(l, gs + 2, s2);
                });
                const bool last = s + 1 == nst;
                if (last && ti + 1 < count) point_mis(next, (ti + 1) & 1);
                products(std::integral_constant<int, 3>{}, o3, sc0, [&](int at) {
                    // past the list's last stage: an old one, not used
#pragma unroll
                    for (int i = at * kOps / kProd; i < (at + 1) * kOps / kProd; ++i) {
                        read_op(i, gs + 1, 0, o0);
                        read_scale(i, gs + 1, last ? 0 : s + 1, sc1);
                    }
                });
                sc0 = sc1;
            }
            const bool whole = vec && cur.m0 + S::BM <= cur.m1 && (cur.nt + 1) * kOutCols <= a.N;   // uniform
            if (whole)
                store_tile(cur, std::true_type{});
            else
                store_tile(cur, std::false_type{});
            stored = whole;
            clear();
            cur = next;
        }
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    }
}

// ----------------------------------------------------------- few-row kernel ---
// Up to 32 rows of a group by 32 columns (SwiGLU: 32 gate and 32 up rows of B) per
// workgroup; its waves take every eighth run of 256 codes of K, fed straight from memory,
// and add up through LDS in wave order.  What bounds it is B's bytes, read once: lane half
// h takes blocks 4 h + s of a run, 64 consecutive bytes of a row in four loads.  At 1 row of
// 4096 x 4096 (8.9 MB, 1.9 us at a copy's rate) its 5.6 us are mostly latency: a launch, the
// operands' first bytes, the waves' sums.
constexpr int kFewWaves = 8, kFewRows = 32;

// Groups of a row table: row slot s belongs to the last group g whose first slot
// bounds[g] / 32 + g is <= s (a group of c rows never needs more than the
// bounds[g + 1] / 32 + 1 - bounds[g] / 32 slots up to the next group's first), so a
// workgroup finds its rows from the bounds alone, and where there is nothing to do it ends.
struct Rows {
    int g;
    int64_t m0, m1;           // rows [m0, m1); m0 >= m1: nothing to do
};

// The rows of a slot, the same on all lanes, by the wave together.
__device__ __forceinline__ Rows rows_of_slot(const MxGemm& a, int64_t slot)
{
    if (!a.bounds) {
        const int64_t m0 = slot * kFewRows;
        return {0, m0, m0 + kFewRows < a.M ? m0 + kFewRows : a.M};
    }
    // 64 groups are compared at a time, one per lane: two rounds of loads up to 4096 groups
    int g = 0, span = a.G;
    const int lane = threadIdx.x & 63;
    while (span > 1) {
        const int step = (span + 63) >> 6, at = g + lane * step;
        const bool le = lane * step < span && (int64_t)(bound_of(a, at) / kFewRows) + at <= slot;
        const int n = __popcll(__ballot(le));             // a run of lanes from 0 for bounds that ascend
        const int skip = (n > 0 ? n - 1 : 0) * step;
        g += skip;
        span = span - skip < step ? span - skip : step;
    }
    g = __builtin_amdgcn_readfirstlane(g);
    const int64_t b0 = bound_of(a, g), b1 = bound_of(a, g + 1);
    int64_t m0 = b0 + (slot - (b0 / kFewRows + g)) * kFewRows;
    const int64_t m1 = m0 + kFewRows < b1 ? m0 + kFewRows : b1;
    if (m0 < b0) m0 = m1;                                 // bounds that do not ascend: nothing before the group's rows
    return {g, m0, m1};
}

template <int kT, bool kSwiglu, bool kAligned>
__global__ __launch_bounds__(64 * kFewWaves) void k_mx_few(MxGemm a)
{
    constexpr int NT = kSwiglu ? 2 : 1;
    __shared__ float red[kFewWaves][NT][32][33];
    const Rows t = rows_of_slot(a, blockIdx.x);
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

// The most tiles of BM rows that the groups can have, and the few-row kernel's slots.
int64_t slots_of(const MxGemm& g, int BM) { return g.bounds ? g.M / BM + g.G : (g.M + BM - 1) / BM; }

template <class S, int kT, bool kSwiglu, int kMode>
hipError_t launch_tile(const MxGemm& g, hipStream_t st)
{
    constexpr int lds = MxLds<S, kMode>::kBytes;
    const int n_tiles = (int)nblk(g.N, kSwiglu ? S::BN / 2 : S::BN);
    const int64_t slots = slots_of(g, S::BM), total = slots * n_tiles;   // at most 2^30 (kMxMostTiles)
    // more than the default limit of dynamic LDS
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&k_mx_tile<S, kT, kSwiglu, kMode>),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
    // as many workgroups as the chip holds at once: 256 CUs, 160 KiB of LDS each
    constexpr int kGrid = 256 * (163840 / lds);
    const unsigned grid = 8 * nblk(total, 8);
    hipLaunchKernelGGL((k_mx_tile<S, kT, kSwiglu, kMode>), dim3(grid < (unsigned)kGrid ? grid : (unsigned)kGrid), dim3(64 * S::NW), lds,
                       st, g, n_tiles, slots);
    return hipGetLastError();
}

template <int kT, bool kSwiglu, int kMode>
hipError_t launch_shape(const MxGemm& g, hipStream_t st)
{
    const int64_t rows = g.M / g.G;       // rows a group has on average
    // tiles of a shape: what a grouped product has at most
    auto tiles = [&](int BM, int BN) { return slots_of(g, BM) * (int64_t)nblk(g.N, kSwiglu ? BN / 2 : BN); };
    // the tiled kernel reaches A through the row table by 32 bits of offset
    const bool far = (g.rows || g.row_div > 1) && g.a_rows * (g.K / 2) > (int64_t)UINT32_MAX;
    // Fewer tiles than a quarter of the CUs: the few-row kernel's workgroups are narrower and their
    // waves share K.  64 x 4096 x 4096: 7.5 us against 10.5; 128 rows (64 tiles): 13.2 against 10.6;
    // 64 groups of 8 rows, N = K = 2048 (more than 1024 tiles): 34.6 against 28.0.
    if (far || (rows <= 64 && tiles(64, 128) < 64)) {
        hipLaunchKernelGGL((k_mx_few<kT, kSwiglu, kMode != kScale1>), dim3((unsigned)slots_of(g, kFewRows), nblk(g.N, 32)),
                           dim3(64 * kFewWaves), 0, st, g);
        return hipGetLastError();
    }
    // 256 x 256 tiles move the fewest bytes a product but start and end slowest: worth it over
    // many stages, tiles that fill the chip more than once and groups that fill their last tile well
    // enough.  8192 x 4096 at K = 4096: 89 us against 94 of 128 x 128 tiles, K = 8192: 151, 175; K = 2880: 87, 90;
    // K = 2560: 67, 62; K = 2048: 59, 52; 4096 x 4096 x 4096 (256 tiles): 51, 51; 32 groups of 512 rows, N = 2048,
    // K = 4096: 95, 96, K = 6144: 140, 170; of 320 rows: 90, 77 and 126, 117.
    if (rows >= 448 && g.K >= 2816 && tiles(256, 256) >= 384) return launch_tile<Tile256, kT, kSwiglu, kMode>(g, st);
    // 128 x 128 tiles where they fill the chip's two workgroups a CU and the rows fill a good part of
    // a tile: 2048 x 4096 x 4096 27 us against 32 of 64 x 128; 128 groups of 72 rows, N = 768, K = 2048, SwiGLU
    // 45, 50, of 64 44, 45, of 56 44, 44, of 40 43, 39; 64 groups of 40 rows (N = K = 2048) 30.8, 29.6;
    // 512 x 4096 x 4096 (128 tiles) 14.6, 12.0.
    if (rows >= 60 && tiles(128, 128) >= 512) return launch_tile<Tile128, kT, kSwiglu, kMode>(g, st);
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
