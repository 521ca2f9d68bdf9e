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
#include "moe_tile_numbers.h"

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

// ------------------------------------------------------------- tiled kernel ---
// WM x WN waves, each TM x TN tiles of 32 x 32: BM rows of A by BN rows of B, K in stages of
// 64 values (128 bytes a row, a cache line) through two LDS slots.
template <int WM_, int WN_, int TM_, int TN_>
struct Shape {
    static constexpr int WM = WM_, WN = WN_, TM = TM_, TN = TN_;
    static constexpr int NW = WM * WN, BM = 32 * WM * TM, BN = 32 * WN * TN, kRows = BM + BN;
    // 1 KiB data loads per wave and stage: of A's rows, of B's
    static constexpr int NLA = BM / 8 / NW, NLB = BN / 8 / NW, NL = NLA + NLB;
    static_assert(NLA * NW * 8 == BM && NLB * NW * 8 == BN, "whole loads");
    static constexpr int kDataBytes = kRows * 128;
    static constexpr int kRowsOff = 2 * kDataBytes;       // row indices of two tiles
    static constexpr int kListOff = kRowsOff + 2 * BM * 4;
    static constexpr int kLds = kListOff + kListMost * (int)sizeof(ListedTile);
};

// What a chunk past the end of K is loaded from.
__device__ const uint4 kZeros = {0, 0, 0, 0};

// Persistent workgroups: each takes every so-many-th tile of its XCD's run (workgroups go
// round-robin over the 8 XCDs), one after the other without a pause in its stages -- the last two
// stages of a tile issue the first two of the next, whose pointers are made under the products,
// and the epilogue's stores drain under them.  kTail: K ends inside a stage, or there is one alone.
template <class S, int kIn, int kT, bool kSwiglu, bool kTail>
__global__ __launch_bounds__(64 * S::NW) void k_gemm16_tile(Gemm16 a, int n_tiles, int64_t n_slots)
{
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5, j = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / S::WN, wn = wave % S::WN;
    const int chunks = a.K / 8;                           // of 16 bytes
    // at least two stages (a stage past the end of K adds 0): a stage issues the one two further,
    // which is then in this tile or the next
    const int nst = chunks > 8 ? (chunks + 7) >> 3 : 2;
    constexpr int kOutCols = kSwiglu ? S::BN / 2 : S::BN;
    int32_t* s_rows = reinterpret_cast<int32_t*>(lds + S::kRowsOff);
    ListedTile* s_list = reinterpret_cast<ListedTile*>(lds + S::kListOff);
    const uint32_t lds0 = lds_addr(lds);

    // A base per operand and tile, an offset per lane and load.  32 bits of offset: the host checked
    // that a tile's rows, or all of A where a table names them, span less.
    const uint8_t* a_at;
    const uint8_t* b_at;
    uint32_t dofs[S::NL];
    constexpr int kOps = S::TM + S::TN, kProd = S::TM * S::TN;
    const int sa_base = wm * S::TM * 32 + j, sb_base = S::BM + wn * S::TN * 32 + j;
    auto op_row = [&](int i) { return i < S::TM ? sa_base + i * 32 : sb_base + (i - S::TM) * 32; };

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
    // row q of its rows of B, relative to the tile's first (SwiGLU: 32 gate rows and their 32 up
    // rows in turn, the up rows relative to the first up row)
    auto b_ofs = [&](const ListedTile& t, int q) -> uint32_t {
        const int n = kSwiglu ? (q >> 6) * 32 + (q & 31) : q, last = a.N - 1 - t.nt * kOutCols;
        return (uint32_t)(n < last ? n : last);
    };
    const int64_t up = kSwiglu ? (int64_t)a.N * a.b_stride : 0;     // bytes from a gate row to its up row
    auto point_data = [&](const ListedTile& t, int buf) {
        a_at = a.a + (by_table ? 0 : t.m0) * a.a_stride;
        b_at = a.b + t.g * a.b_group + (int64_t)(t.nt * kOutCols) * a.b_stride;
#pragma unroll
        for (int l = 0; l < S::NL; ++l) {
            const bool is_a = l < S::NLA;
            const int q = (is_a ? wave * S::NLA + l : wave * S::NLB + l - S::NLA) * 8 + (lane >> 3);
            dofs[l] = is_a ? a_ofs(t, buf, q) * (uint32_t)a.a_stride : b_ofs(t, q) * (uint32_t)a.b_stride;
            dofs[l] += ((lane & 7) ^ swz(q)) * 16;
        }
    };
    // Stages are counted through a list's tiles; a stage sits in slot gs % 2.
    auto issue_data = [&](int l, int gs, int s) {
        const bool is_a = l < S::NLA;
        const int ql = is_a ? wave * S::NLA + l : wave * S::NLB + l - S::NLA;       // load of the operand: 8 rows
        const uint32_t to = lds0 + (gs & 1) * S::kDataBytes + ((is_a ? 0 : S::BM / 8) + ql) * 1024;
        const uint8_t* base = (is_a ? a_at : b_at + (kSwiglu && (ql & 4) ? up : 0)) + s * 128;
        if constexpr (!kTail) {
            g2lds16_at(base, dofs[l], to);
        } else {
            const int c = (lane & 7) ^ swz(ql * 8 + (lane >> 3));
            g2lds16(c < chunks - s * 8 ? base + dofs[l] : reinterpret_cast<const uint8_t*>(&kZeros), to);
        }
    };
    // the row indices of tile t into s_rows[buf] (past its end: the last one again)
    auto issue_rows = [&](const ListedTile& t, int buf) {
        if (!a.rows || wave * 64 >= S::BM) return;
        static_assert(S::BM <= 64 * S::NW, "one index a thread");
        const int at = wave * 64 + lane, last = t.m1 - 1 - t.m0;
        if (S::BM < 64 && lane >= S::BM) return;
        g2lds4(a.rows + t.m0 + (at < last ? at : last), lds0 + S::kRowsOff + (buf * S::BM + wave * 64) * 4);
    };

    struct Ops {
        v4i v[kOps];
    };
    auto read_op = [&](int i, int gs, int step, Ops& o) {
        o.v[i] = *reinterpret_cast<const v4i*>(lds + (gs & 1) * S::kDataBytes + op_row(i) * 128 + (((4 * h + step) ^ swz(j)) << 4));
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
    auto products = [&](const Ops& o, auto between) {
#pragma unroll
        for (int i = 0; i < S::TM; ++i)
#pragma unroll
            for (int n = 0; n < S::TN; ++n) {
                acc[i][n] = mfma16<kIn>(o.v[S::TM + n], o.v[i], acc[i][n]);
                between(i * S::TN + n);
                __builtin_amdgcn_sched_barrier(0);
            }
    };

    // Stores straight from the result registers.  A lane holds 4 consecutive columns of row j per
    // register quad g: columns 8 g + 4 h.  Exchanges between lanes make 16 bytes a lane and 64
    // consecutive bytes a row of them: of 16-bit types quads 2 p and 2 p + 1 between the lane halves
    // (each then has 8 columns, of quad 2 p + h), and of all types two such vectors between lanes 16
    // apart, so that the first store takes rows 0-15 of the tile and the second rows 16-31, lane group
    // j / 16 the first or the second vector.
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

    TileNumbers<S::NW, S::BM> num(a, reinterpret_cast<uint32_t*>(lds), n_slots);
    static_assert(TileNumbers<S::NW, S::BM>::kBytes <= 2 * S::kDataBytes, "inside the stages' slots");
    const TileRun run = tile_run(num.slots, n_tiles);
    for (int64_t list0 = run.first; list0 < run.end; list0 += (int64_t)run.step * kListMost) {
        const int count = num.list(a, s_list, list0, run, n_tiles);
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
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int l = 0; l < S::NL; ++l) issue_data(l, u, u);
        asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
        Ops o0, o1, o2, o3;
#pragma unroll
        for (int i = 0; i < kOps; ++i) read_op(i, 0, 0, o0);
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
                products(o0, [&](int at) {
#pragma unroll
                    for (int i = at * 2 * kOps / kProd; i < (at + 1) * 2 * kOps / kProd; ++i) {
                        if (i < kOps)
                            read_op(i, gs, 1, o1);
                        else
                            read_op(i - kOps, gs, 2, o2);
                    }
                });
                products(o1, [&](int at) {
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
                products(o2, [&](int at) {
#pragma unroll
                    for (int l = at * S::NL / kProd; l < (at + 1) * S::NL / kProd; ++l) issue_data(l, gs + 2, s2);
                });
                products(o3, [&](int at) {
                    // past the list's last stage: an old one, not used
#pragma unroll
                    for (int i = at * kOps / kProd; i < (at + 1) * kOps / kProd; ++i) read_op(i, gs + 1, 0, o0);
                });
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

using Tile256 = Shape<2, 2, 4, 4>;        // 256 x 256
using Tile128 = Shape<2, 2, 2, 2>;        // 128 x 128
using Tile64 = Shape<2, 2, 1, 2>;         // 64 x 128

template <class S, int kIn, int kT, bool kSwiglu, bool kTail>
hipError_t launch_tile(const Gemm16& g, hipStream_t st)
{
    const int n_tiles = (int)nblk(g.N, kSwiglu ? S::BN / 2 : S::BN);
    const int64_t slots = slots_of(g, S::BM), total = slots * n_tiles;   // at most 2^30 (kGemm16MostTiles)
    // more than the default limit of dynamic LDS
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&k_gemm16_tile<S, kIn, kT, kSwiglu, kTail>),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, S::kLds);
    if (e != hipSuccess) return e;
    // as many workgroups as the chip holds at once: 256 CUs, 160 KiB of LDS each
    constexpr int kGrid = 256 * (163840 / S::kLds);
    const unsigned grid = 8 * nblk(total, 8);
    hipLaunchKernelGGL((k_gemm16_tile<S, kIn, kT, kSwiglu, kTail>), dim3(grid < (unsigned)kGrid ? grid : (unsigned)kGrid), dim3(64 * S::NW),
                       S::kLds, st, g, n_tiles, slots);
    return hipGetLastError();
}

template <int kIn, int kT, bool kSwiglu, bool kTail>
hipError_t launch_shape(const Gemm16& g, hipStream_t st)
{
    const int64_t rows = g.M / g.G;       // rows a group has on average
    // tiles of a shape: what a grouped product has at most
    auto tiles = [&](int BM, int BN) { return slots_of(g, BM) * (int64_t)nblk(g.N, kSwiglu ? BN / 2 : BN); };
    // the tiled kernel reaches a tile's rows, or all of A through the row table, by 32 bits of offset
    const int64_t a_span = (g.rows || g.row_div > 1 ? g.a_rows : 256) * g.a_stride, b_span = 256 * g.b_stride;
    const bool far = a_span > (int64_t)UINT32_MAX || b_span > (int64_t)UINT32_MAX;
    if (far || (rows <= 64 && tiles(64, 128) < 64)) {
        hipLaunchKernelGGL((k_gemm16_few<kIn, kT, kSwiglu>), dim3((unsigned)slots_of(g, kFewRows), nblk(g.N, 32)), dim3(64 * kFewWaves), 0, st, g);
        return hipGetLastError();
    }
    if (rows >= 256 && tiles(256, 256) >= 384) return launch_tile<Tile256, kIn, kT, kSwiglu, kTail>(g, st);
    if (rows >= 60 && tiles(128, 128) >= 512) return launch_tile<Tile128, kIn, kT, kSwiglu, kTail>(g, st);
    return launch_tile<Tile64, kIn, kT, kSwiglu, kTail>(g, st);
}

template <int kIn, int kT, bool kSwiglu>
hipError_t launch_tail(const Gemm16& g, hipStream_t st)
{
    return g.K % 64 || g.K < 128 ? launch_shape<kIn, kT, kSwiglu, true>(g, st) : launch_shape<kIn, kT, kSwiglu, false>(g, st);
}

template <int kIn>
hipError_t launch_typed(const Gemm16& g, hipStream_t st)
{
    if (g.out_type == kF32) return g.swiglu ? launch_tail<kIn, kF32, true>(g, st) : launch_tail<kIn, kF32, false>(g, st);
    return g.swiglu ? launch_tail<kIn, kIn, true>(g, st) : launch_tail<kIn, kIn, false>(g, st);
}

}  // namespace

hipError_t launch_gemm16(const Gemm16& g, hipStream_t st)
{
    if (g.M == 0) return hipSuccess;
    return g.in_type == kBF16 ? launch_typed<kBF16>(g, st) : launch_typed<kF16>(g, st);
}

}  // namespace moe
