// HIP kernels (CDNA4 / gfx950) of products of 16-bit matrices (bf16 or fp16), dense or over the
// groups of a row table:
//   out[r, n] = sum_k A[src(r), k] B[g(r), n, k]
// in fp32, with SwiGLU of gate and up rows of B where asked for, rounded once.  Included by one source a
// type, so that they compile at once.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "moe_dtype.h"
#include "moe_gemm16.h"
#include "moe_mfma16.h"
#include "moe_tile.h"
#include "moe_tile_numbers.h"

namespace moe {

namespace {

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

// Rows [m0, m1) of group g; m0 >= m1: nothing to do.
struct Rows {
    int g;
    int64_t m0, m1;
};

// The rows of tile number x of the groups' tiles of BM rows that hold any, the same on all lanes, by each
// wave for itself.
template <int BM>
__device__ __forceinline__ Rows rows_of_tile(const Gemm16& a, int64_t x)
{
    if (!a.bounds) return {0, x * BM, x * BM + BM < a.M ? x * BM + BM : a.M};
    constexpr int kPer = 8;                               // groups a lane
    const int lane = threadIdx.x & 63;
    for (int base = 0; base < a.G; base += 64 * kPer) {
        int b[kPer + 1];
        uint32_t n = 0;
#pragma unroll
        for (int i = 0; i <= kPer; ++i) {
            const int g = base + lane * kPer + i;
            b[i] = bound_of(a, g < a.G ? g : a.G);
        }
        auto tiles = [&](int i) { return b[i + 1] > b[i] ? (uint32_t)(b[i + 1] - b[i] + BM - 1) / BM : 0u; };
#pragma unroll
        for (int i = 0; i < kPer; ++i) n += tiles(i);     // 2^23 a group at most, which leaves the next one none where bounds do not ascend
        uint32_t upto = n;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const uint32_t y = (uint32_t)__shfl_up((int)upto, o);
            if (lane >= o) upto += y;
        }
        const uint32_t all = (uint32_t)__builtin_amdgcn_readlane((int)upto, 63);
        if (x >= all) {
            x -= all;
            continue;
        }
        const int at = __builtin_ctzll(__ballot((int64_t)upto > x));   // the lane that has it
        int64_t left = x - (upto - n);
        int g = 0, m0 = 0, m1 = 0;
        bool found = false;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const uint32_t t = tiles(i);
            if (!found && left < (int64_t)t) {
                g = base + lane * kPer + i;
                m0 = b[i] + (int)left * BM;
                m1 = m0 + BM < b[i + 1] ? m0 + BM : b[i + 1];
                found = true;
            }
            if (!found) left -= t;
        }
        return {__builtin_amdgcn_readlane(g, at), __builtin_amdgcn_readlane(m0, at), __builtin_amdgcn_readlane(m1, at)};
    }
    return {0, 0, 0};
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
// 64 values (128 bytes a row, a cache line) through NS LDS slots.
template <int WM_, int WN_, int TM_, int TN_, int NS_>
struct Shape {
    static constexpr int WM = WM_, WN = WN_, TM = TM_, TN = TN_, NS = NS_;
    static constexpr int NW = WM * WN, BM = 32 * WM * TM, BN = 32 * WN * TN, kRows = BM + BN;
    // 1 KiB data loads per wave and stage: of A's rows, of B's
    static constexpr int NLA = BM / 8 / NW, NLB = BN / 8 / NW, NL = NLA + NLB;
    static_assert(NLA * NW * 8 == BM && NLB * NW * 8 == BN, "whole loads");
    static constexpr int kDataBytes = kRows * 128;
    static constexpr int kRowsOff = NS * kDataBytes;      // row indices of two tiles
    static constexpr int kListOff = kRowsOff + 2 * BM * 4;
    static constexpr int kLds = kListOff + kListMost * (int)sizeof(ListedTile);
};

// Persistent workgroups: each takes every so-many-th tile of its XCD's run (workgroups go
// round-robin over the 8 XCDs), one after the other without a pause in its stages -- the last NS
// stages of a tile issue the first NS of the next, whose pointers are made under the products,
// and the epilogue's stores drain under them.  Not so 256 x 256 tiles, whose 512 registers a wave do not hold all that: 16 to
// 27 are spilled, by type, and a tile's end reloads them behind everything that is out, the stores just made and the
// next tile's loads too, some eight times.  kTail: K ends inside a stage, or has fewer than NS; also for a table over 4 GiB of
// A or more.
//
// What bounds it: large dense products the matrix cores and the loads' latency -- 8192 x 4096 x 4096, bf16, 215 to
// 224 us or 1.25 PFLOP/s (a library product 217), the matrix cores busy 58% of the cycles: a fifth of a stage's
// lines come from beyond the L2, a 256 x 256 tile's two slots leave them one stage's time, and its end waits as said.  (Words a line read
// ahead into the L2 cost 6 to 60%: more requests.)  Over groups memory -- gate/up of 1024 tokens over 128 experts
// (805 MB of B) 159 to 170 us, 5 TB/s; down of 65536 rows in 256 groups (N = 4096, K = 1536; 4.0 GB, 4.9 by the L2's
// misses) 1.2 ms, in 128 x 256 tiles through three slots (two slots of 256 x 256 1.38, and 1.36 with tiles numbered
// across groups).
template <class S, int kIn, int kT, bool kSwiglu, bool kTail>
__global__ __launch_bounds__(64 * S::NW) void k_gemm16_tile(Gemm16 a, int n_tiles, int64_t n_slots)
{
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5, j = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / S::WN, wn = wave % S::WN;
    const int chunks = a.K / 8;                           // of 16 bytes
    // at least NS stages (a stage past the end of K adds 0): a stage issues the one NS further, which is
    // then in this tile or the next
    constexpr int NS = S::NS;
    const int nst = chunks > 8 * (NS - 1) ? (chunks + 7) >> 3 : NS;
    constexpr int kOutCols = kSwiglu ? S::BN / 2 : S::BN;
    int32_t* s_rows = reinterpret_cast<int32_t*>(lds + S::kRowsOff);
    ListedTile* s_list = reinterpret_cast<ListedTile*>(lds + S::kListOff);
    const uint32_t lds0 = lds_addr(lds);

    // A base per operand and tile, an offset per lane and load, 32 bits of bytes, or of 16 bytes with kTail: the
    // host checked that a tile's rows, or all of A where a table names them, span less.
    constexpr int kUnit = kTail ? 16 : 1;
    const uint8_t* a_at;
    const uint8_t* b_at;
    uint32_t dofs[S::NL];
    constexpr int kOps = S::TM + S::TN, kProd = S::TM * S::TN;
    const int sa_base = wm * S::TM * 32 + j, sb_base = S::BM + wn * S::TN * 32 + j;
    auto op_row = [&](int i) { return i < S::TM ? sa_base + i * 32 : sb_base + (i - S::TM) * 32; };

    // row q of tile t's rows of A, relative to a_at's row: from the row table (indices in
    // s_rows[buf]) relative to A, else to the tile's first
    const bool in_order = !a.rows && a.row_div == 1;
    auto first_of = [&](const ListedTile& t) { return a.rows ? 0 : in_order ? t.m0 : t.m0 / a.row_div; };
    auto a_ofs = [&](const ListedTile& t, int buf, int q) -> uint32_t {
        const int last = t.m1 - 1 - t.m0, at = q < last ? q : last;
        if (in_order) return (uint32_t)at;
        int r = a.rows ? s_rows[buf * S::BM + at] : t.m0 + at;
        if (a.row_div > 1) r /= a.row_div;
        return (uint32_t)((r < 0 ? 0 : (r >= a.a_rows ? (int)(a.a_rows - 1) : r)) - first_of(t));
    };
    // row q of its rows of B, relative to the tile's first (SwiGLU: 32 gate rows and their 32 up
    // rows in turn, the up rows relative to the first up row)
    auto b_ofs = [&](const ListedTile& t, int q) -> uint32_t {
        const int n = kSwiglu ? (q >> 6) * 32 + (q & 31) : q, last = a.N - 1 - t.nt * kOutCols;
        return (uint32_t)(n < last ? n : last);
    };
    const int64_t up = kSwiglu ? (int64_t)a.N * a.b_stride : 0;     // bytes from a gate row to its up row
    auto point_data = [&](const ListedTile& t, int buf) {
        a_at = a.a + first_of(t) * a.a_stride;
        b_at = a.b + t.g * a.b_group + (int64_t)(t.nt * kOutCols) * a.b_stride;
#pragma unroll
        for (int l = 0; l < S::NL; ++l) {
            const bool is_a = l < S::NLA;
            const int q = (is_a ? wave * S::NLA + l : wave * S::NLB + l - S::NLA) * 8 + (lane >> 3);
            dofs[l] = is_a ? a_ofs(t, buf, q) * (uint32_t)(a.a_stride / kUnit) : b_ofs(t, q) * (uint32_t)(a.b_stride / kUnit);
            dofs[l] += ((lane & 7) ^ swz(q)) * (16 / kUnit);
        }
    };
    // Stages go through the slots in turn, through a list's tiles.
    auto issue_data = [&](int l, int slot, int s) {
        const bool is_a = l < S::NLA;
        const int ql = is_a ? wave * S::NLA + l : wave * S::NLB + l - S::NLA;       // load of the operand: 8 rows
        const uint32_t to = lds0 + slot * S::kDataBytes + ((is_a ? 0 : S::BM / 8) + ql) * 1024;
        const uint8_t* base = (is_a ? a_at : b_at + (kSwiglu && (ql & 4) ? up : 0)) + s * 128;
        if constexpr (!kTail) {
            g2lds16_at(base, dofs[l], to);
        } else {
            const int c = (lane & 7) ^ swz(ql * 8 + (lane >> 3));
            g2lds16(c < chunks - s * 8 ? base + (uint64_t)dofs[l] * kUnit : reinterpret_cast<const uint8_t*>(&kZeros), to);
        }
    };
    // the row indices of tile t into s_rows[buf] (past its end: the last one again)
    auto issue_rows = [&](const ListedTile& t, int buf) {
        if (!a.rows || wave * 64 >= S::BM) return;
        static_assert(S::BM % 64 == 0 && S::BM <= 64 * S::NW, "one index a thread, whole waves");
        const int at = wave * 64 + lane, last = t.m1 - 1 - t.m0;
        g2lds4(a.rows + t.m0 + (at < last ? at : last), lds0 + S::kRowsOff + (buf * S::BM + wave * 64) * 4);
    };

    struct Ops {
        v4i v[kOps];
    };
    auto read_op = [&](int i, int slot, int step, Ops& o) {
        o.v[i] = *reinterpret_cast<const v4i*>(lds + slot * S::kDataBytes + op_row(i) * 128 + (((4 * h + step) ^ swz(j)) << 4));
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
        for (int u = 0; u < NS; ++u)
#pragma unroll
            for (int l = 0; l < S::NL; ++l) issue_data(l, u, u);
        asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
        Ops o0, o1, o2, o3;
#pragma unroll
        for (int i = 0; i < kOps; ++i) read_op(i, 0, 0, o0);
        clear();
        int slot = 0;
        bool stored = false;                              // the last tile's kStores stores are out, behind the loads
        for (int ti = 0; ti < count; ++ti) {
            ListedTile next = cur;
            for (int s = 0; s < nst; ++s) {
                // A stage, four steps of kProd products.  Steps 0 and 1 read the operands of steps 1 to 3;
                // then every wave has read its share of the slot, and the barrier frees it for the stage NS
                // further and admits the next stage, whose loads have had NS - 1 stages' time (the loads of the
                // NS - 2 stages behind it, and stores, may still be out).  Step 2 issues the loads of the stage
                // NS further, step 3 reads step 0 of the next.  Each memory instruction is placed behind a
                // product of its own, in whose 32 cycles it issues.
                const int after = slot + 1 < NS ? slot + 1 : 0;
                products(o0, [&](int at) {
#pragma unroll
                    for (int i = at * 2 * kOps / kProd; i < (at + 1) * 2 * kOps / kProd; ++i) {
                        if (i < kOps)
                            read_op(i, slot, 1, o1);
                        else
                            read_op(i - kOps, slot, 2, o2);
                    }
                });
                products(o1, [&](int at) {
#pragma unroll
                    for (int i = at * kOps / kProd; i < (at + 1) * kOps / kProd; ++i) read_op(i, slot, 3, o3);
                });
                constexpr int kBehind = (NS - 2) * S::NL, kMost = kBehind + kStores < 63 ? kBehind + kStores : 63;
                if (stored) {
                    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(kMost) : "memory");
                    stored = false;
                } else {
                    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(kBehind) : "memory");
                }
                // past the list's last tile: its first stages again, not used
                const int s2 = s + NS < nst ? s + NS : s + NS - nst;
                if (s + NS == nst && ti + 1 < count) {    // this tile's loads are all issued: on to the next
                    next = listed(ti + 1);
                    point_data(next, (ti + 1) & 1);
                    if (ti + 2 < count) issue_rows(listed(ti + 2), ti & 1);   // its buffer: this tile's, pointed long ago
                }
                products(o2, [&](int at) {
#pragma unroll
                    for (int l = at * S::NL / kProd; l < (at + 1) * S::NL / kProd; ++l) issue_data(l, slot, s2);
                });
                products(o3, [&](int at) {
                    // past the list's last stage: an old one, not used
#pragma unroll
                    for (int i = at * kOps / kProd; i < (at + 1) * kOps / kProd; ++i) read_op(i, after, 0, o0);
                });
                slot = after;
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
// Up to 16 kR rows of a group by 16 kN / NG columns (SwiGLU, NG = 2: 16 gate and 16 up rows of B) per
// workgroup; its waves take every eighth 64 values of K, fed straight from memory, four such units' loads
// out at a time, and add up through LDS in wave order.  What bounds it is B's bytes, read once: gate/up of one token,
// 8 experts (N = 768, K = 2048, 50 MB) 13 us, 3.8 TB/s; one row of 4096 x 4096 7.7 us, 4.3 TB/s.
constexpr int kFewWaves = 8;

// kR row tiles; kN tiles of 16 rows of B (SwiGLU: half of them gate, half up); from tile x0 and column tile y0 on
template <int kIn, int kT, bool kSwiglu, int kR, int kN>
__global__ __launch_bounds__(64 * kFewWaves) void k_gemm16_few(Gemm16 a, int64_t x0, int y0)
{
    constexpr int BM = 16 * kR, kCols = kSwiglu ? 8 * kN : 16 * kN;
    __shared__ float red[kFewWaves][BM][16 * kN + 4];
    const Rows t = rows_of_tile<BM>(a, x0 + blockIdx.x);
    if (t.m0 >= t.m1) return;                             // uniform
    const int tid = threadIdx.x, lane = tid & 63, i = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int chunks = a.K / 8, n0 = (y0 + (int)blockIdx.y) * kCols;
    const uint8_t* x[kR];
    const uint8_t* w[kN];
#pragma unroll
    for (int q = 0; q < kR; ++q) x[q] = a.a + a_row(a, t.m0 + 16 * q + i < t.m1 ? t.m0 + 16 * q + i : t.m1 - 1) * a.a_stride + 32 * g;
#pragma unroll
    for (int q = 0; q < kN; ++q) {
        const int at = n0 + 16 * (kSwiglu ? q / 2 : q) + i, n = at < a.N ? at : a.N - 1;
        w[q] = a.b + t.g * a.b_group + (int64_t)(kSwiglu && (q & 1) ? n + a.N : n) * a.b_stride + 32 * g;
    }
    v4f acc[kR][kN];
#pragma unroll
    for (int q = 0; q < kR; ++q)
#pragma unroll
        for (int n = 0; n < kN; ++n) acc[q][n] = v4f{0, 0, 0, 0};
    // two units; lane group g has chunks u + 2 g, + 1 of one that starts at chunk u; past the end of K 0
    constexpr int kStep = 8 * kFewWaves;
    struct Frag {
        v4i x[4][kR], w[4][kN];
    };
    auto load = [&](Frag& f, int u0) {
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int u = u0 + (s >> 1) * kStep;
            const bool in = u + 8 <= chunks || u + 2 * g + (s & 1) < chunks;
            const int64_t at = (int64_t)(u + (s & 1)) * 16;
#pragma unroll
            for (int n = 0; n < kN; ++n) f.w[s][n] = in ? *reinterpret_cast<const v4i*>(w[n] + at) : v4i{0, 0, 0, 0};
#pragma unroll
            for (int q = 0; q < kR; ++q) f.x[s][q] = in ? *reinterpret_cast<const v4i*>(x[q] + at) : v4i{0, 0, 0, 0};
        }
    };
    auto multiply = [&](const Frag& f) {
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int n = 0; n < kN; ++n)
#pragma unroll
                for (int q = 0; q < kR; ++q) acc[q][n] = mfma16x16<kIn>(f.w[s][n], f.x[s][q], acc[q][n]);
    };
    Frag f0, f1;
    const int u0 = wave * 8;
    if (u0 < chunks) load(f0, u0);
    if (u0 + 2 * kStep < chunks) load(f1, u0 + 2 * kStep);
    for (int u = u0; u < chunks; u += 4 * kStep) {
        multiply(f0);
        if (u + 4 * kStep < chunks) load(f0, u + 4 * kStep);
        if (u + 2 * kStep >= chunks) break;
        multiply(f1);
        if (u + 6 * kStep < chunks) load(f1, u + 6 * kStep);
    }
#pragma unroll
    for (int q = 0; q < kR; ++q)
#pragma unroll
        for (int n = 0; n < kN; ++n) *reinterpret_cast<v4f*>(&red[wave][16 * q + i][16 * n + 4 * g]) = acc[q][n];
    __syncthreads();
    typedef typename Elem<kT>::type T;
    for (int e = tid; e < BM * kCols; e += 64 * kFewWaves) {
        const int row = e / kCols, col = e % kCols, at = kSwiglu ? col / 16 * 32 + col % 16 : col;
        if (t.m0 + row >= t.m1 || n0 + col >= a.N) continue;
        float z = 0.0f, z2 = 0.0f;
#pragma unroll
        for (int v = 0; v < kFewWaves; ++v) {
            z += red[v][row][at];
            if (kSwiglu) z2 += red[v][row][at + 16];
        }
        static_cast<T*>(a.out)[(t.m0 + row) * a.out_stride + n0 + col] = from_f32<kT>(kSwiglu ? silu_mul(z, z2) : z);
    }
}

}  // namespace

// ----------------------------------------------------------------- launches ---
namespace {

// The most tiles of BM rows that the groups can have.
int64_t slots_of(const Gemm16& g, int BM)
{
    const int64_t n = g.bounds ? g.M / BM + g.G : (g.M + BM - 1) / BM;
    return n < g.M ? n : g.M;
}

// Few tiles leave a workgroup a CU to itself: deep rings, whose loads have up to seven stages' time.
// (64 x 128 through two slots took 37 us for 64 x 4096 x 4096, a load's latency a stage; 64 x 64 through
// eight 18.)
using Deep64 = Shape<2, 2, 1, 1, 8>;      // 64 x 64
using DeepWide = Shape<2, 2, 1, 2, 6>;    // 64 x 128
using Deep128 = Shape<2, 2, 2, 2, 4>;     // 128 x 128
using Tile128 = Shape<2, 2, 2, 2, 2>;     // 128 x 128, two workgroups a CU
using TileWide = Shape<2, 2, 2, 4, 3>;    // 128 x 256
using Tile256 = Shape<2, 2, 4, 4, 2>;     // 256 x 256

// as many workgroups as the chip holds at once: 256 CUs, 160 KiB of LDS each
template <class S>
constexpr int kGrid = 256 * (163840 / S::kLds);

template <class S, int kIn, int kT, bool kSwiglu, bool kTail>
hipError_t launch_kernel(const Gemm16& g, hipStream_t st)
{
    const int n_tiles = (int)nblk(g.N, kSwiglu ? S::BN / 2 : S::BN);
    const int64_t slots = slots_of(g, S::BM), total = slots * n_tiles;   // at most 2^30 (kGemm16MostTiles)
    // more than the default limit of dynamic LDS
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&k_gemm16_tile<S, kIn, kT, kSwiglu, kTail>),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, S::kLds);
    if (e != hipSuccess) return e;
    const unsigned grid = 8 * nblk(total, 8);
    hipLaunchKernelGGL((k_gemm16_tile<S, kIn, kT, kSwiglu, kTail>), dim3(grid < (unsigned)kGrid<S> ? grid : (unsigned)kGrid<S>),
                       dim3(64 * S::NW), S::kLds, st, g, n_tiles, slots);
    return hipGetLastError();
}

template <class S, int kIn, int kT, bool kSwiglu>
hipError_t launch_tile(const Gemm16& g, hipStream_t st)
{
    // a table over 4 GiB of A or more: offsets in 16 bytes, up to 64 GiB
    const bool wide = g.rows && g.a_stride > (int64_t)UINT32_MAX / g.a_rows;
    return wide || g.K % 64 || g.K < 64 * S::NS ? launch_kernel<S, kIn, kT, kSwiglu, true>(g, st) : launch_kernel<S, kIn, kT, kSwiglu, false>(g, st);
}

template <int kIn, int kT, bool kSwiglu, int kR, int kN>
hipError_t launch_few(const Gemm16& g, hipStream_t st)
{
    // A launch takes less than 2^32 threads along x and 65536 workgroups along y: more rows or columns take several.
    constexpr int64_t kMostX = 1 << 22, kMostY = 32768;
    const int64_t xs = slots_of(g, 16 * kR), ys = nblk(g.N, (kSwiglu ? 8 : 16) * kN);
    for (int64_t x0 = 0; x0 < xs; x0 += kMostX)
        for (int64_t y0 = 0; y0 < ys; y0 += kMostY)
            hipLaunchKernelGGL((k_gemm16_few<kIn, kT, kSwiglu, kR, kN>), dim3((unsigned)std::min(xs - x0, kMostX), (unsigned)std::min(ys - y0, kMostY)),
                               dim3(64 * kFewWaves), 0, st, g, x0, (int)y0);
    return hipGetLastError();
}

// What a shape's tiles would take, in us at K = 4096 but for the operands' way from memory, which is the same
// for all: the rounds of tiles that the chip goes through, each as long as measured on dense products
// (bf16, K = 4096; 128 x 128 in twos: half a round takes 43).
template <class S>
int rounds_time(const Gemm16& g, int a_round)
{
    // tiles as the groups have them on average: half a tile each is empty
    const int64_t some = g.M < g.G ? g.M : g.G, half = g.M / S::BM + g.G / 2;
    const int64_t slots = g.bounds ? std::min(std::max(half, some), slots_of(g, S::BM)) : slots_of(g, S::BM);
    const int64_t tiles = slots * (int64_t)nblk(g.N, g.swiglu ? S::BN / 2 : S::BN), rest = tiles % kGrid<S>;
    const int64_t t = tiles / kGrid<S> * a_round + (rest == 0 ? 0 : rest <= kGrid<S> - 256 ? 43 : a_round);
    return (int)(t < INT32_MAX ? t : INT32_MAX);
}

template <int kIn, int kT, bool kSwiglu>
hipError_t launch_shape(const Gemm16& g, hipStream_t st)
{
    // The tiled kernel reaches a tile's rows by 32 bits of offset (of bytes: 256 rows at most 16 MB apart), all of A through the
    // row table by 32 bits of 16 bytes (64 GiB; 8192 of 524,400 rows by 4096 x 4096, 260 us).  Beyond that the few-row kernel
    // takes any number of rows, and B again for every 16 of them (8192 x 4096 x 4096: 2.7 ms against 0.25).
    const bool far_a = g.rows ? g.a_stride / 16 > (int64_t)UINT32_MAX / g.a_rows : g.a_stride > (int64_t)UINT32_MAX / Tile256::BM;
    const bool far = far_a || g.b_stride > (int64_t)UINT32_MAX / Tile256::BN;
    // Too few tiles to fill the chip, whose waves the few-row kernel has share K.  Groups of a row or two: gate/up of
    // 8 rows (N = 768, K = 2048) 13 us against 17 of 64 x 128 tiles, of 16 rows 20, 22, of 32 rows 43, 43; down of 16 rows
    // (N = 2048, K = 768) 13.5, 13.4.  One matrix 4096 x 4096: 1 row 7.7 us against 18 of 64 x 64, 16 rows 10, 18, 32
    // rows 16.6, 17.9, 48 rows 20, 18; with SwiGLU (N = 1536) 32 rows 15.4, 23, 64 rows 19, 23; 1024 x 2048: 64 rows 6.1, 10.8.
    const int64_t tiles16 = slots_of(g, 16) * (int64_t)nblk(g.N, 16);
    const bool few = far || (g.bounds ? g.M <= 24 : g.M <= (kSwiglu ? 64 : 32) || tiles16 <= 256);
    if constexpr (kSwiglu) {
        if (few && !g.bounds && g.M > 32) return launch_few<kIn, kT, true, 2, 2>(g, st);
        if (few) return launch_few<kIn, kT, true, 1, 2>(g, st);
    } else {
        // 32 columns a workgroup: half the reads of A where there are workgroups enough (20 rows: 16.0 us, 17.8)
        if (few && tiles16 <= 256) return launch_few<kIn, kT, false, 1, 1>(g, st);
        if (few) return launch_few<kIn, kT, false, 1, 2>(g, st);
    }
    // The shape whose tiles are through first.  Measured at 4096 x 4096, us of 64 x 64, 64 x 128, 128 x 128, the same in
    // twos, 128 x 256, 256 x 256: 64 rows 18, 23, 30, 41, 49, 81; 512: 35, 26, 32, 42, 50, 84; 1024: 64, 48, 37, 50, 53, 87;
    // 2048: 122, 92, 68, 66, 68, 95; 5000: 314, 228, 174, 158, 174, 190; 8192: -, 318, -, 271, 249, 221.  Over groups, where B's
    // bytes are most of it: 512 rows in 64 groups (N = K = 2048) 108, 115, 119, 126, 126, 146; gate/up of 64 rows in
    // each of 128 (N = 768, K = 2048) -, 180, 160, 161, 159, 196; down of 256 in each of 256 (N = 4096, K = 1536) 1902, 1576,
    // 1359, 1298, 1205, 1380.
    const int t[] = {kSwiglu ? INT32_MAX : rounds_time<Deep64>(g, 18), rounds_time<DeepWide>(g, 24), rounds_time<Deep128>(g, 36),
                     rounds_time<Tile128>(g, 68), rounds_time<TileWide>(g, 62), rounds_time<Tile256>(g, 108)};
    int best = 0;
    for (int i = 1; i < 6; ++i) best = t[i] < t[best] ? i : best;
    if constexpr (!kSwiglu) {                             // gate and up rows are 32 each in a wave
        if (best == 0) return launch_tile<Deep64, kIn, kT, kSwiglu>(g, st);
    }
    if (best == 1) return launch_tile<DeepWide, kIn, kT, kSwiglu>(g, st);
    if (best == 2) return launch_tile<Deep128, kIn, kT, kSwiglu>(g, st);
    if (best == 3) return launch_tile<Tile128, kIn, kT, kSwiglu>(g, st);
    if (best == 4) return launch_tile<TileWide, kIn, kT, kSwiglu>(g, st);
    return launch_tile<Tile256, kIn, kT, kSwiglu>(g, st);
}

template <int kIn>
hipError_t launch_gemm16_typed(const Gemm16& g, hipStream_t st)
{
    if (g.out_type == kF32) return g.swiglu ? launch_shape<kIn, kF32, true>(g, st) : launch_shape<kIn, kF32, false>(g, st);
    return g.swiglu ? launch_shape<kIn, kIn, true>(g, st) : launch_shape<kIn, kIn, false>(g, st);
}

}  // namespace

}  // namespace moe
