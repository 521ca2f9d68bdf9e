// Launch interface of the row-table kernels (host side of moe_rows.hip): pairs grouped by
// expert, and the experts' rows back to tokens.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_layout.h"

namespace moe {

constexpr int kGroupMostGroups = 1024;                    // a workgroup keeps 16 counters a group in LDS
constexpr int64_t kGroupMostPairs = 1 << 27;
constexpr int64_t kCombineMostTokens = 1 << 23;           // a workgroup of 256 threads each in one launch

// Pairs a workgroup places, and how many workgroups do: one up to kGroupOne pairs, else of
// kGroupChunk pairs, more where that would be more than kGroupMostBlocks workgroups.
constexpr int kGroupOne = 4096, kGroupChunk = 1024, kGroupMostBlocks = 256;
static inline int64_t group_chunk(int64_t pairs)
{
    if (pairs <= kGroupOne) return kGroupOne;
    const int64_t c = (pairs + kGroupMostBlocks - 1) / kGroupMostBlocks;
    return (c + kGroupChunk - 1) / kGroupChunk * kGroupChunk;
}
static inline int group_blocks(int64_t pairs) { return (int)((pairs + group_chunk(pairs) - 1) / group_chunk(pairs)); }
// counts of every workgroup's pairs a group, where there are several
static inline uint64_t group_ws(int64_t pairs, int groups)
{
    const int b = group_blocks(pairs);
    return b > 1 ? ((uint64_t)b * groups * 4 + 255) / 256 * 256 : 0;
}

struct GroupRows {
    const int32_t* eidx;      // [pairs] group of each pair; outside [0, E): in none
    int64_t pairs;
    int E;
    int32_t* counts;          // [E], optional
    int32_t* bounds;          // [E + 1]
    int32_t* rows;            // [pairs], optional
    int32_t* pos;             // [pairs], optional
    int32_t* ws;              // [blocks, E]
};

struct CombineRows {
    const void* d;            // [d_rows, n], rows d_stride apart
    int64_t d_stride, d_rows;
    int d_type;
    const float* weights;     // [T, k]
    const int32_t* pos;       // [T, k] row of d; outside [0, d_rows): none
    const void* base;         // [T, n] or null
    int64_t base_stride;
    int base_type;
    void* y;                  // [T, n]
    int64_t y_stride;
    int y_type;
    int64_t T;
    int n, k;
};

hipError_t launch_group_rows(const GroupRows& g, hipStream_t st);
hipError_t launch_combine_rows(const CombineRows& c, hipStream_t st);

}  // namespace moe
