// Launch interface of the low-rank adapters (host side of moe_lora.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_layout.h"

namespace moe {

constexpr int kLoraMostRank = 256, kLoraMostAdapters = 1 << 20;
constexpr int64_t kLoraMostRows = 1 << 23;                // tiles of 16 rows, 256 threads each, in one launch

// Parts of K whose sums are kept apart (each workgroup sums one): enough workgroups to fill the
// chip from the few tiles of 16 rows that a small batch has, each with at least kLoraUnit of K.
constexpr int kLoraTile = 16, kLoraUnit = 256;
static inline int lora_parts(int64_t M, int K)
{
    const int64_t tiles = (M + kLoraTile - 1) / kLoraTile, want = (512 + tiles - 1) / tiles, most = (K + kLoraUnit - 1) / kLoraUnit;
    const int64_t p = want < most ? want : most;
    return (int)(p < 16 ? p : 16);
}
// sums of the parts, [parts][M][r] fp32: enough for M rows or fewer (tiles * ceil(512 / tiles) < tiles + 512)
static inline uint64_t lora_ws(int64_t M, int K, int r)
{
    const int64_t rows = (M + kLoraTile - 1) / kLoraTile * kLoraTile, most = (K + kLoraUnit - 1) / kLoraUnit;
    const int64_t all = rows * (most < 16 ? most : 16), few = rows + 512 * kLoraTile;
    return ((uint64_t)(all < few ? all : few) * r * 4 + 255) / 256 * 256;
}

struct LoraAdd {
    const uint8_t* x;         // [M, K], rows x_stride bytes apart
    int64_t x_stride;
    const uint8_t* a;         // [n, r, K]
    const uint8_t* b;         // [n, N, r]
    int in_type;              // of x, a and b: kBF16 or kF16
    const int32_t* adapters;  // [M]; outside [0, n): none
    int n;
    const float* scales;      // [n] or null
    const void* base;         // [M, N] or null
    int64_t base_stride;
    int base_type;
    void* out;                // [M, N]
    int64_t out_stride;
    int out_type;
    int64_t M;
    int N, K, r;
    float* ws;
};

hipError_t launch_lora_add(const LoraAdd& l, hipStream_t st);

}  // namespace moe
