// Launch interface of the low-rank adapters (host side of moe_lora.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_dtype.h"

namespace moe {

constexpr int kLoraMostRank = 256, kLoraMostAdapters = 1 << 20;
constexpr int64_t kLoraMostRows = 1 << 23;                // tiles of 16 rows, 256 threads each, in one launch

// Above this many rows the tiles are larger, see moe_lora.hip.
constexpr int kLoraFewRows = 1024;
static inline bool lora_few(int64_t M) { return M <= kLoraFewRows; }
// Rows of a tile of x A^T, and parts of K whose sums are kept apart (each workgroup sums
// one): enough workgroups to fill the chip from the few tiles of a small batch, each with at least
// kLoraUnit of K.
constexpr int kLoraUnit = 256, kLoraMostParts = 16, kLoraFill = 512;
static inline int lora_tile(int64_t M, int r) { return lora_few(M) ? 16 : r <= 32 ? 128 : 64; }
static inline int lora_parts(int64_t M, int K, int r)
{
    const int64_t tiles = (M + lora_tile(M, r) - 1) / lora_tile(M, r), want = (kLoraFill + tiles - 1) / tiles;
    const int64_t most = (K + kLoraUnit - 1) / kLoraUnit, p = want < most ? want : most;
    return (int)(p < kLoraMostParts ? p : kLoraMostParts);
}
// sums of the parts, [parts][M][r] fp32: enough for M rows or fewer (tiles * ceil(kLoraFill / tiles) < tiles + kLoraFill)
static inline uint64_t lora_ws(int64_t M, int K, int r)
{
    const int64_t rows = (M + 127) / 128 * 128, most = (K + kLoraUnit - 1) / kLoraUnit;
    const int64_t all = rows * (most < kLoraMostParts ? most : kLoraMostParts), few = rows + (int64_t)kLoraFill * lora_tile(kLoraFewRows + 1, r);
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
