// Launch interface of the 16-bit products (host side of moe_gemm16_kernels.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_dtype.h"

namespace moe {

// What one launch takes, as of the MXFP4 products.
constexpr int64_t kGemm16MostRows = 1 << 27;              // M
constexpr int64_t kGemm16MostTiles = 1 << 30;             // its tiles, the smallest being 32 x 32

struct Gemm16 {
    const uint8_t* a;         // [a_rows, K] bf16 or fp16, rows a_stride bytes apart; a_rows < 2^31
    int64_t a_stride, a_rows;
    const int32_t* rows;      // row r of the product reads A row rows[r] / row_div (null: r / row_div)
    int row_div;
    const uint8_t* b;         // [G, NB, K], NB = N or 2 N (SwiGLU: gate rows, then up rows)
    int64_t b_stride, b_group;   // bytes between rows, between groups
    const int32_t* bounds;    // [G + 1] on the device (null: one group of all M rows)
    int G;
    int64_t M;
    int N, K;
    int swiglu;
    int in_type;              // of A and B: kBF16 or kF16
    void* out;                // [M, N]
    int64_t out_stride;
    int out_type;             // kF32 or in_type
};

hipError_t launch_gemm16_bf16(const Gemm16& g, hipStream_t st);
hipError_t launch_gemm16_f16(const Gemm16& g, hipStream_t st);
inline hipError_t launch_gemm16(const Gemm16& g, hipStream_t st)
{
    if (g.M == 0) return hipSuccess;
    return g.in_type == kBF16 ? launch_gemm16_bf16(g, st) : launch_gemm16_f16(g, st);
}

}  // namespace moe
