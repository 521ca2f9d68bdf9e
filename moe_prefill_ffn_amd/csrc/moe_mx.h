// Launch interface of the MXFP4 kernels (host side of moe_mx.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_layout.h"

namespace moe {

// What one launch takes: a launch has fewer than 2^32 threads (four a block of 32; 512 for 32 rows
// and a group's last ones), and the tiled kernel counts its tiles in 32 bits.
constexpr int64_t kMxMostBlocks = (1 << 30) - 64;     // M * K / 32 of quantise and dequantise: whole workgroups of 64
constexpr int64_t kMxMostRows = 1 << 27;              // M of a product
constexpr int64_t kMxMostTiles = 1 << 30;             // its tiles, the smallest being 64 x 64

struct MxQuant {
    const void* x;            // quantise: [M, K] in; dequantise: out
    void* y;
    int dtype;
    int64_t M, stride;        // rows, elements between rows of x (or y)
    int K;
    uint8_t* codes;           // [M, K / 2]
    uint8_t* scales;          // [M, K / 32]
};

struct MxGemm {
    const uint8_t* a_codes;   // [a_rows, K / 2], a_rows < 2^31
    const uint8_t* a_scales;  // [a_rows, K / 32]
    int64_t a_rows;
    const int32_t* rows;      // row r of the product reads A row rows[r] / row_div (null: r / row_div)
    int row_div;
    const uint8_t* b_codes;   // [G, NB, K / 2], NB = N or 2 N (SwiGLU: gate rows, then up rows)
    const uint8_t* b_scales;
    const int32_t* bounds;    // [G + 1] on the device (null: one group of all M rows)
    int G;
    int64_t M;
    int N, K;
    int swiglu;
    void* out;                // [M, N]
    int64_t out_stride;
    int dtype;
};

hipError_t launch_mx_quantize(const MxQuant& q, hipStream_t st);
hipError_t launch_mx_dequantize(const MxQuant& q, hipStream_t st);
hipError_t launch_mx_gemm(const MxGemm& g, hipStream_t st);

}  // namespace moe
