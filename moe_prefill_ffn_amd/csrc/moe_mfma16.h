// The 16-bit matrix instruction of 16 x 16 tiles, and the zeros that loads past the end of K take.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_dtype.h"
#include "moe_tile.h"

namespace moe {

namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));

// First operand: 16 rows of weights (of an adapter), lane i = lane % 16 holds one; second: rows of activations.
// Lane group g = lane / 16 takes 8 values of the summed dimension and gets four consecutive results, columns
// 4 g .. 4 g + 3 of the first, of row i of the second operand.
template <int kIn>
__device__ __forceinline__ v4f mfma16x16(v4i w, v4i x, v4f c)
{
    if constexpr (kIn == kBF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, w), __builtin_bit_cast(v8bf, x), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, w), __builtin_bit_cast(v8h, x), c, 0, 0, 0);
}

// What a chunk past the end of K is loaded from.
__device__ const uint4 kZeros = {0, 0, 0, 0};

}  // namespace

}  // namespace moe
