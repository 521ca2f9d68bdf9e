// Element types of the tensors that callers hand over (MOE_F32 / MOE_BF16 / MOE_F16):
// loads to and stores from fp32.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_layout.h"

namespace moe {

enum DType { kF32 = 0, kBF16 = 1, kF16 = 2 };
MOE_HD static inline int dtype_bytes(int t) { return t == kF32 ? 4 : 2; }

template <int kT> struct Elem;
template <> struct Elem<kF32> { typedef float type; };
template <> struct Elem<kBF16> { typedef __bf16 type; };
template <> struct Elem<kF16> { typedef _Float16 type; };

// One rounding to the nearest, ties to even (the conversion instructions' own).
template <int kT>
__device__ __forceinline__ typename Elem<kT>::type from_f32(float v) { return (typename Elem<kT>::type)v; }

// n consecutive elements (n * size <= 16 bytes, aligned to n * size)
template <int kT, int n>
__device__ __forceinline__ void load_n(const void* p, float (&v)[n])
{
    typedef typename Elem<kT>::type T;
    typedef T Tn __attribute__((ext_vector_type(n)));
    const Tn t = *reinterpret_cast<const Tn*>(p);
#pragma unroll
    for (int i = 0; i < n; ++i) v[i] = (float)t[i];
}

template <int kT, int n>
__device__ __forceinline__ void store_n(void* p, const float (&v)[n])
{
    typedef typename Elem<kT>::type T;
    typedef T Tn __attribute__((ext_vector_type(n)));
    Tn t;
#pragma unroll
    for (int i = 0; i < n; ++i) t[i] = from_f32<kT>(v[i]);
    *reinterpret_cast<Tn*>(p) = t;
}

}  // namespace moe
