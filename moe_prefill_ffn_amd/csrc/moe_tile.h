// What the kernels of products over a row table share: loads straight into LDS, the order of
// rows in LDS, the groups' bounds, SwiGLU.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));

namespace {

inline unsigned nblk(int64_t n, int per) { return (unsigned)((n + per - 1) / per); }

// A bound of the groups of `a` (bounds, M), clamped into [0, M].
template <class Args>
__device__ __forceinline__ int bound_of(const Args& a, int g)
{
    const int64_t b = a.bounds[g];
    return (int)(b < 0 ? 0 : b > a.M ? a.M : b);
}

// silu(g) u by the hardware's exp2 and reciprocal (an ulp each).  exp(-g) = 2^t (1 + ln2 r), t the
// rounded -g log2(e) and r what the rounding left, so that a large |g| costs no bits.
__device__ __forceinline__ float silu_mul(float g, float u)
{
    const float log2e = 0x1.715476p+0f, log2e_lo = 0x1.4ae0c0p-26f;   // the fp32 nearest log2(e), and the rest
    const float t = -g * log2e;
    const float r = __builtin_fmaf(-g, log2e, -t) - g * log2e_lo;
    const float p = __builtin_amdgcn_exp2f(t);
    // past the range of exp (p = 0 or infinity) there is nothing to correct
    const float e = t > -126.0f && t < 128.0f ? __builtin_fmaf(p, 0x1.62e430p-1f * r, p) : p;
    return g * __builtin_amdgcn_rcpf(1.0f + e) * u;
}

// Direct global->LDS loads, lane i's bytes at wave_base + size * i; inline asm so that the
// compiler does not drain them (the ring waits for them itself).
__device__ __forceinline__ uint32_t lds_addr(const void* p)
{
    return __builtin_amdgcn_readfirstlane(
        (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p);
}
__device__ __forceinline__ void g2lds16(const void* g, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %1\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(g), "s"(lds) : "memory", "m0");
}
// the same from a wave-uniform base and 32 bits of offset a lane
__device__ __forceinline__ void g2lds16_at(const uint8_t* base, uint32_t off, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %2\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "s"(lds) : "memory", "m0");
}
__device__ __forceinline__ void g2lds4(const void* g, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %1\n\tglobal_load_lds_dword %0, off" ::"v"(g), "s"(lds) : "memory", "m0");
}

// Chunk c (16 bytes, one block) of a 128-byte row r sits in slot c ^ swz(r): any 8
// consecutive rows touch 8 distinct 16-byte bank groups of 128 bytes, any 16 rows 16
// distinct ones of 256.
__device__ __forceinline__ int swz(int r) { return (r ^ ((r >> 3) & 1)) & 7; }

constexpr int kListMost = 256;                            // tiles a workgroup lists at a time

struct ListedTile {
    int g, m0, m1, nt;
};

}  // namespace

}  // namespace moe
