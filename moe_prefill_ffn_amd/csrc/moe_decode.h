// Launch interface of the few-token layer's kernels (host side of moe_decode.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_layout.h"

namespace moe {

constexpr int kDecodeMaxPairs = 1024;   // n_tokens * top_k of one call
// Most rows of one expert that share one read of its weights.  Two fill one result register quad of
// each lane half and 26 KB of LDS at 4096 columns; four cost a quad more and the LDS of a workgroup a CU:
// 4096 x 1536, 8 of 256 experts, 16 tokens 201 us against 230 of four rows, 24 alike 278 against 302, 24
// skewed 149, 146, 128 tokens 824, 762; at 16384 columns four do not fit.
constexpr int kChunkRows = 2;

// One work item of the expert products: (token, slot) pairs of one expert.
struct DecodeChunk {
    int32_t expert, n;
    int32_t pair[kChunkRows];  // 16 bytes
};

struct DecodeWs {
    uint64_t eidx, wts, counts, nchunks, chunks, xl, xs, hl, hs, dm, total;
    int max_chunks;
};

static inline DecodeWs decode_ws(int d, int f, int E, int k, int T)
{
    DecodeWs L;
    const uint64_t R = (uint64_t)T * k;
    // sum over experts of ceil(rows / kChunkRows): at most one partial chunk per reached expert
    L.max_chunks = (int)(R / kChunkRows) + (int)(R < (uint64_t)E ? R : (uint64_t)E);
    uint64_t o = 0;
    auto take = [&](uint64_t bytes) { uint64_t at = o; o = align_up(o + bytes, 256); return at; };
    L.eidx = take(R * 4);
    L.wts = take(R * 4);
    L.counts = take((uint64_t)E * 4);
    L.nchunks = take(4);
    L.chunks = take((uint64_t)L.max_chunks * sizeof(DecodeChunk));
    L.xl = take((uint64_t)T * 3 * d);
    L.xs = take((uint64_t)T * (d / 32) * 4);
    L.hl = take(R * 3 * f);
    L.hs = take(R * (f / 32) * 4);
    L.dm = take(R * d * 4);
    L.total = o;
    return L;
}

struct DecodeLaunch {
    int T, d, f, E, k, dtype;
    const void* x;
    int64_t x_stride;          // elements
    const float* logits;
    int64_t logits_stride;
    void* y;
    int64_t y_stride;
    const uint8_t* blob;
    uint64_t expert_stride, gu_q_off, gu_s_off, d_q_off, d_s_off;
    uint8_t* ws;
    DecodeWs L;
    int32_t* eidx_out;         // optional exports
    float* wts_out;
    bool need_counts;          // the rows per expert (DecodeWs::counts) are read after the routing
};

// Routing, the chunk table and x's fixed-point form; nothing where the products route themselves.
hipError_t launch_decode_route(const DecodeLaunch& D, hipStream_t st);
// The experts with rows from the pinned host blob into the slot that D reads, after a route with need_counts.
hipError_t launch_decode_load(const DecodeLaunch& D, const uint8_t* src, uint8_t* dst, unsigned long long* stats, hipStream_t st);
// Both expert products (the last reader of the weights), and the combine where they hold it.
hipError_t launch_decode_products(const DecodeLaunch& D, hipStream_t st);
// The combine, where the products left it.
hipError_t launch_decode_combine(const DecodeLaunch& D, hipStream_t st);

}  // namespace moe
