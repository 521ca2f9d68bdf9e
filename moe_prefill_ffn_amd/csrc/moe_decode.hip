// HIP kernels (CDNA4 / gfx950) of the MoE FFN layer for a few tokens: the layer of
// moe_kernels.hip on the same packed Q4 blob, for the one-token steps after a prompt.
//
//   route     top-k of the E logits (ties to the lower expert), w = softmax over the k;
//             a logit of -inf marks an expert that is not available: its slot has no
//             work and weight 0
//   gate/up   z = x [W_g | W_u]^T, h = z_g / (1 + exp(-z_g)) * z_u
//   down      dm = h W_d^T
//   combine   y[t] = sum_j w[t, j] dm[t, j], j ascending
//
// What bounds it: the bytes of the experts reached (0.5625 per weight); a token brings
// two operations per weight, far below the matrix cores' rate.  So the activations are
// carried with more bits than a quantised product would need: a block of 32 values is held
// as 24-bit integers times one power of two, split into three signed bytes ("limbs"), and the
// int8 matrix instruction multiplies the limbs with the 4-bit codes exactly.  The limbs of a
// few tokens share the rows of one instruction, which would idle otherwise.  Per 32-block the
// limb sums are joined and scaled into an fp32 accumulator.  A value is off by at most 1.01 * 2^-23 of
// its block's largest: bf16 x down to 2^-15 of it and fp16 x down to 2^-12 is exact.  (Two limbs
// for 16-bit types, 2^-15 of the largest: their error next to a large value is not hidden by the
// output's rounding where that value's weight is small.  A block's value 300 times the others, its
// weights smaller in proportion: 1e-3 of the output, six roundings of fp16.)
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "moe_decode.h"
#include "moe_dtype.h"
#include "moe_math.h"

namespace moe {

// The active-expert load of the prompt path (moe_kernels.hip).
__global__ __launch_bounds__(256) void k_expert_load(const uint8_t* __restrict__ src, uint8_t* __restrict__ dst,
                                                     const int32_t* __restrict__ counts, int E, uint64_t expert_bytes,
                                                     unsigned long long* __restrict__ stats);

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v16i __attribute__((ext_vector_type(16)));

namespace {

// -------------------------------------------------------------- fixed point ---
// Integers q of 24 bits in three limbs.  Exponent field of the scale of a block whose largest
// magnitude has the fp32 bits u: with E = that field, the value is q * 2^(E - 149) and
// |q| <= 0x7F7F7F, so that signed bytes hold it.  2^17 added to the mantissa moves the top 1/64
// of a binade to the next one (q would pass that).  E >= 23 keeps the scale normal: below a
// largest value of 2^-104 the last place stays at 2^-126.
constexpr int kLimbs = 3;
__device__ __forceinline__ int fix_exp(uint32_t u)
{
    const int e = (int)((u + (1u << 17)) >> 23);
    return e < 8 * kLimbs - 1 ? 8 * kLimbs - 1 : e;
}
// the block scale; NaN for a block that holds an infinity or a NaN
__device__ __forceinline__ float fix_scale(uint32_t u, int e)
{
    return u >= 0x7f800000u ? __builtin_nanf("") : __uint_as_float((uint32_t)(e - (8 * kLimbs - 2)) << 23);
}
__device__ __forceinline__ int fix_code(float v, int e) { return (int)__builtin_rintf(ldexpf(v, 125 + 8 * kLimbs - e)); }

// q = l0 + 256 l1 + 65536 l2 with signed bytes
__device__ __forceinline__ void limbs(int q, int (&l)[kLimbs])
{
    l[0] = (int8_t)q;
    q = (q - l[0]) >> 8;
    l[1] = (int8_t)q;
    l[2] = (q - l[1]) >> 8;
}

// Limb l of a chunk's token m is row 4 m + l of the instruction's 32 rows, so that a lane gets the
// limb sums of a (token, column) in neighbouring result registers: register quad i of lane half h
// holds rows 8 i + 4 h .. 8 i + 4 h + 3, token 2 i + h.
constexpr int kRowStep = 4;
constexpr int kPerHalf = kChunkRows / 2;                  // tokens of a lane half
static_assert(kPerHalf * 2 == kChunkRows && kChunkRows * kRowStep <= 32, "rows of one instruction");

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }
__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// ------------------------------------------------------------------ routing ---
// Keys order the logits (larger first), -0 as +0; equal keys go to the lower expert: the
// order of the prompt path's routing.  Never 0, which marks a taken slot.
__device__ __forceinline__ uint32_t route_key(float v)
{
    uint32_t u = v == 0.0f ? 0u : __float_as_uint(v);
    u = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
    return u ? u : 1u;
}
constexpr uint32_t kKeyMinusInf = 0x007fffffu;            // route_key(-inf)

// Reductions over a wave by lane moves inside the VALU (a shuffle through LDS takes ten times
// as long, and a token's routing is a chain of them).  The result is on every lane.
template <int kCtrl>
__device__ __forceinline__ uint32_t dpp0(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kCtrl, 0xf, 0xf, false);
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v)
{
    v = umax(v, dpp0<0x111>(v));                          // row_shr 1, 2, 4, 8: rows of 16 lanes
    v = umax(v, dpp0<0x112>(v));
    v = umax(v, dpp0<0x114>(v));
    v = umax(v, dpp0<0x118>(v));
    v = umax(v, dpp0<0x142>(v));                          // row_bcast 15, 31: row into the next
    v = umax(v, dpp0<0x143>(v));
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
__device__ __forceinline__ float add_dpp(float v, uint32_t moved) { return v + __uint_as_float(moved); }
__device__ __forceinline__ float wave_sum(float v)
{
    v = add_dpp(v, dpp0<0x111>(__float_as_uint(v)));
    v = add_dpp(v, dpp0<0x112>(__float_as_uint(v)));
    v = add_dpp(v, dpp0<0x114>(__float_as_uint(v)));
    v = add_dpp(v, dpp0<0x118>(__float_as_uint(v)));
    v = add_dpp(v, dpp0<0x142>(__float_as_uint(v)));
    v = add_dpp(v, dpp0<0x143>(__float_as_uint(v)));
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), 63));
}

// One token by one wave: slot(j, e, key) for its first k slots; e = -1: not available.
template <int NK, class F>   // keys per lane: E <= 64 * NK
__device__ __forceinline__ void route_token(const float* __restrict__ lt, int E, int k, F slot)
{
    const int lane = threadIdx.x & 63;
    uint32_t key[NK];
#pragma unroll
    for (int i = 0; i < NK; ++i) {
        const int e = lane + 64 * i;
        const uint32_t u = route_key(lt[e < E ? e : E - 1]);
        key[i] = e < E ? u : 0u;
    }
    for (int j = 0; j < k; ++j) {
        uint32_t m = key[0];
#pragma unroll
        for (int i = 1; i < NK; ++i) m = umax(m, key[i]);
        m = wave_max(m);
        // the lowest expert that holds it: experts lane + 64 i, so the lowest i, then lane
        int e = -1;
#pragma unroll
        for (int i = NK - 1; i >= 0; --i) {
            const uint64_t has = __ballot(key[i] == m);
            e = has ? 64 * i + (int)__builtin_ctzll(has) : e;
        }
#pragma unroll
        for (int i = 0; i < NK; ++i) key[i] = lane + 64 * i == e ? 0u : key[i];
        slot(j, m == kKeyMinusInf ? -1 : e, m);
    }
}

// the logit of a key
__device__ __forceinline__ float key_logit(uint32_t u)
{
    return __uint_as_float((u & 0x80000000u) ? (u & 0x7fffffffu) : ~u);
}

// Weights of one token's k slots by one wave, from the experts (-1: weight 0) and the logits in
// z (LDS), which they replace: softmax over the available ones; all 0 where there is none.
__device__ __forceinline__ void route_weights(int k, const int* eidx, float* z)
{
    const int lane = threadIdx.x & 63;
    __builtin_amdgcn_wave_barrier();
    const float top = z[0];
    float part = 0.0f;
    for (int j = lane; j < k; j += 64) part += eidx[j] < 0 ? 0.0f : exp_cw(z[j] - top);
    const float sum = wave_sum(part);
    for (int j = lane; j < k; j += 64) z[j] = eidx[j] < 0 ? 0.0f : exp_cw(z[j] - top) / sum;
    __builtin_amdgcn_wave_barrier();
}

constexpr int kRouteThreads = 1024;
constexpr int kRouteWaves = kRouteThreads / 64;
constexpr int kMaxE = 1024;

struct RouteArgs {
    const float* logits;
    int64_t logits_stride;
    int T, E, k;
    int32_t* eidx;
    float* wts;
    int32_t* counts;
    int32_t* nchunks;
    DecodeChunk* chunks;
    int32_t* eidx_out;
    float* wts_out;
    const void* x;
    int64_t x_stride;
    int d;
    int8_t* xl;
    float* xs;
};

// Workgroup 0 routes every token (a token per wave at a time) and lists the chunks: per
// expert its pairs in groups of kChunkRows.  A pair's row inside its chunk depends on
// the order of LDS atomics; nothing else does, since every row is computed by itself.
__device__ __forceinline__ void route_all(const RouteArgs& a)
{
    __shared__ int s_eidx[kDecodeMaxPairs];
    __shared__ float s_z[kDecodeMaxPairs];
    __shared__ int s_cnt[kMaxE], s_first[kMaxE], s_fill[kMaxE];
    __shared__ int s_wave[kRouteWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int R = a.T * a.k;
    s_cnt[tid] = 0;
    s_fill[tid] = 0;
    for (int t = wave; t < a.T; t += kRouteWaves) {
        const float* lt = a.logits + (int64_t)t * a.logits_stride;
        int* te = s_eidx + t * a.k;
        float* tz = s_z + t * a.k;
        auto slot = [&](int j, int e, uint32_t key) {
            if (lane == 0) {
                te[j] = e;
                tz[j] = key_logit(key);
            }
        };
        if (a.E <= 128)
            route_token<2>(lt, a.E, a.k, slot);
        else if (a.E <= 256)
            route_token<4>(lt, a.E, a.k, slot);
        else
            route_token<16>(lt, a.E, a.k, slot);
        route_weights(a.k, te, tz);
    }
    __syncthreads();
    const int e_of = tid < R ? s_eidx[tid] : -1;          // R <= kRouteThreads
    if (tid < R) {
        a.eidx[tid] = e_of;
        a.wts[tid] = s_z[tid];
        if (a.eidx_out) a.eidx_out[tid] = e_of;
        if (a.wts_out) a.wts_out[tid] = s_z[tid];
        if (e_of >= 0) atomicAdd(&s_cnt[e_of], 1);
    }
    __syncthreads();
    const int c = tid < a.E ? s_cnt[tid] : 0;
    const int nc = (c + kChunkRows - 1) / kChunkRows;
    int incl = nc;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int y = __shfl_up(incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 63) s_wave[wave] = incl;
    __syncthreads();
    int before = 0, total = 0;
    for (int i = 0; i < kRouteWaves; ++i) {
        before += i < wave ? s_wave[i] : 0;
        total += s_wave[i];
    }
    const int first = before + incl - nc;
    s_first[tid] = first;
    if (tid < a.E) {
        a.counts[tid] = c;
        for (int i = 0; i < nc; ++i) {
            a.chunks[first + i].expert = tid;
            a.chunks[first + i].n = c - i * kChunkRows < kChunkRows ? c - i * kChunkRows : kChunkRows;
        }
    }
    if (tid == 0) *a.nchunks = total;
    __syncthreads();
    if (e_of >= 0) {
        const int r = atomicAdd(&s_fill[e_of], 1);
        a.chunks[s_first[e_of] + r / kChunkRows].pair[r % kChunkRows] = tid;
    }
}

// Four values of a block of 32 by each of 8 lanes: their limbs as a word per plane, and the
// block's scale.
__device__ __forceinline__ void block_to_fixed(const float (&v)[4], uint32_t (&w)[kLimbs], float& scale)
{
    uint32_t u = umax(umax(abs_bits(v[0]), abs_bits(v[1])), umax(abs_bits(v[2]), abs_bits(v[3])));
    u = umax(u, dpp0<0xB1>(u));                           // quad_perm: lane ^ 1
    u = umax(u, dpp0<0x4E>(u));                           // quad_perm: lane ^ 2
    u = umax(u, dpp0<0x141>(u));                          // row_half_mirror: the other quad of the 8
    const int e = fix_exp(u);
    w[0] = w[1] = w[2] = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        int l[kLimbs];
        limbs(u >= 0x7f800000u ? 0 : fix_code(v[i], e), l);
#pragma unroll
        for (int j = 0; j < kLimbs; ++j) w[j] |= (uint32_t)(l[j] & 0xff) << (8 * i);
    }
    scale = fix_scale(u, e);
}

// x in fixed point: 8 lanes per block of 32, limb plane l of token t at xl[(3 t + l) d].
template <int kT>
__device__ __forceinline__ void x_to_fixed(const RouteArgs& a, int64_t first)
{
    const int nb = a.d / 32;
    const int64_t blk = first + (threadIdx.x >> 3);
    if (blk >= (int64_t)a.T * nb) return;                 // uniform over the 8-lane group
    const int sub = threadIdx.x & 7;
    const int t = (int)((uint32_t)blk / (uint32_t)nb), b = (int)blk - t * nb;
    float v[4], scale;
    uint32_t w[kLimbs];
    load_n<kT, 4>(static_cast<const uint8_t*>(a.x) +
                  ((int64_t)t * a.x_stride + b * 32 + sub * 4) * dtype_bytes(kT), v);
    block_to_fixed(v, w, scale);
#pragma unroll
    for (int j = 0; j < kLimbs; ++j)
        *reinterpret_cast<uint32_t*>(a.xl + ((int64_t)t * kLimbs + j) * a.d + b * 32 + sub * 4) = w[j];
    if (sub == 0) a.xs[(int64_t)t * nb + b] = scale;
}

template <int kT>
__global__ __launch_bounds__(kRouteThreads) void k_decode_route(RouteArgs a)
{
    if (blockIdx.x == 0) {
        route_all(a);
        return;
    }
    x_to_fixed<kT>(a, (int64_t)(blockIdx.x - 1) * (kRouteThreads / 8));
}

// ---------------------------------------------------------- expert products ---
// Eight codes of a word as bytes holding 16 x the weight (see moe_kernels.hip's grouped
// GEMM: the code with its top bit flipped is the weight in 4-bit two's complement).
__device__ __forceinline__ v4i unpack16x(uint32_t w0, uint32_t w1)
{
    v4i b;
    b.x = (int)(((w0 << 4) & 0xF0F0F0F0u) ^ 0x80808080u);
    b.y = (int)((w0 & 0xF0F0F0F0u) ^ 0x80808080u);
    b.z = (int)(((w1 << 4) & 0xF0F0F0F0u) ^ 0x80808080u);
    b.w = (int)((w1 & 0xF0F0F0F0u) ^ 0x80808080u);
    return b;
}

// Where one wave reads the weights: this lane's words of tile 0, tile t further by *_step.
struct WeightAt {
    const uint8_t* q;
    const uint8_t* s;
    int64_t q_step, s_step;
};
__device__ __forceinline__ WeightAt weights_at(const uint8_t* expert, uint64_t q_off, uint64_t s_off, int tile, int K)
{
    const int lane = threadIdx.x & 63, npairs = k_pairs(K), ngroups = scale_groups(K);
    return {expert + q_off + (uint64_t)tile * npairs * 1024 + lane * 16,
            expert + s_off + ((uint64_t)tile * ngroups * 32 + (lane & 31)) * 16, (int64_t)npairs * 1024,
            (int64_t)ngroups * 512};
}

// The weights of U K pairs of NT 32-column tiles in registers, all in flight at first; a pair's
// registers take the pair U further as soon as it is used, so that U * NT KiB a wave stay in
// flight.
template <int NT, int U>
struct Ring {
    uint4 q[U][NT];
    uint32_t s[U][NT];        // the scales of the pair's two blocks for this lane's column

    __device__ __forceinline__ void load(int u, const WeightAt& w, int pr)
    {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            q[u][t] = *reinterpret_cast<const uint4*>(w.q + t * w.q_step + (int64_t)pr * 1024);
            s[u][t] = *reinterpret_cast<const uint32_t*>(w.s + t * w.s_step + (pr >> 2) * 512 + (pr & 3) * 4);
        }
    }
    __device__ __forceinline__ void fill(const WeightAt& w, int p0, int p1)
    {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (p0 + u < p1) load(u, w, p0 + u);          // uniform
    }
};

// acc[t][i] += block b's products for token i of this lane half: q = 0 / 1, the first / second
// block of ring slot u.
//   a          the 16 bytes of the block that this lane feeds
//   scl(i, b)  the scale of that token's block
template <int kTok, int NT, int U, class Scl>
__device__ __forceinline__ void block_product(float (&acc)[NT][kTok], const Ring<NT, U>& r, int u, int q, v4i a, int b, Scl scl)
{
    const v16i zero = {0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
    v16i s[NT];
    float ws[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const v4i w = q ? unpack16x(r.q[u][t].z, r.q[u][t].w) : unpack16x(r.q[u][t].x, r.q[u][t].y);
        s[t] = __builtin_amdgcn_mfma_i32_32x32x32_i8(a, w, zero, 0, 0, 0);
        const uint16_t hb = (uint16_t)(q ? r.s[u][t] >> 16 : r.s[u][t] & 0xffffu);
        ws[t] = (float)__builtin_bit_cast(_Float16, hb) * 0.0625f;
    }
#pragma unroll
    for (int i = 0; i < kTok; ++i) {
        const float x = scl(i, b);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            // 16 x the limb sums; s0 + 256 s1 is a multiple of 16 below 2^28: exact in fp32
            const float low = (float)(s[t][4 * i] + (s[t][4 * i + 1] << 8));
            const float v = __builtin_fmaf((float)s[t][4 * i + 2], 65536.0f, low);
            acc[t][i] = __builtin_fmaf(v, ws[t] * x, acc[t][i]);
        }
    }
    __builtin_amdgcn_sched_barrier(0);                    // one block's sums at a time in registers
}

// K pairs [p0, p1) of a filled ring, the activations in LDS: act(b) gives the bytes of block b
// that this lane feeds.
template <int kTok, int NT, int U, class Act, class Scl>
__device__ __forceinline__ void ring_product(float (&acc)[NT][kTok], Ring<NT, U>& r, const WeightAt& w, int p0, int p1,
                                             int nb, Act act, Scl scl)
{
    for (int pb = p0; pb < p1; pb += U) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int pr = pb + u;
            if (pr >= p1) break;                          // uniform
            block_product<kTok>(acc, r, u, 0, act(2 * pr), 2 * pr, scl);
            // the padded block of an odd count is left out
            if (2 * pr + 1 < nb) block_product<kTok>(acc, r, u, 1, act(2 * pr + 1), 2 * pr + 1, scl);
            if (pr + U < p1) r.load(u, w, pr + U);
        }
    }
}

struct GateUpArgs {
    RouteArgs r;              // routing and x
    const int32_t* nchunks;
    const DecodeChunk* chunks;
    const uint8_t* blob;
    uint64_t expert_stride, q_off, s_off;
    int8_t* hl;               // h in fixed point: limb plane l of pair p at hl[(3 p + l) f]
    float* hs;                // its block scales [pairs][f / 32]
    int f;
};

// h = silu(gate) * up of pair p, 32 columns by a 32-lane half, in fixed point.
__device__ __forceinline__ void store_h(const GateUpArgs& g, int p, int fb, float gate, float up)
{
    const int j32 = threadIdx.x & 31;
    const float hv = gate / (1.0f + exp_cw(-gate)) * up;
    uint32_t u = abs_bits(hv);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) u = umax(u, (uint32_t)__shfl_xor((int)u, o));
    const int e = fix_exp(u);
    int l[kLimbs];
    limbs(u >= 0x7f800000u ? 0 : fix_code(hv, e), l);
    int8_t* o = g.hl + (int64_t)p * kLimbs * g.f + fb * 32 + j32;
#pragma unroll
    for (int i = 0; i < kLimbs; ++i) o[i * g.f] = (int8_t)l[i];
    if (j32 == 0) g.hs[(int64_t)p * (g.f / 32) + fb] = fix_scale(u, e);
}

// ------------------------------------------------------- few pairs: gate/up ---
// Workgroup (f-block, pair) finds its pair's expert itself -- every wave routes the token, in
// registers -- and turns the token's x into fixed point in LDS, so that no launch comes before
// it.  Pairs of the same expert each read its weights (from a cache).  The workgroups of
// f-block 0 and slot 0 leave the token's routing for the next kernel.
//
// One token, 8 experts of d = 2048, f = 768 (14 MB): 7.6 us, of which the weights' bytes are 3;
// the rest is the launch, the logits' way and eight slots' routing, the sums.  d = 4096,
// f = 1536 (57 MB): 14.8 us, 3.8 TB/s.
template <int kT, int kPairWaves>
__global__ __launch_bounds__(64 * kPairWaves) void k_decode_pair_gate_up(GateUpArgs g)
{
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];   // xl [3][d], then xs [d / 32]
    __shared__ float s_red[kPairWaves][2][32];
    __shared__ int s_eidx[kMaxE];
    __shared__ float s_z[kMaxE];
    const RouteArgs& r = g.r;
    const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5, j32 = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int p = blockIdx.y, t = p / r.k, j = p - t * r.k, fb = blockIdx.x;
    const int d = r.d, nb = d / 32, npairs = k_pairs(d);
    int8_t* xl = reinterpret_cast<int8_t*>(lds);
    float* xs = reinterpret_cast<float*>(lds + kLimbs * d);
    const bool record = fb == 0 && j == 0;                // uniform
    const float* lt = r.logits + (int64_t)t * r.logits_stride;

    int e = -1;
    auto slot = [&](int jj, int ee, uint32_t key) {
        if (jj == j) e = ee;
        if (record && wave == 0 && lane == 0) {
            s_eidx[jj] = ee;
            s_z[jj] = key_logit(key);
        }
    };
    const int slots = record && wave == 0 ? r.k : j + 1;
    if (r.E <= 128)
        route_token<2>(lt, r.E, slots, slot);
    else if (r.E <= 256)
        route_token<4>(lt, r.E, slots, slot);
    else
        route_token<16>(lt, r.E, slots, slot);
    e = __builtin_amdgcn_readfirstlane(e);
    const int p0 = wave * npairs / kPairWaves, p1 = (wave + 1) * npairs / kPairWaves;
    const WeightAt w = weights_at(g.blob + (uint64_t)(e < 0 ? 0 : e) * g.expert_stride, g.q_off, g.s_off, 2 * fb, d);
    Ring<2, 4> ring;
    if (e >= 0) ring.fill(w, p0, p1);                     // in flight while x is turned
    if (record && wave == 0) {
        route_weights(r.k, s_eidx, s_z);
        for (int i = lane; i < r.k; i += 64) {
            r.eidx[p + i] = s_eidx[i];
            r.wts[p + i] = s_z[i];
            if (r.eidx_out) r.eidx_out[p + i] = s_eidx[i];
            if (r.wts_out) r.wts_out[p + i] = s_z[i];
        }
    }
    if (e < 0) return;                                    // the same on every wave

    for (int blk = tid >> 3; blk < nb; blk += 64 * kPairWaves / 8) {
        const int sub = tid & 7;
        float v[4], scale;
        uint32_t x[kLimbs];
        load_n<kT, 4>(static_cast<const uint8_t*>(r.x) +
                      ((int64_t)t * r.x_stride + blk * 32 + sub * 4) * dtype_bytes(kT), v);
        block_to_fixed(v, x, scale);
#pragma unroll
        for (int l = 0; l < kLimbs; ++l) *reinterpret_cast<uint32_t*>(xl + l * d + blk * 32 + sub * 4) = x[l];
        if (sub == 0) xs[blk] = scale;
    }
    __syncthreads();

    auto act = [&](int b) -> v4i {
        v4i a = {0, 0, 0, 0};
        if (j32 < kLimbs) a = *reinterpret_cast<const v4i*>(xl + j32 * d + b * 32 + 16 * h);
        return a;
    };
    float acc[2][1] = {};
    if (p0 < p1) ring_product<1>(acc, ring, w, p0, p1, nb, act, [&](int, int b) { return xs[b]; });
    if (h == 0) {
        s_red[wave][0][j32] = acc[0][0];
        s_red[wave][1][j32] = acc[1][0];
    }
    __syncthreads();
    if (tid >= 32) return;
    float z[2] = {};
#pragma unroll
    for (int v = 0; v < kPairWaves; ++v) {
        z[0] += s_red[v][0][j32];
        z[1] += s_red[v][1][j32];
    }
    store_h(g, p, fb, z[0], z[1]);
}

// ----------------------------------------------------- chunks: gate/up, down ---
struct DownArgs {
    const int32_t* nchunks;   // null: pair p is the chunk of itself
    const DecodeChunk* chunks;
    const int32_t* eidx;
    const float* wts;
    const uint8_t* blob;
    uint64_t expert_stride, q_off, s_off;
    const int8_t* hl;
    const float* hs;
    int T, k, d, f, ksplit;
    float* dm;                // [pairs][d]; not written for a pair without an expert
    void* y;
    int64_t y_stride;
};

struct ChunkArgs {
    GateUpArgs g;
    DownArgs d;
};

// LDS of a chunk kernel: the rows' activations (rows kPad apart in bank groups), their block
// scales.
constexpr int kActPad = 32;
constexpr int chunk_lds(int K) { return kChunkRows * (kLimbs * (K + kActPad) + K / 32 * 4); }

// Rows that share an expert's weights: a chunk of the route kernel's list (up to kChunkRows), or a
// pair by itself.  A workgroup takes a chunk by two 32-column tiles -- the gate and the up tile of
// an f-block, or two tiles of the down matrix -- its waves split K and add up through LDS.  A
// fixed number of workgroups goes through the items, since only the device knows how many there
// are; the chunks of an expert follow each other at a multiple of 8 workgroups, so that one XCD
// reads a tile for all of them (the first from memory, the others from its L2).
//
// 24 tokens of d = 4096, f = 1536, skewed routing, some 36 of 256 experts reached (380 MB): gate/up 86 us,
// down 53; of alike routing, 137 experts (1.4 GB): 169 and 96.  The first is bound by the expansion of the codes
// and the sums' join, paid again for every chunk of an expert, the second by memory (5.5 TB/s).
constexpr int kChunkWaves = 4;

template <bool kGateUp>
__global__ __launch_bounds__(64 * kChunkWaves) __attribute__((amdgpu_waves_per_eu(4))) void k_decode_chunk(ChunkArgs a)
{
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    __shared__ float s_red[kChunkWaves][2][kChunkRows][32];
    const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5, j32 = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int K = kGateUp ? a.g.r.d : a.d.f, nb = K / 32, npairs = k_pairs(K);
    const int tiles = kGateUp ? a.g.f / 32 * 2 : a.d.d / 32, tile2 = (tiles + 1) / 2, stride = (tile2 + 7) & ~7;
    const int32_t* nchunks = kGateUp ? a.g.nchunks : a.d.nchunks;
    const int items = (nchunks ? *nchunks : a.d.T * a.d.k) * stride;
    const int p0 = wave * npairs / kChunkWaves, p1 = (wave + 1) * npairs / kChunkWaves;
    int8_t* s_act = reinterpret_cast<int8_t*>(lds);
    float* s_scale = reinterpret_cast<float*>(lds + kChunkRows * kLimbs * (K + kActPad));
    const int8_t* acts = kGateUp ? a.g.r.xl : a.d.hl;
    const float* scales = kGateUp ? a.g.r.xs : a.d.hs;

    for (int it = blockIdx.x; it < items; it += gridDim.x) {
        const int ci = it / stride, nt = 2 * (it - ci * stride);
        if (nt >= tiles) continue;
        const DecodeChunk* ch = (kGateUp ? a.g.chunks : a.d.chunks) + ci;
        const int e = nchunks ? ch->expert : a.d.eidx[ci], n = nchunks ? ch->n : 1;
        if (e < 0) continue;
        const bool two = nt + 1 < tiles;
        WeightAt w = weights_at(kGateUp ? a.g.blob + (uint64_t)e * a.g.expert_stride : a.d.blob + (uint64_t)e * a.d.expert_stride,
                                kGateUp ? a.g.q_off : a.d.q_off, kGateUp ? a.g.s_off : a.d.s_off, nt, K);
        if (!two) w.q_step = w.s_step = 0;                // an odd count's last tile twice, stored once
        Ring<2, 4> ring;
        ring.fill(w, p0, p1);                             // in flight while the activations are staged
        int pair[kChunkRows];
#pragma unroll
        for (int m = 0; m < kChunkRows; ++m) pair[m] = nchunks ? ch->pair[m < n ? m : 0] : ci;
        __syncthreads();                                  // the previous item's LDS is read
#pragma unroll
        for (int m = 0; m < kChunkRows; ++m) {
            if (m >= n) break;                            // uniform
            const int64_t src = kGateUp ? pair[m] / a.g.r.k : pair[m];
            for (int i = tid * 16; i < kLimbs * K; i += 64 * kChunkWaves * 16) {
                const int l = (i >= K) + (i >= 2 * K);    // K is a multiple of 32: a piece is in one plane
                *reinterpret_cast<uint4*>(s_act + (m * kLimbs + l) * (K + kActPad) + i - l * K) =
                    *reinterpret_cast<const uint4*>(acts + src * kLimbs * K + i);
            }
            for (int i = tid; i < nb; i += 64 * kChunkWaves) s_scale[m * nb + i] = scales[src * nb + i];
        }
        __syncthreads();
        const int m_a = j32 / kRowStep, l_a = j32 % kRowStep;           // the A row this lane feeds
        const bool on = m_a < n && l_a < kLimbs;
        const int8_t* al = s_act + (m_a * kLimbs + l_a) * (K + kActPad) + 16 * h;
        auto act = [&](int b) -> v4i {
            v4i v = {0, 0, 0, 0};
            if (on) v = *reinterpret_cast<const v4i*>(al + b * 32);
            return v;
        };
        // an absent token's column is not stored: whatever its place in the array holds will do
        const float* xs = s_scale + h * nb;
        float acc[2][kPerHalf] = {};
        if (p0 < p1)
            ring_product<kPerHalf>(acc, ring, w, p0, p1, nb, act, [&](int i, int b) { return xs[2 * i * nb + b]; });
#pragma unroll
        for (int i = 0; i < kPerHalf; ++i) {
            s_red[wave][0][2 * i + h][j32] = acc[0][i];
            s_red[wave][1][2 * i + h][j32] = acc[1][i];
        }
        __syncthreads();
        // gate/up: row m by a half wave; down: row m's tile t by a half wave
        if (kGateUp) {
            const int m = tid >> 5;
            if (m < n) {                                  // uniform over the 32-lane half
                float z[2] = {};
#pragma unroll
                for (int v = 0; v < kChunkWaves; ++v) {
                    z[0] += s_red[v][0][m][j32];
                    z[1] += s_red[v][1][m][j32];
                }
                store_h(a.g, nchunks ? ch->pair[m] : ci, nt >> 1, z[0], z[1]);
            }
        } else {
            const int m = tid >> 6, t = (tid >> 5) & 1;
            if (m < n && (t == 0 || two)) {
                float z = 0.0f;
#pragma unroll
                for (int v = 0; v < kChunkWaves; ++v) z += s_red[v][t][m][j32];
                a.d.dm[(int64_t)(nchunks ? ch->pair[m] : ci) * a.d.d + (nt + t) * 32 + j32] = z;
            }
        }
        static_assert(kChunkRows <= kChunkWaves, "a wave per row");
    }
}

// ------------------------------------------- few pairs: down and combine in one ---
// A workgroup owns 32 columns of y for all tokens.  Its 16 waves take the (pair, K split) units
// in turn, the pairs' h in LDS, and leave the units' rows there, where each token's slots are
// added up in slot order.  One token, 4 experts of d = 2048, f = 768 (3.5 MB): 5.1 us; 8 of d = 2048, f = 512
// (4.7 MB): 5.6; 4 of d = 4096, f = 1536 (14 MB): 7.8 us; a chain of the first bytes' latency, the ring and
// two passes through LDS, since its d / 32 workgroups leave CUs idle.
constexpr int kPairDownWaves = 16;
constexpr int kFusedPairs = 8;                            // pairs, at most

struct PairDownLds {
    int hl, hs, dm, bytes;
    MOE_HD PairDownLds(int R, int f, int ksplit)
    {
        hl = 0;
        hs = R * kLimbs * f;
        dm = hs + R * (f / 32) * 4;
        bytes = dm + R * ksplit * 32 * 4;
    }
};

template <int kT>
__global__ __launch_bounds__(64 * kPairDownWaves) void k_decode_pair_down(DownArgs g)
{
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    __shared__ float s_w[kFusedPairs];
    const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5, j32 = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int R = g.T * g.k, nb = g.f / 32, npairs = k_pairs(g.f), nt = blockIdx.x;
    const PairDownLds L(R, g.f, g.ksplit);
    int8_t* s_hl = reinterpret_cast<int8_t*>(lds);
    float* s_hs = reinterpret_cast<float*>(lds + L.hs);
    float* s_dm = reinterpret_cast<float*>(lds + L.dm);   // [ksplit][pairs][32]

    const int units = R * g.ksplit;
    Ring<1, 6> ring;
    WeightAt w{};
    int e = -1, p0 = 0, p1 = 0;
    auto open = [&](int u) {                              // unit u's weights on their way
        const int p = u / g.ksplit, ks = u - p * g.ksplit;
        e = g.eidx[p];
        p0 = ks * npairs / g.ksplit;
        p1 = (ks + 1) * npairs / g.ksplit;
        w = weights_at(g.blob + (uint64_t)(e < 0 ? 0 : e) * g.expert_stride, g.q_off, g.s_off, nt, g.f);
        if (e >= 0) ring.fill(w, p0, p1);
    };
    if (wave < units) open(wave);
    if (tid < R) s_w[tid] = g.wts[tid];
    for (int i = tid * 16; i < L.hs; i += 64 * kPairDownWaves * 16)   // 3 R f: a multiple of 32
        *reinterpret_cast<uint4*>(s_hl + i) = *reinterpret_cast<const uint4*>(g.hl + i);
    for (int i = tid; i < R * nb; i += 64 * kPairDownWaves) s_hs[i] = g.hs[i];
    __syncthreads();
    for (int u = wave; u < units; u += kPairDownWaves) {
        if (u != wave) open(u);
        const int p = u / g.ksplit, ks = u - p * g.ksplit;
        float acc[1][1] = {};
        if (e >= 0) {
            const int8_t* al = s_hl + (p * kLimbs + j32) * g.f + 16 * h;
            auto act = [&](int b) -> v4i {
                v4i a = {0, 0, 0, 0};
                if (j32 < kLimbs) a = *reinterpret_cast<const v4i*>(al + b * 32);
                return a;
            };
            ring_product<1>(acc, ring, w, p0, p1, nb, act, [&](int, int b) { return s_hs[p * nb + b]; });
        }
        if (h == 0) s_dm[(ks * R + p) * 32 + j32] = acc[0][0];
    }
    __syncthreads();
    typedef typename Elem<kT>::type E;
    for (int i = tid; i < g.T * 32; i += 64 * kPairDownWaves) {
        const int t = i >> 5, col = i & 31;
        float a = 0.0f;
        for (int j = 0; j < g.k; ++j) {
            const int p = t * g.k + j;
            float v = 0.0f;                               // 0 with weight 0 where there is no expert
            for (int ks = 0; ks < g.ksplit; ++ks) v += s_dm[(ks * R + p) * 32 + col];
            a = __builtin_fmaf(s_w[p], v, a);
        }
        static_cast<E*>(g.y)[(int64_t)t * g.y_stride + nt * 32 + col] = from_f32<kT>(a);
    }
}

// ------------------------------------------------------------------ combine ---
// y[t] = sum over j of w[t, j] dm[t, j].  Eight slots' rows, weights and experts are loaded
// together, none of them waiting for another: a slot without an expert reads its row too (it
// holds what the workspace held) and drops it.
template <int kT>
__global__ __launch_bounds__(256) void k_decode_combine(const float* __restrict__ dm,
                                                        const float* __restrict__ wts,
                                                        const int32_t* __restrict__ eidx, int k,
                                                        int d, void* __restrict__ y, int64_t y_stride)
{
    const int t = blockIdx.y, c = ((int)blockIdx.x * 256 + (int)threadIdx.x) * 4;
    if (c >= d) return;
    float acc[4] = {};
    for (int j0 = 0; j0 < k; j0 += 8) {
        float4 v[8];
        float w[8];
        int e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int p = t * k + (j0 + i < k ? j0 + i : k - 1);
            v[i] = *reinterpret_cast<const float4*>(dm + (int64_t)p * d + c);
            w[i] = wts[p];
            e[i] = eidx[p];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (j0 + i >= k || e[i] < 0) continue;        // uniform
            acc[0] = __builtin_fmaf(w[i], v[i].x, acc[0]);
            acc[1] = __builtin_fmaf(w[i], v[i].y, acc[1]);
            acc[2] = __builtin_fmaf(w[i], v[i].z, acc[2]);
            acc[3] = __builtin_fmaf(w[i], v[i].w, acc[3]);
        }
    }
    store_n<kT, 4>(static_cast<uint8_t*>(y) + ((int64_t)t * y_stride + c) * dtype_bytes(kT), acc);
}

unsigned nblk(int64_t n, int per) { return (unsigned)((n + per - 1) / per); }

}  // namespace

// ----------------------------------------------------------------- launches ---
namespace {

// Pairs by themselves need no route kernel, but those that share an expert read its weights again,
// from a cache.  With experts drawn alike the re-reads are (R - D) experts' bytes, D = E (1 - (1 - k / E)^T)
// the experts reached; about 100 MB of them cost what the route kernel does, whatever the sizes.  Pairs
// against chunks: 4096 x 1536, 8 of 256 experts, 8 tokens (70 MB) 121 us, 122, 12 tokens (158 MB) 171, 166; 8 of
// 32, 3 tokens (58 MB) 46.5, 49.5, 5 tokens (166 MB) 69, 61; 2048 x 768, 8 of 16, 6 tokens (86 MB) 25.7, 26.8,
// 8 tokens (128 MB) 30.5, 30.0; 8 of 128, 16 tokens (121 MB) 59, 57; 1024 x 512, 2 of 8, 48 tokens (78 MB) 20, 25.
constexpr double kPairReread = 100e6;
constexpr int kPairMost = 128;                            // as far as that was measured

// The fused down and combine (a workgroup a column tile) against a wave for every (pair, K split) of two
// tiles and a combine: it saves a launch, and its waves have more of K to go through.  Up to four pairs their K
// splits are the waves of one round; more win while there is little h.  The width of y does not matter.
// Fused, not: 2 pairs of 1024 x 768 9.1 us, 11.3, of 128 x 2048 10.2, 12.5; 4 pairs of 1024 x 1536 12.3, 13.8, of
// 2048 x 4096 21.5, 22.8; 7 pairs of 1024 x 768 (5376 values) 11.3, 11.5; 8 pairs of 2048 x 512 (4096) 13.8, 14.2,
// of 2048 x 768 (6144) 15.4, 15.2; 5 pairs of 1024 x 1536 (7680) 14.0, 13.8; 8 pairs of 4096 x 1536 28.1, 27.5, of
// 2048 x 4096 32, 27.
constexpr int kFusedH = 5632;                             // values of h of more than kFusedFew pairs
constexpr int kFusedFew = 4;
constexpr int kFusedLds = 64 << 10;                       // as far as that was measured

bool by_pairs(const DecodeLaunch& D)
{
    const int R = D.T * D.k;
    if (R > kPairMost || D.need_counts) return false;
    double missed = 1.0;                                  // the share of experts no token reaches
    for (int t = 0; t < D.T; ++t) missed *= 1.0 - (double)D.k / D.E;
    return (R - D.E * (1.0 - missed)) * (double)D.expert_stride <= kPairReread;
}

// K splits that give every wave of the fused down kernel a unit
int down_ksplit(const DecodeLaunch& D)
{
    const int R = D.T * D.k, np = k_pairs(D.f);
    int ks = 1;
    while (R * ks < kPairDownWaves && 2 * ks <= np && ks < 8) ks *= 2;
    return ks;
}

bool down_fused(const DecodeLaunch& D)
{
    const int R = D.T * D.k;
    return by_pairs(D) && R <= kFusedPairs && (R <= kFusedFew || R * D.f <= kFusedH) &&
           PairDownLds(R, D.f, down_ksplit(D)).bytes <= kFusedLds;
}

RouteArgs route_args(const DecodeLaunch& D)
{
    RouteArgs a;
    a.logits = D.logits;
    a.logits_stride = D.logits_stride;
    a.T = D.T;
    a.E = D.E;
    a.k = D.k;
    a.eidx = reinterpret_cast<int32_t*>(D.ws + D.L.eidx);
    a.wts = reinterpret_cast<float*>(D.ws + D.L.wts);
    a.counts = reinterpret_cast<int32_t*>(D.ws + D.L.counts);
    a.nchunks = reinterpret_cast<int32_t*>(D.ws + D.L.nchunks);
    a.chunks = reinterpret_cast<DecodeChunk*>(D.ws + D.L.chunks);
    a.eidx_out = D.eidx_out;
    a.wts_out = D.wts_out;
    a.x = D.x;
    a.x_stride = D.x_stride;
    a.d = D.d;
    a.xl = reinterpret_cast<int8_t*>(D.ws + D.L.xl);
    a.xs = reinterpret_cast<float*>(D.ws + D.L.xs);
    return a;
}

GateUpArgs gate_up_args(const DecodeLaunch& D)
{
    GateUpArgs g;
    g.r = route_args(D);
    g.nchunks = g.r.nchunks;
    g.chunks = g.r.chunks;
    g.blob = D.blob;
    g.expert_stride = D.expert_stride;
    g.q_off = D.gu_q_off;
    g.s_off = D.gu_s_off;
    g.hl = reinterpret_cast<int8_t*>(D.ws + D.L.hl);
    g.hs = reinterpret_cast<float*>(D.ws + D.L.hs);
    g.f = D.f;
    return g;
}

DownArgs down_args(const DecodeLaunch& D)
{
    DownArgs g;
    const bool pairs = by_pairs(D);
    g.nchunks = pairs ? nullptr : reinterpret_cast<const int32_t*>(D.ws + D.L.nchunks);
    g.chunks = reinterpret_cast<const DecodeChunk*>(D.ws + D.L.chunks);
    g.eidx = reinterpret_cast<const int32_t*>(D.ws + D.L.eidx);
    g.wts = reinterpret_cast<const float*>(D.ws + D.L.wts);
    g.blob = D.blob;
    g.expert_stride = D.expert_stride;
    g.q_off = D.d_q_off;
    g.s_off = D.d_s_off;
    g.hl = reinterpret_cast<const int8_t*>(D.ws + D.L.hl);
    g.hs = reinterpret_cast<const float*>(D.ws + D.L.hs);
    g.T = D.T;
    g.k = D.k;
    g.d = D.d;
    g.f = D.f;
    g.ksplit = down_ksplit(D);
    g.dm = reinterpret_cast<float*>(D.ws + D.L.dm);
    g.y = D.y;
    g.y_stride = D.y_stride;
    return g;
}

template <int kT>
hipError_t route_typed(const DecodeLaunch& D, hipStream_t st)
{
    if (by_pairs(D)) return hipSuccess;                   // the gate/up kernel routes
    const dim3 grid(1 + nblk((int64_t)D.T * (D.d / 32), kRouteThreads / 8));
    hipLaunchKernelGGL(k_decode_route<kT>, grid, dim3(kRouteThreads), 0, st, route_args(D));
    return hipGetLastError();
}

// The limit is the process's, for every thread that launches the kernel: always the most that any call
// needs (`most`), so that none can lower it between another's setting and launch.
constexpr int kMaxDim = 16384;                            // d and f, as the handle checked
constexpr int pair_lds(int d) { return kLimbs * d + d / 32 * 4; }
template <class K>
hipError_t lds_limit(K kernel, int bytes, int most)
{
    if (bytes <= 16 << 10) return hipSuccess;             // within the default limit next to the static arrays
    return hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, most);
}

// chunks: the most there can be; tile2: two-tile columns of the matrix
template <bool kGateUp>
hipError_t launch_chunk(const DecodeLaunch& D, int chunks, int K, int tile2, hipStream_t st)
{
    const int64_t items = (int64_t)chunks * align_up(tile2, 8);
    const int lds = chunk_lds(K);
    const hipError_t e = lds_limit(&k_decode_chunk<kGateUp>, lds, chunk_lds(kMaxDim));
    if (e != hipSuccess) return e;
    ChunkArgs a;
    a.g = gate_up_args(D);
    a.d = down_args(D);
    hipLaunchKernelGGL(k_decode_chunk<kGateUp>, dim3((unsigned)(items < 1024 ? items : 1024)), dim3(64 * kChunkWaves), lds, st, a);
    return hipGetLastError();
}

template <int kT>
hipError_t products_typed(const DecodeLaunch& D, hipStream_t st)
{
    hipError_t e = hipSuccess;
    if (by_pairs(D)) {
        const int lds = pair_lds(D.d);
        const dim3 grid(D.f / 32, D.T * D.k);
        // two workgroups of eight waves fill a CU, four of four: more than the first hold would
        // wait for a second round.  Fewer are done sooner by more waves, and so are any whose eight
        // waves have more than a ring of K pairs each.  The layer with eight waves, four: 2048 x 768, 8 of 128
        // experts, 1 token (192 workgroups) 15.3 us, 15.7, 2 tokens 18.4, 18.3, 3 tokens (576) 23.6, 22.3, 5
        // tokens 29.0, 27.5; 4096 x 1536, 8 of 256, 4 tokens (1536) 67, 69.5
        if (grid.x * grid.y > 512 && k_pairs(D.d) <= 8 * 4) {
            e = lds_limit(&k_decode_pair_gate_up<kT, 4>, lds, pair_lds(kMaxDim));
            if (e != hipSuccess) return e;
            hipLaunchKernelGGL((k_decode_pair_gate_up<kT, 4>), grid, dim3(64 * 4), lds, st, gate_up_args(D));
        } else {
            e = lds_limit(&k_decode_pair_gate_up<kT, 8>, lds, pair_lds(kMaxDim));
            if (e != hipSuccess) return e;
            hipLaunchKernelGGL((k_decode_pair_gate_up<kT, 8>), grid, dim3(64 * 8), lds, st, gate_up_args(D));
        }
    } else {
        e = launch_chunk<true>(D, D.L.max_chunks, D.d, D.f / 32, st);
        if (e != hipSuccess) return e;
    }
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    const DownArgs g = down_args(D);
    if (down_fused(D)) {
        const int lds = PairDownLds(D.T * D.k, D.f, g.ksplit).bytes;
        e = lds_limit(&k_decode_pair_down<kT>, lds, kFusedLds);
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL(k_decode_pair_down<kT>, dim3(D.d / 32), dim3(64 * kPairDownWaves), lds, st, g);
    } else {
        return launch_chunk<false>(D, by_pairs(D) ? D.T * D.k : D.L.max_chunks, D.f, (D.d / 32 + 1) / 2, st);
    }
    return hipGetLastError();
}

template <int kT>
hipError_t combine_typed(const DecodeLaunch& D, hipStream_t st)
{
    if (down_fused(D)) return hipSuccess;
    const DownArgs g = down_args(D);
    hipLaunchKernelGGL(k_decode_combine<kT>, dim3(nblk(D.d / 4, 256), D.T), dim3(256), 0, st, g.dm, g.wts, g.eidx, D.k, D.d, D.y,
                       D.y_stride);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_decode_route(const DecodeLaunch& D, hipStream_t st)
{
    return D.dtype == kF32 ? route_typed<kF32>(D, st) : D.dtype == kBF16 ? route_typed<kBF16>(D, st) : route_typed<kF16>(D, st);
}

hipError_t launch_decode_load(const DecodeLaunch& D, const uint8_t* src, uint8_t* dst, unsigned long long* stats, hipStream_t st)
{
    hipLaunchKernelGGL(k_expert_load, dim3(512), dim3(256), 0, st, src, dst, reinterpret_cast<const int32_t*>(D.ws + D.L.counts), D.E,
                       D.expert_stride, stats);
    return hipGetLastError();
}

hipError_t launch_decode_products(const DecodeLaunch& D, hipStream_t st)
{
    return D.dtype == kF32 ? products_typed<kF32>(D, st)
                           : D.dtype == kBF16 ? products_typed<kBF16>(D, st) : products_typed<kF16>(D, st);
}

hipError_t launch_decode_combine(const DecodeLaunch& D, hipStream_t st)
{
    return D.dtype == kF32 ? combine_typed<kF32>(D, st)
                           : D.dtype == kBF16 ? combine_typed<kBF16>(D, st) : combine_typed<kF16>(D, st);
}

}  // namespace moe
