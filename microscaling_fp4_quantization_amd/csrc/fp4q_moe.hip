// fp4q_moe.hip -- a mixture-of-experts layer for a few tokens (moe_layer).
//
// For at most 64 tokens x, experts e with quantized weights G_e, U_e (gate and up,
// inter x dim) and D_e (down, dim x inter):
//   l = x Wr^T;  the top_k largest of each token, with softmax weights p
//   h_e = silu(G_e x) * (U_e x);   y = sum_e p_e D_e h_e
//
// Three launches:
//  k_moe_route  router logits by 16 experts x 16 tokens x a range of K, on the bf16
//               matrix cores; the last workgroup to finish adds the ranges, picks the
//               tokens' experts and lists each expert's tokens (k_moe_plan: the list
//               alone, for a given routing);
//  k_moe_up     one workgroup per (expert in use, 16 rows of h): gate and up products
//               of the expert's tokens, K split over its waves, and silu(g) u;
//  k_moe_down   one workgroup per 16 rows of y: its waves share out the (expert, K
//               chunk) pairs in order, each adding into a tile of its own, and the
//               tiles meet in wave order.
// Sums are formed in a fixed order: the same inputs give the same bits.
//
// The layer is a pass over the weights of the experts in use.  They go from memory
// to registers, 16 rows x 128 elements per wave and step: lane l holds row l % 16
// and the 32 consecutive elements 32 (l / 16) of the step (16 bytes of 4-bit codes),
// and the token fragment is read the same way, so that every element meets its
// partner.  The weights are widened to bf16, which holds each exactly (an E2M1 value
// times a power of two or a UE4M3 scale, or an E4M3 value; per-tensor and tile
// scales are applied to the binary32 sums).  Activations that bf16 does not hold go
// as a sum of bf16 parts, each the rounding of what the ones before it leave: 3 for
// binary32 x (24 bits, all of it); h as 2 parts (16 bits: rounding it to one would
// add an error as large as a bf16 output's own) or 3 for a binary32 output.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <stdio.h>

#include <algorithm>

#include "fp4q_gemm_tile.h"
#include "fp4q_launch.h"

namespace fp4q {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v2f __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

constexpr int kMaxTokens = kMoeMaxTokens, kMaxExperts = kMoeMaxExperts, kMaxTopK = kMoeMaxTopK;
constexpr int kMaxPairs = kMaxTokens * kMaxTopK;
constexpr int kStep = 128;       // K elements per wave and step
constexpr int kRows = 16;        // weight rows per fragment
constexpr int kMx = 0, kNv = 1, kF8 = 2;  // weight formats

struct Weights {
    const uint8_t* codes;  // (experts * rows) x K, packed
    const void* scales;
    const float* g;        // NULL: 1
    int g_step;            // 1: one g per expert, 0: one for all
};

struct MoeParams {
    const void* x;
    int T, D, I, E, k;
    Weights w13, w2;
    const void* router;
    int renorm;
    int* ids;          // T x k
    float* wts;        // T x k
    void* y;
    int yt;            // 0 bf16, 1 f32
    uint32_t* count;   // workgroups of the router that are done, zero between calls
    struct Plan* plan;
    float* logits;     // ranges x T x E partial sums
    int ranges;        // K ranges of the router product
    uint16_t* h;       // parts x (T k) x I
};

__device__ __forceinline__ uint32_t load32(Rsrc r, int off) { return __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0); }
__device__ __forceinline__ u32x4_t load128(Rsrc r, int off) { return __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0); }

__device__ __forceinline__ v4f mma(bf16x8_t a, bf16x8_t b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// ---------------------------------------------------------------------------
// Operands: 32 elements of a lane as four fragments of 8.

struct Frag {
    bf16x8_t v[4];
};

__device__ __forceinline__ Frag frag_of(const u32x4_t (&w)[4]) {
    return Frag{{__builtin_bit_cast(bf16x8_t, w[0]), __builtin_bit_cast(bf16x8_t, w[1]),
                 __builtin_bit_cast(bf16x8_t, w[2]), __builtin_bit_cast(bf16x8_t, w[3])}};
}

// Binary32 as bf16 parts: what is left after a part is exact, so three parts hold
// all 24 bits of a value whose last bits do not fall below the smallest number.
// (An infinity or NaN leaves nothing.)
__device__ __forceinline__ float left(float f, uint32_t part) {
    return (part & 0x7F800000u) == 0x7F800000u ? 0.0f : f - __uint_as_float(part);
}
template <int P>
__device__ __forceinline__ void split8(const float (&f)[8], bf16x8_t (&out)[P]) {
    float rest[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) rest[e] = f[e];
#pragma unroll
    for (int p = 0; p < P; ++p) {
        u32x4_t w;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            w[q] = pack_bf16x2(rest[2 * q], rest[2 * q + 1]);
            rest[2 * q] = left(rest[2 * q], w[q] << 16);
            rest[2 * q + 1] = left(rest[2 * q + 1], w[q] & 0xFFFF0000u);
        }
        out[p] = __builtin_bit_cast(bf16x8_t, w);
    }
}

// 32 consecutive elements at element offset `at` (kDropped: zeros) of a window of
// bf16 (P = 1) or binary32 (P = 3) values, as P parts.
template <int P>
struct Act;
template <>
struct Act<1> {
    u32x4_t w[4];
    __device__ __forceinline__ void load(Rsrc r, int at) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = load128(r, at < 0 ? kDropped : at * 2 + 16 * i);
    }
    __device__ __forceinline__ void parts(Frag (&f)[1]) const { f[0] = frag_of(w); }
};
template <>
struct Act<3> {
    u32x4_t w[8];
    __device__ __forceinline__ void load(Rsrc r, int at) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = load128(r, at < 0 ? kDropped : at * 4 + 16 * i);
    }
    __device__ __forceinline__ void parts(Frag (&f)[3]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(w[2 * i + e / 4][e % 4]);
            bf16x8_t o[3];
            split8<3>(v, o);
            f[0].v[i] = o[0], f[1].v[i] = o[1], f[2].v[i] = o[2];
        }
    }
};

// 32 weights of a lane: codes, and the scales of its blocks.
template <int FMT>
struct Raw {
    u32x4_t w[FMT == kF8 ? 2 : 1];
    uint32_t s;
};

// A fragment row window: 16 rows of K elements with their scales, from global row
// `row0` of the stacked matrix.
template <int FMT>
struct Rows {
    Rsrc codes, scales;
    int K, kb;
    const float* tile;  // kF8: the tile scales of these rows, one per step
    __device__ __forceinline__ Rows(const Weights& w, int64_t row0, int K_) : K(K_) {
        const int rowb = FMT == kF8 ? K : K / 2;
        kb = FMT == kMx ? K / 32 : FMT == kNv ? K / 16 : (K + kStep - 1) / kStep;
        codes = make_rsrc(w.codes + row0 * rowb, (int64_t)kRows * rowb);
        if (FMT == kF8) tile = static_cast<const float*>(w.scales) + row0 / 128 * kb;
        else scales = make_rsrc(static_cast<const uint8_t*>(w.scales) + row0 * kb, (int64_t)kRows * kb);
    }
    // Step c of the lane of row r, quarter q; past K: zeros.
    __device__ __forceinline__ Raw<FMT> load(int c, int r, int q) const {
        Raw<FMT> o;
        const int k = c * kStep + 32 * q;
        const bool in = k < K;
        if (FMT == kF8) {
            o.w[0] = load128(codes, in ? r * K + k : kDropped);
            o.w[FMT == kF8] = load128(codes, in ? r * K + k + 16 : kDropped);
            o.s = __float_as_uint(tile[c < kb ? c : 0]);
        } else {
            o.w[0] = load128(codes, in ? r * (K / 2) + k / 2 : kDropped);
            if (FMT == kMx) o.s = __builtin_amdgcn_raw_buffer_load_b8(scales, in ? r * kb + k / 32 : kDropped, 0, 0);
            else o.s = __builtin_amdgcn_raw_buffer_load_b16(scales, in ? r * kb + k / 16 : kDropped, 0, 0);
        }
        return o;
    }
};

__device__ __forceinline__ bf16x8_t join8(bf16x2_t a, bf16x2_t b, bf16x2_t c, bf16x2_t d) {
    return bf16x8_t{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// Weights to bf16, exactly.  For kF8 without the tile scale.
template <int FMT>
__device__ __forceinline__ Frag widen(const Raw<FMT>& x) {
    Frag f;
    if (FMT == kMx) {
        const float s = __uint_as_float(x.s << 23);  // the conversion takes the scale's exponent
#pragma unroll
        for (int i = 0; i < 4; ++i)
            f.v[i] = join8(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x.w[0][i], s, 0),
                           __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x.w[0][i], s, 1),
                           __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x.w[0][i], s, 2),
                           __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x.w[0][i], s, 3));
    } else if (FMT == kNv) {
        // At most 6 significant bits: the upper half of the binary32 product.
        const float sc[2] = {__builtin_amdgcn_cvt_f32_fp8((int)x.s, 0), __builtin_amdgcn_cvt_f32_fp8((int)x.s, 1)};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float s = sc[i / 2];
            const v2f a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(x.w[0][i], 1.0f, 0);
            const v2f b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(x.w[0][i], 1.0f, 1);
            const v2f c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(x.w[0][i], 1.0f, 2);
            const v2f d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(x.w[0][i], 1.0f, 3);
            const u32x4_t o = {pack_bf16x2(a[0] * s, a[1] * s), pack_bf16x2(b[0] * s, b[1] * s),
                               pack_bf16x2(c[0] * s, c[1] * s), pack_bf16x2(d[0] * s, d[1] * s)};
            f.v[i] = __builtin_bit_cast(bf16x8_t, o);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int lo = (int)x.w[FMT == kF8 ? i / 2 : 0][2 * (i % 2)], hi = (int)x.w[FMT == kF8 ? i / 2 : 0][2 * (i % 2) + 1];
            f.v[i] = join8(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false),
                           __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true),
                           __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false),
                           __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true));
        }
    }
    return f;
}

// acc += W x over a step (kF8: under the step's tile scale), parts smallest first.
template <int FMT, int P>
__device__ __forceinline__ v4f mma_step(const Frag& w, const Frag (&x)[P], uint32_t s, v4f acc) {
    v4f t = FMT == kF8 ? v4f{} : acc;
#pragma unroll
    for (int p = P - 1; p >= 0; --p)
#pragma unroll
        for (int i = 0; i < 4; ++i) t = mma(w.v[i], x[p].v[i], t);
    if (FMT != kF8) return t;
    const float f = __uint_as_float(s);
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] = fmaf(t[e], f, acc[e]);
    return acc;
}

// ---------------------------------------------------------------------------
// Which experts are in use, by whom.  Experts in use are numbered in order
// ("slots"); the tokens of a slot, in order, are the pairs off .. off + n - 1.  An id
// outside 0 .. E - 1 names none; a token that names an expert twice is one pair under
// the sum of its weights.
struct Slot {
    uint64_t mask;   // its tokens
    int e, off;
};
struct Plan {
    Slot slot[kMaxExperts];
    float wt[kMaxPairs];
    uint8_t tok[kMaxPairs];
    int slots;
};
struct PlanScratch {
    uint64_t mask[kMaxExperts];  // by expert
    uint16_t off[kMaxExperts];
};

// Made by one workgroup from the ids and weights in `ids`, `wts` (T x k; LDS or
// memory).  GIVEN: a caller's routing, where a token may name an expert twice.
template <bool GIVEN>
__device__ __forceinline__ void make_plan(Plan& out, PlanScratch& s, const int* ids, const float* wts, int T, int k, int E) {
    const int lane = threadIdx.x % kWave, n = T * k;
    for (int e = threadIdx.x; e < E; e += blockDim.x) s.mask[e] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        const int e = ids[i];
        if (e >= 0 && e < E) atomicOr((unsigned long long*)&s.mask[e], 1ull << (i / k));
    }
    __syncthreads();
    if (threadIdx.x < kWave) {
        int slots = 0, pairs = 0;
        for (int e0 = 0; e0 < E; e0 += kWave) {
            const int e = e0 + lane;
            const uint64_t mask = e < E ? s.mask[e] : 0;
            const int c = __popcll(mask);
            const uint64_t below = (1ull << lane) - 1;
            int before = 0, all = 0;  // pairs of the lanes below, and of all, bit by bit (c is at most 64)
#pragma unroll
            for (int bit = 0; bit < 7; ++bit) {
                const uint64_t with = __builtin_amdgcn_ballot_w64((c >> bit) & 1);
                before += __popcll(with & below) << bit;
                all += __popcll(with) << bit;
            }
            const uint64_t used = __builtin_amdgcn_ballot_w64(c > 0);
            if (c > 0) {
                const int off = pairs + before;
                s.off[e] = (uint16_t)off;
                out.slot[slots + __popcll(used & below)] = Slot{mask, e, off};
            }
            slots += __popcll(used);
            pairs += all;
        }
        if (lane == 0) out.slots = slots;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        const int e = ids[i], t = i / k, j = i - t * k;
        if (e < 0 || e >= E) continue;
        float w = wts[i];
        if (GIVEN) {
            bool first = true;
            w = 0.0f;
            for (int o = 0; o < k; ++o)
                if (ids[t * k + o] == e) {
                    if (o < j) first = false;
                    w += wts[t * k + o];
                }
            if (!first) continue;
        }
        const int at = s.off[e] + __popcll(s.mask[e] & ((1ull << t) - 1));
        out.tok[at] = (uint8_t)t;
        out.wt[at] = w;
    }
}

// Given routing.
__global__ __launch_bounds__(1024) void k_moe_plan(MoeParams p) {
    __shared__ PlanScratch s;
    make_plan<true>(*p.plan, s, p.ids, p.wts, p.T, p.k, p.E);
}

// The i-th token of a mask (i below its count).
__device__ __forceinline__ int token_of(uint64_t mask, int i) {
    int at = 0;
#pragma unroll
    for (int w = 32; w >= 1; w /= 2) {
        const int c = __popcll(mask & ((1ull << w) - 1));
        if (i >= c) i -= c, mask >>= w, at += w;
    }
    return at;
}

// ---------------------------------------------------------------------------
// The router.

constexpr int kRouteWaves = 16;
constexpr int kMaxRanges = 8;

// A reduction over each row of 16 lanes, by rotations: the same value in all of them.
template <typename F>
__device__ __forceinline__ uint32_t row_reduce(uint32_t v, F f) {
    v = f(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x121, 0xF, 0xF, true));  // row_ror:1, 2, 4, 8
    v = f(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x122, 0xF, 0xF, true));
    v = f(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x124, 0xF, 0xF, true));
    return f(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x128, 0xF, 0xF, true));
}
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
    return row_reduce(v, [](uint32_t a, uint32_t b) { return max(a, b); });
}
__device__ __forceinline__ uint32_t row_min(uint32_t v) {
    return row_reduce(v, [](uint32_t a, uint32_t b) { return min(a, b); });
}
__device__ __forceinline__ float row_sum(float v) {
    return __uint_as_float(row_reduce(__float_as_uint(v), [](uint32_t a, uint32_t b) {
        return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
    }));
}

// 8 consecutive elements of a row, as bf16 parts.
template <int P>
__device__ __forceinline__ void load8(Rsrc r, int at, bf16x8_t (&out)[P]) {
    if (P == 1) {
        out[0] = __builtin_bit_cast(bf16x8_t, load128(r, at < 0 ? kDropped : at * 2));
    } else {
        const u32x4_t a = load128(r, at < 0 ? kDropped : at * 4), b = load128(r, at < 0 ? kDropped : at * 4 + 16);
        float f[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = __uint_as_float(a[e]), f[4 + e] = __uint_as_float(b[e]);
        split8<P>(f, out);
    }
}

// Picks the experts of four tokens at once, one per row of 16 lanes: lane r of the row
// holds the logits of experts r, 16 + r, ... in v.  Each round takes the largest left,
// the lowest index among equals; lane j keeps the j-th.  (A whole wave per token took
// 6.8 us of 64 tokens' routing where this takes about 1.5: the rounds are chains of
// short steps, the same for one token as for four.)
template <int R>
__device__ __forceinline__ void pick(const MoeParams& p, int t, int r, const float (&v)[R], int* ids, float* wts) {
    uint32_t key[R];  // ordered as the logits are
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const uint32_t b = __float_as_uint(v[i] + 0.0f);  // -0 and 0 are equal
        const uint32_t o = b & 0x80000000u ? ~b : b | 0x80000000u;
        key[i] = 16 * i + r < p.E ? max(o, 1u) : 0u;  // 0: not there, or taken
    }
    uint32_t top = 0, mine = 0;
    int chosen = 0;
    for (int j = 0; j < p.k; ++j) {
        uint32_t m = key[0];
#pragma unroll
        for (int i = 1; i < R; ++i) m = max(m, key[i]);
        m = row_max(m);
        uint32_t e = 0xFFFFFFFFu;
#pragma unroll
        for (int i = R - 1; i >= 0; --i) e = key[i] == m ? 16 * i + r : e;
        e = row_min(e);
#pragma unroll
        for (int i = 0; i < R; ++i) key[i] = e == (uint32_t)(16 * i + r) ? 0u : key[i];
        if (j == 0) top = m;
        if (r == j) mine = m, chosen = (int)e;
    }
    auto logit = [](uint32_t o) { return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o); };
    const float l0 = logit(top);
    const float w = r < p.k ? expf(logit(mine) - l0) : 0.0f;
    float total = w;
    if (!p.renorm) {
        total = 0.0f;
#pragma unroll
        for (int i = 0; i < R; ++i) total += 16 * i + r < p.E ? expf(v[i] - l0) : 0.0f;
    }
    total = row_sum(total);
    if (r < p.k && t < p.T) {
        p.ids[t * p.k + r] = ids[t * p.k + r] = chosen;
        p.wts[t * p.k + r] = wts[t * p.k + r] = w / total;
    }
}

// PX, PR: bf16 parts of x and of the router's weights (products of parts beyond the
// third order, below 2^-24 of the whole, are left out).
template <int PX, int PR, int R>
__global__ __launch_bounds__(kRouteWaves * kWave) void k_moe_route(MoeParams p) {
    __shared__ float red[kRouteWaves][256];
    __shared__ int last;
    __shared__ PlanScratch scratch;
    __shared__ int ids[kMaxPairs];
    __shared__ float wts[kMaxPairs];
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int r = lane % 16, q = lane / 16;
    const int etiles = (p.E + 15) / 16;
    const int e0 = (int)(blockIdx.x % etiles) * 16;
    const int range = (int)(blockIdx.x / etiles) % p.ranges;
    const int tile = (int)(blockIdx.x / etiles) / p.ranges, t0 = tile * 16;
    const int xb = PX == 1 ? 2 : 4, rb = PR == 1 ? 2 : 4;
    const int rows_x = min(16, p.T - t0), rows_r = min(16, p.E - e0);
    const Rsrc rx = make_rsrc(static_cast<const char*>(p.x) + (int64_t)t0 * p.D * xb, (int64_t)rows_x * p.D * xb);
    const Rsrc rr = make_rsrc(static_cast<const char*>(p.router) + (int64_t)e0 * p.D * rb, (int64_t)rows_r * p.D * rb);
    const int steps = p.D / 32;  // D is a multiple of 32
    constexpr int U = 2;         // steps in flight
    v4f acc = {};
    for (int s0 = range * kRouteWaves + wave; s0 < steps; s0 += U * p.ranges * kRouteWaves) {
        bf16x8_t x[U][PX], w[U][PR];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int s = s0 + u * p.ranges * kRouteWaves, k = s * 32 + 8 * q;
            load8<PX>(rx, s < steps && r < rows_x ? r * p.D + k : -1, x[u]);
            load8<PR>(rr, s < steps && r < rows_r ? r * p.D + k : -1, w[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int o = 2; o >= 0; --o)  // small products first
#pragma unroll
                for (int i = 0; i <= o; ++i)
                    if (i < PR && o - i < PX) acc = mma(w[u][i < PR ? i : 0], x[u][o - i < PX ? o - i : 0], acc);
    }
    // Lane: token r, experts 4 q .. 4 q + 3.
    *reinterpret_cast<v4f*>(&red[wave][r * 16 + 4 * q]) = acc;
    __syncthreads();
    if (threadIdx.x < 256) {
        const int t = threadIdx.x / 16, e = threadIdx.x % 16;
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kRouteWaves; ++w) sum += red[w][threadIdx.x];
        if (t < rows_x && e < rows_r) p.logits[((int64_t)range * p.T + t0 + t) * p.E + e0 + e] = sum;
    }
    __syncthreads();
    // The last workgroup to get here sees everyone's sums (none waits): the barrier
    // orders the workgroup's sums before thread 0, which releases and acquires for it.
    if (threadIdx.x == 0) {
        const uint32_t n = __hip_atomic_fetch_add(p.count, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
        last = n + 1 == gridDim.x;
        if (last) __hip_atomic_store(p.count, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    if (!last) return;
    // Four tokens per wave: 16 waves take all there can be.
    static_assert(4 * kRouteWaves >= kMaxTokens, "a row of lanes per token");
    if (4 * wave < p.T) {
        const int t = 4 * wave + q;
        const float* src = p.logits + (int64_t)min(t, p.T - 1) * p.E;
        float v[R];
        // A range's sums of all experts are loaded together; where registers allow,
        // all ranges' (one trip to memory).
#pragma unroll
        for (int i = 0; i < R; ++i) v[i] = src[min(16 * i + r, p.E - 1)];
        if (R <= 8) {
            float part[kMaxRanges - 1][R <= 8 ? R : 1];
#pragma unroll
            for (int g = 1; g < kMaxRanges; ++g)
#pragma unroll
                for (int i = 0; i < R; ++i)
                    part[g - 1][R <= 8 ? i : 0] = src[(int64_t)min(g, p.ranges - 1) * p.T * p.E + min(16 * i + r, p.E - 1)];
#pragma unroll
            for (int g = 1; g < kMaxRanges; ++g)
#pragma unroll
                for (int i = 0; i < R; ++i) v[i] += g < p.ranges ? part[g - 1][R <= 8 ? i : 0] : 0.0f;
        } else {
            for (int g = 1; g < p.ranges; ++g) {
                float part[R];
#pragma unroll
                for (int i = 0; i < R; ++i) part[i] = src[(int64_t)g * p.T * p.E + min(16 * i + r, p.E - 1)];
#pragma unroll
                for (int i = 0; i < R; ++i) v[i] += part[i];
            }
        }
        pick<R>(p, t, r, v, ids, wts);
    }
    __syncthreads();
    make_plan<false>(*p.plan, scratch, ids, wts, p.T, p.k, p.E);
}

// ---------------------------------------------------------------------------
// Gate and up.

constexpr int kUpWaves = 8;

// NT: token tiles of 16.  PH: parts of h.
template <int FMT, int NT, int PX>
__global__ __launch_bounds__(kUpWaves * kWave) void k_moe_up(MoeParams p, int parts_h) {
    constexpr int U = FMT == kF8 || PX > 1 ? 2 : 4;  // steps in flight
    __shared__ float red[kUpWaves][2][256];
    const int itiles = p.I / kRows;
    const int slot = (int)(blockIdx.x / itiles), i0 = (int)(blockIdx.x % itiles) * kRows;
    const Slot sl = p.plan->slot[slot];
    if (slot >= p.plan->slots) return;
    const int e = sl.e, n = __popcll(sl.mask), off = sl.off;
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int r = lane % 16, q = lane / 16;
    const int64_t row = (int64_t)e * 2 * p.I + i0;
    const Rows<FMT> gate(p.w13, row, p.D), up(p.w13, row + p.I, p.D);
    const Rsrc rx = make_rsrc(p.x, (int64_t)p.T * p.D * (PX == 1 ? 2 : 4));
    int src[NT];  // element offset of the lane's token, or none
#pragma unroll
    for (int t = 0; t < NT; ++t) src[t] = 16 * t + r < n ? token_of(sl.mask, 16 * t + r) * p.D : -1;

    v4f ag[NT], au[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) ag[t] = au[t] = v4f{};
    const int steps = (p.D + kStep - 1) / kStep;
    for (int c0 = wave; c0 < steps; c0 += kUpWaves * U) {
        Raw<FMT> rg[U], ru[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = c0 + u * kUpWaves;  // past the last: zeros
            rg[u] = gate.load(c, r, q);
            ru[u] = up.load(c, r, q);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = (c0 + u * kUpWaves) * kStep + 32 * q;
            const Frag wg = widen<FMT>(rg[u]), wu = widen<FMT>(ru[u]);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                if (16 * t >= n) break;
                Act<PX> a;
                a.load(rx, src[t] >= 0 && k < p.D ? src[t] + k : -1);
                Frag x[PX];
                a.parts(x);
                ag[t] = mma_step<FMT, PX>(wg, x, rg[u].s, ag[t]);
                au[t] = mma_step<FMT, PX>(wu, x, ru[u].s, au[t]);
            }
        }
    }
    const float g = p.w13.g ? p.w13.g[e * p.w13.g_step] : 1.0f;
    const int64_t plane = (int64_t)p.T * p.k * p.I;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        if (16 * t >= n) break;
        // Lane: token 16 t + r, rows 4 q .. 4 q + 3.
        *reinterpret_cast<v4f*>(&red[wave][0][r * 16 + 4 * q]) = ag[t];
        *reinterpret_cast<v4f*>(&red[wave][1][r * 16 + 4 * q]) = au[t];
        __syncthreads();
        const int m = 16 * t + (int)threadIdx.x / 16;
        if (threadIdx.x < 256 && m < n) {
            float sg = 0.0f, su = 0.0f;
#pragma unroll
            for (int w = 0; w < kUpWaves; ++w) sg += red[w][0][threadIdx.x], su += red[w][1][threadIdx.x];
            sg *= g, su *= g;
            float h = sg / (1.0f + expf(-sg)) * su;
            uint16_t* dst = p.h + (int64_t)(off + m) * p.I + i0 + threadIdx.x % 16;
            for (int a = 0; a < parts_h; ++a) {
                const uint32_t b = to_bf16(h);
                dst[a * plane] = (uint16_t)b;
                h = left(h, b << 16);
            }
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// Down, and the sum over a token's experts.

constexpr int kDownWaves = 16;

template <int FMT, int NT, int PH>
__global__ __launch_bounds__(kDownWaves * kWave) void k_moe_down(MoeParams p) {
    constexpr int U = FMT == kF8 ? 2 : 4;
    __shared__ float wt[kMaxPairs];
    __shared__ uint8_t tok[kMaxPairs];
    extern __shared__ __attribute__((aligned(16))) float ytile[];  // waves x T x 16
    for (int i = threadIdx.x; i < p.T * p.k; i += kDownWaves * kWave) wt[i] = p.plan->wt[i], tok[i] = p.plan->tok[i];
    __syncthreads();
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int r = lane % 16, q = lane / 16;
    const int d0 = (int)blockIdx.x * kRows;
    float* mine = ytile + wave * p.T * 16;
    for (int i = lane; i < p.T * 16; i += kWave) mine[i] = 0.0f;

    const int steps = (p.I + kStep - 1) / kStep;
    const int total = p.plan->slots * steps;
    int at = total * wave / kDownWaves;
    const int end = total * (wave + 1) / kDownWaves;
    const int64_t plane = (int64_t)p.T * p.k * p.I;
    while (at < end) {
        const int slot = at / steps, c_lo = at % steps, c_hi = min(steps, c_lo + end - at);
        at += c_hi - c_lo;
        const Slot sl = p.plan->slot[slot];
        const int e = sl.e, n = __popcll(sl.mask), off = sl.off;
        const Rows<FMT> down(p.w2, (int64_t)e * p.D + d0, p.I);
        Rsrc rh[PH];
#pragma unroll
        for (int a = 0; a < PH; ++a)
            rh[a] = make_rsrc(p.h + a * plane + (int64_t)off * p.I, (int64_t)n * p.I * 2);
        v4f acc[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[t] = v4f{};
        for (int c0 = c_lo; c0 < c_hi; c0 += U) {
            Raw<FMT> raw[U];
#pragma unroll
            for (int u = 0; u < U; ++u) raw[u] = down.load(c0 + u < c_hi ? c0 + u : steps, r, q);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (c0 + u >= c_hi) break;
                const int k = (c0 + u) * kStep + 32 * q;
                const Frag w = widen<FMT>(raw[u]);
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    if (16 * t >= n) break;
                    Frag x[PH];
#pragma unroll
                    for (int a = 0; a < PH; ++a) {
                        Act<1> h;
                        h.load(rh[a], 16 * t + r < n && k < p.I ? (16 * t + r) * p.I + k : -1);
                        x[a] = frag_of(h.w);
                    }
                    acc[t] = mma_step<FMT, PH>(w, x, raw[u].s, acc[t]);
                }
            }
        }
        const float g = p.w2.g ? p.w2.g[e * p.w2.g_step] : 1.0f;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            // Lane: token 16 t + r of the slot (no token twice), rows 4 q .. 4 q + 3.
            if (16 * t + r >= n) continue;
            const float w = wt[off + 16 * t + r] * g;
            v4f* dst = reinterpret_cast<v4f*>(mine + tok[off + 16 * t + r] * 16 + 4 * q);
            v4f v = *dst;
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = fmaf(acc[t][i], w, v[i]);
            *dst = v;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < p.T * 16; i += kDownWaves * kWave) {
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kDownWaves; ++w) sum += ytile[w * p.T * 16 + i];
        const int64_t o = (int64_t)(i / 16) * p.D + d0 + i % 16;
        if (p.yt == 1) static_cast<float*>(p.y)[o] = sum;
        else static_cast<uint16_t*>(p.y)[o] = (uint16_t)to_bf16(sum);
    }
}

// ---------------------------------------------------------------------------

template <int FMT, int NT>
void launch_products(const MoeParams& p, bool x32, int parts_h, hipStream_t stream) {
    const int slots = std::min(p.T * p.k, p.E);
    const dim3 up((unsigned)(slots * (p.I / kRows))), down((unsigned)(p.D / kRows));
    if (x32) FP4Q_LAUNCH((k_moe_up<FMT, NT, 3>), up, dim3(kUpWaves * kWave), 0, stream, p, parts_h);
    else FP4Q_LAUNCH((k_moe_up<FMT, NT, 1>), up, dim3(kUpWaves * kWave), 0, stream, p, parts_h);
    const unsigned lds = (unsigned)(kDownWaves * p.T * 16 * 4);
    if (parts_h == 3) FP4Q_LAUNCH((k_moe_down<FMT, NT, 3>), down, dim3(kDownWaves * kWave), lds, stream, p);
    else FP4Q_LAUNCH((k_moe_down<FMT, NT, 2>), down, dim3(kDownWaves * kWave), lds, stream, p);
}

template <int FMT>
void launch_tiles(const MoeParams& p, bool x32, int parts_h, hipStream_t stream) {
    if (p.T <= 16) launch_products<FMT, 1>(p, x32, parts_h, stream);
    else if (p.T <= 32) launch_products<FMT, 2>(p, x32, parts_h, stream);
    else launch_products<FMT, 4>(p, x32, parts_h, stream);
}

// Ranges of K for the router: two steps of 32 per wave keep its loads in flight
// together, and 8 ranges are as many partial sums as are worth adding.
int route_ranges(int64_t D) {
    return (int)std::max<int64_t>(1, std::min<int64_t>(kMaxRanges, D / 32 / (2 * kRouteWaves)));
}

constexpr size_t kCountBytes = 256;
size_t up256(size_t n) { return (n + 255) / 256 * 256; }
const size_t kPlanBytes = up256(sizeof(Plan));

template <int PX, int PR>
void launch_route(const MoeParams& p, hipStream_t stream) {
    const dim3 grid((unsigned)((p.E + 15) / 16 * p.ranges * ((p.T + 15) / 16))), block(kRouteWaves * kWave);
    if (p.E <= 64) FP4Q_LAUNCH((k_moe_route<PX, PR, 4>), grid, block, 0, stream, p);
    else if (p.E <= 128) FP4Q_LAUNCH((k_moe_route<PX, PR, 8>), grid, block, 0, stream, p);
    else FP4Q_LAUNCH((k_moe_route<PX, PR, kMaxExperts / 16>), grid, block, 0, stream, p);
}

}  // namespace

size_t moe_workspace_bytes(int64_t T, int64_t D, int64_t I, int64_t E, int64_t k) {
    return kCountBytes + kPlanBytes + up256((size_t)(route_ranges(D) * T * E * 4)) + (size_t)(3 * T * k * I * 2);
}

int launch_moe(const MoeJob& j, char* msg, size_t msg_len) {
    if (j.T == 0) return 0;
    hipStream_t stream = static_cast<hipStream_t>(j.stream);
    char* ws = static_cast<char*>(j.ws);
    MoeParams p{};
    p.x = j.x;
    p.T = (int)j.T, p.D = (int)j.D, p.I = (int)j.I, p.E = (int)j.E, p.k = (int)j.k;
    p.w13 = Weights{j.w13.codes, j.w13.scales, j.w13.g, j.w13.g_per_expert ? 1 : 0};
    p.w2 = Weights{j.w2.codes, j.w2.scales, j.w2.g, j.w2.g_per_expert ? 1 : 0};
    p.router = j.router;
    p.renorm = j.renorm;
    p.ids = j.ids;
    p.wts = j.wts;
    p.y = j.y;
    p.yt = j.yt;
    p.ranges = route_ranges(j.D);
    p.count = reinterpret_cast<uint32_t*>(ws);
    p.plan = reinterpret_cast<Plan*>(ws + kCountBytes);
    p.logits = reinterpret_cast<float*>(ws + kCountBytes + kPlanBytes);
    p.h = reinterpret_cast<uint16_t*>(ws + kCountBytes + kPlanBytes + up256((size_t)(p.ranges * j.T * j.E * 4)));
    if (p.router) {
        if (j.xt == 0 && j.rt == 0) launch_route<1, 1>(p, stream);
        else if (j.xt == 0) launch_route<1, 3>(p, stream);
        else if (j.rt == 0) launch_route<3, 1>(p, stream);
        else launch_route<3, 3>(p, stream);
    } else {
        FP4Q_LAUNCH(k_moe_plan, dim3(1), dim3(1024), 0, stream, p);
    }
    const int parts_h = j.yt == 1 ? 3 : 2;
    if (j.fmt == 0) launch_tiles<kMx>(p, j.xt == 1, parts_h, stream);
    else if (j.fmt == 1) launch_tiles<kNv>(p, j.xt == 1, parts_h, stream);
    else launch_tiles<kF8>(p, j.xt == 1, parts_h, stream);
    const hipError_t e = hipGetLastError();
    if (e == hipSuccess) return 0;
    snprintf(msg, msg_len, "moe kernel launch: %s", hipGetErrorString(e));
    return (int)e;
}

}  // namespace fp4q
