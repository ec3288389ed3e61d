// fp4q_moe.hip -- a mixture-of-experts layer for a few tokens (moe_layer).
//
// For at most 64 tokens x, experts e with quantized weights G_e, U_e (gate and up,
// inter x dim) and D_e (down, dim x inter):
//   l = x Wr^T;  the top_k largest of each token, with softmax weights p
//   h_e = silu(G_e x) * (U_e x);   y = sum_e p_e D_e h_e
//
// Four launches:
//  k_moe_route  router logits by 16 experts x 16 tokens x a range of K, on the bf16
//               matrix cores; the last workgroup to finish adds the ranges, picks the
//               tokens' experts and lists each expert's tokens (k_moe_plan: the list
//               alone, for a given routing);
//  k_moe_up     gate and up products, and silu(g) u; or k_moe_many, which does the same
//               for more tokens and
//  k_moe_many   the down products of each (token, expert) pair, by K ranges;
//  k_moe_combine  their weighted sum.
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
//
// Measured: 64 tokens, 64 experts of 4096 x 1024 in E4M3 (805 MB) 190 us, its two
// products at 4.5 and 5.0 TB/s; 11 tokens, 8 experts of 4096 x 14336 in NVFP4 (793 MB)
// 189 to 197 us, at 4.4 and 4.0 TB/s with the vector unit, which widens the weights, busy
// in half of the cycles (E4M3: a seventh);
// one token on 8 of 64 experts of 4096 x 1024 in MXFP4 (53 MB) 30 us, of which the
// products 12.5 and 7.3, router 7.7 and combine 4.4: four launches of work too short to
// fill memory.  (The combine inside the down kernel, by the last workgroup of each 128
// rows, saved the launch but took 37 us: each workgroup's release writes back its L2.)
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
    uint16_t* xp;      // x as bf16 parts: x itself, or 3 x T x D made of binary32 x
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
// all 24 bits of a value whose last bits do not fall below the smallest number.  The
// first part stops at bf16's largest number, which the largest binary32 ones would round
// past; what is left of an infinity or NaN is itself, and of its own part nothing.
__device__ __forceinline__ float first_part(float f) { return __builtin_amdgcn_fmed3f(f, -0x1.FEp127f, 0x1.FEp127f); }
__device__ __forceinline__ float left(float f, uint32_t part) {
    return (part & 0x7F800000u) == 0x7F800000u ? 0.0f : f - __uint_as_float(part);
}
template <int P>
__device__ __forceinline__ void split8(const float (&f)[8], bf16x8_t (&out)[P]) {
    static_assert(P > 1, "an infinity is in the second part");
    float rest[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) rest[e] = f[e];
#pragma unroll
    for (int p = 0; p < P; ++p) {
        u32x4_t w;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            w[q] = p == 0 ? pack_bf16x2(first_part(rest[2 * q]), first_part(rest[2 * q + 1]))
                          : pack_bf16x2(rest[2 * q], rest[2 * q + 1]);
            rest[2 * q] = left(rest[2 * q], w[q] << 16);
            rest[2 * q + 1] = left(rest[2 * q + 1], w[q] & 0xFFFF0000u);
        }
        out[p] = __builtin_bit_cast(bf16x8_t, w);
    }
}

// 32 consecutive bf16 values at element offset `at` (negative: zeros) of a window.
struct Act {
    u32x4_t w[4];
    __device__ __forceinline__ void load(Rsrc r, int at) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = load128(r, at < 0 ? kDropped : at * 2 + 16 * i);
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
    int K, kb, end;     // `end`: no element from here on is read
    const float* tile;  // kF8: the tile scales of these rows, one per step
    __device__ __forceinline__ Rows(const Weights& w, int64_t row0, int K_, int end_) : K(K_), end(end_) {
        const int rowb = FMT == kF8 ? K : K / 2;
        kb = FMT == kMx ? K / 32 : FMT == kNv ? K / 16 : (K + kStep - 1) / kStep;
        codes = make_rsrc(w.codes + row0 * rowb, (int64_t)kRows * rowb);
        if (FMT == kF8) tile = static_cast<const float*>(w.scales) + row0 / 128 * kb;
        else scales = make_rsrc(static_cast<const uint8_t*>(w.scales) + row0 * kb, (int64_t)kRows * kb);
    }
    // Step c of the lane of row r, quarter q; from `end` on: zeros.
    __device__ __forceinline__ Raw<FMT> load(int c, int r, int q) const {
        Raw<FMT> o;
        const int k = c * kStep + 32 * q;
        const bool in = k < end;
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

// Two steps at once: a lane's row has their 8 (MX) or 16 (NV) scale bytes in one load
// where rows of scales start on that boundary, instead of four loads of one or two bytes,
// each of which touches 16 cache lines.
template <int FMT>
struct Raw2 {
    u32x4_t w[2][FMT == kF8 ? 2 : 1];
    uint32_t s[2][2];
    __device__ __forceinline__ Raw<FMT> step(int u, int q) const {
        Raw<FMT> o;
        o.w[0] = w[u][0];
        if (FMT == kF8) o.w[FMT == kF8] = w[u][FMT == kF8];
        if (FMT == kMx) o.s = (s[u][0] >> (8 * q)) & 0xFFu;
        else if (FMT == kNv) o.s = (q & 2 ? s[u][1] : s[u][0]) >> (16 * (q & 1));
        else o.s = s[u][0];
        return o;
    }
};
template <int FMT>
__device__ __forceinline__ bool whole_scales(const Rows<FMT>& rows, const void* scales) {
    constexpr int kBytes = FMT == kMx ? 8 : 16;
    return rows.kb % kBytes == 0 && (uint32_t)(uintptr_t)scales % kBytes == 0;
}
// Steps 2 c and 2 c + 1; whole: whole_scales of the matrix.
template <int FMT>
__device__ __forceinline__ Raw2<FMT> load2(const Rows<FMT>& rows, int c, int r, int q, bool whole) {
    Raw2<FMT> o;
    if (FMT == kF8 || !whole) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const Raw<FMT> x = rows.load(2 * c + u, r, q);
            o.w[u][0] = x.w[0];
            if (FMT == kF8) o.w[u][FMT == kF8] = x.w[FMT == kF8];
            o.s[u][0] = o.s[u][1] = FMT == kF8 ? x.s : x.s << (FMT == kMx ? 8 * q : 16 * (q & 1));
        }
    } else {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int k = (2 * c + u) * kStep + 32 * q;
            o.w[u][0] = load128(rows.codes, k < rows.end ? r * (rows.K / 2) + k / 2 : kDropped);
        }
        const bool in = 2 * c * kStep < rows.end;  // K is a multiple of 256 here
        if (FMT == kMx) {
            const u32x2_t v = __builtin_amdgcn_raw_buffer_load_b64(rows.scales, in ? r * rows.kb + 8 * c : kDropped, 0, 0);
            o.s[0][0] = v[0], o.s[1][0] = v[1], o.s[0][1] = o.s[1][1] = 0;
        } else {
            const u32x4_t v = load128(rows.scales, in ? r * rows.kb + 16 * c : kDropped);
            o.s[0][0] = v[0], o.s[0][1] = v[1], o.s[1][0] = v[2], o.s[1][1] = v[3];
        }
    }
    return o;
}

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

// 8 consecutive elements of a row, as bf16 parts.
template <int P>
__device__ __forceinline__ void load8(Rsrc r, int at, bf16x8_t (&out)[P]) {
    if constexpr (P == 1) {
        out[0] = __builtin_bit_cast(bf16x8_t, load128(r, at < 0 ? kDropped : at * 2));
    } else {
        const u32x4_t a = load128(r, at < 0 ? kDropped : at * 4), b = load128(r, at < 0 ? kDropped : at * 4 + 16);
        float f[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = __uint_as_float(a[e]), f[4 + e] = __uint_as_float(b[e]);
        split8<P>(f, out);
    }
}

// ---------------------------------------------------------------------------
// Which experts are in use, by whom: "slots" of an expert and up to 16 of its tokens (a
// matrix-core fragment), in order of experts and tokens; the tokens of a slot are the
// pairs off .. off + n - 1.  An id outside 0 .. E - 1 names no expert; a token that names
// one twice is one pair under the sum of its weights.
constexpr int kMaxSlots = kMaxExperts + kMaxPairs / 16;
struct Slot {
    uint64_t mask;   // its tokens
    int e, off;
};
struct Plan {
    Slot slot[kMaxSlots];
    short pair[kMaxPairs];    // of each token's choices in turn; -1: none
    float weight[kMaxPairs];  // and their weights
    int slots;
};
struct PlanScratch {
    uint64_t mask[kMaxExperts];  // by expert
    uint16_t off[kMaxExperts];
};

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
            // Slots of the lanes below, and of all: at most four each.
            const int ns = (c + 15) / 16;
            int first = slots;
#pragma unroll
            for (int bit = 0; bit < 3; ++bit) {
                const uint64_t with = __builtin_amdgcn_ballot_w64((ns >> bit) & 1);
                first += __popcll(with & below) << bit;
                slots += __popcll(with) << bit;
            }
            const int off = pairs + before;
            if (c > 0) s.off[e] = (uint16_t)off;
            uint64_t left = mask;
            for (int i = 0; i < ns; ++i) {
                const int n = min(16, c - 16 * i);
                const uint64_t part = n < 16 || c == 16 * (i + 1) ? left : left & ((1ull << token_of(left, 16)) - 1);
                out.slot[first + i] = Slot{part, e, off + 16 * i};
                left &= ~part;
            }
            pairs += all;
        }
        if (lane == 0) out.slots = slots;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        const int e = ids[i], t = i / k;
        out.pair[i] = -1;
        out.weight[i] = 0.0f;
        if (e < 0 || e >= E) continue;
        float w = wts[i];
        if (GIVEN) {
            const int j = i - t * k;
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
        out.pair[i] = (short)at;
        out.weight[i] = w;
    }
}

// Given routing: the first workgroup lists the experts' tokens, the others make the
// parts of binary32 x.
__global__ __launch_bounds__(1024) void k_moe_plan(MoeParams p) {
    __shared__ PlanScratch s;
    if (blockIdx.x > 0) {
        const Rsrc rx = make_rsrc(p.x, (int64_t)p.T * p.D * 4);
        const int n = p.T * p.D;  // a multiple of 8; at most 2^26
        for (int at = ((int)(blockIdx.x - 1) * 1024 + (int)threadIdx.x) * 8; at < n; at += (int)(gridDim.x - 1) * 8192) {
            bf16x8_t part[3];
            load8<3>(rx, at, part);
#pragma unroll
            for (int a = 0; a < 3; ++a) *reinterpret_cast<bf16x8_t*>(p.xp + (int64_t)a * n + at) = part[a];
        }
        return;
    }
    make_plan<true>(*p.plan, s, p.ids, p.wts, p.T, p.k, p.E);
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
        if (PX == 3 && e0 == 0) {
            // x's parts, for the products: each step is in one wave of these workgroups.
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int s = s0 + u * p.ranges * kRouteWaves;
                if (s < steps && r < rows_x)
#pragma unroll
                    for (int a = 0; a < PX; ++a)
                        *reinterpret_cast<bf16x8_t*>(p.xp + ((int64_t)a * p.T + t0 + r) * p.D + s * 32 + 8 * q) = x[u][a];
            }
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
    // The last workgroup to get here sees everyone's sums (none waits): each wave waits for
    // its own stores (the barrier does not), then thread 0 releases and acquires for all.
    wait_vm<0>();
    __syncthreads();
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
// Gate and up, where there are few (slot, rows) pairs to spread over the chip: a
// workgroup per 16 rows of h, its waves sharing out K, so that one token's few experts
// still put hundreds of workgroups to work.  Each wave reads its tokens' values from
// the caches itself.

constexpr int kUpWaves = 8;

// h of a pair's element from the sums of gate and up, as bf16 parts.
__device__ __forceinline__ void put_h(const MoeParams& p, float sg, float su, int64_t at, int parts_h) {
    const int64_t plane = (int64_t)p.T * p.k * p.I;
    float h = sg / (1.0f + expf(-sg)) * su;
    for (int a = 0; a < parts_h; ++a) {
        const uint32_t b = pack_bf16x2(a == 0 ? first_part(h) : h, 0.0f) & 0xFFFFu;
        p.h[at + a * plane] = (uint16_t)b;
        h = left(h, b << 16);
    }
}

// PX: parts of x.
template <int FMT, int PX>
__global__ __launch_bounds__(kUpWaves * kWave, 4) void k_moe_up(MoeParams p, int parts_h) {
    constexpr int U = PX > 1 ? 1 : FMT == kF8 ? 2 : 4;  // steps in flight
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
    const Rows<FMT> gate(p.w13, row, p.D, p.D), up(p.w13, row + p.I, p.D, p.D);
    Rsrc rx[PX];
#pragma unroll
    for (int a = 0; a < PX; ++a) rx[a] = make_rsrc(p.xp + (int64_t)a * p.T * p.D, (int64_t)p.T * p.D * 2);
    const int src = r < n ? token_of(sl.mask, r) * p.D : -1;  // element offset of the lane's token, or none

    v4f ag = {}, au = {};
    const int steps = (p.D + kStep - 1) / kStep;
    for (int c0 = wave; c0 < steps; c0 += kUpWaves * U) {
        Raw<FMT> rg[U], ru[U];
        Act x[U][PX];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = c0 + u * kUpWaves, k = c * kStep + 32 * q;  // past the last: zeros
            rg[u] = gate.load(c, r, q);
            ru[u] = up.load(c, r, q);
#pragma unroll
            for (int a = 0; a < PX; ++a) x[u][a].load(rx[a], src >= 0 && k < p.D ? src + k : -1);
        }
        __builtin_amdgcn_sched_barrier(0);  // every load before the first wait
#pragma unroll
        for (int u = 0; u < U; ++u) {
            Frag f[PX];
#pragma unroll
            for (int a = 0; a < PX; ++a) f[a] = frag_of(x[u][a].w);
            ag = mma_step<FMT, PX>(widen<FMT>(rg[u]), f, rg[u].s, ag);
            au = mma_step<FMT, PX>(widen<FMT>(ru[u]), f, ru[u].s, au);
        }
    }
    // Lane: token r, rows 4 q .. 4 q + 3.
    *reinterpret_cast<v4f*>(&red[wave][0][r * 16 + 4 * q]) = ag;
    *reinterpret_cast<v4f*>(&red[wave][1][r * 16 + 4 * q]) = au;
    __syncthreads();
    const int m = (int)threadIdx.x / 16;
    if (threadIdx.x < 256 && m < n) {
        const float g = p.w13.g ? p.w13.g[e * p.w13.g_step] : 1.0f;
        float sg = 0.0f, su = 0.0f;
#pragma unroll
        for (int w = 0; w < kUpWaves; ++w) sg += red[w][0][threadIdx.x], su += red[w][1][threadIdx.x];
        put_h(p, sg * g, su * g, (int64_t)(off + m) * p.I + i0 + threadIdx.x % 16, parts_h);
    }
}

// ---------------------------------------------------------------------------
// Down, and gate and up where there are many pairs: a workgroup per slot and 128 rows
// (64 of gate and the same 64 of up, or 128 of down), four waves of two fragments each.
// The slot's token values go to LDS once for the 128 rows, a step of 128 elements of
// each part at a time, by direct loads; two stages, so that the next one's values and
// weights are on their way while one is multiplied.  (With 16 rows per workgroup the
// caches deliver the values eight times as often: at 64 tokens the down product took
// 108 us so, and 63 so.)
//
// A stage holds 16 tokens x 256 bytes per part.  The sixteen 16-byte pieces of token
// t's row sit at slot piece ^ (t + 4) % 16, which spreads the lanes that one
// ds_read_b128 serves together (0-3, 12-15, 20-23, 24-27, ...; lane l reads piece
// 4 (l / 16) + i of token l % 16) over all bank groups.
constexpr int kManyWaves = 4;
constexpr int kManyRows = 32 * kManyWaves;
constexpr int kPart = 16 * 256;  // bytes of a stage's part

// DOWN: this K range's z[pair] = g D_e h in binary32, added up by k_moe_combine; else h.
template <int FMT, int P, bool DOWN>
__global__ __launch_bounds__(kManyWaves * kWave) void k_moe_many(MoeParams p, float* z, int ranges, int parts_h) {
    constexpr int S = 2;  // steps per stage
    constexpr int kStage = S * P * kPart;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * kStage];
    const int K = DOWN ? p.I : p.D;
    const int groups = ((DOWN ? p.D : 2 * p.I) + kManyRows - 1) / kManyRows;
    const int group = (int)(blockIdx.x % groups), range = (int)(blockIdx.x / groups) % ranges;
    const int slot = (int)(blockIdx.x / groups) / ranges;
    const Slot sl = p.plan->slot[slot];
    if (slot >= p.plan->slots) return;
    const int e = sl.e, n = __popcll(sl.mask), off = sl.off;
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int r = lane % 16, q = lane / 16;
    // The wave's two fragments: rows row and row + 16 of down, or row of gate and of up.
    // Both sizes are multiples of 32: a wave has both fragments or none.
    const int row = DOWN ? group * kManyRows + 32 * wave : group * (kManyRows / 2) + 16 * wave;
    const bool any = row < (DOWN ? p.D : p.I);
    const int64_t row0 = any ? (DOWN ? (int64_t)e * p.D + row : (int64_t)e * 2 * p.I + row) : 0;
    const int stages = (K + S * kStep - 1) / (S * kStep);
    const int c_lo = stages * range / ranges, c_hi = stages * (range + 1) / ranges;
    const int end = min(K, c_hi * S * kStep);  // the last stage's early loads go no further
    const Rows<FMT> w0(DOWN ? p.w2 : p.w13, row0, K, end), w1(DOWN ? p.w2 : p.w13, any ? row0 + (DOWN ? 16 : p.I) : 0, K, end);

    // Direct load `wave` of a part moves tokens 4 wave .. 4 wave + 3, 256 bytes each.
    const uint16_t* vals = DOWN ? p.h + (int64_t)off * p.I : p.xp;
    const int64_t part_step = DOWN ? (int64_t)p.T * p.k * p.I : (int64_t)p.T * p.D;
    const int64_t part_size = (int64_t)(DOWN ? n : p.T) * K * 2;
    const int m = 4 * wave + lane / 16;
    const int src = m < n ? (DOWN ? m : token_of(sl.mask, m)) * K : -1;
    const int piece = (lane % 16) ^ ((m + 4) % 16);
    auto issue = [&](int c) {
#pragma unroll
        for (int u = 0; u < S; ++u) {
            const int k = (c * S + u) * kStep + 8 * piece;
            const int at = src >= 0 && k < end ? (src + k) * 2 : kDropped;
#pragma unroll
            for (int a = 0; a < P; ++a)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(
                    make_rsrc(vals + a * part_step, part_size),
                    (LdsPtr)(lds + (c & 1) * kStage + (u * P + a) * kPart + wave * 1024), 16, at, 0, 0, 0);
        }
    };

    v4f acc[2] = {};
    const bool whole = whole_scales(w0, DOWN ? p.w2.scales : p.w13.scales);
    issue(c_lo);
    Raw2<FMT> n0 = load2(w0, c_lo, r, q, whole), n1 = load2(w1, c_lo, r, q, whole);
    for (int c = c_lo; c < c_hi; ++c) {
        // Stage c has landed, and no wave still reads stage c - 1.
        __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) lgkmcnt(0)
        asm volatile("s_barrier" ::: "memory");
        const Raw2<FMT> now[2] = {n0, n1};
        issue(c + 1);
        n0 = load2(w0, c + 1, r, q, whole), n1 = load2(w1, c + 1, r, q, whole);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int u = 0; u < S; ++u) {
            Frag x[P];
#pragma unroll
            for (int a = 0; a < P; ++a)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    x[a].v[i] = *reinterpret_cast<const bf16x8_t*>(lds + (c & 1) * kStage + (u * P + a) * kPart + r * 256 +
                                                                   ((4 * q + i) ^ ((r + 4) % 16)) * 16);
#pragma unroll
            for (int f = 0; f < 2; ++f) {
                const Raw<FMT> w = now[f].step(u, q);
                acc[f] = mma_step<FMT, P>(widen<FMT>(w), x, w.s, acc[f]);
            }
        }
    }
    wait_all_barrier();
    // Lane: token r, rows 4 q .. 4 q + 3 of each fragment.
    if (!any || r >= n) return;
    const Weights& w = DOWN ? p.w2 : p.w13;
    const float g = w.g ? w.g[e * w.g_step] : 1.0f;
    const int64_t pair = off + r;
    if (DOWN) {
        float* dst = z + ((int64_t)range * p.T * p.k + pair) * p.D + row + 4 * q;
#pragma unroll
        for (int f = 0; f < 2; ++f) *reinterpret_cast<v4f*>(dst + 16 * f) = acc[f] * g;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) put_h(p, acc[0][i] * g, acc[1][i] * g, pair * p.I + row + 4 * q + i, parts_h);
    }
}

// y[t] = sum over the token's choices of weight times z, z by K ranges.  Four columns
// per thread; the four threads of a quad take the choices in turn and meet in their
// order, so that a single token still keeps many loads in flight.
__global__ __launch_bounds__(256) void k_moe_combine(MoeParams p, const float* z, int ranges) {
    const int cols = p.D / 4, s = threadIdx.x % 4;
    const int i = (int)blockIdx.x * 64 + (int)threadIdx.x / 4;
    const int t = min(i / cols, p.T - 1), d = i % cols * 4;  // quads past the last repeat it, unstored
    const int64_t plane = (int64_t)p.T * p.k * p.D;
    v4f sum = {};
    for (int j = s; j < p.k; j += 4) {
        const int pair = p.plan->pair[t * p.k + j];
        const float w = p.plan->weight[t * p.k + j];
        if (pair < 0) continue;
        const float* src = z + (int64_t)pair * p.D + d;
        v4f v = {};
        for (int g0 = 0; g0 < ranges; g0 += 4) {
            v4f part[4];
#pragma unroll
            for (int g = 0; g < 4; ++g) part[g] = *reinterpret_cast<const v4f*>(src + min(g0 + g, ranges - 1) * plane);
#pragma unroll
            for (int g = 0; g < 4; ++g)
                if (g0 + g < ranges) v += part[g];
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) sum[c] = fmaf(v[c], w, sum[c]);
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        sum[c] += __shfl_xor(sum[c], 1);
        sum[c] += __shfl_xor(sum[c], 2);
    }
    if (s != 0 || i >= p.T * cols) return;
    // y need not start on more than its element's boundary.
    typedef float Four __attribute__((ext_vector_type(4), aligned(4)));
    typedef uint32_t Two __attribute__((ext_vector_type(2), aligned(2)));
    const int64_t o = (int64_t)t * p.D + d;
    if (p.yt == 1) *reinterpret_cast<Four*>(static_cast<float*>(p.y) + o) = sum;
    else *reinterpret_cast<Two*>(static_cast<uint16_t*>(p.y) + o) = u32x2_t{pack_bf16x2(sum[0], sum[1]), pack_bf16x2(sum[2], sum[3])};
}

// ---------------------------------------------------------------------------

// Slots there may be.
int64_t max_slots(int64_t T, int64_t E, int64_t k) { return std::min(T * k, E + T * k / 16); }

// K ranges of the down product: as many as fill the chip four workgroups deep, of two
// steps or more.
int down_ranges(int64_t T, int64_t D, int64_t I, int64_t E, int64_t k) {
    const int64_t groups = max_slots(T, E, k) * ((D + kManyRows - 1) / kManyRows);
    const int64_t stages = (I + 2 * kStep - 1) / (2 * kStep);
    return (int)std::max<int64_t>(1, std::min<int64_t>({(1024 + groups - 1) / groups, stages / 2, 16}));
}

template <int FMT>
void launch_products(const MoeParams& p, float* z, bool x32, int parts_h, hipStream_t stream) {
    const int slots = (int)max_slots(p.T, p.E, p.k);
    const int up_groups = (2 * p.I + kManyRows - 1) / kManyRows, down_groups = (p.D + kManyRows - 1) / kManyRows;
    const dim3 block(kManyWaves * kWave);
    // Which form of gate and up: 128 rows per workgroup where that makes enough
    // workgroups, fewer of them where slots are at least half full, since 16 rows per
    // workgroup fetch a slot's values eight times as often.  Measured (us, 128 rows / 16
    // rows; the product alone, and the whole layer where said): 128 workgroups (one token, 8
    // experts of 4096 x 1024) 25 / 13, 256 (two tokens) 27 / 22, 448 (one token, 2 of 4096 x
    // 14336) 34 / 36, 512 (four tokens, NVFP4 2048 x 1024) 20 / 27, 3072 (64 tokens, E4M3)
    // 114 / 157; layers with half-full slots: 174 workgroups (29 tokens, 15 of 864 x 352)
    // 27.6 / 26.2, 238 (49 tokens, 5 of 1920 x 896, binary32) 50 / 55, 256 (64 tokens, 8 of
    // 2048 x 1024) 34 / 36, binary32 42 / 49.
    const bool full = p.T * p.k >= 8 * slots;
    if (slots * up_groups >= (full ? 224 : 384)) {
        const dim3 grid((unsigned)(slots * up_groups));
        if (x32) FP4Q_LAUNCH((k_moe_many<FMT, 3, false>), grid, block, 0, stream, p, z, 1, parts_h);
        else FP4Q_LAUNCH((k_moe_many<FMT, 1, false>), grid, block, 0, stream, p, z, 1, parts_h);
    } else {
        const dim3 grid((unsigned)(slots * (p.I / kRows)));
        if (x32) FP4Q_LAUNCH((k_moe_up<FMT, 3>), grid, dim3(kUpWaves * kWave), 0, stream, p, parts_h);
        else FP4Q_LAUNCH((k_moe_up<FMT, 1>), grid, dim3(kUpWaves * kWave), 0, stream, p, parts_h);
    }
    const int ranges = down_ranges(p.T, p.D, p.I, p.E, p.k);
    const dim3 grid((unsigned)(slots * down_groups * ranges));
    if (parts_h == 3) FP4Q_LAUNCH((k_moe_many<FMT, 3, true>), grid, block, 0, stream, p, z, ranges, parts_h);
    else FP4Q_LAUNCH((k_moe_many<FMT, 2, true>), grid, block, 0, stream, p, z, ranges, parts_h);
    FP4Q_LAUNCH(k_moe_combine, dim3((unsigned)((p.T * (p.D / 4) + 63) / 64)), dim3(256), 0, stream, p, (const float*)z, ranges);
}

// Ranges of K for the router: as many as make 64 workgroups, with no less than half a step of
// 32 per wave; 32 where over 128 experts make the last workgroup add one range after the
// other.  Measured (us, so / with two steps per wave whatever the tiles): 49 tokens,
// 5 experts of 1920, binary32, 10.9 / 17.6 (32 workgroups / 4); one token, 64 of 4096, 7.7 /
// 8.3 (32 / 16); 64 tokens, 64 of 4096, 11.0 (64); 64 tokens, 500 of 4096, binary32,
// 46.9 / 54.2 (128 / 512); 16 tokens, 200 of 2048, 15.8 (26; 17.3 with 52).
int route_ranges(int64_t T, int64_t D, int64_t E) {
    const int64_t tiles = (E + 15) / 16 * ((T + 15) / 16), steps = D / 32;
    const int64_t most = std::min<int64_t>(kMaxRanges, (2 * steps + kRouteWaves - 1) / kRouteWaves);
    return (int)std::max<int64_t>(1, std::min<int64_t>(most, (E <= 128 ? 64 : 32) / tiles));
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
    const size_t logits = up256((size_t)(route_ranges(T, D, E) * T * E * 4)), parts = up256((size_t)(3 * T * D * 2));
    const size_t h = up256((size_t)(3 * T * k * I * 2)), z = (size_t)(down_ranges(T, D, I, E, k) * T * k * D * 4);
    return kCountBytes + kPlanBytes + logits + parts + h + z;
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
    p.ranges = route_ranges(j.T, j.D, j.E);
    p.count = reinterpret_cast<uint32_t*>(ws);
    p.plan = reinterpret_cast<Plan*>(ws += kCountBytes);
    p.logits = reinterpret_cast<float*>(ws += kPlanBytes);
    ws += up256((size_t)(p.ranges * j.T * j.E * 4));
    // Binary32 x in parts; bf16 x is its own.
    p.xp = j.xt == 1 ? reinterpret_cast<uint16_t*>(ws) : static_cast<uint16_t*>(const_cast<void*>(j.x));
    p.h = reinterpret_cast<uint16_t*>(ws += up256((size_t)(3 * j.T * j.D * 2)));
    ws += up256((size_t)(3 * j.T * j.k * j.I * 2));
    float* z = reinterpret_cast<float*>(ws);
    if (p.router) {
        if (j.xt == 0 && j.rt == 0) launch_route<1, 1>(p, stream);
        else if (j.xt == 0) launch_route<1, 3>(p, stream);
        else if (j.rt == 0) launch_route<3, 1>(p, stream);
        else launch_route<3, 3>(p, stream);
    } else {
        const int64_t parts = j.xt == 1 ? std::min<int64_t>((j.T * j.D + 8191) / 8192, 256) : 0;
        FP4Q_LAUNCH(k_moe_plan, dim3((unsigned)(1 + parts)), dim3(1024), 0, stream, p);
    }
    const int parts_h = j.yt == 1 ? 3 : 2;
    if (j.fmt == 0) launch_products<kMx>(p, z, j.xt == 1, parts_h, stream);
    else if (j.fmt == 1) launch_products<kNv>(p, z, j.xt == 1, parts_h, stream);
    else launch_products<kF8>(p, z, j.xt == 1, parts_h, stream);
    const hipError_t e = hipGetLastError();
    if (e == hipSuccess) return 0;
    snprintf(msg, msg_len, "moe kernel launch: %s", hipGetErrorString(e));
    return (int)e;
}

}  // namespace fp4q
