// fp4q_int8.hip -- 8-bit integers with one binary32 scale per row (int8_quantize_rows) and
// products of two such operands (int8_gemm).
//
//   s = max(RN32(max |x| / 127), 2^-126) of a row, code = RN32(x / s) to the nearest whole
//   number, ties to even
//   C[m][n] = RN(acc sa[m] sb[n] + bias[n]),  acc = sum over k of A[m][k] B[n][k]
//
// acc is a whole number below 2^31 (K <= 131056), which the matrix cores form exactly, so
// that every kernel and every split of K gives the same acc, and C, a function of acc and of
// its row's and column's own scales, the same bits whatever the other rows are.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <stdio.h>

#include <algorithm>
#include <type_traits>

#include "fp4q_fp8_tile.h"
#include "fp4q_launch.h"

namespace fp4q {
namespace {

// ---------------------------------------------------------------------------
// Quantizer.  WAVES waves per row (one: four rows per workgroup), a thread holding up to
// CHUNKS pieces of 8 elements, so that the row is read once; longer rows are read twice.
// A row that holds a NaN or an infinity gets that scale (NaN or infinity) and codes of 0:
// on use all of it is NaN.

constexpr float kMinScale = 0x1p-126f;
// Scales for which the corrected quotient is RN32(x / s) wherever it can matter: from 2^-60
// up, |x| < 2^-100 means a quotient below 2^-40, code 0.
constexpr float kFastLo = 0x1p-60f, kFastHi = 0x1p100f;

struct I8QuantParams {
    const void* x;
    int64_t rows, cols, ld;
    int8_t* codes;
    float* scales;
    unsigned first;  // this launch's first workgroup
};

// Eight elements from column c on; what does not exist is +0.
template <int XT>
__device__ __forceinline__ void load8(float (&v)[8], const void* row, int64_t c, int64_t cols) {
    typedef typename std::conditional<XT == 0, uint16_t, uint32_t>::type Bits;
    struct __attribute__((packed, aligned(sizeof(Bits)))) Eight { Bits e[8]; };
    const Bits* src = static_cast<const Bits*>(row) + c;
    auto f32 = [](Bits b) { return __uint_as_float(XT == 0 ? (uint32_t)b << 16 : (uint32_t)b); };
    if (c + 8 <= cols) {
        const Eight w = *reinterpret_cast<const Eight*>(src);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = f32(w.e[e]);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = c + e < cols ? f32(src[e]) : 0.0f;
    }
}

__device__ __forceinline__ float max8(const float (&v)[8], float m) {
#pragma unroll
    for (int e = 0; e < 8; ++e) m = __builtin_elementwise_maximum(m, fabsf(v[e]));  // keeps a NaN
    return m;
}

// Maximum over a wave, in every lane.
__device__ __forceinline__ float wave_max(float m) {
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) m = __builtin_elementwise_maximum(m, __shfl_xor(m, d));
    return m;
}

struct RowScale {
    float s, r;   // scale, 1 / s
    bool fast, bad;
    __device__ __forceinline__ explicit RowScale(float amax) {
        s = amax / 127.0f;
        s = s < kMinScale ? kMinScale : s;  // (keeps a NaN)
        r = 1.0f / s;
        fast = s >= kFastLo && s <= kFastHi;
        bad = !(s < __builtin_inff());
    }
    __device__ __forceinline__ int code(float x) const {
        float q = x * r;
        if (fast) q = fmaf(-fmaf(q, s, -x), r, q);
        else q = x / s;
        return bad ? 0 : (int)rintf(q);
    }
    __device__ __forceinline__ uint2 codes(const float (&v)[8]) const {
        uint32_t w[2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
            w[h] = (uint32_t)(code(v[4 * h]) & 255) | (uint32_t)(code(v[4 * h + 1]) & 255) << 8 |
                   (uint32_t)(code(v[4 * h + 2]) & 255) << 16 | (uint32_t)code(v[4 * h + 3]) << 24;
        return make_uint2(w[0], w[1]);
    }
};

template <int XT, int WAVES, int CHUNKS>
__global__ __launch_bounds__(WAVES == 1 ? 256 : WAVES * kWave) void k_int8_quantize(I8QuantParams p) {
    __shared__ float part[WAVES];
    constexpr int kStep = WAVES * kWave * 8;  // elements per chunk of all threads
    const int64_t group = p.first + blockIdx.x;
    const int64_t row = WAVES == 1 ? group * 4 + threadIdx.x / kWave : group;
    if (WAVES == 1 && row >= p.rows) return;
    const int t = WAVES == 1 ? threadIdx.x % kWave : threadIdx.x;
    const char* src = static_cast<const char*>(p.x) + row * p.cols * (XT == 0 ? 2 : 4);
    int8_t* dst = p.codes + row * p.ld;
    float v[CHUNKS][8], m = 0.0f;
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) load8<XT>(v[c], src, min((int64_t)c * kStep + t * 8, p.cols), p.cols);
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) m = max8(v[c], m);
    for (int64_t at = (int64_t)CHUNKS * kStep + t * 8; at < p.cols; at += kStep) {
        float u[8];
        load8<XT>(u, src, at, p.cols);
        m = max8(u, m);
    }
    m = wave_max(m);
    if (WAVES > 1) {
        if (t % kWave == 0) part[t / kWave] = m;
        __syncthreads();
        m = part[0];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) m = __builtin_elementwise_maximum(m, part[w]);
    }
    const RowScale sc(m);
    if (t == 0) p.scales[row] = sc.s;
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
        const int64_t at = (int64_t)c * kStep + t * 8;
        if (at < p.ld) *reinterpret_cast<uint2*>(dst + at) = sc.codes(v[c]);
    }
    for (int64_t at = (int64_t)CHUNKS * kStep + t * 8; at < p.ld; at += kStep) {
        float u[8];
        load8<XT>(u, src, min(at, p.cols), p.cols);
        *reinterpret_cast<uint2*>(dst + at) = sc.codes(u);
    }
}

// ---------------------------------------------------------------------------
// Products

struct I8Params {
    const int8_t* a;
    const float* sa;   // M
    const int8_t* b;
    const float* sb;   // N
    const void* bias;  // N, or NULL
    int bt;            // its type: 0 bf16, 1 f32
    int64_t M, N, K;
    int S;             // K blocks
    void* c;
    int ct;            // 0 bf16, 1 f32
    bool whole;        // C's rows start on 16 bytes
    int splits;        // K ranges per tile (1: C directly)
    int* partial;      // splits > 1: splits x M x N
    unsigned first;    // this launch's first workgroup
};

__device__ __forceinline__ v4i mma(v4i b, v4i a, v4i c) { return __builtin_amdgcn_mfma_i32_16x16x64_i8(b, a, c, 0, 0, 0); }

// The same where every accumulation register is taken: written as a builtin, the compiler turned
// the sums through a spare register, four moves a product.
__device__ __forceinline__ void mma_in_place(v4i& c, v4i b, v4i a) {
    asm volatile("v_mfma_i32_16x16x64_i8 %0, %1, %2, %0" : "+a"(c) : "v"(b), "v"(a));
}

// acc sa sb + bias: acc and the scales' product are rounded to binary32, then one fused
// multiply-add.  Where that product is not a normal number, in binary64.
__device__ __forceinline__ float value(int acc, float sa, float sb, float bias) {
    const float f = sa * sb;
    const float slow = (float)((double)acc * ((double)sa * (double)sb) + (double)bias);
    return fabsf(f) >= 0x1p-126f && fabsf(f) < __builtin_inff() ? fmaf((float)acc, f, bias) : slow;
}

__device__ __forceinline__ float bias_at(const I8Params& p, int64_t n) {
    if (!p.bias) return 0.0f;
    if (p.bt == 1) return static_cast<const float*>(p.bias)[n];
    return __uint_as_float((uint32_t) static_cast<const uint16_t*>(p.bias)[n] << 16);
}

// What a tile of T x T needs after its sums, brought to LDS before them: loads there would be
// waited for with nothing else to do.  Rows and columns past the last repeat it.
template <int T>
struct Ends {
    float sa[T], sb[T], bias[T];
    __device__ __forceinline__ void load(const I8Params& p, int64_t m0, int64_t n0) {
        for (int t = threadIdx.x; t < T; t += 256) {
            const int64_t n = min(n0 + t, p.N - 1);
            sa[t] = p.sa[min(m0 + t, p.M - 1)];
            sb[t] = p.sb[n];
            bias[t] = bias_at(p, n);
        }
    }
};

// A wave's sums to values, given to put(i, j, v4f) fragment by fragment, or as the bits of whole
// numbers for a K range's partial sums.  Lane l, register e of acc[i][j]: row of A a0 + 16 j +
// l % 16, row of B b0 + 16 i + 4 (l / 16) + e, within the tile.
template <int T, int NA, int NB, class Put>
__device__ __forceinline__ void finish(const v4i (&acc)[NB][NA], const Ends<T>& ends, bool partial, int a0, int b0, int lane, Put put) {
    if (partial) {
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
            for (int j = 0; j < NA; ++j) put(i, j, __builtin_bit_cast(v4f, acc[i][j]));
        return;
    }
    float sa[NA], lo_a = __builtin_inff(), hi_a = 0.0f, lo_b = lo_a, hi_b = 0.0f;
#pragma unroll
    for (int j = 0; j < NA; ++j) {
        sa[j] = ends.sa[a0 + j * kF16 + lane % kF16];
        lo_a = __builtin_elementwise_minimum(lo_a, fabsf(sa[j]));
        hi_a = __builtin_elementwise_maximum(hi_a, fabsf(sa[j]));
    }
    const int col = b0 + 4 * (lane / kF16);
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            lo_b = __builtin_elementwise_minimum(lo_b, fabsf(ends.sb[col + i * kF16 + e]));
            hi_b = __builtin_elementwise_maximum(hi_b, fabsf(ends.sb[col + i * kF16 + e]));
        }
    // Whether all scales' products are normal numbers: then value()'s first form alone.
    const bool normal = lo_a * lo_b >= 0x1p-126f && hi_a * hi_b < __builtin_inff();
    auto all = [&](auto plain) {
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const v4f sb = *reinterpret_cast<const v4f*>(ends.sb + col + i * kF16), bias = *reinterpret_cast<const v4f*>(ends.bias + col + i * kF16);
#pragma unroll
            for (int j = 0; j < NA; ++j) {
                v4f v;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    v[e] = decltype(plain)::value ? fmaf((float)acc[i][j][e], sa[j] * sb[e], bias[e]) : value(acc[i][j][e], sa[j], sb[e], bias[e]);
                put(i, j, v);
                __builtin_amdgcn_sched_barrier(0);  // few values in flight
            }
        }
    };
    if (__builtin_expect(__builtin_amdgcn_ballot_w64(!normal) == 0, 1)) all(std::true_type{});
    else all(std::false_type{});
}

// tile_of for fewer than 2^31 tiles, as numbers in scalar registers (the buffer windows that they
// give must be known to be the whole wave's).
__device__ __forceinline__ void tile_at(unsigned g, int64_t rows, int64_t cols, int side, int64_t& m0, int64_t& n0) {
    const unsigned tiles_m = (unsigned)((rows + side - 1) / side), tiles_n = (unsigned)((cols + side - 1) / side);
    const unsigned T = tiles_m * tiles_n, xcd = g % 8, idx = g / 8, per = T / 8, rem = T % 8;
    const unsigned t = xcd * per + min(xcd, rem) + idx;
    const unsigned span = kGroupM * tiles_n, band = t / span, in = t - band * span, first = band * kGroupM;
    const unsigned gm = min(tiles_m - first, (unsigned)kGroupM), n = in / gm;
    m0 = (int64_t)__builtin_amdgcn_readfirstlane(first + in - n * gm) * side;
    n0 = (int64_t)__builtin_amdgcn_readfirstlane(n) * side;
}

// A 256 x 256 tile of C by four waves of 128 x 128, one per SIMD, whose sums fill half of its
// registers: such a wave reads 32 KB of LDS for its 2048 cycles of products per K block, where
// eight waves of 128 x 64 read 192 KB together, as long as the products take.  A K block (128
// bytes per row, a cache line) per stage, two stages.  The operands of the next half block are
// read while this half's products run, so that a stage is free half a block before its products
// end: one barrier per block, and loads go out a block and a half before they are read.
constexpr int kBigThreads = 256;
constexpr int kBigF = 8;                            // fragments of 16 rows per wave and side
constexpr int kBigLoads = (BM + BN) / 8 / 4;        // direct loads per wave and stage

template <int EB>
__device__ __forceinline__ void store_big(const v4i (&acc)[kBigF][kBigF], const Ends<256>& ends, bool partial, uint8_t* lds, void* c,
                                          Rsrc rc, int wave, int lane, int64_t rows_a, int64_t n0, int64_t N, bool whole) {
    typedef EpiPlan<EB> P;
    const int wm = wave / 2, wn = wave % 2;
#pragma unroll
    for (int h = 0; h < P::kPasses; ++h) {
        if (wm * WM / P::kRowsPass == h)
            finish(acc, ends, partial, wm * WM, wn * 128, lane, [&](int i, int j, v4f v) {
                put_quad<EB>(lds, wm * WM + j * kF16 + lane % kF16 - h * P::kRowsPass, (wn * 128 + i * kF16) / 4 + lane / kF16, v[0],
                             v[1], v[2], v[3]);
            });
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 2; ++k) {  // four waves in place of eight
            if (whole) store_pass<EB>(lds, h, c, rc, wave * 2 + k, lane, rows_a, n0, N, true);
            else store_pass<EB>(lds, h, c, rc, wave * 2 + k, lane, rows_a, n0, N, false);
        }
        if (h + 1 < P::kPasses) __syncthreads();
    }
}

__global__ __launch_bounds__(kBigThreads, 1) void k_gemm_i8(I8Params p) {
    __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * kCodeBytes + sizeof(Ends<256>)];
    Ends<256>& ends = *reinterpret_cast<Ends<256>*>(lds + 2 * kCodeBytes);
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wm = wave / 2, wn = wave % 2;
    const int splits = p.splits;
    const unsigned group = p.first + blockIdx.x;
    const int split = __builtin_amdgcn_readfirstlane(group % (unsigned)splits);
    int64_t m0, n0;
    tile_at(group / (unsigned)splits, p.M, p.N, BM, m0, n0);
    const int64_t rows_a = p.M - m0 < BM ? p.M - m0 : BM;
    const int64_t rows_b = p.N - n0 < BN ? p.N - n0 : BN;
    const int K = (int)p.K, S = p.S;
    const int per = __builtin_amdgcn_readfirstlane((S + splits - 1) / splits);
    const int s_lo = split * per, s_hi = s_lo + per < S ? s_lo + per : S;
    const Rsrc ra = make_rsrc(p.a + m0 * K, rows_a * K);
    const Rsrc rb = make_rsrc(p.b + n0 * K, rows_b * K);
    // Load q of a wave moves rows 8 d .. 8 d + 7, d = wave + 4 (q % 8), of A (q < 8) or B, into
    // the slots of op_offset: lane l row 8 d + l / 8, slot l % 8.
    const int piece = (lane % 8) ^ (4 * (wave & 1) + lane / 16);
    const int lane_off = (lane / 8) * K + piece * 16;
    auto issue = [&](int s, int q) {
        const int k0 = s * kBlock;
        const int base = k0 + piece * 16 < (s < s_hi ? K : 0) ? lane_off + k0 : kPastWindow;
        const int d = wave + 4 * (q % (kBigLoads / 2));
        uint8_t* dst = lds + (s & 1) * kCodeBytes + (q < kBigLoads / 2 ? 0 : BM * kRowStage) + d * 8 * kRowStage;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(q < kBigLoads / 2 ? ra : rb, (LdsPtr)dst, 16, base + 8 * d * K, 0, 0, 0);
    };
    v4i acc[kBigF][kBigF];
#pragma unroll
    for (int i = 0; i < kBigF; ++i)
#pragma unroll
        for (int j = 0; j < kBigF; ++j) acc[i][j] = v4i{};
    const int a_row = wm * WM + lane % kF16, b_row = wn * 128 + lane % kF16;
    int a_at[2], b_at[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        a_at[h] = op_offset(a_row, lane, h);
        b_at[h] = BM * kRowStage + op_offset(b_row, lane, h);
    }
    auto read = [&](const uint8_t* at, int frag) { return *reinterpret_cast<const v4i*>(at + frag * kF16 * kRowStage); };
    v4i a[2][kBigF], b[2][kBigF];
    ends.load(p, m0, n0);
    if (s_lo < s_hi) {  // K = 0 has no operands to read
#pragma unroll
        for (int q = 0; q < kBigLoads; ++q) issue(s_lo, q);
#pragma unroll
        for (int q = 0; q < kBigLoads; ++q) issue(s_lo + 1, q);
        // Both stages have landed.  The zeros of the sums are written before the pause: the
        // compiler does not know the products below for matrix instructions.
#pragma unroll
        for (int i = 0; i < kBigF; ++i)
#pragma unroll
            for (int j = 0; j < kBigF; ++j) asm volatile("" : "+a"(acc[i][j]));
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_nop 15\n\ts_barrier" ::: "memory");
        const uint8_t* here = lds + (s_lo & 1) * kCodeBytes;
#pragma unroll
        for (int i = 0; i < kBigF; ++i) b[0][i] = read(here + b_at[0], i);
#pragma unroll
        for (int j = 0; j < kBigF; ++j) a[0][j] = read(here + a_at[0], j);
    }
    for (int s = s_lo; s < s_hi; ++s) {
        const uint8_t* here = lds + (s & 1) * kCodeBytes;
        const uint8_t* next = lds + (~s & 1) * kCodeBytes;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (h == 1) {
                // The next stage has landed, and no wave reads this one any more.
                __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) lgkmcnt(0)
                asm volatile("s_barrier" ::: "memory");
            }
            const uint8_t* from = h == 0 ? here : next;
#pragma unroll
            for (int j = 0; j < kBigF; ++j) {
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int i = 0; i < kBigF; ++i) {
                    mma_in_place(acc[i][j], b[h][i], a[h][j]);
                    if (i == 1) {
                        __builtin_amdgcn_sched_barrier(0);
                        b[1 - h][j] = read(from + b_at[1 - h], j);
                        a[1 - h][j] = read(from + a_at[1 - h], j);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                    if (h == 1 && i == 4) {
                        __builtin_amdgcn_sched_barrier(0);
                        issue(s + 2, 2 * j);
                        issue(s + 2, 2 * j + 1);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
            }
        }
    }
    // LDS is reused below, and the last products are done before their sums are read.
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_nop 15\n\ts_nop 15\n\ts_barrier" ::: "memory");
#pragma unroll
    for (int i = 0; i < kBigF; ++i)
#pragma unroll
        for (int j = 0; j < kBigF; ++j) asm volatile("" : "+a"(acc[i][j]));
    void* c = splits > 1 ? static_cast<void*>(p.partial + (int64_t)split * p.M * p.N) : p.c;
    const int ct = splits > 1 ? 1 : p.ct;
    void* tile = static_cast<char*>(c) + m0 * p.N * (ct == 1 ? 4 : 2);
    const Rsrc rc = make_rsrc(tile, rows_a * p.N * (ct == 1 ? 4 : 2));
    const bool whole = splits > 1 ? (p.N & 3) == 0 : p.whole;
    if (ct == 1) store_big<4>(acc, ends, splits > 1, lds, tile, rc, wave, lane, rows_a, n0, p.N, whole);
    else store_big<2>(acc, ends, false, lds, tile, rc, wave, lane, rows_a, n0, p.N, whole);
}

// Tiles of T x T (128 or 64), four waves of T / 2 x T / 2 through two LDS stages; several
// workgroups share a CU and cover each other's waits.
template <int T>
struct I8Mid {
    static constexpr int kF = T / 2 / kF16;
    static constexpr int kStage = 2 * T * kRowStage;
    static constexpr int kLoads = 2 * T / 8 / 4;
    static constexpr int kPitch = T + 4;
    static constexpr int kTile = 2 * kStage > T * kPitch * 4 ? 2 * kStage : T * kPitch * 4;
    static constexpr int kLds = kTile + (int)sizeof(Ends<T>);
};

template <int T>
__global__ __launch_bounds__(256, T == 128 ? 2 : 4) void k_gemm_i8_mid(I8Params p) {
    typedef I8Mid<T> P;
    constexpr int F = P::kF;
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wm = wave / 2, wn = wave % 2;
    const int splits = p.splits;
    const unsigned group = p.first + blockIdx.x;
    const int split = __builtin_amdgcn_readfirstlane(group % (unsigned)splits);
    int64_t m0, n0;
    tile_at(group / (unsigned)splits, p.M, p.N, T, m0, n0);
    const int rows_a = (int)(p.M - m0 < T ? p.M - m0 : T), rows_b = (int)(p.N - n0 < T ? p.N - n0 : T);
    const int K = (int)p.K, S = p.S;
    const int per = __builtin_amdgcn_readfirstlane((S + splits - 1) / splits);
    const int s_lo = split * per, s_hi = s_lo + per < S ? s_lo + per : S;
    const Rsrc ra = make_rsrc(p.a + m0 * K, (int64_t)rows_a * K);
    const Rsrc rb = make_rsrc(p.b + n0 * K, (int64_t)rows_b * K);
    const int piece = (lane % 8) ^ (4 * (wave & 1) + lane / 16);
    const int lane_off = (lane / 8) * K + piece * 16;
    auto issue = [&](int s) {
        uint8_t* stage = lds + (s & 1) * P::kStage;
        const int k0 = s * kBlock;
        const int base = k0 + piece * 16 < (s < s_hi ? K : 0) ? lane_off + k0 : kPastWindow;
#pragma unroll
        for (int q = 0; q < P::kLoads; ++q) {
            const int d = 4 * q + wave;
            const bool is_a = q < P::kLoads / 2;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(is_a ? ra : rb, (LdsPtr)(stage + d * 8 * kRowStage), 16,
                                                     base + (is_a ? 8 * d : 8 * d - T) * K, 0, 0, 0);
        }
    };
    v4i acc[F][F];
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
        for (int j = 0; j < F; ++j) acc[i][j] = v4i{};
    const int a_row = wm * (T / 2) + lane % kF16, b_row = wn * (T / 2) + lane % kF16;
    const int a_lo = op_offset(a_row, lane, 0), a_hi = op_offset(a_row, lane, 1);
    const int b_lo = T * kRowStage + op_offset(b_row, lane, 0), b_hi = T * kRowStage + op_offset(b_row, lane, 1);
    Ends<T>& ends = *reinterpret_cast<Ends<T>*>(lds + P::kTile);
    if (s_lo < s_hi) issue(s_lo);
    ends.load(p, m0, n0);
    for (int s = s_lo; s < s_hi; ++s) {
        const uint8_t* here = lds + (s & 1) * P::kStage;
        // Stage s has landed, and no wave still reads stage s - 1.
        __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) lgkmcnt(0)
        asm volatile("s_barrier" ::: "memory");
        issue(s + 1);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            v4i a[F], b[F];
#pragma unroll
            for (int i = 0; i < F; ++i) {
                b[i] = *reinterpret_cast<const v4i*>(here + (h ? b_hi : b_lo) + i * kF16 * kRowStage);
                a[i] = *reinterpret_cast<const v4i*>(here + (h ? a_hi : a_lo) + i * kF16 * kRowStage);
            }
#pragma unroll
            for (int j = 0; j < F; ++j)
#pragma unroll
                for (int i = 0; i < F; ++i) acc[i][j] = mma(b[i], a[j], acc[i][j]);
        }
    }
    wait_all_barrier();  // LDS is reused below
    float* st = reinterpret_cast<float*>(lds);
    finish(acc, ends, splits > 1, wm * (T / 2), wn * (T / 2), lane, [&](int i, int j, v4f v) {
        *reinterpret_cast<v4f*>(st + (a_row + j * kF16) * P::kPitch + wn * (T / 2) + i * kF16 + 4 * (lane / kF16)) = v;
    });
    __syncthreads();
    void* c = splits > 1 ? static_cast<void*>(p.partial + (int64_t)split * p.M * p.N) : p.c;
    const int ct = splits > 1 ? 1 : p.ct;
    const int eb = ct == 1 ? 4 : 2;
    void* tile = static_cast<char*>(c) + m0 * p.N * eb;
    const Rsrc rc = make_rsrc(tile, (int64_t)rows_a * p.N * eb);
    const bool whole = splits > 1 ? (p.N & 3) == 0 : p.whole;
    const int units = T * eb / 16;  // 16-byte units per row
    for (int u = threadIdx.x; u < rows_a * units; u += 256) {
        const int r = u / units, col = u % units * (16 / eb);
        const float* src = st + r * P::kPitch + col;
        u32x4_t v;
        if (ct == 1) {
            v = *reinterpret_cast<const u32x4_t*>(src);
        } else {
            const v4f x = *reinterpret_cast<const v4f*>(src), y = *reinterpret_cast<const v4f*>(src + 4);
            v = u32x4_t{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3])};
        }
        if (whole) __builtin_amdgcn_raw_buffer_store_b128(v, rc, col < rows_b ? (int)((r * p.N + n0 + col) * eb) : kDropped, 0, kStoreNT);
        else if (col >= rows_b) continue;
        else if (ct == 1) store_unit<4>(tile, r, n0 + col, p.N, v);
        else store_unit<2>(tile, r, n0 + col, p.N, v);
    }
}

// The sums of K ranges added, and their values.
__global__ __launch_bounds__(256) void k_i8_ranges(I8Params p) {
    const int64_t count = p.M * p.N;
    const int64_t step = (int64_t)gridDim.x * 256;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < count; i += step) {
        int acc = 0;
        for (int r = 0; r < p.splits; ++r) acc += p.partial[r * count + i];
        const int64_t m = i / p.N, n = i - m * p.N;
        const float v = value(acc, p.sa[m], p.sb[n], bias_at(p, n));
        if (p.ct == 1) static_cast<float*>(p.c)[i] = v;
        else static_cast<uint16_t*>(p.c)[i] = (uint16_t)pack_bf16x2(v, v);
    }
}

// At most 16 rows of A: C is a pass over B.  A workgroup takes 16 rows of B, its waves K blocks
// in turn, operands straight into registers; their sums meet in LDS.
constexpr int kFewMaxM = 16;
constexpr int kFewRows = 16;
constexpr int kFewMaxWaves = 16;

__global__ __launch_bounds__(kFewMaxWaves * kWave) void k_gemm_i8_few(I8Params p) {
    constexpr int U = 2;
    __shared__ __attribute__((aligned(16))) int red[kFewMaxWaves * 256];
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int waves = blockDim.x / kWave;
    const int64_t n0 = (int64_t)blockIdx.x * kFewRows;
    const int rows_b = (int)(p.N - n0 < kFewRows ? p.N - n0 : kFewRows);
    const int K = (int)p.K, M = (int)p.M, S = p.S;
    const int r = lane % 16, q = lane / 16;
    const Rsrc rb = make_rsrc(p.b + n0 * K, (int64_t)rows_b * K);
    const Rsrc ra = make_rsrc(p.a, (int64_t)M * K);
    v4i acc = {};
    for (int s0 = wave; s0 < S; s0 += waves * U) {
        u32x4_t b[U][2], a[U][2];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int s = s0 + u * waves, pos = s * kBlock + h * 64 + q * 16;
                const int off = s < S && pos < K ? r * K + pos : kDropped;
                b[u][h] = __builtin_amdgcn_raw_buffer_load_b128(rb, off, 0, 0);
                a[u][h] = __builtin_amdgcn_raw_buffer_load_b128(ra, off, 0, 0);
            }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) acc = mma(__builtin_bit_cast(v4i, b[u][h]), __builtin_bit_cast(v4i, a[u][h]), acc);
    }
    *reinterpret_cast<v4i*>(red + (wave * 16 + r) * 16 + 4 * q) = acc;
    __syncthreads();
    for (int e = threadIdx.x; e < 256; e += blockDim.x) {
        int sum = 0;
        for (int w = 0; w < waves; ++w) sum += red[w * 256 + e];
        const int m = e / 16, n = e % 16;
        if (m < M && n < rows_b) {
            const int64_t at = m * p.N + n0 + n;
            const float v = value(sum, p.sa[m], p.sb[n0 + n], bias_at(p, n0 + n));
            if (p.ct == 1) static_cast<float*>(p.c)[at] = v;
            else static_cast<uint16_t*>(p.c)[at] = (uint16_t)pack_bf16x2(v, v);
        }
    }
}

// Which tile, and how many K ranges per tile: the pair whose modelled time is least, in
// microseconds (a K block of one workgroup while its CU is shared, `each`, and its latency when
// it is not, `alone`; a workgroup's start and epilogue; how many share a CU).
constexpr int64_t kMaxPartialBytes = (int64_t)1 << 28;
struct Choice {
    int tile, splits;
};
struct TileCost {
    int tile, per_cu;
    double alone, each, fixed;
};
constexpr TileCost kTileCosts[] = {{256, 1, 1.2, 1.2, 6.0}, {128, 2, 0.6, 0.42, 4.0}, {64, 4, 0.4, 0.2, 3.0}};
constexpr int kCus = 256;
constexpr int kRanges[] = {1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64};

Choice choose(int64_t M, int64_t N, int64_t K) {
    const int64_t S = (K + kBlock - 1) / kBlock;
    Choice best{128, 1};
    double least = 1e300;
    for (const TileCost& c : kTileCosts) {
        const int64_t tiles = ((M + c.tile - 1) / c.tile) * ((N + c.tile - 1) / c.tile);
        for (const int sp : kRanges) {
            const int64_t per = (S + sp - 1) / sp;
            if (sp > 1 && (sp > S || tiles * sp > 4 * kCus || 4 * sp * M * N > kMaxPartialBytes)) break;
            if (sp > 1 && per * (sp - 1) >= S) continue;  // a range would be empty
            const int64_t groups = (tiles * sp + kCus - 1) / kCus, full = groups / c.per_cu, rest = groups % c.per_cu;
            double t = (double)full * ((double)per * std::max(c.alone, c.each * c.per_cu) + c.fixed);
            if (rest) t += (double)per * std::max(c.alone, c.each * (double)rest) + c.fixed;
            if (sp > 1) t += 3.0 + 8.0 * (double)sp * (double)M * (double)N / 8e6;
            if (t < least) least = t, best = Choice{c.tile, sp};
        }
    }
    return best;
}

int status(const char* what, char* msg, size_t msg_len) {
    const hipError_t e = hipGetLastError();
    if (e == hipSuccess) return 0;
    snprintf(msg, msg_len, "%s kernel launch: %s", what, hipGetErrorString(e));
    return (int)e;
}

template <int WAVES, int CHUNKS>
void launch_quantize_as(I8QuantParams p, int xt, hipStream_t stream) {
    const int64_t groups = WAVES == 1 ? (p.rows + 3) / 4 : p.rows;
    for (int64_t first = 0; first < groups; first += kMaxGrid / 2) {  // (workgroups of up to 1024 threads)
        const dim3 grid((unsigned)std::min(groups - first, kMaxGrid / 2)), block(WAVES == 1 ? 256 : WAVES * kWave);
        p.first = (unsigned)first;
        if (xt == 0) FP4Q_LAUNCH((k_int8_quantize<0, WAVES, CHUNKS>), grid, block, 0, stream, p);
        else FP4Q_LAUNCH((k_int8_quantize<1, WAVES, CHUNKS>), grid, block, 0, stream, p);
    }
}

}  // namespace

size_t int8_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    if (M <= kFewMaxM) return 0;
    const int sp = choose(M, N, K).splits;
    return sp > 1 ? (size_t)(4 * sp * M * N) : 0;
}

int launch_int8_quantize(const Int8QuantJob& j, char* msg, size_t msg_len) {
    if (j.rows == 0) return 0;
    const I8QuantParams p{j.x, j.rows, j.cols, (j.cols + 15) / 16 * 16, j.codes, j.scales, 0};
    hipStream_t stream = static_cast<hipStream_t>(j.stream);
    const int64_t chunks = (p.ld / 8 + kWave - 1) / kWave;  // of a wave
    if (j.rows <= 512 && chunks > 2) {
        if (chunks <= 4) launch_quantize_as<4, 1>(p, j.xt, stream);
        else launch_quantize_as<16, 2>(p, j.xt, stream);
    } else if (chunks <= 2) launch_quantize_as<1, 2>(p, j.xt, stream);
    else if (chunks <= 4) launch_quantize_as<1, 4>(p, j.xt, stream);
    else if (chunks <= 8) launch_quantize_as<4, 2>(p, j.xt, stream);
    else if (chunks <= 16) launch_quantize_as<4, 4>(p, j.xt, stream);
    else if (chunks <= 32) launch_quantize_as<8, 4>(p, j.xt, stream);
    else launch_quantize_as<16, 4>(p, j.xt, stream);
    return status("int8 quantize", msg, msg_len);
}

int launch_int8_gemm(const Int8GemmJob& j, char* msg, size_t msg_len) {
    if (j.M == 0 || j.N == 0) return 0;
    hipStream_t stream = static_cast<hipStream_t>(j.stream);
    const int S = (int)((j.K + kBlock - 1) / kBlock);
    const bool whole = j.N * (j.ct == 1 ? 4 : 2) % 16 == 0 && (uintptr_t)j.c % 16 == 0;
    I8Params p{j.a_codes, j.a_scales, j.b_codes, j.b_scales, j.bias, j.bt, j.M, j.N, j.K, S, j.c, j.ct, whole, 1,
               static_cast<int*>(j.ws), 0};
    if (j.M <= kFewMaxM) {
        const int64_t groups = (j.N + kFewRows - 1) / kFewRows;
        int waves = groups <= 256 ? kFewMaxWaves : groups <= 1024 ? 8 : 4;
        while (waves > 1 && waves >= 2 * S) waves /= 2;
        FP4Q_LAUNCH(k_gemm_i8_few, dim3((unsigned)groups), dim3(waves * kWave), 0, stream, p);
        return status("int8 gemm", msg, msg_len);
    }
    const Choice ch = choose(j.M, j.N, j.K);
    p.splits = ch.splits;
    const int64_t groups = ((j.M + ch.tile - 1) / ch.tile) * ((j.N + ch.tile - 1) / ch.tile) * ch.splits;
    if (groups > INT32_MAX) {
        snprintf(msg, msg_len, "int8 gemm: %lld x %lld x %lld needs more workgroups than one launch holds", (long long)j.M,
                 (long long)j.N, (long long)j.K);
        return (int)hipErrorInvalidConfiguration;
    }
    for (int64_t first = 0; first < groups; first += kMaxGrid) {
        const dim3 grid((unsigned)std::min(groups - first, kMaxGrid));
        p.first = (unsigned)first;
        if (ch.tile == 256) FP4Q_LAUNCH(k_gemm_i8, grid, dim3(kBigThreads), 0, stream, p);
        else if (ch.tile == 128) FP4Q_LAUNCH(k_gemm_i8_mid<128>, grid, dim3(256), I8Mid<128>::kLds, stream, p);
        else FP4Q_LAUNCH(k_gemm_i8_mid<64>, grid, dim3(256), I8Mid<64>::kLds, stream, p);
    }
    if (p.splits > 1)
        FP4Q_LAUNCH(k_i8_ranges, dim3((unsigned)std::min<int64_t>((j.M * j.N + 255) / 256, 2048)), dim3(256), 0, stream, p);
    return status("int8 gemm", msg, msg_len);
}

}  // namespace fp4q
