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
// on use all of it is NaN.  Bound by memory: 8192 x 18944 bf16, 466 MB, 87 to 89 us (5.3 TB/s).

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

// Whether the fused form alone gives value()'s bits: f is a normal number, or a smaller one meets a
// sum of 0, as in a batch's padding, whose rows of zeros have the least scale that there is.  (One such
// row in 256 of 8192 x 18944 x 3584 bf16 sent every tile to the full form: 1083 us, now 461 to 505.)
__device__ __forceinline__ bool plain_value(int acc, float f) {
    return fabsf(f) < __builtin_inff() && (fabsf(f) >= 0x1p-126f || acc == 0);
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
    // Of 256 threads, each brings (T < 256: the first T do) one row's and one column's.
    __device__ __forceinline__ void fetch(float (&v)[3], const I8Params& p, int64_t m0, int64_t n0) const {
        const int t = threadIdx.x % T;
        const int64_t n = min(n0 + t, p.N - 1);
        v[0] = p.sa[min(m0 + t, p.M - 1)];
        v[1] = p.sb[n];
        v[2] = bias_at(p, n);
    }
    __device__ __forceinline__ void put(const float (&v)[3]) {
        if (threadIdx.x < T) sa[threadIdx.x] = v[0], sb[threadIdx.x] = v[1], bias[threadIdx.x] = v[2];
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
    // Whether value()'s first form alone will do: all scales' products are normal numbers, or, looked
    // at one by one, those that are not have nothing to scale.
    bool plain = lo_a * lo_b >= 0x1p-126f && hi_a * hi_b < __builtin_inff();
    if (__builtin_expect(__builtin_amdgcn_ballot_w64(!plain) != 0, 0)) {
        unsigned bad = 0;
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const v4f sb = *reinterpret_cast<const v4f*>(ends.sb + col + i * kF16);
#pragma unroll
            for (int j = 0; j < NA; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) bad |= plain_value(acc[i][j][e], sa[j] * sb[e]) ? 0 : 1;
        }
        plain = bad == 0;
    }
    auto all = [&](auto first) {
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const v4f sb = *reinterpret_cast<const v4f*>(ends.sb + col + i * kF16), bias = *reinterpret_cast<const v4f*>(ends.bias + col + i * kF16);
#pragma unroll
            for (int j = 0; j < NA; ++j) {
                v4f v;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    v[e] = decltype(first)::value ? fmaf((float)acc[i][j][e], sa[j] * sb[e], bias[e]) : value(acc[i][j][e], sa[j], sb[e], bias[e]);
                put(i, j, v);
                __builtin_amdgcn_sched_barrier(0);  // few values in flight
            }
        }
    };
    if (__builtin_expect(__builtin_amdgcn_ballot_w64(!plain) == 0, 1)) all(std::true_type{});
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

// Tiles of 256 x 256 (F = 8) by four waves of 128 x 128, one per SIMD, whose sums fill half of
// its registers: such a wave reads 32 KB of LDS for its 2048 cycles of products per K block,
// where eight waves of 128 x 64 read 192 KB together, as long as the products take.  A K block
// (128 bytes per row, a cache line) per stage, two stages.  The operands of the next half block
// are read while this half's products run, so that a stage is free half a block before its
// products end: one barrier per block, and loads go out a block and a half before they are read.
// Workgroups are persistent: a tile's first two stages are loaded while the tile before is
// scaled and stored, straight from registers, so that LDS is free.  4096 x 4096 x 14336 to bf16:
// 157 to 177 us by box (2.7 to 3.1 POP/s), the matrix cores busy in 70% to 72% of the cycles at 1.9 GHz;
// 125 us with operands of zero, so that power is part of what bounds it.
//
// For that a lane's columns are neighbours: fragment i of a wave's B holds at position r its row
// 4 F (r / 4) + 4 i + r % 4, so that lane l ends up with columns 4 F (l / 16) .. + 4 F - 1 of row
// l % 16 of each fragment of A.  B's slots in LDS go by ((row / 2) % 2 + 2 (row / 4 F)) % 8 in the
// place of (row / 2) % 8, which keeps the rows that are read together in distinct banks.
constexpr int kBigThreads = 256;
constexpr int kSpread = 4096;                       // LDS bytes that a wave spreads its rows through

// One tile (of one K range) of a product.
template <int F>
struct BigTile {
    static constexpr int T = 32 * F;               // rows and columns
    static constexpr int kStage = 2 * T * kRowStage;
    static constexpr int kLoads = 2 * T / 8 / 4;   // direct loads per wave and stage
    int64_t m0, n0;
    int rows_a, rows_b, s_lo, s_hi, split;
    Rsrc ra, rb;

    __device__ __forceinline__ BigTile(const I8Params& p, int64_t m, int64_t n, int range) : m0(m), n0(n), split(range) {
        rows_a = (int)(p.M - m0 < T ? p.M - m0 : T);
        rows_b = (int)(p.N - n0 < T ? p.N - n0 : T);
        const int per = __builtin_amdgcn_readfirstlane((p.S + p.splits - 1) / p.splits);
        s_lo = split * per;
        s_hi = s_lo + per < p.S ? s_lo + per : p.S;
        ra = make_rsrc(p.a + m0 * p.K, (int64_t)rows_a * p.K);
        rb = make_rsrc(p.b + n0 * p.K, (int64_t)rows_b * p.K);
    }
    // Load q of a stage moves rows 8 d .. 8 d + 7, d = wave + 4 (q % half), of A (the first half
    // of the loads) or B: lane l row 8 d + l / 8, slot l % 8.  `at` holds the lane's offset of each
    // load, so that the loop over K moves nothing but the stage's scalar offset.
    int at[kLoads];
    __device__ __forceinline__ void offsets(int K, int wave, int lane) {
#pragma unroll
        for (int q = 0; q < kLoads; ++q) at[q] = (8 * load_row(q, wave) + lane / 8) * K + 16 * load_piece(q, wave, lane);
    }
    static __device__ __forceinline__ int load_row(int q, int wave) { return wave + 4 * (q % (kLoads / 2)); }
    static __device__ __forceinline__ int load_piece(int q, int wave, int lane) {
        return (lane % 8) ^ (q < kLoads / 2 ? 4 * (wave & 1) + lane / 16 : lane / 16 % 2 + 2 * (2 * load_row(q, wave) / F % 4));
    }
    // Before the loads of stage s: pieces past K or the range are not read (zeros take their place).
    __device__ __forceinline__ void cut(int K, int s, int wave, int lane) {
        if (__builtin_expect((s + 1) * kBlock <= K && s < s_hi, 1)) return;
        if (s >= s_hi) {
#pragma unroll
            for (int q = 0; q < kLoads; ++q) at[q] = kPastWindow;
            return;
        }
#pragma unroll
        for (int q = 0; q < kLoads; ++q) at[q] = s * kBlock + 16 * load_piece(q, wave, lane) < K ? at[q] : kPastWindow;
    }
    __device__ __forceinline__ void issue(uint8_t* lds, int wave, int s, int q) const {
        const bool is_a = q < kLoads / 2;
        uint8_t* dst = lds + (s & 1) * kStage + (is_a ? 0 : T * kRowStage) + load_row(q, wave) * 8 * kRowStage;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(is_a ? ra : rb, (LdsPtr)dst, 16, at[q], s * kBlock, 0, 0);
    }
    __device__ __forceinline__ void first_stages(uint8_t* lds, int K, int wave, int lane) {
        if (s_lo >= s_hi) return;  // K = 0 has no operands to read
        offsets(K, wave, lane);
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            cut(K, s_lo + n, wave, lane);
#pragma unroll
            for (int q = 0; q < kLoads; ++q) issue(lds, wave, s_lo + n, q);
        }
    }
    // The sums, from two stages that have landed.
    __device__ __forceinline__ void sums(v4i (&acc)[F][F], uint8_t* lds, int K, int wave, int lane) {
        const int r = lane % kF16, wm = wave / 2, wn = wave % 2;
        const int a_row = wm * 16 * F + r, b_row = wn * 16 * F + 4 * F * (r / 4) + r % 4;
        int a_at[2], b_at[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            a_at[h] = op_offset(a_row, lane, h);
            const int slot = (lane / kF16 + 4 * h) ^ (r / 2 % 2 + 2 * (r / 4));
            b_at[h] = T * kRowStage + b_row * kRowStage + slot * 16;
        }
        auto read_a = [&](const uint8_t* stage, int h, int j) { return *reinterpret_cast<const v4i*>(stage + a_at[h] + j * kF16 * kRowStage); };
        auto read_b = [&](const uint8_t* stage, int h, int i) { return *reinterpret_cast<const v4i*>(stage + b_at[h] + i * 4 * kRowStage); };
#pragma unroll
        for (int i = 0; i < F; ++i)
#pragma unroll
            for (int j = 0; j < F; ++j) acc[i][j] = v4i{};
        // The zeros are written before the pause: the compiler does not know the products below
        // for matrix instructions.
#pragma unroll
        for (int i = 0; i < F; ++i)
#pragma unroll
            for (int j = 0; j < F; ++j) asm volatile("" : "+a"(acc[i][j]));
        asm volatile("s_nop 15" ::: "memory");
        if (s_lo >= s_hi) return;
        v4i a[2][F], b[2][F];
        {
            const uint8_t* here = lds + (s_lo & 1) * kStage;
#pragma unroll
            for (int i = 0; i < F; ++i) b[0][i] = read_b(here, 0, i);
#pragma unroll
            for (int j = 0; j < F; ++j) a[0][j] = read_a(here, 0, j);
        }
        for (int s = s_lo; s < s_hi; ++s) {
            const uint8_t* here = lds + (s & 1) * kStage;
            const uint8_t* next = lds + (~s & 1) * kStage;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (h == 1) {
                    // The next stage has landed, and no wave reads this one any more.
                    __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) lgkmcnt(0)
                    asm volatile("s_barrier" ::: "memory");
                    cut(K, s + 2, wave, lane);
                }
                const uint8_t* from = h == 0 ? here : next;
#pragma unroll
                for (int j = 0; j < F; ++j) {
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int i = 0; i < F; ++i) {
                        mma_in_place(acc[i][j], b[h][i], a[h][j]);
                        if (i == 1) {
                            __builtin_amdgcn_sched_barrier(0);
                            b[1 - h][j] = read_b(from, 1 - h, j);
                            __builtin_amdgcn_sched_barrier(0);
                        }
                        if (i == F / 2 + 1) {
                            __builtin_amdgcn_sched_barrier(0);
                            a[1 - h][j] = read_a(from, 1 - h, j);
                            __builtin_amdgcn_sched_barrier(0);
                        }
                        if (h == 1 && i % 4 == 3) {
                            __builtin_amdgcn_sched_barrier(0);
                            constexpr int kEach = kLoads * 4 / (F * F);
#pragma unroll
                            for (int e = 0; e < kEach; ++e) issue(lds, wave, s + 2, (j * (F / 4) + i / 4) * kEach + e);
                            __builtin_amdgcn_sched_barrier(0);
                        }
                    }
                }
            }
        }
        // The last products are done before their sums are read.
        asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
#pragma unroll
        for (int i = 0; i < F; ++i)
#pragma unroll
            for (int j = 0; j < F; ++j) asm volatile("" : "+a"(acc[i][j]));
    }
    // A sum out of its accumulation register.  (Left to the compiler, all of them moved at once.)
    static __device__ __forceinline__ int sum_of(const v4i& c, int e) {
        int v;
        asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(v) : "a"(c[e]));
        return v;
    }
    // The values of the sums (PARTIAL: the sums) to memory, EB bytes each, 16 bytes a store.
    // HOW: 0 C's rows start on 16 bytes, 1 they do not, 2 element by element and by value()'s
    // full form, for a tile whose rows end inside 16 bytes or whose scales need it.
    template <int EB, bool PARTIAL, int HOW>
    __device__ __forceinline__ void store(const v4i (&acc)[F][F], const I8Params& p, const Ends<T>& ends, uint8_t* spread, int wave, int lane) const {
        typedef uint32_t Unit __attribute__((ext_vector_type(4), aligned(2)));
        const int wm = wave / 2, wn = wave % 2, r = lane % kF16, q = lane / kF16, col = wn * 16 * F + 4 * F * q;
        char* c = PARTIAL ? reinterpret_cast<char*>(p.partial + (int64_t)split * p.M * p.N) : static_cast<char*>(p.c);
        c += m0 * p.N * EB;
        const Rsrc rc = make_rsrc(c, rows_a * p.N * EB);
        v4f sb[F], bias[F];
#pragma unroll
        for (int i = 0; i < F; ++i) {
            sb[i] = *reinterpret_cast<const v4f*>(ends.sb + col + 4 * i);
            bias[i] = *reinterpret_cast<const v4f*>(ends.bias + col + 4 * i);
        }
        float sa;
        auto at = [&](int i, int j, int e) {
            const int sum = sum_of(acc[i][j], e);
            if (PARTIAL) return __int_as_float(sum);
            return HOW == 2 ? value(sum, sa, sb[i][e], bias[i][e]) : fmaf((float)sum, sa * sb[i][e], bias[i][e]);
        };
        if (HOW == 2) {
#pragma unroll
            for (int j = 0; j < F; ++j) {
                const int row = wm * 16 * F + j * kF16 + r;
                sa = ends.sa[row];
#pragma unroll
                for (int i = 0; i < F; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int n = col + 4 * i + e, off = row < rows_a && n < rows_b ? (int)((row * p.N + n0 + n) * EB) : kDropped;
                        const float v = at(i, j, e);
                        if (EB == 4) __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), rc, off, 0, 0);
                        else __builtin_amdgcn_raw_buffer_store_b16((unsigned short)pack_bf16x2(v, v), rc, off, 0, 0);
                    }
                __builtin_amdgcn_sched_barrier(0);  // few values in flight
            }
            return;
        }
        // The rows of a fragment of A go through the wave's own 4 KB of LDS, kRows in a step, so
        // that a store covers whole lines.  (A lane's 64 bytes stored by itself, 16 at a time, took
        // 170 us for 8192 x 16384 bf16, half as long as its products.)  Unit u of row r sits at
        // u ^ r: a write's rows and a read's units fall in distinct banks.
        constexpr int kUnits = F * EB;                       // of 16 bytes, in a row of the wave
        constexpr int kMine = F * EB / 4;                    // those of a lane
        constexpr int kPerRead = kWave / kUnits;             // rows
        constexpr int kReads = kPerRead < 8 ? 4 : 2;
        constexpr int kRows = kReads * kPerRead;             // in a step
        constexpr int kSteps = F * 16 / kRows;
        static_assert(kRows <= 16 && kRows * kUnits * 16 <= kSpread, "a step is part of a fragment");
        u32x4_t w[kReads], v[kMine];
        auto store_step = [&](int step) {
#pragma unroll
            for (int t = 0; t < kReads; ++t) {
                const int m = wm * 16 * F + step * kRows + t * kPerRead + lane / kUnits, n = wn * 16 * F + lane % kUnits * (16 / EB);
                const bool in = m < rows_a && n < rows_b;
                const int64_t off = ((int64_t)m * p.N + n0 + n) * EB;
                if (HOW == 0) __builtin_amdgcn_raw_buffer_store_b128(w[t], rc, in ? (int)off : kDropped, 0, kStoreNT);
                else if (in) *reinterpret_cast<Unit*>(c + off) = w[t];
            }
        };
#pragma unroll
        for (int step = 0; step < kSteps; ++step) {
            __builtin_amdgcn_sched_barrier(0);  // few values in flight
            const int j = step * kRows / 16, h = step % (16 / kRows);
            if (h == 0) {
                sa = PARTIAL ? 0.0f : ends.sa[wm * 16 * F + j * kF16 + r];
#pragma unroll
                for (int k = 0; k < kMine; ++k)
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        v[k][u] = EB == 4 ? __float_as_uint(at(k, j, u))
                                          : pack_bf16x2(at(2 * k + u / 2, j, u % 2 * 2), at(2 * k + u / 2, j, u % 2 * 2 + 1));
            }
            if (r / kRows == h) {
#pragma unroll
                for (int k = 0; k < kMine; ++k)
                    *reinterpret_cast<u32x4_t*>(spread + (r % kRows * kUnits + ((q * kMine + k) ^ r) % kUnits) * 16) = v[k];
            }
            asm volatile("" ::: "memory");  // (a wave's LDS accesses run in order)
#pragma unroll
            for (int t = 0; t < kReads; ++t) {
                const int rr = t * kPerRead + lane / kUnits, u = lane % kUnits;
                w[t] = *reinterpret_cast<const u32x4_t*>(spread + (rr * kUnits + (u ^ (h * kRows + rr)) % kUnits) * 16);
            }
            asm volatile("" ::: "memory");
            store_step(step);
        }
    }
    // Whether the first form of value() alone will do for the wave, as in finish(): the scales' products
    // one by one (about 3 us) in the fragments of A alone where one may be no normal number.
    __device__ __forceinline__ bool plain(const v4i (&acc)[F][F], const Ends<T>& ends, int wave, int lane) const {
        float lo_a = __builtin_inff(), hi_a = 0.0f, lo_b = lo_a, hi_b = 0.0f;
        for (int t = lane; t < T; t += kWave) {
            lo_a = __builtin_elementwise_minimum(lo_a, fabsf(ends.sa[t])), hi_a = __builtin_elementwise_maximum(hi_a, fabsf(ends.sa[t]));
            lo_b = __builtin_elementwise_minimum(lo_b, fabsf(ends.sb[t])), hi_b = __builtin_elementwise_maximum(hi_b, fabsf(ends.sb[t]));
        }
#pragma unroll
        for (int d = 1; d < kWave; d *= 2) {
            lo_a = __builtin_elementwise_minimum(lo_a, __shfl_xor(lo_a, d)), hi_a = __builtin_elementwise_maximum(hi_a, __shfl_xor(hi_a, d));
            lo_b = __builtin_elementwise_minimum(lo_b, __shfl_xor(lo_b, d)), hi_b = __builtin_elementwise_maximum(hi_b, __shfl_xor(hi_b, d));
        }
        if (__builtin_expect(__builtin_amdgcn_ballot_w64(!(lo_a * lo_b >= 0x1p-126f && hi_a * hi_b < __builtin_inff())) == 0, 1)) return true;
        const int col = wave % 2 * 16 * F + 4 * F * (lane / kF16);
        unsigned bad = 0;
#pragma unroll
        for (int j = 0; j < F; ++j) {
            const float sa = ends.sa[wave / 2 * 16 * F + j * kF16 + lane % kF16];
            if (__builtin_amdgcn_ballot_w64(!(fabsf(sa) * lo_b >= 0x1p-126f && fabsf(sa) * hi_b < __builtin_inff())) == 0) continue;
#pragma unroll
            for (int i = 0; i < F; ++i) {
                const v4f sb = *reinterpret_cast<const v4f*>(ends.sb + col + 4 * i);
#pragma unroll
                for (int e = 0; e < 4; ++e) bad |= plain_value(sum_of(acc[i][j], e), sa * sb[e]) ? 0 : 1;
                __builtin_amdgcn_sched_barrier(0);  // few values in flight
            }
        }
        return __builtin_amdgcn_ballot_w64(bad != 0) == 0;
    }
    template <int EB, bool PARTIAL>
    __device__ __forceinline__ void store(const v4i (&acc)[F][F], const I8Params& p, const Ends<T>& ends, uint8_t* spread, int wave, int lane, bool plain) const {
        const bool whole = PARTIAL ? (p.N & 3) == 0 : p.whole;
        if (plain && whole) store<EB, PARTIAL, 0>(acc, p, ends, spread, wave, lane);
        else if (plain && rows_b % (16 / EB) == 0) store<EB, PARTIAL, 1>(acc, p, ends, spread, wave, lane);
        else store<EB, PARTIAL, 2>(acc, p, ends, spread, wave, lane);
    }
};

template <int F>
__device__ __forceinline__ void store_any(const BigTile<F>& tile, const v4i (&acc)[F][F], const I8Params& p, const Ends<32 * F>& ends,
                                          uint8_t* spread, int wave, int lane) {
    const bool plain = p.splits > 1 || tile.plain(acc, ends, wave, lane);
    asm volatile("" : "+v"(lane));  // addresses are formed here, not kept through the sums
    if (p.splits > 1) tile.template store<4, true>(acc, p, ends, spread, wave, lane, plain);
    else if (p.ct == 1) tile.template store<4, false>(acc, p, ends, spread, wave, lane, plain);
    else tile.template store<2, false>(acc, p, ends, spread, wave, lane, plain);
}

// Items: a tile and a K range each, dealt to the workgroups in turn.  `quarters`: the last so many
// tiles (without K ranges), too few to give each workgroup one, go out as four tiles of 128 x 128
// each, one to a workgroup.
__global__ __launch_bounds__(kBigThreads, 1) void k_gemm_i8(I8Params p, unsigned items, unsigned quarters) {
    typedef BigTile<8> Tile;
    typedef BigTile<4> Quarter;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * Tile::kStage + sizeof(Ends<Tile::T>) + 4 * kSpread];
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int K = (int)p.K;
    uint8_t* spread = lds + 2 * Tile::kStage + sizeof(Ends<Tile::T>) + wave * kSpread;
    float end[3];
    if (blockIdx.x < items) {
        Ends<Tile::T>& ends = *reinterpret_cast<Ends<Tile::T>*>(lds + 2 * Tile::kStage);
        auto item = [&](unsigned g) {
            int64_t m0, n0;
            tile_at(g / (unsigned)p.splits, p.M, p.N, Tile::T, m0, n0);
            return Tile(p, m0, n0, __builtin_amdgcn_readfirstlane(g % (unsigned)p.splits));
        };
        Tile tile = item(blockIdx.x);
        tile.first_stages(lds, K, wave, lane);
        ends.fetch(end, p, tile.m0, tile.n0);
        for (unsigned g = blockIdx.x; g < items; g += gridDim.x) {
            ends.put(end);
            asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");  // both stages have landed
            v4i acc[8][8];
            tile.sums(acc, lds, K, wave, lane);
            asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");  // no wave reads or fills a stage any more
            const Tile done = tile;
            if (g + gridDim.x < items) {
                tile = item(g + gridDim.x);
                tile.first_stages(lds, K, wave, lane);
                ends.fetch(end, p, tile.m0, tile.n0);
            }
            __builtin_amdgcn_sched_barrier(0);
            store_any<8>(done, acc, p, ends, spread, wave, lane);
            __syncthreads();  // `ends` is read before the next tile's take its place
        }
    }
    // Quarters of one tile go to workgroups 8 apart: to one XCD.
    const unsigned left = blockIdx.x / 32 * 8 + blockIdx.x % 8, quarter = blockIdx.x / 8 % 4;
    if (left >= quarters) return;
    int64_t m0, n0;
    tile_at(items + left, p.M, p.N, Tile::T, m0, n0);
    m0 += quarter / 2 * Quarter::T;
    n0 += quarter % 2 * Quarter::T;
    if (m0 >= p.M || n0 >= p.N) return;
    Ends<Quarter::T>& ends = *reinterpret_cast<Ends<Quarter::T>*>(lds + 2 * Tile::kStage);
    Quarter tile(p, m0, n0, 0);
    tile.first_stages(lds, K, wave, lane);
    ends.fetch(end, p, m0, n0);
    ends.put(end);
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    v4i acc[4][4];
    tile.sums(acc, lds, K, wave, lane);
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    store_any<4>(tile, acc, p, ends, spread, wave, lane);
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
    float end[3];
    ends.fetch(end, p, m0, n0);
    ends.put(end);
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
// in turn, operands straight into registers, the next blocks' on their way while these are
// multiplied; their sums meet in LDS.
// XT >= 0: one row of A, not codes but x itself (0 bf16, 1 f32), which each workgroup quantizes
// into LDS with the first of B's blocks on their way: about 2 us where each CU has one workgroup,
// less than a launch of its own.  Where a CU has several, one after the other, it is not (1 x 4096
// x 14336: 23.1 us against 18.3 and the launch), nor for more rows (8 x 4096: 13 us).
constexpr int kFewMaxM = 16;
constexpr int kFewRows = 16;
constexpr int kFewMaxWaves = 16;
constexpr int kFewMaxCodes = 1 << 15;  // of x, in LDS

template <int XT>
__global__ __launch_bounds__(kFewMaxWaves * kWave) void k_gemm_i8_few(I8Params p, const void* x, int cols) {
    constexpr bool OWN = XT >= 0;
    __shared__ __attribute__((aligned(16))) int red[kFewMaxWaves * 256];
    __shared__ __attribute__((aligned(16))) int8_t codes[OWN ? kFewMaxCodes : 16];
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int waves = blockDim.x / kWave;
    const int64_t n0 = (int64_t)blockIdx.x * kFewRows;
    const int rows_b = (int)(p.N - n0 < kFewRows ? p.N - n0 : kFewRows);
    const int K = (int)p.K, M = (int)p.M, S = p.S;
    const int r = lane % 16, q = lane / 16;
    const Rsrc rb = make_rsrc(p.b + n0 * K, (int64_t)rows_b * K);
    const Rsrc ra = make_rsrc(p.a, OWN ? 0 : (int64_t)M * K);
    struct Block { u32x4_t a[2], b[2]; };
    auto place = [&](int s, int h) {
        const int pos = s * kBlock + h * 64 + q * 16;
        return s < S && pos < K ? r * K + pos : kDropped;
    };
    auto load = [&](Block& t, int s) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            t.b[h] = __builtin_amdgcn_raw_buffer_load_b128(rb, place(s, h), 0, 0);
            if (!OWN) t.a[h] = __builtin_amdgcn_raw_buffer_load_b128(ra, place(s, h), 0, 0);
        }
    };
    // One block read ahead (1 x 18944 x 3584: 17.6 us by events; two at once 18.4, four 19.5, two
    // and none ahead 20.8).
    Block now, next;
    load(now, wave);
    float scale = 0.0f;
    if (OWN) {
        constexpr int kHeld = 3;  // pieces of 8 that a thread keeps
        float* part = reinterpret_cast<float*>(red);  // each wave's maximum
        float v[kHeld][8], u[8], top = 0.0f;
        const int at0 = threadIdx.x * 8, step = blockDim.x * 8;
#pragma unroll
        for (int c = 0; c < kHeld; ++c) load8<XT>(v[c], x, min(at0 + c * step, cols), cols);
#pragma unroll
        for (int c = 0; c < kHeld; ++c) top = max8(v[c], top);
        for (int at = at0 + kHeld * step; at < cols; at += step) {
            load8<XT>(u, x, at, cols);
            top = max8(u, top);
        }
        top = wave_max(top);
        if (lane == 0) part[wave] = top;
        __syncthreads();
        for (int w = 0; w < waves; ++w) top = __builtin_elementwise_maximum(top, part[w]);
        const RowScale sc(top);
        scale = sc.s;
#pragma unroll
        for (int c = 0; c < kHeld; ++c)
            if (at0 + c * step < K) *reinterpret_cast<uint2*>(codes + at0 + c * step) = sc.codes(v[c]);
        for (int at = at0 + kHeld * step; at < K; at += step) {
            load8<XT>(u, x, min(at, cols), cols);
            *reinterpret_cast<uint2*>(codes + at) = sc.codes(u);
        }
        __syncthreads();
    }
    v4i acc = {};
    for (int s = wave; s < S; s += waves) {
        load(next, s + waves);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (OWN) {
                const int off = place(s, h);
                now.a[h] = u32x4_t{0, 0, 0, 0};
                if (r == 0 && off != kDropped) now.a[h] = *reinterpret_cast<const u32x4_t*>(codes + off);
            }
            acc = mma(__builtin_bit_cast(v4i, now.b[h]), __builtin_bit_cast(v4i, now.a[h]), acc);
        }
        now = next;
    }
    *reinterpret_cast<v4i*>(red + (wave * 16 + r) * 16 + 4 * q) = acc;
    __syncthreads();
    for (int e = threadIdx.x; e < 256; e += blockDim.x) {
        const int m = e / 16, n = e % 16;
        if (m >= M || n >= rows_b) continue;
        int sum = 0;
        for (int w = 0; w < waves; ++w) sum += red[w * 256 + e];
        const int64_t at = m * p.N + n0 + n;
        const float v = value(sum, OWN ? scale : p.sa[m], p.sb[n0 + n], bias_at(p, n0 + n));
        if (p.ct == 1) static_cast<float*>(p.c)[at] = v;
        else static_cast<uint16_t*>(p.c)[at] = (uint16_t)pack_bf16x2(v, v);
    }
}

// Which tile, and how many K ranges per tile: the pair whose modelled time is least, in
// microseconds (a K block of one workgroup while its CU is shared, `each`, and its latency when
// it is not, `alone`; a workgroup's start and epilogue; how many share a CU).  Choices beside the
// tile and ranges that come next, us to bf16: 17 x 3584 x 18944 (64, 8) 25, (128, 8) 28; 64 x 18944 x 3584
// (64, 1) and (64, 2) 26, (128, 1) 30, and of 17 rows (64, 1) 25, where (64, 2) takes 21; 333 x 1031 x 1008 (64, 1) 6.7, (64, 2) 9.6; 512 x 3584
// x 18944 (128, 4) 65, (256, 8) 62; 1024 rows (256, 4) 86 to 90, (128, 2) 106; 2048 rows (256, 2) 139 to 149,
// (128, 1) 160; 2048^3 (128, 1) 16.1, (64, 1) 17.3; 4096^3 (256, 1) 56, (128, 1) 70 to 76.  Latency that
// nothing hides is not in it: 333 x 1031 x 1008 is 3.9 us by the model.
constexpr int64_t kMaxPartialBytes = (int64_t)1 << 28;
struct Choice {
    int tile, splits;
};
struct TileCost {
    int tile, per_cu;
    double alone, each, fixed;
};
constexpr TileCost kTileCosts[] = {{256, 1, 1.35, 1.35, 7.0}, {128, 2, 0.58, 0.48, 2.5}, {64, 4, 0.3, 0.195, 1.5}};
constexpr int kCus = 256;
constexpr int kRanges[] = {1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64};

// How many of the tiles of 256 x 256, dealt to all CUs in turn, are left for a last round in which
// four workgroups can share each.
int64_t quartered(int64_t tiles, int splits) {
    const int64_t rest = tiles % kCus;
    return splits == 1 && tiles > kCus && rest <= kCus / 4 ? rest : 0;
}

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
            const int64_t quarters = c.tile == 256 ? quartered(tiles, sp) : 0;
            const int64_t groups = (tiles * sp - quarters + kCus - 1) / kCus, full = groups / c.per_cu, rest = groups % c.per_cu;
            double t = (double)full * ((double)per * std::max(c.alone, c.each * c.per_cu) + c.fixed);
            if (rest) t += (double)per * std::max(c.alone, c.each * (double)rest) + c.fixed;
            if (quarters) t += (double)per * 0.6 + 4.0;
            if (sp > 1) t += 4.0 + 8.0 * (double)sp * (double)M * (double)N / 8e6;
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

bool int8_linear_in_one(int64_t M, int64_t N, int64_t K) { return M == 1 && K <= kFewMaxCodes && N <= kFewRows * kCus; }

int launch_int8_quantize(const Int8QuantJob& j, char* msg, size_t msg_len) {
    if (j.rows == 0) return 0;
    const I8QuantParams p{j.x, j.rows, j.cols, (j.cols + 15) / 16 * 16, j.codes, j.scales, 0};
    hipStream_t stream = static_cast<hipStream_t>(j.stream);
    const int64_t chunks = (p.ld / 8 + kWave - 1) / kWave;  // of a wave
    // Up to 512 rows, fewer than fill the chip by themselves: more waves a row.  (us, launches one after the
    // other, beside what more rows take: 256 x 2048 3.3 and 4.3, 512 x 2048 3.6 and 4.3, 2048 x 2048 5.8 and
    // 4.9; 1 x 3584 3.3 and 3.2, 512 x 3584 4.9 and 3.9, 2048 x 3584 11.8 and 7.2; 1 x 8192 3.4 and 4.0, 512 x
    // 8192 5.3 and 4.9; 1 x 18944 4.0 and 4.3, 512 x 18944 8.8 and 9.2, 2048 x 18944 28 and 27.  A row of
    // more than 16384 is read in part again: 1 x 32768 6.3 and 4.6.)
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
        const dim3 grid((unsigned)groups), block(waves * kWave);
        if (j.xt < 0) FP4Q_LAUNCH((k_gemm_i8_few<-1>), grid, block, 0, stream, p, nullptr, 0);
        else if (j.xt == 0) FP4Q_LAUNCH((k_gemm_i8_few<0>), grid, block, 0, stream, p, j.x, (int)j.cols);
        else FP4Q_LAUNCH((k_gemm_i8_few<1>), grid, block, 0, stream, p, j.x, (int)j.cols);
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
        if (ch.tile == 256) {
            const int64_t quarters = quartered(groups, p.splits);
            FP4Q_LAUNCH(k_gemm_i8, dim3((unsigned)std::min<int64_t>(groups, kCus)), dim3(kBigThreads), 0, stream, p,
                        (unsigned)(groups - quarters), (unsigned)quarters);
            break;
        }
        if (ch.tile == 128) FP4Q_LAUNCH(k_gemm_i8_mid<128>, grid, dim3(256), I8Mid<128>::kLds, stream, p);
        else FP4Q_LAUNCH(k_gemm_i8_mid<64>, grid, dim3(256), I8Mid<64>::kLds, stream, p);
    }
    if (p.splits > 1)
        FP4Q_LAUNCH(k_i8_ranges, dim3((unsigned)std::min<int64_t>((j.M * j.N + 255) / 256, 2048)), dim3(256), 0, stream, p);
    return status("int8 gemm", msg, msg_len);
}

}  // namespace fp4q
