// fp4q_fp8_gemm.hip -- products of E4M3 operands with one binary32 scale per 128
// elements along K (fp8_gemm_b128).
//
// C[m][n] = sum over K blocks s of sa[s][m] sb[s][n] P_s[m][n],
// P_s[m][n] = sum over the block's 128 elements of A[m][k] B[n][k].
//
// The scales are arbitrary binary32 numbers, which the matrix cores' power-of-two
// block scales cannot apply: each P_s is formed from zero and added to the binary32 sum by a fused
// multiply-add under the product of the two scales.  A's scales go by row of A,
// which is a lane of the result; B's are one number per 128 x 128 ("tile"), so
// that the factor is one per lane and fragment, or one per row of B ("row"),
// which costs a multiplication more per element.  Where the product of two scales
// passes binary32's range they go one after the other (d sb, then the sum with sa:
// both are at least 1 there, so that d sb overflows only where d sa sb does).  No K
// loop tests for that: an infinite factor leaves an infinity or NaN in its sum, whatever
// follows, and a wave that finds one in its sums forms them again (sums_again).
//
// The matrix cores' 8-bit form keeps a product only to about 2^-17 of the largest
// that it adds (measured over 128 Normal products: 1.4e-5 of the result, 2^-15.5 of
// sum |a b| at worst, whatever the instruction's depth).  That is a hundredth of a
// bf16 rounding, so a bf16 C takes it.  A binary32 C is computed on the bf16 form,
// at half the rate: E4M3 values are exact in bf16, and its sums are binary32 ones
// (1e-8 of the result on the same products).
//
// Kernels:
//  k_gemm_fp8        a workgroup of 8 waves computes a 256 x 256 tile of C, as
//                    the FP4 kernels do, one K block of 128 bytes per row (a
//                    cache line) per stage, through two LDS stages; a bf16 C;
//  k_gemm_fp8_mid    the same in 128 x 128 or 64 x 64 tiles, for products that the
//                    large tile leaves the chip idle with, and for a binary32 C;
//  k_gemm_fp8_few    at most 16 rows of A: one pass over B, 16 rows of B per
//                    workgroup, K blocks dealt to its waves in turn; bound by the
//                    read of B, so always on the bf16 form.
//
// Measured: 8192 x 18944 x 3584 bf16 475 to 494 us (2.25 to 2.34 PFLOP/s; 515 on inputs
// that change from pass to pass, where the library's product under one scale per tensor
// took 424), 4096 x 4096 x 14336 186 us (2.59), with row scales 14336 x 4096 x 4096 251
// (1.92); binary32 C 4096 x 14336 x 4096 430 us (1.12 PFLOP/s on the bf16 cores); 1 x 3584
// x 18944 13.8 us (4.9 TB/s of B).
// What bounds the large tile: at 4096 x 4096 x 14336, one tile per CU, its cycles are
// half as many again as the matrix cores need.  Timing copies of it took 143 us without
// the direct loads into LDS, 147 without the reads of LDS, about 170 with half of either,
// 185 without any wait or barrier and 160 without the scaling: loads and reads of LDS
// contend, whatever their order (next operands read a stage ahead, B past LDS, persistent
// workgroups: none was faster).
//
// All accesses go through range-checked windows: rows past M or N and K pieces
// past K read zeros (code +0), stores outside C are dropped.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <stdio.h>

#include <algorithm>
#include <type_traits>

#include "fp4q_gemm_tile.h"
#include "fp4q_launch.h"

namespace fp4q {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));

constexpr int kBlock = 128;                     // K elements per scale and per stage
constexpr int kLoads = (BM + BN) / 8 / kWaves;  // code loads per wave per stage
constexpr int kScaleBytes = (BM + BN) * 4;      // a stage's scales: one float per row of A and of B
constexpr int kStageBytes = kCodeBytes + kScaleBytes;
constexpr int kFmtE4M3 = 0;                     // matrix-core operand format
static_assert(2 * kStageBytes >= kEpiBytes, "the epilogue stages the tile through the idle stages");
static_assert(kLoads / 2 * kWaves * 8 == BM && (BM + BN) == kWaves * kWave, "load plan");

struct F8Params {
    const uint8_t* a;
    const float* sa;   // blocks x M
    const uint8_t* b;
    const float* sb;   // blocks x N, or ceil(N / 128) x blocks
    int64_t M, N, K;
    int S;             // K blocks
    void* c;
    int ct;            // 0 bf16, 1 f32
    bool whole;        // C's rows start on 16 bytes
    int splits;        // K ranges per tile (1: C directly)
    float* partial;    // splits > 1: splits x M x N
    unsigned first;    // this launch's first workgroup (of tiles times K ranges)
};

// 16 x 16 x 128 products.  Lane l supplies 32 bytes of row l % 16 of each operand,
// those of quarter l / 16 of the block, and receives column l % 16 of the second
// operand, rows 4 (l / 16) .. + 3 of the first.  The 8-bit form is the one without
// block scales (scale operands of 0), which ran at 4.9 PFLOP/s from registers at two
// waves per SIMD, where the 32 x 32 x 64 one with scales reached 4.4.  On the bf16
// cores step t takes the lane's bytes 8 t .. 8 t + 7 of both operands, so that every
// element meets its partner once.
__device__ __forceinline__ v4f mma16(v8i b, v8i a) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, v4f{}, kFmtE4M3, kFmtE4M3, 0, 0, 0, 0);
}
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
struct Wide {
    bf16x8_t v[4];
};
__device__ __forceinline__ bf16x8_t widen8(int lo, int hi) {
    const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
    const bf16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
    const bf16x2_t c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
    const bf16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
    return bf16x8_t{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}
__device__ __forceinline__ Wide widen(v8i x) {
    return Wide{{widen8(x[0], x[1]), widen8(x[2], x[3]), widen8(x[4], x[5]), widen8(x[6], x[7])}};
}
__device__ __forceinline__ v4f mma16(const Wide& b, const Wide& a) {
    v4f c = {};
#pragma unroll
    for (int t = 0; t < 4; ++t) c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b.v[t], a.v[t], c, 0, 0, 0);
    return c;
}

__device__ __forceinline__ v8i join(v4i a, v4i b) { return v8i{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}; }

// An operand as the products take it: the codes, or their bf16 values.
template <bool WIDE>
struct Operand {
    typedef v8i T;
    static __device__ __forceinline__ v8i of(v8i x) { return x; }
};
template <>
struct Operand<true> {
    typedef Wide T;
    static __device__ __forceinline__ Wide of(v8i x) { return widen(x); }
};

constexpr int kF16 = 16;                          // rows per fragment
constexpr int TA = WM / kF16, TB = WN / kF16;     // fragments of a wave's tile: 8 of A, 4 of B

// A row's eight 16-byte pieces sit in LDS at slot piece ^ (row / 2) % 8.  Lane l
// takes pieces l / 16 and 4 + l / 16 of row l % 16 of a fragment (a permutation of
// the block's elements, the same for both operands): the lanes that a ds_read_b128
// serves together (0-3, 12-15, 20-23, 24-27, and so on) then meet 16 distinct bank
// groups.  Fragments are 16 rows apart, which leaves the slots alone.
__device__ __forceinline__ int op_offset(int row, int lane, int half) {
    return row * kRowStage + ((lane / kF16 + 4 * half) ^ ((row / 2) & 7)) * 16;
}
__device__ __forceinline__ v8i read_op(const uint8_t* lo, const uint8_t* hi, int frag) {
    return join(*reinterpret_cast<const v4i*>(lo + frag * kF16 * kRowStage),
                *reinterpret_cast<const v4i*>(hi + frag * kF16 * kRowStage));
}

constexpr float kInf = __builtin_inff();

// acc + d sa sb, under the scales' product or, where that is infinite, one after the other.
__device__ __forceinline__ float scaled_sum(float d, float sa, float sb, float acc) {
    const float f = sa * sb;
    const bool over = fabsf(f) == kInf;
    return fmaf(over ? d * sb : d, over ? sa : f, acc);
}

// Whether one of a wave's sums is infinite or NaN.
template <int NA, int NB>
__device__ __forceinline__ bool not_finite(const v4f (&acc)[NB][NA]) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int j = 0; j < NA; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) m = __builtin_elementwise_maximum(m, fabsf(acc[i][j][e]));  // keeps a NaN
    return __builtin_amdgcn_ballot_w64(!(m < kInf)) != 0;
}

// A wave's sums formed again, for scales whose product passes binary32's range: operands and
// scales straight from memory, no LDS and no barrier.  FA and FB fragments of 16 rows from
// row a0 and b0 of the tile (whose first rows are m0 and n0), K blocks s_lo .. s_hi - 1.
template <bool BROW, bool WIDE, int NA, int NB>
__device__ __forceinline__ void sums_again(v4f (&acc)[NB][NA], const F8Params& p, Rsrc ra, Rsrc rb, int64_t m0, int64_t n0, int rows_a,
                           int rows_b, int a0, int b0, int s_lo, int s_hi, int lane) {
    const int K = (int)p.K, r = lane % kF16, q = lane / kF16;
    const Rsrc rst = make_rsrc(p.sb + n0 / kBlock * p.S, (int64_t)((rows_b + kBlock - 1) / kBlock) * p.S * 4);
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int j = 0; j < NA; ++j) acc[i][j] = v4f{};
    auto codes = [&](Rsrc w, int row, int s) {
        u32x4_t half[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int pos = s * kBlock + h * 64 + q * 16;
            half[h] = __builtin_amdgcn_raw_buffer_load_b128(w, pos < K ? row * K + pos : kDropped, 0, 0);
        }
        return Operand<WIDE>::of(join(__builtin_bit_cast(v4i, half[0]), __builtin_bit_cast(v4i, half[1])));
    };
    auto scale = [](Rsrc w, int at) { return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(w, at * 4, 0, 0)); };
    for (int s = s_lo; s < s_hi; ++s) {
        const Rsrc rsa = make_rsrc(p.sa + s * p.M + m0, rows_a * 4);
        const Rsrc rsb = make_rsrc(BROW ? p.sb + s * p.N + n0 : p.sb, rows_b * 4);
        for (int i = 0; i < NB; ++i) {
            const typename Operand<WIDE>::T b = codes(rb, b0 + i * kF16 + r, s);
            float sb[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int row = b0 + i * kF16 + 4 * q + e;
                sb[e] = BROW ? scale(rsb, row) : scale(rst, row / kBlock * p.S + s);
            }
#pragma unroll
            for (int j = 0; j < NA; ++j) {
                const int row = a0 + j * kF16 + r;
                const v4f d = mma16(b, codes(ra, row, s));
                const float sa = scale(rsa, row);
#pragma unroll
                for (int k = 0; k < NB; ++k)  // (registers have no run-time index)
                    if (k == i)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[k][j][e] = scaled_sum(d[e], sa, sb[e], acc[k][j][e]);
            }
        }
    }
}

// The epilogue of the FP4 kernels (store_tile) for these fragments.  It is written
// out here because theirs, cut in two to share its second half, ran 1.5% slower.
template <int EB>
struct EpiPlan {
    static constexpr int kPitch = BN * EB;                   // LDS bytes per row
    static constexpr int kRowsPass = kEpiBytes / kPitch;     // 256 (bf16) or 128 (f32)
    static constexpr int kPasses = BM / kRowsPass;
    static constexpr int kRowsInstr = 1024 / kPitch;         // rows per wave-wide 1 KB store
    static constexpr int kInstr = kRowsPass / kRowsInstr / kWaves;
    static_assert(kRowsPass % WM == 0 && kInstr * kRowsInstr * kWaves == kRowsPass, "epilogue plan");
};

// 16 bytes of a row of C whose rows start on no 16-byte boundary: one unaligned store, or
// element by element where the row ends within them.  (5451 x 2053 x 384, binary32: 28.6 us
// with every element stored by itself, 22.2 so; 1856 x 9099 x 1920, bf16: 60 and 54, where 9104
// columns take 50.)
template <int EB>
__device__ __forceinline__ void store_unit(void* c, int64_t row, int64_t col, int64_t N, u32x4_t v) {
    typedef uint32_t Unit __attribute__((ext_vector_type(4), aligned(2)));
    char* at = static_cast<char*>(c) + (row * N + col) * EB;
    if (col + 16 / EB <= N) {
        __builtin_nontemporal_store(v, reinterpret_cast<Unit*>(at));
        return;
    }
#pragma unroll
    for (int e = 0; e < 16 / EB; ++e) {
        if (col + e >= N) break;
        if (EB == 4) reinterpret_cast<uint32_t*>(at)[e] = v[e & 3];
        else reinterpret_cast<uint16_t*>(at)[e] = (uint16_t)(v[e / 2 & 3] >> (16 * (e & 1)));
    }
}

// Four columns of group `grp` of LDS row r.
template <int EB>
__device__ __forceinline__ void put_quad(uint8_t* lds, int r, int grp, float a, float b, float c, float d) {
    *reinterpret_cast<typename Quad<EB>::T*>(lds + r * EpiPlan<EB>::kPitch + (grp ^ (r & 31)) * 4 * EB) =
        Quad<EB>::pack(a, b, c, d);
}

// Stores the rows of pass h from LDS, after a barrier.  c: C's row 0 of the tile.
template <int EB>
__device__ __forceinline__ void store_pass(const uint8_t* lds, int h, void* c, Rsrc rc, int wave, int lane,
                                           int64_t rows_a, int64_t n0, int64_t N, bool whole) {
    typedef EpiPlan<EB> P;
#pragma unroll
    for (int k = 0; k < P::kInstr; ++k) {
        const int r = (wave * P::kInstr + k) * P::kRowsInstr + lane / (P::kPitch / 16);
        const int q = lane % (P::kPitch / 16);  // 16-byte unit within the row
        u32x4_t v;
        if (EB == 4) {
            v = *reinterpret_cast<const u32x4_t*>(lds + r * P::kPitch + ((q ^ (r & 31)) * 16));
        } else {
            const int grp = (2 * q) ^ (r & 31);
            v = *reinterpret_cast<const u32x4_t*>(lds + r * P::kPitch + (grp >> 1) * 16);
            if (r & 1) v = u32x4_t{v[2], v[3], v[0], v[1]};
        }
        const int64_t row = h * P::kRowsPass + r, col = n0 + q * (16 / EB);
        const bool in = row < rows_a && col < N;
        if (whole) __builtin_amdgcn_raw_buffer_store_b128(v, rc, in ? (int)(row * N * EB + col * EB) : kDropped, 0, kStoreNT);
        else if (in) store_unit<EB>(c, row, col, N, v);
    }
}

// Lane l, register e of acc[i][j]: row of A wm * WM + 16 j + l % 16, row of B
// wn * WN + 16 i + 4 (l / 16) + e.
template <int EB>
__device__ __forceinline__ void store_tile16(const v4f (&acc)[TB][TA], uint8_t* lds, void* c, Rsrc rc, int wave, int wm,
                                             int wn, int lane, int64_t rows_a, int64_t n0, int64_t N, bool whole) {
    typedef EpiPlan<EB> P;
#pragma unroll
    for (int h = 0; h < P::kPasses; ++h) {
        if (wm * WM / P::kRowsPass == h) {
#pragma unroll
            for (int j = 0; j < TA; ++j)
#pragma unroll
                for (int i = 0; i < TB; ++i)
                    put_quad<EB>(lds, wm * WM + j * kF16 + lane % kF16 - h * P::kRowsPass,
                                 (wn * WN + i * kF16) / 4 + lane / kF16, acc[i][j][0], acc[i][j][1], acc[i][j][2],
                                 acc[i][j][3]);
        }
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        if (whole) store_pass<EB>(lds, h, c, rc, wave, lane, rows_a, n0, N, true);
        else store_pass<EB>(lds, h, c, rc, wave, lane, rows_a, n0, N, false);
        if (h + 1 < P::kPasses) asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    }
}

template <bool BROW>
__global__ __launch_bounds__(kThreads) void k_gemm_fp8(F8Params p) {
    __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * kStageBytes];
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wm = wave >> 2, wn = wave & 3;  // 2 x 4 waves of 128 x 64
    const int64_t tiles_m = (p.M + BM - 1) / BM, tiles_n = (p.N + BN - 1) / BN;
    const int splits = p.splits;
    const unsigned group = p.first + blockIdx.x;
    const int split = (int)(group % splits);
    int64_t tm, tn;
    tile_of(group / splits, tiles_m, tiles_n, tm, tn);
    const int64_t m0 = tm * BM, n0 = tn * BN;
    const int64_t rows_a = p.M - m0 < BM ? p.M - m0 : BM;
    const int64_t rows_b = p.N - n0 < BN ? p.N - n0 : BN;
    // Every offset below fits 32 bits: K <= 2^22, so a window is at most 2^30 bytes.
    const int K = (int)p.K, S = p.S;
    const int per = (S + splits - 1) / splits;
    const int s_lo = split * per, s_hi = s_lo + per < S ? s_lo + per : S;
    const Rsrc ra = make_rsrc(p.a + m0 * K, rows_a * K);
    const Rsrc rb = make_rsrc(p.b + n0 * K, rows_b * K);

    // Code load q of a wave moves rows 8 d .. 8 d + 7, d = wave + 8 (q % 4), of A
    // (q < 4) or B: lane l fetches row 8 d + l / 8 into slot l % 8 of that row (row /
    // 2 = 4 d + l / 16 and d = wave mod 2, so that the piece is the same for every q).
    const int piece = (lane % 8) ^ (4 * (wave & 1) + lane / 16);
    const int lane_off = (lane / 8) * K + piece * 16;
    // Scales of a stage: waves 0-3 bring 64 rows of A each, waves 4-7 of B; B's tile
    // scales are spread to one per row.  Chosen once per wave, so that the K loop
    // has no branch: a stage's window starts sc_step floats after the one before.
    const bool sc_a = wave < 4;
    const int sc_row = (wave % 4) * kWave + lane;
    const float* sc_base = sc_a ? p.sa + m0 : BROW ? p.sb + n0 : p.sb + n0 / kBlock * S;
    const int64_t sc_step = sc_a ? p.M : BROW ? p.N : 1;
    const int sc_size = (int)(sc_a ? rows_a : BROW ? rows_b : (rows_b + kBlock - 1) / kBlock * S) * 4;
    const int sc_shrink = sc_a || BROW ? 0 : 4;  // the tile scales' window ends where it did
    const int sc_off = (sc_a || BROW ? sc_row : sc_row / kBlock * S) * 4;
    // Load L of stage s: the code loads, then the scales.  A stage past the range
    // reads zero codes (and some other stage's scales).
    auto issue = [&](int s, int L) {
        uint8_t* stage = lds + (s & 1) * kStageBytes;
        if (L < kLoads) {
            const int k0 = s * kBlock;
            const int base = k0 + piece * 16 < (s < s_hi ? K : 0) ? lane_off + k0 : kPastWindow;
            const int d = wave + kWaves * (L % (kLoads / 2));
            uint8_t* dst = stage + (L < kLoads / 2 ? 0 : BM * kRowStage) + d * 8 * kRowStage;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(L < kLoads / 2 ? ra : rb, (LdsPtr)dst, 16, base + 8 * d * K, 0, 0, 0);
        } else {
            const int at = s < s_hi ? s : s_lo;
            const Rsrc rs = make_rsrc(sc_base + at * sc_step, sc_size - at * sc_shrink);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (LdsPtr)(stage + kCodeBytes + wave * kWave * 4), 4, sc_off, 0, 0, 0);
        }
    };

    v4f acc[TB][TA];
#pragma unroll
    for (int i = 0; i < TB; ++i)
#pragma unroll
        for (int j = 0; j < TA; ++j) acc[i][j] = v4f{};

    // Groups of products: the fragments of B against fragment j of A.  While a group's
    // products run, the previous group's are scaled into the sums, the next
    // fragment of A is read and loads of the next stage go out, kEarly per group: early
    // enough to land within the stage, without a burst that fills the load queue.
    // With one scale of B for all (kCarry), the last group's products of a stage are
    // scaled in the next one, while its first operands are on their way from LDS.
    constexpr bool kCarry = !BROW;
    constexpr int kEarly = 2;
    v4f t[2][TB];
    float f_old = 0.0f, sb_old = 0.0f;
#pragma unroll
    for (int i = 0; i < TB; ++i) t[1][i] = v4f{};
    const int a_row = wm * WM + lane % kF16;  // within the tile
    const int b_row = wn * WN + lane % kF16;
    const int a_lo = op_offset(a_row, lane, 0), a_hi = op_offset(a_row, lane, 1);
    const int b_lo = BM * kRowStage + op_offset(b_row, lane, 0), b_hi = BM * kRowStage + op_offset(b_row, lane, 1);
    auto scale_in = [&](int i, int j, const v4f& d, float f, const v4f& sb) {
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = fmaf(d[e], BROW ? sb[e] * f : f, acc[i][j][e]);
    };
    if (s_lo < s_hi) {  // K = 0 has no operands to read
#pragma unroll
        for (int L = 0; L <= kLoads; ++L) issue(s_lo, L);
    }
    for (int s = s_lo; s < s_hi; ++s) {
        const uint8_t* here = lds + (s & 1) * kStageBytes;
        const float* fa = reinterpret_cast<const float*>(here + kCodeBytes) + a_row;
        const float* fb = reinterpret_cast<const float*>(here + kCodeBytes) + BM + wn * WN;
        // Stage s has landed, and no wave still reads stage s - 1.  (The compiler's own
        // wait, so that it adds none before the first operands arrive.)
        __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) lgkmcnt(0)
        asm volatile("s_barrier" ::: "memory");
        v8i a_next = read_op(here + a_lo, here + a_hi, 0);
        v8i b[TB];
        v4f sb[BROW ? TB : 1];
#pragma unroll
        for (int i = 0; i < TB; ++i) {
            __builtin_amdgcn_sched_barrier(0);  // the first products wait for as few reads as can be
            b[i] = read_op(here + b_lo, here + b_hi, i);
        }
        __builtin_amdgcn_sched_barrier(0);
        float f_next = fa[0];
        const float sb_tile = BROW ? 1.0f : fb[0];
        if (BROW) {
#pragma unroll
            for (int i = 0; i < TB; ++i) sb[BROW ? i : 0] = *reinterpret_cast<const v4f*>(fb + i * kF16 + 4 * (lane / kF16));
        }
#pragma unroll
        for (int j = 0; j < TA; ++j) {
            const v8i a = a_next;
            const float f = f_next;
            if (j + 1 < TA) {
                a_next = read_op(here + a_lo, here + a_hi, j + 1);
                f_next = fa[(j + 1) * kF16];
            }
            __builtin_amdgcn_sched_barrier(0);
            const float scale = BROW ? f_old : f_old * sb_old;
#pragma unroll
            for (int i = 0; i < TB; ++i) {
                t[j % 2][i] = mma16(b[i], a);
                if (kCarry || j > 0) scale_in(i, (j + TA - 1) % TA, t[(j + 1) % 2][i], scale, sb[BROW ? i : 0]);
                __builtin_amdgcn_sched_barrier(0);
                if (i == 0) {
#pragma unroll
                    for (int e = 0; e < kEarly; ++e)
                        if (j * kEarly + e <= kLoads) issue(s + 1, j * kEarly + e);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
            f_old = f;
            if (j == 0) sb_old = sb_tile;
        }
        if (!kCarry) {
#pragma unroll
            for (int i = 0; i < TB; ++i) scale_in(i, TA - 1, t[1][i], f_old, sb[BROW ? i : 0]);
        }
    }
    if (kCarry) {
#pragma unroll
        for (int i = 0; i < TB; ++i) scale_in(i, TA - 1, t[1][i], f_old * sb_old, v4f{});
    }
    if (__builtin_expect(not_finite(acc), 0))
        sums_again<BROW, false>(acc, p, ra, rb, m0, n0, (int)rows_a, (int)rows_b, wm * WM, wn * WN, s_lo, s_hi, lane);
    wait_all_barrier();  // LDS is reused below

    void* c = splits > 1 ? static_cast<void*>(p.partial + (int64_t)split * p.M * p.N) : p.c;
    const int ct = splits > 1 ? 1 : p.ct;
    const int eb = ct == 1 ? 4 : 2;
    void* tile = static_cast<char*>(c) + m0 * p.N * eb;
    const Rsrc rc = make_rsrc(tile, rows_a * p.N * eb);
    const bool whole = splits > 1 ? (p.N & 3) == 0 : p.whole;
    int l = lane;  // opaque: the epilogue's addresses are not kept in registers through the K loop
    asm volatile("" : "+v"(l));
    if (ct == 1) store_tile16<4>(acc, lds, tile, rc, wave, wm, wn, l, rows_a, n0, p.N, whole);
    else store_tile16<2>(acc, lds, tile, rc, wave, wm, wn, l, rows_a, n0, p.N, whole);
}

// ---------------------------------------------------------------------------
// Products with too few 256 x 256 tiles to fill the chip: the same in tiles of T x T
// (128 or 64), four waves of T / 2 x T / 2, through two LDS stages; two or four
// workgroups share a CU and cover each other's waits (a third stage, which leaves room
// for fewer, was 5% slower at T = 64 and 1.4 times as slow at T = 128).

template <int T>
struct MidPlan {
    static constexpr int kF = T / 2 / kF16;                // fragments per wave and side
    static constexpr int kCode = 2 * T * kRowStage;        // a stage's codes: T rows of A, T of B
    static constexpr int kStage = kCode + 2 * T * 4;       // and scales
    static constexpr int kCodeLoads = 2 * T / 8 / 4;       // direct loads per wave and stage
    static constexpr int kPitch = T + 4;                   // floats per row of the staged result: 16-byte
                                                           // writes of 16 rows fall in distinct banks
    static constexpr int kLds = 2 * kStage > T * kPitch * 4 ? 2 * kStage : T * kPitch * 4;
};

template <int T, bool BROW, bool WIDE>
__global__ __launch_bounds__(256, T == 128 ? 2 : 4) void k_gemm_fp8_mid(F8Params p) {
    typedef MidPlan<T> P;
    typedef Operand<WIDE> Op;
    constexpr int F = P::kF;
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wm = wave / 2, wn = wave % 2;
    const int64_t tiles_m = (p.M + T - 1) / T, tiles_n = (p.N + T - 1) / T;
    const int splits = p.splits;
    const unsigned group = p.first + blockIdx.x;
    const int split = (int)(group % splits);
    int64_t tm, tn;
    tile_of(group / splits, tiles_m, tiles_n, tm, tn);
    const int64_t m0 = tm * T, n0 = tn * T;
    const int rows_a = (int)(p.M - m0 < T ? p.M - m0 : T), rows_b = (int)(p.N - n0 < T ? p.N - n0 : T);
    const int K = (int)p.K, S = p.S;
    const int per = (S + splits - 1) / splits;
    const int s_lo = split * per, s_hi = s_lo + per < S ? s_lo + per : S;
    const Rsrc ra = make_rsrc(p.a + m0 * K, (int64_t)rows_a * K);
    const Rsrc rb = make_rsrc(p.b + n0 * K, (int64_t)rows_b * K);

    // Code load q of a wave moves rows 8 d .. 8 d + 7 of the 2 T (A's, then B's), d =
    // 4 q + wave; slots as in the tile kernel (T is a multiple of 16).
    const int piece = (lane % 8) ^ (4 * (wave & 1) + lane / 16);
    const int lane_off = (lane / 8) * K + piece * 16;
    // Scales: waves 0 and 1 bring A's, 2 and 3 B's, 64 each (T = 64: the same twice).
    const bool sc_a = wave < 2;
    const int sc_row = (wave % 2 * kWave + lane) % T;
    const float* sc_base = sc_a ? p.sa + m0 : BROW ? p.sb + n0 : p.sb + n0 / kBlock * S;
    const int64_t sc_step = sc_a ? p.M : BROW ? p.N : 1;
    const int sc_size = (sc_a ? rows_a : BROW ? rows_b : S) * 4;
    const int sc_shrink = sc_a || BROW ? 0 : 4;
    const int sc_off = sc_a || BROW ? sc_row * 4 : 0;  // a tile's 64 or 128 rows are in one block of B
    auto issue = [&](int s) {
        uint8_t* stage = lds + (s & 1) * P::kStage;
        const int k0 = s * kBlock;
        const int base = k0 + piece * 16 < (s < s_hi ? K : 0) ? lane_off + k0 : kPastWindow;
#pragma unroll
        for (int q = 0; q < P::kCodeLoads; ++q) {
            const int d = 4 * q + wave;
            const bool is_a = q < P::kCodeLoads / 2;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(is_a ? ra : rb, (LdsPtr)(stage + d * 8 * kRowStage), 16,
                                                     base + (is_a ? 8 * d : 8 * d - T) * K, 0, 0, 0);
        }
        const int at = s < s_hi ? s : s_lo;
        const Rsrc rs = make_rsrc(sc_base + at * sc_step, sc_size - at * sc_shrink);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            rs, (LdsPtr)(stage + P::kCode + ((sc_a ? 0 : T) + wave % 2 * kWave % T) * 4), 4, sc_off, 0, 0, 0);
    };

    v4f acc[F][F];
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
        for (int j = 0; j < F; ++j) acc[i][j] = v4f{};
    const int a_row = wm * (T / 2) + lane % kF16, b_row = wn * (T / 2) + lane % kF16;
    const int a_lo = op_offset(a_row, lane, 0), a_hi = op_offset(a_row, lane, 1);
    const int b_lo = T * kRowStage + op_offset(b_row, lane, 0), b_hi = T * kRowStage + op_offset(b_row, lane, 1);
    if (s_lo < s_hi) issue(s_lo);  // K = 0 has no operands to read
    for (int s = s_lo; s < s_hi; ++s) {
        const uint8_t* here = lds + (s & 1) * P::kStage;
        // Stage s has landed, and no wave still reads stage s - 1.
        __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) lgkmcnt(0)
        asm volatile("s_barrier" ::: "memory");
        issue(s + 1);
        const float* fa = reinterpret_cast<const float*>(here + P::kCode) + a_row;
        const float* fb = reinterpret_cast<const float*>(here + P::kCode) + T + wn * (T / 2);
        typename Op::T b[F];
        v4f sb[BROW ? F : 1];
#pragma unroll
        for (int i = 0; i < F; ++i) {
            b[i] = Op::of(read_op(here + b_lo, here + b_hi, i));
            if (BROW) sb[i] = *reinterpret_cast<const v4f*>(fb + i * kF16 + 4 * (lane / kF16));
        }
        const float sb_tile = BROW ? 1.0f : fb[0];
#pragma unroll
        for (int j = 0; j < F; ++j) {
            const typename Op::T a = Op::of(read_op(here + a_lo, here + a_hi, j));
            const float f = fa[j * kF16] * sb_tile;
            v4f t[F];
#pragma unroll
            for (int i = 0; i < F; ++i) t[i] = mma16(b[i], a);
#pragma unroll
            for (int i = 0; i < F; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][j][e] = fmaf(t[i][e], BROW ? sb[i][e] * f : f, acc[i][j][e]);
        }
    }
    if (__builtin_expect(not_finite(acc), 0))
        sums_again<BROW, WIDE>(acc, p, ra, rb, m0, n0, rows_a, rows_b, wm * (T / 2), wn * (T / 2), s_lo, s_hi, lane);
    wait_all_barrier();  // LDS is reused below

    // The tile as binary32 in LDS, then whole row segments to memory.
    float* st = reinterpret_cast<float*>(lds);
#pragma unroll
    for (int j = 0; j < F; ++j)
#pragma unroll
        for (int i = 0; i < F; ++i)
            *reinterpret_cast<v4f*>(st + (a_row + j * kF16) * P::kPitch + wn * (T / 2) + i * kF16 + 4 * (lane / kF16)) =
                acc[i][j];
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

// ---------------------------------------------------------------------------
// At most 16 rows of A: C is a pass over B.  A workgroup takes 16 rows of B; its
// waves take K blocks in turn, so that together they stream whole runs of each
// row, and their sums meet in LDS (added in binary64, in wave order).  Lane l holds
// bytes 16 (l / 16) .. + 15 of both halves of the block of row l % 16 of each operand,
// read straight into registers: B is used once, A comes from the caches.  (More rows
// of A take 64 x 64 tiles: 32 x 3584 x 18944 took 36 us here against 22.)
constexpr int kFewMaxM = 16;
constexpr int kFewRows = 16;
constexpr int kFewMaxWaves = 16;

template <bool BROW>
__global__ __launch_bounds__(kFewMaxWaves * kWave) void k_gemm_fp8_few(F8Params p) {
    constexpr int U = 2;  // K blocks in flight per wave (1 x 3584 x 3584: 4.9 us, 5.9 with 4)
    __shared__ __attribute__((aligned(16))) float red[kFewMaxWaves * 256];
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int waves = blockDim.x / kWave;
    const int64_t n0 = (int64_t)blockIdx.x * kFewRows;
    const int rows_b = (int)(p.N - n0 < kFewRows ? p.N - n0 : kFewRows);
    const int K = (int)p.K, M = (int)p.M, S = p.S;
    const int r = lane % 16, q = lane / 16;
    const Rsrc rb = make_rsrc(p.b + n0 * K, (int64_t)rows_b * K);
    const Rsrc ra = make_rsrc(p.a, (int64_t)M * K);
    const Rsrc rsa = make_rsrc(p.sa, (int64_t)S * M * 4);
    const float* sb_tile = p.sb + n0 / kBlock * S;

    v4f acc[1][1] = {};
    auto sums = [&](auto careful) {
        constexpr bool CAREFUL = decltype(careful)::value;
        for (int s0 = wave; s0 < S; s0 += waves * U) {
            u32x4_t b[U][2], a[U][2];
            float sa[U], sb[U][4];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int s = s0 + u * waves;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int pos = s * kBlock + h * 64 + q * 16;
                    const int off = s < S && pos < K ? r * K + pos : kDropped;
                    b[u][h] = __builtin_amdgcn_raw_buffer_load_b128(rb, off, 0, 0);
                    a[u][h] = __builtin_amdgcn_raw_buffer_load_b128(ra, off, 0, 0);
                }
                sa[u] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rsa, s < S ? (s * M + r) * 4 : kDropped, 0, 0));
                if (BROW) {
                    const Rsrc rs = make_rsrc(p.sb + (int64_t)(s < S ? s : 0) * p.N + n0, rows_b * 4);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        sb[u][e] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, (4 * q + e) * 4, 0, 0));
                } else {
                    sb[u][0] = sb_tile[s < S ? s : 0];
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const Wide bw = widen(join(__builtin_bit_cast(v4i, b[u][0]), __builtin_bit_cast(v4i, b[u][1])));
                const Wide aw = widen(join(__builtin_bit_cast(v4i, a[u][0]), __builtin_bit_cast(v4i, a[u][1])));
                const v4f d = mma16(bw, aw);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float t = sb[u][BROW ? e : 0];
                    acc[0][0][e] = CAREFUL ? scaled_sum(d[e], sa[u], t, acc[0][0][e]) : fmaf(d[e], sa[u] * t, acc[0][0][e]);
                }
            }
        }
    };
    sums(std::false_type{});
    if (__builtin_expect(not_finite(acc), 0)) {
        acc[0][0] = v4f{};
        sums(std::true_type{});
    }
    // Register e of lane l: row of A l % 16, row of B 4 (l / 16) + e.
    *reinterpret_cast<v4f*>(red + (wave * 16 + r) * 16 + 4 * q) = acc[0][0];
    __syncthreads();
    for (int e = threadIdx.x; e < 256; e += blockDim.x) {
        double sum = 0.0;
        for (int w = 0; w < waves; ++w) sum += red[w * 256 + e];
        const int m = e / 16, n = e % 16;
        if (m < M && n < rows_b) {
            const int64_t at = m * p.N + n0 + n;
            if (p.ct == 1) static_cast<float*>(p.c)[at] = (float)sum;
            else static_cast<uint16_t*>(p.c)[at] = (uint16_t)to_bf16((float)sum);
        }
    }
}

// Which tile, and how many K ranges per tile: the pair that makes the modelled time
// least.  A function of the shape and the output's type only, so that the workspace's
// size is too.
constexpr int64_t kMaxPartialBytes = (int64_t)1 << 28;

struct Choice {
    int tile;    // 256, 128 or 64
    int splits;
};

// Costs in microseconds, fitted to measured products (100 x 3584 x 3584 to 14336 x
// 4096 x 4096): a K block of one workgroup while its CU is shared (`each`, on the 8-bit
// and on the bf16 cores) and its latency when it is not (`alone`), a workgroup's start and
// epilogue, and how many share a CU.  A binary32 C takes the smaller tiles alone: on the
// bf16 cores the large one gained 4% at best (4096 x 4096 x 14336: 392 us against 407) and
// lost 10% where K is short (8192 x 8192 x 512: 105 against 95).
struct TileCost {
    int tile, per_cu;
    double alone, each, each_wide, fixed;
};
constexpr TileCost kTileCosts[] = {{256, 1, 1.5, 1.5, 0.0, 6.0}, {128, 2, 0.7, 0.53, 0.95, 4.0}, {64, 4, 0.45, 0.22, 0.30, 3.0}};
constexpr int kCus = 256;
constexpr int kRanges[] = {1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64};

Choice choose(int64_t M, int64_t N, int64_t K, bool wide) {
    const int64_t S = (K + kBlock - 1) / kBlock;
    const bool may_split = N * 4 < ((int64_t)1 << 23);
    Choice best{128, 1};
    double least = 1e300;
    for (const TileCost& c : kTileCosts) {
        if (wide && c.each_wide == 0.0) continue;
        const int64_t tiles = ((M + c.tile - 1) / c.tile) * ((N + c.tile - 1) / c.tile);
        const double each = wide ? c.each_wide : c.each;
        for (const int sp : kRanges) {
            const int64_t per = (S + sp - 1) / sp;
            if (sp > 1 && (sp > S || !may_split || tiles * sp > 4 * kCus || 4 * sp * M * N > kMaxPartialBytes)) break;
            if (sp > 1 && per * (sp - 1) >= S) continue;  // a range would be empty
            // Workgroups on the busiest CU, a full share at a time.
            const int64_t groups = (tiles * sp + kCus - 1) / kCus, full = groups / c.per_cu, rest = groups % c.per_cu;
            double t = (double)full * ((double)per * std::max(c.alone, each * c.per_cu) + c.fixed);
            if (rest) t += (double)per * std::max(c.alone, each * (double)rest) + c.fixed;
            // The partial products' trip through memory, and the launch that adds them.
            if (sp > 1) t += 3.0 + 8.0 * (double)sp * (double)M * (double)N / 8e6;
            if (t < least) least = t, best = Choice{c.tile, sp};
        }
    }
    return best;
}

template <bool BROW, bool WIDE>
void launch_tile(F8Params p, int tile, int64_t groups, hipStream_t stream) {
    for (int64_t first = 0; first < groups; first += kMaxGrid) {
        const dim3 grid((unsigned)std::min(groups - first, kMaxGrid));
        p.first = (unsigned)first;
        if (!WIDE && tile == 256)
            FP4Q_LAUNCH(k_gemm_fp8<BROW>, grid, dim3(kThreads), 0, stream, p);
        else if (tile == 128)
            FP4Q_LAUNCH((k_gemm_fp8_mid<128, BROW, WIDE>), grid, dim3(256), MidPlan<128>::kLds, stream, p);
        else
            FP4Q_LAUNCH((k_gemm_fp8_mid<64, BROW, WIDE>), grid, dim3(256), MidPlan<64>::kLds, stream, p);
    }
}

}  // namespace

size_t fp8_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K, int ct) {
    if (M <= kFewMaxM) return 0;
    const int sp = choose(M, N, K, ct == 1).splits;
    return sp > 1 ? (size_t)(4 * sp * M * N) : 0;
}

int launch_fp8_gemm(const Fp8GemmJob& j, char* msg, size_t msg_len) {
    if (j.M == 0 || j.N == 0) return 0;
    hipStream_t stream = static_cast<hipStream_t>(j.stream);
    const int S = (int)((j.K + kBlock - 1) / kBlock);
    const bool whole = j.N * (j.ct == 1 ? 4 : 2) % 16 == 0 && (uintptr_t)j.c % 16 == 0;
    F8Params p{j.a_codes, j.a_scales, j.b_codes, j.b_scales, j.M, j.N, j.K, S, j.c, j.ct, whole, 1,
               static_cast<float*>(j.ws), 0};
    if (j.M <= kFewMaxM) {
        // Enough waves to keep memory busy whatever N: 16 per workgroup while
        // there are fewer workgroups than CUs.
        const int64_t groups = (j.N + kFewRows - 1) / kFewRows;
        int waves = groups <= 256 ? kFewMaxWaves : groups <= 1024 ? 8 : 4;
        while (waves > 1 && waves >= 2 * S) waves /= 2;
        if (j.b_row) FP4Q_LAUNCH(k_gemm_fp8_few<true>, dim3((unsigned)groups), dim3(waves * kWave), 0, stream, p);
        else FP4Q_LAUNCH(k_gemm_fp8_few<false>, dim3((unsigned)groups), dim3(waves * kWave), 0, stream, p);
    } else {
        const bool wide = j.ct == 1;
        const Choice ch = choose(j.M, j.N, j.K, wide);
        p.splits = ch.splits;
        const int64_t groups = ((j.M + ch.tile - 1) / ch.tile) * ((j.N + ch.tile - 1) / ch.tile) * ch.splits;
        if (groups > INT32_MAX) {
            snprintf(msg, msg_len, "fp8 gemm: %lld x %lld x %lld needs more workgroups than one launch holds",
                     (long long)j.M, (long long)j.N, (long long)j.K);
            return (int)hipErrorInvalidConfiguration;
        }
        if (j.b_row && wide) launch_tile<true, true>(p, ch.tile, groups, stream);
        else if (j.b_row) launch_tile<true, false>(p, ch.tile, groups, stream);
        else if (wide) launch_tile<false, true>(p, ch.tile, groups, stream);
        else launch_tile<false, false>(p, ch.tile, groups, stream);
        if (p.splits > 1) launch_splitk_reduce(p.partial, p.splits, j.M * j.N, j.c, j.ct, j.stream);
    }
    const hipError_t e = hipGetLastError();
    if (e == hipSuccess) return 0;
    snprintf(msg, msg_len, "fp8 gemm kernel launch: %s", hipGetErrorString(e));
    return (int)e;
}

}  // namespace fp4q
