// fp4q_fp8_tile.h -- what the products of 8-bit operands share (fp4q_fp8_gemm.hip,
// fp4q_grouped.hip, fp4q_int8.hip): matrix-core operands and their places in LDS, and the
// epilogue of a 256 x 256 tile.  Device code only; each including file gets its own copy.
#pragma once

#include "fp4q_gemm_tile.h"

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

// Tiles of T x T (128 or 64) of four waves of T / 2 x T / 2, two LDS stages.
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

}  // namespace
}  // namespace fp4q
