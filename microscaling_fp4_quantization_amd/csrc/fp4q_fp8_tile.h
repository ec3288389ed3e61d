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

// One tile of a product of E4M3 operands: where its rows, K blocks and scales are.
struct F8Tile {
    Rsrc ra, rb;            // rows of K bytes
    int rows_a, rows_b;
    int K, s_lo, s_hi;      // K blocks s_lo .. s_hi - 1 of the rows' K bytes
    const float* sa;        // the scales of A's rows in block s start at sa + s * sa_step, sa_size bytes
    int64_t sa_step;
    int sa_size;
    const float* sb;        // B's at sb + s * sb_step, sb_size bytes less sb_shrink for each s:
    int64_t sb_step;
    int sb_size, sb_shrink;
    int sb_tile;            // 0: one a row; else tile scales, sb_tile of them along K, and the
    int sb_phase;           // tile's first row is this one of its block (BROW; else 0)
    const int* rows;        // GATHER: row r of the tile is row rows[r] of A (none: zeros)
    int rows_all;           // of A

    // Row r of the tile in A, or -1.
    template <bool GATHER>
    __device__ __forceinline__ int a_row(int r) const {
        if (!GATHER) return r;
        const int at = r < rows_a ? rows[r] : -1;
        return at >= 0 && at < rows_all ? at : -1;
    }
    template <bool BROW>
    __device__ __forceinline__ int sb_at(int r) const {
        if (!BROW) return r / kBlock * sb_tile;
        return sb_tile ? (r + sb_phase) / kBlock * sb_tile : r;
    }
};

// A wave's sums formed again, for scales whose product passes binary32's range: operands and
// scales straight from memory, no LDS and no barrier.  NA and NB fragments of 16 rows from
// row a0 and b0 of the tile.
template <bool BROW, bool WIDE, bool GATHER, int NA, int NB>
__device__ __forceinline__ void sums_again(v4f (&acc)[NB][NA], const F8Tile& t, int a0, int b0, int lane) {
    const int r = lane % kF16, q = lane / kF16;
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int j = 0; j < NA; ++j) acc[i][j] = v4f{};
    auto codes = [&](Rsrc w, int row, int s) {
        u32x4_t half[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int pos = s * kBlock + h * 64 + q * 16;
            half[h] = __builtin_amdgcn_raw_buffer_load_b128(w, row >= 0 && pos < t.K ? row * t.K + pos : kDropped, 0, 0);
        }
        return Operand<WIDE>::of(join(__builtin_bit_cast(v4i, half[0]), __builtin_bit_cast(v4i, half[1])));
    };
    auto scale = [](Rsrc w, int at) { return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(w, at < 0 ? kDropped : at * 4, 0, 0)); };
    for (int s = t.s_lo; s < t.s_hi; ++s) {
        const Rsrc rsa = make_rsrc(t.sa + s * t.sa_step, t.sa_size);
        const Rsrc rsb = make_rsrc(t.sb + s * t.sb_step, t.sb_size - s * t.sb_shrink);
        for (int i = 0; i < NB; ++i) {
            const typename Operand<WIDE>::T b = codes(t.rb, b0 + i * kF16 + r, s);
            float sb[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) sb[e] = scale(rsb, t.sb_at<BROW>(b0 + i * kF16 + 4 * q + e));
#pragma unroll
            for (int j = 0; j < NA; ++j) {
                const int row = t.a_row<GATHER>(a0 + j * kF16 + r);
                const v4f d = mma16(b, codes(t.ra, row, s));
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

// A wave's loads of a 256 x 256 tile, with the lane's offset of each formed once, so that the loop
// over K moves a scalar one alone: A's rows may be anywhere (formed in the loop, their offsets took
// more registers than there are).
template <bool GATHER>
struct F8Loads {
    int at[kLoads];
    int sc_off;
    // Load L moves rows 8 d .. 8 d + 7, d = wave + 8 (L % 4), of A (L < 4) or B, as in tile_sums;
    // scales alike.
    static __device__ __forceinline__ int piece(int wave, int lane) { return (lane % 8) ^ (4 * (wave & 1) + lane / 16); }
    template <bool BROW>
    __device__ __forceinline__ void init(const F8Tile& t, int wave, int lane) {
#pragma unroll
        for (int L = 0; L < kLoads; ++L) {
            const int r = 8 * (wave + kWaves * (L % (kLoads / 2))) + lane / 8;
            const int row = L < kLoads / 2 ? t.a_row<GATHER>(r) : r;
            at[L] = row >= 0 ? row * t.K + piece(wave, lane) * 16 : kDropped;
        }
        const int r = (wave % 4) * kWave + lane, row = wave < 4 ? t.a_row<GATHER>(r) : t.sb_at<BROW>(r);
        sc_off = row >= 0 ? row * 4 : kDropped;
    }
    // Before the loads of stage s: pieces past K or s_hi are not read (zeros take their place).
    __device__ __forceinline__ void cut(const F8Tile& t, int s, int wave, int lane) {
        if (__builtin_expect((s + 1) * kBlock <= t.K && s < t.s_hi, 1)) return;
        const bool in = s < t.s_hi && s * kBlock + piece(wave, lane) * 16 < t.K;
#pragma unroll
        for (int L = 0; L < kLoads; ++L) at[L] = in ? at[L] : kDropped;
    }
    __device__ __forceinline__ void issue(const F8Tile& t, uint8_t* lds, int wave, int s, int L) const {
        uint8_t* stage = lds + (s & 1) * kStageBytes;
        if (L < kLoads) {
            const int d = wave + kWaves * (L % (kLoads / 2));
            uint8_t* dst = stage + (L < kLoads / 2 ? 0 : BM * kRowStage) + d * 8 * kRowStage;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(L < kLoads / 2 ? t.ra : t.rb, (LdsPtr)dst, 16, at[L], s * kBlock, 0, 0);
        } else {
            const bool sc_a = wave < 4;
            const int here = s < t.s_hi ? s : t.s_lo;
            const Rsrc rs = make_rsrc((sc_a ? t.sa : t.sb) + here * (sc_a ? t.sa_step : t.sb_step),
                                      (sc_a ? t.sa_size : t.sb_size) - here * (sc_a ? 0 : t.sb_shrink));
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (LdsPtr)(stage + kCodeBytes + wave * kWave * 4), 4, sc_off, 0, 0, 0);
        }
    }
    template <bool BROW>
    __device__ __forceinline__ void first_stage(const F8Tile& t, uint8_t* lds, int wave, int lane) {
        if (t.s_lo >= t.s_hi) return;  // K = 0 has no operands to read
        init<BROW>(t, wave, lane);
        cut(t, t.s_lo, wave, lane);
#pragma unroll
        for (int L = 0; L <= kLoads; ++L) issue(t, lds, wave, t.s_lo, L);
    }
};

// The sums of a 256 x 256 tile by 8 waves (2 x 4 of 128 x 64), through two LDS stages of
// kStageBytes.  BROW: B's scales differ within 64 rows; else one goes for all of a wave's.  SKIP:
// many tiles hold fewer rows of A than they have room for, and a wave that has none multiplies none
// (the waves of the other half share its SIMDs).  AHEAD: `loads` brings the stages, the first one
// already.
template <bool BROW, bool GATHER, bool SKIP, bool AHEAD>
__device__ __forceinline__ void tile_sums(v4f (&acc)[TB][TA], const F8Tile& t, uint8_t* lds, int wave, int lane, F8Loads<GATHER>& loads) {
    const int wm = wave >> 2, wn = wave & 3;
    const bool idle = wm * WM >= t.rows_a;
    // Code load q of a wave moves rows 8 d .. 8 d + 7, d = wave + 8 (q % 4), of A
    // (q < 4) or B: lane l fetches row 8 d + l / 8 into slot l % 8 of that row (row /
    // 2 = 4 d + l / 16 and d = wave mod 2, so that the piece is the same for every q).
    const int K = t.K, s_lo = t.s_lo, s_hi = t.s_hi;
    const int piece = (lane % 8) ^ (4 * (wave & 1) + lane / 16);
    const int lane_off = (lane / 8) * K + piece * 16;
    // Scales of a stage: waves 0-3 bring 64 rows of A each, waves 4-7 of B; B's tile
    // scales are spread to one per row.  Chosen once per wave, so that the K loop
    // has no branch: a stage's window starts sc_step floats after the one before.
    const bool sc_a = wave < 4;
    const int sc_row = (wave % 4) * kWave + lane;
    const float* sc_base = sc_a ? t.sa : t.sb;
    const int64_t sc_step = sc_a ? t.sa_step : t.sb_step;
    const int sc_size = sc_a ? t.sa_size : t.sb_size;
    const int sc_shrink = sc_a ? 0 : t.sb_shrink;  // tile scales' window ends where it did
    const int sc_off = (sc_a ? sc_row : t.sb_at<BROW>(sc_row)) * 4;
    // Load L of stage s: the code loads, then the scales.  A stage past the range
    // reads zero codes (and some other stage's scales).
    auto issue = [&](int s, int L) {
        if (AHEAD) return loads.issue(t, lds, wave, s, L);
        uint8_t* stage = lds + (s & 1) * kStageBytes;
        if (L < kLoads) {
            const int k0 = s * kBlock;
            const int base = k0 + piece * 16 < (s < s_hi ? K : 0) ? lane_off + k0 : kPastWindow;
            const int d = wave + kWaves * (L % (kLoads / 2));
            uint8_t* dst = stage + (L < kLoads / 2 ? 0 : BM * kRowStage) + d * 8 * kRowStage;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(L < kLoads / 2 ? t.ra : t.rb, (LdsPtr)dst, 16, base + 8 * d * K, 0, 0, 0);
        } else {
            const int at = s < s_hi ? s : s_lo;
            const Rsrc rs = make_rsrc(sc_base + at * sc_step, sc_size - at * sc_shrink);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (LdsPtr)(stage + kCodeBytes + wave * kWave * 4), 4, sc_off, 0, 0, 0);
        }
    };

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
    v4f d[2][TB];
    float f_old = 0.0f, sb_old = 0.0f;
#pragma unroll
    for (int i = 0; i < TB; ++i) d[1][i] = v4f{};
    const int a_row = wm * WM + lane % kF16;  // within the tile
    const int b_row = wn * WN + lane % kF16;
    const int a_lo = op_offset(a_row, lane, 0), a_hi = op_offset(a_row, lane, 1);
    const int b_lo = BM * kRowStage + op_offset(b_row, lane, 0), b_hi = BM * kRowStage + op_offset(b_row, lane, 1);
    auto scale_in = [&](int i, int j, const v4f& p, float f, const v4f& sb) {
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = fmaf(p[e], BROW ? sb[e] * f : f, acc[i][j][e]);
    };
    if (!AHEAD && s_lo < s_hi) {  // K = 0 has no operands to read
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
        if (AHEAD) loads.cut(t, s + 1, wave, lane);
        if (SKIP && idle) {
#pragma unroll
            for (int L = 0; L <= kLoads; ++L) issue(s + 1, L);
            continue;
        }
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
                d[j % 2][i] = mma16(b[i], a);
                if (kCarry || j > 0) scale_in(i, (j + TA - 1) % TA, d[(j + 1) % 2][i], scale, sb[BROW ? i : 0]);
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
            for (int i = 0; i < TB; ++i) scale_in(i, TA - 1, d[1][i], f_old, sb[BROW ? i : 0]);
        }
    }
    if (kCarry) {
#pragma unroll
        for (int i = 0; i < TB; ++i) scale_in(i, TA - 1, d[1][i], f_old * sb_old, v4f{});
    }
    if (__builtin_expect(not_finite(acc), 0))
        sums_again<BROW, false, GATHER>(acc, t, wm * WM, wn * WN, lane);
}

// The sums of a T x T tile by 4 waves, through two LDS stages.
template <int T, bool BROW, bool WIDE, bool GATHER, bool SKIP>
__device__ __forceinline__ void mid_sums(v4f (&acc)[MidPlan<T>::kF][MidPlan<T>::kF], const F8Tile& t, uint8_t* lds, int wave, int lane) {
    typedef MidPlan<T> P;
    typedef Operand<WIDE> Op;
    constexpr int F = P::kF;
    const int wm = wave / 2, wn = wave % 2;
    const bool idle = wm * (T / 2) >= t.rows_a;
    // Code load q of a wave moves rows 8 d .. 8 d + 7 of the 2 T (A's, then B's), d =
    // 4 q + wave; slots as in the tile kernel (T is a multiple of 16).
    const int K = t.K, s_lo = t.s_lo, s_hi = t.s_hi;
    const int piece = (lane % 8) ^ (4 * (wave & 1) + lane / 16);
    const int lane_off = (lane / 8) * K + piece * 16;
    int a_off[GATHER ? P::kCodeLoads / 2 : 1];
    if (GATHER) {
#pragma unroll
        for (int q = 0; q < P::kCodeLoads / 2; ++q) {
            const int row = t.a_row<GATHER>(8 * (4 * q + wave) + lane / 8);
            a_off[GATHER ? q : 0] = row >= 0 ? row * K + piece * 16 : -1;
        }
    }
    // Scales: waves 0 and 1 bring A's, 2 and 3 B's, 64 each (T = 64: the same twice).
    const bool sc_a = wave < 2;
    const int sc_row = (wave % 2 * kWave + lane) % T;
    const float* sc_base = sc_a ? t.sa : t.sb;
    const int64_t sc_step = sc_a ? t.sa_step : t.sb_step;
    const int sc_size = sc_a ? t.sa_size : t.sb_size;
    const int sc_shrink = sc_a ? 0 : t.sb_shrink;
    const int sc_at = sc_a ? t.a_row<GATHER>(sc_row) : BROW ? t.sb_at<BROW>(sc_row) : 0;  // else one block holds the tile's rows of B
    const int sc_off = GATHER && sc_at < 0 ? kDropped : sc_at * 4;
    auto issue = [&](int s) {
        uint8_t* stage = lds + (s & 1) * P::kStage;
        const int k0 = s * kBlock;
        const int base = k0 + piece * 16 < (s < s_hi ? K : 0) ? lane_off + k0 : kPastWindow;
#pragma unroll
        for (int q = 0; q < P::kCodeLoads; ++q) {
            const int d = 4 * q + wave;
            const bool is_a = q < P::kCodeLoads / 2;
            int off = base + (is_a ? 8 * d : 8 * d - T) * K;
            if (GATHER && is_a) off = base == kPastWindow || a_off[GATHER ? q : 0] < 0 ? kDropped : a_off[GATHER ? q : 0] + k0;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(is_a ? t.ra : t.rb, (LdsPtr)(stage + d * 8 * kRowStage), 16, off, 0, 0, 0);
        }
        const int at = s < s_hi ? s : s_lo;
        const Rsrc rs = make_rsrc(sc_base + at * sc_step, sc_size - at * sc_shrink);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            rs, (LdsPtr)(stage + P::kCode + ((sc_a ? 0 : T) + wave % 2 * kWave % T) * 4), 4, sc_off, 0, 0, 0);
    };

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
        if (SKIP && idle) continue;
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
            v4f d[F];
#pragma unroll
            for (int i = 0; i < F; ++i) d[i] = mma16(b[i], a);
#pragma unroll
            for (int i = 0; i < F; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][j][e] = fmaf(d[i][e], BROW ? sb[i][e] * f : f, acc[i][j][e]);
        }
    }
    if (__builtin_expect(not_finite(acc), 0))
        sums_again<BROW, WIDE, GATHER>(acc, t, wm * (T / 2), wn * (T / 2), lane);
}

// The tile through LDS (after a barrier) as binary32, then whole row segments to memory.  tile: C's
// row 0 of the tile, N elements a row (ct: 0 bf16, 1 f32), columns from n0 on.
template <int T>
__device__ __forceinline__ void store_mid(const v4f (&acc)[MidPlan<T>::kF][MidPlan<T>::kF], uint8_t* lds, void* tile, int ct, int rows_a,
                                          int rows_b, int64_t n0, int64_t N, bool whole, int wave, int lane) {
    typedef MidPlan<T> P;
    constexpr int F = P::kF;
    const int wn = wave % 2, a_row = wave / 2 * (T / 2) + lane % kF16;
    const int eb = ct == 1 ? 4 : 2;
    const Rsrc rc = make_rsrc(tile, (int64_t)rows_a * N * eb);
    float* st = reinterpret_cast<float*>(lds);
#pragma unroll
    for (int j = 0; j < F; ++j)
#pragma unroll
        for (int i = 0; i < F; ++i)
            *reinterpret_cast<v4f*>(st + (a_row + j * kF16) * P::kPitch + wn * (T / 2) + i * kF16 + 4 * (lane / kF16)) =
                acc[i][j];
    __syncthreads();
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
        if (whole) __builtin_amdgcn_raw_buffer_store_b128(v, rc, col < rows_b ? (int)((r * N + n0 + col) * eb) : kDropped, 0, kStoreNT);
        else if (col >= rows_b) continue;
        else if (ct == 1) store_unit<4>(tile, r, n0 + col, N, v);
        else store_unit<2>(tile, r, n0 + col, N, v);
    }
}

}  // namespace
}  // namespace fp4q
