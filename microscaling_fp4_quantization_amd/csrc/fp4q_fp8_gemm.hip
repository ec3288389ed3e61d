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
// which costs a multiplication more per element.
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
//                    cache line) per stage, through two LDS stages;
//  k_gemm_fp8_few    at most 64 rows of A: one pass over B, 16 rows of B per
//                    workgroup, K blocks dealt to its waves in turn; bound by the
//                    read of B, so always on the bf16 form.
//
// All accesses go through range-checked windows: rows past M or N and K pieces
// past K read zeros (code +0), stores outside C are dropped.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <stdio.h>

#include <algorithm>

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
    int splits;        // K ranges per tile (1: C directly)
    float* partial;    // splits > 1: splits x M x N
};

// 32 x 32 x 64 products of E4M3 operands (block scales of 1).
constexpr int kOne = 0x7F7F7F7F;
__device__ __forceinline__ v16f mma32(v8i b, v8i a, v16f c) {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b, a, c, kFmtE4M3, kFmtE4M3, 0, kOne, 0, kOne);
}

// The same on the bf16 cores, and 16 x 16 x 128: step t takes the lane's bytes 8 t ..
// 8 t + 7 of both operands, so that every element meets its partner once.
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
__device__ __forceinline__ v16f mma32(const Wide& b, const Wide& a, v16f c) {
#pragma unroll
    for (int t = 0; t < 4; ++t) c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(b.v[t], a.v[t], c, 0, 0, 0);
    return c;
}
__device__ __forceinline__ v4f mma16(const Wide& b, const Wide& a, v4f c) {
#pragma unroll
    for (int t = 0; t < 4; ++t) c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b.v[t], a.v[t], c, 0, 0, 0);
    return c;
}

__device__ __forceinline__ v8i join(v4i a, v4i b) { return v8i{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}; }

// Lane l's operand of depth T (64 of the stage's 128 elements): pieces 4 T +
// 2 (l / 32) and the next of row l % 32, stored at slot (piece + row / 2) % 8.
template <int T>
__device__ __forceinline__ v8i read_op(const uint8_t* codes, int row, int lane) {
    const int p = 4 * T + 2 * (lane / kFrag), rot = row / 2;
    const v4i lo = *reinterpret_cast<const v4i*>(codes + row * kRowStage + ((p + rot) & 7) * 16);
    const v4i hi = *reinterpret_cast<const v4i*>(codes + row * kRowStage + ((p + 1 + rot) & 7) * 16);
    return join(lo, hi);
}

template <bool BROW, bool WIDE>
__global__ __launch_bounds__(kThreads) void k_gemm_fp8(F8Params p) {
    __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * kStageBytes];
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wm = wave >> 2, wn = wave & 3;  // 2 x 4 waves of 128 x 64
    const int64_t tiles_m = (p.M + BM - 1) / BM, tiles_n = (p.N + BN - 1) / BN;
    const int splits = p.splits, split = (int)(blockIdx.x % splits);
    int64_t tm, tn;
    tile_of(blockIdx.x / splits, tiles_m, tiles_n, tm, tn);
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
    // (q < 4) or B: lane l fetches row 8 d + l / 8 into slot l % 8 of that row,
    // which holds piece (l % 8 - row / 2) % 8 (the same for every q: row / 2 = 4 d +
    // l / 16 and d = wave mod 2).
    const int piece = ((lane % 8) - 4 * (wave & 1) - lane / 16) & 7;
    const int lane_off = (lane / 8) * K + piece * 16;
    auto issue = [&](uint8_t* stage, int s) {
        const int k0 = s * kBlock;
        const int base = k0 + piece * 16 < K ? lane_off + k0 : kPastWindow;
#pragma unroll
        for (int q = 0; q < kLoads; ++q) {
            const bool is_a = q < kLoads / 2;
            const int d = wave + kWaves * (q % (kLoads / 2));
            uint8_t* dst = stage + (is_a ? 0 : BM * kRowStage) + d * 8 * kRowStage;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(is_a ? ra : rb, (LdsPtr)dst, 16, base + 8 * d * K, 0, 0, 0);
        }
        // Scales: waves 0-3 bring 64 rows of A each, waves 4-7 of B; B's tile
        // scales are spread to one per row.
        const int r = (wave % 4) * kWave + lane;
        uint8_t* dst = stage + kCodeBytes + wave * kWave * 4;
        if (wave < 4) {
            const Rsrc rs = make_rsrc(p.sa + (int64_t)s * p.M + m0, rows_a * 4);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (LdsPtr)dst, 4, r * 4, 0, 0, 0);
        } else if (BROW) {
            const Rsrc rs = make_rsrc(p.sb + (int64_t)s * p.N + n0, rows_b * 4);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (LdsPtr)dst, 4, r * 4, 0, 0, 0);
        } else {
            const Rsrc rs = make_rsrc(p.sb + n0 / kBlock * S, (rows_b + kBlock - 1) / kBlock * S * 4);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (LdsPtr)dst, 4, (r / kBlock * S + s) * 4, 0, 0, 0);
        }
    };

    v16f acc[FB][FA];
#pragma unroll
    for (int i = 0; i < FB; ++i)
#pragma unroll
        for (int j = 0; j < FA; ++j) acc[i][j] = v16f{};

    const int a_row = wm * WM + lane % kFrag;  // within the tile
    const int b_row = wn * WN + lane % kFrag;
    if (s_lo < s_hi) issue(lds + (s_lo & 1) * kStageBytes, s_lo);
    for (int s = s_lo; s < s_hi; ++s) {
        const uint8_t* here = lds + (s & 1) * kStageBytes;
        // Stage s has landed, and no wave still reads stage s - 1.
        wait_all_barrier();
        if (s + 1 < s_hi) issue(lds + ((s + 1) & 1) * kStageBytes, s + 1);
        const uint8_t* ca = here;
        const uint8_t* cb = here + BM * kRowStage;
        const float* fa = reinterpret_cast<const float*>(here + kCodeBytes);
        const float* fb = fa + BM;
        if (!BROW && !WIDE) {
            const float sb = fb[wn * WN];
            v8i b[FB][2];
#pragma unroll
            for (int i = 0; i < FB; ++i) {
                b[i][0] = read_op<0>(cb, b_row + i * kFrag, lane);
                b[i][1] = read_op<1>(cb, b_row + i * kFrag, lane);
            }
#pragma unroll
            for (int j = 0; j < FA; ++j) {
                const v8i a0 = read_op<0>(ca, a_row + j * kFrag, lane);
                const v8i a1 = read_op<1>(ca, a_row + j * kFrag, lane);
                const float f = fa[a_row + j * kFrag] * sb;
                v16f t[FB];
#pragma unroll
                for (int i = 0; i < FB; ++i) t[i] = mma32(b[i][0], a0, v16f{});
#pragma unroll
                for (int i = 0; i < FB; ++i) t[i] = mma32(b[i][1], a1, t[i]);
#pragma unroll
                for (int i = 0; i < FB; ++i)
#pragma unroll
                    for (int e = 0; e < 16; ++e) acc[i][j][e] = fmaf(t[i][e], f, acc[i][j][e]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < FB; ++i) {
                const v8i b0 = read_op<0>(cb, b_row + i * kFrag, lane);
                const v8i b1 = read_op<1>(cb, b_row + i * kFrag, lane);
                Wide w0, w1;
                if (WIDE) w0 = widen(b0), w1 = widen(b1);
                // Result register e of lane l is row 8 (e / 4) + 4 (l / 32) + e % 4.
                v4f sb[4];
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    if (BROW) sb[g] = *reinterpret_cast<const v4f*>(fb + wn * WN + i * kFrag + 8 * g + 4 * (lane / kFrag));
                    else sb[g] = v4f{} + fb[wn * WN];
                }
                v8i a0 = read_op<0>(ca, a_row, lane), a1 = read_op<1>(ca, a_row, lane);
#pragma unroll
                for (int j = 0; j < FA; ++j) {
                    const float f = fa[a_row + j * kFrag];
                    v16f t;
                    if (WIDE) {
                        t = mma32(w0, widen(a0), v16f{});
                        t = mma32(w1, widen(a1), t);
                    } else {
                        t = mma32(b0, a0, v16f{});
                        t = mma32(b1, a1, t);
                    }
                    if (j + 1 < FA) {
                        a0 = read_op<0>(ca, a_row + (j + 1) * kFrag, lane);
                        a1 = read_op<1>(ca, a_row + (j + 1) * kFrag, lane);
                    }
                    __builtin_amdgcn_sched_barrier(0);  // no more of A at once than the registers hold
                    if (BROW) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) acc[i][j][e] = fmaf(t[e] * sb[e / 4][e % 4], f, acc[i][j][e]);
                    } else {
                        const float g = f * sb[0][0];
#pragma unroll
                        for (int e = 0; e < 16; ++e) acc[i][j][e] = fmaf(t[e], g, acc[i][j][e]);
                    }
                }
            }
        }
    }
    wait_all_barrier();  // LDS is reused below

    void* c = splits > 1 ? static_cast<void*>(p.partial + (int64_t)split * p.M * p.N) : p.c;
    const int ct = splits > 1 ? 1 : p.ct;
    const int eb = ct == 1 ? 4 : 2;
    const Rsrc rc = make_rsrc(static_cast<char*>(c) + m0 * p.N * eb, rows_a * p.N * eb);
    if (((p.N * eb) & 15) != 0) store_direct(acc, rc, ct, wm, wn, lane, rows_a, n0, p.N);
    else if (ct == 1) store_tile<4>(acc, lds, rc, wave, wm, wn, lane, rows_a, n0, p.N);
    else store_tile<2>(acc, lds, rc, wave, wm, wn, lane, rows_a, n0, p.N);
}

// ---------------------------------------------------------------------------
// At most 64 rows of A: C is a pass over B.  A workgroup takes 16 rows of B; its
// waves take K blocks in turn, so that together they stream whole runs of each
// row, and their sums meet in LDS (added in binary64, in wave order).  Lane l holds
// row l % 16 and elements 32 (l / 16) .. + 31 of the block of each operand, both
// read straight into registers: B is used once, A comes from the caches.
constexpr int kFewMaxM = 64;
constexpr int kFewRows = 16;
constexpr int kFewMaxWaves = 16;

template <int MT, bool BROW>
__global__ __launch_bounds__(kFewMaxWaves * kWave) void k_gemm_fp8_few(F8Params p) {
    constexpr int U = MT == 1 ? 4 : 2;  // K blocks in flight per wave
    extern __shared__ __attribute__((aligned(16))) float red[];  // waves x MT x 16 x 16
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

    v4f acc[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[t] = v4f{};
    for (int s0 = wave; s0 < S; s0 += waves * U) {
        v4i b[U][2], a[U][MT][2];
        float sa[U][MT], sb[U][4];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int s = s0 + u * waves;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int pos = s * kBlock + q * 32 + h * 16;
                const bool in = s < S && pos < K;
                b[u][h] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rb, in ? r * K + pos : kDropped, 0, 0));
#pragma unroll
                for (int t = 0; t < MT; ++t)
                    a[u][t][h] = __builtin_bit_cast(
                        v4i, __builtin_amdgcn_raw_buffer_load_b128(ra, in ? (t * 16 + r) * K + pos : kDropped, 0, 0));
            }
#pragma unroll
            for (int t = 0; t < MT; ++t)
                sa[u][t] = __builtin_bit_cast(
                    float, __builtin_amdgcn_raw_buffer_load_b32(rsa, s < S ? (s * M + t * 16 + r) * 4 : kDropped, 0, 0));
            if (BROW) {
                const Rsrc rs = make_rsrc(p.sb + (int64_t)(s < S ? s : 0) * p.N + n0, rows_b * 4);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    sb[u][e] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rs, (4 * q + e) * 4, 0, 0));
            } else {
                sb[u][0] = sb_tile[s < S ? s : 0];
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const Wide bw = widen(join(b[u][0], b[u][1]));
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                const v4f d = mma16(bw, widen(join(a[u][t][0], a[u][t][1])), v4f{});
                const float f = BROW ? sa[u][t] : sa[u][t] * sb[u][0];
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[t][e] = fmaf(BROW ? d[e] * sb[u][e] : d[e], f, acc[t][e]);
            }
        }
    }
    // Register e of lane l: row of A 16 t + l % 16, row of B 4 (l / 16) + e.
#pragma unroll
    for (int t = 0; t < MT; ++t)
        *reinterpret_cast<v4f*>(red + ((wave * MT + t) * 16 + r) * 16 + 4 * q) = acc[t];
    __syncthreads();
    for (int e = threadIdx.x; e < MT * 256; e += blockDim.x) {
        double sum = 0.0;
        for (int w = 0; w < waves; ++w) sum += red[w * MT * 256 + e];
        const int m = e / 16, n = e % 16;
        if (m < M && n < rows_b) {
            const int64_t at = m * p.N + n0 + n;
            if (p.ct == 1) static_cast<float*>(p.c)[at] = (float)sum;
            else static_cast<uint16_t*>(p.c)[at] = (uint16_t)to_bf16((float)sum);
        }
    }
}

// K ranges per tile: as for the FP4 products, the count that makes the modelled
// time least (rounds of workgroups x stages, plus the partial products' trip
// through memory), in units of a stage.  A function of the shape only.
constexpr int kChipGroups = 256;
constexpr double kStageTraffic = 5e6;  // bytes of memory traffic in one stage's time
constexpr int64_t kMaxPartialBytes = (int64_t)1 << 28;

int splits_for(int64_t M, int64_t N, int64_t K) {
    const int64_t S = (K + kBlock - 1) / kBlock;
    const int64_t tiles = ((M + BM - 1) / BM) * ((N + BN - 1) / BN);
    if (S < 2 || tiles >= 2 * kChipGroups || N * 4 >= ((int64_t)1 << 23)) return 1;
    auto cost = [&](int64_t sp) {
        const double rounds = (double)((tiles * sp + kChipGroups - 1) / kChipGroups);
        const double run = rounds * (double)((S + sp - 1) / sp + 3);
        return sp == 1 ? run : run + 4.0 + 8.0 * (double)sp * (double)M * (double)N / kStageTraffic;
    };
    int64_t best = 1;
    for (int64_t sp = 2; sp <= std::min<int64_t>(S, 64); ++sp) {
        if (4 * sp * M * N > kMaxPartialBytes) break;
        if ((S + sp - 1) / sp * (sp - 1) >= S) continue;  // a range would be empty
        if (cost(sp) < cost(best)) best = sp;
    }
    return (int)best;
}

template <int MT, bool BROW>
void launch_few(const F8Params& p, int waves, hipStream_t stream) {
    const unsigned grid = (unsigned)((p.N + kFewRows - 1) / kFewRows);
    FP4Q_LAUNCH((k_gemm_fp8_few<MT, BROW>), dim3(grid), dim3(waves * kWave), waves * MT * 256 * 4, stream, p);
}

}  // namespace

size_t fp8_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    if (M <= kFewMaxM) return 0;
    const int sp = splits_for(M, N, K);
    return sp > 1 ? (size_t)(4 * sp * M * N) : 0;
}

int launch_fp8_gemm(const Fp8GemmJob& j, char* msg, size_t msg_len) {
    if (j.M == 0 || j.N == 0) return 0;
    hipStream_t stream = static_cast<hipStream_t>(j.stream);
    const int S = (int)((j.K + kBlock - 1) / kBlock);
    F8Params p{j.a_codes, j.a_scales, j.b_codes, j.b_scales, j.M, j.N, j.K, S, j.c, j.ct, 1,
               static_cast<float*>(j.ws)};
    if (j.M <= kFewMaxM) {
        // Enough waves to keep memory busy whatever N: 16 per workgroup while
        // there are fewer workgroups than CUs.
        const int64_t groups = (j.N + kFewRows - 1) / kFewRows;
        int waves = groups <= 256 ? 16 : groups <= 1024 ? 8 : 4;
        while (waves > 1 && waves >= 2 * S) waves /= 2;
        const int mt = j.M <= 16 ? 1 : j.M <= 32 ? 2 : 4;
        if (j.b_row) {
            if (mt == 1) launch_few<1, true>(p, waves, stream);
            else if (mt == 2) launch_few<2, true>(p, waves, stream);
            else launch_few<4, true>(p, waves, stream);
        } else {
            if (mt == 1) launch_few<1, false>(p, waves, stream);
            else if (mt == 2) launch_few<2, false>(p, waves, stream);
            else launch_few<4, false>(p, waves, stream);
        }
    } else {
        const int64_t tiles = ((j.M + BM - 1) / BM) * ((j.N + BN - 1) / BN);
        p.splits = splits_for(j.M, j.N, j.K);
        if (tiles * p.splits > INT32_MAX) {
            snprintf(msg, msg_len, "fp8 gemm: %lld x %lld x %lld needs more workgroups than one launch holds",
                     (long long)j.M, (long long)j.N, (long long)j.K);
            return (int)hipErrorInvalidConfiguration;
        }
        const dim3 grid((unsigned)(tiles * p.splits));
        const bool wide = j.ct == 1;
        if (j.b_row && wide) FP4Q_LAUNCH((k_gemm_fp8<true, true>), grid, dim3(kThreads), 0, stream, p);
        else if (j.b_row) FP4Q_LAUNCH((k_gemm_fp8<true, false>), grid, dim3(kThreads), 0, stream, p);
        else if (wide) FP4Q_LAUNCH((k_gemm_fp8<false, true>), grid, dim3(kThreads), 0, stream, p);
        else FP4Q_LAUNCH((k_gemm_fp8<false, false>), grid, dim3(kThreads), 0, stream, p);
        if (p.splits > 1) launch_splitk_reduce(p.partial, p.splits, j.M * j.N, j.c, j.ct, j.stream);
    }
    const hipError_t e = hipGetLastError();
    if (e == hipSuccess) return 0;
    snprintf(msg, msg_len, "fp8 gemm kernel launch: %s", hipGetErrorString(e));
    return (int)e;
}

}  // namespace fp4q
