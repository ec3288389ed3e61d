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

#include "fp4q_fp8_tile.h"
#include "fp4q_launch.h"

namespace fp4q {
namespace {

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

template <bool BROW>
__device__ __forceinline__ F8Tile dense_tile(const F8Params& p, int64_t m0, int64_t n0, int rows_a, int rows_b, int s_lo, int s_hi) {
    F8Tile t;
    t.K = (int)p.K;
    t.ra = make_rsrc(p.a + m0 * t.K, (int64_t)rows_a * t.K);
    t.rb = make_rsrc(p.b + n0 * t.K, (int64_t)rows_b * t.K);
    t.rows_a = rows_a, t.rows_b = rows_b, t.s_lo = s_lo, t.s_hi = s_hi;
    t.sa = p.sa + m0, t.sa_step = p.M, t.sa_size = rows_a * 4;
    t.sb = BROW ? p.sb + n0 : p.sb + n0 / kBlock * p.S;
    t.sb_step = BROW ? p.N : 1;
    t.sb_size = (BROW ? rows_b : (rows_b + kBlock - 1) / kBlock * p.S) * 4;
    t.sb_shrink = BROW ? 0 : 4;
    t.sb_tile = BROW ? 0 : p.S;
    t.sb_phase = 0;
    return t;
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
    const int S = p.S;
    const int per = (S + splits - 1) / splits;
    const int s_lo = split * per, s_hi = s_lo + per < S ? s_lo + per : S;
    const F8Tile t = dense_tile<BROW>(p, m0, n0, (int)rows_a, (int)rows_b, s_lo, s_hi);
    v4f acc[TB][TA];
    F8Loads<false> none;
    tile_sums<BROW, false, false, false>(acc, t, lds, wave, lane, none);
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

template <int T, bool BROW, bool WIDE>
__global__ __launch_bounds__(256, T == 128 ? 2 : 4) void k_gemm_fp8_mid(F8Params p) {
    typedef MidPlan<T> P;
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int64_t tiles_m = (p.M + T - 1) / T, tiles_n = (p.N + T - 1) / T;
    const int splits = p.splits;
    const unsigned group = p.first + blockIdx.x;
    const int split = (int)(group % splits);
    int64_t tm, tn;
    tile_of(group / splits, tiles_m, tiles_n, tm, tn);
    const int64_t m0 = tm * T, n0 = tn * T;
    const int rows_a = (int)(p.M - m0 < T ? p.M - m0 : T), rows_b = (int)(p.N - n0 < T ? p.N - n0 : T);
    const int S = p.S;
    const int per = (S + splits - 1) / splits;
    const int s_lo = split * per, s_hi = s_lo + per < S ? s_lo + per : S;
    v4f acc[P::kF][P::kF];
    mid_sums<T, BROW, WIDE, false, false>(acc, dense_tile<BROW>(p, m0, n0, rows_a, rows_b, s_lo, s_hi), lds, wave, lane);
    wait_all_barrier();  // LDS is reused below
    void* c = splits > 1 ? static_cast<void*>(p.partial + (int64_t)split * p.M * p.N) : p.c;
    const int ct = splits > 1 ? 1 : p.ct;
    const int eb = ct == 1 ? 4 : 2;
    void* tile = static_cast<char*>(c) + m0 * p.N * eb;
    const bool whole = splits > 1 ? (p.N & 3) == 0 : p.whole;
    store_mid<T>(acc, lds, tile, ct, rows_a, rows_b, n0, p.N, whole, wave, lane);
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
