// fp4q_grouped.hip -- products of E4M3 operands grouped by expert, with group sizes that the
// device alone knows (fp8_grouped_gemm_b128, fp8_grouped_linear), and the sort of a batch's
// slots by expert that makes the groups (expert_order).
//
//   C[i] = A[tokens[i]] W_e^T for the rows i of group e, offsets[e] <= i < offsets[e + 1]
//   dW_e = dY_e^T X_e, the rows of group e being the contraction
//
// The sums of a tile are fp8_gemm_b128's (fp4q_fp8_tile.h); what is here is where a tile's rows
// are.  A launch has workgroups for the most tiles that any sizes of its groups give (each group
// that holds a row ends inside at most one tile); a workgroup counts the tiles that there are,
// takes its own in the same order over the XCDs as the dense product, and finds its group.  Rows
// of A are gathered as they are read: a token's codes are stored once, however many experts it has.
//
// What bounds them: few rows, memory (8 rows on 8 experts of 14336 x 4096: 60 to 71 us); many rows,
// what bounds the dense product, and the tiles in which a group ends (65536 rows on 64 experts of
// 2048 x 4096, bf16 C: 594 to 642 us gathered; the dense product of that size 488 to 508; a binary32 C,
// in tiles of 128 on the bf16 cores, 1058 to 1207).
//
// A bf16 C's sums of 128 products are those of the 8-bit cores, which hold about 16 bits, twice as fast
// as the bf16 ones: one element in 60 to 90 is another bf16 number than with sums in binary32, next to it but
// where terms cancel, and the error against 64 bits is the same to three digits.  The blocks' sums are
// added in binary32.  A binary32 C, and the pass over the weights, take the bf16 cores.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <stdio.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "fp4q_fp8_tile.h"
#include "fp4q_groups.h"
#include "fp4q_launch.h"

namespace fp4q {
namespace {

struct GroupedParams {
    const uint8_t* a;
    const float* sa;     // blocks x a_rows
    int a_rows;
    const uint8_t* b;    // (experts x N) x K
    const float* sb;
    int sb_rows;         // rows per expert as its tile scales count them: N, or N rounded up to 128
    const int* tokens;
    Groups groups;
    int N, K;
    int S;               // K blocks
    char* c;
    int ct;              // 0 bf16, 1 f32
    bool whole;          // C's rows start on 16 bytes
    unsigned first;      // this launch's first workgroup
};

// Which of tiles_m by tiles_n tiles is the `idx`-th of an XCD's share (tile_of's order, for fewer
// than 2^31), where the share has so many.
__device__ __forceinline__ unsigned share_of(unsigned tiles, unsigned xcd) { return tiles / 8 + (xcd < tiles % 8 ? 1 : 0); }
__device__ __forceinline__ void tile_at(unsigned xcd, unsigned idx, unsigned tiles_m, unsigned tiles_n, int& tm, int& tn) {
    const unsigned T = tiles_m * tiles_n, t = xcd * (T / 8) + min(xcd, T % 8) + idx;
    const unsigned span = kGroupM * tiles_n, band = t / span, in = t - band * span, first = band * kGroupM;
    const unsigned gm = min(tiles_m - first, (unsigned)kGroupM), n = in / gm;
    tm = __builtin_amdgcn_readfirstlane(first + in - n * gm);
    tn = __builtin_amdgcn_readfirstlane(n);
}

// The tile of a workgroup: `side` rows of one group and as many of its expert's.  False: none.
template <bool GATHER>
__device__ __forceinline__ bool grouped_tile(const GroupedParams& p, int side, F8Tile& t, int& row0, int& n0) {
    const unsigned tiles_m = group_tiles(p.groups, side), tiles_n = (p.N + side - 1) / side, group = p.first + blockIdx.x;
    if (group / 8 >= share_of(tiles_m * tiles_n, group % 8)) return false;
    int tm, tn;
    tile_at(group % 8, group / 8, tiles_m, tiles_n, tm, tn);
    const GroupTile g = group_tile(p.groups, side, tm);
    if (g.group < 0) return false;
    const bool rest = g.group >= p.groups.count;  // rows of no group: no products
    const int e = rest ? 0 : g.group;
    row0 = g.row;
    n0 = tn * side;
    t.K = p.K;
    t.rows_a = min(side, g.end - g.row);
    t.rows_b = min(side, p.N - n0);
    t.s_lo = 0;
    t.s_hi = rest ? 0 : p.S;
    t.rows = GATHER ? p.tokens + row0 : nullptr;
    t.rows_all = p.a_rows;
    t.ra = GATHER ? make_rsrc(p.a, (int64_t)p.a_rows * p.K) : make_rsrc(p.a + (int64_t)row0 * p.K, (int64_t)t.rows_a * p.K);
    t.rb = make_rsrc(p.b + ((int64_t)e * p.N + n0) * p.K, (int64_t)t.rows_b * p.K);
    t.sa = GATHER ? p.sa : p.sa + row0;
    t.sa_step = p.a_rows;
    t.sa_size = (GATHER ? p.a_rows : t.rows_a) * 4;
    const int64_t at = (int64_t)e * p.sb_rows + n0;
    t.sb_phase = (int)(at % kBlock);
    t.sb = p.sb + at / kBlock * p.S;
    t.sb_step = 1;
    t.sb_size = (t.sb_phase + t.rows_b + kBlock - 1) / kBlock * p.S * 4;
    t.sb_shrink = 4;
    t.sb_tile = p.S;
    return true;
}

// BROW: an expert's rows do not start on a block of tile scales.
template <bool BROW, bool GATHER>
__global__ __launch_bounds__(kThreads) void k_grouped(GroupedParams p) {
    __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * kStageBytes];
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    F8Tile t;
    int row0, n0;
    if (!grouped_tile<GATHER>(p, BM, t, row0, n0)) return;
    F8Loads<GATHER> loads;
    loads.template first_stage<BROW>(t, lds, wave, lane);
    v4f acc[TB][TA];
    tile_sums<BROW, GATHER, true, true>(acc, t, lds, wave, lane, loads);
    wait_all_barrier();  // LDS is reused below
    char* c = p.c + (int64_t)row0 * p.N * 2;  // (a binary32 C takes the smaller tiles)
    const Rsrc rc = make_rsrc(c, (int64_t)t.rows_a * p.N * 2);
    int l = lane;  // opaque: the epilogue's addresses are not kept in registers through the K loop
    asm volatile("" : "+v"(l));
    store_tile16<2>(acc, lds, c, rc, wave, wave >> 2, wave & 3, l, t.rows_a, n0, p.N, p.whole);
}

template <int T, bool BROW, bool WIDE, bool GATHER>
__global__ __launch_bounds__(256, T == 128 ? 2 : 4) void k_grouped_mid(GroupedParams p) {
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    F8Tile t;
    int row0, n0;
    if (!grouped_tile<GATHER>(p, T, t, row0, n0)) return;
    v4f acc[MidPlan<T>::kF][MidPlan<T>::kF];
    mid_sums<T, BROW, WIDE, GATHER, true>(acc, t, lds, wave, lane);
    wait_all_barrier();  // LDS is reused below
    store_mid<T>(acc, lds, p.c + (int64_t)row0 * p.N * (p.ct == 1 ? 4 : 2), p.ct, t.rows_a, t.rows_b, n0, p.N, p.whole, wave, lane);
}

// Few rows per group: a pass over the matrices of the experts that have any.  A workgroup takes 16
// rows of one expert's matrix against its group, 16 rows of that at a time, its waves K blocks in
// turn, the next block on its way; bound by the read of B, so always on the bf16 form.  Half a
// wave's registers go to blocks on their way, so that eight waves share a SIMD.
constexpr int kFewRows = 16;
constexpr int kFewMaxWaves = 8;

template <bool BROW, bool GATHER>
__global__ __launch_bounds__(kFewMaxWaves * kWave) void k_grouped_few(GroupedParams p) {
    constexpr int SB = BROW ? 4 : 1;  // scales of a lane's four rows of B
    __shared__ __attribute__((aligned(16))) float red[kFewMaxWaves * 256];
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int waves = blockDim.x / kWave;
    const unsigned tiles_n = (p.N + kFewRows - 1) / kFewRows, group = p.first + blockIdx.x;
    const GroupTile g = nonempty_group(p.groups, (int)(group / tiles_n));
    if (g.group < 0) return;
    const bool rest = g.group >= p.groups.count;
    const int e = rest ? 0 : g.group, n0 = (int)(group % tiles_n) * kFewRows;
    const int rows_b = min(kFewRows, p.N - n0);
    const int K = p.K, S = rest ? 0 : p.S;
    const int r = lane % 16, q = lane / 16;
    const Rsrc rb = make_rsrc(p.b + ((int64_t)e * p.N + n0) * K, (int64_t)rows_b * K);
    const int64_t at = (int64_t)e * p.sb_rows + n0;
    const float* sb = p.sb + at / kBlock * p.S;  // of the first row's block
    int sb_at[SB];
#pragma unroll
    for (int k = 0; k < SB; ++k) sb_at[k] = BROW ? (int)((at % kBlock + min(4 * q + k, rows_b - 1)) / kBlock) * p.S : 0;

    struct Block { u32x4_t a[2], b[2]; float sa, sb[SB]; };
    auto place = [&](int s, int h) {
        const int pos = s * kBlock + h * 64 + q * 16;
        return s < S && pos < K ? pos : -1;
    };
    auto load_b = [&](Block& t, int s) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int pos = place(s, h);
            t.b[h] = __builtin_amdgcn_raw_buffer_load_b128(rb, pos >= 0 ? r * K + pos : kDropped, 0, 0);
        }
#pragma unroll
        for (int k = 0; k < SB; ++k) t.sb[k] = sb[sb_at[k] + (s < S ? s : 0)];
    };
    Block now, next;
    if (S > 0) load_b(now, wave);  // on its way while the rows of A are found
    for (int row0 = g.row; row0 < g.end; row0 += 16) {
        const int m = row0 + r;
        const int token = m >= g.end ? -1 : GATHER ? p.tokens[m] : m - row0;
        const bool there = token >= 0 && token < p.a_rows;
        const Rsrc ra = GATHER ? make_rsrc(p.a, (int64_t)p.a_rows * K) : make_rsrc(p.a + (int64_t)row0 * K, (int64_t)min(16, g.end - row0) * K);
        const float* sa = GATHER ? p.sa : p.sa + row0;
        const int sa_size = (GATHER ? p.a_rows : min(16, g.end - row0)) * 4;
        auto load_a = [&](Block& t, int s) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int pos = place(s, h);
                t.a[h] = __builtin_amdgcn_raw_buffer_load_b128(ra, there && pos >= 0 ? token * K + pos : kDropped, 0, 0);
            }
            const Rsrc rs = make_rsrc(sa + (int64_t)(s < S ? s : 0) * p.a_rows, sa_size);
            t.sa = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, there && s < S ? token * 4 : kDropped, 0, 0));
        };
        v4f acc[1][1] = {};
        auto sums = [&](auto careful) {
            constexpr bool CAREFUL = decltype(careful)::value;
            for (int s = wave; s < S; s += waves) {
                load_b(next, s + waves);
                load_a(next, s + waves);
                const Wide bw = widen(join(__builtin_bit_cast(v4i, now.b[0]), __builtin_bit_cast(v4i, now.b[1])));
                const Wide aw = widen(join(__builtin_bit_cast(v4i, now.a[0]), __builtin_bit_cast(v4i, now.a[1])));
                const v4f d = mma16(bw, aw);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float t = now.sb[BROW ? k : 0];
                    acc[0][0][k] = CAREFUL ? scaled_sum(d[k], now.sa, t, acc[0][0][k]) : fmaf(d[k], now.sa * t, acc[0][0][k]);
                }
                now = next;
            }
        };
        if (S > 0) {
            if (row0 != g.row) load_b(now, wave);
            load_a(now, wave);
        }
        sums(std::false_type{});
        if (__builtin_expect(not_finite(acc), 0)) {
            acc[0][0] = v4f{};
            load_b(now, wave);
            load_a(now, wave);
            sums(std::true_type{});
        }
        // Register k of lane l: row of A l % 16, row of B 4 (l / 16) + k.
        *reinterpret_cast<v4f*>(red + (wave * 16 + r) * 16 + 4 * q) = acc[0][0];
        __syncthreads();
        for (int i = threadIdx.x; i < 256; i += blockDim.x) {
            double sum = 0.0;
            for (int w = 0; w < waves; ++w) sum += red[w * 256 + i];
            const int mm = row0 + i / 16, n = i % 16;
            if (mm < g.end && n < rows_b) {
                const int64_t to = (int64_t)mm * p.N + n0 + n;
                if (p.ct == 1) reinterpret_cast<float*>(p.c)[to] = (float)sum;
                else reinterpret_cast<uint16_t*>(p.c)[to] = (uint16_t)to_bf16((float)sum);
            }
        }
        __syncthreads();  // `red` is read before the next rows' sums take its place
    }
}

// dW: M x N per expert, the group's blocks of 128 (transposed, zeros past its rows) the contraction.
struct OuterParams {
    const uint8_t* a;    // M x pitch
    const float* sa;     // blocks x M
    const uint8_t* b;    // N x pitch
    const float* sb;     // blocks x N
    Groups groups;
    int M, N, pitch;
    char* c;             // experts x M x N
    int ct;
    bool whole;
    unsigned first;
};

// Each XCD takes a share of every expert's tiles (a run of tile_at's order within one), so that it
// has its share of the large groups; up to 64 experts in order of their size, the largest first,
// so that none of those starts when the others are done.  (16 experts of 4096 x 2048 and 16384 rows
// in all, bf16: 199 to 236 us; 390 with the experts one after the other in tile_at's runs.)
__device__ __forceinline__ bool outer_tile(const OuterParams& p, int side, unsigned group, F8Tile& t, int& m0, int& n0, int& e) {
    const unsigned tiles_m = (p.M + side - 1) / side, tiles_n = (p.N + side - 1) / side;
    const unsigned share = (tiles_m * tiles_n + 7) / 8;
    if (group / 8 / share >= (unsigned)p.groups.count) return false;
    int tm, tn;
    if (group / 8 % share >= share_of(tiles_m * tiles_n, group % 8)) return false;
    tile_at(group % 8, group / 8 % share, tiles_m, tiles_n, tm, tn);
    const int lane = threadIdx.x % kWave;
    e = (int)(group / 8 / share);
    if (p.groups.count <= kWave) {
        int lo, hi, rank = 0;
        p.groups.range(lane, lo, hi);
        const int mine = hi - lo;
        for (int o = 0; o < p.groups.count; ++o) {
            const int other = __builtin_amdgcn_readlane(mine, o);
            rank += other > mine || (other == mine && o < lane) ? 1 : 0;
        }
        e = __builtin_ctzll(__builtin_amdgcn_ballot_w64(lane < p.groups.count && rank == e));
    }
    m0 = tm * side;
    n0 = tn * side;
    // Blocks of the groups before e, and its own.
    int before = 0, mine = 0;
    for (int c = 0; c <= e; c += kWave) {
        int lo, hi;
        p.groups.range(c + lane, lo, hi);
        const int blocks = c + lane <= e ? (hi - lo + kBlock - 1) / kBlock : 0;
        before += __builtin_amdgcn_readlane(wave_sums(blocks), 63);
        if (e - c < kWave) mine = __builtin_amdgcn_readlane(blocks, e - c);
    }
    t.K = p.pitch;
    t.s_lo = min(before - mine, p.pitch / kBlock);
    t.s_hi = min(before, p.pitch / kBlock);
    t.rows_a = min(side, p.M - m0);
    t.rows_b = min(side, p.N - n0);
    t.ra = make_rsrc(p.a + (int64_t)m0 * p.pitch, (int64_t)t.rows_a * p.pitch);
    t.rb = make_rsrc(p.b + (int64_t)n0 * p.pitch, (int64_t)t.rows_b * p.pitch);
    t.sa = p.sa + m0, t.sa_step = p.M, t.sa_size = t.rows_a * 4;
    t.sb = p.sb + n0, t.sb_step = p.N, t.sb_size = t.rows_b * 4, t.sb_shrink = 0;
    t.sb_tile = 0, t.sb_phase = 0;
    return true;
}

__global__ __launch_bounds__(kThreads) void k_grouped_outer(OuterParams p) {
    __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * kStageBytes];
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    F8Tile t;
    int m0, n0, e;
    if (!outer_tile(p, BM, p.first + blockIdx.x, t, m0, n0, e)) return;
    F8Loads<false> loads;
    loads.template first_stage<true>(t, lds, wave, lane);
    v4f acc[TB][TA];
    tile_sums<true, false, false, true>(acc, t, lds, wave, lane, loads);
    wait_all_barrier();  // LDS is reused below
    char* c = p.c + ((int64_t)e * p.M + m0) * p.N * 2;  // (a binary32 C takes the smaller tiles)
    const Rsrc rc = make_rsrc(c, (int64_t)t.rows_a * p.N * 2);
    int l = lane;
    asm volatile("" : "+v"(l));
    store_tile16<2>(acc, lds, c, rc, wave, wave >> 2, wave & 3, l, t.rows_a, n0, p.N, p.whole);
}

template <int T, bool WIDE>
__global__ __launch_bounds__(256, T == 128 ? 2 : 4) void k_grouped_outer_mid(OuterParams p) {
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    F8Tile t;
    int m0, n0, e;
    if (!outer_tile(p, T, p.first + blockIdx.x, t, m0, n0, e)) return;
    v4f acc[MidPlan<T>::kF][MidPlan<T>::kF];
    mid_sums<T, true, WIDE, false, false>(acc, t, lds, wave, lane);
    wait_all_barrier();  // LDS is reused below
    store_mid<T>(acc, lds, p.c + ((int64_t)e * p.M + m0) * p.N * (p.ct == 1 ? 4 : 2), p.ct, t.rows_a, t.rows_b, n0, p.N, p.whole, wave, lane);
}

// Which tile: the one whose modelled time is least, in microseconds, for `tiles(side)` of them with
// `blocks` K blocks each (the numbers of the dense product: a K block of one workgroup while its
// CU is shared, on the 8-bit and on the bf16 cores, and its latency when it is not; a workgroup's
// start and end; how many share a CU).  The read of B is not in it: where that is what bounds a
// product, it takes longer (512 rows on 64 experts of 2048 x 4096: 123 to 127 us in tiles of 64, 62 here),
// and the tiles that can be chosen then take about the same (of 128: 126 to 130).
struct TileCost {
    int tile, per_cu;
    double alone, each, each_wide, fixed;
};
constexpr TileCost kTileCosts[] = {{256, 1, 1.5, 1.5, 0.0, 6.0}, {128, 2, 0.7, 0.53, 0.95, 4.0}, {64, 4, 0.45, 0.22, 0.30, 3.0}};
constexpr int kCus = 256;

template <class Tiles>
int choose(bool wide, double blocks, Tiles tiles) {
    int best = 128;
    double least = 1e300;
    for (const TileCost& c : kTileCosts) {
        if (wide && c.each_wide == 0.0) continue;
        const double each = wide ? c.each_wide : c.each, groups = tiles(c.tile) / kCus;
        const double full = std::floor(groups / c.per_cu), rest = groups - full * c.per_cu;
        double t = full * (blocks * std::max(c.alone, each * c.per_cu) + c.fixed);
        if (rest > 0) t += blocks * std::max(c.alone, each * rest) + c.fixed;
        if (t < least) least = t, best = c.tile;
    }
    return best;
}

int status(const char* what, char* msg, size_t msg_len) {
    const hipError_t e = hipGetLastError();
    if (e == hipSuccess) return 0;
    snprintf(msg, msg_len, "%s kernel launch: %s", what, hipGetErrorString(e));
    return (int)e;
}

int too_many(const char* what, char* msg, size_t msg_len) {
    snprintf(msg, msg_len, "%s: more workgroups than 2^31", what);
    return (int)hipErrorInvalidConfiguration;
}

template <bool BROW, bool GATHER>
void launch_tiles(GroupedParams p, int tile, int64_t groups, hipStream_t stream) {
    for (int64_t first = 0; first < groups; first += kMaxGrid) {
        const dim3 grid((unsigned)std::min(groups - first, kMaxGrid));
        p.first = (unsigned)first;
        if (tile == 256) FP4Q_LAUNCH((k_grouped<BROW, GATHER>), grid, dim3(kThreads), 0, stream, p);
        else if (tile == 128 && p.ct == 1) FP4Q_LAUNCH((k_grouped_mid<128, BROW, true, GATHER>), grid, dim3(256), MidPlan<128>::kLds, stream, p);
        else if (tile == 128) FP4Q_LAUNCH((k_grouped_mid<128, BROW, false, GATHER>), grid, dim3(256), MidPlan<128>::kLds, stream, p);
        else if (p.ct == 1) FP4Q_LAUNCH((k_grouped_mid<64, BROW, true, GATHER>), grid, dim3(256), MidPlan<64>::kLds, stream, p);
        else FP4Q_LAUNCH((k_grouped_mid<64, BROW, false, GATHER>), grid, dim3(256), MidPlan<64>::kLds, stream, p);
    }
}

}  // namespace

int launch_grouped_gemm(const GroupedGemmJob& j, char* msg, size_t msg_len) {
    const char* what = "grouped gemm";
    if (j.rows == 0 || j.N == 0) return 0;
    hipStream_t stream = static_cast<hipStream_t>(j.stream);
    const int64_t eb = j.ct == 1 ? 4 : 2;
    GroupedParams p{j.a_codes, j.a_scales, (int)j.a_rows, j.b_codes, j.b_scales,
                    (int)(j.stacked ? j.N : (j.N + kBlock - 1) / kBlock * kBlock), j.tokens,
                    Groups{j.offsets, (int)j.experts, (int)j.rows, j.clear_rest}, (int)j.N, (int)j.K,
                    (int)((j.K + kBlock - 1) / kBlock), static_cast<char*>(j.c), j.ct, j.N * eb % 16 == 0 && (uintptr_t)j.c % 16 == 0, 0};
    // Groups that hold a row, at most: as the kernel is chosen (a product's is the same, and so are its
    // bits, whether the other rows are cleared or not), and with all rows of no group.
    const int64_t some = std::min(j.rows, j.chosen_by);
    const int64_t most = std::min(j.rows, j.experts + (j.clear_rest ? 2 : 0));
    const bool gather = j.tokens != nullptr, brow = j.stacked && j.N % kBlock != 0;
    // Up to eight rows a group on average: a pass over the weights.  (64 experts of 2048 x 4096, launches
    // one after the other, over three sets of weights or one alike, against 64 x 64 tiles.  The same rows
    // for each expert: 64 rows 110 to 130 us and 123 to 126; 256 rows 112 to 127 and 123 to 127; 512 rows
    // 120 to 138 and 123 to 127; 640 rows 131 to 147 and 125 to 127; 1024 rows 143 to 153 and 126 to 128.
    // Routed, the largest groups several times the mean: 128 rows 83 to 84 and 101 to 104; 256 rows 101 to
    // 103 and 111 to 114; 384 rows 116 to 118 both; 512 rows 128 to 131 and 123 to 125; 640 rows 142 to 146
    // and 122 to 127.  The sizes are not known here: should one expert own all of 512 rows, 147 to 150 us,
    // in tiles 16 to 19.)
    if (j.rows <= 8 * some) {
        const int64_t groups = most * ((j.N + kFewRows - 1) / kFewRows);
        if (groups > INT32_MAX) return too_many(what, msg, msg_len);
        // Eight waves, of two K blocks or more each.  (64 experts of 2048 x 4096, 64 rows of 8 tokens,
        // weights from memory, by events: 99 us; with 4 waves 105, with 16 143.  32 experts of
        // 1024 x 1024, 32 rows: 13.5 with 8, 10.5 with 4.)
        int waves = kFewMaxWaves;
        while (waves > 1 && waves * 2 > p.S) waves /= 2;
        for (int64_t first = 0; first < groups; first += kMaxGrid) {
            const dim3 grid((unsigned)std::min(groups - first, kMaxGrid)), block(waves * kWave);
            p.first = (unsigned)first;
            if (brow && gather) FP4Q_LAUNCH((k_grouped_few<true, true>), grid, block, 0, stream, p);
            else if (brow) FP4Q_LAUNCH((k_grouped_few<true, false>), grid, block, 0, stream, p);
            else if (gather) FP4Q_LAUNCH((k_grouped_few<false, true>), grid, block, 0, stream, p);
            else FP4Q_LAUNCH((k_grouped_few<false, false>), grid, block, 0, stream, p);
        }
        return status(what, msg, msg_len);
    }
    // A group ends in the middle of a tile, on average.
    const int tile = choose(j.ct == 1, p.S, [&](int t) {
        return std::max((double)some, (double)j.rows / t + 0.5 * (double)some) * (double)((j.N + t - 1) / t);
    });
    const int64_t groups = (j.rows + (tile - 1) * most) / tile * ((j.N + tile - 1) / tile);
    if (groups > INT32_MAX) return too_many(what, msg, msg_len);
    if (brow && gather) launch_tiles<true, true>(p, tile, groups, stream);
    else if (brow) launch_tiles<true, false>(p, tile, groups, stream);
    else if (gather) launch_tiles<false, true>(p, tile, groups, stream);
    else launch_tiles<false, false>(p, tile, groups, stream);
    return status(what, msg, msg_len);
}

int launch_grouped_outer(const GroupedOuterJob& j, char* msg, size_t msg_len) {
    const char* what = "grouped weight gradient";
    if (j.M == 0 || j.N == 0) return 0;
    hipStream_t stream = static_cast<hipStream_t>(j.stream);
    const int64_t blocks = fp8_group_blocks(j.rows, j.experts), eb = j.ct == 1 ? 4 : 2;
    OuterParams p{j.a_codes, j.a_scales, j.b_codes, j.b_scales, Groups{j.offsets, (int)j.experts, (int)j.rows, false}, (int)j.M, (int)j.N,
                  (int)(blocks * kBlock), static_cast<char*>(j.c), j.ct, j.N * eb % 16 == 0 && (uintptr_t)j.c % 16 == 0, 0};
    auto tiles = [&](int t) { return j.experts * ((j.M + t - 1) / t) * ((j.N + t - 1) / t); };
    const int tile = choose(j.ct == 1, (double)j.rows / 128 / (double)j.experts + 0.5, [&](int t) { return (double)tiles(t); });
    const int64_t groups = (tiles(tile) / j.experts + 7) / 8 * 8 * j.experts;
    if (groups > INT32_MAX) return too_many(what, msg, msg_len);
    for (int64_t first = 0; first < groups; first += kMaxGrid) {
        const dim3 grid((unsigned)std::min(groups - first, kMaxGrid));
        p.first = (unsigned)first;
        if (tile == 256) FP4Q_LAUNCH(k_grouped_outer, grid, dim3(kThreads), 0, stream, p);
        else if (tile == 128 && j.ct == 1) FP4Q_LAUNCH((k_grouped_outer_mid<128, true>), grid, dim3(256), MidPlan<128>::kLds, stream, p);
        else if (tile == 128) FP4Q_LAUNCH((k_grouped_outer_mid<128, false>), grid, dim3(256), MidPlan<128>::kLds, stream, p);
        else if (j.ct == 1) FP4Q_LAUNCH((k_grouped_outer_mid<64, true>), grid, dim3(256), MidPlan<64>::kLds, stream, p);
        else FP4Q_LAUNCH((k_grouped_outer_mid<64, false>), grid, dim3(256), MidPlan<64>::kLds, stream, p);
    }
    return status(what, msg, msg_len);
}

// ---------------------------------------------------------------------------
// The slots of a batch by expert: a counting sort that keeps the slots' order.  A workgroup of 16
// waves takes a run of slots, a wave a run of that; a wave counts its slots of each expert, 64 at a
// time (the lanes with a lane's own expert are found bit by bit), and then places them behind
// those of the experts before, of the workgroups before and of the waves before.  Up to kOneRun
// slots take one workgroup and one launch; more take a launch that counts and one that places.
// (40 slots: 2.7 us.  131072 slots of 128 experts: 3.3 us to count, 8.4 to place, of which the
// counts of the 128 runs, each thread reading one expert's in a row, once took 25.)

namespace {

constexpr int kOrderWaves = 16;
constexpr int kOrderThreads = kOrderWaves * kWave;
constexpr int kOneRun = 4096;
constexpr int kMostRuns = 128;
constexpr int kBuckets = 513;  // experts, and the slots of none

struct OrderParams {
    const void* ids;
    bool wide;
    int64_t slots;
    int top_k, experts;
    int64_t run;         // slots per workgroup, a multiple of kOrderThreads
    int runs;
    int* counts;         // runs x (experts + 1)
    int *offsets, *order, *token, *position;
};

__device__ __forceinline__ int bucket_of(const OrderParams& p, int64_t slot) {
    const int64_t id = p.wide ? static_cast<const int64_t*>(p.ids)[slot] : static_cast<const int*>(p.ids)[slot];
    return id >= 0 && id < p.experts ? (int)id : p.experts;
}

// Lanes of the wave with this lane's bucket (those of `in` alone).
__device__ __forceinline__ uint64_t same(int bucket, bool in, int bits) {
    uint64_t m = __builtin_amdgcn_ballot_w64(in);
    for (int b = 0; b < bits; ++b) {
        const uint64_t one = __builtin_amdgcn_ballot_w64((bucket >> b & 1) != 0);
        m &= bucket >> b & 1 ? one : ~one;
    }
    return m;
}

// Adds this workgroup's slots of each bucket to counts[wave][bucket] in LDS, then turns them into
// sums over the waves before; total[bucket]: all waves'.
__device__ __forceinline__ void count_run(const OrderParams& p, int64_t lo, int64_t hi, int (*counts)[kBuckets], int* total) {
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave, buckets = p.experts + 1;
    for (int i = threadIdx.x; i < kOrderWaves * kBuckets; i += kOrderThreads) counts[0][i] = 0;
    __syncthreads();
    const int64_t per = p.run / kOrderWaves, mine = lo + wave * per, end = min(hi, mine + per);
    for (int64_t s = mine + lane; s < end; s += kWave) atomicAdd(&counts[wave][bucket_of(p, s)], 1);
    __syncthreads();
    for (int b = threadIdx.x; b < buckets; b += kOrderThreads) {
        int sum = 0;
        for (int w = 0; w < kOrderWaves; ++w) {
            const int n = counts[w][b];
            counts[w][b] = sum;
            sum += n;
        }
        total[b] = sum;
    }
    __syncthreads();
}

__global__ __launch_bounds__(kOrderThreads) void k_order_count(OrderParams p) {
    __shared__ int counts[kOrderWaves][kBuckets];
    __shared__ int total[kBuckets];
    const int64_t lo = blockIdx.x * p.run;
    count_run(p, lo, min(lo + p.run, p.slots), counts, total);
    for (int b = threadIdx.x; b <= p.experts; b += kOrderThreads) p.counts[(int64_t)blockIdx.x * (p.experts + 1) + b] = total[b];
}

__global__ __launch_bounds__(kOrderThreads) void k_order_place(OrderParams p) {
    __shared__ int counts[kOrderWaves][kBuckets];
    __shared__ int total[kBuckets];   // this run's, then all runs'
    __shared__ int before[kBuckets];  // of the runs before
    __shared__ int start[kBuckets];   // of the buckets before
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave, buckets = p.experts + 1;
    const int64_t lo = blockIdx.x * p.run, hi = min(lo + p.run, p.slots);
    count_run(p, lo, hi, counts, total);
    // The other runs' slots: kParts threads a bucket, each some of the runs, reads side by side.
    for (int b = threadIdx.x; b < buckets; b += kOrderThreads) before[b] = 0;
    if (p.runs > 1) {
        __syncthreads();
        for (int b = threadIdx.x; b < buckets; b += kOrderThreads) total[b] = 0;
        __syncthreads();
        const int parts = kOrderThreads / buckets > 0 ? kOrderThreads / buckets : 1;
        const int part = threadIdx.x / buckets, each = (p.runs + parts - 1) / parts;
        const int r_end = min(p.runs, (part + 1) * each);
        if (part < parts) {
            const int b = threadIdx.x - part * buckets;
            int sum = 0, all = 0;
            for (int r0 = part * each; r0 < r_end; r0 += 16) {
                int n[16];
#pragma unroll
                for (int r = 0; r < 16; ++r) n[r] = p.counts[(int64_t)min(r0 + r, p.runs - 1) * buckets + b];
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int one = r0 + r < r_end ? n[r] : 0;
                    all += one;
                    sum += r0 + r < (int)blockIdx.x ? one : 0;
                }
            }
            atomicAdd(&before[b], sum);
            atomicAdd(&total[b], all);
        }
    }
    __syncthreads();
    if (wave == 0) {
        int sum = 0;
        for (int c = 0; c < buckets; c += kWave) {
            const int n = c + lane < buckets ? total[c + lane] : 0, sums = wave_sums(n);
            if (c + lane < buckets) start[c + lane] = sum + sums - n;
            sum += __builtin_amdgcn_readlane(sums, 63);
        }
    }
    __syncthreads();
    if (blockIdx.x == 0)
        for (int b = threadIdx.x; b < buckets; b += kOrderThreads) p.offsets[b] = start[b];
    const int64_t per = p.run / kOrderWaves, mine = lo + wave * per, end = min(hi, mine + per);
    const int bits = 32 - __builtin_clz(p.experts);  // of a bucket
    int* next = counts[wave];
    for (int64_t s0 = mine; s0 < end; s0 += kWave) {
        const int64_t s = s0 + lane;
        const bool in = s < end;
        const int b = in ? bucket_of(p, s) : 0;
        const uint64_t mates = same(b, in, bits), below = mates & ((1ull << lane) - 1);
        const int at = in ? start[b] + before[b] + next[b] + __builtin_popcountll(below) : 0;
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // read before the first of them moves it on
        if (in && below == 0) next[b] += __builtin_popcountll(mates);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        if (in) {
            p.order[at] = (int)s;
            p.token[at] = (int)((unsigned)s / (unsigned)p.top_k);
            p.position[s] = at;
        }
    }
}

// Slots per workgroup, and workgroups.
void order_runs(int64_t slots, int64_t& run, int& runs) {
    const int64_t least = slots <= kOneRun ? slots : kOrderThreads;
    run = std::max(least, (slots + kMostRuns - 1) / kMostRuns);
    run = std::max<int64_t>(run, 1);
    run = (run + kOrderThreads - 1) / kOrderThreads * kOrderThreads;
    runs = (int)std::max<int64_t>(1, (slots + run - 1) / run);
}

}  // namespace

size_t expert_order_workspace_bytes(int64_t slots, int64_t experts) {
    int64_t run;
    int runs;
    order_runs(slots, run, runs);
    return runs > 1 ? (size_t)(4 * runs * (experts + 1)) : 0;
}

int launch_expert_order(const ExpertOrderJob& j, char* msg, size_t msg_len) {
    hipStream_t stream = static_cast<hipStream_t>(j.stream);
    OrderParams p{j.ids, j.wide, j.tokens * j.top_k, (int)j.top_k, (int)j.experts, 0, 0, static_cast<int*>(j.ws),
                  j.offsets, j.order, j.token, j.position};
    order_runs(p.slots, p.run, p.runs);
    if (p.runs > 1) FP4Q_LAUNCH(k_order_count, dim3(p.runs), dim3(kOrderThreads), 0, stream, p);
    FP4Q_LAUNCH(k_order_place, dim3(p.runs), dim3(kOrderThreads), 0, stream, p);
    return status("expert order", msg, msg_len);
}

}  // namespace fp4q
