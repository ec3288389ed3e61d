// fp4q_fp8_quantize.hip -- E4M3 codes with one binary32 scale per 128 elements
// (fp8_quantize_b128), of a matrix and, from the same read, of its transpose.
//
// For a block of 128 elements along a row (row scales) or of 128 x 128 (tile
// scales), with a = max |x|:
//   s = max(RN32(a / 448), 2^-126)       448 is the largest E4M3 value
//   c = E4M3 nearest to RN32(x / s), ties to even
// The floor of s keeps s and 1 / s normal numbers, so an all-zero block needs no
// case of its own; |x / s| is at most 448 (1 + 2^-23), which rounds to 448: the
// conversion never saturates.
//
// One workgroup of 256 threads takes a 128 x 128 tile.  Thread (i, j) of 16 x 16
// holds rows 8 i .. 8 i + 7 by columns 8 j .. 8 j + 7, so that both packings come
// out of registers: 8 codes along a row are one 8-byte store of the row-major
// codes, 8 along a column one 8-byte piece of the transposed ones, which pass
// through LDS to leave as whole 128-byte rows.  Row maxima are a DPP maximum over
// the 16 threads of a row group; column maxima cross the workgroup through LDS.
//
// Memory-bound: 2 or 4 bytes in and 1 or 2 out per element, against about 8
// vector instructions (12 with both outputs).  Measured: 8192 x 3584 bf16, row
// scales, both outputs, 119 MB in 22.8 us (5.2 TB/s, where a large copy reached 4.7);
// 4861 x 5000 binary32, tile scales, both, 146 MB in 28 us (5.2 TB/s); 7 x 896 in
// 5.1 us, the time of any launch that waits for memory twice.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <stdio.h>

#include "fp4q_launch.h"

namespace fp4q {
namespace {

constexpr int kTile = 128;      // rows and columns of a workgroup's tile
constexpr int kThreads = 256;
constexpr int kSide = 8;        // rows and columns of a thread's part
constexpr int kPitch = kTile + 8;  // LDS bytes per transposed row: 8-byte writes of 4 columns x 16 row groups
                                   // then fall in distinct banks, and rows start on 8 bytes
constexpr float kMinScale = 0x1p-126f;
// Scales for which the corrected quotient below is RN32(x / s) wherever it can
// matter: from 2^-60 up, |x| < 2^-100 means a quotient below 2^-40, a zero code.
constexpr float kFastLo = 0x1p-60f, kFastHi = 0x1p100f;

struct Fp8Params {
    const void* x;
    int64_t rows, cols;
    int64_t ld, ld_t;        // bytes per row of codes and of codes_t
    int64_t tiles_c;         // tiles along the columns
    unsigned first;          // this launch's first tile
    uint8_t* codes;          // NULL: not wanted
    float* scales;
    uint8_t* codes_t;        // NULL: not wanted
    float* scales_t;
};

template <int T>
struct Elem;
template <>
struct Elem<0> {
    typedef uint16_t Bits;
    static __device__ __forceinline__ float f32(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
};
template <>
struct Elem<1> {
    typedef uint32_t Bits;
    static __device__ __forceinline__ float f32(uint32_t b) { return __uint_as_float(b); }
};

// Maximum over the 16 lanes of a DPP row.
__device__ __forceinline__ float row16_max(float v) {
    int b = __float_as_int(v);
    v = fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(b, b, 0x121, 0xF, 0xF, true)));  // row_ror:1
    b = __float_as_int(v);
    v = fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(b, b, 0x122, 0xF, 0xF, true)));  // row_ror:2
    b = __float_as_int(v);
    v = fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(b, b, 0x124, 0xF, 0xF, true)));  // row_ror:4
    b = __float_as_int(v);
    v = fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(b, b, 0x128, 0xF, 0xF, true)));  // row_ror:8
    return v;
}

// Lanes 0 .. 7 of each DPP row, to all of it.
__device__ __forceinline__ void from_lanes(float (&out)[8], float v) {
    const int b = __float_as_int(v);
    out[0] = __int_as_float(__builtin_amdgcn_update_dpp(0, b, 0x150, 0xF, 0xF, true));  // row_newbcast:0
    out[1] = __int_as_float(__builtin_amdgcn_update_dpp(0, b, 0x151, 0xF, 0xF, true));
    out[2] = __int_as_float(__builtin_amdgcn_update_dpp(0, b, 0x152, 0xF, 0xF, true));
    out[3] = __int_as_float(__builtin_amdgcn_update_dpp(0, b, 0x153, 0xF, 0xF, true));
    out[4] = __int_as_float(__builtin_amdgcn_update_dpp(0, b, 0x154, 0xF, 0xF, true));
    out[5] = __int_as_float(__builtin_amdgcn_update_dpp(0, b, 0x155, 0xF, 0xF, true));
    out[6] = __int_as_float(__builtin_amdgcn_update_dpp(0, b, 0x156, 0xF, 0xF, true));
    out[7] = __int_as_float(__builtin_amdgcn_update_dpp(0, b, 0x157, 0xF, 0xF, true));
}

__device__ __forceinline__ float scale_of(float amax) { return fmaxf(amax / 448.0f, kMinScale); }

__device__ __forceinline__ bool fast_scale(float s) { return s >= kFastLo && s <= kFastHi; }

// RN32(x / s) from r = RN32(1 / s): the reciprocal product corrected once by its
// exact remainder, negated so that -0 stays -0.
__device__ __forceinline__ float quotient(float x, float s, float r) {
    const float q = x * r;
    const float n = fmaf(q, s, -x);
    return fmaf(-n, r, q);
}

__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}

// 8 codes of v[0], v[stride], ... under one scale each (sc, rc indexed alike).
template <bool FAST>
__device__ __forceinline__ uint2 codes8(const float (&v)[8], const float (&s)[8], const float (&r)[8]) {
    float q[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) q[k] = FAST ? quotient(v[k], s[k], r[k]) : v[k] / s[k];
    return make_uint2(pack4(q[0], q[1], q[2], q[3]), pack4(q[4], q[5], q[6], q[7]));
}

struct Fp8Lds {
    float part[16][kTile];            // column maxima of each row group
    float col_s[kTile], col_r[kTile];
};

// One workgroup's tile.  TILE: one scale per 128 x 128, else one per 128 of a row (and,
// for the transposed output, of a column).  OUT, TOUT: which outputs are wanted; flip: 128
// transposed rows, with TOUT.
template <int XT, bool TILE, bool OUT, bool TOUT>
__device__ __forceinline__ void quantize_tile(const Fp8Params& p, unsigned tile, Fp8Lds& lds, uint8_t* flip) {
    typedef typename Elem<XT>::Bits Bits;
    auto& part = lds.part;
    auto& col_s = lds.col_s;
    auto& col_r = lds.col_r;
    const int t = threadIdx.x, i = t / 16, j = t % 16;
    const int64_t tile_r = tile / p.tiles_c, tile_c = tile % p.tiles_c;
    const int64_t r0 = tile_r * kTile, c0 = tile_c * kTile;
    const int64_t row0 = r0 + kSide * i, col0 = c0 + kSide * j;
    const int n_rows = (int)min((int64_t)kSide, max((int64_t)0, p.rows - row0));
    const int n_cols = (int)min((int64_t)kSide, max((int64_t)0, p.cols - col0));

    // Rows need not start on any boundary past their element's: 8 elements are one
    // unaligned wide load (two for binary32), or single loads where the row ends
    // within them.  What does not exist is +0: its loads are of the nearest element
    // that does (no branch, so that all are in flight together), and dropped.
    struct __attribute__((packed, aligned(sizeof(Bits)))) Eight { Bits e[8]; };
    float v[8][8];
    if (n_cols == kSide && n_rows > 0) {
        Eight w[8];
#pragma unroll
        for (int a = 0; a < 8; ++a)
            w[a] = *reinterpret_cast<const Eight*>(static_cast<const Bits*>(p.x) + (row0 + min(a, n_rows - 1)) * p.cols + col0);
#pragma unroll
        for (int a = 0; a < 8; ++a)
#pragma unroll
            for (int b = 0; b < 8; ++b) v[a][b] = a < n_rows ? Elem<XT>::f32(w[a].e[b]) : 0.0f;
    } else if (n_cols > 0 && n_rows > 0) {
#pragma unroll
        for (int a = 0; a < 8; ++a) {
            const Bits* src = static_cast<const Bits*>(p.x) + (row0 + min(a, n_rows - 1)) * p.cols + col0;
#pragma unroll
            for (int b = 0; b < 8; ++b) v[a][b] = Elem<XT>::f32(src[min(b, n_cols - 1)]);
        }
#pragma unroll
        for (int a = 0; a < 8; ++a)
#pragma unroll
            for (int b = 0; b < 8; ++b) v[a][b] = a < n_rows && b < n_cols ? v[a][b] : 0.0f;
    } else {
#pragma unroll
        for (int a = 0; a < 8; ++a)
#pragma unroll
            for (int b = 0; b < 8; ++b) v[a][b] = 0.0f;
    }

    float rm[8], cm[8];
#pragma unroll
    for (int a = 0; a < 8; ++a) {
        rm[a] = 0.0f;
#pragma unroll
        for (int b = 0; b < 8; ++b) rm[a] = fmaxf(rm[a], fabsf(v[a][b]));
        rm[a] = row16_max(rm[a]);
    }
    if (!TILE && TOUT) {
#pragma unroll
        for (int b = 0; b < 8; ++b) {
            cm[b] = 0.0f;
#pragma unroll
            for (int a = 0; a < 8; ++a) cm[b] = fmaxf(cm[b], fabsf(v[a][b]));
            part[i][kSide * j + b] = cm[b];
        }
        __syncthreads();
        if (t < kTile) {
            float m = part[0][t];
#pragma unroll
            for (int g = 1; g < 16; ++g) m = fmaxf(m, part[g][t]);
            const float s = scale_of(m);
            col_s[t] = s;
            col_r[t] = 1.0f / s;
            if (c0 + t < p.cols) p.scales_t[tile_r * p.cols + c0 + t] = s;
        }
        __syncthreads();
    }

    float s[8], r[8];
    if (TILE) {
        float m = rm[0];
#pragma unroll
        for (int a = 1; a < 8; ++a) m = fmaxf(m, rm[a]);
        if (j == 0) part[0][i] = m;
        __syncthreads();
        m = part[0][0];
#pragma unroll
        for (int g = 1; g < 16; ++g) m = fmaxf(m, part[0][g]);
        const float sc = scale_of(m), rc = 1.0f / sc;
#pragma unroll
        for (int a = 0; a < 8; ++a) s[a] = sc, r[a] = rc;
        if (t == 0) {
            if (OUT) p.scales[tile_r * p.tiles_c + tile_c] = sc;
            if (TOUT) p.scales_t[tile_c * ((p.rows + kTile - 1) / kTile) + tile_r] = sc;
        }
    } else if (OUT) {
        // Lane j of a row group forms the scale of its row j (mod 8), and hands it out.
        float m = rm[0];
#pragma unroll
        for (int a = 1; a < 8; ++a) m = j % 8 == a ? rm[a] : m;
        const float mine = scale_of(m), inv = 1.0f / mine;
        from_lanes(s, mine);
        from_lanes(r, inv);
        if (j < n_rows) p.scales[tile_c * p.rows + row0 + j] = mine;
    }

    if (OUT) {
        bool fast = true;
#pragma unroll
        for (int a = 0; a < 8; ++a) fast = fast && fast_scale(s[a]);
        const bool all_fast = __builtin_amdgcn_ballot_w64(!fast) == 0;  // wave-uniform
        if (col0 < p.ld) {
            uint8_t* dst = p.codes + row0 * p.ld + col0;
#pragma unroll
            for (int a = 0; a < 8; ++a) {
                const float ss[8] = {s[a], s[a], s[a], s[a], s[a], s[a], s[a], s[a]};
                const float rr[8] = {r[a], r[a], r[a], r[a], r[a], r[a], r[a], r[a]};
                const uint2 w = all_fast ? codes8<true>(v[a], ss, rr) : codes8<false>(v[a], ss, rr);
                if (a < n_rows) *reinterpret_cast<uint2*>(dst + a * p.ld) = w;
            }
        }
    }
    if (TOUT) {
        if (!TILE) {
#pragma unroll
            for (int b = 0; b < 8; ++b) {
                s[b] = col_s[kSide * j + b];
                r[b] = col_r[kSide * j + b];
            }
        }
        bool fast = true;
#pragma unroll
        for (int b = 0; b < 8; ++b) fast = fast && fast_scale(s[b]);
        const bool all_fast = __builtin_amdgcn_ballot_w64(!fast) == 0;
#pragma unroll
        for (int b = 0; b < 8; ++b) {
            const float ss[8] = {s[b], s[b], s[b], s[b], s[b], s[b], s[b], s[b]};
            const float rr[8] = {r[b], r[b], r[b], r[b], r[b], r[b], r[b], r[b]};
            const float col[8] = {v[0][b], v[1][b], v[2][b], v[3][b], v[4][b], v[5][b], v[6][b], v[7][b]};
            const uint2 w = all_fast ? codes8<true>(col, ss, rr) : codes8<false>(col, ss, rr);
            *reinterpret_cast<uint2*>(flip + (kSide * j + b) * kPitch + kSide * i) = w;
        }
        __syncthreads();
        // 128 transposed rows of 128 bytes: 8 threads per row, 16 bytes each.
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int c = k * 32 + t / 8;
            const int64_t at = r0 + 16 * (t % 8);
            const uint2 lo = *reinterpret_cast<const uint2*>(flip + c * kPitch + 16 * (t % 8));
            const uint2 hi = *reinterpret_cast<const uint2*>(flip + c * kPitch + 16 * (t % 8) + 8);
            if (c0 + c < p.cols && at < p.ld_t)
                *reinterpret_cast<uint4*>(p.codes_t + (c0 + c) * p.ld_t + at) = make_uint4(lo.x, lo.y, hi.x, hi.y);
        }
    }
}

template <int XT, bool TILE, bool OUT, bool TOUT>
__global__ __launch_bounds__(kThreads) void k_fp8_quantize(Fp8Params p) {
    __shared__ Fp8Lds lds;
    __shared__ __attribute__((aligned(16))) uint8_t flip[TOUT ? kTile * kPitch : 16];
    quantize_tile<XT, TILE, OUT, TOUT>(p, p.first + blockIdx.x, lds, flip);
}

// A linear layer's input (row scales) and weight (tile scales), both outputs of each, in
// one launch: small layers fill the chip with neither.  (509 x 896 and 4864 x 896 binary32:
// 11.6 us, 7.6 and 11 one after the other; 4096 x 4096 and 14336 x 4096 bf16: 57, 17 and 44.)
template <int XT, int WT>
__global__ __launch_bounds__(kThreads) void k_fp8_quantize_two(Fp8Params x, Fp8Params w, unsigned x_tiles) {
    __shared__ Fp8Lds lds;
    __shared__ __attribute__((aligned(16))) uint8_t flip[kTile * kPitch];
    if (blockIdx.x < x_tiles) quantize_tile<XT, false, true, true>(x, blockIdx.x, lds, flip);
    else quantize_tile<WT, true, true, true>(w, blockIdx.x - x_tiles, lds, flip);
}

template <int XT, bool TILE>
void launch_outs(const Fp8Params& p, unsigned grid, void* stream_) {
    hipStream_t stream = static_cast<hipStream_t>(stream_);
    if (p.codes && p.codes_t) FP4Q_LAUNCH((k_fp8_quantize<XT, TILE, true, true>), dim3(grid), dim3(kThreads), 0, stream, p);
    else if (p.codes) FP4Q_LAUNCH((k_fp8_quantize<XT, TILE, true, false>), dim3(grid), dim3(kThreads), 0, stream, p);
    else FP4Q_LAUNCH((k_fp8_quantize<XT, TILE, false, true>), dim3(grid), dim3(kThreads), 0, stream, p);
}

}  // namespace

namespace {
Fp8Params params_of(const Fp8QuantJob& j) {
    Fp8Params p{};
    p.x = j.x;
    p.rows = j.rows;
    p.cols = j.cols;
    p.ld = (j.cols + 15) / 16 * 16;
    p.ld_t = (j.rows + 15) / 16 * 16;
    p.tiles_c = (j.cols + kTile - 1) / kTile;
    p.codes = j.codes;
    p.scales = j.scales;
    p.codes_t = j.codes_t;
    p.scales_t = j.scales_t;
    return p;
}
int64_t tiles_of(const Fp8Params& p) { return p.tiles_c * ((p.rows + kTile - 1) / kTile); }
int launch_status(char* msg, size_t msg_len) {
    const hipError_t e = hipGetLastError();
    if (e == hipSuccess) return 0;
    snprintf(msg, msg_len, "fp8 quantize kernel launch: %s", hipGetErrorString(e));
    return (int)e;
}
}  // namespace

int launch_fp8_quantize_two(const Fp8QuantJob& x, const Fp8QuantJob& w, char* msg, size_t msg_len) {
    const bool all = x.rows > 0 && x.cols > 0 && w.rows > 0 && w.cols > 0 && !x.tile && w.tile && x.codes && x.codes_t &&
                     w.codes && w.codes_t;
    const Fp8Params px = params_of(x), pw = params_of(w);
    const int64_t tx = tiles_of(px), tiles = tx + tiles_of(pw);
    if (!all || tiles > kMaxGrid) {
        const int rc = launch_fp8_quantize(x, msg, msg_len);
        return rc ? rc : launch_fp8_quantize(w, msg, msg_len);
    }
    hipStream_t stream = static_cast<hipStream_t>(x.stream);
    const dim3 grid((unsigned)tiles), block(kThreads);
    const unsigned n = (unsigned)tx;
    if (x.xt == 0 && w.xt == 0) FP4Q_LAUNCH((k_fp8_quantize_two<0, 0>), grid, block, 0, stream, px, pw, n);
    else if (x.xt == 0) FP4Q_LAUNCH((k_fp8_quantize_two<0, 1>), grid, block, 0, stream, px, pw, n);
    else if (w.xt == 0) FP4Q_LAUNCH((k_fp8_quantize_two<1, 0>), grid, block, 0, stream, px, pw, n);
    else FP4Q_LAUNCH((k_fp8_quantize_two<1, 1>), grid, block, 0, stream, px, pw, n);
    return launch_status(msg, msg_len);
}

int launch_fp8_quantize(const Fp8QuantJob& j, char* msg, size_t msg_len) {
    if (j.rows == 0 || j.cols == 0) return 0;
    Fp8Params p = params_of(j);
    const int64_t tiles = tiles_of(p);
    if (tiles > INT32_MAX) {
        snprintf(msg, msg_len, "fp8 quantize: %lld x %lld needs more workgroups than one launch holds",
                 (long long)j.rows, (long long)j.cols);
        return (int)hipErrorInvalidConfiguration;
    }
    for (int64_t first = 0; first < tiles; first += kMaxGrid) {
        const unsigned grid = (unsigned)(tiles - first < kMaxGrid ? tiles - first : kMaxGrid);
        p.first = (unsigned)first;
        if (j.xt == 0) {
            if (j.tile) launch_outs<0, true>(p, grid, j.stream);
            else launch_outs<0, false>(p, grid, j.stream);
        } else {
            if (j.tile) launch_outs<1, true>(p, grid, j.stream);
            else launch_outs<1, false>(p, grid, j.stream);
        }
    }
    return launch_status(msg, msg_len);
}

}  // namespace fp4q
