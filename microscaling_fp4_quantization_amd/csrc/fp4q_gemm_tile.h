// fp4q_gemm_tile.h -- what the 256 x 256 tile GEMMs share (fp4q_gemm.hip,
// fp4q_fp8_gemm.hip): the tile and its waves, buffer windows, the order of
// tiles over the XCDs, waits, and the epilogue.  Device code only; each
// including file gets its own copy.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp4q {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef unsigned int u32x2_t __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));
typedef __amdgpu_buffer_rsrc_t Rsrc;
typedef __attribute__((address_space(3))) void* LdsPtr;

constexpr int kWave = 64;
constexpr int kWaves = 8;
constexpr int kThreads = kWave * kWaves;
constexpr int BM = 256, BN = 256;          // workgroup tile: rows of A, rows of B
constexpr int kFrag = 32;                  // rows per matrix-core operand
constexpr int WM = 128, WN = 64;           // wave tile: rows of A, rows of B
constexpr int FA = WM / kFrag, FB = WN / kFrag;
constexpr int kRowStage = 128;             // code bytes per row per stage (one cache line)
constexpr int kCodeBytes = (BM + BN) * kRowStage;  // a stage's codes in LDS (64 KB)
constexpr int kEpiBytes = 2 * kCodeBytes;  // LDS the epilogue stages the tile through
constexpr int kDropped = (int)0x80000000;  // an offset past every buffer window
constexpr int kPastWindow = 1 << 30;       // every window is at most 2^30 bytes
constexpr int kRsrcWord3 = 0x00020000;
// Cache policy of the stores of C: non-temporal.  C is written once and not
// read back here; cached, it evicts the operand rows the other tiles of the
// XCD are about to read (measured: a fifth of the time of a 8192 x 18944 x
// 3584 product).
constexpr int kStoreNT = 2;

__device__ __forceinline__ Rsrc make_rsrc(const void* base, int64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, (int)bytes, kRsrcWord3);
}

// Round-to-nearest-even binary32 -> bf16 bits.
__device__ __forceinline__ uint32_t to_bf16(float f) {
    const uint32_t b = __float_as_uint(f);
    return (b + 0x7FFFu + ((b >> 16) & 1u)) >> 16;
}

// Tile of workgroup g: the 8 XCDs take workgroups round robin, so tiles are
// renumbered to give each XCD a contiguous run, walked in groups of kGroupM
// tile rows so that concurrently running tiles share operand rows in its L2.
constexpr int kGroupM = 4;

__device__ __forceinline__ void tile_of(int64_t g, int64_t tiles_m, int64_t tiles_n, int64_t& tm,
                                        int64_t& tn) {
    const int64_t T = tiles_m * tiles_n;
    const int64_t xcd = g % 8, idx = g / 8, per = T / 8, rem = T % 8;
    const int64_t t = xcd < rem ? xcd * (per + 1) + idx : rem * (per + 1) + (xcd - rem) * per + idx;
    const int64_t span = (int64_t)kGroupM * tiles_n;
    const int64_t first = (t / span) * kGroupM;
    const int64_t gm = tiles_m - first < kGroupM ? tiles_m - first : kGroupM;
    tm = first + (t % span) % gm;
    tn = (t % span) / gm;
}

// Wait for all of this wave's loads (the next stage's codes and scales) and
// LDS reads, then barrier.  The memory clobber keeps LDS accesses from moving
// across.
__device__ __forceinline__ void wait_all_barrier() {
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// Wait until at most N of this wave's loads are in flight, then barrier.  A
// workgroup fence would wait for all of them (the later stage too).  The wait
// is the compiler's builtin, so that it knows the scale registers loaded
// before those N have landed (and adds no wait of its own for them).
template <int N>
__device__ __forceinline__ void wait_loads_barrier() {
    static_assert(N >= 0 && N < 16, "vmcnt range");
    __builtin_amdgcn_s_waitcnt(0x0F70 | N);  // vmcnt(N), expcnt and lgkmcnt unconstrained
    asm volatile("s_barrier" ::: "memory");
}

// Wait for this wave's LDS reads, then barrier: afterwards no wave reads the
// stage buffer any more.  (The compiler's builtin again, so that its own
// bookkeeping of outstanding LDS reads agrees.)
__device__ __forceinline__ void lds_reads_barrier() {
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0), vmcnt and expcnt unconstrained
    asm volatile("s_barrier" ::: "memory");
}

// s_waitcnt vmcnt(N) for N < 64 (the count's high bits sit at bits 14-15),
// expcnt and lgkmcnt unconstrained.
template <int N>
__device__ __forceinline__ void wait_vm() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x0F70);
}

// Four results in the output format: EB = 4 binary32, EB = 2 bf16 (round to
// nearest even), packed in 16 or 8 bytes.
template <int EB>
struct Quad;
template <>
struct Quad<4> {
    typedef u32x4_t T;
    static __device__ __forceinline__ T pack(float a, float b, float c, float d) {
        return u32x4_t{__float_as_uint(a), __float_as_uint(b), __float_as_uint(c), __float_as_uint(d)};
    }
};
// Two binary32 values to bf16 in one v_cvt_pk_bf16_f32, which rounds to
// nearest even as to_bf16 does (for every input but NaN, which stays NaN):
// the epilogue's conversions took about 2 us of a 30 us tile as integer
// arithmetic.
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{lo, hi}, bf16x2_t));
}

template <>
struct Quad<2> {
    typedef u32x2_t T;
    static __device__ __forceinline__ T pack(float a, float b, float c, float d) {
        return u32x2_t{pack_bf16x2(a, b), pack_bf16x2(c, d)};
    }
};

// Epilogue through LDS, for rows of C that are whole 16-byte units: the tile
// is written to LDS row-major (in passes of as many rows as 128 KB holds),
// then stored with each lane moving 16 contiguous bytes, so that a store
// covers whole cache lines.  In LDS the 4-column group k of row r sits at
// group k ^ (r % 32): the 32 rows a wave writes at once then fall in distinct
// banks, and a 16-byte read holds the same two groups, possibly swapped.
template <int EB>
__device__ __forceinline__ void store_tile(const v16f (&acc)[FB][FA], uint8_t* lds, Rsrc rc, int wave,
                                           int wm, int wn, int lane, int64_t rows_a, int64_t n0,
                                           int64_t N) {
    constexpr int kPitch = BN * EB;                   // LDS bytes per row
    constexpr int kRowsPass = kEpiBytes / kPitch;     // 256 (bf16) or 128 (f32)
    constexpr int kPasses = BM / kRowsPass;
    constexpr int kRowsInstr = 1024 / kPitch;         // rows per wave-wide 1 KB store
    constexpr int kInstr = kRowsPass / kRowsInstr / kWaves;
    typedef typename Quad<EB>::T QT;
    static_assert(kRowsPass % WM == 0 && kInstr * kRowsInstr * kWaves == kRowsPass, "epilogue plan");
#pragma unroll
    for (int h = 0; h < kPasses; ++h) {
        if (wm * WM / kRowsPass == h) {
#pragma unroll
            for (int j = 0; j < FA; ++j) {
                const int r = wm * WM + j * kFrag + lane % kFrag - h * kRowsPass;
#pragma unroll
                for (int i = 0; i < FB; ++i)
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const int grp = (wn * WN + i * kFrag + 8 * g) / 4 + lane / kFrag;
                        *reinterpret_cast<QT*>(lds + r * kPitch + (grp ^ (r & 31)) * 4 * EB) =
                            Quad<EB>::pack(acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2],
                                           acc[i][j][4 * g + 3]);
                    }
            }
        }
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
        for (int k = 0; k < kInstr; ++k) {
            const int r = (wave * kInstr + k) * kRowsInstr + lane / (kPitch / 16);
            const int q = lane % (kPitch / 16);  // 16-byte unit within the row
            u32x4_t v;
            if (EB == 4) {
                v = *reinterpret_cast<const u32x4_t*>(lds + r * kPitch + ((q ^ (r & 31)) * 16));
            } else {
                const int grp = (2 * q) ^ (r & 31);
                v = *reinterpret_cast<const u32x4_t*>(lds + r * kPitch + (grp >> 1) * 16);
                if (r & 1) v = u32x4_t{v[2], v[3], v[0], v[1]};
            }
            const int64_t row = h * kRowsPass + r, col = n0 + q * (16 / EB);
            const int off = row < rows_a && col < N ? (int)(row * N * EB + col * EB) : kDropped;
            __builtin_amdgcn_raw_buffer_store_b128(v, rc, off, 0, kStoreNT);
        }
        if (h + 1 < kPasses) asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    }
}

// Epilogue straight from the accumulators, element by element (rows of C
// that are not whole 16-byte units).
__device__ __forceinline__ void store_direct(const v16f (&acc)[FB][FA], Rsrc rc, int ct, int wm, int wn,
                                             int lane, int64_t rows_a, int64_t n0, int64_t N) {
    const int eb = ct == 1 ? 4 : 2;
#pragma unroll
    for (int j = 0; j < FA; ++j) {
        const int row = wm * WM + j * kFrag + lane % kFrag;
#pragma unroll
        for (int i = 0; i < FB; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int64_t col = n0 + wn * WN + i * kFrag + 8 * (r / 4) + 4 * (lane / kFrag) + r % 4;
                const int off = row < rows_a && col < N ? (int)((row * N + col) * eb) : kDropped;
                if (ct == 1)
                    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(acc[i][j][r]), rc, off, 0,
                                                          kStoreNT);
                else
                    __builtin_amdgcn_raw_buffer_store_b16((unsigned short)to_bf16(acc[i][j][r]), rc, off, 0,
                                                          kStoreNT);
            }
    }
}

}  // namespace
}  // namespace fp4q
