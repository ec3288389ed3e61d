// Internal interface between the C ABI layer (fp4q_abi.cpp) and the kernel
// launchers (fp4q_kernels.hip).  Plain types only; arguments arrive here
// already validated.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace fp4q {

// Workspace layout (bytes from the start of ws).  Every slot is written before
// it is read within one call, so the workspace needs no initial contents.
constexpr int kMaxGroups = 16384;           // upper bound on any grid size
constexpr size_t kWsAmax = 0;               // uint32 per-workgroup |x| maxima
// Per-workgroup error terms, one array per term (structure of arrays):
// [non-max | max | zero-rounding | sum x^2] as double, then the zero-block count.
constexpr size_t kWsPartials = kWsAmax + 4 * (size_t)kMaxGroups;
// sum x^2 per workgroup of the amax pre-pass (dynamic mode), as double
constexpr size_t kWsAmaxSumsq = kWsPartials + 5 * 8 * (size_t)kMaxGroups;
constexpr size_t kWsBytes = kWsAmaxSumsq + 8 * (size_t)kMaxGroups;

struct QuantJob {
    const void* x;
    int xt;            // 0 bf16, 1 f32
    int64_t n;         // rows * cols
    int64_t rows, cols;
    int block;         // 8..256
    int fmt;           // 0 MXFP4, 1 UE4M3, 2 UE5M3
    int gmode;         // 0 none, 1 dynamic, 2 given, 3 per row
    float* g;          // device: dynamic out / given in / one per row out
    int rotate;        // 0, 16, 32
    uint8_t* codes;
    uint8_t* scales;
    float* block_mse;  // nullable
    int mse_kind;      // 0 abs, 1 rel
    void* stats;       // nullable, fp4q_stats layout
    void* ws;
    void* stream;
    int radius = -1;   // >= 0: per-block scale search over this many neighbours
    // MXFP4 pass of fp4_quantize_mx_nv: the quantize kernel also writes its
    // per-workgroup max |x| (binary32 bits) to amax_out, and the reduction
    // kernel turns them into the NVFP4 per-tensor scale at g_from_amax.
    uint32_t* amax_out = nullptr;
    float* g_from_amax = nullptr;
    // NVFP4 pass of fp4_quantize_mx_nv: stores with the nontemporal bit.
    bool nv_of_pair = false;
};

struct DequantJob {
    const uint8_t* codes;
    const uint8_t* scales;
    int fmt;
    int block;
    const float* g;    // nullable (UE4M3)
    int64_t n;
    int rotate;
    void* out;
    int ot;            // 0 bf16, 1 f32
    void* stream;
};

struct MseJob {
    const void* x;
    int xt;
    const uint8_t* codes;
    const uint8_t* scales;
    int fmt;
    int block;
    const float* g;    // nullable (UE4M3)
    int64_t n;
    int rotate;
    float* block_mse;
    int mse_kind;
    void* stats;
    void* ws;
    void* stream;
};

struct RotateJob {
    const void* x;
    int xt;
    int64_t n;
    int rotate;
    float* out;
    void* stream;
};

struct GemmJob {
    const uint8_t* a_codes;
    const uint8_t* a_scales;
    const uint8_t* b_codes;
    const uint8_t* b_scales;
    int64_t M, N, K;
    void* c;
    int ct;            // 0 bf16, 1 f32
    void* ws;          // gemm_workspace_bytes(M, N, K) bytes: packed scales
    void* stream;
};

size_t gemm_workspace_bytes(int64_t M, int64_t N, int64_t K);

struct GemmNvJob {
    const uint8_t* a_codes;
    const uint8_t* a_scales;  // UE4M3 per 16 elements
    const uint8_t* b_codes;
    const uint8_t* b_scales;
    const float* ga;          // per-tensor scales (device), nullable
    const float* gb;
    int64_t M, N, K;
    void* c;
    int ct;                   // 0 bf16, 1 f32
    void* ws;                 // gemm_nvfp4_workspace_bytes(M, N, K) bytes: partials
    void* stream;
};

size_t gemm_nvfp4_workspace_bytes(int64_t M, int64_t N, int64_t K);

// E4M3 codes with a binary32 scale per 128 elements of a row (tile false) or per
// 128 x 128 (tile true); codes or codes_t may be NULL.
struct Fp8QuantJob {
    const void* x;
    int xt;            // 0 bf16, 1 f32
    int64_t rows, cols;
    bool tile;
    uint8_t* codes;
    float* scales;
    uint8_t* codes_t;
    float* scales_t;
    void* stream;
};

// Product of two such operands; b_row: B has row scales (else tile scales).
struct Fp8GemmJob {
    const uint8_t* a_codes;
    const float* a_scales;
    const uint8_t* b_codes;
    const float* b_scales;
    bool b_row;
    int64_t M, N, K;
    void* c;
    int ct;            // 0 bf16, 1 f32
    void* ws;          // fp8_gemm_workspace_bytes(M, N, K, ct) bytes: partial products
    void* stream;
};

size_t fp8_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K, int ct);

// Rows in groups: group e owns rows offsets[e] .. offsets[e + 1] - 1 (device, groups + 1 of them).
// Row scales; the transpose holds fp8_group_blocks() blocks of 128 columns, each group's own from a
// whole block on: codes_t cols x (128 blocks), scales_t blocks x cols.
struct Fp8GroupQuantJob {
    const void* x;
    int xt;            // 0 bf16, 1 f32
    int64_t rows, cols;
    const int* offsets;
    int64_t groups;
    uint8_t* codes;    // nullable, as codes_t
    float* scales;     // ceil(cols / 128) x rows
    uint8_t* codes_t;
    float* scales_t;
    void* stream;
};
// Blocks that the groups take at most.
int64_t fp8_group_blocks(int64_t rows, int64_t groups);

// One matrix per expert, tile scales of each: codes (experts x rows) x ld, codes_t experts x cols x
// ld_t (nullable), scales and scales_t alike.
struct Fp8ExpertQuantJob {
    const void* w;
    int wt;            // 0 bf16, 1 f32
    int64_t experts, rows, cols;
    uint8_t* codes;
    float* scales;
    uint8_t* codes_t;
    float* scales_t;
    void* stream;
};

// A product per group of A's rows with its expert's matrix: C[i] = A[tokens[i]] W_e^T.
struct GroupedGemmJob {
    const uint8_t* a_codes;
    const float* a_scales;   // ceil(K / 128) x a_rows
    int64_t a_rows;
    const uint8_t* b_codes;  // (experts x N) x K
    const float* b_scales;
    bool stacked;            // tile scales of the stacked matrix; else of each expert's
    const int* offsets;
    int64_t experts;
    const int* tokens;       // nullable: row i of C is row i of A
    int64_t rows, N, K;
    void* c;
    int ct;                  // 0 bf16, 1 f32
    bool clear_rest;         // rows of no group: zeros, else left as they are
    int64_t chosen_by;       // groups that a kernel is chosen for
    void* stream;
};

// A weight gradient per group: dW_e = At_e Bt_e^T over the group's blocks of transposed operands
// as Fp8GroupQuantJob writes them.
struct GroupedOuterJob {
    const uint8_t* a_codes;  // M x (128 blocks)
    const float* a_scales;   // blocks x M
    const uint8_t* b_codes;  // N x (128 blocks)
    const float* b_scales;
    const int* offsets;
    int64_t experts, rows, M, N;
    void* c;                 // experts x M x N
    int ct;
    void* stream;
};

// The slots of a routing by expert.
struct ExpertOrderJob {
    const void* ids;   // tokens x top_k
    bool wide;         // int64 (else int32)
    int64_t tokens, top_k, experts;
    int* offsets;      // experts + 1
    int* order;        // slot of each sorted row
    int* token;        // its token
    int* position;     // sorted row of each slot
    void* ws;          // expert_order_workspace_bytes() bytes
    void* stream;
};
size_t expert_order_workspace_bytes(int64_t slots, int64_t experts);

// 8-bit integers with a binary32 scale per row.
struct Int8QuantJob {
    const void* x;
    int xt;            // 0 bf16, 1 f32
    int64_t rows, cols;
    int8_t* codes;
    float* scales;
    void* stream;
};

// Product of two such operands, with a bias per column.
struct Int8GemmJob {
    const int8_t* a_codes;
    const float* a_scales;
    const int8_t* b_codes;
    const float* b_scales;
    const void* bias;  // nullable
    int bt;            // 0 bf16, 1 f32
    int64_t M, N, K;
    void* c;
    int ct;            // 0 bf16, 1 f32
    void* ws;          // int8_gemm_workspace_bytes(M, N, K) bytes: sums of K ranges
    void* stream;
    // Where int8_linear_in_one(M, N, K): A's values (M x cols, K = cols rounded up to 16) in the place
    // of a_codes and a_scales.
    int xt = -1;       // 0 bf16, 1 f32; -1: A is given as codes
    const void* x = nullptr;
    int64_t cols = 0;
};

size_t int8_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K);
// Whether a product of unquantized A takes one launch: one row, and few rows of B.
bool int8_linear_in_one(int64_t M, int64_t N, int64_t K);

// Mixture-of-experts layer for a few tokens.
struct MoeWeights {
    const uint8_t* codes;  // (E * rows) x K
    const void* scales;
    const float* g;        // nullable (1)
    bool g_per_expert;
};
struct MoeJob {
    const void* x;
    int xt;                // 0 bf16, 1 f32
    int64_t T, D, I, E, k;
    int fmt;               // 0 MXFP4, 1 UE4M3 block 16, 2 E4M3 block 128
    MoeWeights w13, w2;
    const void* router;    // nullable: ids and wts are given
    int rt;
    int renorm;
    int* ids;
    float* wts;
    void* y;
    int yt;
    void* ws;              // moe_workspace_bytes(...) bytes, its first 256 zero
    void* stream;
};

constexpr int64_t kMoeMaxTokens = 64, kMoeMaxExperts = 512, kMoeMaxTopK = 16, kMoeMaxSize = 1 << 20;
size_t moe_workspace_bytes(int64_t T, int64_t D, int64_t I, int64_t E, int64_t k);

// Launch timing (fp4q_profile_events): while the calling thread has event
// pairs left, every kernel launch records the next pair on its stream around
// itself.  Streams and events are passed as void*.
void profile_set(void* const* events, int n_pairs);
int profile_count();
void profile_before(void* stream);
void profile_after(void* stream);

// A kernel launch bracketed by the timing hooks (used for every launch).
#define FP4Q_LAUNCH(kernel, grid, block, shmem, stream, ...)                       \
    do {                                                                           \
        ::fp4q::profile_before(stream);                                            \
        hipLaunchKernelGGL(kernel, grid, block, shmem, stream, __VA_ARGS__);       \
        ::fp4q::profile_after(stream);                                             \
    } while (0)

// A grid holds fewer than 2^32 threads: more workgroups (of up to 512 threads) than this go out
// in several launches, each told its first one.  (A second grid dimension needs a test for the
// workgroups past the last, which cost small products 3%.)
constexpr int64_t kMaxGrid = 1 << 22;

// The library's static device scratch for the allocation-free entry point:
// its device address on the current device (looked up once per device) and
// its size (kWsBytes).  Returns 0, else a HIP error code with `msg` set.
int scratch_workspace(void** ptr, size_t* bytes, char* msg, size_t msg_len);

// Each returns 0 on success, else a HIP error code; `msg` gets a description.
int launch_quantize(const QuantJob& j, char* msg, size_t msg_len);
// MXFP4 (mx) then dynamic NVFP4 (nv) of the same unrotated tensor, the NVFP4
// per-tensor scale taken from the MXFP4 pass's maxima (no amax pass).
int launch_quantize_mx_nv(const QuantJob& mx, const QuantJob& nv, char* msg, size_t msg_len);
// The same for n <= kMaxBatchTensors tensors in one launch per pass: mx[i] and
// nv[i] describe tensor i (same dtype, NVFP4 block 16 or 32, and the same
// outputs wanted for every tensor); one reduction launch per pass.
constexpr int kMaxBatchTensors = 16;
int launch_quantize_mx_nv_batch(const QuantJob* mx, const QuantJob* nv, int n, char* msg,
                                size_t msg_len);
int launch_dequantize(const DequantJob& j, char* msg, size_t msg_len);
int launch_block_mse(const MseJob& j, char* msg, size_t msg_len);
int launch_rotate(const RotateJob& j, char* msg, size_t msg_len);
int launch_gemm(const GemmJob& j, char* msg, size_t msg_len);
int launch_gemm_nvfp4(const GemmNvJob& j, char* msg, size_t msg_len);
int launch_fp8_quantize(const Fp8QuantJob& j, char* msg, size_t msg_len);
// x under row scales and w under tile scales: one launch where both outputs of both are wanted.
int launch_fp8_quantize_two(const Fp8QuantJob& x, const Fp8QuantJob& w, char* msg, size_t msg_len);
int launch_fp8_gemm(const Fp8GemmJob& j, char* msg, size_t msg_len);
int launch_fp8_quantize_groups(const Fp8GroupQuantJob& j, char* msg, size_t msg_len);
int launch_fp8_quantize_experts(const Fp8ExpertQuantJob& j, char* msg, size_t msg_len);
// Both: one launch where all outputs of both are wanted.
int launch_fp8_quantize_grouped(const Fp8GroupQuantJob& x, const Fp8ExpertQuantJob& w, char* msg, size_t msg_len);
int launch_grouped_gemm(const GroupedGemmJob& j, char* msg, size_t msg_len);
int launch_grouped_outer(const GroupedOuterJob& j, char* msg, size_t msg_len);
int launch_expert_order(const ExpertOrderJob& j, char* msg, size_t msg_len);
int launch_int8_quantize(const Int8QuantJob& j, char* msg, size_t msg_len);
int launch_int8_gemm(const Int8GemmJob& j, char* msg, size_t msg_len);
int launch_moe(const MoeJob& j, char* msg, size_t msg_len);

// Adds the binary32 partial products of `splits` K ranges (splits x count, range
// by range) in binary64 and writes c (ct: 0 bf16, 1 f32); partial and c are
// device pointers, the stream a hipStream_t.
void launch_splitk_reduce(const float* partial, int splits, int64_t count, void* c, int ct, void* stream);

}  // namespace fp4q
