// train.h -- types shared by the C ABI and the kernels of the training-step
// operators (include/conv_bwd_train.h).
#pragma once
#include <stdint.h>
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace cbd {

// Launch that may begin while the kernel before it in the stream still runs: the
// kernel sets itself up (barriers, tensor memory) and then waits in pdl_wait()
// before it touches global memory.
template <typename... P, typename... A>
inline cudaError_t launch_early(void (*kernel)(P...), int grid, int block, size_t smem, cudaStream_t s, const A &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}
#ifdef __CUDACC__
// every thread: the kernels before this one are done and their writes visible
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// the next kernel may set itself up
__device__ __forceinline__ void pdl_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
#endif

constexpr int kMaxExperts = 1024;  // the expert tables of a launch live in shared memory

enum : int { kExpForward = 0, kExpData = 1, kExpWeight = 2 };

// Expert product on CUDA cores (any sizes, strides and alignment).
constexpr int kMaxRows = 0x7fffffff;
struct ExpertSimtParams {
    const void *a;           // x (forward), dy (data, weight)
    const void *b;           // w (forward, data), x (weight)
    const void *a_end, *b_end;
    void *out;               // y, dx or dw
    const int32_t *offsets;  // [experts + 1]
    int32_t *status;
    int64_t lda, ldb, ldo;   // row strides of the row-sorted tensors (ldb: weight only; ldo: forward, data)
    int32_t experts, rows, K, N;
    int32_t accumulate;
    int32_t wide;            // 1: tiles of 128 x 128, else 64 x 64
    int32_t chunk;           // contraction indices of a piece (kMaxRows: a tile is not split)
    int32_t grid;
    float *parts;            // 64 x 64 sums of each piece of split tiles
    int32_t *arrived;        // their counters
};
// most pieces of a launch with split tiles, for an SM
constexpr int kSimtPieces = 2;
cudaError_t launch_experts_few_f32(const ExpertSimtParams &p, int dir, int num_sms, cudaStream_t s);
cudaError_t launch_experts_f32(const ExpertSimtParams &p, int dir, cudaStream_t s);
cudaError_t launch_experts_b16(const ExpertSimtParams &p, int dir, cudaStream_t s);

// Expert product on tensor cores over pairs of SMs (bf16; filters or their gradients on 16 bytes, rows at any address).
struct ExpertPairParams {  // 128-byte aligned through CUtensorMap
    CUtensorMap a;           // forward, data: w {K, N, experts}; weight: dy {N, rows}
    CUtensorMap b;           // forward: x {K, rows}; data: dy {N, rows}; weight: x {K, rows}
    CUtensorMap o;           // weight: dw {K, N, experts} in fp32
    void *out;               // forward, data: y, dx
    const int32_t *offsets;
    int32_t *status;
    int64_t wait_budget;
    int64_t ldo;
    int32_t experts, rows, K, N;
    int32_t accumulate;
    int32_t out_lines;       // forward, data: the output rows take 16-byte stores
    // where TMA cannot load the rows (else null): x (forward) or dy, its end and row stride
    const void *rows_at, *rows_end;
    int64_t ldb;
    const void *rows2_at, *rows2_end;  // weight: x
    int64_t ldb2;
};
cudaError_t launch_experts_pair(const ExpertPairParams &p, int dir, int grid, cudaStream_t s);

// Expert product for few rows per expert (bf16, forward and data).
struct ExpertStreamParams {
    CUtensorMap a;  // w {K, N, experts}
    CUtensorMap b;  // x {K, rows} or dy {N, rows}
    void *out;
    const int32_t *offsets;
    int32_t *status;
    float *parts;      // [blocks][2][kStreamRows][128] parts of tiles that several blocks share
    int32_t *arrived;  // [blocks] arrivals of the tile that starts in a block and ends in another, 0 between launches
    int32_t *drawn;    // counter of the tiles that blocks drew, 0 between launches
    int64_t wait_budget, ldo;
    int32_t experts, rows, K, N;
};
constexpr int kStreamRows = 16;  // most rows of a tile
cudaError_t launch_experts_stream(const ExpertStreamParams &p, int dir, int grid, cudaStream_t s);

// Gradient clipping: the tensors are cut into chunks of kClipChunk bytes.
constexpr int kClipChunk = 32768;
constexpr int kNormBlocks = 3, kScaleBlocks = 2;  // blocks per SM
constexpr int kClipPtrs = 1000;  // tensors per launch (their pointers travel as kernel parameters)
struct __align__(16) ClipChunk {
    int64_t start;   // first element
    int32_t n;       // elements
    int16_t tensor;  // index within the launch's pointer table
    int16_t bf16;
};
struct ClipParams {
    const ClipChunk *chunks;  // of this launch's tensors; at least one entry
    double *partials;        // one per block of every norm launch
    uint32_t *ticket, *turn;
    int32_t *status;
    int64_t wait_budget;
    float *norm, *coef;
    int32_t num_chunks;
    int32_t partial_base;    // first partial of this launch
    int32_t partial_total;   // partials of all launches (the last launch sums them), 0: not the last
    int32_t want_coef;
    float max_norm;
};
// `g` and `o` (NULL for the norm): the launch's `tensors` pointers, on the host
cudaError_t launch_clip_norm(const ClipParams &p, const void *const *g, int tensors, int grid, cudaStream_t s);
cudaError_t launch_clip_scale(const ClipParams &p, const void *const *g, void *const *o, int tensors, int grid, cudaStream_t s);
// norm and scaling in one launch of num_chunks blocks, at most clip_fused_blocks
int clip_fused_blocks(int num_sms);
cudaError_t launch_clip_fused(const ClipParams &p, const void *const *g, void *const *o, int tensors, cudaStream_t s);

// Policy loss.
enum : int { kPolForward = 0, kPolBackward = 1, kPolBoth = 2 };
struct PolicyParams {
    const void *logits;
    void *dlogits;
    const int32_t *actions;
    const float *advantage, *weight, *old_logp, *ref_logp;
    const float *lse_in, *coef_in, *grad;  // backward
    float *loss, *logp, *lse, *coef;       // forward (lse and coef NULL in the fused form)
    double *partials;                      // one per block
    uint32_t *ticket;
    int32_t *status;
    int64_t ld, ldd;
    int64_t wait_budget;
    int32_t tokens, vocab;
    float clip_lo, clip_hi, kl, scale;     // clamp bounds 1 - clip_low, 1 + clip_high
};
int policy_max_blocks(int num_sms);        // upper bound of any launch's blocks
cudaError_t launch_policy(const PolicyParams &p, int dtype, int mode, int num_sms, cudaStream_t s);

// Log-probabilities of given tokens, entropy, alternatives.
constexpr int kLogpTop = 32;     // most alternatives of a row
constexpr int kLogpPart = 272;   // bytes of a row's part in the workspace
struct LogpParams {
    const void *logits;
    void *dlogits;
    const int32_t *tokens;                               // NULL: no given tokens
    float *logp, *entropy, *lse, *top_logp;              // forward
    int32_t *top_tokens;
    const float *lse_in, *entropy_in, *grad_logp, *grad_entropy;  // backward
    void *work;                                          // [rows][parts] parts
    int32_t *arrived;                                    // [rows] parts that are there, 0 between launches
    int32_t *status;
    int64_t ld, ldd;
    int64_t wait_budget;
    int32_t rows, vocab, top, parts;
    float scale;
};
int logp_most_items(int num_sms);  // upper bound of rows * parts where parts > 1
int logp_parts(int64_t rows, int64_t vocab, int dtype, int num_sms);
cudaError_t launch_logp(const LogpParams &p, int dtype, bool backward, int num_sms, cudaStream_t s);

// Orthogonalised updates.
struct OrthPrepParams {
    const void *grad;        // [batch] matrices, `ls` elements apart, rows `ld` apart
    float *momentum;         // dense, or NULL
    __half *hi, *lo;         // [batch][rows][pitch]
    double *partial;         // [batch][parts][2]: SquareSum's two
    int32_t *done;           // [batch], cleared
    int64_t ls, ld;
    int32_t batch, rows, cols, pitch, parts, bf16, nesterov;
    float beta;
};
cudaError_t launch_orth_prep(const OrthPrepParams &p, cudaStream_t s);
// All the products, as a list of phases over the plan's matrices: 0 and 1 hold X in turn, the others are symmetric.
constexpr int kOrthMostSteps = 64, kOrthJoined = 3;  // kOrthJoined: steps of one polynomial
constexpr int kOrthMostPhases = 240;                 // of 64 steps: 11 for three joined, 3 for one
constexpr int kOrthMatrices = 8;
constexpr int kOrthSplits = 3;  // most pieces of a tile's contraction
constexpr float kOrthUp = 1024.f, kOrthUpPoly = 256.f;  // what the planes' values are multiplied by
enum : int8_t { kOrthGram = 0, kOrthSquare = 1, kOrthProduct = 2 };  // over the larger side; of symmetric matrices; X's
struct OrthPhase {
    int32_t first, need;           // its first item; warps that have finished with a matrix before
    int8_t kind, a, b, out;
    int8_t poly, last;             // mul a b + add a + diag; the result
    float mul, add, diag;
};
struct OrthMaps {
    CUtensorMap rows128[2], rows64[2], store[2];  // of planes hi and lo: boxes of 128 and 64 rows, of a warp's 32
};
struct OrthParams {
    OrthMaps maps[kOrthMatrices];
    const __half *at[kOrthMatrices][2];
    void *result;                  // the result, or the step on the weights
    float *weight;
    __nv_bfloat16 *copy;
    float4 *parts;                 // sums of tiles whose contraction is split
    int32_t *arrived;              // their counters, 0 between tiles
    int32_t *done;                 // [batch] warps that have finished a tile
    int32_t *status;
    int64_t wait_budget;
    int64_t ldo, lse;              // of the caller's tensors: rows, matrices
    int32_t rows, cols, batch, matrices, phases;
    int32_t tiles_sym, tiles_all;  // tiles of a matrix: symmetric, X
    int32_t splits[3];             // by kind
    int32_t own_tiles, own_pieces; // split tiles and their pieces: the most that a matrix has of one kind
    int32_t segment;               // k-blocks of one accumulator
    int32_t bf16, pitch_gram;
    float rate, keep;
    OrthPhase phase[kOrthMostPhases + 1];  // and the end
};
// The places of a split tile's counters and of its pieces' sums.  A matrix has its own: one may be in another product than the
// next, and a place has another tile in every kind of product.
__host__ __device__ inline int orth_counter_place(const OrthParams &p, int e, int tile) { return e * p.own_tiles + tile; }
__host__ __device__ inline int orth_piece_place(const OrthParams &p, int e, int tile, int splits) { return e * p.own_pieces + tile * splits; }
int orth_pairs(int num_sms);
// Matrices whose smaller side is at most kOrthSmall, their larger side in `cluster` slices of `slice` columns.
constexpr int kOrthSmall = 128, kOrthSlice = 256;
struct OrthSmallParams {
    const void *grad;
    float *momentum;
    void *result;
    float *weight;
    __nv_bfloat16 *copy;
    int32_t *status;
    int64_t wait_budget;
    int64_t ls, ld, lse, ldo;      // of the input, of the result
    int32_t rows, cols, batch, steps, cluster, slice;
    int32_t bf16, nesterov;        // bf16: of the input and the result
    float beta, rate, keep;
    float coef[3 * kOrthMostSteps];
};
cudaError_t launch_orth_small(const OrthSmallParams &p, cudaStream_t s);
#ifdef __CUDACC__
// A sum of squares: of those far from both ends of fp32 in fp32, of the others in fp64 (a conversion and an addition of fp64
// for every element would take longer than the memory).  What an addition in fp32 leaves goes into the next one: a thread may
// add 2^16 numbers (2^34 elements by 304 blocks), equal ones with errors that all point one way.
struct SquareSum {
    float safe, lost;
    double rest;
    template <int N>
    __device__ __forceinline__ void add(const float (&x)[N]) {
        float q = 0.f;
#pragma unroll
        for (int j = 0; j < N; ++j) q = fmaf(x[j], x[j], q);
        if (q > 0x1p-60f && q < 0x1p100f) {
            const float y = q - lost, t = safe + y;
            lost = (t - safe) - y;
            safe = t;
        } else {
#pragma unroll 1
            for (int j = 0; j < N; ++j) {
                float y = x[0];
#pragma unroll
                for (int l = 1; l < N; ++l) y = l == j ? x[l] : y;
                if (y != 0.f) rest += (double)y * (double)y;
            }
        }
    }
    // over the lanes of a warp
    __device__ __forceinline__ void join() {
#pragma unroll
        for (int d = 16; d; d >>= 1) safe += __shfl_xor_sync(0xffffffffu, safe, d);
        if (__any_sync(0xffffffffu, rest != 0.0)) {
#pragma unroll
            for (int d = 16; d; d >>= 1) rest += __shfl_xor_sync(0xffffffffu, rest, d);
        }
    }
};
// 2^10 / sqrt(sum of squares) in three factors that neither overflow nor underflow (the norm is anywhere from 2^-149 on):
// zeros for a matrix of zeros, NaN where the norm is not finite.  (Exponent and mantissa by hand, the root in fp32 with one
// step of Newton, good to 2^-23: in fp64 it took some thousand clocks, which in a small matrix everyone waits for.)
__device__ __forceinline__ void orth_factors(const SquareSum &s, float &f0, float &f1, float &f2) {
    int x;
    float m;  // sum = m 2^x, m in [1, 4), x even
    if (s.rest == 0.0 && s.safe > 0x1p-100f && s.safe < 0x1p120f) {
        const int bits = __float_as_int(s.safe);
        x = (bits >> 23) - 127;
        x -= x & 1;
        m = __int_as_float(bits - (x << 23));
    } else {
        const double sum = (double)s.safe + s.rest;
        if (!(sum > 0.0) || sum > 1e300) {
            f0 = f1 = f2 = sum == 0.0 ? 0.f : __int_as_float(0x7fffffff);
            return;
        }
        const long long bits = __double_as_longlong(sum);
        x = (int)(bits >> 52) - 1023;  // (squares of fp32 numbers are normal fp64 numbers)
        x -= x & 1;
        m = (float)__longlong_as_double(bits - ((long long)x << 52));
    }
    float r = rsqrtf(m);
    r = r * fmaf(-0.5f * m * r, r, 1.5f);
    const int k = 10 - x / 2, h = k / 2;
    f0 = __int_as_float((127 + h) << 23);
    f1 = __int_as_float((127 + k - h) << 23);
    f2 = r;
}
#endif
// wide: tiles of 256 x 256, else 256 x 128
cudaError_t launch_orth_steps(const OrthParams &p, bool wide, int pairs, cudaStream_t s);

}  // namespace cbd
