// train.h -- types shared by the C ABI and the kernels of the training-step
// operators (include/conv_bwd_train.h).
#pragma once
#include <stdint.h>
#include <cuda.h>
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

}  // namespace cbd
