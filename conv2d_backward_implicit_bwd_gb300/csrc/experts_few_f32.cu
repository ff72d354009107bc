// experts_few_f32.cu -- fp32 expert products with few rows per expert:
//   y[i][n]  = sum_k x[i][k]  w[e][n][k]
//   dx[i][k] = sum_n dy[i][n] w[e][n][k]
//
// Every filter that has a row is read once and that read is the time, so the
// filters go straight to registers, 16 bytes a lane where the addresses allow it,
// and up to eight rows of an expert are multiplied with what a lane holds.
//
// forward: a warp takes four filter rows, its lanes go along k, and the lanes' sums
// are added by shuffles.  data: a block takes 128 (or 32) columns, a warp an eighth
// of n, and the warps' sums are added in shared memory in their order.
//
// Bound by memory at one row: 64 filters of 2048 x 1024 (537 MB, floor 80 us) 93 us
// forward, 80 data (on tiles of 64 x 64 200 and 172); then by the rows' reads from
// L1: 102 and 92 at four rows, 141 and 118 at eight.  Filters that pass by L1 leave
// the rows in it: 122 and 196 us forward otherwise.
#include <algorithm>

#include "expert_pieces.cuh"

namespace cbd {

namespace {

constexpr int NT = 256, WARPS = NT / 32;
constexpr int ROWS = 8;  // of an expert at a time
constexpr int NJ = 4;    // forward: filter rows of a warp
constexpr int UN = 8;    // data: filter rows in flight

template <int V>
struct Quad;
template <>
struct Quad<4> {
    float4 v;
    __device__ __forceinline__ void load(const float *p) { v = *reinterpret_cast<const float4 *>(p); }
    // of a filter: read once, and not to push the rows out of L1  (no read-only load: the launch begins while the kernel
    // before it, which may still write the filters, runs)
    __device__ __forceinline__ void pass(const float *p) {
        asm volatile("ld.global.L1::no_allocate.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p));
    }
    __device__ __forceinline__ float dot(const Quad &o, float s) const { return fmaf(v.w, o.v.w, fmaf(v.z, o.v.z, fmaf(v.y, o.v.y, fmaf(v.x, o.v.x, s)))); }
    __device__ __forceinline__ void add(float a, const Quad &o) {
        v.x = fmaf(a, o.v.x, v.x);
        v.y = fmaf(a, o.v.y, v.y);
        v.z = fmaf(a, o.v.z, v.z);
        v.w = fmaf(a, o.v.w, v.w);
    }
    __device__ __forceinline__ void store(float *p) const { *reinterpret_cast<float4 *>(p) = v; }
    __device__ __forceinline__ void zero() { v = make_float4(0.f, 0.f, 0.f, 0.f); }
};
template <>
struct Quad<1> {
    float v;
    __device__ __forceinline__ void load(const float *p) { v = *p; }
    __device__ __forceinline__ void pass(const float *p) { asm volatile("ld.global.L1::no_allocate.f32 %0, [%1];" : "=f"(v) : "l"(p)); }
    __device__ __forceinline__ float dot(const Quad &o, float s) const { return fmaf(v, o.v, s); }
    __device__ __forceinline__ void add(float a, const Quad &o) { v = fmaf(a, o.v, v); }
    __device__ __forceinline__ void store(float *p) const { *p = v; }
    __device__ __forceinline__ void zero() { v = 0.f; }
};

// One to R rows by up to NJ filter rows.  Rows past the last are the first again, and not stored: no load waits for a
// branch (with one, four rows took 237 us and eight 425 at 64 filters of 2048 x 1024).
template <int V, int R>
__device__ __forceinline__ void forward_rows(const ExpertSimtParams &p, const float *w, const float *x, float *out, int r, int nj) {
    const int lane = threadIdx.x % 32;
    const float *wj[NJ], *xi[R];
#pragma unroll
    for (int j = 0; j < NJ; ++j) wj[j] = w + (j < nj ? (int64_t)j * p.K : 0);
#pragma unroll
    for (int i = 0; i < R; ++i) xi[i] = x + (i < r ? i * p.lda : 0);
    float acc[NJ][R] = {};
    Quad<V> next[NJ];
    int k = lane * V;
    if (k < p.K) {
#pragma unroll
        for (int j = 0; j < NJ; ++j) next[j].pass(wj[j] + k);
    }
#pragma unroll 1
    for (; k < p.K; k += 32 * V) {
        Quad<V> cur[NJ], a[R];
#pragma unroll
        for (int j = 0; j < NJ; ++j) cur[j] = next[j];
#pragma unroll
        for (int i = 0; i < R; ++i) a[i].load(xi[i] + k);
        if (k + 32 * V < p.K) {
#pragma unroll
            for (int j = 0; j < NJ; ++j) next[j].pass(wj[j] + k + 32 * V);
        }
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int j = 0; j < NJ; ++j) acc[j][i] = cur[j].dot(a[i], acc[j][i]);
    }
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            float s = acc[j][i];
#pragma unroll
            for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
            if (lane == j && j < nj && i < r) out[i * p.ldo + j] = s;
        }
}

template <int V>
__global__ void __launch_bounds__(NT, 2) experts_few_forward_kernel(const __grid_constant__ ExpertSimtParams p) {
    __shared__ ExpertTable tab;
    __shared__ int32_t zero;
    const int nt = (p.N + NJ - 1) / NJ;
    if (threadIdx.x == 0) zero = 0;
    __syncthreads();
    pdl_next();
    if (threadIdx.x < 32)
        build_expert_table_early(tab, p.offsets, &zero, p.experts, p.rows, ROWS, nt, false, blockIdx.x == 0 ? p.status : nullptr);
    else
        pdl_wait();
    __syncthreads();
    const int total = tab.tile[p.experts];
    for (int t = blockIdx.x * WARPS + threadIdx.x / 32; t < total; t += gridDim.x * WARPS) {
        const int e = expert_of_tile(tab, p.experts, t), l = t - tab.tile[e], q = l / nt, n0 = (l - q * nt) * NJ;
        const int r = min(ROWS, tab.len(e) - q * ROWS), nj = min(NJ, p.N - n0);
        const int64_t row0 = tab.off[e] + q * ROWS;
        const float *w = static_cast<const float *>(p.b) + ((int64_t)e * p.N + n0) * p.K, *x = static_cast<const float *>(p.a) + row0 * p.lda;
        float *out = static_cast<float *>(p.out) + row0 * p.ldo + n0;
        if (r == 1)
            forward_rows<V, 1>(p, w, x, out, r, nj);
        else if (r <= 4)
            forward_rows<V, 4>(p, w, x, out, r, nj);
        else
            forward_rows<V, 8>(p, w, x, out, r, nj);
    }
    zero_free_rows<float>(p, tab, p.N);
}

// One to R rows of dy by the filter rows [n, end) of a warp, V columns a lane.
template <int V, int R>
__device__ __forceinline__ void data_rows(const ExpertSimtParams &p, const float *w, const float *dy, float *part, int r, int n, int end) {
    Quad<V> acc[R];
    const float *di[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        acc[i].zero();
        di[i] = dy + (i < r ? i * p.lda : 0);
    }
#pragma unroll 1
    for (; n + UN <= end; n += UN) {
        Quad<V> f[UN];
        __align__(16) float d[R][UN];
#pragma unroll
        for (int u = 0; u < UN; ++u) f[u].pass(w + (int64_t)(n + u) * p.K);
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int u = 0; u < UN; u += V) reinterpret_cast<Quad<V> *>(&d[i][u])->load(di[i] + n + u);
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int u = 0; u < UN; ++u) acc[i].add(d[i][u], f[u]);
    }
    for (; n < end; ++n) {
        Quad<V> f;
        f.pass(w + (int64_t)n * p.K);
#pragma unroll
        for (int i = 0; i < R; ++i) acc[i].add(di[i][n], f);
    }
#pragma unroll
    for (int i = 0; i < R; ++i)
        if (i < r) acc[i].store(part + i * 32 * V);
}

template <int V>
__global__ void __launch_bounds__(NT, 2) experts_few_data_kernel(const __grid_constant__ ExpertSimtParams p) {
    constexpr int W = 32 * V;  // columns
    __shared__ ExpertTable tab;
    __shared__ __align__(16) float part[WARPS][ROWS][W];
    __shared__ int32_t zero;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, kt = (p.K + W - 1) / W;
    if (threadIdx.x == 0) zero = 0;
    __syncthreads();
    pdl_next();
    if (threadIdx.x < 32)
        build_expert_table_early(tab, p.offsets, &zero, p.experts, p.rows, ROWS, kt, false, blockIdx.x == 0 ? p.status : nullptr);
    else
        pdl_wait();
    __syncthreads();
    const int total = tab.tile[p.experts], chunk = ((p.N + WARPS - 1) / WARPS + UN - 1) / UN * UN;
    const int n_lo = min(p.N, warp * chunk), n_hi = min(p.N, n_lo + chunk);
    for (int t = blockIdx.x; t < total; t += gridDim.x) {
        const int e = expert_of_tile(tab, p.experts, t), l = t - tab.tile[e], q = l / kt, k0 = (l - q * kt) * W;
        const int r = min(ROWS, tab.len(e) - q * ROWS), k = k0 + lane * V;
        const int64_t row0 = tab.off[e] + q * ROWS;
        const float *w = static_cast<const float *>(p.b) + (int64_t)e * p.N * p.K + k, *dy = static_cast<const float *>(p.a) + row0 * p.lda;
        float *mine = &part[warp][0][lane * V];
        if (k < p.K) {
            if (r == 1)
                data_rows<V, 1>(p, w, dy, mine, r, n_lo, n_hi);
            else if (r <= 4)
                data_rows<V, 4>(p, w, dy, mine, r, n_lo, n_hi);
            else
                data_rows<V, 8>(p, w, dy, mine, r, n_lo, n_hi);
        }
        __syncthreads();
        float *out = static_cast<float *>(p.out) + row0 * p.ldo + k0;
        for (int s = threadIdx.x; s < r * W; s += NT) {
            const int i = s / W, c = s - i * W;
            float sum = 0.f;
#pragma unroll
            for (int v = 0; v < WARPS; ++v) sum += part[v][i][c];
            if (k0 + c < p.K) out[i * p.ldo + c] = sum;
        }
        __syncthreads();
    }
    zero_free_rows<float>(p, tab, p.K);
}

}  // namespace

cudaError_t launch_experts_few_f32(const ExpertSimtParams &p, int dir, int num_sms, cudaStream_t s) {
    const bool quads = (((uintptr_t)p.a | (uintptr_t)p.b) & 15) == 0 && (p.K | p.lda) % 4 == 0 && (dir == kExpForward || p.N % 4 == 0);
    const int64_t groups = std::min<int64_t>(p.rows, (int64_t)p.rows / ROWS + p.experts);  // most of up to eight rows
    if (dir == kExpForward) {
        const int64_t blocks = (groups * ((p.N + NJ - 1) / NJ) + WARPS - 1) / WARPS;
        const int grid = (int)std::max<int64_t>(1, std::min<int64_t>(blocks, 2 * num_sms));
        return quads ? launch_early(experts_few_forward_kernel<4>, grid, NT, 0, s, p) : launch_early(experts_few_forward_kernel<1>, grid, NT, 0, s, p);
    }
    // (32 columns a block where 128 would leave SMs without one)
    const bool wide = quads && groups * ((p.K + 127) / 128) >= num_sms;
    const int64_t blocks = groups * ((p.K + (wide ? 127 : 31)) / (wide ? 128 : 32));
    const int grid = (int)std::max<int64_t>(1, std::min<int64_t>(blocks, 2 * num_sms));
    return wide ? launch_early(experts_few_data_kernel<4>, grid, NT, 0, s, p) : launch_early(experts_few_data_kernel<1>, grid, NT, 0, s, p);
}

}  // namespace cbd
