// experts_simt.cu -- matrix products grouped by expert on CUDA cores, for
// fp32 tensors and for bf16 tensors whose sizes, strides or alignment the
// tensor-core kernels cannot load.
//
// Expert e owns rows [offsets[e], offsets[e+1]) and filter w[e] [N][K]:
//   forward  y[i][n]     = sum_k x[i][k]  w[e][n][k]
//   data     dx[i][k]    = sum_n dy[i][n] w[e][n][k]
//   weight   dw[e][n][k] (+)= sum_{i in e} dy[i][n] x[i][k]
// as C[i][j] = sum_l A[i][l] B[j][l] over tiles of 64 x 64 with l in slices of
// 16: 256 threads of 4 x 4 outputs, the next slice in registers while the
// current one is multiplied.  Each output is summed in fp32 in the order of
// l, so results do not depend on the schedule.
#include <cuda_bf16.h>

#include "expert_table.cuh"

namespace cbd {

namespace {

constexpr int BT = 64, BL = 16, NT = 256;

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void put(float *p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

// 64 x 16 elements of an operand: element (i, l) at src[i * si + l * sl], with
// the unit stride known at compile time so that neighbouring threads read
// neighbouring elements.
template <typename T, bool L_CONTIG>
__device__ __forceinline__ void fetch(float (&v)[4], const T *src, int64_t stride, int i_lim, int64_t l0, int64_t l_lim) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int i = L_CONTIG ? (int)threadIdx.x / 16 + 16 * q : (int)threadIdx.x % 64;
        const int64_t l = l0 + (L_CONTIG ? (int)threadIdx.x % 16 : (int)threadIdx.x / 64 + 4 * q);
        v[q] = (i < i_lim && l < l_lim) ? to_f32(L_CONTIG ? src[i * stride + l] : src[l * stride + i]) : 0.f;
    }
}
template <bool L_CONTIG>
__device__ __forceinline__ void park(float (*s)[BT + 4], const float (&v)[4]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int i = L_CONTIG ? (int)threadIdx.x / 16 + 16 * q : (int)threadIdx.x % 64;
        const int l = L_CONTIG ? (int)threadIdx.x % 16 : (int)threadIdx.x / 64 + 4 * q;
        s[l][i] = v[q];
    }
}

template <typename T, typename O, int DIR>
__global__ void __launch_bounds__(NT) experts_simt_kernel(const ExpertSimtParams p) {
    constexpr bool A_L = DIR != kExpWeight;   // A's contraction index is contiguous
    constexpr bool B_L = DIR == kExpForward;  // B's
    __shared__ ExpertTable tab;
    __shared__ __align__(16) float sa[BL][BT + 4];  // read as float4: rows of 17 x 16 bytes
    __shared__ __align__(16) float sb[BL][BT + 4];
    const int cols = DIR == kExpForward ? p.N : p.K;
    const int n_tiles = (cols + BT - 1) / BT, m_tiles = (p.N + BT - 1) / BT;  // m_tiles: weight only
    pdl_next();
    pdl_wait();
    if (threadIdx.x < 32)
        build_expert_table<BT>(tab, p.offsets, p.experts, p.rows, DIR == kExpWeight ? m_tiles * n_tiles : n_tiles,
                               DIR != kExpWeight ? kTilesByRows : p.accumulate ? kTilesNonEmpty : kTilesEach,
                               blockIdx.x == 0 ? p.status : nullptr);
    __syncthreads();
    const int total = tab.tile[p.experts];
    const T *A = static_cast<const T *>(p.a), *B = static_cast<const T *>(p.b);
    O *out = static_cast<O *>(p.out);
    const int ti = (threadIdx.x / 16) * 4, tj = (threadIdx.x % 16) * 4;

    for (int t = blockIdx.x; t < total; t += gridDim.x) {
        const int e = expert_of_tile(tab, p.experts, t), mb = (t - tab.tile[e]) / n_tiles, nb = (t - tab.tile[e]) % n_tiles;
        const int64_t r0 = tab.off[e], len = tab.len(e);
        const int64_t L = DIR == kExpForward ? p.K : DIR == kExpData ? p.N : len;
        const int i_lim = (int)min((int64_t)BT, (DIR == kExpWeight ? (int64_t)p.N : len) - (int64_t)mb * BT);
        const int j_lim = min(BT, cols - nb * BT);
        const T *a, *b;
        int64_t sa_, sb_;
        if constexpr (DIR == kExpWeight) {
            a = A + r0 * p.lda + (int64_t)mb * BT;
            b = B + r0 * p.ldb + (int64_t)nb * BT;
            sa_ = p.lda;
            sb_ = p.ldb;
        } else {
            a = A + (r0 + (int64_t)mb * BT) * p.lda;
            sa_ = p.lda;
            b = B + (int64_t)e * p.N * p.K + (DIR == kExpForward ? (int64_t)nb * BT * p.K : (int64_t)nb * BT);
            sb_ = p.K;
        }
        float acc[4][4] = {};
        float va[4], vb[4];
        fetch<T, A_L>(va, a, sa_, i_lim, 0, L);
        fetch<T, B_L>(vb, b, sb_, j_lim, 0, L);
        for (int64_t l0 = 0; l0 < L; l0 += BL) {
            __syncthreads();
            park<A_L>(sa, va);
            park<B_L>(sb, vb);
            __syncthreads();
            if (l0 + BL < L) {
                fetch<T, A_L>(va, a, sa_, i_lim, l0 + BL, L);
                fetch<T, B_L>(vb, b, sb_, j_lim, l0 + BL, L);
            }
#pragma unroll
            for (int l = 0; l < BL; ++l) {
                const float4 x = *reinterpret_cast<const float4 *>(&sa[l][ti]), y = *reinterpret_cast<const float4 *>(&sb[l][tj]);
                const float xa[4] = {x.x, x.y, x.z, x.w}, yb[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(xa[i], yb[j], acc[i][j]);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (ti + i >= i_lim) break;
            O *row;
            if constexpr (DIR == kExpWeight)
                row = out + ((int64_t)e * p.N + (int64_t)mb * BT + ti + i) * p.K + (int64_t)nb * BT;
            else
                row = out + (r0 + (int64_t)mb * BT + ti + i) * p.ldo + (int64_t)nb * BT;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (tj + j < j_lim) {
                    float v = acc[i][j];
                    if (DIR == kExpWeight && p.accumulate) v += to_f32(row[tj + j]);
                    put(row + tj + j, v);
                }
        }
    }

    if constexpr (DIR != kExpWeight) {
        const int lo = tab.off[0], hi = tab.off[p.experts];
        const int64_t nfill = (int64_t)lo + (p.rows - hi);
        for (int64_t f = blockIdx.x; f < nfill; f += gridDim.x) {
            O *row = out + (f < lo ? f : hi + (f - lo)) * p.ldo;
            for (int c = threadIdx.x; c < cols; c += NT) put(row + c, 0.f);
        }
    }
}

template <typename T>
cudaError_t launch_dir(const ExpertSimtParams &p, int dir, int grid, cudaStream_t s) {
    if (dir == kExpForward) return launch_early(experts_simt_kernel<T, T, kExpForward>, grid, NT, 0, s, p);
    if (dir == kExpData) return launch_early(experts_simt_kernel<T, T, kExpData>, grid, NT, 0, s, p);
    return launch_early(experts_simt_kernel<T, float, kExpWeight>, grid, NT, 0, s, p);
}

}  // namespace

cudaError_t launch_experts_simt(const ExpertSimtParams &p, int dtype, int dir, int num_sms, cudaStream_t s) {
    const int64_t nt = ((dir == kExpForward ? p.N : p.K) + BT - 1) / BT;
    const int64_t most = dir == kExpWeight ? (int64_t)p.experts * ((p.N + BT - 1) / BT) * nt
                                           : ((int64_t)p.rows / BT + p.experts) * nt + 1;
    const int grid = (int)(most < (int64_t)num_sms * 6 ? (most > 0 ? most : 1) : (int64_t)num_sms * 6);
    return dtype == 1 ? launch_dir<__nv_bfloat16>(p, dir, grid, s) : launch_dir<float>(p, dir, grid, s);
}

}  // namespace cbd
