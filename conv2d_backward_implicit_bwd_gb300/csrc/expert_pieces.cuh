// expert_pieces.cuh -- what the expert products on plain loads share (fp32, and
// bf16 that TMA cannot load): the schedule and the join of split tiles.
//
// Expert e owns rows [offsets[e], offsets[e+1]) and filter w[e] [N][K]:
//   forward  y[i][n]     = sum_k x[i][k]  w[e][n][k]
//   data     dx[i][k]    = sum_n dy[i][n] w[e][n][k]
//   weight   dw[e][n][k] (+)= sum_{i in e} dy[i][n] x[i][k]
// as C[i][j] = sum_l A[i][l] B[j][l] over square tiles.  Where the tiles are fewer
// than the SMs, a tile's contraction is cut in chunks ("pieces") of their own
// blocks: each writes its fp32 sums to the workspace, and the last of a tile to
// arrive adds them in the order of the chunks and stores.  No block waits for
// another, and the order of every sum follows from the sizes alone.
#pragma once
#include <cuda_bf16.h>

#include "expert_table.cuh"

namespace cbd {

template <int DIR, int BT>
struct ExpertPieces {
    int n_tiles, m_tiles, splits;  // column tiles, row tiles (weight), pieces of a tile (forward, data)
    __device__ __forceinline__ explicit ExpertPieces(const ExpertSimtParams &p)
        : n_tiles(((DIR == kExpForward ? p.N : p.K) + BT - 1) / BT), m_tiles((p.N + BT - 1) / BT),
          splits((int)(((uint32_t)(DIR == kExpForward ? p.K : p.N) + (uint32_t)p.chunk - 1) / (uint32_t)p.chunk)) {}
    __device__ __forceinline__ void build(ExpertTable &tab, const int32_t *zero, const ExpertSimtParams &p) const {
        constexpr bool W = DIR == kExpWeight;
        build_expert_table_early(tab, p.offsets, zero, p.experts, p.rows, W ? (uint32_t)p.chunk : BT, n_tiles * (W ? m_tiles : splits),
                                 W && !p.accumulate, blockIdx.x == 0 ? p.status : nullptr);
    }
};

// Piece t: its tile, operands and part of the contraction.
template <int DIR, int BT, typename T>
struct ExpertPiece {
    int e, nb, i_lim, j_lim;   // expert; column tile; valid rows and columns
    int part, parts;           // which of how many pieces of the tile
    int depth;                 // of this piece
    int64_t row;               // first row of the output: of the tensor, or of the filter (weight)
    const T *a, *b;            // the piece's first elements
    int64_t stride_a, stride_b;  // of the index that is not contiguous
    __device__ __forceinline__ ExpertPiece(const ExpertSimtParams &p, const ExpertTable &tab, const ExpertPieces<DIR, BT> &ps, int t) {
        e = expert_of_tile(tab, p.experts, t);
        const int64_t r0 = tab.off[e];
        const int len = tab.len(e), l = t - tab.tile[e], whole = DIR == kExpForward ? p.K : DIR == kExpData ? p.N : len;
        parts = DIR == kExpWeight ? max(1, (int)(((uint32_t)len + (uint32_t)p.chunk - 1) / (uint32_t)p.chunk)) : ps.splits;
        const int tile = l / parts;
        part = l - tile * parts;
        const int mb = tile / ps.n_tiles;
        nb = tile - mb * ps.n_tiles;
        const int64_t l0 = (int64_t)part * p.chunk;
        depth = (int)min((int64_t)p.chunk, (int64_t)whole - l0);
        i_lim = min(BT, (DIR == kExpWeight ? p.N : len) - mb * BT);
        j_lim = min(BT, (DIR == kExpForward ? p.N : p.K) - nb * BT);
        const T *A = static_cast<const T *>(p.a), *B = static_cast<const T *>(p.b);
        stride_a = p.lda;
        if constexpr (DIR == kExpWeight) {
            row = (int64_t)e * p.N + (int64_t)mb * BT;
            a = A + (r0 + l0) * p.lda + (int64_t)mb * BT;
            b = B + (r0 + l0) * p.ldb + (int64_t)nb * BT;
            stride_b = p.ldb;
        } else {
            row = r0 + (int64_t)mb * BT;
            a = A + row * p.lda + l0;
            b = B + (int64_t)e * p.N * p.K + (DIR == kExpForward ? (int64_t)nb * BT * p.K + l0 : l0 * p.K + (int64_t)nb * BT);
            stride_b = p.K;
        }
    }
};

// All threads of a block, V sums of each: true in the block that holds the whole sum.
template <int V, int NT, typename P>
__device__ __forceinline__ bool join_parts(float (&v)[V], const ExpertSimtParams &p, const P &w, int t, volatile int32_t *flag) {
    static_assert(V % 4 == 0 && V * NT == 64 * 64, "a piece's place in the workspace");
    float4 *mine = reinterpret_cast<float4 *>(p.parts) + (int64_t)t * (V / 4 * NT) + threadIdx.x;
#pragma unroll
    for (int q = 0; q < V / 4; ++q) __stcg(mine + q * NT, make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]));
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
        int32_t *count = p.arrived + (t - w.part);
        const bool last = atomicAdd(count, 1) == w.parts - 1;
        if (last) *count = 0;
        *flag = last;
        __threadfence();
    }
    __syncthreads();
    const bool last = *flag;
    __syncthreads();  // the flag is written again
    if (!last) return false;
    __threadfence();
#pragma unroll
    for (int q = 0; q < V; ++q) v[q] = 0.f;
    mine -= (int64_t)w.part * (V / 4 * NT);
    for (int c = 0; c < w.parts; ++c, mine += V / 4 * NT) {
        float4 x[V / 4];
#pragma unroll
        for (int q = 0; q < V / 4; ++q) x[q] = __ldcg(mine + q * NT);
#pragma unroll
        for (int q = 0; q < V / 4; ++q) {
            v[4 * q] += x[q].x;
            v[4 * q + 1] += x[q].y;
            v[4 * q + 2] += x[q].z;
            v[4 * q + 3] += x[q].w;
        }
    }
    return true;
}

// forward, data: rows of no expert get zeros
template <typename O>
__device__ __forceinline__ void zero_free_rows(const ExpertSimtParams &p, const ExpertTable &tab, int cols) {
    const int lo = tab.off[0], hi = tab.off[p.experts];
    const int64_t nfill = (int64_t)lo + (p.rows - hi);
    for (int64_t f = blockIdx.x; f < nfill; f += gridDim.x) {
        O *row = static_cast<O *>(p.out) + (f < lo ? f : hi + (f - lo)) * p.ldo;
        for (int c = threadIdx.x; c < cols; c += blockDim.x) row[c] = O(0.f);
    }
}

}  // namespace cbd
