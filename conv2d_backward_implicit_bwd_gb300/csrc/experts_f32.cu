// experts_f32.cu -- matrix products grouped by expert in fp32 on CUDA cores.
//
// 256 threads hold a tile of 128 x 128 (8 x 8 sums each) or 64 x 64 (4 x 4); the
// operands come through four stages of shared memory with 4-byte asynchronous
// copies, which take any alignment and turn a row-major operand around on the way.
// Two products an instruction (fma.f32x2): the sums of two neighbouring columns.
// Each output is summed in fp32 in the order of the contraction.
//
// Bound by the FMA pipe and the instructions around it: 8192 rows by 8 filters of
// 1001 x 1001 381 us (43 TFLOP/s; single FMAs 416 us, A stored twice to save the
// broadcasts 544 us, one block of 255 registers an SM 409 us).  Small products wait
// on latency: 1500 rows as one expert, weight of 100 x 100, 10 us (unsplit 71 us).
#include "expert_pieces.cuh"

namespace cbd {

namespace {

constexpr int NT = 256, ST = 4;

// BT x BL elements of an operand: element (i, l) at src[i * stride + l], or at src[l * stride + i], to s[l][i];
// zeros past `left`; what lies past i_lim only reaches sums that nobody stores (narrow tiles leave it as it was).  `quads`: four neighbours at a time (the latter layout, on 16 bytes).
template <bool L_CONTIG, int BT, int BL>
__device__ __forceinline__ void copy(float *s, const float *src, int64_t stride, int i_lim, int left, bool quads) {
    if (!L_CONTIG && quads) {
        constexpr int W = BT / 4, STEP = NT / W;
        const int u = (int)threadIdx.x % W * 4, v = (int)threadIdx.x / W, bytes = max(0, min(4, i_lim - u)) * 4;
        const float *at = src + v * stride + u;
        uint32_t dst = smem_u32(s + v * (BT + 4) + u);
#pragma unroll
        for (int q = 0; q < BL / STEP; ++q) {
            const bool ok = v + q * STEP < left && bytes;
            if (BT == 128 || bytes) asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(ok ? at : src), "r"(ok ? bytes : 0) : "memory");
            at += STEP * stride;
            dst += STEP * (BT + 4) * 4;
        }
        return;
    }
    constexpr int Q = BT * BL / NT, W = L_CONTIG ? BL : BT, STEP = NT / W;
    const int u = (int)threadIdx.x % W, v = (int)threadIdx.x / W;
    const float *at = src + v * stride + u;
    uint32_t dst = smem_u32(s + (L_CONTIG ? u * (BT + 4) + v : v * (BT + 4) + u));
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        const int x = v + q * STEP;
        const bool in = (L_CONTIG ? x : u) < i_lim, ok = in && (L_CONTIG ? u : x) < left;
        if (BT == 128 || in) asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(ok ? at : src), "r"(ok ? 4 : 0) : "memory");
        at += STEP * stride;
        dst += L_CONTIG ? STEP * 4 : STEP * (BT + 4) * 4;
    }
}
__device__ __forceinline__ uint64_t both(float x) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ void fma2(uint64_t &d, uint64_t a, uint64_t b) { asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(d) : "l"(a), "l"(b)); }

template <int BT>
struct Cfg {
    static constexpr int BL = BT == 128 ? 16 : 32, LD = BT + 4, SMEM = ST * 2 * BL * LD * 4;
};

template <int DIR, int BT>
__global__ void __launch_bounds__(NT, 2) experts_f32_kernel(const __grid_constant__ ExpertSimtParams p) {
    constexpr bool A_L = DIR != kExpWeight;   // A's contraction index is contiguous
    constexpr bool B_L = DIR == kExpForward;  // B's
    constexpr int BL = Cfg<BT>::BL, LD = Cfg<BT>::LD, M = BT / 16, G = M / 4;
    extern __shared__ __align__(16) float stages[];
    __shared__ ExpertTable tab;
    __shared__ int32_t flag;
    const ExpertPieces<DIR, BT> ps(p);
    if (threadIdx.x == 0) flag = 0;
    __syncthreads();
    pdl_next();
    if (threadIdx.x < 32)
        ps.build(tab, &flag, p);
    else
        pdl_wait();
    __syncthreads();
    const int total = tab.tile[p.experts];
    const int ti = (threadIdx.x / 16) * 4, tj = (threadIdx.x % 16) * 4;

    for (int t = blockIdx.x; t < total; t += gridDim.x) {
        const ExpertPiece<DIR, BT, float> w(p, tab, ps, t);
        const int slices = (w.depth + BL - 1) / BL;
        const bool quads_a = !A_L && ((reinterpret_cast<uintptr_t>(w.a) | (uintptr_t)w.stride_a * 4) & 15) == 0;
        const bool quads_b = !B_L && ((reinterpret_cast<uintptr_t>(w.b) | (uintptr_t)w.stride_b * 4) & 15) == 0;
        const bool busy = BT == 128 || (int)threadIdx.x / 32 * 8 < w.i_lim;  // any of this warp's 8 rows
        auto issue = [&](int k) {
            if (k < slices) {
                float *s = stages + (k % ST) * (2 * BL * LD);
                const int64_t l = (int64_t)k * BL;
                copy<A_L, BT, BL>(s, w.a + (A_L ? l : l * w.stride_a), w.stride_a, w.i_lim, w.depth - k * BL, quads_a);
                copy<B_L, BT, BL>(s + BL * LD, w.b + (B_L ? l : l * w.stride_b), w.stride_b, w.j_lim, w.depth - k * BL, quads_b);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        uint64_t acc[M][M / 2];  // rows ti + 64 g + 0..3, columns tj + 64 g + 0..3
#pragma unroll
        for (int i = 0; i < M; ++i)
#pragma unroll
            for (int j = 0; j < M / 2; ++j) acc[i][j] = 0;
        __syncthreads();  // the stages are free
#pragma unroll
        for (int k = 0; k < ST - 1; ++k) issue(k);
#pragma unroll 1
        for (int k = 0; k < slices; ++k) {
            asm volatile("cp.async.wait_group %0;" ::"n"(ST - 2) : "memory");
            __syncthreads();
            issue(k + ST - 1);
            if (!busy) continue;
            const float *sa = stages + (k % ST) * (2 * BL * LD) + ti, *sb = stages + (k % ST) * (2 * BL * LD) + BL * LD + tj;
#pragma unroll
            for (int l = 0; l < BL; ++l) {
                float4 a[G];
                ulonglong2 b[G];
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    a[g] = *reinterpret_cast<const float4 *>(sa + l * LD + 64 * g);
                    b[g] = *reinterpret_cast<const ulonglong2 *>(sb + l * LD + 64 * g);
                }
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    const uint64_t x[4] = {both(a[g].x), both(a[g].y), both(a[g].z), both(a[g].w)};
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int h = 0; h < G; ++h) {
                            fma2(acc[4 * g + i][2 * h], x[i], b[h].x);
                            fma2(acc[4 * g + i][2 * h + 1], x[i], b[h].y);
                        }
                }
            }
        }
        float v[M * M];
#pragma unroll
        for (int i = 0; i < M; ++i)
#pragma unroll
            for (int j = 0; j < M / 2; ++j) asm("mov.b64 {%0, %1}, %2;" : "=f"(v[i * M + 2 * j]), "=f"(v[i * M + 2 * j + 1]) : "l"(acc[i][j]));
        if constexpr (BT == 64) {
            if (w.parts > 1 && !join_parts<M * M, NT>(v, p, w, t, &flag)) continue;
        }
        float *out = static_cast<float *>(p.out) + w.row * (DIR == kExpWeight ? p.K : p.ldo) + (int64_t)w.nb * BT;
#pragma unroll
        for (int i = 0; i < M; ++i) {
            const int r = (i / 4) * 64 + ti + i % 4;
            if (r >= w.i_lim) break;
            float *row = out + r * (DIR == kExpWeight ? (int64_t)p.K : p.ldo);
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const int c = g * 64 + tj;
                float4 x = make_float4(v[i * M + 4 * g], v[i * M + 4 * g + 1], v[i * M + 4 * g + 2], v[i * M + 4 * g + 3]);
                if (c + 3 < w.j_lim && (reinterpret_cast<uintptr_t>(row + c) & 15) == 0) {
                    float4 *at = reinterpret_cast<float4 *>(row + c);
                    if (DIR == kExpWeight && p.accumulate) {
                        const float4 o = *at;
                        x = make_float4(x.x + o.x, x.y + o.y, x.z + o.z, x.w + o.w);
                    }
                    *at = x;
                } else {
                    const float y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (c + j < w.j_lim) row[c + j] = DIR == kExpWeight && p.accumulate ? row[c + j] + y[j] : y[j];
                }
            }
        }
    }
    if constexpr (DIR != kExpWeight) zero_free_rows<float>(p, tab, DIR == kExpForward ? p.N : p.K);
}

template <int DIR, int BT>
cudaError_t launch_one(const ExpertSimtParams &p, cudaStream_t s) {
    static bool attr_set[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !attr_set[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(experts_f32_kernel<DIR, BT>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<BT>::SMEM);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) attr_set[dev] = true;
    }
    return launch_early(experts_f32_kernel<DIR, BT>, p.grid, NT, Cfg<BT>::SMEM, s, p);
}
template <int DIR>
cudaError_t launch_dir(const ExpertSimtParams &p, cudaStream_t s) {
    return p.wide ? launch_one<DIR, 128>(p, s) : launch_one<DIR, 64>(p, s);
}

}  // namespace

cudaError_t launch_experts_f32(const ExpertSimtParams &p, int dir, cudaStream_t s) {
    return dir == kExpForward ? launch_dir<kExpForward>(p, s) : dir == kExpData ? launch_dir<kExpData>(p, s) : launch_dir<kExpWeight>(p, s);
}

}  // namespace cbd
