// experts_b16.cu -- matrix products grouped by expert for bf16 tensors that TMA
// cannot load: widths, strides or addresses that are no multiple of 16 bytes.
//
// The loads are the time here: single elements, or two where the addresses allow
// it.  So the matrix instruction is the warp-level m16n8k16 on shared memory that
// ordinary stores fill, 256 threads for a tile of 128 x 128 or 64 x 64 in slices of
// 32, two slices of loads in registers ahead.  Each operand stays as it lies in
// memory, contraction or tile index contiguous, and ldmatrix turns it where needed.
//
// Bound by the loads' instructions: 8192 rows by 8 filters of 1028 x 1028 (pairs)
// 112 us forward, 85 us data, 124 us weight; of 1001 x 1001 (single elements) 158,
// 122 and 215 us (fp32 FMAs on the same loads 545 to 660 us).
//
// weight adds its accumulators to fp32 registers every 512 rows, as the tensor
// core's own sums truncate.
#include <type_traits>

#include "expert_pieces.cuh"

namespace cbd {

namespace {

constexpr int NT = 256, BL = 32;
constexpr int SEGMENT = 512 / BL;

template <bool L_CONTIG, int BT>
struct Slab {  // [BT][BL] or [BL][BT], rows padded to odd multiples of 16 bytes
    static constexpr int LD = L_CONTIG ? BL + 8 : BT + 8, BYTES = (L_CONTIG ? BT : BL) * LD * 2;
};

// BT x 32 elements of an operand, two neighbours to a register; zeros past i_lim and `left`.
template <bool L_CONTIG, int BT>
__device__ __forceinline__ void fetch(uint32_t (&r)[BT / 16], const uint16_t *src, int64_t stride, int i_lim, int left, bool pairs) {
    constexpr int W = L_CONTIG ? BL / 2 : BT / 2, STEP = NT / W;
    const int u = (int)threadIdx.x % W * 2, v = (int)threadIdx.x / W;
    const int along = L_CONTIG ? left : i_lim, across = L_CONTIG ? i_lim : left;
    const uint16_t *at = src + v * stride + u;
    if (pairs && u + 1 < along) {
#pragma unroll
        for (int q = 0; q < BT / 16; ++q, at += STEP * stride)
            r[q] = v + q * STEP < across ? *reinterpret_cast<const uint32_t *>(at) : 0u;
    } else {
#pragma unroll
        for (int q = 0; q < BT / 16; ++q, at += STEP * stride) {
            const bool ok = v + q * STEP < across;
            const uint32_t lo = ok && u < along ? at[0] : 0u, hi = ok && u + 1 < along ? at[1] : 0u;
            r[q] = lo | hi << 16;
        }
    }
}
template <bool L_CONTIG, int BT>
__device__ __forceinline__ void park(uint8_t *s, const uint32_t (&r)[BT / 16]) {
    constexpr int W = L_CONTIG ? BL / 2 : BT / 2, STEP = NT / W;
    uint8_t *at = s + ((int)threadIdx.x / W * Slab<L_CONTIG, BT>::LD + (int)threadIdx.x % W * 2) * 2;
#pragma unroll
    for (int q = 0; q < BT / 16; ++q) *reinterpret_cast<uint32_t *>(at + q * STEP * Slab<L_CONTIG, BT>::LD * 2) = r[q];
}
// four 8 x 8 blocks of (tile index, contraction) at (i, l): (0, 0), (8, 0), (0, 8), (8, 8), or with SWAP the middle two
// exchanged
template <bool L_CONTIG, int BT, bool SWAP>
__device__ __forceinline__ void ld4(uint32_t (&r)[4], uint32_t s, int i, int l) {
    const int lane = threadIdx.x % 32, b = lane / 8;
    const int di = SWAP ? b / 2 : b % 2, dl = SWAP ? b % 2 : b / 2;
    if constexpr (L_CONTIG) {
        const uint32_t at = s + (uint32_t)((i + di * 8 + lane % 8) * Slab<L_CONTIG, BT>::LD + l + dl * 8) * 2;
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
    } else {
        const uint32_t at = s + (uint32_t)((l + dl * 8 + lane % 8) * Slab<L_CONTIG, BT>::LD + i + di * 8) * 2;
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
    }
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void put2(__nv_bfloat16 *at, float x, float y, bool second, bool) {
    if (second && (reinterpret_cast<uintptr_t>(at) & 3) == 0) {
        *reinterpret_cast<__nv_bfloat162 *>(at) = __floats2bfloat162_rn(x, y);
    } else {
        at[0] = __float2bfloat16_rn(x);
        if (second) at[1] = __float2bfloat16_rn(y);
    }
}
__device__ __forceinline__ void put2(float *at, float x, float y, bool second, bool add) {
    at[0] = add ? at[0] + x : x;
    if (second) at[1] = add ? at[1] + y : y;
}

template <int DIR, int BT>
__global__ void __launch_bounds__(NT, BT == 128 && DIR == kExpWeight ? 1 : 2) experts_b16_kernel(const __grid_constant__ ExpertSimtParams p) {
    constexpr bool A_L = DIR != kExpWeight;   // A's contraction index is contiguous
    constexpr bool B_L = DIR == kExpForward;  // B's
    constexpr int A_BYTES = Slab<A_L, BT>::BYTES, B_BYTES = Slab<B_L, BT>::BYTES;
    constexpr int T = BT / 32;  // a warp's tiles of 16 rows and of 8 columns: BT / 2 x BT / 4
    typedef typename std::conditional<DIR == kExpWeight, float, __nv_bfloat16>::type O;
    __shared__ ExpertTable tab;
    extern __shared__ __align__(16) uint8_t slabs[];
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
    const int total = tab.tile[p.experts], lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int wi = warp / 4 * (BT / 2), wj = warp % 4 * (BT / 4);

    for (int t = blockIdx.x; t < total; t += gridDim.x) {
        const ExpertPiece<DIR, BT, uint16_t> w(p, tab, ps, t);
        const int slices = (w.depth + BL - 1) / BL;
        const bool pairs_a = (reinterpret_cast<uintptr_t>(w.a) & 3) == 0 && w.stride_a % 2 == 0;
        const bool pairs_b = (reinterpret_cast<uintptr_t>(w.b) & 3) == 0 && w.stride_b % 2 == 0;
        uint32_t ra[2][BT / 16], rb[2][BT / 16];
        float acc[T][T][4] = {}, sum[DIR == kExpWeight ? T * T * 4 : 1] = {};
        auto load = [&](int k, uint32_t (&a)[BT / 16], uint32_t (&b)[BT / 16]) {
            if (k >= slices) return;
            const int64_t l = (int64_t)k * BL;
            fetch<A_L, BT>(a, w.a + (A_L ? l : l * w.stride_a), w.stride_a, w.i_lim, w.depth - k * BL, pairs_a);
            fetch<B_L, BT>(b, w.b + (B_L ? l : l * w.stride_b), w.stride_b, w.j_lim, w.depth - k * BL, pairs_b);
        };
        auto step = [&](int k, int h) {
            uint8_t *s = slabs + h * (A_BYTES + B_BYTES);
            park<A_L, BT>(s, ra[h]);
            park<B_L, BT>(s + A_BYTES, rb[h]);
            load(k + 2, ra[h], rb[h]);
            // (this slab is written again after the next slice's barrier, which follows every read of it)
            __syncthreads();
            const uint32_t sa = smem_u32(s), sb = smem_u32(s + A_BYTES);
#pragma unroll
            for (int l = 0; l < BL; l += 16) {
                uint32_t a[T][4], b[T / 2][4];
#pragma unroll
                for (int i = 0; i < T; ++i) ld4<A_L, BT, false>(a[i], sa, wi + i * 16, l);
#pragma unroll
                for (int j = 0; j < T / 2; ++j) ld4<B_L, BT, true>(b[j], sb, wj + j * 16, l);
#pragma unroll
                for (int i = 0; i < T; ++i)
#pragma unroll
                    for (int j = 0; j < T; ++j) mma(acc[i][j], a[i], b[j / 2][j % 2 * 2], b[j / 2][j % 2 * 2 + 1]);
            }
        };
        auto flush = [&] {
            if constexpr (DIR == kExpWeight) {
#pragma unroll
                for (int q = 0; q < T * T * 4; ++q) {
                    sum[q] += (&acc[0][0][0])[q];
                    (&acc[0][0][0])[q] = 0.f;
                }
            }
        };
        load(0, ra[0], rb[0]);
        load(1, ra[1], rb[1]);
        __syncthreads();  // the slabs are free
#pragma unroll 1
        for (int k = 0; k < slices; k += 2) {
            if (DIR == kExpWeight && k % SEGMENT == 0) flush();
            step(k, 0);
            if (k + 1 < slices) step(k + 1, 1);
        }
        flush();
        float v[T * T * 4];
#pragma unroll
        for (int q = 0; q < T * T * 4; ++q) v[q] = DIR == kExpWeight ? sum[DIR == kExpWeight ? q : 0] : (&acc[0][0][0])[q];
        if constexpr (BT == 64) {
            if (w.parts > 1 && !join_parts<T * T * 4, NT>(v, p, w, t, &flag)) continue;
        }
        const int64_t ldo = DIR == kExpWeight ? (int64_t)p.K : p.ldo;
        O *out = static_cast<O *>(p.out) + w.row * ldo + (int64_t)w.nb * BT;
#pragma unroll
        for (int i = 0; i < T; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = wi + i * 16 + h * 8 + lane / 4;
                if (r >= w.i_lim) continue;
#pragma unroll
                for (int j = 0; j < T; ++j) {
                    const int c = wj + j * 8 + lane % 4 * 2;
                    if (c < w.j_lim) put2(out + r * ldo + c, v[(i * T + j) * 4 + 2 * h], v[(i * T + j) * 4 + 2 * h + 1], c + 1 < w.j_lim, p.accumulate);
                }
            }
    }
    if constexpr (DIR != kExpWeight) zero_free_rows<__nv_bfloat16>(p, tab, DIR == kExpForward ? p.N : p.K);
}

template <int DIR, int BT>
cudaError_t launch_one(const ExpertSimtParams &p, cudaStream_t s) {
    constexpr int SMEM = 2 * (Slab<DIR != kExpWeight, BT>::BYTES + Slab<DIR == kExpForward, BT>::BYTES);
    static bool attr_set[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !attr_set[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(experts_b16_kernel<DIR, BT>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) attr_set[dev] = true;
    }
    return launch_early(experts_b16_kernel<DIR, BT>, p.grid, NT, SMEM, s, p);
}
template <int DIR>
cudaError_t launch_dir(const ExpertSimtParams &p, cudaStream_t s) {
    return p.wide ? launch_one<DIR, 128>(p, s) : launch_one<DIR, 64>(p, s);
}

}  // namespace

cudaError_t launch_experts_b16(const ExpertSimtParams &p, int dir, cudaStream_t s) {
    return dir == kExpForward ? launch_dir<kExpForward>(p, s) : dir == kExpData ? launch_dir<kExpData>(p, s) : launch_dir<kExpWeight>(p, s);
}

}  // namespace cbd
