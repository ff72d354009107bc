// experts_b16.cu -- matrix products grouped by expert for bf16 tensors whose widths,
// filters or filter gradients are no multiple of 16 bytes (TMA cannot move those).
//
// The loads are the time here: single elements, two where the addresses allow it, or
// (weight) 16-byte lines that are shifted into place.  So the matrix instruction is the warp-level m16n8k16 on shared memory that
// ordinary stores fill, 256 threads for a tile of 128 x 128 or 64 x 64 in slices of
// 32, two slices of loads in registers ahead.  Each operand stays as it lies in
// memory, contraction or tile index contiguous, and ldmatrix turns it where needed.
//
// Bound by the loads' instructions: 8192 rows by 8 filters of 1028 x 1028 (pairs)
// 112 us forward, 85 us data, 124 us weight; of 1001 x 1001 (single elements, lines)
// 158, 122 and 157 us (fp32 FMAs on the same loads 545 to 660 us).
//
// weight adds its accumulators to fp32 registers every 512 rows, as the tensor
// core's own sums truncate.
#include <type_traits>

#include "expert_pieces.cuh"
#include "lines.cuh"

namespace cbd {

namespace {

constexpr int NT = 256, BL = 32;
constexpr int SEGMENT = 512 / BL;

template <bool L_CONTIG, int BT>
struct Slab {  // [BT][BL] or [BL][BT], rows padded to odd multiples of 16 bytes
    static constexpr int LD = L_CONTIG ? BL + 8 : BT + 8, BYTES = (L_CONTIG ? BT : BL) * LD * 2;
};

// BT x 32 elements of an operand on their way to shared memory; zeros past `left`, anything past i_lim.
template <bool L_CONTIG, int BT, bool LINES>
struct Slice;

// Two neighbours to a register, read one by one or, on 4-byte addresses, together.
template <bool L_CONTIG, int BT>
struct Slice<L_CONTIG, BT, false> {
    uint32_t r[BT / 16];
    static constexpr int W = L_CONTIG ? BL / 2 : BT / 2, STEP = NT / W;
    __device__ __forceinline__ void fetch(const uint16_t *src, int64_t stride, int i_lim, int left, const void *, const void *) {
        const int u = (int)threadIdx.x % W * 2, v = (int)threadIdx.x / W;
        const int along = L_CONTIG ? left : i_lim, across = L_CONTIG ? i_lim : left;
        const bool words = (reinterpret_cast<uintptr_t>(src) & 3) == 0 && stride % 2 == 0;
        const uint16_t *at = src + v * stride + u;
        if (words && u + 1 < along) {
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
    __device__ __forceinline__ void park(uint8_t *s) const {
        uint8_t *at = s + ((int)threadIdx.x / W * Slab<L_CONTIG, BT>::LD + (int)threadIdx.x % W * 2) * 2;
#pragma unroll
        for (int q = 0; q < BT / 16; ++q) *reinterpret_cast<uint32_t *>(at + q * STEP * Slab<L_CONTIG, BT>::LD * 2) = r[q];
    }
};

// Tile index contiguous: a 16-byte line of a row to a thread, shifted with its neighbour's (the row's last thread reads the
// line after its own as well).
template <int BT>
struct Slice<false, BT, true> {
    static constexpr int W = BT / 8, STEP = NT / W, Q = BL / STEP;
    uint4 line[Q], after[Q];
    int shift[Q];
    __device__ __forceinline__ void fetch(const uint16_t *src, int64_t stride, int i_lim, int left, const void *begin_, const void *end_) {
        const uintptr_t begin = reinterpret_cast<uintptr_t>(begin_), end = reinterpret_cast<uintptr_t>(end_);
        const int c = (int)threadIdx.x % W, v = (int)threadIdx.x / W;
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const int l = v + q * STEP;
            const uintptr_t row = reinterpret_cast<uintptr_t>(src + l * stride);
            const int s = (int)(row & 15) / 2;
            shift[q] = s;
            const uintptr_t at = row - 2 * s + 16 * c;
            line[q] = after[q] = make_uint4(0u, 0u, 0u, 0u);
            if (l < left && 8 * c - s < i_lim) line[q] = load_line(at, begin, end);
            if (l < left && c == W - 1 && s && 8 * W - s < i_lim) after[q] = load_line(at + 16, begin, end);
        }
    }
    __device__ __forceinline__ void park(uint8_t *sm) const {
        const int c = (int)threadIdx.x % W, v = (int)threadIdx.x / W;
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            uint4 hi;
            hi.x = __shfl_down_sync(0xffffffffu, line[q].x, 1);
            hi.y = __shfl_down_sync(0xffffffffu, line[q].y, 1);
            hi.z = __shfl_down_sync(0xffffffffu, line[q].z, 1);
            hi.w = __shfl_down_sync(0xffffffffu, line[q].w, 1);
            if (c == W - 1) hi = after[q];
            *reinterpret_cast<uint4 *>(sm + ((v + q * STEP) * Slab<false, BT>::LD + c * 8) * 2) = shifted(line[q], hi, shift[q]);
        }
    }
};
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

template <int DIR, int BT, bool LINES>
__global__ void __launch_bounds__(NT, BT == 128 && DIR == kExpWeight ? 1 : 2) experts_b16_kernel(const __grid_constant__ ExpertSimtParams p) {
    constexpr bool A_L = DIR != kExpWeight;   // A's contraction index is contiguous
    constexpr bool B_L = DIR == kExpForward;  // B's
    static_assert(!LINES || DIR == kExpWeight, "lines for operands whose tile index is contiguous");
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
        Slice<A_L, BT, LINES> ra[2];
        Slice<B_L, BT, LINES> rb[2];
        float acc[T][T][4] = {}, sum[DIR == kExpWeight ? T * T * 4 : 1] = {};
        auto load = [&](int k, Slice<A_L, BT, LINES> &a, Slice<B_L, BT, LINES> &b) {
            if (k >= slices) return;
            const int64_t l = (int64_t)k * BL;
            a.fetch(w.a + (A_L ? l : l * w.stride_a), w.stride_a, w.i_lim, w.depth - k * BL, p.a, p.a_end);
            b.fetch(w.b + (B_L ? l : l * w.stride_b), w.stride_b, w.j_lim, w.depth - k * BL, p.b, p.b_end);
        };
        auto step = [&](int k, int h) {
            uint8_t *s = slabs + h * (A_BYTES + B_BYTES);
            ra[h].park(s);
            rb[h].park(s + A_BYTES);
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

template <int DIR, int BT, bool LINES>
cudaError_t launch_one(const ExpertSimtParams &p, cudaStream_t s) {
    constexpr int SMEM = 2 * (Slab<DIR != kExpWeight, BT>::BYTES + Slab<DIR == kExpForward, BT>::BYTES);
    static bool attr_set[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !attr_set[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(experts_b16_kernel<DIR, BT, LINES>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) attr_set[dev] = true;
    }
    return launch_early(experts_b16_kernel<DIR, BT, LINES>, p.grid, NT, SMEM, s, p);
}
template <int DIR, bool LINES = false>
cudaError_t launch_dir(const ExpertSimtParams &p, cudaStream_t s) {
    return p.wide ? launch_one<DIR, 128, LINES>(p, s) : launch_one<DIR, 64, LINES>(p, s);
}

}  // namespace

cudaError_t launch_experts_b16(const ExpertSimtParams &p, int dir, cudaStream_t s) {
    if (dir == kExpForward) return launch_dir<kExpForward>(p, s);
    if (dir == kExpData) return launch_dir<kExpData>(p, s);
    // Two neighbours on 4-byte addresses cost less than shifting lines: 8192 rows by 8 filters of 1028 x 1028 125 against
    // 204 us; single ones more: of 1001 x 1001 171 against 163, 16384 rows by 16 of them 495 against 289.  (data, whose
    // rows come in singles or pairs all the same: lines 141 against 122.)
    const bool words = (((uintptr_t)p.a | (uintptr_t)p.b) & 3) == 0 && (p.lda | p.ldb) % 2 == 0;
    return words ? launch_dir<kExpWeight>(p, s) : launch_dir<kExpWeight, true>(p, s);
}

}  // namespace cbd
