// policy_loss.cu -- clipped policy loss with a KL term over logits rows:
// forward, backward, and both in one launch.
//
// Per row: m = max z, s = sum exp(scale (z - m)) in one pass (the running sum
// is rescaled when the maximum grows), logp = scale (z_a - m) - log s, the
// loss and its derivative c = dloss/dlogp from four floats, then
// dz_v = c scale ([v = a] - exp(scale (z_v - m)) / s) in a second pass.
//
// Rows above 16 KB stream through a ring of 16 KB buffers in shared memory that
// one thread fills with bulk copies, three blocks per SM: up to 192 KB of reads
// stay in flight whatever the arithmetic does.  The fused form's second pass reads
// the row again, from L2 where its block has just had it: memory sees each logit
// once and each gradient once.  Narrower rows take a warp each and load into
// registers.  Bound by memory; measured at 6.68 TB/s: 8192 rows of 32768 bf16 fused
// 184 us (0.87), 1021 rows of 50257 fp32 forward 37 us (0.83), 300 rows of 128000
// bf16 backward 23.5 us (0.98, part of the logits still in L2).
// What the choice rests on (us, before launches were overlapped; the ring against
// rows loaded into registers): fused 190 (204), forward 38 (43), backward 25 (32).
// Two blocks of 512 workers took 225 fused, with the row kept in the ring between
// its passes 268: the ends of a pass, which only other rows' work can hide, weigh
// more than the second read from L2.
#include <cuda_bf16.h>
#include <math.h>

#include "device_util.cuh"
#include "internal.h"
#include "train.h"

namespace cbd {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int NT = 256;
constexpr int UNR = 4;  // 16-byte loads of a thread in flight

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <typename T>
struct Vec;
template <>
struct Vec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void unpack(const uint4 &u, float (&v)[4]) {
        v[0] = __uint_as_float(u.x);
        v[1] = __uint_as_float(u.y);
        v[2] = __uint_as_float(u.z);
        v[3] = __uint_as_float(u.w);
    }
    static __device__ __forceinline__ uint4 pack(const float (&v)[4]) {
        return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    }
    static __device__ __forceinline__ float get(const float *p) { return *p; }
    static __device__ __forceinline__ void put(float *p, float v) { *p = v; }
};
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void unpack(const uint4 &u, float (&v)[8]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ uint4 pack(const float (&v)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    static __device__ __forceinline__ float get(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
    static __device__ __forceinline__ void put(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }
};

// s = sum 2^(z c - off) over the elements so far, off = m c rounded, for a
// reference m: the first maximum, replaced where an element lies more than 2^16
// above it, so the sum neither overflows nor is rescaled often.  One FMA for each
// exponential; off's rounding is the same for a row's every term and cancels.
// Past |m c| = 256 it would be more than 2^-17: there the difference z - m is
// taken first (and rest is what off lacks, where sums of both meet).  -inf
// elements add 0; a NaN reaches s (fmaxf drops it from the maximum); m = -inf has
// no exponentials.  (FMAs are written out where the compiler could choose:
// forward and the fused form give the same bits.)
struct MaxSum {
    float m, s;
};
struct Exps {
    bool near;
    float base, off, rest, c;
    __device__ __forceinline__ Exps(float m, float c_) : c(c_) {
        const float mc = __fmul_rn(m, c_);
        near = fabsf(mc) < 256.f;
        base = near || m == -INFINITY ? 0.f : m;
        off = near ? mc : 0.f;
        rest = near ? fmaf(m, c_, -mc) : 0.f;
    }
    template <bool NEAR>
    __device__ __forceinline__ float at(float z) const {
        return ex2(NEAR ? fmaf(z, c, -off) : (z - base) * c);
    }
    __device__ __forceinline__ float at_any(float z) const { return near ? at<true>(z) : at<false>(z); }
    // the factor that brings a sum over another reference m to this one's terms
    __device__ __forceinline__ float from(float m, float m_here) const {
        if (m == -INFINITY || m == m_here) return 1.f;
        const Exps o(m, c);
        return near && o.near ? ex2(o.off - off) : ex2(fmaf(m - m_here, c, rest - o.rest));
    }
};
// a thread's elements
struct Run {
    MaxSum r;
    float lim, room;
    Exps e;
    __device__ __forceinline__ explicit Run(float c) : r{-INFINITY, 0.f}, lim(-INFINITY), room(16.f / c), e(-INFINITY, c) {}
    template <int N>
    __device__ __forceinline__ void take(const float (&v)[N]) {
        float m = v[0];
#pragma unroll
        for (int i = 1; i < N; ++i) m = fmaxf(m, v[i]);
        if (m > lim) {
            e = Exps(m, e.c);
            r.s = __fmul_rn(r.s, e.from(r.m, m));
            r.m = m;
            lim = m + room;
        }
        float s = 0.f;
        if (e.near) {
#pragma unroll
            for (int i = 0; i < N; ++i) s += e.at<true>(v[i]);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) s += e.at<false>(v[i]);
        }
        r.s = __fadd_rn(r.s, s);
    }
};
// The sums of N neighbouring lanes over one reference, in a fixed order; every lane gets it.
template <int N>
__device__ __forceinline__ MaxSum join(MaxSum r, float c) {
    float m = r.m;
#pragma unroll
    for (int d = N / 2; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    r.s = __fmul_rn(r.s, Exps(m, c).from(r.m, m));
    r.m = m;
#pragma unroll
    for (int d = N / 2; d; d >>= 1) r.s = __fadd_rn(r.s, __shfl_xor_sync(0xffffffffu, r.s, d));
    return r;
}
// log of the row's sum over exp((z - m) scale): the reference's own term, as it
// was computed, is 1, so a row with one entry left has 0
__device__ __forceinline__ float log_sum(const MaxSum &r, float c) { return logf(r.m == -INFINITY ? r.s : r.s / Exps(r.m, c).at_any(r.m)); }

// dz of an element: cs ([chosen] - p)
template <int MODE>
struct Grad {
    float cs, csi;  // csi exp(...) = cs p
    Exps e;
    float lse, scale;
    __device__ __forceinline__ Grad() : cs(0.f), csi(0.f), e(0.f, 1.f), lse(0.f), scale(0.f) {}
    template <bool NEAR>
    __device__ __forceinline__ float other(float z) const {
        return -csi * (MODE == kPolBackward ? ex2(fmaf(z, scale, -lse) * kLog2e) : e.at<NEAR>(z));
    }
    __device__ __forceinline__ float one(float z, bool chosen) const {
        const float g = e.near ? other<true>(z) : other<false>(z);
        return chosen ? cs + g : g;
    }
    // a vector whose first element is e0
    template <int N>
    __device__ __forceinline__ void vec(const float (&z)[N], float (&o)[N], int e0, int a) const {
        if (MODE == kPolBackward || e.near) {
#pragma unroll
            for (int j = 0; j < N; ++j) o[j] = other<true>(z[j]);
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j) o[j] = other<false>(z[j]);
        }
        if ((unsigned)(a - e0) < (unsigned)N) {
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (j == a - e0) o[j] += cs;
        }
    }
};

// A row's numbers, read ahead of their use.
struct RowIn {
    int a;
    float w, adv, old, ref;  // backward: coef, lse in w, adv
};
template <int MODE>
__device__ __forceinline__ RowIn row_in(const PolicyParams &p, int64_t t) {
    RowIn r;
    r.a = p.actions[t];
    if constexpr (MODE == kPolBackward) {
        r.w = p.coef_in[t];
        r.adv = p.lse_in[t];
        r.old = r.ref = 0.f;
    } else {
        r.w = p.weight[t];
        r.adv = p.advantage[t];
        r.old = p.old_logp ? p.old_logp[t] : 0.f;
        r.ref = p.ref_logp ? p.ref_logp[t] : 0.f;
    }
    return r;
}
__device__ __forceinline__ bool row_live(const PolicyParams &p, const RowIn &in) { return in.a >= 0 && in.a < p.vocab && in.w != 0.f; }

// What they give: loss, derivative.
__device__ __forceinline__ void row_loss(const PolicyParams &p, const RowIn &in, float logp, float &l, float &k) {
    const float adv = in.adv;
    const float ratio = p.old_logp ? expf(logp - in.old) : 1.f;
    const float ra = ratio * adv, ca = fminf(fmaxf(ratio, p.clip_lo), p.clip_hi) * adv;
    const bool unclipped = !(ra > ca);
    l = -(unclipped ? ra : ca);
    k = unclipped ? -ra : 0.f;
    if (p.ref_logp && p.kl > 0.f) {
        const float d = in.ref - logp, ed = expm1f(d);
        l = fmaf(p.kl, ed - d, l);
        k = fmaf(-p.kl, ed, k);
    }
    if (!p.old_logp && logp != logp) l = k = logp;  // no distribution: r = 1 would hide it
}

// The blocks' loss sums in order, by the block that finishes last: a fixed sum.
template <int N>
__device__ __forceinline__ void join_loss(const PolicyParams &p, double mine, double *sums, int *flag) {
    if (threadIdx.x == 0) {
        p.partials[blockIdx.x] = mine;
        __threadfence();
        *flag = atomicAdd(p.ticket, 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (!*flag) return;
    __threadfence();
    double s = 0.0;
    for (int i = threadIdx.x; i < (int)gridDim.x; i += N) s += __ldcg(p.partials + i);
    sums[threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.x < 32) {
        s = 0.0;
        for (int i = threadIdx.x; i < N; i += 32) s += sums[i];
#pragma unroll
        for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        if (threadIdx.x == 0) {
            *p.loss = (float)s;
            *p.ticket = 0;
        }
    }
}

// ---- narrow rows: a warp each ------------------------------------------------
template <typename T, int MODE>
__global__ void __launch_bounds__(NT) policy_warp_kernel(const PolicyParams p) {
    constexpr int ROWS = NT / 32;
    constexpr int VN = Vec<T>::N;
    __shared__ double block_loss[ROWS], sums[NT];
    __shared__ int flag;
    const int lane = threadIdx.x % 32, sub = threadIdx.x / 32;
    const int V = p.vocab;
    const float c = p.scale * kLog2e;
    double loss = 0.0;

    pdl_next();
    pdl_wait();
    const int64_t step = (int64_t)gridDim.x * ROWS;
    RowIn next = {};
    if (p.tokens > 0) next = row_in<MODE>(p, min((int64_t)blockIdx.x * ROWS + sub, (int64_t)p.tokens - 1));
    for (int64_t t = (int64_t)blockIdx.x * ROWS + sub; t < p.tokens; t += step) {
        const T *z = static_cast<const T *>(p.logits) + t * p.ld;
        T *dz = MODE == kPolForward ? nullptr : static_cast<T *>(p.dlogits) + t * p.ldd;
        const RowIn in = next;
        next = row_in<MODE>(p, min(t + step, (int64_t)p.tokens - 1));
        const int a = in.a;
        const bool live = row_live(p, in);
        if (a >= V && lane == 0) record_status(p.status, kDevFaultIndex);
        // elements before the first 16-byte boundary, 16-byte vectors, the rest
        const int head = min(V, (int)((16 - ((uintptr_t)z & 15)) % 16 / sizeof(T)));
        const int nv = (V - head) / VN;
        const uint4 *zv = reinterpret_cast<const uint4 *>(z + head);

        Grad<MODE> grad;
        if constexpr (MODE == kPolBackward) {
            if (live) {
                grad.cs = grad.csi = in.w * (p.grad ? *p.grad : 1.f) * p.scale;
                grad.lse = in.adv;
                grad.scale = p.scale;
            }
        } else if (live) {
            Run run(c);
            for (int i = lane; i < head; i += 32) {
                const float v[1] = {Vec<T>::get(z + i)};
                run.take(v);
            }
            int i = lane;
            for (; i + (UNR - 1) * 32 < nv; i += UNR * 32) {
                uint4 u[UNR];
#pragma unroll
                for (int q = 0; q < UNR; ++q) u[q] = zv[i + q * 32];
                float v[UNR * VN];
#pragma unroll
                for (int q = 0; q < UNR; ++q) {
                    float w[VN];
                    Vec<T>::unpack(u[q], w);
#pragma unroll
                    for (int k = 0; k < VN; ++k) v[q * VN + k] = w[k];
                }
                run.take(v);
            }
            for (; i < nv; i += 32) {
                float w[VN];
                Vec<T>::unpack(zv[i], w);
                run.take(w);
            }
            for (int k = head + nv * VN + lane; k < V; k += 32) {
                const float v[1] = {Vec<T>::get(z + k)};
                run.take(v);
            }
            const float za = Vec<T>::get(z + a);
            const MaxSum r = join<32>(run.r, c);
            __syncwarp();  // every lane has read its row: dlogits may overwrite it
            const float logs = log_sum(r, c);
            const float logp = fmaf(za - r.m, p.scale, -logs);
            const float w = in.w;
            float l, k;
            row_loss(p, in, logp, l, k);
            if (lane == 0) {
                loss += (double)w * (double)l;
                p.logp[t] = logp;
                if (p.lse) p.lse[t] = fmaf(r.m, p.scale, logs);
                if (p.coef) p.coef[t] = w * k;
            }
            grad.cs = w * k * p.scale;
            grad.csi = grad.cs / r.s;
            grad.e = Exps(r.m, c);
        } else if (lane == 0) {
            p.logp[t] = 0.f;
            if (p.lse) p.lse[t] = 0.f;
            if (p.coef) p.coef[t] = 0.f;
        }

        if constexpr (MODE != kPolForward) {
            const bool same = (((uintptr_t)z ^ (uintptr_t)dz) & 15) == 0;
            const int dhead = live && !same ? V : min(V, (int)((16 - ((uintptr_t)dz & 15)) % 16 / sizeof(T)));
            const int dnv = (V - dhead) / VN;
            uint4 *dv = reinterpret_cast<uint4 *>(dz + dhead);
            if (!live) {
                for (int i = lane; i < dhead; i += 32) Vec<T>::put(dz + i, 0.f);
                for (int i = lane; i < dnv; i += 32) dv[i] = make_uint4(0u, 0u, 0u, 0u);
                for (int k = dhead + dnv * VN + lane; k < V; k += 32) Vec<T>::put(dz + k, 0.f);
            } else {
                for (int i = lane; i < dhead; i += 32) Vec<T>::put(dz + i, grad.one(Vec<T>::get(z + i), i == a));
                auto one = [&](int i, const uint4 &u) {
                    float w[VN], o[VN];
                    Vec<T>::unpack(u, w);
                    grad.vec(w, o, dhead + i * VN, a);
                    dv[i] = Vec<T>::pack(o);
                };
                int i = lane;
                for (; i + (UNR - 1) * 32 < dnv; i += UNR * 32) {
                    uint4 u[UNR];
#pragma unroll
                    for (int q = 0; q < UNR; ++q) u[q] = zv[i + q * 32];
#pragma unroll
                    for (int q = 0; q < UNR; ++q) one(i + q * 32, u[q]);
                }
                for (; i < dnv; i += 32) one(i, zv[i]);
                for (int k = dhead + dnv * VN + lane; k < V; k += 32) Vec<T>::put(dz + k, grad.one(Vec<T>::get(z + k), k == a));
            }
        }
    }

    if constexpr (MODE != kPolBackward) {
        if (lane == 0) block_loss[sub] = loss;
        __syncthreads();
        double mine = 0.0;
        if (threadIdx.x == 0)
            for (int i = 0; i < ROWS; ++i) mine += block_loss[i];
        join_loss<NT>(p, mine, sums, &flag);
    }
}

// ---- wide rows ---------------------------------------------------------------
constexpr int CHUNK = 16384, RING = 4, WORKERS = 256, RING_BLOCKS = 3;  // of a block, blocks per SM
constexpr int EACH = CHUNK / 16 / WORKERS;             // vectors of a thread in a chunk
constexpr int kRingSmem = CHUNK * RING + 64 * 8;

struct RowAt {
    int head, nv, chunks;  // elements before the first 16-byte boundary, 16-byte vectors, chunks of them
};
template <typename T>
__device__ __forceinline__ RowAt row_at(const T *z, int V) {
    RowAt r;
    r.head = min(V, (int)((16 - ((uintptr_t)z & 15)) % 16 / sizeof(T)));
    r.nv = (V - r.head) / Vec<T>::N;
    r.chunks = (r.nv + CHUNK / 16 - 1) / (CHUNK / 16);  // (in vectors: a row of 2^30 entries has 2^32 bytes)
    return r;
}
template <typename T, int MODE>
__global__ void __launch_bounds__(WORKERS + 32, RING_BLOCKS) policy_ring_kernel(const PolicyParams p) {
    constexpr int VN = Vec<T>::N;
    extern __shared__ __align__(128) uint8_t ring[];
    uint64_t *bars = reinterpret_cast<uint64_t *>(ring + CHUNK * RING);
    __shared__ MaxSum sh[2][WORKERS / 32];
    __shared__ double sums[WORKERS + 32];
    __shared__ int flag;
    __shared__ int abort_;
    __shared__ volatile float fin[3];  // both: what the row's second pass needs
    volatile int32_t *abort_flag = &abort_;
    const uint32_t full0 = smem_u32(bars), empty0 = smem_u32(bars + RING);
    const int V = p.vocab, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const float c = p.scale * kLog2e;
    if (threadIdx.x == 0) {
        for (int i = 0; i < RING; ++i) {
            mbar_init(full0 + 8 * i, 1);
            mbar_init(empty0 + 8 * i, WORKERS / 32);
        }
        abort_ = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    pdl_next();
    pdl_wait();
    __syncthreads();
    double loss = 0.0;
    if (warp == WORKERS / 32) {
        // ------------------------------------------------------------ loads
        if (lane == 0) {
            uint64_t keep, drop;
            asm("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(keep));
            asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(drop));
            uint32_t it = 0;
            bool ok = true;
            RowIn next = row_in<MODE>(p, blockIdx.x);
            for (int64_t t = blockIdx.x; t < p.tokens && ok; t += gridDim.x) {
                const RowIn in = next;
                next = row_in<MODE>(p, min(t + gridDim.x, (int64_t)p.tokens - 1));
                if (!row_live(p, in)) continue;
                const T *z = static_cast<const T *>(p.logits) + t * p.ld;
                const RowAt r = row_at(z, V);
                const char *src = reinterpret_cast<const char *>(z + r.head);
                constexpr int PASSES = MODE == kPolBoth ? 2 : 1;
                for (int k = 0; k < PASSES * r.chunks && ok; ++k, ++it) {
                    const uint32_t b = it % RING, ph = (it / RING) & 1;
                    ok = mbar_wait_bounded(empty0 + 8 * b, ph ^ 1, p.wait_budget, abort_flag, p.status, kDevTimeoutProducer);
                    if (!ok) break;
                    const int chunk = k >= r.chunks ? k - r.chunks : k, bytes = min(CHUNK / 16, r.nv - chunk * (CHUNK / 16)) * 16;
                    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(full0 + 8 * b), "r"(bytes) : "memory");
                    // the fused form keeps a row in L2 until its second reading
                    const uint64_t policy = MODE == kPolBoth && k < r.chunks ? keep : drop;
                    asm volatile("cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(smem_u32(ring) + b * CHUNK),
                                 "l"(src + (int64_t)chunk * CHUNK), "r"(bytes), "r"(full0 + 8 * b), "l"(policy)
                                 : "memory");
                }
            }
            if (!ok) {
                for (int q = 0; q < 100; ++q) __nanosleep(1000);
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ workers
        const int tid = threadIdx.x;
        uint32_t it = 0;
        bool ok = true;  // after a wait that ran out: nothing is stored, the barriers are kept
        int turn = 0;    // which of sh's two slots; flips with the barrier that guards it, so not on masked rows
        RowIn next = row_in<MODE>(p, blockIdx.x);
        for (int64_t t = blockIdx.x; t < p.tokens; t += gridDim.x) {
            const RowIn in = next;
            next = row_in<MODE>(p, min(t + gridDim.x, (int64_t)p.tokens - 1));
            const T *z = static_cast<const T *>(p.logits) + t * p.ld;
            T *dz = MODE == kPolForward ? nullptr : static_cast<T *>(p.dlogits) + t * p.ldd;
            const int a = in.a;
            if (a >= V && tid == 0) record_status(p.status, kDevFaultIndex);
            if (!row_live(p, in)) {
                if constexpr (MODE != kPolBackward) {
                    if (tid == 0) {
                        p.logp[t] = 0.f;
                        if (p.lse) p.lse[t] = 0.f;
                        if (p.coef) p.coef[t] = 0.f;
                    }
                }
                if constexpr (MODE != kPolForward) {
                    const RowAt d = row_at(dz, V);
                    uint4 *dv = reinterpret_cast<uint4 *>(dz + d.head);
                    if (tid < d.head) Vec<T>::put(dz + tid, 0.f);
                    for (int i = tid; i < d.nv; i += WORKERS) dv[i] = make_uint4(0u, 0u, 0u, 0u);
                    for (int i = d.head + d.nv * VN + tid; i < V; i += WORKERS) Vec<T>::put(dz + i, 0.f);
                }
                continue;
            }
            const RowAt r = row_at(z, V);
            const int tail = r.head + r.nv * VN;  // first element after the vectors
            // the row's ends: at most one element of a thread before and after the vectors
            const bool has_head = tid < r.head, has_tail = tail + tid < V;
            const float zh = has_head ? Vec<T>::get(z + tid) : -INFINITY, zt = has_tail ? Vec<T>::get(z + tail + tid) : -INFINITY;
            auto landed = [&](uint32_t i) {
                if (ok) ok = mbar_wait_bounded(full0 + 8 * (i % RING), (i / RING) & 1, p.wait_budget, abort_flag, p.status, kDevTimeoutEpilogue);
            };
            auto release = [&](uint32_t i) {
                __syncwarp();
                if (lane == 0) mbar_arrive(empty0 + 8 * (i % RING));
            };
            Grad<MODE> grad;
            if constexpr (MODE == kPolBackward) {
                grad.cs = grad.csi = in.w * (p.grad ? *p.grad : 1.f) * p.scale;
                grad.lse = in.adv;
                grad.scale = p.scale;
            } else {
                const float za = Vec<T>::get(z + a);
                Run run(c);
                if (has_head || has_tail) {
                    const float v[2] = {zh, zt};
                    run.take(v);
                }
                for (int k = 0; k < r.chunks; ++k) {
                    landed(it + k);
                    const uint4 *buf = reinterpret_cast<const uint4 *>(ring + ((it + k) % RING) * CHUNK);
                    const int n = min(CHUNK / 16, r.nv - k * (CHUNK / 16));
                    if (n == CHUNK / 16) {
                        float v[EACH * VN];
#pragma unroll
                        for (int q = 0; q < EACH; ++q) {
                            float w[VN];
                            Vec<T>::unpack(buf[tid + q * WORKERS], w);
#pragma unroll
                            for (int j = 0; j < VN; ++j) v[q * VN + j] = w[j];
                        }
                        run.take(v);
                    } else {
                        for (int i = tid; i < n; i += WORKERS) {
                            float w[VN];
                            Vec<T>::unpack(buf[i], w);
                            run.take(w);
                        }
                    }
                    release(it + k);
                }
                it += r.chunks;
                const MaxSum part = join<32>(run.r, c);
                // (a slot is written again two live rows later, after the barrier that warp 0 meets when it has read it)
                MaxSum *slot = sh[turn];
                turn ^= 1;
                if (lane == 0) slot[warp] = part;
                asm volatile("bar.sync 1, %0;" ::"n"(WORKERS) : "memory");
                if (warp == 0) {  // one warp ends the row; the others issue nothing meanwhile
                    const MaxSum m = join<WORKERS / 32>(slot[lane % (WORKERS / 32)], c);
                    const float logs = log_sum(m, c), logp = fmaf(za - m.m, p.scale, -logs), w = in.w;
                    float l, k;
                    row_loss(p, in, logp, l, k);
                    if (lane == 0) {
                        if (ok) {
                            loss += (double)w * (double)l;
                            p.logp[t] = logp;
                            if (p.lse) p.lse[t] = fmaf(m.m, p.scale, logs);
                            if (p.coef) p.coef[t] = w * k;
                        }
                        if constexpr (MODE == kPolBoth) {
                            const float cs = w * k * p.scale;
                            fin[0] = cs;
                            fin[1] = cs / m.s;
                            fin[2] = m.m;
                        }
                    }
                }
                if constexpr (MODE == kPolBoth) {
                    asm volatile("bar.sync 1, %0;" ::"n"(WORKERS) : "memory");
                    grad.cs = fin[0];
                    grad.csi = fin[1];
                    grad.e = Exps(fin[2], c);
                }
            }
            if constexpr (MODE != kPolForward) {
                if (ok && has_head) Vec<T>::put(dz + tid, grad.one(zh, tid == a));
                if (ok && has_tail) Vec<T>::put(dz + tail + tid, grad.one(zt, tail + tid == a));
                const bool same = (((uintptr_t)z ^ (uintptr_t)dz) & 15) == 0;
                for (int k = 0; k < r.chunks; ++k) {
                    landed(it + k);
                    const uint4 *buf = reinterpret_cast<const uint4 *>(ring + ((it + k) % RING) * CHUNK);
                    const int v0 = k * (CHUNK / 16), n = ok ? min(CHUNK / 16, r.nv - v0) : 0;
                    auto vector = [&](int i, const uint4 &u) {
                        float w[VN], o[VN];
                        Vec<T>::unpack(u, w);
                        const int e0 = r.head + (v0 + i) * VN;
                        grad.vec(w, o, e0, a);
                        if (same) {
                            __stcs(reinterpret_cast<uint4 *>(dz + e0), Vec<T>::pack(o));
                        } else {
#pragma unroll
                            for (int j = 0; j < VN; ++j) Vec<T>::put(dz + e0 + j, o[j]);
                        }
                    };
                    if (n == CHUNK / 16) {
                        uint4 u[EACH];
#pragma unroll
                        for (int q = 0; q < EACH; ++q) u[q] = buf[tid + q * WORKERS];
#pragma unroll
                        for (int q = 0; q < EACH; ++q) vector(tid + q * WORKERS, u[q]);
                    } else {
                        for (int i = tid; i < n; i += WORKERS) vector(i, buf[i]);
                    }
                    release(it + k);
                }
                it += r.chunks;
            }
        }
    }
    __syncthreads();
    if constexpr (MODE != kPolBackward) join_loss<WORKERS + 32>(p, loss, sums, &flag);
}

constexpr int kBlocksPerSm = 8;

template <typename T>
cudaError_t launch_warp(const PolicyParams &p, int mode, int num_sms, cudaStream_t s) {
    const int64_t need = (p.tokens + NT / 32 - 1) / (NT / 32);
    const int grid = (int)(need < 1 ? 1 : need < policy_max_blocks(num_sms) ? need : policy_max_blocks(num_sms));
    if (mode == kPolForward) return launch_early(policy_warp_kernel<T, kPolForward>, grid, NT, 0, s, p);
    if (mode == kPolBackward) return launch_early(policy_warp_kernel<T, kPolBackward>, grid, NT, 0, s, p);
    return launch_early(policy_warp_kernel<T, kPolBoth>, grid, NT, 0, s, p);
}
template <typename T, int MODE>
cudaError_t launch_ring_mode(const PolicyParams &p, int num_sms, cudaStream_t s) {
    static bool attr_set[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !attr_set[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(policy_ring_kernel<T, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingSmem);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) attr_set[dev] = true;
    }
    int grid = RING_BLOCKS * num_sms;
    if (MODE == kPolBoth) {  // rows between their two readings: at most 64 MB, half of L2
        const int64_t rows = (64LL << 20) / ((int64_t)p.vocab * (int64_t)sizeof(T));
        if (rows < grid) grid = rows > num_sms ? (int)rows : num_sms;
    }
    return launch_early(policy_ring_kernel<T, MODE>, p.tokens < grid ? p.tokens : grid, WORKERS + 32, kRingSmem, s, p);
}
template <typename T>
cudaError_t launch_ring(const PolicyParams &p, int mode, int num_sms, cudaStream_t s) {
    return mode == kPolForward    ? launch_ring_mode<T, kPolForward>(p, num_sms, s)
           : mode == kPolBackward ? launch_ring_mode<T, kPolBackward>(p, num_sms, s)
                                  : launch_ring_mode<T, kPolBoth>(p, num_sms, s);
}

}  // namespace

int policy_max_blocks(int num_sms) { return num_sms * kBlocksPerSm; }

cudaError_t launch_policy(const PolicyParams &p, int dtype, int mode, int num_sms, cudaStream_t s) {
    // (one rule for every mode: forward and the fused form add in the same order)
    const bool narrow = (int64_t)p.vocab * (dtype == 1 ? 2 : 4) <= 16384 || p.tokens == 0;
    if (dtype == 1) return narrow ? launch_warp<__nv_bfloat16>(p, mode, num_sms, s) : launch_ring<__nv_bfloat16>(p, mode, num_sms, s);
    return narrow ? launch_warp<float>(p, mode, num_sms, s) : launch_ring<float>(p, mode, num_sms, s);
}

}  // namespace cbd
