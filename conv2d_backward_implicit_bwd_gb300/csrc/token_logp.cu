// token_logp.cu -- log-probabilities of given tokens, entropy and the largest
// alternatives of logits rows; gradients of log-probability and entropy.
//
// Forward, one pass over a row: with a running reference m, c = scale log2(e) and
// d_v = c (z_v - m),
//   s = sum 2^d,  t = sum 2^d d,
//   lse = scale m + log s,  logp = scale (z_a - m) - log s,  H = log s - ln2 t / s.
// H adds two non-negative numbers where m is the maximum; the reference follows the
// maximum within 2^1 (a wider step would leave t with terms of d up to it, whose
// rounding H, near 0 in confident rows, would show).
//
// Alternatives: keys of 64 bits, the value's order above the inverted index, so the
// largest of any set is unique (ties go to the lowest index) and the result does not
// depend on the order of work.  A warp keeps its 32 best sorted over its lanes.  A
// batch whose maximum is below the bound costs a comparison; else its elements at or
// above the bound go to a queue, and 32 of them at a time are sorted (15 exchanges)
// and merged (6).  The bound is the larger of the warp's own last place and the
// smallest of the block's posts: each warp posts its ceil(top / 8)-th best, so
// `top` elements of the row lie at or above that.  An empty list takes its first bound
// from the batch's lane maxima (without it every element of the first batch is a
// candidate).
//
// Rows above 16 KB stream through a ring of 16 KB buffers that one thread fills with
// bulk copies, as in the policy loss; where rows are few each is cut into parts, and
// the block that ends a row last joins the parts' sums and lists in their order.
// Narrower rows take a warp each.
#include <cuda_bf16.h>
#include <math.h>

#include <algorithm>

#include "device_util.cuh"
#include "internal.h"
#include "train.h"
#include "vocab_rows.cuh"

namespace cbd {

namespace {

constexpr int NT = 256;
constexpr int UNR = 4;  // 16-byte loads of a thread in flight
constexpr float kLn2 = 0.6931471805599453f;
constexpr uint32_t kAll = 0xffffffffu;

struct Sums {
    float m, s, t;
};
// r over the reference m instead of its own
__device__ __forceinline__ Sums rebased(const Sums &r, float m, float c) {
    const float up = Exps(m, c).shift(r.m, m), f = ex2(up);
    return {m, r.s * f, fmaf(r.s, up, r.t) * f};
}
struct Run {
    Sums r;
    float lim, room;
    Exps e;
    __device__ __forceinline__ explicit Run(float c) : r{-INFINITY, 0.f, 0.f}, lim(-INFINITY), room(1.f / c), e(-INFINITY, c) {}
    template <bool NEAR, int N>
    __device__ __forceinline__ void add(const float (&v)[N]) {
        float s = 0.f, t = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float d = NEAR ? fmaf(v[i], e.c, -e.off) : (v[i] - e.base) * e.c, p = ex2(d);
            s += p;
            t = fmaf(p, fmaxf(d, -200.f), t);  // (2^-inf * -inf is not 0)
        }
        r.s += s;
        r.t += t;
    }
    // returns the elements' maximum
    template <int N>
    __device__ __forceinline__ float take(const float (&v)[N]) {
        float m = v[0];
#pragma unroll
        for (int i = 1; i < N; ++i) m = fmaxf(m, v[i]);
        if (m > lim) {
            r = rebased(r, m, e.c);
            e = Exps(m, e.c);
            lim = m + room;
        }
        if (e.near)
            add<true>(v);
        else
            add<false>(v);
        return m;
    }
};
// The sums of N neighbouring lanes over one reference, in a fixed order; every lane gets it.
template <int N>
__device__ __forceinline__ Sums join(Sums r, float c) {
    float m = r.m;
#pragma unroll
    for (int d = N / 2; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, d));
    r = rebased(r, m, c);
#pragma unroll
    for (int d = N / 2; d; d >>= 1) {
        r.s += __shfl_xor_sync(kAll, r.s, d);
        r.t += __shfl_xor_sync(kAll, r.t, d);
    }
    return r;
}
// log of the sum over exp((z - m) scale): the reference's own term, as it was computed, is 1
__device__ __forceinline__ float log_sum(const Sums &r, float c) { return logf(r.m == -INFINITY ? r.s : r.s / Exps(r.m, c).at_any(r.m)); }
// (a row without a distribution: s = 0 and t / s is NaN)
__device__ __forceinline__ float entropy(const Sums &r) {
    const float h = logf(r.s) - kLn2 * (r.t / r.s);
    return h < 0.f ? 0.f : h;
}

// ---- the largest elements ------------------------------------------------------
__device__ __forceinline__ uint32_t ordered(float v) {
    const uint32_t b = __float_as_uint(v + 0.f);  // (-0 ties with 0)
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint64_t key) {
    const uint32_t b = (uint32_t)(key >> 32);
    return __uint_as_float(b & 0x80000000u ? b ^ 0x80000000u : ~b);
}
__device__ __forceinline__ uint64_t key_of(float v, uint32_t index) { return (uint64_t)ordered(v) << 32 | (kAll - index); }
template <typename K>
__device__ __forceinline__ K exchange(K x, int d, bool keep_larger) {
    const K o = __shfl_xor_sync(kAll, x, d);
    return (x > o) == keep_larger ? x : o;
}
template <typename K>
__device__ __forceinline__ K sorted_falling(K x, int lane) {
#pragma unroll
    for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
        for (int j = k / 2; j; j >>= 1) x = exchange(x, j, ((lane & j) == 0) == ((lane & k) == 0));
    return x;
}
// the 32 largest of two falling lists, falling
__device__ __forceinline__ uint64_t merged(uint64_t a, uint64_t b, int lane) {
    const uint64_t o = __shfl_sync(kAll, b, 31 - lane);
    a = a > o ? a : o;
#pragma unroll
    for (int j = 16; j; j >>= 1) a = exchange(a, j, (lane & j) == 0);
    return a;
}
constexpr int kQueue = 64;
// A warp's list: lane i has the i-th best, 0 where there is none yet.
struct List {
    uint64_t key, last;  // last: the top-th
    float bound;         // of values that may still enter
    int count;           // queued
    uint64_t *queue;     // [kQueue], the warp's own
    int top, lane;
    __device__ __forceinline__ List(uint64_t *q, int top_, int lane_) : key(0), last(0), bound(-INFINITY), count(0), queue(q), top(top_), lane(lane_) {}
    __device__ __forceinline__ void flush() {
        __syncwarp();
        const int first = count > 32 ? count - 32 : 0;
        const uint64_t mine = first + lane < count ? queue[first + lane] : 0;
        __syncwarp();
        count = first;
        key = merged(key, sorted_falling(mine, lane), lane);
        last = __shfl_sync(kAll, key, top - 1);
        if (last) bound = fmaxf(bound, value_of(last));
    }
    // (by the whole warp)
    __device__ __forceinline__ void offer(bool there, float v, int index) {
        const uint64_t k = key_of(v, (uint32_t)index);
        const bool in = there && v >= bound && k > last;
        const uint32_t who = __ballot_sync(kAll, in);
        if (who == 0) return;
        if (in) queue[count + __popc(who & ((1u << lane) - 1))] = k;
        count += __popc(who);
        if (count >= 32) flush();
    }
    __device__ __forceinline__ void end() {
        while (count > 0) flush();
    }
    // a first bound from the maxima of the lanes' elements
    __device__ __forceinline__ uint32_t first(float m) {
        const uint32_t by = sorted_falling(m == m ? ordered(m) : 0u, lane);
        const uint32_t at = __shfl_sync(kAll, by, top - 1);
        if (at) bound = fmaxf(bound, value_of((uint64_t)at << 32));
        return by;
    }
};

// What a row's end writes.
__device__ __forceinline__ void put_sums(const LogpParams &p, int64_t t, const Sums &r, float za, float c) {
    const float logs = log_sum(r, c);
    if (p.logp) p.logp[t] = fmaf(za - r.m, p.scale, -logs);
    p.entropy[t] = entropy(r);
    p.lse[t] = fmaf(r.m, p.scale, logs);
}
__device__ __forceinline__ void put_list(const LogpParams &p, int64_t t, const Sums &r, uint64_t key, int lane, float c) {
    if (lane >= p.top) return;
    const float logs = log_sum(r, c);
    // (elements that are not numbers enter no list: -1 where too few are left)
    p.top_logp[t * p.top + lane] = key ? fmaf(value_of(key) - r.m, p.scale, -logs) : __uint_as_float(0x7fffffffu);
    p.top_tokens[t * p.top + lane] = key ? (int32_t)(kAll - (uint32_t)key) : -1;
}
__device__ __forceinline__ void put_masked(const LogpParams &p, int64_t t, int lane) {
    if (lane == 0) {
        if (p.logp) p.logp[t] = 0.f;
        p.entropy[t] = 0.f;
        p.lse[t] = 0.f;
    }
    if (lane < p.top) {
        p.top_logp[t * p.top + lane] = 0.f;
        p.top_tokens[t * p.top + lane] = -1;
    }
}

// ---- narrow rows: a warp each ------------------------------------------------
template <typename T, bool TOP>
__global__ void __launch_bounds__(NT) logp_warp_kernel(const LogpParams p) {
    constexpr int ROWS = NT / 32;
    constexpr int VN = Vec<T>::N;
    __shared__ uint64_t queues[TOP ? ROWS : 1][kQueue];
    const int lane = threadIdx.x % 32, sub = threadIdx.x / 32;
    const int V = p.vocab;
    const float c = p.scale * kLog2e;
    pdl_next();
    pdl_wait();
    const int64_t step = (int64_t)gridDim.x * ROWS;
    for (int64_t t = (int64_t)blockIdx.x * ROWS + sub; t < p.rows; t += step) {
        const T *z = static_cast<const T *>(p.logits) + t * p.ld;
        const int a = p.tokens ? p.tokens[t] : 0;
        if (a >= V && lane == 0) record_status(p.status, kDevFaultIndex);
        if (a < 0 || a >= V) {
            put_masked(p, t, lane);
            continue;
        }
        // elements before the first 16-byte boundary, 16-byte vectors, the rest
        const int head = min(V, (int)((16 - ((uintptr_t)z & 15)) % 16 / sizeof(T)));
        const int nv = (V - head) / VN, tail = head + nv * VN;
        const uint4 *zv = reinterpret_cast<const uint4 *>(z + head);
        const float za = Vec<T>::get(z + a);
        Run run(c);
        List list(queues[TOP ? sub : 0], TOP ? p.top : 1, lane);
        const bool has_head = lane < head, has_tail = tail + lane < V;
        const float ends[2] = {has_head ? Vec<T>::get(z + lane) : -INFINITY, has_tail ? Vec<T>::get(z + tail + lane) : -INFINITY};
        for (int i0 = 0; i0 < nv; i0 += UNR * 32) {
            uint4 u[UNR];
            float v[UNR * VN];
#pragma unroll
            for (int q = 0; q < UNR; ++q)
                if (i0 + q * 32 + lane < nv) u[q] = zv[i0 + q * 32 + lane];
#pragma unroll
            for (int q = 0; q < UNR; ++q) {
                float w[VN];
                Vec<T>::unpack(u[q], w);
#pragma unroll
                for (int k = 0; k < VN; ++k) v[q * VN + k] = i0 + q * 32 + lane < nv ? w[k] : -INFINITY;
            }
            const float m = run.take(v);
            if constexpr (TOP) {
                if (list.last == 0) list.first(m);
                if (__any_sync(kAll, m >= list.bound)) {
#pragma unroll
                    for (int q = 0; q < UNR; ++q)
#pragma unroll
                        for (int k = 0; k < VN; ++k) list.offer(i0 + q * 32 + lane < nv, v[q * VN + k], head + (i0 + q * 32 + lane) * VN + k);
                }
            }
        }
        run.take(ends);
        const Sums r = join<32>(run.r, c);
        if constexpr (TOP) {
            list.offer(has_head, ends[0], lane);
            list.offer(has_tail, ends[1], tail + lane);
            list.end();
            put_list(p, t, r, list.key, lane, c);
        }
        if (lane == 0) put_sums(p, t, r, za, c);
        __syncwarp();
    }
}

// dz = p (a + b u) + cs [chosen], u = scale z - lse
struct Slope {
    float scale, lse, a, b, cs;
    int chosen;
    __device__ __forceinline__ float at(float z) const {
        const float u = fmaf(z, scale, -lse);
        return ex2(u * kLog2e) * fmaf(b, fmaxf(u, -1e4f), a);  // (2^-inf * -inf is not 0)
    }
    __device__ __forceinline__ float one(float z, int i) const { return i == chosen ? at(z) + cs : at(z); }
    template <int N>
    __device__ __forceinline__ void vec(const float (&z)[N], float (&o)[N], int e0) const {
#pragma unroll
        for (int j = 0; j < N; ++j) o[j] = at(z[j]);
        if ((unsigned)(chosen - e0) < (unsigned)N) {
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (j == chosen - e0) o[j] += cs;
        }
    }
};
// A row's numbers, read ahead of their use.
struct GradIn {
    int a;
    float lse, h, gl, ge;
};
__device__ __forceinline__ GradIn grad_in(const LogpParams &p, int64_t t) {
    GradIn r;
    r.a = p.tokens ? p.tokens[t] : 0;
    r.lse = p.lse_in[t];
    r.h = p.entropy_in ? p.entropy_in[t] : 0.f;
    r.gl = p.grad_logp ? p.grad_logp[t] : 0.f;
    r.ge = p.grad_entropy ? p.grad_entropy[t] : 0.f;
    return r;
}
__device__ __forceinline__ bool grad_live(const LogpParams &p, const GradIn &in) { return in.a >= 0 && in.a < p.vocab && (in.gl != 0.f || in.ge != 0.f); }
__device__ __forceinline__ Slope slope(const LogpParams &p, const GradIn &in) {
    Slope s;
    s.scale = p.scale;
    s.lse = in.lse;
    s.b = -p.scale * in.ge;
    s.a = -p.scale * fmaf(in.ge, in.h, in.gl);
    s.cs = p.scale * in.gl;
    s.chosen = p.grad_logp ? in.a : -1;
    return s;
}

template <typename T>
__global__ void __launch_bounds__(NT) logp_grad_warp_kernel(const LogpParams p) {
    constexpr int ROWS = NT / 32;
    constexpr int VN = Vec<T>::N;
    const int lane = threadIdx.x % 32, sub = threadIdx.x / 32;
    const int V = p.vocab;
    pdl_next();
    pdl_wait();
    const int64_t step = (int64_t)gridDim.x * ROWS, first = (int64_t)blockIdx.x * ROWS + sub;
    if (first >= p.rows) return;
    GradIn next = grad_in(p, first);
    for (int64_t t = first; t < p.rows; t += step) {
        const T *z = static_cast<const T *>(p.logits) + t * p.ld;
        T *dz = static_cast<T *>(p.dlogits) + t * p.ldd;
        const GradIn in = next;
        next = grad_in(p, min(t + step, (int64_t)p.rows - 1));
        const bool live = grad_live(p, in);
        if (in.a >= V && lane == 0) record_status(p.status, kDevFaultIndex);
        const Slope g = slope(p, in);
        const bool same = (((uintptr_t)z ^ (uintptr_t)dz) & 15) == 0;
        const int head = live && !same ? V : min(V, (int)((16 - ((uintptr_t)dz & 15)) % 16 / sizeof(T)));
        const int nv = (V - head) / VN, tail = head + nv * VN;
        const uint4 *zv = reinterpret_cast<const uint4 *>(z + head);
        uint4 *dv = reinterpret_cast<uint4 *>(dz + head);
        if (!live) {
            for (int i = lane; i < head; i += 32) Vec<T>::put(dz + i, 0.f);
            for (int i = lane; i < nv; i += 32) dv[i] = make_uint4(0u, 0u, 0u, 0u);
            for (int k = tail + lane; k < V; k += 32) Vec<T>::put(dz + k, 0.f);
            continue;
        }
        for (int i = lane; i < head; i += 32) Vec<T>::put(dz + i, g.one(Vec<T>::get(z + i), i));
        auto one = [&](int i, const uint4 &u) {
            float w[VN], o[VN];
            Vec<T>::unpack(u, w);
            g.vec(w, o, head + i * VN);
            dv[i] = Vec<T>::pack(o);
        };
        int i = lane;
        for (; i + (UNR - 1) * 32 < nv; i += UNR * 32) {
            uint4 u[UNR];
#pragma unroll
            for (int q = 0; q < UNR; ++q) u[q] = zv[i + q * 32];
#pragma unroll
            for (int q = 0; q < UNR; ++q) one(i + q * 32, u[q]);
        }
        for (; i < nv; i += 32) one(i, zv[i]);
        for (int k = tail + lane; k < V; k += 32) Vec<T>::put(dz + k, g.one(Vec<T>::get(z + k), k));
    }
}

// ---- wide rows ---------------------------------------------------------------
constexpr int CHUNK = 16384, RING = 4, WORKERS = 256, RING_BLOCKS = 3;  // of a block, blocks per SM
constexpr int WARPS = WORKERS / 32;
constexpr int EACH = CHUNK / 16 / WORKERS;  // vectors of a thread in a chunk
constexpr int kRingSmem = CHUNK * RING + 64 * 8;

// The vectors [v0, v1) of row t that an item covers, with the elements before the row's first 16-byte boundary if it is
// the first part and those after the last vector if it is the last.
template <typename T>
struct Item {
    const T *z;
    int head, v0, v1, tail;
    bool first, last;
    __device__ __forceinline__ Item(const T *z_, int V, int part, int parts) : z(z_) {
        head = min(V, (int)((16 - ((uintptr_t)z & 15)) % 16 / sizeof(T)));
        const int nv = (V - head) / Vec<T>::N;
        v0 = (int)((int64_t)nv * part / parts);
        v1 = (int)((int64_t)nv * (part + 1) / parts);
        tail = head + nv * Vec<T>::N;
        first = part == 0;
        last = part == parts - 1;
    }
    __device__ __forceinline__ int chunks() const { return (v1 - v0 + CHUNK / 16 - 1) / (CHUNK / 16); }  // (in vectors: a row has up to 2^32 bytes)
    __device__ __forceinline__ int vectors(int chunk) const { return min(CHUNK / 16, v1 - v0 - chunk * (CHUNK / 16)); }
};

struct Ring {
    uint64_t full[RING], empty[RING];
};
__device__ __forceinline__ void ring_init(Ring &r, int *abort_) {
    if (threadIdx.x == 0) {
        for (int i = 0; i < RING; ++i) {
            mbar_init(smem_u32(&r.full[i]), 1);
            mbar_init(smem_u32(&r.empty[i]), WARPS);
        }
        *abort_ = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
}
// one thread: the item's chunks into the ring
template <typename T>
__device__ __forceinline__ bool ring_fill(uint8_t *ring, Ring &bars, const Item<T> &item, uint32_t &it, uint64_t policy, int64_t budget, volatile int32_t *abort_flag, int32_t *status) {
    const char *src = reinterpret_cast<const char *>(item.z + item.head) + (int64_t)item.v0 * 16;
    const int chunks = item.chunks();
    for (int k = 0; k < chunks; ++k, ++it) {
        const uint32_t b = it % RING, ph = (it / RING) & 1;
        if (!mbar_wait_bounded(smem_u32(&bars.empty[b]), ph ^ 1, budget, abort_flag, status, kDevTimeoutProducer)) return false;
        const int bytes = item.vectors(k) * 16;
        const uint32_t full = smem_u32(&bars.full[b]);
        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(full), "r"(bytes) : "memory");
        asm volatile("cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(smem_u32(ring) + b * CHUNK),
                     "l"(src + (int64_t)k * CHUNK), "r"(bytes), "r"(full), "l"(policy)
                     : "memory");
    }
    return true;
}

// A part's share of its row, in the workspace.
struct __align__(16) Part {
    Sums r;
    uint32_t pad;
    uint64_t key[32];
};
static_assert(sizeof(Part) == kLogpPart, "workspace");

template <typename T, bool TOP>
__global__ void __launch_bounds__(WORKERS + 32, RING_BLOCKS) logp_ring_kernel(const LogpParams p) {
    constexpr int VN = Vec<T>::N;
    extern __shared__ __align__(128) uint8_t ring[];
    Ring &bars = *reinterpret_cast<Ring *>(ring + CHUNK * RING);
    __shared__ Sums sh[2][WARPS];
    __shared__ uint64_t lists[TOP ? 2 : 1][TOP ? WARPS : 1][32];
    __shared__ uint64_t queues[TOP ? WARPS : 1][kQueue];
    __shared__ float posts[2][WARPS];
    __shared__ int abort_;
    volatile int32_t *abort_flag = &abort_;
    const int V = p.vocab, warp = threadIdx.x / 32, lane = threadIdx.x % 32, parts = p.parts;
    const float c = p.scale * kLog2e;
    ring_init(bars, &abort_);
    if (threadIdx.x < 2 * WARPS) (&posts[0][0])[threadIdx.x] = -INFINITY;
    pdl_next();
    pdl_wait();
    __syncthreads();
    const int64_t items = (int64_t)p.rows * parts;
    auto live = [&](int64_t t) { return !p.tokens || (unsigned)p.tokens[t] < (unsigned)V; };
    if (warp == WARPS) {
        // ------------------------------------------------------------ loads
        if (lane == 0) {
            uint64_t drop;
            asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(drop));
            uint32_t it = 0;
            bool ok = true;
            for (int64_t w = blockIdx.x; w < items && ok; w += gridDim.x) {
                const int64_t t = w / parts;
                if (!live(t)) continue;
                ok = ring_fill(ring, bars, Item<T>(static_cast<const T *>(p.logits) + t * p.ld, V, (int)(w - t * parts), parts), it, drop, p.wait_budget, abort_flag, p.status);
            }
            if (!ok) {
                for (int q = 0; q < 100; ++q) __nanosleep(1000);
            }
        }
        __syncwarp();
        return;
    }
    // ---------------------------------------------------------------- workers
    const int tid = threadIdx.x;
    uint32_t it = 0;
    bool ok = true;  // after a wait that ran out: nothing is stored, the barriers are kept
    int turn = 0;    // which of the two slots; flips with the barrier that guards it, so not on masked rows
    for (int64_t w = blockIdx.x; w < items; w += gridDim.x) {
        const int64_t t = w / parts;
        const int part = (int)(w - t * parts);
        if (!live(t)) {
            if (part == 0 && warp == 0) {
                if (lane == 0 && p.tokens[t] >= V) record_status(p.status, kDevFaultIndex);
                put_masked(p, t, lane);
            }
            continue;
        }
        const T *z = static_cast<const T *>(p.logits) + t * p.ld;
        const Item<T> item(z, V, part, parts);
        const float za = warp == 0 && p.logp ? Vec<T>::get(z + p.tokens[t]) : 0.f;
        // the row's ends: at most one element of a thread before and after the vectors
        const bool has_head = item.first && tid < item.head, has_tail = item.last && item.tail + tid < V;
        const float ends[2] = {has_head ? Vec<T>::get(z + tid) : -INFINITY, has_tail ? Vec<T>::get(z + item.tail + tid) : -INFINITY};
        Run run(c);
        List list(queues[TOP ? warp : 0], TOP ? p.top : 1, lane);
        volatile float *post = posts[turn];  // (each has one writer and only rises: whatever a reader sees is a bound)
        const int place = TOP ? (p.top + WARPS - 1) / WARPS - 1 : 0;  // of the posted element
        // a batch's elements, still in the buffer, that may be among the largest
        auto pick = [&](const uint4 *buf, int n, float m, int e0) {
            if (list.last == 0) {
                const uint32_t by = __shfl_sync(kAll, list.first(m), place);
                if (by && lane == 0) post[warp] = fmaxf(post[warp], value_of((uint64_t)by << 32));
                __syncwarp();
            }
            float low = post[0];
#pragma unroll
            for (int q = 1; q < WARPS; ++q) low = fminf(low, post[q]);
            list.bound = fmaxf(list.bound, low);
            list.bound = __shfl_sync(kAll, list.bound, 0);  // (the posts may rise between two lanes' loads)
            if (!__any_sync(kAll, m >= list.bound)) return;
#pragma unroll 1
            for (int i = tid; i - lane < n; i += WORKERS) {
                const bool there = i < n;
                uint4 u = make_uint4(0u, 0u, 0u, 0u);
                if (there) u = buf[i];
                float v[VN];
                Vec<T>::unpack(u, v);
                float top = v[0];
#pragma unroll
                for (int k = 1; k < VN; ++k) top = fmaxf(top, v[k]);
                if (!__any_sync(kAll, there && top >= list.bound)) continue;
#pragma unroll
                for (int k = 0; k < VN; ++k) list.offer(there, v[k], e0 + i * VN + k);
            }
            const uint64_t mine = __shfl_sync(kAll, list.key, place);
            if (mine && lane == 0) post[warp] = fmaxf(post[warp], value_of(mine));
        };
        const int chunks = item.chunks();
        for (int k = 0; k < chunks; ++k) {
            const uint32_t b = (it + k) % RING;
            if (ok) ok = mbar_wait_bounded(smem_u32(&bars.full[b]), ((it + k) / RING) & 1, p.wait_budget, abort_flag, p.status, kDevTimeoutEpilogue);
            ok = __all_sync(kAll, ok);
            const uint4 *buf = reinterpret_cast<const uint4 *>(ring + b * CHUNK);
            const int n = item.vectors(k);
            float m;
            if (n == CHUNK / 16) {
                float v[EACH * VN];
#pragma unroll
                for (int q = 0; q < EACH; ++q) {
                    float u[VN];
                    Vec<T>::unpack(buf[tid + q * WORKERS], u);
#pragma unroll
                    for (int j = 0; j < VN; ++j) v[q * VN + j] = u[j];
                }
                m = run.take(v);
            } else {
                m = -INFINITY;
                for (int i = tid; i < n; i += WORKERS) {
                    float u[VN];
                    Vec<T>::unpack(buf[i], u);
                    m = fmaxf(m, run.take(u));
                }
                __syncwarp();
            }
            if constexpr (TOP) pick(buf, n, m, item.head + (item.v0 + k * (CHUNK / 16)) * VN);
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bars.empty[b]));
        }
        it += chunks;
        run.take(ends);
        const Sums mine = join<32>(run.r, c);
        // (a slot is written again two live items later, after the barrier that warp 0 meets when it has read it)
        const int slot = turn;
        turn ^= 1;
        if (lane == 0) sh[slot][warp] = mine;
        if constexpr (TOP) {
            list.offer(has_head, ends[0], tid);
            list.offer(has_tail, ends[1], item.tail + tid);
            list.end();
            lists[slot][warp][lane] = list.key;
            if (lane == 0) posts[turn][warp] = -INFINITY;  // for the next item; nobody reads them before the barrier
        }
        asm volatile("bar.sync 1, %0;" ::"n"(WORKERS) : "memory");
        if (warp == 0) {  // one warp ends the item; the others go on
            const Sums r = join<WARPS>(sh[slot][lane % WARPS], c);
            uint64_t key = 0;
            if constexpr (TOP) {
                key = lists[slot][0][lane];
#pragma unroll 1
                for (int q = 1; q < WARPS; ++q) key = merged(key, lists[slot][q][lane], lane);
            }
            if (parts == 1) {
                if (ok && lane == 0) put_sums(p, t, r, za, c);
                if (TOP && ok) put_list(p, t, r, key, lane, c);
            } else {
                Part *row = static_cast<Part *>(p.work) + t * parts;
                if (lane == 0) row[part].r = r;
                if (TOP) row[part].key[lane] = key;
                __threadfence();
                __syncwarp();
                int arrived = 0;
                if (lane == 0) arrived = atomicAdd(p.arrived + t, 1);
                arrived = __shfl_sync(kAll, arrived, 0);
                if (arrived == parts - 1) {
                    __threadfence();
                    if (lane == 0) p.arrived[t] = 0;
                    Sums all = {-INFINITY, 0.f, 0.f};
                    key = 0;
                    for (int q0 = 0; q0 < parts; q0 += 32) {
                        const int q = q0 + lane;
                        Sums one = {-INFINITY, 0.f, 0.f};
                        if (q < parts) one = {__ldcg(&row[q].r.m), __ldcg(&row[q].r.s), __ldcg(&row[q].r.t)};
                        one = join<32>(one, c);
                        const float m = fmaxf(all.m, one.m);
                        all = rebased(all, m, c);
                        one = rebased(one, m, c);
                        all.s += one.s;
                        all.t += one.t;
                    }
                    if constexpr (TOP) {
#pragma unroll 1
                        for (int q = 0; q < parts; ++q) key = merged(key, __ldcg(reinterpret_cast<const unsigned long long *>(&row[q].key[lane])), lane);
                    }
                    if (ok && lane == 0) put_sums(p, t, all, za, c);
                    if (TOP && ok) put_list(p, t, all, key, lane, c);
                }
            }
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(WORKERS + 32, RING_BLOCKS) logp_grad_ring_kernel(const LogpParams p) {
    constexpr int VN = Vec<T>::N;
    extern __shared__ __align__(128) uint8_t ring[];
    Ring &bars = *reinterpret_cast<Ring *>(ring + CHUNK * RING);
    __shared__ int abort_;
    volatile int32_t *abort_flag = &abort_;
    const int V = p.vocab, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    ring_init(bars, &abort_);
    pdl_next();
    pdl_wait();
    __syncthreads();
    const int64_t last = (int64_t)p.rows - 1;
    if (warp == WARPS) {
        // ------------------------------------------------------------ loads
        if (lane == 0) {
            uint64_t drop;
            asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(drop));
            uint32_t it = 0;
            bool ok = true;
            GradIn next = grad_in(p, blockIdx.x);
            for (int64_t t = blockIdx.x; t < p.rows && ok; t += gridDim.x) {
                const GradIn in = next;
                next = grad_in(p, min(t + gridDim.x, last));
                if (!grad_live(p, in)) continue;
                ok = ring_fill(ring, bars, Item<T>(static_cast<const T *>(p.logits) + t * p.ld, V, 0, 1), it, drop, p.wait_budget, abort_flag, p.status);
            }
            if (!ok) {
                for (int q = 0; q < 100; ++q) __nanosleep(1000);
            }
        }
        __syncwarp();
        return;
    }
    // ---------------------------------------------------------------- workers
    const int tid = threadIdx.x;
    uint32_t it = 0;
    bool ok = true;  // after a wait that ran out nothing is stored
    GradIn next = grad_in(p, blockIdx.x);
    for (int64_t t = blockIdx.x; t < p.rows; t += gridDim.x) {
        const GradIn in = next;
        next = grad_in(p, min(t + gridDim.x, last));
        const T *z = static_cast<const T *>(p.logits) + t * p.ld;
        T *dz = static_cast<T *>(p.dlogits) + t * p.ldd;
        if (in.a >= V && tid == 0) record_status(p.status, kDevFaultIndex);
        if (!grad_live(p, in)) {
            const Item<T> d(dz, V, 0, 1);
            uint4 *dv = reinterpret_cast<uint4 *>(dz + d.head);
            if (tid < d.head) Vec<T>::put(dz + tid, 0.f);
            for (int i = tid; i < d.v1; i += WORKERS) dv[i] = make_uint4(0u, 0u, 0u, 0u);
            for (int i = d.tail + tid; i < V; i += WORKERS) Vec<T>::put(dz + i, 0.f);
            continue;
        }
        const Slope g = slope(p, in);
        const Item<T> item(z, V, 0, 1);
        if (ok && tid < item.head) Vec<T>::put(dz + tid, g.one(Vec<T>::get(z + tid), tid));
        if (ok && item.tail + tid < V) Vec<T>::put(dz + item.tail + tid, g.one(Vec<T>::get(z + item.tail + tid), item.tail + tid));
        const bool same = (((uintptr_t)z ^ (uintptr_t)dz) & 15) == 0;
        const int chunks = item.chunks();
        for (int k = 0; k < chunks; ++k, ++it) {
            const uint32_t b = it % RING;
            if (ok) ok = mbar_wait_bounded(smem_u32(&bars.full[b]), (it / RING) & 1, p.wait_budget, abort_flag, p.status, kDevTimeoutEpilogue);
            const uint4 *buf = reinterpret_cast<const uint4 *>(ring + b * CHUNK);
            const int v0 = k * (CHUNK / 16), n = ok ? item.vectors(k) : 0;
            auto vector = [&](int i, const uint4 &u) {
                float w[VN], o[VN];
                Vec<T>::unpack(u, w);
                const int e0 = item.head + (v0 + i) * VN;
                g.vec(w, o, e0);
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
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bars.empty[b]));
        }
    }
}

template <typename K>
cudaError_t launch_ring(K kernel, bool (&attr_set)[64], const LogpParams &p, int64_t items, int num_sms, cudaStream_t s) {
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !attr_set[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingSmem);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) attr_set[dev] = true;
    }
    const int64_t most = (int64_t)RING_BLOCKS * num_sms;
    return launch_early(kernel, (int)(items < most ? items : most), WORKERS + 32, kRingSmem, s, p);
}
template <typename T, bool TOP>
cudaError_t launch_forward(const LogpParams &p, bool narrow, int num_sms, cudaStream_t s) {
    if (narrow) {
        const int64_t need = (p.rows + NT / 32 - 1) / (NT / 32), most = 8LL * num_sms;
        return launch_early(logp_warp_kernel<T, TOP>, (int)(need < most ? need : most), NT, 0, s, p);
    }
    static bool attr_set[64] = {};
    return launch_ring(logp_ring_kernel<T, TOP>, attr_set, p, (int64_t)p.rows * p.parts, num_sms, s);
}
template <typename T>
cudaError_t launch_backward(const LogpParams &p, bool narrow, int num_sms, cudaStream_t s) {
    if (narrow) {
        const int64_t need = (p.rows + NT / 32 - 1) / (NT / 32), most = 8LL * num_sms;
        return launch_early(logp_grad_warp_kernel<T>, (int)(need < most ? need : most), NT, 0, s, p);
    }
    static bool attr_set[64] = {};
    return launch_ring(logp_grad_ring_kernel<T>, attr_set, p, p.rows, num_sms, s);
}

bool narrow_rows(const LogpParams &p, int dtype) { return (int64_t)p.vocab * (dtype == 1 ? 2 : 4) <= 16384; }

}  // namespace

int logp_most_items(int num_sms) { return RING_BLOCKS * num_sms; }

// Parts of a row: as many as the blocks that would else stay idle, each of 8 KB at least.
int logp_parts(int64_t rows, int64_t vocab, int dtype, int num_sms) {
    const int64_t bytes = vocab * (dtype == 1 ? 2 : 4), slots = (int64_t)RING_BLOCKS * num_sms;
    if (bytes <= 16384 || rows >= slots) return 1;
    return (int)std::max<int64_t>(1, std::min(slots / rows, bytes / 8192));
}

cudaError_t launch_logp(const LogpParams &p, int dtype, bool backward, int num_sms, cudaStream_t s) {
    const bool narrow = narrow_rows(p, dtype);
    if (backward) return dtype == 1 ? launch_backward<__nv_bfloat16>(p, narrow, num_sms, s) : launch_backward<float>(p, narrow, num_sms, s);
    if (p.top) return dtype == 1 ? launch_forward<__nv_bfloat16, true>(p, narrow, num_sms, s) : launch_forward<float, true>(p, narrow, num_sms, s);
    return dtype == 1 ? launch_forward<__nv_bfloat16, false>(p, narrow, num_sms, s) : launch_forward<float, false>(p, narrow, num_sms, s);
}

}  // namespace cbd
