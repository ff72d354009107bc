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
// depend on the order of work.  The pass itself keeps little for them: each thread has
// its elements' maximum anyway, and that of its other chunks.  `top` elements lie at or
// above the top-th largest of 32 maxima, each of eight threads' elements (or of 64, of four);
// only threads whose maximum is there have candidates (some two dozen for 20
// alternatives), mostly in the one chunk that it came from, and that chunk's vectors are
// read again, from L2, by the warp that ends the row, while the others are at the next
// one.  It sorts the elements that reach the bound 32 at a time.  (8192 rows of 32768
// with 20 alternatives 125 us, without any 90: what the ending warps issue, and their
// second reading; candidates taken out during the pass against a rising bound 551,
// taken out by the workers after it 188.)
//
// Which lane sums which element goes by the row's address (what precedes its first 16
// bytes), and how many blocks take part by the number of rows: lse, logp and entropy of a
// row may differ in their last bits between addresses, row strides and batches.
//
// Wide rows stream through a ring of 16 KB buffers that one thread fills with
// bulk copies, as in the policy loss; where rows are few each is cut into parts, and
// the block that ends a row last joins the parts' sums and lists in their order.
// Rows up to 16 KB, many rows up to 32 KB, take a warp each (20000 rows of 12000 bf16 91 us,
// through the ring 155; 1500 of them 17, 15).
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
constexpr float kLn2 = 0.6931471805599453f;
constexpr uint32_t kAll = 0xffffffffu;

struct Sums {
    float m, s, t;
};
// r over the reference m instead of its own, which lies no higher.  (Between the type's lowest value and others the exponent
// is -inf in fp32: held where 2^up is 0 already, as 0 * -inf is not 0.)
__device__ __forceinline__ Sums rebased(const Sums &r, float m, float c) {
    const float up = fmaxf(Exps(m, c).shift(r.m, m), -200.f), f = ex2(up);
    return {m, r.s * f, fmaf(r.s, up, r.t) * f};
}
// the largest element of some vectors (what is no number counts last)
template <typename T, int N>
__device__ __forceinline__ float largest(const uint4 (&u)[N]) {
    if constexpr (sizeof(T) == 4) {
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < N; ++i) m = fmaxf(m, fmaxf(fmaxf(__uint_as_float(u[i].x), __uint_as_float(u[i].y)), fmaxf(__uint_as_float(u[i].z), __uint_as_float(u[i].w))));
        return m;
    } else {  // two at a time
        auto two = [](const uint32_t &w) { return *reinterpret_cast<const __nv_bfloat162 *>(&w); };
        __nv_bfloat162 m = two(u[0].x);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (i) m = __hmax2(m, two(u[i].x));
            m = __hmax2(__hmax2(m, two(u[i].y)), __hmax2(two(u[i].z), two(u[i].w)));
        }
        const float2 f = __bfloat1622float2(m);
        return fmaxf(f.x, f.y);
    }
}

__device__ __forceinline__ uint32_t ordered(float v) {
    const uint32_t b = __float_as_uint(v + 0.f);  // (-0 ties with 0)
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint64_t key) {
    const uint32_t b = (uint32_t)(key >> 32);
    return __uint_as_float(b & 0x80000000u ? b ^ 0x80000000u : ~b);
}
__device__ __forceinline__ uint32_t ordered_number(float v) { return ordered(v == v ? v : -INFINITY); }
__device__ __forceinline__ float warp_max(float m) { return value_of((uint64_t)__reduce_max_sync(kAll, ordered_number(m)) << 32); }

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pair(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 both(uint64_t x) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t x, uint64_t y, uint64_t z) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t x, uint64_t y) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    return r;
}
// A warp's elements: every lane has its own sums over the warp's reference, so that the reference is seldom moved (one for
// each lane was moved in most batches by some lane, for 1.5 instructions an element).  2^-inf * -inf is not 0: a batch whose
// t is no number is summed again with d held at -200, and so are the later ones (logits of -inf come many in a row or not at
// all).  take() is called by the whole warp.
struct Run {
    Sums r;
    float lim, room;
    bool held;
    Exps e;
    __device__ __forceinline__ Run(float c, float room_) : r{-INFINITY, 0.f, 0.f}, lim(-INFINITY), room(room_), held(false), e(-INFINITY, c) {}
    template <int N>
    __device__ __forceinline__ float2 plain(const float (&v)[N]) const {
        const uint64_t c2 = pair(e.c, e.c), off2 = pair(-e.off, -e.off);
        uint64_t s2 = 0, t2 = 0;
#pragma unroll
        for (int i = 0; i + 1 < N; i += 2) {
            const uint64_t d2 = fma2(pair(v[i], v[i + 1]), c2, off2);
            const float2 d = both(d2);
            const uint64_t p2 = pair(ex2(d.x), ex2(d.y));
            s2 = add2(s2, p2);
            t2 = fma2(p2, d2, t2);
        }
        const float2 s = both(s2), t = both(t2);
        return make_float2(s.x + s.y, t.x + t.y);
    }
    template <int N>
    __device__ __forceinline__ float2 careful(const float (&v)[N]) const {
        float s = 0.f, t = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float d = e.near ? fmaf(v[i], e.c, -e.off) : (v[i] - e.base) * e.c, p = ex2(d);
            s += p;
            t = fmaf(p, fmaxf(d, -200.f), t);
        }
        return make_float2(s, t);
    }
    // elements and their maximum; lanes without any take part with values whose terms are 0
    template <int N>
    __device__ __forceinline__ void take(float (&v)[N], float m, bool there = true) {
        if (__any_sync(kAll, m > lim)) {
            m = warp_max(m);
            r = rebased(r, m, e.c);
            e = Exps(m, e.c);
            lim = m + room;
        }
        const float dead = e.near && r.m != -INFINITY ? r.m - 300.f * room : -INFINITY;
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = there ? v[k] : dead;
        float2 x = make_float2(0.f, __int_as_float(0x7fffffff));
        if (N % 2 == 0 && e.near && !held) x = plain(v);
        if (__any_sync(kAll, !(x.y == x.y))) {
            x = careful(v);
            held = true;
        }
        r.s += x.x;
        r.t += x.y;
    }
    template <typename T, int N>
    __device__ __forceinline__ float take(const uint4 (&u)[N], bool there = true) {
        constexpr int VN = Vec<T>::N;
        float v[N * VN];
#pragma unroll
        for (int q = 0; q < N; ++q) {
            float w[VN];
            Vec<T>::unpack(u[q], w);
#pragma unroll
            for (int k = 0; k < VN; ++k) v[q * VN + k] = w[k];
        }
        const float m = there ? largest<T>(u) : -INFINITY;
        take(v, m, there);
        return m;
    }
};
// The lanes' sums over their common reference, in a fixed order; every lane gets them.
__device__ __forceinline__ Sums total(Sums r) {
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        r.s += __shfl_xor_sync(kAll, r.s, d);
        r.t += __shfl_xor_sync(kAll, r.t, d);
    }
    return r;
}
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
template <typename K>
__device__ __forceinline__ K merged(K a, K b, int lane) {
    const K o = __shfl_sync(kAll, b, 31 - lane);
    a = a > o ? a : o;
#pragma unroll
    for (int j = 16; j; j >>= 1) a = exchange(a, j, (lane & j) == 0);
    return a;
}
// A bound of the `top` largest from two elements of each lane (as ordered()): the top-th of the lanes' larger ones; for many
// the top-th of all 64, above which there are 64 ln(64 / (64 - top)) elements to expect instead of 32 ln(32 / (32 - top)): 24, 31
// at 20, 44, 130 at 32.
// For few the maximum is taken off again and again, which takes less than a sorting network (8192 rows of 32768 bf16, one
// alternative 104 us, sorted 108; eight 110, 114; ten 112, 115; by the maximum sixteen 122, sorted 120.  4000 rows of 4096 fp32,
// three 24.9, 25.2; ten 27.8, 27.3.)
__device__ __forceinline__ uint32_t bound_of(uint32_t a, uint32_t b, int top, int lane) {
    if (top <= 10) {
        uint32_t x = max(a, b), m = 0;
#pragma unroll 1
        for (int i = 0; i < top; ++i) {
            m = __reduce_max_sync(kAll, x);
            if (lane == __ffs(__ballot_sync(kAll, x == m)) - 1) x = 0;
        }
        return m;
    }
    const uint32_t s = sorted_falling(top > 16 ? a : max(a, b), lane);
    return __shfl_sync(kAll, top > 16 ? merged(s, sorted_falling(b, lane), lane) : s, top - 1);
}
constexpr int kQueue = 64;
// A warp's best: lane i has the i-th, 0 where there is none; what came last waits in the queue.
struct List {
    uint64_t key, last;  // last: the top-th
    float bound;         // of values that may still enter
    int count;           // queued
    uint64_t *queue;     // [kQueue], the warp's own
    int top, lane;
    __device__ __forceinline__ List(uint64_t *q, int top_, float bound_, int lane_) : key(0), last(0), bound(bound_), count(0), queue(q), top(top_), lane(lane_) {}
    __device__ __forceinline__ void flush() {
        __syncwarp();
        const int first = count > 32 ? count - 32 : 0;
        const uint64_t mine = first + lane < count ? queue[first + lane] : 0;
        __syncwarp();
        count = first;
        key = merged(key, sorted_falling(mine, lane), lane);
        const uint64_t place = __shfl_sync(kAll, key, top - 1);
        if (place > last) {
            last = place;
            bound = fmaxf(bound, value_of(last));
        }
    }
    // (by the whole warp)
    __device__ __forceinline__ void offer(bool there, float v, int index) { offer(there && v >= bound ? key_of(v, (uint32_t)index) : 0); }
    __device__ __forceinline__ void offer(uint64_t k) {
        const bool in = k > last;
        const uint32_t who = __ballot_sync(kAll, in);
        if (who == 0) return;
        if (in) queue[count + __popc(who & ((1u << lane) - 1))] = k;
        count += __popc(who);
        if (count >= 32) flush();
    }
    // a vector's elements, the first of them with this index; `there` goes by lane
    template <typename T>
    __device__ __forceinline__ void offer_vector(bool there, const uint4 &u, int index) {
        constexpr int VN = Vec<T>::N;
        const uint4 one[1] = {u};
        if (!__any_sync(kAll, there && largest<T>(one) >= bound)) return;
        float v[VN];
        Vec<T>::unpack(u, v);
        uint32_t high = 0;
#pragma unroll
        for (int k = 0; k < VN; ++k) high |= (there && v[k] >= bound ? 1u : 0u) << k;
        while (__any_sync(kAll, high != 0)) {  // mostly once or never
            const int k = high ? __ffs(high) - 1 : 0;
            float x = v[0];
#pragma unroll
            for (int j = 1; j < VN; ++j) x = k == j ? v[j] : x;
            offer(high != 0, x, index + k);
            high &= high - 1;
        }
    }
    __device__ __forceinline__ void end() {
        while (count > 0) flush();
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
    constexpr int UNR = 2;  // vectors of a lane in a batch (four: 65536 rows of 4096 bf16 107 us instead of 97, of 1000 69 instead of 46)
    __shared__ uint64_t queues[TOP ? ROWS : 1][kQueue];
    const int lane = threadIdx.x % 32, sub = threadIdx.x / 32;
    const int V = p.vocab;
    const float c = p.scale * kLog2e, room = 1.f / c;
    pdl_next();
    pdl_wait();
    const int64_t step = (int64_t)gridDim.x * ROWS;
    auto token = [&](int64_t t) { return p.tokens ? p.tokens[min(t, (int64_t)p.rows - 1)] : 0; };  // (read a row ahead)
    int following = token((int64_t)blockIdx.x * ROWS + sub);
    for (int64_t t = (int64_t)blockIdx.x * ROWS + sub; t < p.rows; t += step) {
        const T *z = static_cast<const T *>(p.logits) + t * p.ld;
        const int a = following;
        following = token(t + step);
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
        Run run(c, room);
        const bool has_head = lane < head, has_tail = tail + lane < V;
        float ends[2] = {has_head ? Vec<T>::get(z + lane) : -INFINITY, has_tail ? Vec<T>::get(z + tail + lane) : -INFINITY};
        float best = -INFINITY, second = -INFINITY;  // of the batches, and of the others
        int where = 0;
        auto seen = [&](float m, int i) {
            if constexpr (TOP) {
                second = fmaxf(second, fminf(best, m));
                where = m > best ? i : where;
                best = fmaxf(best, m);
            }
        };
        uint4 next[UNR];
        auto fetch = [&](int i) {
#pragma unroll
            for (int q = 0; q < UNR; ++q) next[q] = zv[min(i + q * 32, nv - 1)];
        };
        if (nv > 0) fetch(lane);
        for (int i = lane; i - lane < nv; i += UNR * 32) {
            uint4 u[UNR];
#pragma unroll
            for (int q = 0; q < UNR; ++q) u[q] = next[q];
            if (i - lane + UNR * 32 < nv) fetch(i + UNR * 32);
            if (i - lane + UNR * 32 <= nv) {
                seen(run.template take<T>(u), i);
                continue;
            }
            float m = -INFINITY;
#pragma unroll
            for (int q = 0; q < UNR; ++q) {
                if (i - lane + q * 32 >= nv) break;
                const uint4 one[1] = {u[q]};
                m = fmaxf(m, run.template take<T>(one, i + q * 32 < nv));
            }
            seen(m, i);
        }
        if (__any_sync(kAll, has_head || has_tail)) run.take(ends, fmaxf(ends[0], ends[1]));
        const Sums r = total(run.r);
        if constexpr (TOP) {
            // Candidates are the lanes' ends, and mostly one batch of a lane, else all of its vectors, read by the warp
            // or, where these are few beside the lanes and the candidates many, by the lane (20000 rows of bf16, by the lane and by the
            // warp: 1000 columns with five alternatives 39 and 35 us, with 20 47 and 51, with 32 54 and 59; 500 with 20 42 and 41;
            // 2000 with 20 66 and 62).
            const uint32_t mine = ordered_number(best), other = ordered_number(second);
            const uint32_t low = bound_of(ordered_number(fmaxf(best, fmaxf(ends[0], ends[1]))), other, p.top, lane);
            const bool in = mine >= low, few = nv <= 128 && p.top > 16, more = in && (few || other >= low);
            List list(queues[sub], p.top, value_of((uint64_t)low << 32), lane);
            list.offer(has_head, ends[0], lane);
            list.offer(has_tail, ends[1], tail + lane);
            uint4 u[UNR];
#pragma unroll
            for (int q = 0; q < UNR; ++q) {
                u[q] = make_uint4(0u, 0u, 0u, 0u);
                if (in && !more && where + q * 32 < nv) u[q] = zv[where + q * 32];
            }
#pragma unroll
            for (int q = 0; q < UNR; ++q) list.offer_vector<T>(in && !more && where + q * 32 < nv, u[q], head + (where + q * 32) * VN);
            uint32_t who = __ballot_sync(kAll, more);
            if (few || __popc(who) * ((nv + 1023) / 1024) > (nv + 31) / 32) {
                for (int k = lane; k - lane < nv; k += 32) {
                    const bool there = more && k < nv;
                    uint4 w = make_uint4(0u, 0u, 0u, 0u);
                    if (there) w = zv[k];
                    list.offer_vector<T>(there, w, head + k * VN);
                }
                who = 0;
            }
            for (; who; who &= who - 1) {
                const int of = __ffs(who) - 1;
                for (int k = of + lane * 32; k - lane * 32 < nv; k += 1024) {
                    uint4 w = make_uint4(0u, 0u, 0u, 0u);
                    if (k < nv) w = zv[k];
                    list.offer_vector<T>(k < nv, w, head + k * VN);
                }
            }
            list.end();
            put_list(p, t, r, list.key, lane, c);
        }
        if (lane == 0) put_sums(p, t, r, za, c);
        __syncwarp();
    }
}

// dz = p (a + b u) + cs [chosen], u = scale z - lse with scale z rounded first, as it is in lse where that is large: u does not
// pass 0 there.  (With one rounding, rows of the type's lowest value had u anywhere within the last bit of lse, 2^103, and p infinite.)
struct Slope {
    float scale, lse, a, b, cs;
    int chosen;
    __device__ __forceinline__ float at(float z) const {
        const float u = __fmul_rn(z, scale) - lse;
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
    r.h = p.grad_entropy ? p.entropy_in[t] : 0.f;  // (unasked for otherwise, whatever it holds)
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
    constexpr int UNR = 4;  // 16-byte loads of a thread in flight
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
constexpr int CHUNK = 16384, WORKERS = 256;
constexpr int WARPS = WORKERS / 32;
constexpr int EACH = CHUNK / 16 / WORKERS;  // vectors of a thread in a chunk
constexpr int MOST_RING = 6;
// Blocks per SM, buffers of a block, warps that end items and the slots that they get them in.  (8192 rows of 32768 bf16: two
// blocks of six buffers 90 us, without the exponentials 83; three of four 96.  With 20 alternatives and three warps to end
// them 125, with two 147.)
constexpr int BLOCKS = 2;
template <bool TOP>
struct Shape {
    static constexpr int RING = 6, ENDS = TOP ? 3 : 1, SLOTS = TOP ? 3 : 2;
    static_assert(ENDS <= SLOTS, "a warp waits for the use of a slot that comes next (the parity of a later one reads as done)");
    static constexpr int THREADS = WORKERS + 32 + 32 * ENDS, SMEM = CHUNK * RING + 256;
};
// the gradient's
constexpr int GRAD_BLOCKS = 3, GRAD_RING = 4, GRAD_SMEM = CHUNK * GRAD_RING + 256;

template <typename T>
struct Item {
    const T *z;
    int head, v0, v1, tail;
    bool first, last;
    __device__ __forceinline__ Item(const T *z_, int V, int part, int parts) : z(z_) {
        head = min(V, (int)((16 - ((uintptr_t)z & 15)) % 16 / sizeof(T)));
        const int nv = (V - head) / Vec<T>::N;
        v0 = 0;
        v1 = nv;
        if (parts > 1) {
            const int each = nv / parts, more = nv - each * parts;  // the first `more` parts have one more
            v0 = each * part + min(part, more);
            v1 = v0 + each + (part < more ? 1 : 0);
        }
        tail = head + nv * Vec<T>::N;
        first = part == 0;
        last = part == parts - 1;
    }
    __device__ __forceinline__ int chunks() const { return (v1 - v0 + CHUNK / 16 - 1) / (CHUNK / 16); }  // (in vectors: a row has up to 2^32 bytes)
    __device__ __forceinline__ int vectors(int chunk) const { return min(CHUNK / 16, v1 - v0 - chunk * (CHUNK / 16)); }
};

struct Ring {
    uint64_t full[MOST_RING], empty[MOST_RING];
    uint64_t filled[4], free[4];  // slots of the items' ends
};
template <int RING>
__device__ __forceinline__ void ring_init(Ring &r, int *abort_) {
    if (threadIdx.x == 0) {
        for (int i = 0; i < RING; ++i) {
            mbar_init(smem_u32(&r.full[i]), 1);
            mbar_init(smem_u32(&r.empty[i]), WARPS);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(smem_u32(&r.filled[i]), WARPS);
            mbar_init(smem_u32(&r.free[i]), 1);
        }
        *abort_ = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
}
// one thread: the item's chunks into the ring
template <int RING, typename T>
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

// A block's items: row and part, and the row's token, read an item ahead.
struct Walk {
    const LogpParams &p;
    int64_t at, items;
    int next;
    __device__ __forceinline__ explicit Walk(const LogpParams &p_) : p(p_), at(blockIdx.x), items((int64_t)p_.rows * p_.parts), next(token(min(at, items - 1))) {}
    __device__ __forceinline__ int64_t row(int64_t i) const { return p.parts == 1 ? i : (int64_t)((uint32_t)i / (uint32_t)p.parts); }  // (parts only where items are few)
    __device__ __forceinline__ int token(int64_t i) const { return p.tokens ? p.tokens[row(i)] : 0; }
    __device__ __forceinline__ bool take(int64_t &t, int &part, int &of) {
        if (at >= items) return false;
        t = row(at);
        part = (int)(at - t * p.parts);
        of = next;
        at += gridDim.x;
        next = token(min(at, items - 1));
        return true;
    }
    __device__ __forceinline__ bool live(int of) const { return (unsigned)of < (unsigned)p.vocab; }
};

static_assert(sizeof(Ring) <= 256, "behind the buffers");

// A part's share of its row, in the workspace.
struct __align__(16) Part {
    Sums r;
    uint32_t pad;
    uint64_t key[32];
};
static_assert(sizeof(Part) == kLogpPart, "workspace");

constexpr int kFewParts = 4;
// The largest of all parts' lists, by one warp, a part to a lane.  (Of a few parts, whose lists are read beside their sums: merged one by
// one.  Rows of 128000 bf16, five alternatives, the other way: 150 rows of two parts 15.6, 18.0 us; 100 of three 13.6, 15.9; 76 of four
// 13.0, 15.3.  Merging would still be ahead at five to eight, 60 rows of five 12.4, 13.8, 38 of eight 11.7, 12.2, for eight more
// registers a lane.)
__device__ __forceinline__ uint64_t best_of_parts(const Part *row, int parts, int top, uint64_t *queue, int lane) {
    List list(queue, top, -INFINITY, lane);
    for (int q0 = 0; q0 < parts; q0 += 32) {
        const bool there = q0 + lane < parts;
        const unsigned long long *from = reinterpret_cast<const unsigned long long *>(row[there ? q0 + lane : 0].key);
        uint64_t k[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) k[i] = there ? __ldcg(from + i) : 0;
        // `top` keys lie at or above the top-th of the parts' first ones
        const uint64_t low = __shfl_sync(kAll, sorted_falling(k[0], lane), top - 1);
        if (low > list.last) list.last = low - 1;
        for (int i = 0; i < 32; ++i) {
            const uint64_t x = i < 4 ? k[0] : there ? __ldcg(from + i) : 0;
            k[0] = k[1], k[1] = k[2], k[2] = k[3];
            if (!__any_sync(kAll, x > list.last)) break;
            list.offer(x);
        }
    }
    list.end();
    return list.key;
}

template <typename T, bool TOP>
__global__ void __launch_bounds__(Shape<TOP>::THREADS, BLOCKS) logp_ring_kernel(const LogpParams p) {
    using S = Shape<TOP>;
    constexpr int VN = Vec<T>::N, RING = S::RING;
    extern __shared__ __align__(128) uint8_t ring[];
    Ring &bars = *reinterpret_cast<Ring *>(ring + CHUNK * RING);
    __shared__ Sums sh[S::SLOTS][WARPS];
    // of each thread, as ordered(): its largest element, the largest of its other chunks; the chunk
    __shared__ uint32_t best_of[TOP ? S::SLOTS : 1][TOP ? WORKERS : 1], second_of[TOP ? S::SLOTS : 1][TOP ? WORKERS : 1], chunk_of[TOP ? S::SLOTS : 1][TOP ? WORKERS : 1];
    __shared__ uint64_t queues[TOP ? S::ENDS : 1][kQueue];
    __shared__ uint32_t chosen[TOP ? S::ENDS : 1][WORKERS];
    __shared__ int abort_;
    volatile int32_t *abort_flag = &abort_;
    const int V = p.vocab, warp = threadIdx.x / 32, lane = threadIdx.x % 32, parts = p.parts;
    const float c = p.scale * kLog2e, room = 1.f / c;
    ring_init<RING>(bars, &abort_);
    pdl_next();
    pdl_wait();
    __syncthreads();
    Walk walk(p);
    int64_t t;
    int part, token;
    if (warp == WARPS) {
        // ------------------------------------------------------------ loads
        if (lane == 0) {
            uint64_t policy;  // alternatives are read again from L2
            if (TOP)
                asm("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(policy));
            else
                asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
            uint32_t it = 0;
            bool ok = true;
            while (ok && walk.take(t, part, token)) {
                if (!walk.live(token)) continue;
                ok = ring_fill<RING>(ring, bars, Item<T>(static_cast<const T *>(p.logits) + t * p.ld, V, part, parts), it, policy, p.wait_budget, abort_flag, p.status);
            }
            if (!ok) {
                for (int q = 0; q < 100; ++q) __nanosleep(1000);
            }
        }
        __syncwarp();
        return;
    }
    // Workers and the warps that end the items hand the slots to and fro; the n-th live item of a block has slot n % SLOTS
    // and warp n % ENDS.
    int n = 0;
    bool ok = true;  // after a wait that ran out: nothing is stored, the barriers are kept
    if (warp > WARPS) {
        // ------------------------------------------------------------ ends of items
        const int me = warp - WARPS - 1;
        while (walk.take(t, part, token)) {
            if (!walk.live(token)) {
                if (part == 0 && me == 0) {
                    if (lane == 0 && token >= V) record_status(p.status, kDevFaultIndex);
                    put_masked(p, t, lane);
                }
                continue;
            }
            const int slot = n % S::SLOTS, turn = n % S::ENDS, use = n / S::SLOTS;
            ++n;
            if (turn != me) continue;
            const T *z = static_cast<const T *>(p.logits) + t * p.ld;
            const float za = p.logp ? Vec<T>::get(z + token) : 0.f;
            if (ok) ok = mbar_wait_bounded(smem_u32(&bars.filled[slot]), use & 1, p.wait_budget, abort_flag, p.status, kDevTimeoutPartial);
            ok = __all_sync(kAll, ok);
            Sums r = join<WARPS>(sh[slot][lane % WARPS], c);
            uint64_t key = 0;
            if constexpr (TOP) {
                const Item<T> item(z, V, part, parts);
                uint32_t m[WARPS], high[2] = {0, 0};
#pragma unroll
                for (int k = 0; k < WARPS; ++k) {
                    m[k] = best_of[slot][k * 32 + lane];
                    high[k % 2] = max(high[k % 2], m[k]);
                }
                const uint32_t low = bound_of(high[0], high[1], p.top, lane);
                // where candidates are: mostly one chunk of a thread, else all of its chunks
                int threads = 0;
                uint32_t many = 0;  // bit k: thread 32 k + lane has them in several chunks
#pragma unroll
                for (int k = 0; k < WARPS; ++k) {
                    const int of = k * 32 + lane;
                    const bool in = m[k] >= low, more = in && second_of[slot][of] >= low;
                    many |= (more ? 1u : 0u) << k;
                    const uint32_t who = __ballot_sync(kAll, in && !more);
                    if (who >> lane & 1) chosen[me][threads + __popc(who & ((1u << lane) - 1))] = chunk_of[slot][of] * (CHUNK / 16) + of;
                    threads += __popc(who);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bars.free[slot]));
                List list(queues[me], p.top, value_of((uint64_t)low << 32), lane);
                const bool has_head = item.first && lane < item.head, has_tail = item.last && item.tail + lane < V;
                list.offer(has_head, has_head ? Vec<T>::get(z + lane) : 0.f, lane);
                list.offer(has_tail, has_tail ? Vec<T>::get(z + item.tail + lane) : 0.f, item.tail + lane);
                const uint4 *row = reinterpret_cast<const uint4 *>(z + item.head) + item.v0;
                const int nv = item.v1 - item.v0;
                constexpr int AHEAD = 4;
                for (int j = lane; j - lane < threads * EACH; j += 32 * AHEAD) {
                    uint4 u[AHEAD];
                    int at[AHEAD];
#pragma unroll
                    for (int q = 0; q < AHEAD; ++q) {
                        const int k = j + 32 * q;
                        at[q] = k < threads * EACH ? (int)chosen[me][k / EACH] + k % EACH * WORKERS : nv;
                        u[q] = make_uint4(0u, 0u, 0u, 0u);
                        if (at[q] < nv) u[q] = __ldcg(row + at[q]);
                    }
#pragma unroll
                    for (int q = 0; q < AHEAD; ++q)
                        if (j - lane + 32 * q < threads * EACH) list.offer_vector<T>(at[q] < nv, u[q], item.head + (item.v0 + at[q]) * VN);
                }
#pragma unroll 1
                for (int k = 0; k < WARPS; ++k)
                    for (uint32_t who = __ballot_sync(kAll, many >> k & 1); who; who &= who - 1) {
                        const int of = k * 32 + __ffs(who) - 1;
                        for (int j = of + lane * WORKERS; j - lane * WORKERS < nv; j += 32 * WORKERS) {
                            uint4 u = make_uint4(0u, 0u, 0u, 0u);
                            if (j < nv) u = __ldcg(row + j);
                            list.offer_vector<T>(j < nv, u, item.head + (item.v0 + j) * VN);
                        }
                    }
                list.end();
                key = list.key;
            } else {
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bars.free[slot]));
            }
            if (parts > 1) {
                Part *row = static_cast<Part *>(p.work) + t * parts;
                if (lane == 0) row[part].r = r;
                if (TOP) row[part].key[lane] = key;
                __threadfence();
                __syncwarp();
                int arrived = 0;
                if (lane == 0) arrived = atomicAdd(p.arrived + t, 1);
                arrived = __shfl_sync(kAll, arrived, 0);
                if (arrived != parts - 1) continue;
                __threadfence();
                if (lane == 0) p.arrived[t] = 0;
                uint64_t lists[TOP ? kFewParts : 1];
                if constexpr (TOP) {
#pragma unroll
                    for (int q = 0; q < kFewParts; ++q) lists[q] = parts <= kFewParts && q < parts ? __ldcg(reinterpret_cast<const unsigned long long *>(&row[q].key[lane])) : 0;
                }
                r = {-INFINITY, 0.f, 0.f};
                for (int q0 = 0; q0 < parts; q0 += 32) {
                    const int q = q0 + lane;
                    Sums one = {-INFINITY, 0.f, 0.f};
                    if (q < parts) one = {__ldcg(&row[q].r.m), __ldcg(&row[q].r.s), __ldcg(&row[q].r.t)};
                    one = join<32>(one, c);
                    const float m = fmaxf(r.m, one.m);
                    r = rebased(r, m, c);
                    one = rebased(one, m, c);
                    r.s += one.s;
                    r.t += one.t;
                }
                if constexpr (TOP) {
                    if (parts <= kFewParts) {
                        key = lists[0];
#pragma unroll
                        for (int q = 1; q < kFewParts; ++q)
                            if (q < parts) key = merged(key, lists[q], lane);
                    } else {
                        key = best_of_parts(row, parts, p.top, queues[me], lane);
                    }
                }
            }
            if (!ok || *abort_flag) continue;
            if (lane == 0) put_sums(p, t, r, za, c);
            if (TOP) put_list(p, t, r, key, lane, c);
        }
        return;
    }
    // ---------------------------------------------------------------- workers
    const int tid = threadIdx.x;
    uint32_t it = 0;
    while (walk.take(t, part, token)) {
        if (!walk.live(token)) continue;
        const T *z = static_cast<const T *>(p.logits) + t * p.ld;
        const Item<T> item(z, V, part, parts);
        // the row's ends: at most one element of a thread before and after the vectors
        const bool has_head = item.first && tid < item.head, has_tail = item.last && item.tail + tid < V;
        float ends[2] = {has_head ? Vec<T>::get(z + tid) : -INFINITY, has_tail ? Vec<T>::get(z + item.tail + tid) : -INFINITY};
        Run run(c, room);
        float best = -INFINITY, second = -INFINITY;
        int where = 0;
        const int chunks = item.chunks();
        for (int k = 0; k < chunks; ++k, ++it) {
            const uint32_t b = it % RING;
            if (ok) ok = mbar_wait_bounded(smem_u32(&bars.full[b]), (it / RING) & 1, p.wait_budget, abort_flag, p.status, kDevTimeoutEpilogue);
            ok = __all_sync(kAll, ok);
            const uint4 *buf = reinterpret_cast<const uint4 *>(ring + b * CHUNK);
            const int count = item.vectors(k);
            float m = -INFINITY;
            if (count == CHUNK / 16) {
                uint4 u[EACH];
#pragma unroll
                for (int q = 0; q < EACH; ++q) u[q] = buf[tid + q * WORKERS];
                m = run.template take<T>(u);
            } else {
                for (int i = tid; i - lane < count; i += WORKERS) {
                    const uint4 u[1] = {buf[min(i, count - 1)]};
                    m = fmaxf(m, run.template take<T>(u, i < count));
                }
            }
            if constexpr (TOP) {
                second = fmaxf(second, fminf(best, m));
                where = m > best ? k : where;
                best = fmaxf(best, m);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bars.empty[b]));
        }
        if (__any_sync(kAll, has_head || has_tail)) run.take(ends, fmaxf(ends[0], ends[1]));
        const Sums mine = total(run.r);
        const int slot = n % S::SLOTS, use = n / S::SLOTS;
        ++n;
        if (ok) ok = mbar_wait_bounded(smem_u32(&bars.free[slot]), (use & 1) ^ 1, p.wait_budget, abort_flag, p.status, kDevTimeoutEpilogue);
        ok = __all_sync(kAll, ok);
        if (lane == 0) sh[slot][warp] = mine;
        if constexpr (TOP) {
            best_of[slot][tid] = ordered_number(best);
            second_of[slot][tid] = ordered_number(second);
            chunk_of[slot][tid] = (uint32_t)where;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars.filled[slot]));
    }
}

template <typename T>
__global__ void __launch_bounds__(WORKERS + 32, GRAD_BLOCKS) logp_grad_ring_kernel(const LogpParams p) {
    constexpr int VN = Vec<T>::N, RING = GRAD_RING;
    extern __shared__ __align__(128) uint8_t ring[];
    Ring &bars = *reinterpret_cast<Ring *>(ring + CHUNK * RING);
    __shared__ int abort_;
    volatile int32_t *abort_flag = &abort_;
    const int V = p.vocab, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    ring_init<RING>(bars, &abort_);
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
                ok = ring_fill<RING>(ring, bars, Item<T>(static_cast<const T *>(p.logits) + t * p.ld, V, 0, 1), it, drop, p.wait_budget, abort_flag, p.status);
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
cudaError_t launch_ring(K kernel, bool (&attr_set)[64], const LogpParams &p, int64_t items, int blocks, int threads, int smem, cudaStream_t s) {
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !attr_set[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) attr_set[dev] = true;
    }
    return launch_early(kernel, (int)(items < blocks ? items : blocks), threads, smem, s, p);
}
template <typename T, bool TOP>
cudaError_t launch_forward(const LogpParams &p, bool narrow, int num_sms, cudaStream_t s) {
    if (narrow) {
        const int64_t need = (p.rows + NT / 32 - 1) / (NT / 32), most = 8LL * num_sms;
        return launch_early(logp_warp_kernel<T, TOP>, (int)(need < most ? need : most), NT, 0, s, p);
    }
    static bool attr_set[64] = {};
    return launch_ring(logp_ring_kernel<T, TOP>, attr_set, p, (int64_t)p.rows * p.parts, BLOCKS * num_sms, Shape<TOP>::THREADS, Shape<TOP>::SMEM, s);
}
template <typename T>
cudaError_t launch_backward(const LogpParams &p, bool narrow, int num_sms, cudaStream_t s) {
    if (narrow) {
        const int64_t need = (p.rows + NT / 32 - 1) / (NT / 32), most = 8LL * num_sms;
        return launch_early(logp_grad_warp_kernel<T>, (int)(need < most ? need : most), NT, 0, s, p);
    }
    static bool attr_set[64] = {};
    return launch_ring(logp_grad_ring_kernel<T>, attr_set, p, p.rows, GRAD_BLOCKS * num_sms, WORKERS + 32, GRAD_SMEM, s);
}

// A warp each: rows of up to 16 KB, and of up to 32 KB where there are sixteen to an SM.
bool narrow_rows(const LogpParams &p, int dtype, int num_sms) {
    const int64_t bytes = (int64_t)p.vocab * (dtype == 1 ? 2 : 4);
    return bytes <= 16384 || (bytes <= 32768 && p.rows >= 16 * num_sms);
}

}  // namespace

int logp_most_items(int num_sms) { return BLOCKS * num_sms; }

// Parts of a row: as many as the blocks that would else stay idle, each of 8 KB at least.  (64 rows of 128000 bf16 9.5 us, two
// or three items to a block 11.3 and 13.3; one row with 20 alternatives 11.4, in parts of 4 KB 13.5, of 16 KB 12.4.)
int logp_parts(int64_t rows, int64_t vocab, int dtype, int num_sms) {
    const int64_t bytes = vocab * (dtype == 1 ? 2 : 4), slots = (int64_t)BLOCKS * num_sms;
    if (bytes <= 16384 || rows >= slots) return 1;
    return (int)std::max<int64_t>(1, std::min(slots / rows, bytes / 8192));
}

cudaError_t launch_logp(const LogpParams &p, int dtype, bool backward, int num_sms, cudaStream_t s) {
    const bool narrow = narrow_rows(p, dtype, num_sms);
    if (backward) return dtype == 1 ? launch_backward<__nv_bfloat16>(p, narrow, num_sms, s) : launch_backward<float>(p, narrow, num_sms, s);
    if (p.top) return dtype == 1 ? launch_forward<__nv_bfloat16, true>(p, narrow, num_sms, s) : launch_forward<float, true>(p, narrow, num_sms, s);
    return dtype == 1 ? launch_forward<__nv_bfloat16, false>(p, narrow, num_sms, s) : launch_forward<float, false>(p, narrow, num_sms, s);
}

}  // namespace cbd
