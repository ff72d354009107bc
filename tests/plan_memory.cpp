// plan_memory.cpp -- the library's plan code on a CUDA runtime that does nothing
// before it must: copies and memsets wait in their stream's queue until something
// synchronises that stream, as a busy GPU may let them.  A program for
// test_plan_memory.py; argv[1] names the plan to make.  Ends with 0 if create left
// nothing queued, every buffer that create writes was written, and a run with
// another device current is refused.
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <map>
#include <string>
#include <vector>

#include <cuda.h>
#include <cuda_runtime.h>

#include "../conv2d_backward_implicit_bwd_gb300/csrc/internal.h"
#ifdef TRAIN
#include "../conv2d_backward_implicit_bwd_gb300/csrc/train.h"
#include "../include/conv_bwd_train.h"
#endif
#include "../include/conv_bwd_data.h"

namespace {

struct Op {
    void *dst;
    std::vector<uint8_t> bytes;
};
std::map<cudaStream_t, std::vector<Op>> queued;  // nullptr: the legacy default stream
std::map<void *, size_t> held;                   // device memory, 0xA5 until written
int written = 0, device = 0;

cudaError_t put(cudaStream_t s, void *dst, std::vector<uint8_t> bytes) {
    queued[s].push_back({dst, std::move(bytes)});
    return cudaSuccess;
}
int pending() {
    int n = 0;
    for (auto &q : queued) n += (int)q.second.size();
    return n;
}
int encode(...) { return 0; }
#ifdef TRAIN
void *at(int i) { return (void *)((uintptr_t)i << 24); }  // an address that nothing reads
#endif

}  // namespace

extern "C" {
void not_reached(void) {
    printf("a call that create has no use for\n");
    exit(3);
}
cudaError_t cudaGetDeviceCount(int *n) { return *n = 1, cudaSuccess; }
cudaError_t cudaGetDevice(int *d) { return *d = device, cudaSuccess; }
cudaError_t cudaSetDevice(int) { return cudaSuccess; }
cudaError_t cudaGetLastError(void) { return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int *v, cudaDeviceAttr a, int) {
    return *v = a == cudaDevAttrMultiProcessorCount ? 152 : a == cudaDevAttrClockRate ? 2000000 : 1, cudaSuccess;
}
cudaError_t cudaMalloc(void **p, size_t n) {
    *p = malloc(n);
    if (!*p) return cudaErrorMemoryAllocation;
    memset(*p, 0xA5, n);
    held[*p] = n;
    return cudaSuccess;
}
cudaError_t cudaFree(void *p) { return held.erase(p), free(p), cudaSuccess; }
cudaError_t cudaMemsetAsync(void *p, int v, size_t n, cudaStream_t s) { return put(s, p, std::vector<uint8_t>(n, (uint8_t)v)); }
cudaError_t cudaMemset(void *p, int v, size_t n) { return cudaMemsetAsync(p, v, n, nullptr); }
cudaError_t cudaMemcpyAsync(void *d, const void *h, size_t n, cudaMemcpyKind, cudaStream_t s) {
    return put(s, d, std::vector<uint8_t>((const uint8_t *)h, (const uint8_t *)h + n));
}
// pageable memory to the device: staged when the call returns, and no more than that
cudaError_t cudaMemcpy(void *d, const void *h, size_t n, cudaMemcpyKind k) { return cudaMemcpyAsync(d, h, n, k, nullptr); }
cudaError_t cudaStreamCreateWithFlags(cudaStream_t *s, unsigned) {
    static uintptr_t next = 16;
    return *s = (cudaStream_t)next++, cudaSuccess;
}
cudaError_t cudaStreamDestroy(cudaStream_t) { return cudaSuccess; }  // what is queued still runs, some time
cudaError_t cudaStreamSynchronize(cudaStream_t s) {
    for (Op &o : queued[s]) memcpy(o.dst, o.bytes.data(), o.bytes.size()), ++written;
    queued[s].clear();
    return cudaSuccess;
}
cudaError_t cudaGetDriverEntryPointByVersion(const char *, void **f, unsigned, unsigned long long, cudaDriverEntryPointQueryResult *q) {
    *f = (void *)encode;
    *q = cudaDriverEntryPointSuccess;
    return cudaSuccess;
}
}

namespace cbd {
#ifdef TRAIN
int policy_max_blocks(int sms) { return sms * 8; }
int clip_fused_blocks(int sms) { return sms * 2; }
#else
int tc2_max_pairs(int sms) { return sms / 2; }
#endif
}  // namespace cbd

int main(int argc, char **argv) {
    const std::string what = argc > 1 ? argv[1] : "";
    conv_bwd_status st = CONV_BWD_ERR_INVALID_ARG;
    int ops = 1;  // at least
    int elsewhere = CONV_BWD_ERR_INVALID_ARG;  // a run's status with another device current
    size_t zeros = 0;  // bytes of the plan's first buffer that start as zeros
#ifdef TRAIN
    if (what == "experts") {
        const conv_bwd_experts_desc d = {4, 64, 64, CONV_BWD_BF16};
        conv_bwd_experts_plan p;
        st = conv_bwd_experts_create(&d, &p);
        zeros = 64 + 152 * 2 * 4;
        device = 1;
        if (!st) elsewhere = conv_bwd_experts_forward(p, 4, at(1), 0, at(2), (const int32_t *)at(3), at(4), 0, nullptr);
    } else if (what == "clip") {
        const int64_t sizes[2] = {70000, 3};
        const int32_t types[2] = {CONV_BWD_F32, CONV_BWD_BF16};
        conv_bwd_clip_plan p;
        st = conv_bwd_clip_create(2, sizes, types, &p);
        ops = 2;  // counters, and the table of chunks
        zeros = 64;
        device = 1;
        void *const g[2] = {at(1), at(2)};
        if (!st) elsewhere = conv_bwd_clip_run(p, g, g, 1.f, (float *)at(3), (float *)at(4), nullptr);
    } else if (what == "policy") {
        const conv_bwd_policy_desc d = {100, CONV_BWD_F32, 0.2f, 0.2f, 0.f, 1.f};
        conv_bwd_policy_plan p;
        st = conv_bwd_policy_create(&d, &p);
        zeros = 64;
        device = 1;
        const float *f = (const float *)at(3);
        if (!st) elsewhere = conv_bwd_policy_forward(p, 4, at(1), 0, (const int32_t *)at(2), f, f, f, f, (float *)at(4), (float *)at(5), (float *)at(6), (float *)at(7), nullptr);
    }
#else
    conv_bwd_desc d = {};
    d.N = 32; d.C = 512; d.K = 512; d.Hi = 28; d.Wi = 28; d.Y = 3; d.X = 3;
    d.pad_h = d.pad_w = 1;
    d.stride_h = d.stride_w = d.dil_h = d.dil_w = d.groups = 1;
    d.layout = CONV_BWD_NHWC_KYXC;
    d.dtype = CONV_BWD_BF16;
    if (what == "status") {
        d.C = d.K = 64;
    } else if (what == "split") {
        d.stride_h = d.stride_w = d.dil_h = d.dil_w = 2;
        ops = 2;  // status word, and the flags of the split contraction
    } else if (what == "streamk") {
        d.C = d.K = 1024;
        setenv("CONVBWD_DEBUG_STREAMK", "1", 1);
        ops = 2;
    }
    conv_bwd_plan p;
    st = conv_bwd_data_create(&d, &p);
#endif
    if (st != CONV_BWD_OK) return printf("create: status %d\n", (int)st), 2;
    if (int n = pending()) return printf("%d of the plan's writes still queued when create returned\n", n), 1;
    if (written < ops) return printf("%d writes, %d expected\n", written, ops), 1;
    if (held.empty()) return printf("no device memory\n"), 2;
    if (elsewhere != CONV_BWD_ERR_INVALID_ARG) return printf("run with another device current: status %d\n", elsewhere), 1;
    if (zeros) {
        if (held.size() != 1 || held.begin()->second < zeros) return printf("unexpected buffers\n"), 2;
        const uint8_t *m = (const uint8_t *)held.begin()->first;
        for (size_t i = 0; i < zeros; ++i)
            if (m[i]) return printf("byte %zu of the counters is %d\n", i, m[i]), 1;
    }
    return 0;
}
