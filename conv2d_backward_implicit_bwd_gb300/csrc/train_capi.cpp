// train_capi.cpp -- C ABI of the training-step operators
// (include/conv_bwd_train.h): argument checks, plans and their workspaces,
// kernel choice and launches.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <memory>
#include <mutex>
#include <new>
#include <utility>
#include <vector>

#include <cuda.h>
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include "../../include/conv_bwd_train.h"
#include "internal.h"
#include "train.h"

using namespace cbd;

namespace {

struct Range {  // NVTX range in the library's domain
    explicit Range(const char *name) {
        static nvtxDomainHandle_t d = nvtxDomainCreateA("conv_bwd_train");
        dom = d;
        nvtxEventAttributes_t a = {};
        a.version = NVTX_VERSION;
        a.size = NVTX_EVENT_ATTRIB_STRUCT_SIZE;
        a.messageType = NVTX_MESSAGE_TYPE_ASCII;
        a.message.ascii = name;
        nvtxDomainRangePushEx(dom, &a);
    }
    ~Range() { nvtxDomainRangePop(dom); }
    nvtxDomainHandle_t dom;
};

// Device part every plan has: the device it was created on and one allocation
// (status word, tickets, partial sums), zeroed at creation.
struct DevicePart {
    bool has_device = false;
    int device = -1, num_sms = 0, clock_khz = 0;
    void *mem = nullptr;
    size_t counters = 64;  // status word and the counters that are 0 between launches
    conv_bwd_status init(size_t bytes) {
        int n = 0;
        if (cudaGetDeviceCount(&n) != cudaSuccess || n == 0) {
            cudaGetLastError();
            return CONV_BWD_OK;
        }
        if (cudaGetDevice(&device) != cudaSuccess ||
            cudaDeviceGetAttribute(&num_sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess)
            return CONV_BWD_ERR_CUDA;
        if (cudaDeviceGetAttribute(&clock_khz, cudaDevAttrClockRate, device) != cudaSuccess || clock_khz <= 0) {
            cudaGetLastError();
            clock_khz = 2000000;
        }
        if (cudaMalloc(&mem, bytes) != cudaSuccess || write_now(mem, nullptr, bytes) != cudaSuccess) {
            cudaGetLastError();
            return CONV_BWD_ERR_CUDA;
        }
        has_device = true;
        return CONV_BWD_OK;
    }
    ~DevicePart() {
        if (mem) cudaFree(mem);
    }
    // whether the current device is the plan's: its memory and the caller's tensors are there
    bool current() const {
        int now = -1;
        return cudaGetDevice(&now) == cudaSuccess && now == device;
    }
    int32_t *status() const { return static_cast<int32_t *>(mem); }
    uint32_t *ticket() const { return static_cast<uint32_t *>(mem) + 4; }
    char *rest() const { return static_cast<char *>(mem) + 64; }
};

conv_bwd_status read_status(const DevicePart &d, void *stream, int32_t *detail) {
    if (detail) *detail = 0;
    if (!d.has_device) return CONV_BWD_ERR_CUDA;
    cudaStream_t s = (cudaStream_t)stream;
    int32_t h = 0;
    if (cudaMemcpyAsync(&h, d.status(), 4, cudaMemcpyDeviceToHost, s) != cudaSuccess) return CONV_BWD_ERR_CUDA;
    if (cudaStreamSynchronize(s) != cudaSuccess) return CONV_BWD_ERR_CUDA;
    if (h == 0) return CONV_BWD_OK;
    if (detail) *detail = h;
    // (a wait that ran out may have left counters behind)
    if (cudaMemsetAsync(d.mem, 0, d.counters, s) != cudaSuccess || cudaStreamSynchronize(s) != cudaSuccess)
        return CONV_BWD_ERR_CUDA;
    return (h & 0xF00) == 0x200 ? CONV_BWD_ERR_DEVICE_FAULT : CONV_BWD_ERR_DEVICE_TIMEOUT;
}

size_t esize(int32_t dt) { return dt == CONV_BWD_BF16 ? 2 : 4; }
bool overlap(const void *a, size_t na, const void *b, size_t nb) {
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return na && nb && x < y + nb && y < x + na;
}
// bytes from the first to the last element of `rows` rows
size_t extent(int64_t rows, int64_t ld, int64_t width, size_t es) {
    return rows > 0 ? ((size_t)(rows - 1) * (size_t)ld + (size_t)width) * es : 0;
}
bool known_dtype(int32_t d) { return d == CONV_BWD_F32 || d == CONV_BWD_BF16; }

template <typename P, typename F>
conv_bwd_status create_plan(P **out, F &&init) {
    try {
        std::unique_ptr<P> p(new P());
        const conv_bwd_status st = init(*p);
        if (st != CONV_BWD_OK) return st;
        *out = p.release();
        return CONV_BWD_OK;
    } catch (...) {  // host memory
        return CONV_BWD_ERR_CUDA;
    }
}

}  // namespace

namespace {

typedef CUresult (*EncodeTiled)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiled encode_tiled() {
    static EncodeTiled fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = (EncodeTiled)f;
    });
    return fn;
}

// Map of a matrix of rows {width, rows} (bf16, row stride ld elements), box 64 x box_rows.
bool map_rows(CUtensorMap *m, const void *ptr, int64_t width, int64_t rows, int64_t ld, uint32_t box_rows) {
    EncodeTiled enc = encode_tiled();
    if (!enc) return false;
    cuuint64_t dims[2] = {(cuuint64_t)width, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)ld * 2};
    cuuint32_t box[2] = {64, box_rows}, one[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(ptr), dims, strides, box, one,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// Map of [experts][N][K] (bf16, or fp32 for the gradients), box bk x bn of one expert, 128 bytes wide.
bool map_filters(CUtensorMap *m, const void *ptr, const conv_bwd_experts_desc &d, bool f32, uint32_t bk, uint32_t bn) {
    EncodeTiled enc = encode_tiled();
    if (!enc) return false;
    const cuuint64_t es = f32 ? 4 : 2;
    cuuint64_t dims[3] = {(cuuint64_t)d.K, (cuuint64_t)d.N, (cuuint64_t)d.experts};
    cuuint64_t strides[2] = {(cuuint64_t)d.K * es, (cuuint64_t)d.K * (cuuint64_t)d.N * es};
    cuuint32_t box[3] = {bk, bn, 1}, one[3] = {1, 1, 1};
    return enc(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(ptr),
               dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

struct conv_bwd_experts_plan_s {
    conv_bwd_experts_desc d;
    size_t off_parts = 0;
    DevicePart dev;
};
struct conv_bwd_clip_plan_s {
    int32_t count = 0;
    std::vector<int64_t> sizes;
    std::vector<int32_t> dtypes;
    struct Launch {  // tensors [first, first + tensors) of one launch
        int32_t first, tensors, chunks, grid, partial_base;
        size_t chunk_off;  // first chunk in the device table
    };
    std::vector<Launch> launches;
    int32_t partial_total = 0;
    size_t off_chunks = 0;
    int fused_blocks = 0;  // blocks of the one-launch kernel that are resident at once
    std::mutex mu;
    DevicePart dev;
};
struct conv_bwd_policy_plan_s {
    conv_bwd_policy_desc d;
    DevicePart dev;
};

struct conv_bwd_logp_plan_s {
    conv_bwd_logp_desc d;
    size_t off_work = 0;
    DevicePart dev;
};

struct conv_bwd_orth_plan_s {
    conv_bwd_orth_desc d;
    int32_t pitch = 0, most_parts = 0, pairs = 0, cluster = 0;  // cluster: the kernel for small matrices
    bool wide = false;
    std::vector<float> coef;
    double *partial = nullptr;
    __half *x[2] = {};  // planes of the first X
    OrthParams run;     // all but the caller's tensors
    DevicePart dev;
};

extern "C" {

// ---- expert products --------------------------------------------------------
conv_bwd_status conv_bwd_experts_create(const conv_bwd_experts_desc *d, conv_bwd_experts_plan *out) {
    if (!out) return CONV_BWD_ERR_INVALID_ARG;
    *out = nullptr;
    if (!d || d->experts < 1 || d->K < 1 || d->N < 1 || !known_dtype(d->dtype)) return CONV_BWD_ERR_INVALID_ARG;
    if (d->experts > kMaxExperts || d->K > (1 << 20) || d->N > (1 << 20) ||
        d->experts * d->K > (1LL << 40) / d->N)
        return CONV_BWD_ERR_UNSUPPORTED;
    return create_plan(out, [&](conv_bwd_experts_plan_s &p) {
        p.d = *d;
        int sms = 0, dev = 0;
        if (cudaGetDevice(&dev) == cudaSuccess &&
            cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            sms = 0;
        cudaGetLastError();
        // status, counters, the parts of tiles that several blocks share (5 MB)
        static_assert(kSimtPieces * 64 * 64 >= 2 * kStreamRows * 128, "parts of either kind");
        p.off_parts = 64 + ((size_t)sms * kSimtPieces * 4 + 255) / 256 * 256 + 192;
        p.dev.counters = p.off_parts;
        return p.dev.init(p.off_parts + (size_t)sms * kSimtPieces * 64 * 64 * 4);
    });
}

conv_bwd_status conv_bwd_experts_destroy(conv_bwd_experts_plan p) {
    delete p;
    return CONV_BWD_OK;
}

// of rows and of tiles: the kernels step past the last one by up to a grid or a slice, in 32 bits
constexpr int64_t kMostRows = 0x7fff0000;

static conv_bwd_status experts_run(conv_bwd_experts_plan p, int dir, int64_t rows, const void *a, int64_t lda,
                                   const void *b, int64_t ldb, const int32_t *offsets, void *out, int64_t ldo,
                                   int32_t accumulate, void *stream) {
    if (!p || rows < 0 || !b || !offsets || (rows > 0 && !a)) return CONV_BWD_ERR_INVALID_ARG;
    if (!out && (rows > 0 || dir == CONV_BWD_EXPERTS_WEIGHT)) return CONV_BWD_ERR_INVALID_ARG;
    const conv_bwd_experts_desc &d = p->d;
    const int64_t wa = dir == CONV_BWD_EXPERTS_FORWARD ? d.K : d.N;  // width of the row-sorted operand a
    const int64_t wo = dir == CONV_BWD_EXPERTS_FORWARD ? d.N : d.K;  // width of out (weight: of the operand b)
    if (lda == 0) lda = wa;
    if (ldb == 0) ldb = d.K;
    if (ldo == 0) ldo = wo;
    if (lda < wa || ldb < d.K || ldo < wo) return CONV_BWD_ERR_INVALID_ARG;
    const size_t es = esize(d.dtype), nw = (size_t)d.experts * d.N * d.K;
    const bool weight = dir == CONV_BWD_EXPERTS_WEIGHT;
    if (((uintptr_t)a | (uintptr_t)b) % es || (uintptr_t)offsets % 4 || (uintptr_t)out % (weight ? 4 : es))
        return CONV_BWD_ERR_MISALIGNED;
    if (rows > kMostRows || lda > (1LL << 31) || ldb > (1LL << 31) || ldo > (1LL << 31)) return CONV_BWD_ERR_UNSUPPORTED;
    // most tiles of any kernel: 64 rows x 64 columns
    const int64_t nt = (wo + 63) / 64;
    const int64_t tiles = weight ? d.experts * ((d.N + 63) / 64) * nt : (rows / 64 + d.experts) * nt;
    if (tiles > kMostRows) return CONV_BWD_ERR_UNSUPPORTED;
    const size_t na = extent(rows, lda, wa, es), nb = weight ? extent(rows, ldb, d.K, es) : nw * es,
                 no = weight ? nw * 4 : extent(rows, ldo, wo, es);
    if (overlap(a, na, out, no) || overlap(b, nb, out, no) || overlap(offsets, (size_t)(d.experts + 1) * 4, out, no))
        return CONV_BWD_ERR_INVALID_ARG;
    if (!p->dev.has_device) return CONV_BWD_ERR_CUDA;
    if (!p->dev.current()) return CONV_BWD_ERR_INVALID_ARG;
    if (rows == 0 && (!weight || accumulate)) return CONV_BWD_OK;
    // Tensor cores on pairs of SMs where TMA can load the filters or store their gradients (bf16, widths and address on 16 bytes); the rows come
    // by TMA if their strides and addresses are on 16 bytes too, else through registers.
    const bool rows_lines = lda % 8 == 0 && (uintptr_t)a % 16 == 0 && (!weight || (ldb % 8 == 0 && (uintptr_t)b % 16 == 0));
    if (d.dtype == CONV_BWD_BF16 && d.K % 8 == 0 && d.N % 8 == 0 && rows > 0 && d.K * d.N < (1LL << 37) &&
        (uintptr_t)(weight ? out : b) % 16 == 0) {
        const int64_t mt = ((dir == kExpData ? d.K : d.N) + 255) / 256, pairs = std::max(1, p->dev.num_sms / 2);
        // Up to eight rows per expert: the filters' bytes are the time.  The few-rows kernel shares them out better where
        // its tiles are many enough to be drawn, or so few that the pairs' 256-wide tiles do not fill two rounds, or
        // where half of a pair's tile would be idle.  Measured (us, it against the pairs; one row per expert, eight
        // rows).  64 experts, drawn: 2048 deep x 1024 44.6 to 47.3, 45.6 to 48.8; 1024 x 2048 43.7 to 44.0, 45.6 to
        // 45.8; 128 x 16384 44.9 to 49.3, 47.4 to 49.9.  Between: 4096 x 512 47.6 to 44.4, 49.8 to 45.6.  Narrow: 16384 x
        // 128 47.5 to 63.0, 52.0 to 63.5.  Few tiles, 8 experts: 4096 deep x 1024 12.6 to 18.8, 18.8 to 19.7; 1024 x
        // 4096 11.5 to 12.0, 15.0 to 15.2, at 16 rows 18.6 to 15.5.
        const int64_t stream_blocks =
            (rows / kStreamRows + std::min<int64_t>(d.experts, rows)) * ((wo + 127) / 128) * ((wa + 63) / 64);
        const int64_t used = std::min<int64_t>(d.experts, rows);
        if (rows_lines && !weight && rows <= 8 * d.experts && (mt * used <= 2 * pairs || (wo + 127) / 128 * used >= 6 * pairs || wo <= 128) && stream_blocks <= 0x7fffffff) {
            ExpertStreamParams sp;
            std::memset(&sp, 0, sizeof(sp));
            const bool ok = map_filters(&sp.a, b, d, false, 64, dir == kExpForward ? 128 : 64) &&
                            map_rows(&sp.b, a, dir == kExpForward ? d.K : d.N, rows, lda, kStreamRows);
            if (!ok) return CONV_BWD_ERR_CUDA;
            sp.out = out; sp.offsets = offsets; sp.status = p->dev.status();
            sp.arrived = reinterpret_cast<int32_t *>(p->dev.rest());
            sp.parts = reinterpret_cast<float *>(static_cast<char *>(p->dev.mem) + p->off_parts);
            sp.drawn = reinterpret_cast<int32_t *>(p->dev.ticket());
            sp.wait_budget = (int64_t)p->dev.clock_khz * 2000;
            sp.ldo = ldo;
            sp.experts = (int32_t)d.experts; sp.rows = (int32_t)rows; sp.K = (int32_t)d.K; sp.N = (int32_t)d.N;
            // at least four blocks of 16 KB for an SM
            const int grid = (int)std::max<int64_t>(1, std::min<int64_t>(p->dev.num_sms, stream_blocks / 4));
            return launch_experts_stream(sp, dir, grid, (cudaStream_t)stream) == cudaSuccess ? CONV_BWD_OK : CONV_BWD_ERR_CUDA;
        }
        ExpertPairParams pp;
        std::memset(&pp, 0, sizeof(pp));
        bool ok;
        if (dir == kExpForward)
            ok = map_filters(&pp.a, b, d, false, 64, 128) && (!rows_lines || map_rows(&pp.b, a, d.K, rows, lda, 64));
        else if (dir == kExpData)
            ok = map_filters(&pp.a, b, d, false, 64, 64) && (!rows_lines || map_rows(&pp.b, a, d.N, rows, lda, 64));
        else
            ok = (!rows_lines || (map_rows(&pp.a, a, d.N, rows, lda, 64) && map_rows(&pp.b, b, d.K, rows, ldb, 64))) &&
                 map_filters(&pp.o, out, d, true, 32, 32);
        if (!ok) return CONV_BWD_ERR_CUDA;
        pp.out = out; pp.offsets = offsets; pp.status = p->dev.status();
        pp.wait_budget = (int64_t)p->dev.clock_khz * 2000;  // two seconds of SM clocks
        pp.ldo = ldo;
        pp.experts = (int32_t)d.experts; pp.rows = (int32_t)rows; pp.K = (int32_t)d.K; pp.N = (int32_t)d.N;
        pp.accumulate = accumulate ? 1 : 0;
        pp.out_lines = ldo % 8 == 0 && (uintptr_t)out % 16 == 0;
        if (!rows_lines) {
            pp.rows_at = a;
            pp.rows_end = static_cast<const char *>(a) + na;
            pp.ldb = lda;
            pp.rows2_at = b;
            pp.rows2_end = static_cast<const char *>(b) + nb;
            pp.ldb2 = ldb;
        }
        const int64_t most = weight ? d.experts * mt * ((d.K + 255) / 256) : mt * (rows / 256 + std::min<int64_t>(d.experts, rows));
        const int grid = (int)(2 * std::max<int64_t>(1, std::min(pairs, most)));
        return launch_experts_pair(pp, dir, grid, (cudaStream_t)stream) == cudaSuccess ? CONV_BWD_OK : CONV_BWD_ERR_CUDA;
    }
    const int64_t sms = std::max(1, p->dev.num_sms);
    auto tiles_of = [&](int64_t bt) {
        const int64_t cols = (wo + bt - 1) / bt;
        return weight ? d.experts * ((d.N + bt - 1) / bt) * cols : (rows / bt + std::min<int64_t>(d.experts, rows)) * cols;
    };
    ExpertSimtParams sp;
    std::memset(&sp, 0, sizeof(sp));
    sp.a = a; sp.b = b; sp.a_end = static_cast<const char *>(a) + na; sp.b_end = static_cast<const char *>(b) + nb; sp.out = out; sp.offsets = offsets; sp.status = p->dev.status();
    sp.lda = lda; sp.ldb = ldb; sp.ldo = ldo;
    sp.experts = (int32_t)d.experts; sp.rows = (int32_t)rows; sp.K = (int32_t)d.K; sp.N = (int32_t)d.N;
    sp.accumulate = accumulate ? 1 : 0;
    sp.chunk = kMaxRows;
    // few rows leave most of a tile idle (measured at the kernel; at 8 rows per expert 141 against 201 us)
    if (!weight && d.dtype == CONV_BWD_F32 && rows <= 8 * d.experts)
        return launch_experts_few_f32(sp, dir, (int)sms, (cudaStream_t)stream) == cudaSuccess ? CONV_BWD_OK : CONV_BWD_ERR_CUDA;
    // wide tiles where they fill the SMs and the tiles' two sides
    sp.wide = tiles_of(128) >= sms && wo > 64 && (weight ? d.N > 64 : rows >= 96 * d.experts);
    int64_t pieces = std::max<int64_t>(1, tiles_of(sp.wide ? 128 : 64));
    if (!sp.wide && pieces <= sms) {
        // few tiles: their contraction in chunks of at least 128, at most two pieces for an SM
        const int64_t depth = weight ? rows : wa, room = kSimtPieces * sms;
        const int64_t least = weight ? rows * pieces / d.experts / (room - pieces) + 1 : (depth + room / pieces - 1) / (room / pieces);
        const int64_t chunk = (std::max<int64_t>(least, 128) + 31) / 32 * 32;
        if (chunk < depth) {
            sp.chunk = (int32_t)chunk;
            pieces = weight ? pieces + depth / chunk * (pieces / d.experts) : pieces * ((depth + chunk - 1) / chunk);
        }
    }
    sp.grid = (int32_t)std::min<int64_t>(pieces, 2 * sms);
    sp.arrived = reinterpret_cast<int32_t *>(p->dev.rest());
    sp.parts = reinterpret_cast<float *>(static_cast<char *>(p->dev.mem) + p->off_parts);
    const cudaError_t e = d.dtype == CONV_BWD_BF16 ? launch_experts_b16(sp, dir, (cudaStream_t)stream) : launch_experts_f32(sp, dir, (cudaStream_t)stream);
    return e == cudaSuccess ? CONV_BWD_OK : CONV_BWD_ERR_CUDA;
}

conv_bwd_status conv_bwd_experts_forward(conv_bwd_experts_plan p, int64_t rows, const void *x, int64_t ldx,
                                         const void *w, const int32_t *offsets, void *y, int64_t ldy, void *stream) {
    Range range("conv_bwd_experts_forward");
    return experts_run(p, kExpForward, rows, x, ldx, w, 0, offsets, y, ldy, 0, stream);
}
conv_bwd_status conv_bwd_experts_data(conv_bwd_experts_plan p, int64_t rows, const void *dy, int64_t lddy,
                                      const void *w, const int32_t *offsets, void *dx, int64_t lddx, void *stream) {
    Range range("conv_bwd_experts_data");
    return experts_run(p, kExpData, rows, dy, lddy, w, 0, offsets, dx, lddx, 0, stream);
}
conv_bwd_status conv_bwd_experts_weight(conv_bwd_experts_plan p, int64_t rows, const void *dy, int64_t lddy,
                                        const void *x, int64_t ldx, const int32_t *offsets, float *dw,
                                        int32_t accumulate, void *stream) {
    Range range("conv_bwd_experts_weight");
    if (rows > 0 && !x) return CONV_BWD_ERR_INVALID_ARG;
    // with no rows x is never read; any non-null pointer stands for it
    return experts_run(p, kExpWeight, rows, dy, lddy, rows > 0 ? x : static_cast<const void *>(offsets), ldx, offsets, dw,
                       0, accumulate, stream);
}
conv_bwd_status conv_bwd_experts_get_status(conv_bwd_experts_plan p, void *stream, int32_t *detail) {
    if (!p) return CONV_BWD_ERR_INVALID_ARG;
    return read_status(p->dev, stream, detail);
}

// ---- gradient clipping --------------------------------------------------------
conv_bwd_status conv_bwd_clip_create(int32_t count, const int64_t *sizes, const int32_t *dtypes,
                                     conv_bwd_clip_plan *out) {
    if (!out) return CONV_BWD_ERR_INVALID_ARG;
    *out = nullptr;
    if (count < 0 || (count > 0 && (!sizes || !dtypes))) return CONV_BWD_ERR_INVALID_ARG;
    if (count > 65536) return CONV_BWD_ERR_UNSUPPORTED;
    int64_t total = 0;
    for (int32_t i = 0; i < count; ++i)
        if (sizes[i] < 0 || !known_dtype(dtypes[i])) return CONV_BWD_ERR_INVALID_ARG;
    for (int32_t i = 0; i < count; ++i) {
        if (sizes[i] >= (1LL << 38)) return CONV_BWD_ERR_UNSUPPORTED;
        total += sizes[i];
        if (total > (1LL << 40)) return CONV_BWD_ERR_UNSUPPORTED;
    }
    return create_plan(out, [&](conv_bwd_clip_plan_s &p) {
        p.count = count;
        p.sizes.assign(sizes, sizes + count);
        p.dtypes.assign(dtypes, dtypes + count);
        int sms = 148, dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
            cudaGetLastError();
            sms = 148;
        }
        std::vector<ClipChunk> chunks;
        for (int32_t first = 0; first == 0 || first < count; first += kClipPtrs) {
            conv_bwd_clip_plan_s::Launch l;
            l.first = first;
            l.tensors = std::min(kClipPtrs, count - first);
            l.chunk_off = chunks.size();
            for (int32_t t = 0; t < l.tensors; ++t) {
                const int64_t per = kClipChunk / (int64_t)esize(dtypes[first + t]), size = sizes[first + t];
                for (int64_t at = 0; at < size; at += per)
                    chunks.push_back({at, (int32_t)std::min(per, size - at), (int16_t)t, (int16_t)(dtypes[first + t] == CONV_BWD_BF16)});
            }
            const size_t n = chunks.size() - l.chunk_off;
            if (n > 0x7fffffff) return CONV_BWD_ERR_UNSUPPORTED;
            l.chunks = (int32_t)n;
            l.grid = (int32_t)std::max<int64_t>(1, std::min<int64_t>(l.chunks, (int64_t)sms * kNormBlocks));
            l.partial_base = p.partial_total;
            p.partial_total += l.grid;
            p.launches.push_back(l);
        }
        chunks.push_back({0, 0, 0, 0});  // a launch without chunks still reads one entry
        int cooperative = 0;
        if (cudaDeviceGetAttribute(&cooperative, cudaDevAttrCooperativeLaunch, dev) == cudaSuccess && cooperative)
            p.fused_blocks = clip_fused_blocks(sms);
        cudaGetLastError();
        p.off_chunks = (64 + (size_t)std::max(p.partial_total, p.fused_blocks) * 8 + 15) / 16 * 16;
        const conv_bwd_status st = p.dev.init(p.off_chunks + chunks.size() * sizeof(ClipChunk));
        if (st != CONV_BWD_OK || !p.dev.has_device) return st;
        if (write_now(static_cast<char *>(p.dev.mem) + p.off_chunks, chunks.data(), chunks.size() * sizeof(ClipChunk)) != cudaSuccess) {
            cudaGetLastError();
            return CONV_BWD_ERR_CUDA;
        }
        return CONV_BWD_OK;
    });
}

conv_bwd_status conv_bwd_clip_destroy(conv_bwd_clip_plan p) {
    delete p;
    return CONV_BWD_OK;
}

static conv_bwd_status clip_launch(conv_bwd_clip_plan p, const void *const *grads, void *const *outs, float max_norm,
                                   float *norm, float *coef, void *stream) {
    if (!p || !norm || (p->count > 0 && !grads)) return CONV_BWD_ERR_INVALID_ARG;
    const bool scale = coef != nullptr;
    if (scale && (std::isnan(max_norm) || max_norm < 0.f || (p->count > 0 && !outs))) return CONV_BWD_ERR_INVALID_ARG;
    bool bad_align = ((uintptr_t)norm | (uintptr_t)coef) % 4;
    for (int32_t i = 0; i < p->count; ++i) {
        if (p->sizes[i] == 0) continue;
        if (!grads[i] || (scale && !outs[i])) return CONV_BWD_ERR_INVALID_ARG;
        const size_t es = esize(p->dtypes[i]), n = (size_t)p->sizes[i] * es;
        if ((uintptr_t)grads[i] % es || (scale && (uintptr_t)outs[i] % es)) bad_align = true;
        if (scale && outs[i] != grads[i] && overlap(grads[i], n, outs[i], n)) return CONV_BWD_ERR_INVALID_ARG;
    }
    if (bad_align) return CONV_BWD_ERR_MISALIGNED;
    if (!p->dev.has_device) return CONV_BWD_ERR_CUDA;
    if (!p->dev.current()) return CONV_BWD_ERR_INVALID_ARG;
    std::lock_guard<std::mutex> lock(p->mu);
    char *m = static_cast<char *>(p->dev.mem);
    ClipParams cp;
    std::memset(&cp, 0, sizeof(cp));
    cp.partials = reinterpret_cast<double *>(p->dev.rest());
    cp.ticket = p->dev.ticket();
    cp.norm = norm;
    cp.coef = coef;
    cp.want_coef = scale ? 1 : 0;
    cp.max_norm = max_norm;
    cp.turn = p->dev.ticket() + 1;
    cp.status = p->dev.status();
    cp.wait_budget = (int64_t)p->dev.clock_khz * 2000;
    const size_t nl = p->launches.size();
    // Gradients that fit the SMs' registers are read once.
    if (scale && nl == 1 && p->launches[0].chunks > 0 && p->launches[0].chunks <= p->fused_blocks) {
        cp.chunks = reinterpret_cast<const ClipChunk *>(m + p->off_chunks);
        cp.num_chunks = p->launches[0].chunks;
        return launch_clip_fused(cp, grads, outs, p->count, (cudaStream_t)stream) == cudaSuccess ? CONV_BWD_OK : CONV_BWD_ERR_CUDA;
    }
    for (int pass = 0; pass < (scale ? 2 : 1); ++pass)
        for (size_t k = 0; k < nl; ++k) {
            const auto &l = p->launches[pass ? nl - 1 - k : k];
            cp.chunks = reinterpret_cast<const ClipChunk *>(m + p->off_chunks) + l.chunk_off;
            cp.num_chunks = l.chunks;
            cp.partial_base = l.partial_base;
            cp.partial_total = k + 1 == nl ? p->partial_total : 0;
            if (pass && l.chunks == 0) continue;
            const void *const *g = grads + l.first;
            const cudaError_t e = pass ? launch_clip_scale(cp, g, outs + l.first, l.tensors, std::min(l.chunks, p->dev.num_sms * kScaleBlocks), (cudaStream_t)stream)
                                       : launch_clip_norm(cp, g, l.tensors, l.grid, (cudaStream_t)stream);
            if (e != cudaSuccess) return CONV_BWD_ERR_CUDA;
        }
    return CONV_BWD_OK;
}

conv_bwd_status conv_bwd_clip_norm(conv_bwd_clip_plan p, const void *const *grads, float *norm, void *stream) {
    Range range("conv_bwd_clip_norm");
    return clip_launch(p, grads, nullptr, 0.f, norm, nullptr, stream);
}
conv_bwd_status conv_bwd_clip_run(conv_bwd_clip_plan p, const void *const *grads, void *const *out, float max_norm,
                                  float *norm, float *coef, void *stream) {
    Range range("conv_bwd_clip_run");
    if (!coef) return CONV_BWD_ERR_INVALID_ARG;
    return clip_launch(p, grads, out, max_norm, norm, coef, stream);
}

conv_bwd_status conv_bwd_clip_get_status(conv_bwd_clip_plan p, void *stream, int32_t *detail) {
    if (!p) return CONV_BWD_ERR_INVALID_ARG;
    return read_status(p->dev, stream, detail);
}

// ---- policy loss --------------------------------------------------------------
conv_bwd_status conv_bwd_policy_create(const conv_bwd_policy_desc *d, conv_bwd_policy_plan *out) {
    if (!out) return CONV_BWD_ERR_INVALID_ARG;
    *out = nullptr;
    if (!d || d->vocab < 1 || !known_dtype(d->dtype)) return CONV_BWD_ERR_INVALID_ARG;
    if (!(d->clip_low >= 0.f && d->clip_low <= 1.f) || !(d->clip_high >= 0.f && std::isfinite(d->clip_high)) ||
        !(d->kl >= 0.f && std::isfinite(d->kl)) || !(d->scale > 0.f && std::isfinite(d->scale)))
        return CONV_BWD_ERR_INVALID_ARG;
    if (d->vocab > (1LL << 30)) return CONV_BWD_ERR_UNSUPPORTED;
    return create_plan(out, [&](conv_bwd_policy_plan_s &p) {
        p.d = *d;
        int sms = 0, dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
            cudaGetLastError();
            sms = 0;
        }
        return p.dev.init(64 + (size_t)policy_max_blocks(sms) * 8 + 8);
    });
}
conv_bwd_status conv_bwd_policy_destroy(conv_bwd_policy_plan p) {
    delete p;
    return CONV_BWD_OK;
}

static conv_bwd_status policy_run(conv_bwd_policy_plan p, int mode, PolicyParams &pp, int64_t tokens, int64_t ld,
                                  int64_t ldd, void *stream) {
    if (!p || tokens < 0) return CONV_BWD_ERR_INVALID_ARG;
    const int64_t V = p->d.vocab;
    if (ld == 0) ld = V;
    if (ldd == 0) ldd = V;
    if (ld < V || ldd < V) return CONV_BWD_ERR_INVALID_ARG;
    const bool fwd = mode != kPolBackward, bwd = mode != kPolForward;
    if (tokens > 0) {
        if (!pp.logits || !pp.actions) return CONV_BWD_ERR_INVALID_ARG;
        if (fwd && (!pp.advantage || !pp.weight || !pp.logp)) return CONV_BWD_ERR_INVALID_ARG;
        if (mode == kPolForward && (!pp.lse || !pp.coef)) return CONV_BWD_ERR_INVALID_ARG;
        if (mode == kPolBackward && (!pp.lse_in || !pp.coef_in)) return CONV_BWD_ERR_INVALID_ARG;
        if (bwd && !pp.dlogits) return CONV_BWD_ERR_INVALID_ARG;
    }
    if (fwd && !pp.loss) return CONV_BWD_ERR_INVALID_ARG;
    const size_t es = esize(p->d.dtype);
    const uintptr_t words = (uintptr_t)pp.actions | (uintptr_t)pp.advantage | (uintptr_t)pp.weight |
                            (uintptr_t)pp.old_logp | (uintptr_t)pp.ref_logp | (uintptr_t)pp.lse_in |
                            (uintptr_t)pp.coef_in | (uintptr_t)pp.grad | (uintptr_t)pp.loss | (uintptr_t)pp.logp |
                            (uintptr_t)pp.lse | (uintptr_t)pp.coef;
    if (words % 4 || ((uintptr_t)pp.logits | (uintptr_t)pp.dlogits) % es) return CONV_BWD_ERR_MISALIGNED;
    if (tokens > 0x7fffffff || ld > (1LL << 31) || ldd > (1LL << 31)) return CONV_BWD_ERR_UNSUPPORTED;
    const size_t nz = extent(tokens, ld, V, es), nd = extent(tokens, ldd, V, es);
    if (bwd && overlap(pp.logits, nz, pp.dlogits, nd) && !(pp.logits == pp.dlogits && ld == ldd))
        return CONV_BWD_ERR_INVALID_ARG;
    if (!p->dev.has_device) return CONV_BWD_ERR_CUDA;
    if (!p->dev.current()) return CONV_BWD_ERR_INVALID_ARG;
    if (tokens == 0 && !fwd) return CONV_BWD_OK;
    pp.partials = reinterpret_cast<double *>(p->dev.rest());
    pp.ticket = p->dev.ticket();
    pp.status = p->dev.status();
    pp.ld = ld;
    pp.ldd = ldd;
    pp.tokens = (int32_t)tokens;
    pp.vocab = (int32_t)V;
    pp.clip_lo = 1.f - p->d.clip_low;
    pp.clip_hi = 1.f + p->d.clip_high;
    pp.kl = p->d.kl;
    pp.scale = p->d.scale;
    pp.wait_budget = (int64_t)p->dev.clock_khz * 2000;
    return launch_policy(pp, p->d.dtype, mode, p->dev.num_sms, (cudaStream_t)stream) == cudaSuccess ? CONV_BWD_OK
                                                                                                    : CONV_BWD_ERR_CUDA;
}

conv_bwd_status conv_bwd_policy_forward(conv_bwd_policy_plan p, int64_t tokens, const void *logits, int64_t ld,
                                        const int32_t *actions, const float *advantage, const float *weight,
                                        const float *old_logp, const float *ref_logp, float *loss, float *logp,
                                        float *lse, float *coef, void *stream) {
    Range range("conv_bwd_policy_forward");
    PolicyParams pp;
    std::memset(&pp, 0, sizeof(pp));
    pp.logits = logits; pp.actions = actions; pp.advantage = advantage; pp.weight = weight;
    pp.old_logp = old_logp; pp.ref_logp = ref_logp;
    pp.loss = loss; pp.logp = logp; pp.lse = lse; pp.coef = coef;
    return policy_run(p, kPolForward, pp, tokens, ld, 0, stream);
}
conv_bwd_status conv_bwd_policy_backward(conv_bwd_policy_plan p, int64_t tokens, const void *logits, int64_t ld,
                                         const int32_t *actions, const float *lse, const float *coef,
                                         const float *grad, void *dlogits, int64_t ldd, void *stream) {
    Range range("conv_bwd_policy_backward");
    PolicyParams pp;
    std::memset(&pp, 0, sizeof(pp));
    pp.logits = logits; pp.actions = actions; pp.lse_in = lse; pp.coef_in = coef; pp.grad = grad;
    pp.dlogits = dlogits;
    return policy_run(p, kPolBackward, pp, tokens, ld, ldd, stream);
}
conv_bwd_status conv_bwd_policy_forward_backward(conv_bwd_policy_plan p, int64_t tokens, const void *logits,
                                                 int64_t ld, const int32_t *actions, const float *advantage,
                                                 const float *weight, const float *old_logp, const float *ref_logp,
                                                 float *loss, float *logp, void *dlogits, int64_t ldd, void *stream) {
    Range range("conv_bwd_policy_forward_backward");
    PolicyParams pp;
    std::memset(&pp, 0, sizeof(pp));
    pp.logits = logits; pp.actions = actions; pp.advantage = advantage; pp.weight = weight;
    pp.old_logp = old_logp; pp.ref_logp = ref_logp;
    pp.loss = loss; pp.logp = logp; pp.dlogits = dlogits;
    return policy_run(p, kPolBoth, pp, tokens, ld, ldd, stream);
}
conv_bwd_status conv_bwd_policy_get_status(conv_bwd_policy_plan p, void *stream, int32_t *detail) {
    if (!p) return CONV_BWD_ERR_INVALID_ARG;
    return read_status(p->dev, stream, detail);
}

// ---- token log-probabilities ----------------------------------------------------
conv_bwd_status conv_bwd_logp_create(const conv_bwd_logp_desc *d, conv_bwd_logp_plan *out) {
    if (!out) return CONV_BWD_ERR_INVALID_ARG;
    *out = nullptr;
    // (scale log2(e) is finite)
    if (!d || d->vocab < 1 || !known_dtype(d->dtype) || d->top < 0 || d->top > d->vocab ||
        !(d->scale > 0.f && d->scale <= 0x1p127f))
        return CONV_BWD_ERR_INVALID_ARG;
    if (d->vocab > (1LL << 30) || d->top > kLogpTop) return CONV_BWD_ERR_UNSUPPORTED;
    return create_plan(out, [&](conv_bwd_logp_plan_s &p) {
        p.d = *d;
        int sms = 0, dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
            cudaGetLastError();
            sms = 0;
        }
        const size_t items = (size_t)logp_most_items(sms);
        p.off_work = 64 + (items * 4 + 63) / 64 * 64;
        p.dev.counters = p.off_work;
        return p.dev.init(p.off_work + items * kLogpPart);
    });
}
conv_bwd_status conv_bwd_logp_destroy(conv_bwd_logp_plan p) {
    delete p;
    return CONV_BWD_OK;
}

static conv_bwd_status logp_run(conv_bwd_logp_plan p, bool backward, LogpParams &lp, int64_t rows, int64_t ld, int64_t ldd,
                                void *stream) {
    if (!p || rows < 0) return CONV_BWD_ERR_INVALID_ARG;
    const conv_bwd_logp_desc &d = p->d;
    const int64_t V = d.vocab;
    if (ld == 0) ld = V;
    if (ldd == 0) ldd = V;
    if (ld < V || ldd < V) return CONV_BWD_ERR_INVALID_ARG;
    if (rows > 0) {
        if (!lp.logits) return CONV_BWD_ERR_INVALID_ARG;
        if (!backward && (!lp.entropy || !lp.lse || !lp.tokens != !lp.logp || (d.top > 0 && (!lp.top_logp || !lp.top_tokens))))
            return CONV_BWD_ERR_INVALID_ARG;
        if (backward && (!lp.lse_in || !lp.dlogits || (!lp.grad_logp && !lp.grad_entropy) || (lp.grad_logp && !lp.tokens) ||
                         (lp.grad_entropy && !lp.entropy_in)))
            return CONV_BWD_ERR_INVALID_ARG;
    }
    const size_t es = esize(d.dtype);
    const uintptr_t words = (uintptr_t)lp.tokens | (uintptr_t)lp.logp | (uintptr_t)lp.entropy | (uintptr_t)lp.lse |
                            (uintptr_t)lp.top_logp | (uintptr_t)lp.top_tokens | (uintptr_t)lp.lse_in |
                            (uintptr_t)lp.entropy_in | (uintptr_t)lp.grad_logp | (uintptr_t)lp.grad_entropy;
    if (words % 4 || ((uintptr_t)lp.logits | (uintptr_t)lp.dlogits) % es) return CONV_BWD_ERR_MISALIGNED;
    if (rows > kMostRows || ld > (1LL << 31) || ldd > (1LL << 31)) return CONV_BWD_ERR_UNSUPPORTED;
    const size_t nz = extent(rows, ld, V, es), nd = extent(rows, ldd, V, es), n = (size_t)rows * 4;
    if (backward) {
        if (overlap(lp.logits, nz, lp.dlogits, nd) && !(lp.logits == lp.dlogits && ld == ldd)) return CONV_BWD_ERR_INVALID_ARG;
        for (const void *in : {(const void *)lp.tokens, (const void *)lp.lse_in, (const void *)lp.entropy_in,
                               (const void *)lp.grad_logp, (const void *)lp.grad_entropy})
            if (in && overlap(in, n, lp.dlogits, nd)) return CONV_BWD_ERR_INVALID_ARG;
    } else {
        const size_t top = n * (size_t)d.top;
        const std::pair<const void *, size_t> outs[] = {{lp.logp, n}, {lp.entropy, n}, {lp.lse, n}, {lp.top_logp, top}, {lp.top_tokens, top}};
        for (const auto &o : outs) {
            if (!o.first) continue;
            if (overlap(lp.logits, nz, o.first, o.second) || (lp.tokens && overlap(lp.tokens, n, o.first, o.second))) return CONV_BWD_ERR_INVALID_ARG;
            for (const auto &q : outs)
                if (&q != &o && q.first && overlap(q.first, q.second, o.first, o.second)) return CONV_BWD_ERR_INVALID_ARG;
        }
    }
    if (!p->dev.has_device) return CONV_BWD_ERR_CUDA;
    if (!p->dev.current()) return CONV_BWD_ERR_INVALID_ARG;
    if (rows == 0) return CONV_BWD_OK;
    lp.work = static_cast<char *>(p->dev.mem) + p->off_work;
    lp.arrived = reinterpret_cast<int32_t *>(p->dev.rest());
    lp.status = p->dev.status();
    lp.ld = ld;
    lp.ldd = ldd;
    lp.wait_budget = (int64_t)p->dev.clock_khz * 2000;
    lp.rows = (int32_t)rows;
    lp.vocab = (int32_t)V;
    lp.top = d.top;
    lp.parts = logp_parts(rows, V, d.dtype, p->dev.num_sms);
    lp.scale = d.scale;
    return launch_logp(lp, d.dtype, backward, p->dev.num_sms, (cudaStream_t)stream) == cudaSuccess ? CONV_BWD_OK : CONV_BWD_ERR_CUDA;
}

conv_bwd_status conv_bwd_logp_forward(conv_bwd_logp_plan p, int64_t rows, const void *logits, int64_t ld, const int32_t *tokens,
                                      float *logp, float *entropy, float *lse, float *top_logp, int32_t *top_tokens, void *stream) {
    Range range("conv_bwd_logp_forward");
    LogpParams lp;
    std::memset(&lp, 0, sizeof(lp));
    lp.logits = logits; lp.tokens = tokens;
    lp.logp = logp; lp.entropy = entropy; lp.lse = lse;
    if (p && p->d.top) { lp.top_logp = top_logp; lp.top_tokens = top_tokens; }
    return logp_run(p, false, lp, rows, ld, 0, stream);
}
conv_bwd_status conv_bwd_logp_backward(conv_bwd_logp_plan p, int64_t rows, const void *logits, int64_t ld, const int32_t *tokens,
                                       const float *lse, const float *entropy, const float *grad_logp, const float *grad_entropy,
                                       void *dlogits, int64_t ldd, void *stream) {
    Range range("conv_bwd_logp_backward");
    LogpParams lp;
    std::memset(&lp, 0, sizeof(lp));
    lp.logits = logits; lp.tokens = tokens;
    lp.lse_in = lse; lp.entropy_in = entropy; lp.grad_logp = grad_logp; lp.grad_entropy = grad_entropy;
    lp.dlogits = dlogits;
    return logp_run(p, true, lp, rows, ld, ldd, stream);
}
conv_bwd_status conv_bwd_logp_get_status(conv_bwd_logp_plan p, void *stream, int32_t *detail) {
    if (!p) return CONV_BWD_ERR_INVALID_ARG;
    return read_status(p->dev, stream, detail);
}

// ---- orthogonalised updates -------------------------------------------------------
// A plane [batch][rows][pitch] of fp16 as the products read and write it.
static bool map_plane(CUtensorMap *m, void *at, int64_t batch, int64_t rows, int64_t cols, int64_t pitch, uint32_t box_cols,
                      uint32_t box_rows) {
    EncodeTiled enc = encode_tiled();
    if (!enc) return false;
    cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)batch};
    cuuint64_t strides[2] = {(cuuint64_t)pitch * 2, (cuuint64_t)pitch * (cuuint64_t)rows * 2};
    cuuint32_t box[3] = {box_cols, box_rows, 1}, one[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, at, dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Whether `steps` steps may go by polynomials of several of them, `joined` at most in one.  X^T X's rounding reaches a
// direction of singular value s by |dQ/d(s^2)| s, which for three steps with a = 3.4445 is what three steps apart lose and for
// five ten times as much; it grows by the fifth power of a.  And all matrices must stay within the planes' range: X
// begins with singular values in [0, 1], and what becomes of those is followed.
static bool orth_may_join(const float *coef, int steps, int joined) {
    for (int k = 0; k < steps; ++k)
        if (std::fabs(coef[3 * k]) > 4.f || std::fabs(coef[3 * k + 1]) > 6.f || std::fabs(coef[3 * k + 2]) > 6.f) return false;
    constexpr int POINTS = 4096;
    for (int i = 0; i <= POINTS; ++i) {
        double x = (double)i / POINTS;
        for (int k0 = 0; k0 < steps; k0 += joined) {
            double gram = x * x, q = 1.0;
            for (int k = k0; k < std::min(k0 + joined, steps); ++k) {
                const double b = coef[3 * k] + (coef[3 * k + 1] + coef[3 * k + 2] * gram) * gram;
                q *= b;
                if (!(std::fabs(b) < 100.0 && std::fabs(q) < 100.0 && std::fabs(b * gram) < 30.0 && gram < 30.0)) return false;
                gram *= b * b;
            }
            x *= q;
        }
    }
    return true;
}
// The products of all steps: joined ones first multiply the symmetric polynomials, and X by their product.
static bool orth_phases(OrthParams &q, const float *coef, int steps, int joined) {
    int64_t first = 0, need = 0, next = 0;
    int n = 0;
    auto add = [&](int kind, int a, int b, int out, float mul, const float *poly = nullptr, bool beside = false) {
        if (!beside) need = next;
        OrthPhase &f = q.phase[n++];
        std::memset(&f, 0, sizeof(f));
        f.first = (int32_t)first;
        f.need = (int32_t)need;
        f.kind = (int8_t)kind; f.a = (int8_t)a; f.b = (int8_t)b; f.out = (int8_t)out;
        f.mul = mul;
        if (poly) {
            f.poly = 1;
            f.mul = poly[2] * (kOrthUpPoly / (kOrthUp * kOrthUp));
            f.add = poly[1] * (kOrthUpPoly / kOrthUp);
            f.diag = poly[0] * kOrthUpPoly;
        }
        const int tiles = kind == kOrthProduct ? q.tiles_all : q.tiles_sym;
        first += (int64_t)q.batch * tiles * q.splits[kind];
        next += 16 * tiles;  // the epilogue warps of a pair
    };
    enum { GRAM = 2, POLY = 3, GRAM2 = 4, TEMP = 5, FACTOR = 6, POLY2 = 7 };
    int x = 0;
    for (int k0 = 0; k0 < steps; k0 += joined) {
        const int m = std::min(joined, steps - k0);
        int gram = GRAM, poly = POLY;
        add(kOrthGram, x, x, gram, 1.f / kOrthUp);
        for (int k = 0; k < m; ++k) {
            const int factor = k ? FACTOR : POLY;  // this step's own
            add(kOrthSquare, gram, gram, factor, 0.f, coef + 3 * (k0 + k));
            if (k + 1 < m) add(kOrthSquare, factor, gram, TEMP, 1.f / kOrthUpPoly);
            if (k) {  // (the pieces of a split tile have one place in the workspace)
                const int to = poly == POLY ? POLY2 : POLY;
                add(kOrthSquare, factor, poly, to, 1.f / kOrthUpPoly, nullptr, k + 1 < m && q.splits[kOrthSquare] == 1);
                poly = to;
            }
            if (k + 1 < m) {
                const int to = gram == GRAM ? GRAM2 : GRAM;
                add(kOrthSquare, TEMP, factor, to, 1.f / kOrthUpPoly);
                gram = to;
            }
        }
        const bool last = k0 + m >= steps, high = q.rows > q.cols;
        add(kOrthProduct, high ? x : poly, high ? poly : x, 1 - x, last ? 1.f / (kOrthUp * kOrthUpPoly) : 1.f / kOrthUpPoly);
        q.phase[n - 1].last = last;
        x = 1 - x;
    }
    q.phases = n;
    q.phase[n].first = (int32_t)first;
    q.matrices = joined > 1 ? kOrthMatrices : 4;
    return first <= kMostRows && next <= kMostRows;
}

conv_bwd_status conv_bwd_orth_create(const conv_bwd_orth_desc *d, conv_bwd_orth_plan *out) {
    if (!out) return CONV_BWD_ERR_INVALID_ARG;
    *out = nullptr;
    if (!d || d->batch < 1 || d->rows < 1 || d->cols < 1 || !known_dtype(d->dtype) || d->steps < 1 || !d->coefficients)
        return CONV_BWD_ERR_INVALID_ARG;
    if (d->batch > 65535 || d->rows > 65536 || d->cols > 65536 || d->batch * d->rows * d->cols > (1LL << 34) || d->steps > 64)
        return CONV_BWD_ERR_UNSUPPORTED;
    for (int i = 0; i < 3 * d->steps; ++i)
        if (!(std::fabs(d->coefficients[i]) <= 32.f)) return CONV_BWD_ERR_INVALID_ARG;
    return create_plan(out, [&](conv_bwd_orth_plan_s &p) {
        p.d = *d;
        p.d.coefficients = nullptr;
        int sms = 0, dev = 0;
        if (cudaGetDevice(&dev) == cudaSuccess &&
            cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            sms = 0;
        cudaGetLastError();
        const int64_t g = std::min(d->rows, d->cols), h = std::max(d->rows, d->cols);
        if (g <= kOrthSmall && h <= 8 * kOrthSlice) {
            for (p.cluster = 1; p.cluster * kOrthSlice < h;) p.cluster *= 2;
            p.coef.assign(d->coefficients, d->coefficients + 3 * d->steps);
            return p.dev.init(64);
        }
        const bool high = d->rows > d->cols;
        p.pitch = (int32_t)((d->cols + 7) / 8 * 8);
        p.most_parts = (int32_t)std::max<int64_t>(1, std::min<int64_t>((d->rows * d->cols + 4095) / 4096, 8LL * sms / d->batch));
        OrthParams &q = p.run;
        std::memset(&q, 0, sizeof(q));
        q.pitch_gram = (int32_t)((g + 7) / 8 * 8);
        q.rows = (int32_t)d->rows; q.cols = (int32_t)d->cols; q.batch = (int32_t)d->batch;
        p.pairs = sms > 1 ? orth_pairs(sms) : 0;
        if (sms > 1 && p.pairs < 1) return CONV_BWD_ERR_CUDA;
        const int64_t pairs = std::max(1, p.pairs);
        auto tiles_all = [&](int64_t w) { return (d->rows + 255) / 256 * ((d->cols + w - 1) / w); };
        auto tiles_sym = [&](int64_t w) {
            const int64_t mt = (g + 255) / 256;
            return mt * ((g + w - 1) / w) - mt * (mt - 1) / 2 * (256 / w);
        };
        // Wide tiles where the symmetric products have one for every pair.  (32 of 1024 x 2048 2197 us, narrow ones 2368; 50 of 489
        // x 1142 792 both ways.  Where they are fewer, in pieces, in an earlier form: 2 of 1024 x 4096, steps apart, 430, narrow ones
        // 413; 1000 x 1000 322, 217.)
        p.wide = tiles_sym(256) * d->batch >= pairs;
        const int64_t w = p.wide ? 256 : 128;
        q.tiles_sym = (int32_t)tiles_sym(w);
        q.tiles_all = (int32_t)tiles_all(w);
        // Pieces of a contraction, where pairs would else be idle: as many as make the shortest round.  (A k-block takes 0.65
        // us, the joining of two pieces 3.3, of three 3.7.  1000 x 1000 207 us, never in pieces 243; 600 x 600 in three of four
        // k-blocks 175, whole 177; 300 x 513 in two of five 142, whole 138.  700 x 700, whose rows are whole lines of memory, would be
        // faster whole than in three: 150, 161.)
        auto splits = [&](int64_t tiles, int64_t depth) {
            const int64_t blocks = (depth + 63) / 64, most = std::min(pairs / (tiles * d->batch), (int64_t)kOrthSplits);
            int32_t best = 1;
            double least = 0.65 * (double)blocks;
            for (int32_t k = 2; k <= most && k <= blocks; ++k) {
                const double takes = 0.65 * (double)((blocks + k - 1) / k) + 3.3 + 0.4 * (k - 2);
                if (takes < least) least = takes, best = k;
            }
            return best;
        };
        q.splits[0] = splits(q.tiles_sym, h);
        q.splits[1] = splits(q.tiles_sym, g);
        q.splits[2] = splits(q.tiles_all, g);
        for (int kind = 0; kind < 3; ++kind) {
            if (q.splits[kind] == 1) continue;
            const int32_t tiles = kind == kOrthProduct ? q.tiles_all : q.tiles_sym;
            q.own_tiles = std::max(q.own_tiles, tiles);
            q.own_pieces = std::max(q.own_pieces, tiles * q.splits[kind]);
        }
        // Three steps at a time (two products over the larger side instead of six, ten symmetric ones instead of three) where
        // X is large beside its Gram matrix, and sooner where products fill the machine than where each is a round of tiles.
        // (Joined, apart: 32 of 1024 x 2048 2197, 2702 us, x 1536 1971, 2171, x 1280 1852, 1907, x 1024 1720, 1606; 2 of 1024 x
        // 4096 303, 384; 1 of 200 x 4096 148, 166; 1000 x 1500 242, 215; 20 of 300 x 512 173, 155, of 256 x 600 142, 143.  Two
        // at a time took 8 to 10 % more than three.)
        const bool join = h >= 2 * g || (p.wide && 4 * h >= 5 * g);
        const int joined = join && orth_may_join(d->coefficients, d->steps, kOrthJoined) ? kOrthJoined : 1;
        if (!orth_phases(q, d->coefficients, d->steps, joined)) return CONV_BWD_ERR_UNSUPPORTED;
        auto lines = [](size_t n) { return (n + 255) / 256 * 256; };
        const bool split = q.splits[0] > 1 || q.splits[1] > 1 || q.splits[2] > 1;
        const size_t arrived = split ? lines((size_t)pairs * 16 * 4) : 0, parts = split ? (size_t)pairs * 256 * w * 4 : 0;
        const size_t done = lines((size_t)d->batch * 4), partial = lines((size_t)d->batch * p.most_parts * 16),
                     whole = lines((size_t)d->batch * d->rows * p.pitch * 2), square = lines((size_t)d->batch * g * q.pitch_gram * 2);
        p.dev.counters = 256 + arrived;
        const conv_bwd_status st = p.dev.init(256 + arrived + parts + done + partial + 4 * whole + (q.matrices - 2) * 2 * square);
        if (st != CONV_BWD_OK || !p.dev.has_device) return st;
        char *at = static_cast<char *>(p.dev.mem) + 256;
        q.arrived = reinterpret_cast<int32_t *>(at);
        at += arrived;
        q.parts = reinterpret_cast<float4 *>(at);
        at += parts;
        q.done = reinterpret_cast<int32_t *>(at);
        at += done;
        p.partial = reinterpret_cast<double *>(at);
        at += partial;
        bool ok = true;
        for (int i = 0; i < q.matrices; ++i) {
            const bool x = i < 2;
            const int64_t rows = x ? d->rows : g, cols = x ? d->cols : g, pitch = x ? p.pitch : q.pitch_gram;
            for (int plane = 0; plane < 2; ++plane, at += x ? whole : square) {
                q.at[i][plane] = reinterpret_cast<__half *>(at);
                ok = ok && map_plane(&q.maps[i].rows128[plane], at, d->batch, rows, cols, pitch, 64, 128) &&
                     map_plane(&q.maps[i].rows64[plane], at, d->batch, rows, cols, pitch, 64, 64) &&
                     map_plane(&q.maps[i].store[plane], at, d->batch, rows, cols, pitch, 64, 32);
                if (i == 0) p.x[plane] = reinterpret_cast<__half *>(at);
            }
        }
        if (!ok) return CONV_BWD_ERR_CUDA;
        q.status = p.dev.status();
        q.wait_budget = (int64_t)p.dev.clock_khz * 2000;
        return CONV_BWD_OK;
    });
}
conv_bwd_status conv_bwd_orth_destroy(conv_bwd_orth_plan p) {
    delete p;
    return CONV_BWD_OK;
}

// What the last product does with its result.
struct OrthOut {
    void *result = nullptr;
    float *weight = nullptr;
    __nv_bfloat16 *copy = nullptr;
    int64_t ldo = 0, lse = 0;
    float rate = 0.f, keep = 1.f;
};
static conv_bwd_status orth_run(conv_bwd_orth_plan p, OrthPrepParams &pp, const OrthOut &o, cudaStream_t s) {
    const conv_bwd_orth_desc &d = p->d;
    if (p->cluster) {
        OrthSmallParams q;
        std::memset(&q, 0, sizeof(q));
        q.grad = pp.grad; q.ls = pp.ls; q.ld = pp.ld;
        q.momentum = pp.momentum; q.beta = pp.beta; q.nesterov = pp.nesterov;
        q.result = o.result; q.weight = o.weight; q.copy = o.copy;
        q.ldo = o.ldo; q.lse = o.lse; q.rate = o.rate; q.keep = o.keep;
        q.status = p->dev.status();
        q.wait_budget = (int64_t)p->dev.clock_khz * 2000;
        q.rows = (int32_t)d.rows; q.cols = (int32_t)d.cols; q.batch = (int32_t)d.batch; q.steps = d.steps;
        q.cluster = p->cluster;
        q.slice = (int32_t)(((std::max(d.rows, d.cols) + p->cluster - 1) / p->cluster + 63) / 64 * 64);
        q.bf16 = d.dtype == CONV_BWD_BF16;
        std::copy(p->coef.begin(), p->coef.end(), q.coef);
        return launch_orth_small(q, s) == cudaSuccess ? CONV_BWD_OK : CONV_BWD_ERR_CUDA;
    }
    pp.hi = p->x[0];
    pp.lo = p->x[1];
    pp.partial = p->partial;
    pp.done = p->run.done;
    pp.batch = (int32_t)d.batch; pp.rows = (int32_t)d.rows; pp.cols = (int32_t)d.cols; pp.pitch = p->pitch;
    pp.parts = p->most_parts;
    pp.bf16 = d.dtype == CONV_BWD_BF16;
    if (launch_orth_prep(pp, s) != cudaSuccess) return CONV_BWD_ERR_CUDA;
    OrthParams q = p->run;
    q.segment = pp.bf16 ? 8 : 2;  // (of what a plan is given: bf16 has been rounded by more than the longer sums lose)
    q.result = o.result;
    q.bf16 = pp.bf16;
    q.weight = o.weight;
    q.copy = o.copy;
    q.ldo = o.ldo;
    q.lse = o.lse;
    q.rate = o.rate;
    q.keep = o.keep;
    return launch_orth_steps(q, p->wide, p->pairs, s) == cudaSuccess ? CONV_BWD_OK : CONV_BWD_ERR_CUDA;
}

// Checks a stack of matrices with row stride ld (0: cols) and matrix stride ls (0: rows ld) and fills the strides in.
static conv_bwd_status orth_strides(const conv_bwd_orth_desc &d, int64_t &ld, int64_t &ls, size_t es, size_t &bytes) {
    if (ld == 0) ld = d.cols;
    if (ld < d.cols) return CONV_BWD_ERR_INVALID_ARG;
    if (ld > (1LL << 31)) return CONV_BWD_ERR_UNSUPPORTED;
    if (ls == 0) ls = ld * d.rows;
    if (ls < ld * (d.rows - 1) + d.cols) return CONV_BWD_ERR_INVALID_ARG;
    if (ls > (1LL << 40)) return CONV_BWD_ERR_UNSUPPORTED;
    bytes = ((size_t)(d.batch - 1) * (size_t)ls + (size_t)(d.rows - 1) * (size_t)ld + (size_t)d.cols) * es;
    return CONV_BWD_OK;
}

conv_bwd_status conv_bwd_orth_apply(conv_bwd_orth_plan p, const void *x, int64_t ldx, int64_t lsx, void *out, int64_t ldo,
                                    int64_t lso, void *stream) {
    Range range("conv_bwd_orth_apply");
    if (!p || !x || !out) return CONV_BWD_ERR_INVALID_ARG;
    const size_t es = esize(p->d.dtype);
    size_t nx, no;
    conv_bwd_status st = orth_strides(p->d, ldx, lsx, es, nx);
    if (st == CONV_BWD_OK) st = orth_strides(p->d, ldo, lso, es, no);
    if (st != CONV_BWD_OK) return st;
    if (((uintptr_t)x | (uintptr_t)out) % es) return CONV_BWD_ERR_MISALIGNED;
    if (overlap(x, nx, out, no) && !(x == out && ldx == ldo && lsx == lso)) return CONV_BWD_ERR_INVALID_ARG;
    if (!p->dev.has_device) return CONV_BWD_ERR_CUDA;
    if (!p->dev.current()) return CONV_BWD_ERR_INVALID_ARG;
    OrthPrepParams pp;
    std::memset(&pp, 0, sizeof(pp));
    pp.grad = x;
    pp.ld = ldx;
    pp.ls = lsx;
    OrthOut o;
    o.result = out;
    o.ldo = ldo;
    o.lse = lso;
    return orth_run(p, pp, o, (cudaStream_t)stream);
}
conv_bwd_status conv_bwd_orth_update(conv_bwd_orth_plan p, float *weight, const void *grad, int64_t ldg, int64_t lsg, float *momentum,
                                     void *copy, float lr, float beta, int32_t nesterov, float decay, float scale, void *stream) {
    Range range("conv_bwd_orth_update");
    if (!p || !weight || !grad || !momentum) return CONV_BWD_ERR_INVALID_ARG;
    if (!std::isfinite(lr) || !std::isfinite(decay) || !std::isfinite(scale) || !(beta >= 0.f && beta <= 1.f)) return CONV_BWD_ERR_INVALID_ARG;
    if (!std::isfinite(lr * scale) || !std::isfinite(lr * decay)) return CONV_BWD_ERR_INVALID_ARG;  // (times a zero of X: NaN)
    const conv_bwd_orth_desc &d = p->d;
    const size_t es = esize(d.dtype), n = (size_t)d.batch * d.rows * d.cols;
    size_t ng;
    const conv_bwd_status st = orth_strides(d, ldg, lsg, es, ng);
    if (st != CONV_BWD_OK) return st;
    if (((uintptr_t)weight | (uintptr_t)momentum) % 4 || (uintptr_t)copy % 2 || (uintptr_t)grad % es) return CONV_BWD_ERR_MISALIGNED;
    if (overlap(weight, 4 * n, momentum, 4 * n) || overlap(weight, 4 * n, grad, ng) || overlap(momentum, 4 * n, grad, ng))
        return CONV_BWD_ERR_INVALID_ARG;
    if (copy && (overlap(copy, 2 * n, weight, 4 * n) || overlap(copy, 2 * n, momentum, 4 * n) || overlap(copy, 2 * n, grad, ng)))
        return CONV_BWD_ERR_INVALID_ARG;
    if (!p->dev.has_device) return CONV_BWD_ERR_CUDA;
    if (!p->dev.current()) return CONV_BWD_ERR_INVALID_ARG;
    OrthPrepParams pp;
    std::memset(&pp, 0, sizeof(pp));
    pp.grad = grad;
    pp.ld = ldg;
    pp.ls = lsg;
    pp.momentum = momentum;
    pp.beta = beta;
    pp.nesterov = nesterov ? 1 : 0;
    OrthOut o;
    o.weight = weight;
    o.copy = static_cast<__nv_bfloat16 *>(copy);
    o.ldo = d.cols;
    o.lse = d.rows * d.cols;
    o.rate = lr * scale;
    o.keep = 1.f - lr * decay;
    return orth_run(p, pp, o, (cudaStream_t)stream);
}
conv_bwd_status conv_bwd_orth_get_status(conv_bwd_orth_plan p, void *stream, int32_t *detail) {
    if (!p) return CONV_BWD_ERR_INVALID_ARG;
    return read_status(p->dev, stream, detail);
}

}  // extern "C"
