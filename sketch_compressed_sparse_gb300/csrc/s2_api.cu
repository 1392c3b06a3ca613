// C ABI of libs2: argument validation and dispatch to the kernels. Every
// entry point checks its arguments completely before anything is launched,
// then queues its kernels on the caller's stream and returns.
#include <cmath>
#include <cstring>
#include <initializer_list>
#include <mutex>

#include "s2.h"  // include/ is on the include path
#include "s2_header_id.h"
#include "s2_internal.h"

namespace s2 {

cudaError_t device_info(DeviceInfo* out) {
    static DeviceInfo cache[64];
    static std::once_flag once[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    cudaError_t err = cudaSuccess;
    std::call_once(once[dev], [&] {
        DeviceInfo di{};
        err = cudaDeviceGetAttribute(&di.sms, cudaDevAttrMultiProcessorCount, dev);
        if (err == cudaSuccess) err = cudaDeviceGetAttribute(&di.l2_bytes, cudaDevAttrL2CacheSize, dev);
        cache[dev] = di;
    });
    if (err != cudaSuccess) return err;
    if (cache[dev].sms <= 0) return cudaErrorInvalidDevice;
    *out = cache[dev];
    return cudaSuccess;
}

int blocks_per_sm(const void* fn, int threads, size_t smem) {
    struct Entry {
        int dev;
        const void* fn;
        int threads;
        size_t smem;
        int per_sm;
    };
    static std::mutex mu;
    static Entry table[512];
    static int used = 0;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) dev = -1;
    {
        std::lock_guard<std::mutex> lock(mu);
        for (int x = 0; x < used; ++x)
            if (table[x].dev == dev && table[x].fn == fn && table[x].threads == threads && table[x].smem == smem)
                return table[x].per_sm;
    }
    int per_sm = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, fn, threads, smem) != cudaSuccess || per_sm < 1) {
        cudaGetLastError();  // a failed query is not a launch error
        return 1;
    }
    std::lock_guard<std::mutex> lock(mu);
    if (used < 512) table[used++] = Entry{dev, fn, threads, smem, per_sm};
    return per_sm;
}

static uint32_t host_fmix32(uint32_t x) {
    x ^= x >> 16;
    x *= 0x85ebca6bu;
    x ^= x >> 13;
    x *= 0xc2b2ae35u;
    x ^= x >> 16;
    return x;
}

RowKeys make_keys(uint32_t seed, uint32_t d) {
    RowKeys k;
    std::memset(&k, 0, sizeof(k));
    const uint32_t golden = 0x9E3779B9u;
    for (uint32_t j = 0; j < d && j < (uint32_t)kMaxRows; ++j) {
        k.kh[j] = host_fmix32(seed ^ (uint32_t)(golden * (2u * j + 1u)));
        k.ks[j] = host_fmix32(seed ^ (uint32_t)(golden * (2u * j + 2u)));
    }
    return k;
}

}  // namespace s2

using namespace s2;

namespace {

constexpr uint64_t kMaxN = 0xffffffffull;  // positions are 32-bit
static_assert(kPrivMaxBytes == S2_SMEM_SKETCH_MAX_BYTES, "shared-memory sketch limit differs from the header");

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Byte ranges [a, a+na) and [b, b+nb) intersect (empty ranges never do).
inline bool overlap(const void* a, uint64_t na, const void* b, uint64_t nb) {
    if (na == 0 || nb == 0 || a == nullptr || b == nullptr) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

inline s2_status check_params(const s2_params& p) {
    if (p.d < 1 || p.d > S2_MAX_ROWS) return S2_ERR_INVALID_ARG;
    if (p.w < 1 || p.w > (1u << 31)) return S2_ERR_INVALID_ARG;
    return S2_OK;
}

inline uint64_t words_of(uint64_t n) { return (n + 31) / 32; }

inline s2_status cuda_status(cudaError_t e) { return e == cudaSuccess ? S2_OK : S2_ERR_CUDA; }

inline size_t round256(size_t x) { return (x + 255) / 256 * 256; }

// Encode W workers: zero the sketches and fill them, in groups of workers
// whose sketches fit in half of L2 together, so that each group's
// sketches are zeroed, updated and written back once.
s2_status encode_impl(const void* grad, s2_dtype dt, uint32_t W, uint64_t n, s2_params p, uint32_t* bitmaps,
                      float* sketches, cudaStream_t stream, uint32_t block = 0,
                      s2_encode_path path = S2_PATH_AUTO) {
    const uint64_t esz = dt == S2_F32 ? 4 : 2;
    const uint64_t nw = words_of(n);
    const uint64_t dw = (uint64_t)p.d * p.w;
    DeviceInfo di{};
    cudaError_t e = device_info(&di);
    if (e != cudaSuccess) return S2_ERR_CUDA;
    const uint64_t sk_bytes = dw * 4;
    uint64_t group = sk_bytes ? ((uint64_t)di.l2_bytes / 2) / sk_bytes : W;
    if (group < 1) group = 1;
    if (group > W) group = W;
    // A sketch too large to stay in L2 while it is built (above 3/4 of L2:
    // its reductions would go to DRAM) is built one worker at a time in
    // `passes` slices of its flattened buckets, each pass re-reading the
    // worker's gradient and updating only its slice. Element bitmaps only.
    // Measured on GB300 (8 workers of 2^27 positions at 10 % density): a
    // 160 MB sketch in two passes 5.6 ms instead of 10.7 ms; a 96 MB sketch
    // 3.7 ms in one pass, 4.1 ms in two.
    const uint64_t slice_cap = (uint64_t)di.l2_bytes / 4 * 3;
    uint64_t passes = 1;
    if (sk_bytes > slice_cap && path != S2_PATH_SMEM && block == 0) {
        passes = (sk_bytes + slice_cap - 1) / slice_cap;
        group = 1;
    }
    // vector loads need every worker row 16-byte aligned
    const bool vec = ((n * esz) % 16 == 0) || W == 1;
    EncodeArgs a;
    std::memset(&a, 0, sizeof(a));
    a.n = n;
    a.nw = nw;
    a.dw = dw;
    a.tasks_per_worker = (uint32_t)((n + kTaskElems - 1) / kTaskElems);
    a.d = p.d;
    a.w = p.w;
    a.keys = make_keys(p.seed, p.d);
    const uint64_t nbw = block ? words_of((n + block - 1) / block) : 0;
    a.block_words = block / 32;
    a.nbw = nbw;
    a.x_lo = 0;
    a.x_span = dw;
    if (block && W * nbw) {  // block bits are set with atomicOr: start from zero
        e = launch_zero(reinterpret_cast<float*>(bitmaps), W * nbw, stream);
        if (e != cudaSuccess) return S2_ERR_CUDA;
    }
    if (path != S2_PATH_L2 && sk_bytes <= kPrivMaxBytes) {
        a.grad = grad;
        a.bitmaps = bitmaps;
        a.sketches = sketches;
        a.workers = W;
        bool launched = false;
        e = launch_encode_smem(a, dt == S2_F32 ? 0 : 1, vec, path == S2_PATH_AUTO, &launched, stream);
        if (e != cudaSuccess) return S2_ERR_CUDA;
        if (launched) return S2_OK;
    }
    for (uint64_t k0 = 0; k0 < W; k0 += group) {
        const uint64_t g = (W - k0) < group ? (W - k0) : group;
        a.grad = static_cast<const char*>(grad) + k0 * n * esz;
        a.bitmaps = bitmaps + k0 * (block ? nbw : nw);
        a.sketches = sketches + k0 * dw;
        a.workers = (uint32_t)g;
        if (passes == 1) {
            e = launch_zero(sketches + k0 * dw, g * dw, stream);
            if (e != cudaSuccess) return S2_ERR_CUDA;
            e = launch_encode(a, dt == S2_F32 ? 0 : 1, vec, stream);
            if (e != cudaSuccess) return S2_ERR_CUDA;
            continue;
        }
        // one worker, slice by slice (the bitmap is rewritten with the same
        // words on every pass; block bits are ORed again)
        const uint64_t span = (dw + passes - 1) / passes;
        for (uint64_t x0 = 0; x0 < dw; x0 += span) {
            a.x_lo = x0;
            a.x_span = (dw - x0) < span ? (dw - x0) : span;
            e = launch_zero(sketches + k0 * dw + x0, a.x_span, stream);
            if (e != cudaSuccess) return S2_ERR_CUDA;
            e = launch_encode(a, dt == S2_F32 ? 0 : 1, vec, stream);
            if (e != cudaSuccess) return S2_ERR_CUDA;
        }
        a.x_lo = 0;
        a.x_span = dw;
    }
    return S2_OK;
}

s2_status check_encode(const void* grad, s2_dtype dt, uint32_t W, uint64_t n, s2_params p, const uint32_t* bitmaps,
                       const float* sketches) {
    s2_status st = check_params(p);
    if (st != S2_OK) return st;
    if (dt != S2_F32 && dt != S2_BF16) return S2_ERR_INVALID_ARG;
    if (n > kMaxN) return S2_ERR_UNSUPPORTED;
    if (W == 0) return S2_OK;
    const uint64_t esz = dt == S2_F32 ? 4 : 2;
    const uint64_t gbytes = (uint64_t)W * n * esz, bbytes = (uint64_t)W * words_of(n) * 4,
                   sbytes = (uint64_t)W * p.d * p.w * 4;
    if (!sketches || (n > 0 && (!grad || !bitmaps))) return S2_ERR_INVALID_ARG;
    if (!aligned(grad, 16) || !aligned(bitmaps, 16) || !aligned(sketches, 16)) return S2_ERR_ALIGNMENT;
    if (overlap(grad, gbytes, bitmaps, bbytes) || overlap(grad, gbytes, sketches, sbytes) ||
        overlap(bitmaps, bbytes, sketches, sbytes))
        return S2_ERR_INVALID_ARG;
    return S2_OK;
}

s2_status check_reduce(const uint32_t* bitmaps, const float* sketches, uint32_t W, uint64_t n, s2_params p,
                       const uint32_t* bitmap_out, const float* sketch_out) {
    s2_status st = check_params(p);
    if (st != S2_OK) return st;
    if (n > kMaxN) return S2_ERR_UNSUPPORTED;
    const uint64_t nw = words_of(n), dw = (uint64_t)p.d * p.w;
    if (!sketch_out || (nw > 0 && !bitmap_out)) return S2_ERR_INVALID_ARG;
    if (W > 0 && (!sketches || (nw > 0 && !bitmaps))) return S2_ERR_INVALID_ARG;
    if (!aligned(bitmaps, 16) || !aligned(sketches, 16) || !aligned(bitmap_out, 16) || !aligned(sketch_out, 16))
        return S2_ERR_ALIGNMENT;
    const uint64_t ib = (uint64_t)W * nw * 4, is = (uint64_t)W * dw * 4;
    if (overlap(bitmaps, ib, bitmap_out, nw * 4) || overlap(bitmaps, ib, sketch_out, dw * 4) ||
        overlap(sketches, is, bitmap_out, nw * 4) || overlap(sketches, is, sketch_out, dw * 4) ||
        overlap(bitmap_out, nw * 4, sketch_out, dw * 4))
        return S2_ERR_INVALID_ARG;
    return S2_OK;
}

s2_status check_decode_dense(const uint32_t* bitmap, const float* sketch, uint64_t n, s2_params p, const float* out) {
    s2_status st = check_params(p);
    if (st != S2_OK) return st;
    if (n > kMaxN) return S2_ERR_UNSUPPORTED;
    if (n == 0) return S2_OK;
    if (!bitmap || !sketch || !out) return S2_ERR_INVALID_ARG;
    if (!aligned(bitmap, 16) || !aligned(sketch, 16) || !aligned(out, 16)) return S2_ERR_ALIGNMENT;
    const uint64_t dw = (uint64_t)p.d * p.w;
    if (overlap(out, n * 4, bitmap, words_of(n) * 4) || overlap(out, n * 4, sketch, dw * 4))
        return S2_ERR_INVALID_ARG;
    return S2_OK;
}

DecodeArgs make_decode_args(const uint32_t* bitmap, const float* sketch, uint64_t n, s2_params p, float scale) {
    DecodeArgs a;
    std::memset(&a, 0, sizeof(a));
    a.bitmap = bitmap;
    a.sketch = sketch;
    a.n = n;
    a.nw = words_of(n);
    a.d = p.d;
    a.w = p.w;
    a.scale = scale;
    a.keys = make_keys(p.seed, p.d);
    return a;
}

// Device address of page-locked host memory at `p` that the current device
// can access in place (16-byte aligned), or nullptr for any other memory.
const void* mapped_host(const void* p) {
    if (!p) return nullptr;
    cudaPointerAttributes at{};
    if (cudaPointerGetAttributes(&at, p) != cudaSuccess) {
        cudaGetLastError();  // an unknown pointer is not an error here
        return nullptr;
    }
    if (at.type != cudaMemoryTypeHost || !at.devicePointer || !aligned(at.devicePointer, 16)) return nullptr;
    return at.devicePointer;
}

struct PipelineLayout {
    size_t grad, bitmaps, sketches, bitmap, sketch, out, dec_ws, total;
};

PipelineLayout pipeline_layout(s2_dtype dt, uint32_t W, uint64_t n, s2_params p) {
    const uint64_t esz = dt == S2_F32 ? 4 : 2, nw = words_of(n), dw = (uint64_t)p.d * p.w;
    PipelineLayout L{};
    size_t off = 0;
    L.grad = off;
    off += round256((size_t)W * n * esz);
    L.bitmaps = off;
    off += round256((size_t)W * nw * 4);
    L.sketches = off;
    off += round256((size_t)W * dw * 4);
    L.bitmap = off;
    off += round256((size_t)nw * 4);
    L.sketch = off;
    off += round256((size_t)dw * 4);
    L.out = off;
    off += round256((size_t)n * 4);
    L.dec_ws = off;
    off += round256(dense_workspace_bytes(n, p.d));
    L.total = off;
    return L;
}

// ---- 8-bit layer ----
constexpr uint64_t kMaxDim8 = 0x7fffffffull;   // sizes travel as 32-bit coordinates
constexpr uint64_t kMaxSpan8 = 1ull << 48;     // elements from a matrix's first to its last row

inline uint64_t blocks8(uint64_t n) { return (n + 127) / 128; }
inline uint64_t size_of(s2_dtype dt) { return dt == S2_F32 ? 4 : 2; }
inline bool dtype_ok(s2_dtype dt) { return dt == S2_F32 || dt == S2_BF16; }
inline bool layout_ok(s2_scale_layout l) { return l == S2_SCALE_ROWS || l == S2_SCALE_TILES; }

// Bytes from the first to the last element of `rows` rows, `ld` elements apart.
inline uint64_t extent(uint64_t rows, uint64_t cols, uint64_t ld, uint64_t esz) {
    return rows && cols ? ((rows - 1) * ld + cols) * esz : 0;
}

// A matrix argument: its row stride covers a row and its bytes are addressable.
inline s2_status check_matrix(uint64_t rows, uint64_t cols, uint64_t ld) {
    if (rows > kMaxDim8 || cols > kMaxDim8 || ld >= (1ull << 35)) return S2_ERR_UNSUPPORTED;  // tensor maps: 2^40 bytes
    if (rows > 1 && ld && rows - 1 > kMaxSpan8 / ld) return S2_ERR_UNSUPPORTED;
    return rows > 1 && ld < cols ? S2_ERR_INVALID_ARG : S2_OK;
}

// Codes: rows start on 16 bytes, as the tiled copies need them.
inline s2_status check_codes(const void* codes, uint64_t rows, uint64_t cols, uint64_t ld) {
    const s2_status st = check_matrix(rows, cols, ld);
    if (st != S2_OK) return st;
    if (!codes) return S2_ERR_INVALID_ARG;
    return aligned(codes, 16) && (rows <= 1 || ld % 16 == 0) ? S2_OK : S2_ERR_ALIGNMENT;
}

// ---- 4-bit layer ----
constexpr uint64_t kMaxItems4 = 0x7fffffffull * 8;  // a warp each, eight warps a block

inline uint64_t bytes4(uint64_t cols) { return (cols + 1) / 2; }
inline uint64_t scales4(uint64_t rows, uint64_t cols) { return blocks8(rows) * blocks8(cols) * 512; }

// A packed matrix: rows of codes start on 16 bytes, and so do the scales.
inline s2_status check_packed4(const void* codes, uint64_t rows, uint64_t cols, uint64_t ldc, const void* scales) {
    if (!scales) return S2_ERR_INVALID_ARG;
    const s2_status st = check_codes(codes, rows, bytes4(cols), ldc);
    if (st != S2_OK) return st;
    return aligned(scales, 16) ? S2_OK : S2_ERR_ALIGNMENT;
}

// Row stride of codes for their tensor map, which wants a multiple of 16; that of a single row is free.
inline uint64_t stride16(uint64_t rows, uint64_t cols, uint64_t ld) { return rows > 1 ? ld : (cols + 15) / 16 * 16; }

inline s2_status first_error(std::initializer_list<s2_status> all) {
    for (s2_status st : all)
        if (st != S2_OK) return st;
    return S2_OK;
}

struct Span {
    const void* p;
    uint64_t bytes;
};
// Some output overlaps an input or another output (the first `outs` spans are outputs).
inline bool clash(std::initializer_list<Span> spans, size_t outs) {
    for (size_t i = 0; i < outs; ++i)
        for (size_t j = i + 1; j < spans.size(); ++j)
            if (overlap(spans.begin()[i].p, spans.begin()[i].bytes, spans.begin()[j].p, spans.begin()[j].bytes))
                return true;
    return false;
}

}  // namespace

extern "C" {

s2_status s2_encode(const void* grad, s2_dtype dt, uint64_t n, s2_params p, uint32_t* bitmap, float* sketch,
                    s2_stream_t stream) {
    s2_status st = check_encode(grad, dt, 1, n, p, bitmap, sketch);
    if (st != S2_OK) return st;
    return encode_impl(grad, dt, 1, n, p, bitmap, sketch, reinterpret_cast<cudaStream_t>(stream));
}

s2_status s2_encode_batched(const void* grad, s2_dtype dt, uint32_t W, uint64_t n, s2_params p, uint32_t* bitmaps,
                            float* sketches, s2_stream_t stream) {
    s2_status st = check_encode(grad, dt, W, n, p, bitmaps, sketches);
    if (st != S2_OK || W == 0) return st;
    return encode_impl(grad, dt, W, n, p, bitmaps, sketches, reinterpret_cast<cudaStream_t>(stream));
}

s2_status s2_encode_batched_path(const void* grad, s2_dtype dt, uint32_t W, uint64_t n, s2_params p,
                                 s2_encode_path path, uint32_t* bitmaps, float* sketches, s2_stream_t stream) {
    if (path != S2_PATH_AUTO && path != S2_PATH_L2 && path != S2_PATH_SMEM) return S2_ERR_INVALID_ARG;
    s2_status st = check_encode(grad, dt, W, n, p, bitmaps, sketches);
    if (st != S2_OK) return st;
    if (path == S2_PATH_SMEM && (uint64_t)p.d * p.w * 4 > S2_SMEM_SKETCH_MAX_BYTES) return S2_ERR_UNSUPPORTED;
    if (W == 0) return S2_OK;
    return encode_impl(grad, dt, W, n, p, bitmaps, sketches, reinterpret_cast<cudaStream_t>(stream), 0, path);
}

s2_status s2_encode_batched_blocks(const void* grad, s2_dtype dt, uint32_t W, uint64_t n, uint32_t block,
                                   s2_params p, uint32_t* block_bitmaps, float* sketches, s2_stream_t stream) {
    s2_status st = check_params(p);
    if (st != S2_OK) return st;
    if (dt != S2_F32 && dt != S2_BF16) return S2_ERR_INVALID_ARG;
    if (block == 0 || block % 32 != 0) return S2_ERR_UNSUPPORTED;
    if (n > kMaxN) return S2_ERR_UNSUPPORTED;
    if (W == 0) return S2_OK;
    const uint64_t esz = dt == S2_F32 ? 4 : 2;
    const uint64_t nbw = words_of((n + block - 1) / block);
    const uint64_t gbytes = (uint64_t)W * n * esz, bbytes = (uint64_t)W * nbw * 4,
                   sbytes = (uint64_t)W * p.d * p.w * 4;
    if (!sketches || (n > 0 && (!grad || !block_bitmaps))) return S2_ERR_INVALID_ARG;
    if (!aligned(grad, 16) || !aligned(block_bitmaps, 16) || !aligned(sketches, 16)) return S2_ERR_ALIGNMENT;
    if (overlap(grad, gbytes, block_bitmaps, bbytes) || overlap(grad, gbytes, sketches, sbytes) ||
        overlap(block_bitmaps, bbytes, sketches, sbytes))
        return S2_ERR_INVALID_ARG;
    return encode_impl(grad, dt, W, n, p, block_bitmaps, sketches, reinterpret_cast<cudaStream_t>(stream), block);
}

s2_status s2_decode_dense_blocks(const uint32_t* block_bitmap, const float* sketch, uint64_t n, uint32_t block,
                                 s2_params p, float scale, float* out, s2_stream_t stream) {
    s2_status st = check_params(p);
    if (st != S2_OK) return st;
    if (block == 0 || block % 32 != 0 || n > kMaxN) return S2_ERR_UNSUPPORTED;
    if (n == 0) return S2_OK;
    if (!block_bitmap || !sketch || !out) return S2_ERR_INVALID_ARG;
    if (!aligned(block_bitmap, 16) || !aligned(sketch, 16) || !aligned(out, 16)) return S2_ERR_ALIGNMENT;
    const uint64_t dw = (uint64_t)p.d * p.w, nbw = words_of((n + block - 1) / block);
    if (overlap(out, n * 4, block_bitmap, nbw * 4) || overlap(out, n * 4, sketch, dw * 4)) return S2_ERR_INVALID_ARG;
    DecodeArgs a = make_decode_args(block_bitmap, sketch, n, p, scale);
    a.nw = nbw;
    a.block = block;
    return cuda_status(launch_decode_dense(a, out, reinterpret_cast<cudaStream_t>(stream)));
}

s2_status s2_block_topk_workspace_size(uint32_t W, uint64_t n, uint32_t block, size_t* bytes) {
    if (!bytes) return S2_ERR_INVALID_ARG;
    if (block == 0 || block % 32 != 0 || n > kMaxN) return S2_ERR_UNSUPPORTED;
    *bytes = topk_workspace_bytes(W, n, block);
    return S2_OK;
}

s2_status s2_block_topk(const float* grad, float* residual, uint32_t W, uint64_t n, uint32_t block, uint64_t K,
                        float* sparse_out, void* workspace, size_t workspace_bytes, s2_stream_t stream) {
    if (block == 0 || block % 32 != 0 || n > kMaxN) return S2_ERR_UNSUPPORTED;
    const uint64_t nb = (n + block - 1) / block, bytes = (uint64_t)W * n * 4;
    if (K > nb) return S2_ERR_INVALID_ARG;
    if (bytes == 0) return S2_OK;
    const size_t need = topk_workspace_bytes(W, n, block);
    if (!grad || !residual || !sparse_out || !workspace || workspace_bytes < need) return S2_ERR_INVALID_ARG;
    if (!aligned(grad, 16) || !aligned(residual, 16) || !aligned(sparse_out, 16) || !aligned(workspace, 16))
        return S2_ERR_ALIGNMENT;
    if (overlap(grad, bytes, residual, bytes) || overlap(grad, bytes, sparse_out, bytes) ||
        overlap(residual, bytes, sparse_out, bytes) || overlap(workspace, need, grad, bytes) ||
        overlap(workspace, need, residual, bytes) || overlap(workspace, need, sparse_out, bytes))
        return S2_ERR_INVALID_ARG;
    return cuda_status(
        launch_block_topk(grad, residual, W, n, block, K, sparse_out, workspace, reinterpret_cast<cudaStream_t>(stream)));
}

s2_status s2_sparse_pack_workspace_size(uint32_t W, uint64_t n, size_t* bytes) {
    if (!bytes) return S2_ERR_INVALID_ARG;
    if (n > kMaxN) return S2_ERR_UNSUPPORTED;
    *bytes = pack_workspace_bytes(W, n);
    return S2_OK;
}

s2_status s2_sparse_pack(const float* grad, uint32_t W, uint64_t n, uint32_t* idx_out, float* val_out,
                         uint64_t capacity, uint64_t* counts_out, void* workspace, size_t workspace_bytes,
                         s2_stream_t stream) {
    if (n > kMaxN) return S2_ERR_UNSUPPORTED;
    if (W == 0) return S2_OK;
    const size_t need = pack_workspace_bytes(W, n);
    const uint64_t gbytes = (uint64_t)W * n * 4, lbytes = (uint64_t)W * capacity * 4;
    if (!counts_out || (n > 0 && (!grad || !workspace || workspace_bytes < need)) ||
        (capacity > 0 && (!idx_out || !val_out)))
        return S2_ERR_INVALID_ARG;
    if (!aligned(grad, 16) || !aligned(idx_out, 4) || !aligned(val_out, 4) || !aligned(counts_out, 8) ||
        !aligned(workspace, 16))
        return S2_ERR_ALIGNMENT;
    const void* outs[4] = {idx_out, val_out, counts_out, workspace};
    const uint64_t osz[4] = {lbytes, lbytes, (uint64_t)W * 8, need};
    for (int o = 0; o < 4; ++o) {
        if (overlap(grad, gbytes, outs[o], osz[o])) return S2_ERR_INVALID_ARG;
        for (int q = o + 1; q < 4; ++q)
            if (overlap(outs[o], osz[o], outs[q], osz[q])) return S2_ERR_INVALID_ARG;
    }
    return cuda_status(launch_sparse_pack(grad, W, n, idx_out, val_out, capacity,
                                          reinterpret_cast<unsigned long long*>(counts_out), workspace,
                                          reinterpret_cast<cudaStream_t>(stream)));
}

s2_status s2_sparse_sum(const uint32_t* idx, const float* val, const uint64_t* counts, uint32_t W, uint64_t capacity,
                        uint64_t n, float* out, s2_stream_t stream) {
    if (n > kMaxN) return S2_ERR_UNSUPPORTED;
    if (n == 0) return S2_OK;
    const uint64_t lbytes = (uint64_t)W * capacity * 4;
    if (!out || (W > 0 && (!counts || (capacity > 0 && (!idx || !val))))) return S2_ERR_INVALID_ARG;
    if (!aligned(out, 16) || !aligned(idx, 4) || !aligned(val, 4) || !aligned(counts, 8)) return S2_ERR_ALIGNMENT;
    if (overlap(out, n * 4, idx, lbytes) || overlap(out, n * 4, val, lbytes) || overlap(out, n * 4, counts, W * 8ull))
        return S2_ERR_INVALID_ARG;
    return cuda_status(launch_sparse_sum(idx, val, reinterpret_cast<const unsigned long long*>(counts), W, capacity, n,
                                         out, reinterpret_cast<cudaStream_t>(stream)));
}

s2_status s2_reduce(const uint32_t* bitmaps, const float* sketches, uint32_t W, uint64_t n, s2_params p,
                    uint32_t* bitmap_out, float* sketch_out, s2_stream_t stream) {
    s2_status st = check_reduce(bitmaps, sketches, W, n, p, bitmap_out, sketch_out);
    if (st != S2_OK) return st;
    const uint64_t nw = words_of(n), dw = (uint64_t)p.d * p.w;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (W == 0) {
        cudaError_t e = launch_zero(sketch_out, dw, s);
        if (e == cudaSuccess && nw) e = launch_zero(reinterpret_cast<float*>(bitmap_out), nw, s);
        return cuda_status(e);
    }
    return cuda_status(launch_reduce(bitmaps, sketches, W, nw, dw, bitmap_out, sketch_out, s));
}

s2_status s2_encode_reduce_fused(const void* grad, s2_dtype dt, uint32_t W, uint64_t n, s2_params p,
                                 uint32_t* bitmap_out, float* sketch_out, s2_stream_t stream) {
    s2_status st = check_params(p);
    if (st != S2_OK) return st;
    if (dt != S2_F32 && dt != S2_BF16) return S2_ERR_INVALID_ARG;
    if (n > kMaxN) return S2_ERR_UNSUPPORTED;
    const uint64_t esz = dt == S2_F32 ? 4 : 2, nw = words_of(n), dw = (uint64_t)p.d * p.w;
    const uint64_t gbytes = (uint64_t)W * n * esz;
    if (!sketch_out || (nw > 0 && !bitmap_out) || (gbytes > 0 && !grad)) return S2_ERR_INVALID_ARG;
    if (!aligned(grad, 16) || !aligned(bitmap_out, 16) || !aligned(sketch_out, 16)) return S2_ERR_ALIGNMENT;
    if (overlap(grad, gbytes, bitmap_out, nw * 4) || overlap(grad, gbytes, sketch_out, dw * 4) ||
        overlap(bitmap_out, nw * 4, sketch_out, dw * 4))
        return S2_ERR_INVALID_ARG;
    FusedArgs a;
    std::memset(&a, 0, sizeof(a));
    a.grad = grad;
    a.bitmap = bitmap_out;
    a.sketch = sketch_out;
    a.n = n;
    a.nw = nw;
    a.workers = W;
    a.d = p.d;
    a.w = p.w;
    a.keys = make_keys(p.seed, p.d);
    return cuda_status(launch_fused(a, dt == S2_F32 ? 0 : 1, reinterpret_cast<cudaStream_t>(stream)));
}

s2_status s2_decode_dense(const uint32_t* bitmap, const float* sketch, uint64_t n, s2_params p, float scale,
                          float* out, s2_stream_t stream) {
    s2_status st = check_decode_dense(bitmap, sketch, n, p, out);
    if (st != S2_OK || n == 0) return st;
    return cuda_status(
        launch_decode_dense(make_decode_args(bitmap, sketch, n, p, scale), out, reinterpret_cast<cudaStream_t>(stream)));
}

s2_status s2_decode_dense_workspace_size(uint64_t n, s2_params p, size_t* bytes) {
    if (!bytes) return S2_ERR_INVALID_ARG;
    s2_status st = check_params(p);
    if (st != S2_OK) return st;
    if (n > kMaxN) return S2_ERR_UNSUPPORTED;
    *bytes = dense_workspace_bytes(n, p.d);
    return S2_OK;
}

s2_status s2_decode_dense_ws(const uint32_t* bitmap, const float* sketch, uint64_t n, s2_params p, float scale,
                             float* out, void* workspace, size_t workspace_bytes, s2_stream_t stream) {
    s2_status st = check_decode_dense(bitmap, sketch, n, p, out);
    if (st != S2_OK || n == 0) return st;
    const size_t need = dense_workspace_bytes(n, p.d);
    if (workspace_bytes < need || (need > 0 && !workspace)) return S2_ERR_INVALID_ARG;
    if (!aligned(workspace, 16)) return S2_ERR_ALIGNMENT;
    const uint64_t dw = (uint64_t)p.d * p.w;
    if (overlap(workspace, need, out, n * 4) || overlap(workspace, need, bitmap, words_of(n) * 4) ||
        overlap(workspace, need, sketch, dw * 4))
        return S2_ERR_INVALID_ARG;
    return cuda_status(launch_decode_dense_ws(make_decode_args(bitmap, sketch, n, p, scale), out,
                                              static_cast<float*>(workspace), reinterpret_cast<cudaStream_t>(stream)));
}

s2_status s2_decode_workspace_size(uint64_t n, size_t* bytes) {
    if (!bytes) return S2_ERR_INVALID_ARG;
    if (n > kMaxN) return S2_ERR_UNSUPPORTED;
    *bytes = compact_workspace_bytes(n);
    return S2_OK;
}

}  // extern "C"

namespace {
// Argument checks shared by both compacted decodes (everything but the workspace).
s2_status check_decode_compact(const uint32_t* bitmap, const float* sketch, uint64_t n, s2_params p,
                               const uint32_t* idx_out, const float* val_out, uint64_t capacity,
                               const uint64_t* count_out, const void* workspace, size_t ws_bytes) {
    s2_status st = check_params(p);
    if (st != S2_OK) return st;
    if (n > kMaxN) return S2_ERR_UNSUPPORTED;
    if (!count_out) return S2_ERR_INVALID_ARG;
    if (n > 0 && (!bitmap || !sketch)) return S2_ERR_INVALID_ARG;
    if (capacity > 0 && (!idx_out || !val_out)) return S2_ERR_INVALID_ARG;
    if (!aligned(bitmap, 16) || !aligned(sketch, 16) || !aligned(workspace, 16) || !aligned(idx_out, 4) ||
        !aligned(val_out, 4) || !aligned(count_out, 8))
        return S2_ERR_ALIGNMENT;
    const uint64_t nw = words_of(n), dw = (uint64_t)p.d * p.w, cap = capacity < n ? capacity : n;
    const void* ins[2] = {bitmap, sketch};
    const uint64_t insz[2] = {nw * 4, dw * 4};
    const void* outs[4] = {idx_out, val_out, count_out, workspace};
    const uint64_t outsz[4] = {cap * 4, cap * 4, 8, ws_bytes};
    for (int i = 0; i < 2; ++i)
        for (int o = 0; o < 4; ++o)
            if (overlap(ins[i], insz[i], outs[o], outsz[o])) return S2_ERR_INVALID_ARG;
    for (int o = 0; o < 4; ++o)
        for (int q = o + 1; q < 4; ++q)
            if (overlap(outs[o], outsz[o], outs[q], outsz[q])) return S2_ERR_INVALID_ARG;
    return S2_OK;
}
}  // namespace

extern "C" {

s2_status s2_decode_compact(const uint32_t* bitmap, const float* sketch, uint64_t n, s2_params p, float scale,
                            uint32_t* idx_out, float* val_out, uint64_t capacity, uint64_t* count_out,
                            void* workspace, size_t workspace_bytes, s2_stream_t stream) {
    if (n <= kMaxN) {
        const size_t need = compact_workspace_bytes(n);
        if (workspace_bytes < need || (need > 0 && !workspace)) {
            s2_status st = check_params(p);
            return st != S2_OK ? st : S2_ERR_INVALID_ARG;
        }
    }
    s2_status st = check_decode_compact(bitmap, sketch, n, p, idx_out, val_out, capacity, count_out, workspace,
                                        n <= kMaxN ? compact_workspace_bytes(n) : 0);
    if (st != S2_OK) return st;
    const uint64_t tiles = compact_tiles(words_of(n));
    uint32_t* counts = static_cast<uint32_t*>(workspace);
    uint32_t* offsets = counts + (round256(tiles * 4) / 4);
    return cuda_status(launch_decode_compact(make_decode_args(bitmap, sketch, n, p, scale), idx_out, val_out, capacity,
                                             reinterpret_cast<unsigned long long*>(count_out), counts, offsets,
                                             reinterpret_cast<cudaStream_t>(stream)));
}

s2_status s2_decode_compact_noalloc(const uint32_t* bitmap, const float* sketch, uint64_t n, s2_params p, float scale,
                                    uint32_t* idx_out, float* val_out, uint64_t capacity, uint64_t* count_out,
                                    s2_stream_t stream) {
    s2_status st = check_decode_compact(bitmap, sketch, n, p, idx_out, val_out, capacity, count_out, nullptr, 0);
    if (st != S2_OK) return st;
    if (n > noalloc_compact_max_n()) return S2_ERR_UNSUPPORTED;
    uint32_t* counts = nullptr;
    uint32_t* offsets = nullptr;
    if (noalloc_compact_scratch(&counts, &offsets) != cudaSuccess) return S2_ERR_CUDA;
    return cuda_status(launch_decode_compact(make_decode_args(bitmap, sketch, n, p, scale), idx_out, val_out, capacity,
                                             reinterpret_cast<unsigned long long*>(count_out), counts, offsets,
                                             reinterpret_cast<cudaStream_t>(stream)));
}

s2_status s2_hash(const uint32_t* idx, uint64_t m, s2_params p, uint32_t* bucket_out, int8_t* sign_out,
                  s2_stream_t stream) {
    s2_status st = check_params(p);
    if (st != S2_OK) return st;
    if (m == 0) return S2_OK;
    if (!idx || !bucket_out || !sign_out) return S2_ERR_INVALID_ARG;
    if (!aligned(idx, 4) || !aligned(bucket_out, 4)) return S2_ERR_ALIGNMENT;
    if (overlap(idx, m * 4, bucket_out, m * p.d * 4) || overlap(idx, m * 4, sign_out, m * p.d) ||
        overlap(bucket_out, m * p.d * 4, sign_out, m * p.d))
        return S2_ERR_INVALID_ARG;
    return cuda_status(
        launch_hash(idx, m, p.d, p.w, make_keys(p.seed, p.d), bucket_out, sign_out, reinterpret_cast<cudaStream_t>(stream)));
}

s2_status s2_pipeline_workspace_size(s2_dtype dt, uint32_t W, uint64_t n, s2_params p, size_t* bytes) {
    if (!bytes) return S2_ERR_INVALID_ARG;
    s2_status st = check_params(p);
    if (st != S2_OK) return st;
    if (dt != S2_F32 && dt != S2_BF16) return S2_ERR_INVALID_ARG;
    if (n > kMaxN) return S2_ERR_UNSUPPORTED;
    *bytes = pipeline_layout(dt, W, n, p).total;
    return S2_OK;
}

s2_status s2_pipeline_dense_host(const void* host_grad, s2_dtype dt, uint32_t W, uint64_t n, s2_params p,
                                 float scale, float* host_out, void* workspace, size_t workspace_bytes,
                                 s2_stream_t stream) {
    s2_status st = check_params(p);
    if (st != S2_OK) return st;
    if (dt != S2_F32 && dt != S2_BF16) return S2_ERR_INVALID_ARG;
    if (n > kMaxN) return S2_ERR_UNSUPPORTED;
    const PipelineLayout L = pipeline_layout(dt, W, n, p);
    if (!workspace || workspace_bytes < L.total) return S2_ERR_INVALID_ARG;
    if (!aligned(workspace, 16)) return S2_ERR_ALIGNMENT;
    if (n > 0 && (!host_out || (W > 0 && !host_grad))) return S2_ERR_INVALID_ARG;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    char* ws = static_cast<char*>(workspace);
    const uint64_t esz = dt == S2_F32 ? 4 : 2;
    void* d_grad = ws + L.grad;
    uint32_t* d_bitmaps = reinterpret_cast<uint32_t*>(ws + L.bitmaps);
    float* d_sketches = reinterpret_cast<float*>(ws + L.sketches);
    uint32_t* d_bitmap = reinterpret_cast<uint32_t*>(ws + L.bitmap);
    float* d_sketch = reinterpret_cast<float*>(ws + L.sketch);
    float* d_out = reinterpret_cast<float*>(ws + L.out);
    // Page-locked host buffers mapped into the device's address space are
    // read and written in place by the kernels (over NVLink-C2C on a
    // Grace-Blackwell node): the encode streams the gradient from host
    // memory once and the decode stores the output there, so no staging
    // copy precedes or follows them. Other host memory is staged through
    // the workspace with copies. A sketch built in several passes (larger
    // than 3/4 of L2) would re-read the gradient per pass: staged too.
    const void* enc_src = d_grad;
    if ((uint64_t)W * n > 0) {
        DeviceInfo di{};
        if (device_info(&di) != cudaSuccess) return S2_ERR_CUDA;
        const bool one_pass = (uint64_t)p.d * p.w * 4 <= (uint64_t)di.l2_bytes / 4 * 3;
        const void* mapped = one_pass ? mapped_host(host_grad) : nullptr;
        if (mapped) {
            enc_src = mapped;
        } else if (cudaMemcpyAsync(d_grad, host_grad, (size_t)W * n * esz, cudaMemcpyHostToDevice, s) !=
                   cudaSuccess) {
            return S2_ERR_CUDA;
        }
        st = encode_impl(enc_src, dt, W, n, p, d_bitmaps, d_sketches, s);
        if (st != S2_OK) return st;
    }
    st = s2_reduce(d_bitmaps, d_sketches, W, n, p, d_bitmap, d_sketch, stream);
    if (st != S2_OK) return st;
    if (n == 0) return S2_OK;
    float* out_mapped = static_cast<float*>(const_cast<void*>(mapped_host(host_out)));
    st = s2_decode_dense_ws(d_bitmap, d_sketch, n, p, scale, out_mapped ? out_mapped : d_out, ws + L.dec_ws,
                            dense_workspace_bytes(n, p.d), stream);
    if (st != S2_OK) return st;
    if (!out_mapped &&
        cudaMemcpyAsync(host_out, d_out, (size_t)n * 4, cudaMemcpyDeviceToHost, s) != cudaSuccess)
        return S2_ERR_CUDA;
    return S2_OK;
}

s2_status s2_pack8(const void* x, s2_dtype dt, uint64_t rows, uint64_t cols, uint64_t ldx, s2_scale_layout layout,
                   uint8_t* codes, uint64_t ldc, uint8_t* scales, uint8_t* codes_t, uint64_t ldct, uint8_t* scales_t,
                   s2_stream_t stream) {
    if (!dtype_ok(dt) || !layout_ok(layout)) return S2_ERR_INVALID_ARG;
    const bool tiles = layout == S2_SCALE_TILES;
    if ((codes_t != nullptr) != (scales_t != nullptr) || (codes_t && !tiles)) return S2_ERR_INVALID_ARG;
    s2_status st = check_matrix(rows, cols, ldx);
    if (st != S2_OK) return st;
    const uint64_t nblk = blocks8(cols), nrow = blocks8(rows);
    if (rows * nblk > 0xffffffffull || (tiles && nrow * nblk > kMaxDim8)) return S2_ERR_UNSUPPORTED;
    if (rows == 0 || cols == 0) return S2_OK;
    if (!x || !scales) return S2_ERR_INVALID_ARG;
    st = first_error({check_codes(codes, rows, cols, ldc), codes_t ? check_codes(codes_t, cols, rows, ldct) : S2_OK});
    if (st != S2_OK) return st;
    if (!aligned(x, size_of(dt))) return S2_ERR_ALIGNMENT;
    const uint64_t ns = (tiles ? nrow : rows) * nblk;
    if (clash({{codes, extent(rows, cols, ldc, 1)}, {scales, ns}, {codes_t, extent(cols, rows, ldct, 1)},
               {scales_t, ns}, {x, extent(rows, cols, ldx, size_of(dt))}}, 4))
        return S2_ERR_INVALID_ARG;
    Pack8Args a{x, ldx, codes, ldc, scales, codes_t, ldct, scales_t, rows, (uint32_t)cols, (uint32_t)nblk,
                (uint32_t)nrow, (uint32_t)(rows * nblk)};
    return cuda_status(launch_pack8(a, dt == S2_F32 ? 0 : 1, tiles, reinterpret_cast<cudaStream_t>(stream)));
}

s2_status s2_unpack8(const uint8_t* codes, uint64_t ldc, const uint8_t* scales, s2_scale_layout layout, uint64_t rows,
                     uint64_t cols, void* out, s2_dtype dt, uint64_t ldo, s2_stream_t stream) {
    if (!dtype_ok(dt) || !layout_ok(layout)) return S2_ERR_INVALID_ARG;
    s2_status st = check_matrix(rows, cols, ldo);
    if (st != S2_OK) return st;
    const uint64_t nblk = blocks8(cols);
    if (rows * nblk > 0xffffffffull) return S2_ERR_UNSUPPORTED;
    if (rows == 0 || cols == 0) return S2_OK;
    if (!out || !scales) return S2_ERR_INVALID_ARG;
    st = check_codes(codes, rows, cols, ldc);
    if (st != S2_OK) return st;
    if (!aligned(out, size_of(dt))) return S2_ERR_ALIGNMENT;
    const uint64_t ns = (layout == S2_SCALE_TILES ? blocks8(rows) : rows) * nblk;
    if (clash({{out, extent(rows, cols, ldo, size_of(dt))}, {codes, extent(rows, cols, ldc, 1)}, {scales, ns}}, 1))
        return S2_ERR_INVALID_ARG;
    Unpack8Args a{codes, ldc, scales, layout == S2_SCALE_TILES ? 7u : 0u, out, ldo, (uint32_t)cols, (uint32_t)nblk,
                  (uint32_t)(rows * nblk)};
    return cuda_status(launch_unpack8(a, dt == S2_F32 ? 0 : 1, reinterpret_cast<cudaStream_t>(stream)));
}

s2_status s2_matmul8(const uint8_t* x, uint64_t ldx, const uint8_t* x_scales, const uint8_t* w, uint64_t ldw,
                     const uint8_t* w_scales, s2_scale_layout w_layout, uint64_t M, uint64_t N, uint64_t K, void* y,
                     s2_dtype dt, uint64_t ldy, s2_stream_t stream) {
    if (!dtype_ok(dt) || !layout_ok(w_layout)) return S2_ERR_INVALID_ARG;
    s2_status st = first_error({check_matrix(M, N, ldy), check_matrix(M, K, ldx), check_matrix(N, K, ldw)});
    if (st != S2_OK) return st;
    if ((M + 15) / 16 * blocks8(N) > 0x7fffffffull) return S2_ERR_UNSUPPORTED;  // the smallest tiles are counted in 32 bits
    if (M == 0 || N == 0) return S2_OK;
    if (!y) return S2_ERR_INVALID_ARG;
    const uint64_t esz = size_of(dt);
    if (!aligned(y, esz)) return S2_ERR_ALIGNMENT;
    if (K == 0)  // an empty sum
        return cuda_status(cudaMemset2DAsync(y, (M > 1 ? ldy : N) * esz, 0, N * esz, M,
                                             reinterpret_cast<cudaStream_t>(stream)));
    if (!x_scales || !w_scales) return S2_ERR_INVALID_ARG;
    st = first_error({check_codes(x, M, K, ldx), check_codes(w, N, K, ldw)});
    if (st != S2_OK) return st;
    const uint64_t nblk = blocks8(K);
    if (clash({{y, extent(M, N, ldy, esz)}, {x, extent(M, K, ldx, 1)}, {x_scales, M * nblk}, {w, extent(N, K, ldw, 1)},
               {w_scales, (w_layout == S2_SCALE_TILES ? blocks8(N) : N) * nblk}}, 1))
        return S2_ERR_INVALID_ARG;
    Matmul8Args a{x, x_scales, w, w_scales, y, stride16(M, K, ldx), stride16(N, K, ldw), ldy,
                  (uint32_t)M, (uint32_t)N, (uint32_t)K, w_layout == S2_SCALE_TILES ? 7u : 0u, dt == S2_F32 ? 0 : 1};
    return cuda_status(launch_matmul8(a, reinterpret_cast<cudaStream_t>(stream)));
}

s2_status s2_wgrad8(const void* dy, uint64_t lddy, const uint8_t* x, uint64_t ldx, const uint8_t* x_scales, uint64_t T,
                    uint64_t N, uint64_t K, void* dw, s2_dtype dt, uint64_t lddw, int accumulate, s2_stream_t stream) {
    if (!dtype_ok(dt)) return S2_ERR_INVALID_ARG;
    s2_status st = first_error({check_matrix(T, N, lddy), check_matrix(T, K, ldx), check_matrix(N, K, lddw)});
    if (st != S2_OK) return st;
    // the smallest tiles are counted in 32 bits, and so are the stages of one of the device's blocks or pairs (at least 64)
    const uint64_t tiles = (N + 31) / 32 * blocks8(K);
    if (tiles > 0x7fffffffull || tiles * ((T + 63) / 64) >= (1ull << 36)) return S2_ERR_UNSUPPORTED;
    if (N == 0 || K == 0) return S2_OK;
    if (!dw) return S2_ERR_INVALID_ARG;
    const uint64_t esz = size_of(dt);
    if (!aligned(dw, esz)) return S2_ERR_ALIGNMENT;
    if (T == 0)  // an empty sum
        return accumulate ? S2_OK
                          : cuda_status(cudaMemset2DAsync(dw, (N > 1 ? lddw : K) * esz, 0, K * esz, N,
                                                          reinterpret_cast<cudaStream_t>(stream)));
    if (!dy || !x_scales) return S2_ERR_INVALID_ARG;
    st = check_codes(x, T, K, ldx);
    if (st != S2_OK) return st;
    if (!aligned(dy, 2)) return S2_ERR_ALIGNMENT;
    if (clash({{dw, extent(N, K, lddw, esz)}, {dy, extent(T, N, lddy, 2)}, {x, extent(T, K, ldx, 1)},
               {x_scales, T * blocks8(K)}}, 1))
        return S2_ERR_INVALID_ARG;
    Wgrad8Args a{dy, x, x_scales, dw, T > 1 ? lddy : (N + 7) / 8 * 8, stride16(T, K, ldx), lddw, (uint32_t)T, (uint32_t)N, (uint32_t)K,
                 dt == S2_F32 ? 0 : 1, accumulate != 0};
    return cuda_status(launch_wgrad8(a, reinterpret_cast<cudaStream_t>(stream)));
}

s2_status s2_pack4_scales_size(uint64_t rows, uint64_t cols, size_t* bytes) {
    if (!bytes) return S2_ERR_INVALID_ARG;
    if (rows > kMaxDim8 || cols > kMaxDim8) return S2_ERR_UNSUPPORTED;
    *bytes = scales4(rows, cols);
    return S2_OK;
}

s2_status s2_pack4(const void* x, s2_dtype dt, uint64_t rows, uint64_t cols, uint64_t ldx, uint8_t* codes, uint64_t ldc,
                   uint8_t* scales, s2_stream_t stream) {
    if (!dtype_ok(dt)) return S2_ERR_INVALID_ARG;
    s2_status st = check_matrix(rows, cols, ldx);
    if (st != S2_OK) return st;
    const uint64_t items = blocks8(rows) * blocks8(cols) * 16;
    if (items > kMaxItems4) return S2_ERR_UNSUPPORTED;
    if (rows == 0 || cols == 0) return S2_OK;
    if (!x) return S2_ERR_INVALID_ARG;
    st = check_packed4(codes, rows, cols, ldc, scales);
    if (st != S2_OK) return st;
    if (!aligned(x, size_of(dt))) return S2_ERR_ALIGNMENT;
    if (clash({{codes, extent(rows, bytes4(cols), ldc, 1)}, {scales, scales4(rows, cols)},
               {x, extent(rows, cols, ldx, size_of(dt))}}, 2))
        return S2_ERR_INVALID_ARG;
    Pack4Args a{x, ldx, codes, ldc, scales, rows, (uint32_t)cols, (uint32_t)blocks8(cols), items / 16, 0};
    return cuda_status(launch_pack4(a, dt == S2_F32 ? 0 : 1, reinterpret_cast<cudaStream_t>(stream)));
}

s2_status s2_unpack4(const uint8_t* codes, uint64_t ldc, const uint8_t* scales, uint64_t rows, uint64_t cols, void* out,
                     s2_dtype dt, uint64_t ldo, s2_stream_t stream) {
    if (!dtype_ok(dt)) return S2_ERR_INVALID_ARG;
    s2_status st = check_matrix(rows, cols, ldo);
    if (st != S2_OK) return st;
    const uint64_t items = blocks8(rows) * blocks8(cols) * 16;
    if (items > kMaxItems4) return S2_ERR_UNSUPPORTED;
    if (rows == 0 || cols == 0) return S2_OK;
    if (!out) return S2_ERR_INVALID_ARG;
    st = check_packed4(codes, rows, cols, ldc, scales);
    if (st != S2_OK) return st;
    if (!aligned(out, size_of(dt))) return S2_ERR_ALIGNMENT;
    if (clash({{out, extent(rows, cols, ldo, size_of(dt))}, {codes, extent(rows, bytes4(cols), ldc, 1)},
               {scales, scales4(rows, cols)}}, 1))
        return S2_ERR_INVALID_ARG;
    Unpack4Args a{codes, ldc, scales, out, ldo, rows, (uint32_t)cols, (uint32_t)blocks8(cols), items};
    return cuda_status(launch_unpack4(a, dt == S2_F32 ? 0 : 1, reinterpret_cast<cudaStream_t>(stream)));
}

s2_status s2_matmul4(const uint8_t* x, uint64_t ldx, const uint8_t* x_scales, const uint8_t* w, uint64_t ldw,
                     const uint8_t* w_scales, uint64_t M, uint64_t N, uint64_t K, void* y, s2_dtype dt, uint64_t ldy,
                     s2_stream_t stream) {
    if (!dtype_ok(dt)) return S2_ERR_INVALID_ARG;
    s2_status st = first_error({check_matrix(M, N, ldy), check_matrix(M, bytes4(K), ldx), check_matrix(N, bytes4(K), ldw)});
    if (st != S2_OK) return st;
    // the smallest tiles are counted in 32 bits; K as a size has the limit of the others
    if (K > kMaxDim8 || (M + 15) / 16 * blocks8(N) > 0x7fffffffull) return S2_ERR_UNSUPPORTED;
    if (M == 0 || N == 0) return S2_OK;
    if (!y) return S2_ERR_INVALID_ARG;
    const uint64_t esz = size_of(dt);
    if (!aligned(y, esz)) return S2_ERR_ALIGNMENT;
    if (K == 0)  // an empty sum
        return cuda_status(cudaMemset2DAsync(y, (M > 1 ? ldy : N) * esz, 0, N * esz, M,
                                             reinterpret_cast<cudaStream_t>(stream)));
    st = first_error({check_packed4(x, M, K, ldx, x_scales), check_packed4(w, N, K, ldw, w_scales)});
    if (st != S2_OK) return st;
    if (clash({{y, extent(M, N, ldy, esz)}, {x, extent(M, bytes4(K), ldx, 1)}, {x_scales, scales4(M, K)},
               {w, extent(N, bytes4(K), ldw, 1)}, {w_scales, scales4(N, K)}}, 1))
        return S2_ERR_INVALID_ARG;
    Matmul4Args a{x, x_scales, w, w_scales, y, stride16(M, bytes4(K), ldx), stride16(N, bytes4(K), ldw), ldy,
                  (uint32_t)M, (uint32_t)N, (uint32_t)K, dt == S2_F32 ? 0 : 1};
    return cuda_status(launch_matmul4(a, reinterpret_cast<cudaStream_t>(stream)));
}

s2_status s2_sample(const void* logits, s2_dtype dt, uint64_t T, uint64_t V, uint64_t ld, const float* temperature,
                    const int32_t* top_k, const float* top_p, const float* min_p, const float* u, int32_t* tokens,
                    s2_stream_t stream) {
    if (!dtype_ok(dt)) return S2_ERR_INVALID_ARG;
    const s2_status st = check_matrix(T, V, ld);
    if (st != S2_OK) return st;
    if (T == 0) return S2_OK;
    if (!tokens || !u) return S2_ERR_INVALID_ARG;
    if (!aligned(tokens, 4) || !aligned(u, 4) || !aligned(temperature, 4) || !aligned(top_k, 4) || !aligned(top_p, 4) ||
        !aligned(min_p, 4))
        return S2_ERR_ALIGNMENT;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (V > 0 && !logits) return S2_ERR_INVALID_ARG;
    if (!aligned(logits, size_of(dt))) return S2_ERR_ALIGNMENT;
    if (clash({{tokens, T * 4}, {logits, extent(T, V, ld, size_of(dt))}, {temperature, T * 4}, {top_k, T * 4},
               {top_p, T * 4}, {min_p, T * 4}, {u, T * 4}}, 1))
        return S2_ERR_INVALID_ARG;
    if (V == 0) return cuda_status(cudaMemsetAsync(tokens, 0xff, T * 4, s));  // -1: nothing to draw
    SampleArgs a{logits, ld, (uint32_t)T, (uint32_t)V, temperature, top_k, top_p, min_p, u, tokens};
    return cuda_status(launch_sample(a, dt == S2_F32 ? 0 : 1, s));
}

s2_status s2_distill(const void* logits, s2_dtype dt, uint64_t T, uint64_t V, uint64_t ld, const int32_t* teacher_idx,
                     const float* teacher, uint64_t K, const int32_t* targets, const float* row_weight,
                     s2_distill_params p, float* loss, void* dlogits, s2_dtype ddt, uint64_t ldd, s2_stream_t stream) {
    if (!dtype_ok(dt) || (dlogits && !dtype_ok(ddt))) return S2_ERR_INVALID_ARG;
    const float ct = (float)(1.44269504088896340736 / p.temperature), inv_t = (float)(1.0 / p.temperature);
    if (!(p.temperature > 0.0f) || !std::isfinite(p.temperature) || !std::isfinite(ct) || !std::isfinite(p.soft) ||
        !std::isfinite(p.hard) || !std::isfinite(p.scale))
        return S2_ERR_INVALID_ARG;
    s2_status st = first_error({check_matrix(T, V, ld), dlogits ? check_matrix(T, V, ldd) : S2_OK});
    if (st != S2_OK) return st;
    if (K > S2_DISTILL_MAX_ENTRIES) return S2_ERR_UNSUPPORTED;
    if (T == 0) return S2_OK;
    if (!loss || (K > 0 && (!teacher_idx || !teacher))) return S2_ERR_INVALID_ARG;
    if (!aligned(loss, 4) || !aligned(teacher_idx, 4) || !aligned(teacher, 4) || !aligned(targets, 4) || !aligned(row_weight, 4))
        return S2_ERR_ALIGNMENT;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (V == 0) return cuda_status(cudaMemsetAsync(loss, 0, T * 4, s));  // no logits, no terms
    if (!logits) return S2_ERR_INVALID_ARG;
    const uint64_t esz = size_of(dt), dsz = size_of(ddt);
    if (!aligned(logits, esz) || !aligned(dlogits, dsz)) return S2_ERR_ALIGNMENT;
    if (clash({{loss, T * 4}, {dlogits, dlogits ? extent(T, V, ldd, dsz) : 0}, {logits, extent(T, V, ld, esz)},
               {teacher_idx, T * K * 4}, {teacher, T * K * 4}, {targets, T * 4}, {row_weight, T * 4}}, 2))
        return S2_ERR_INVALID_ARG;
    DistillArgs a{};
    a.z = logits;
    a.ld = ld;
    a.idx = teacher_idx;
    a.t = teacher;
    a.K = (uint32_t)K;
    a.targets = targets;
    a.row_weight = row_weight;
    a.soft = p.soft;
    a.hard = p.hard;
    a.scale = p.scale;
    a.loss = loss;
    a.dz = dlogits;
    a.ldd = ldd;
    a.T = (uint32_t)T;
    a.V = (uint32_t)V;
    a.wide = dlogits && (reinterpret_cast<uintptr_t>(logits) / esz - reinterpret_cast<uintptr_t>(dlogits) / dsz) % 8 == 0 &&
             (T == 1 || (ld - ldd) % 8 == 0);
    a.use_soft = K > 0 && p.soft != 0.0f;
    a.use_hard = targets && p.hard != 0.0f;
    a.ct = ct;
    a.inv_t = inv_t;
    return cuda_status(launch_distill(a, dt == S2_F32 ? 0 : 1, ddt == S2_F32 ? 0 : 1, s));
}

s2_status s2_wait_faults(uint32_t* host_count) {
    if (!host_count) return S2_ERR_INVALID_ARG;
    return cuda_status(read_wait_faults(host_count));
}

const char* s2_status_string(s2_status st) {
    switch (st) {
        case S2_OK: return "S2_OK";
        case S2_ERR_INVALID_ARG: return "S2_ERR_INVALID_ARG";
        case S2_ERR_ALIGNMENT: return "S2_ERR_ALIGNMENT";
        case S2_ERR_UNSUPPORTED: return "S2_ERR_UNSUPPORTED";
        case S2_ERR_CUDA: return "S2_ERR_CUDA";
    }
    return "S2_UNKNOWN_STATUS";
}

const char* s2_version(void) { return "libs2 0.1 (sm_103a), s2.h " S2_HEADER_WORD; }

}  // extern "C"
