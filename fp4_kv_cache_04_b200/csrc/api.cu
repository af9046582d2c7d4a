// C-ABI entry points of libcsa2: host-side validation, workspace layout and the
// Full / Reindex / Reuse dispatch of a CSA2 layer (CSA2 section of the thecryptopost.io
// DeepSeek-V4.1-Flash article).  Every check runs before anything is enqueued.
#include <cuda.h>

#include <algorithm>
#include <atomic>
#include <cstdio>
#include <cstring>
#include <mutex>

#include "common.cuh"
#include "dense.cuh"
#include "kernels.cuh"

namespace csa2 {

namespace {
thread_local char g_last_error[256] = "";

constexpr size_t WS_HEADER = 256;          // device error word + padding

size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

struct WsLayout {
    bool fused = false;                    // decode indexer: scan + chunk Top-K + merge
    bool prefill_fused = false;            // many-query Full indexer with a streaming Top-K
    size_t scores = 0;                     // materialised scores [rows][scores_ld]
    int64_t scores_ld = 0;
    size_t cand_s = 0, cand_p = 0;         // fused: [B][n_chunks][512] candidates
    size_t chunk_thr = 0;                  // fused: [B][n_chunks] chunk 512th scores
    int n_chunks = 0, chunk = 0;
    size_t blockmax = 0;                   // [B][bm_ld] block maxima (FULL + want_pool)
    int64_t bm_ld = 0;
    int n_split = 1;                       // attention CTAs (one cluster) per query row
    size_t total = WS_HEADER;
};

WsLayout layer_layout(const csa2_layer_args* a) {
    WsLayout L;
    size_t off = WS_HEADER;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off += align_up(bytes, 256);
        return at;
    };
    const int64_t rows = static_cast<int64_t>(a->batch) * a->q_per_seq;
    if (a->mode != CSA2_MODE_REUSE) {
        L.fused = (a->q_per_seq == 1 && a->q_pos == nullptr);
        L.prefill_fused = !L.fused && a->mode == CSA2_MODE_FULL;
        const int64_t ncols = (a->mode == CSA2_MODE_REINDEX) ? POOL_POSITIONS : a->max_n;
        if (L.prefill_fused) {
            // no scratch: scores and candidates stay in shared memory
        } else if (L.fused) {
            L.chunk = (a->mode == CSA2_MODE_REINDEX) ? REINDEX_CHUNK : SCAN_CHUNK;
            L.n_chunks = static_cast<int>(ceil_div(ncols, L.chunk));
            const size_t n = static_cast<size_t>(a->batch) * L.n_chunks * TOPK;
            L.cand_s = take(n * sizeof(float));
            L.cand_p = take(n * sizeof(int32_t));
            L.chunk_thr = take(static_cast<size_t>(a->batch) * L.n_chunks * sizeof(float));
        } else {
            L.scores_ld = padded_ld(ncols);
            L.scores = take(static_cast<size_t>(rows * L.scores_ld) * sizeof(float));
        }
        if (a->mode == CSA2_MODE_FULL && a->want_pool) {
            L.bm_ld = padded_ld(ceil_div(a->max_n, POOL_BLOCK));
            L.blockmax = take(static_cast<size_t>(a->batch * L.bm_ld) * sizeof(float));
        }
    }
    // every attention runs on the single-row kernel (decode rows and prefill rows alike);
    // a row's CTAs merge their partials in their cluster, so it needs no scratch
    const bool swa8 = a->swa_format == CSA2_SWA_FP8;
    L.n_split = attend_rows_split(rows, attend_rows_swa_tiles(a->swa_rows, a->q_pos != nullptr, swa8), swa8);
    L.total = off;
    return L;
}

bool valid_type(int32_t t) { return t == CSA2_T_BF16 || t == CSA2_T_F16 || t == CSA2_T_F32; }

// Workspace of csa2_attend_cache: two partials for each range of the tile list, as many as a cut
// list of that many tiles has (a smaller batch may be cut where a larger one is not).
struct CacheLayout {
    CachePlan plan;
    size_t meta = 0, part = 0, total = 0;
};

// Positions of a row, up to its last tile's end, and rows are counted in 32 bits.
bool cache_sizes_fit(const csa2_cache_args* a) {
    return a->max_n <= INT32_MAX - (CACHE_TILE - 1) && static_cast<int64_t>(a->batch) * a->q_per_seq <= INT32_MAX;
}

CacheLayout cache_layout(const csa2_cache_args* a) {
    CacheLayout L;
    L.plan = cache_plan(static_cast<int64_t>(a->batch) * a->q_per_seq, a->max_n, a->window, a->sinks);
    L.meta = WS_HEADER;
    L.part = L.meta + align_up(static_cast<size_t>(L.plan.room) * 2 * sizeof(int32_t), 256);
    L.total = L.part + align_up(static_cast<size_t>(L.plan.room) * 2 * CACHE_PART_FLOATS * sizeof(float), 256);
    return L;
}

// A second stream per device, for work of one call that may run beside the caller's
// stream (created on first use, outside stream capture; never destroyed).
cudaStream_t side_stream(cudaStream_t caller) {
    static std::mutex mu;
    static cudaStream_t streams[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return nullptr;
    std::lock_guard<std::mutex> lock(mu);
    if (!streams[dev]) {
        cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
        if (cudaStreamIsCapturing(caller, &cap) != cudaSuccess || cap != cudaStreamCaptureStatusNone) return nullptr;
        if (cudaStreamCreateWithFlags(&streams[dev], cudaStreamNonBlocking) != cudaSuccess) streams[dev] = nullptr;
    }
    return streams[dev];
}

// Fork / join of the side stream with events (inside a stream capture these become graph
// edges).  begin() returns the stream to use: the side stream, or the caller's own stream
// when no side stream is available (then join() has nothing to do).
struct SideFork {
    cudaEvent_t e_fork = nullptr, e_join = nullptr;
    cudaStream_t side = nullptr;
    cudaStream_t begin(cudaStream_t s) {
        cudaStream_t st = side_stream(s);
        if (!st || cudaEventCreateWithFlags(&e_fork, cudaEventDisableTiming) != cudaSuccess ||
            cudaEventCreateWithFlags(&e_join, cudaEventDisableTiming) != cudaSuccess ||
            cudaEventRecord(e_fork, s) != cudaSuccess || cudaStreamWaitEvent(st, e_fork, 0) != cudaSuccess) {
            (void)cudaGetLastError();
            return s;
        }
        side = st;
        return st;
    }
    // Instead of joining: records ev where the side work ends (the side stream, or s when
    // the work ran on s); whoever reads its outputs waits for ev.
    csa2_status defer(cudaStream_t s, cudaEvent_t ev) {
        const cudaError_t ce = cudaEventRecord(ev, side ? side : s);
        side = nullptr;
        return ce == cudaSuccess ? CSA2_OK : fail_cuda("csa2_attend ev_pool record", ce);
    }
    csa2_status join(cudaStream_t s) {
        cudaError_t ce = cudaSuccess;
        if (side) {
            ce = cudaEventRecord(e_join, side);
            if (ce == cudaSuccess) ce = cudaStreamWaitEvent(s, e_join, 0);
            side = nullptr;
        }
        return ce == cudaSuccess ? CSA2_OK : fail_cuda("csa2_attend side-stream join", ce);
    }
    ~SideFork() {
        if (e_fork) cudaEventDestroy(e_fork);
        if (e_join) cudaEventDestroy(e_join);
    }
};

csa2_status validate_index(const csa2_index_args* a) {
    if (!a) return CSA2_ERR_INVALID_ARG;
    if (a->batch < 1 || a->q_per_seq < 1 || a->q_per_seq > 65536) return CSA2_ERR_INVALID_ARG;
    if (a->ratio != 1 && a->ratio != 2) return CSA2_ERR_INVALID_ARG;
    if (a->reserved0 != 0 || a->max_n < 1) return CSA2_ERR_INVALID_ARG;
    if (!a->kv_offsets || !a->idx_q || !a->idx_w || !a->idx_k || !a->idx_kscale)
        return CSA2_ERR_INVALID_ARG;
    if (!aligned(a->idx_q, 16) || !aligned(a->idx_k, 16)) return CSA2_ERR_INVALID_ARG;
    return CSA2_OK;
}

IndexParams to_params(const csa2_index_args* a) {
    IndexParams p;
    p.batch = a->batch;
    p.q_per_seq = a->q_per_seq;
    p.ratio = a->ratio;
    p.max_n = a->max_n;
    p.kv_offsets = a->kv_offsets;
    p.q_pos = a->q_pos;
    p.idx_q = a->idx_q;
    p.idx_w = a->idx_w;
    p.idx_k = a->idx_k;
    p.idx_kscale = a->idx_kscale;
    p.pool_blocks = a->pool_blocks;
    p.rows = RowMap{nullptr, 0, 0};                      // the stage API reads packed rows
    return p;
}

// cuTensorMapEncodeTiled through the runtime's driver entry point (no libcuda link).
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                                   CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                   CUtensorMapFloatOOBfill);

EncodeTiledFn encode_tiled() {
    static EncodeTiledFn fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<EncodeTiledFn>(f);
    }();
    return fn;
}

// TMA map over bf16 rows of 512: rank 2 = [rows][512] (boxes of box_rows x 64), rank 3 =
// [seqs][rows][512] (boxes of 1 x box_rows x 64); 128-byte swizzle.  The kernel's TMA
// instruction must have the same rank.
bool make_bf16_rows_map(const uint16_t* base, int64_t rows, int64_t seqs, int box_rows, int rank,
                        CUtensorMap* map) {
    const EncodeTiledFn enc = encode_tiled();
    if (!enc) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(rows),
                                static_cast<cuuint64_t>(seqs)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(rows * D) * 2};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_rows), 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    if (rank != 2 && rank != 3) return false;
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, static_cast<cuuint32_t>(rank), const_cast<uint16_t*>(base), dims,
               strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// TMA map over indexer K viewed as [rows][64] bytes, 64-byte swizzle, boxes of box_rows.
bool make_idx_k_map(const uint8_t* idx_k, int64_t rows, int box_rows, CUtensorMap* map) {
    const EncodeTiledFn enc = encode_tiled();
    if (!enc) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(IDX_DIM), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(IDX_DIM)};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(IDX_DIM), static_cast<cuuint32_t>(box_rows)};
    const cuuint32_t estr[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(idx_k), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// TMA map over rows of `width` bytes, boxes of box_rows x box_width.
bool make_byte_rows_map(const uint8_t* base, int64_t rows, int width, int box_width, int box_rows,
                        CUtensorMapSwizzle swizzle, CUtensorMap* map) {
    const EncodeTiledFn enc = encode_tiled();
    if (!enc) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(width)};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_width), static_cast<cuuint32_t>(box_rows)};
    const cuuint32_t estr[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

bool opt_in_smem(const void* kernel, int bytes) {
    constexpr int kMaxDev = 64, kMaxKernels = 32;
    static const void* kernels[kMaxKernels] = {};
    static bool done[kMaxKernels][kMaxDev] = {};
    static std::mutex mu;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDev) return false;
    std::lock_guard<std::mutex> lock(mu);
    int slot = 0;
    while (slot < kMaxKernels && kernels[slot] != nullptr && kernels[slot] != kernel) ++slot;
    if (slot == kMaxKernels) return false;
    kernels[slot] = kernel;
    if (done[slot][dev]) return true;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
        return false;
    done[slot][dev] = true;
    return true;
}

std::atomic<uint64_t> g_launches{0};

csa2_status fail_cuda(const char* what, cudaError_t e) {
    std::snprintf(g_last_error, sizeof(g_last_error), "%s: %s", what, cudaGetErrorString(e));
    cudaGetLastError();                       // clear a non-sticky error
    return CSA2_ERR_CUDA;
}

csa2_status check_launch(const char* what) {
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) {
        g_launches.fetch_add(1, std::memory_order_relaxed);
        return CSA2_OK;
    }
    std::snprintf(g_last_error, sizeof(g_last_error), "%s: %s", what, cudaGetErrorString(e));
    return CSA2_ERR_CUDA;
}

}  // namespace csa2

using namespace csa2;

extern "C" {

const char* csa2_status_string(csa2_status s) {
    switch (s) {
        case CSA2_OK: return "CSA2_OK";
        case CSA2_ERR_INVALID_ARG: return "CSA2_ERR_INVALID_ARG";
        case CSA2_ERR_UNSUPPORTED: return "CSA2_ERR_UNSUPPORTED";
        case CSA2_ERR_WORKSPACE: return "CSA2_ERR_WORKSPACE";
        case CSA2_ERR_CUDA: return "CSA2_ERR_CUDA";
        case CSA2_ERR_TIMEOUT: return "CSA2_ERR_TIMEOUT";
        case CSA2_ERR_DEVICE: return "CSA2_ERR_DEVICE";
        default: return "CSA2_ERR_UNKNOWN";
    }
}

const char* csa2_last_error(void) { return g_last_error; }

int32_t csa2_abi_version(void) { return CSA2_ABI_VERSION; }

uint64_t csa2_kernel_launches(void) { return g_launches.load(std::memory_order_relaxed); }

csa2_status csa2_quantize_kv(const uint16_t* x, int64_t n_in, int32_t ratio, const int64_t* dst_row,
                             uint8_t* codes, uint8_t* scales, void* stream) {
    if (ratio != 1 && ratio != 2) return CSA2_ERR_INVALID_ARG;
    if (n_in < 0 || n_in % ratio != 0) return CSA2_ERR_INVALID_ARG;
    if (n_in == 0) return CSA2_OK;
    if (!x || !codes || !scales) return CSA2_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(codes, 8)) return CSA2_ERR_INVALID_ARG;
    if (n_in / ratio > (int64_t(1) << 36)) return CSA2_ERR_UNSUPPORTED;
    return launch_quantize(x, n_in, ratio, dst_row, codes, scales, static_cast<cudaStream_t>(stream));
}

csa2_status csa2_append_kv(const uint16_t* latent, const float* idx_proj, int64_t n, const int64_t* dst_row,
                           uint8_t* codes, uint8_t* scales, uint8_t* idx_k, float* idx_kscale, void* stream) {
    if (n < 0) return CSA2_ERR_INVALID_ARG;
    if (n == 0) return CSA2_OK;
    if (!latent || !idx_proj || !dst_row || !codes || !scales || !idx_k || !idx_kscale)
        return CSA2_ERR_INVALID_ARG;
    if (!aligned(latent, 16) || !aligned(idx_proj, 8) || !aligned(codes, 8) || !aligned(idx_k, 2) ||
        !aligned(idx_kscale, 4) || !aligned(dst_row, 8))
        return CSA2_ERR_INVALID_ARG;
    if (n > (int64_t(1) << 36)) return CSA2_ERR_UNSUPPORTED;
    return launch_append(latent, idx_proj, n, dst_row, codes, scales, idx_k, idx_kscale,
                         static_cast<cudaStream_t>(stream));
}

csa2_status csa2_index_score(const csa2_index_args* a, float* scores, int64_t ld, void* stream) {
    const csa2_status st = validate_index(a);
    if (st != CSA2_OK) return st;
    if (!scores) return CSA2_ERR_INVALID_ARG;
    const int64_t ncols = a->pool_blocks ? POOL_POSITIONS : a->max_n;
    if (ld < ncols) return CSA2_ERR_INVALID_ARG;
    return launch_index_score(to_params(a), scores, ld, nullptr, 0, static_cast<cudaStream_t>(stream));
}

csa2_status csa2_topk(const float* scores, int64_t ld, int64_t n_cols, int32_t rows, int32_t k,
                      const int32_t* pool_blocks, int32_t q_per_seq, int32_t* idx_out, void* stream) {
    if (rows < 0 || k < 1 || k > 4096 || q_per_seq < 1) return CSA2_ERR_INVALID_ARG;
    if (n_cols < 0 || n_cols > ld) return CSA2_ERR_INVALID_ARG;
    if (pool_blocks && n_cols > POOL_POSITIONS) return CSA2_ERR_INVALID_ARG;
    if (rows == 0) return CSA2_OK;
    if (!scores || !idx_out) return CSA2_ERR_INVALID_ARG;
    if (n_cols > (int64_t(1) << 31) - 1) return CSA2_ERR_UNSUPPORTED;
    return launch_topk_rows(scores, ld, n_cols, rows, k, pool_blocks, q_per_seq, idx_out,
                            static_cast<cudaStream_t>(stream));
}

size_t csa2_pool_workspace_size(int32_t batch, int64_t max_n) {
    if (batch < 1 || max_n < 1) return 0;
    const int64_t bm_ld = padded_ld(ceil_div(max_n, POOL_BLOCK));
    return WS_HEADER + align_up(static_cast<size_t>(batch * bm_ld) * sizeof(float), 256);
}

csa2_status csa2_build_pool(const float* scores, int64_t ld, const int64_t* kv_offsets, int32_t batch,
                            int64_t max_n, int32_t* pool_blocks, void* workspace,
                            size_t workspace_bytes, void* stream) {
    if (batch < 1 || max_n < 1 || ld < max_n) return CSA2_ERR_INVALID_ARG;
    if (!scores || !kv_offsets || !pool_blocks) return CSA2_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, 256) ||
        workspace_bytes < csa2_pool_workspace_size(batch, max_n))
        return CSA2_ERR_WORKSPACE;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int64_t bm_ld = padded_ld(ceil_div(max_n, POOL_BLOCK));
    float* bm = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + WS_HEADER);
    csa2_status st = launch_block_max(scores, ld, kv_offsets, batch, max_n, bm, bm_ld, s);
    if (st != CSA2_OK) return st;
    return launch_topk_rows(bm, bm_ld, ceil_div(max_n, POOL_BLOCK), batch, POOL_BLOCKS, nullptr, 1,
                            pool_blocks, s, kv_offsets);
}

size_t csa2_workspace_size(const csa2_layer_args* a) {
    if (!a) return 0;
    if (a->batch < 1 || a->q_per_seq < 1 || a->max_n < 1) return WS_HEADER;
    return layer_layout(a).total;
}

csa2_status csa2_attend(const csa2_layer_args* a, void* stream) {
    if (!a) return CSA2_ERR_INVALID_ARG;
    if (a->mode != CSA2_MODE_FULL && a->mode != CSA2_MODE_REINDEX && a->mode != CSA2_MODE_REUSE)
        return CSA2_ERR_INVALID_ARG;
    if (a->batch < 1 || a->q_per_seq < 1 || a->q_per_seq > 65536) return CSA2_ERR_INVALID_ARG;
    if (a->ratio != 1 && a->ratio != 2) return CSA2_ERR_INVALID_ARG;
    if (a->reserved0 != 0 || a->reserved1 != 0 || a->max_n < 1) return CSA2_ERR_INVALID_ARG;
    if (a->swa_format != CSA2_SWA_BF16 && a->swa_format != CSA2_SWA_FP8) return CSA2_ERR_INVALID_ARG;
    if ((a->q_format != CSA2_Q_BF16 && a->q_format != CSA2_Q_NVFP4) || a->reserved2 != 0)
        return CSA2_ERR_INVALID_ARG;
    const bool swa8 = a->swa_format == CSA2_SWA_FP8;
    if (!a->kv_offsets || !a->codes || !a->scales || !a->topk_idx || !a->q || !a->out) return CSA2_ERR_INVALID_ARG;
    if (swa8 ? (!a->swa_kv8 || !a->swa_kscale) : !a->swa_kv) return CSA2_ERR_INVALID_ARG;
    if (swa8 && (!aligned(a->swa_kv8, 16) || !aligned(a->swa_kscale, 4))) return CSA2_ERR_INVALID_ARG;
    if (swa8 && (a->q_per_seq != 1 || a->q_pos != nullptr)) return CSA2_ERR_UNSUPPORTED;
    if (a->mode != CSA2_MODE_REUSE && (!a->idx_q || !a->idx_w || !a->idx_k || !a->idx_kscale))
        return CSA2_ERR_INVALID_ARG;
    if (a->mode == CSA2_MODE_REINDEX && !a->pool_blocks) return CSA2_ERR_INVALID_ARG;
    if (a->want_pool && (a->mode != CSA2_MODE_FULL || !a->pool_blocks || a->q_per_seq != 1))
        return CSA2_ERR_INVALID_ARG;
    if (a->swa_rows < 1) return CSA2_ERR_INVALID_ARG;
    if ((a->pool_k != nullptr) != (a->pool_kscale != nullptr)) return CSA2_ERR_INVALID_ARG;
    if (a->page_table) {
        if (a->page_rows < 128 || a->page_rows % 128 != 0 || a->page_rows > (1 << 24)) return CSA2_ERR_INVALID_ARG;
        if (a->pages_per_seq < ceil_div(a->max_n, a->page_rows)) return CSA2_ERR_INVALID_ARG;
        if (a->mode == CSA2_MODE_REINDEX && (a->q_per_seq != 1 || a->q_pos != nullptr))
            return CSA2_ERR_UNSUPPORTED;
    }
    if (a->pool_k && (!aligned(a->pool_k, 16) || !aligned(a->pool_kscale, 4))) return CSA2_ERR_INVALID_ARG;
    if (a->sel_cache_mode < CSA2_CACHE_OFF || a->sel_cache_mode > CSA2_CACHE_USE)
        return CSA2_ERR_INVALID_ARG;
    if (a->sel_cache_mode != CSA2_CACHE_OFF && (!a->sel_cache || !aligned(a->sel_cache, 16)))
        return CSA2_ERR_INVALID_ARG;
    if (a->sel_cache_mode == CSA2_CACHE_USE && a->mode != CSA2_MODE_REUSE) return CSA2_ERR_INVALID_ARG;
    if (a->mode != CSA2_MODE_REUSE && (a->total_n < 1 || a->total_n > INT32_MAX))
        return CSA2_ERR_INVALID_ARG;
    if (a->q_pos && a->swa_rows < static_cast<int64_t>(a->q_per_seq) + CSA2_WINDOW - 1)
        return CSA2_ERR_INVALID_ARG;
    if (!aligned(a->q, 16) || (!swa8 && !aligned(a->swa_kv, 16)) || !aligned(a->codes, 16) ||
        !aligned(a->scales, 16) ||
        !aligned(a->out, 8) || (a->idx_q && !aligned(a->idx_q, 16)) ||
        (a->idx_k && !aligned(a->idx_k, 16)))
        return CSA2_ERR_INVALID_ARG;
    const WsLayout L = layer_layout(a);
    if (!a->workspace || !aligned(a->workspace, 256) || a->workspace_bytes < L.total)
        return CSA2_ERR_WORKSPACE;

    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    uint8_t* ws = static_cast<uint8_t*>(a->workspace);
    unsigned* err = reinterpret_cast<unsigned*>(ws);
    const int rows = a->batch * a->q_per_seq;
    csa2_status st = CSA2_OK;
    SideFork fork;                                      // the HSI pool select's side stream

    if (a->mode == CSA2_MODE_REINDEX && a->ev_pool) {       // the pool of a deferred Full call
        const cudaError_t ce = cudaStreamWaitEvent(s, static_cast<cudaEvent_t>(a->ev_pool), 0);
        if (ce != cudaSuccess) return fail_cuda("csa2_attend ev_pool wait", ce);
    }
    if (a->mode != CSA2_MODE_REUSE) {
        IndexParams ip;
        ip.batch = a->batch;
        ip.q_per_seq = a->q_per_seq;
        ip.ratio = a->ratio;
        ip.max_n = a->max_n;
        ip.kv_offsets = a->kv_offsets;
        ip.q_pos = a->q_pos;
        ip.idx_q = a->idx_q;
        ip.idx_w = a->idx_w;
        ip.idx_k = a->idx_k;
        ip.idx_kscale = a->idx_kscale;
        ip.pool_blocks = (a->mode == CSA2_MODE_REINDEX) ? a->pool_blocks : nullptr;
        ip.rows = RowMap{a->page_table, a->page_rows, a->pages_per_seq};
        const bool want_bm = (a->mode == CSA2_MODE_FULL && a->want_pool);
        float* bm = want_bm ? reinterpret_cast<float*>(ws + L.blockmax) : nullptr;
        cudaError_t ce;
        // under stream capture the timing events must be event-record nodes of the graph
        cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
        if ((a->ev_index_begin || a->ev_index_end) && (ce = cudaStreamIsCapturing(s, &cap)) != cudaSuccess)
            return fail_cuda("csa2_attend cudaStreamIsCapturing", ce);
        const unsigned ev_flags = cap == cudaStreamCaptureStatusActive ? cudaEventRecordExternal : 0u;
        if (a->ev_index_begin &&
            (ce = cudaEventRecordWithFlags(static_cast<cudaEvent_t>(a->ev_index_begin), s, ev_flags)) !=
                cudaSuccess)
            return fail_cuda("csa2_attend ev_index_begin", ce);
        if (L.fused) {
            ScanSelectArgs sa;
            sa.p = ip;
            sa.chunk = L.chunk;
            sa.n_chunks = L.n_chunks;
            sa.cand_s = reinterpret_cast<float*>(ws + L.cand_s);
            sa.cand_p = reinterpret_cast<int32_t*>(ws + L.cand_p);
            sa.bm = bm;
            sa.bm_ld = L.bm_ld;
            sa.err = err;
            sa.chunk_thr = reinterpret_cast<float*>(ws + L.chunk_thr);
            CUtensorMap tmap;
            const bool pool = a->mode == CSA2_MODE_REINDEX;
            const bool contig = pool && a->pool_k != nullptr;
            sa.pool_kscale = contig ? a->pool_kscale : nullptr;
            const bool map_ok = contig ? make_idx_k_map(a->pool_k, static_cast<int64_t>(a->batch) * POOL_POSITIONS,
                                                        128, &tmap)
                                       : make_idx_k_map(a->idx_k, a->total_n, pool ? POOL_BLOCK : 128, &tmap);
            if (!map_ok) {
                std::snprintf(g_last_error, sizeof(g_last_error), "cuTensorMapEncodeTiled failed");
                return CSA2_ERR_CUDA;
            }
            st = launch_scan_select(sa, tmap, pool, want_bm, s);
        } else if (L.prefill_fused) {
            CUtensorMap tmap;
            if (!make_idx_k_map(a->idx_k, a->total_n, 128, &tmap)) {
                std::snprintf(g_last_error, sizeof(g_last_error), "cuTensorMapEncodeTiled failed");
                return CSA2_ERR_CUDA;
            }
            st = launch_prefill_index(ip, tmap, a->topk_idx, err, s);
        } else {
            st = launch_index_score(ip, reinterpret_cast<float*>(ws + L.scores), L.scores_ld,
                                    bm, L.bm_ld, s);
        }
        if (st != CSA2_OK) return st;
        if (a->ev_index_end &&
            (ce = cudaEventRecordWithFlags(static_cast<cudaEvent_t>(a->ev_index_end), s, ev_flags)) !=
                cudaSuccess)
            return fail_cuda("csa2_attend ev_index_end", ce);
        // The HSI pool select (Top-2,048 blocks) does not depend on the Top-512 select: it
        // runs on a side stream forked from s, beside the merge and the attention (neither
        // reads the pool), and is joined back at the end of the call.
        const cudaStream_t ps = bm ? fork.begin(s) : s;
        if (bm) {
            st = launch_topk_rows(bm, L.bm_ld, ceil_div(a->max_n, POOL_BLOCK), a->batch, POOL_BLOCKS,
                                  nullptr, 1, a->pool_blocks, ps, a->kv_offsets);
            if (st == CSA2_OK && a->pool_k)            // the pool's rows, contiguous, for Reindex
                st = launch_pool_gather(a->pool_blocks, a->kv_offsets, a->batch, a->idx_k, a->idx_kscale,
                                        a->pool_k, a->pool_kscale, ip.rows, ps);
        }
        if (st == CSA2_OK && L.fused) {
            st = launch_merge_select(reinterpret_cast<float*>(ws + L.cand_s),
                                     reinterpret_cast<int32_t*>(ws + L.cand_p),
                                     reinterpret_cast<float*>(ws + L.chunk_thr), L.n_chunks, rows,
                                     a->topk_idx, s);
        } else if (st == CSA2_OK && !L.prefill_fused) {
            const int64_t ncols = (a->mode == CSA2_MODE_REINDEX) ? POOL_POSITIONS : a->max_n;
            st = launch_topk_rows(reinterpret_cast<float*>(ws + L.scores), L.scores_ld, ncols, rows,
                                  TOPK, ip.pool_blocks, a->q_per_seq, a->topk_idx, s);
        }
        if (st != CSA2_OK) {
            (void)fork.join(s);
            return st;
        }
    }

    AttnParams ap;
    ap.batch = a->batch;
    ap.q_per_seq = a->q_per_seq;
    ap.ratio = a->ratio;
    ap.n_split = L.n_split;
    ap.swa_rows = a->swa_rows;
    ap.sm_scale = a->sm_scale;
    ap.kv_offsets = a->kv_offsets;
    ap.q_pos = a->q_pos;
    ap.codes = a->codes;
    ap.scales = a->scales;
    ap.topk_idx = a->topk_idx;
    ap.q = a->q;
    ap.swa_kv = a->swa_kv;
    ap.out = a->out;
    ap.err = err;
    ap.swa_fp8 = swa8 ? 1 : 0;
    ap.swa_kv8 = a->swa_kv8;
    ap.swa_kscale = a->swa_kscale;
    ap.rows = RowMap{a->page_table, a->page_rows, a->pages_per_seq};
    ap.q_nvfp4 = a->q_format == CSA2_Q_NVFP4 ? 1 : 0;
    {
        CUtensorMap tq, tswa;
        memset(&tswa, 0, sizeof(tswa));                  // unused by the FP8 SWA tiles
        if (!make_bf16_rows_map(a->q, static_cast<int64_t>(rows) * HEADS, 1, HEADS, 2, &tq) ||
            (!swa8 && !make_bf16_rows_map(a->swa_kv, a->swa_rows, a->batch, 32, 3, &tswa))) {
            std::snprintf(g_last_error, sizeof(g_last_error), "cuTensorMapEncodeTiled failed (attention)");
            (void)fork.join(s);
            return CSA2_ERR_CUDA;
        }
        st = launch_attend_rows(ap, tq, tswa, s);
    }
    const bool defer = st == CSA2_OK && a->ev_pool && a->mode == CSA2_MODE_FULL && a->want_pool;
    const csa2_status js = defer ? fork.defer(s, static_cast<cudaEvent_t>(a->ev_pool)) : fork.join(s);
    return st != CSA2_OK ? st : js;
}

csa2_status csa2_dequantize_kv(const uint8_t* codes, const uint8_t* scales, int64_t total_rows,
                               const int64_t* src_row, int64_t n, uint16_t* out, void* stream) {
    if (n < 0 || total_rows < 0) return CSA2_ERR_INVALID_ARG;
    if (n == 0) return CSA2_OK;
    if (!codes || !scales || !out || (!src_row && n > total_rows)) return CSA2_ERR_INVALID_ARG;
    if (!aligned(codes, 8) || !aligned(out, 16) || !aligned(src_row, 8)) return CSA2_ERR_INVALID_ARG;
    if (n > (int64_t(1) << 35)) return CSA2_ERR_UNSUPPORTED;
    return launch_dequantize(codes, scales, total_rows, src_row, n, out, static_cast<cudaStream_t>(stream));
}

csa2_status csa2_norm_rope(const csa2_rope_args* a, void* stream) {
    constexpr int32_t known = CSA2_ROPE_NORM | CSA2_ROPE_INVERSE | CSA2_ROPE_HALF;
    if (!a || a->reserved0 != 0 || (a->flags & ~known) != 0 || a->rows < 0) return CSA2_ERR_INVALID_ARG;
    if (!valid_type(a->in_type) || !valid_type(a->out_type)) return CSA2_ERR_INVALID_ARG;
    if (a->heads < 1 || a->dim < 8 || a->dim % 8 != 0 || a->rope_dim < 0 || a->rope_dim > a->dim || a->rope_dim % 2 != 0)
        return CSA2_ERR_INVALID_ARG;
    if (a->heads > 1024 || a->dim > 1024) return CSA2_ERR_UNSUPPORTED;
    if (!(a->eps >= 0.0f) || (a->weight && !(a->flags & CSA2_ROPE_NORM))) return CSA2_ERR_INVALID_ARG;
    if (a->rows == 0) return CSA2_OK;
    if (!a->x || !a->out || (a->rope_dim && (!a->pos || !a->inv_freq))) return CSA2_ERR_INVALID_ARG;
    if (!aligned(a->x, 16) || !aligned(a->out, 16) || !aligned(a->weight, 16) || !aligned(a->pos, 8) ||
        !aligned(a->inv_freq, 4))
        return CSA2_ERR_INVALID_ARG;
    const int xi = a->in_type == CSA2_T_F32 ? 4 : 8, oi = a->out_type == CSA2_T_F32 ? 4 : 8;   // elements per 16 B
    if (a->x_row_stride < 0 || a->x_row_stride % xi != 0 || a->x_head_stride % xi != 0 || a->x_head_stride < 0 ||
        a->out_row_stride < 0 || a->out_row_stride % oi != 0 || a->out_head_stride < 0 || a->out_head_stride % oi != 0)
        return CSA2_ERR_INVALID_ARG;
    // two vectors of out must not overlap: heads inside a row, or rows inside a head
    if (a->heads > 1 && a->out_head_stride < a->dim) return CSA2_ERR_INVALID_ARG;
    const __int128 row_span = static_cast<__int128>(a->heads - 1) * a->out_head_stride + a->dim;
    const __int128 col_span = static_cast<__int128>(a->rows - 1) * a->out_row_stride + a->dim;
    if (a->rows > 1 && !(a->out_row_stride >= row_span ||
                         (a->out_row_stride >= a->dim && (a->heads == 1 || a->out_head_stride >= col_span))))
        return CSA2_ERR_INVALID_ARG;
    if (a->x == a->out && (a->in_type != a->out_type || a->x_row_stride != a->out_row_stride ||
                           a->x_head_stride != a->out_head_stride))
        return CSA2_ERR_INVALID_ARG;
    RopeParams p;
    p.rows = a->rows;
    p.heads = a->heads;
    p.dim = a->dim;
    p.rope_dim = a->rope_dim;
    p.norm = (a->flags & CSA2_ROPE_NORM) != 0;
    p.inverse = (a->flags & CSA2_ROPE_INVERSE) != 0;
    p.half = (a->flags & CSA2_ROPE_HALF) != 0 && a->rope_dim > 0;
    p.x_row_stride = a->x_row_stride;
    p.x_head_stride = a->x_head_stride;
    p.out_row_stride = a->out_row_stride;
    p.out_head_stride = a->out_head_stride;
    p.x = a->x;
    p.out = a->out;
    p.pos = a->pos;
    p.inv_freq = a->inv_freq;
    p.weight = a->weight;
    p.eps = a->eps;
    return launch_norm_rope(p, a->in_type, a->out_type, static_cast<cudaStream_t>(stream));
}

csa2_status csa2_append_rope(const csa2_append_args* a, void* stream) {
    constexpr int32_t known = CSA2_ROPE_NORM | CSA2_ROPE_HALF;
    if (!a || (a->flags & ~known) != 0 || a->n < 0 || a->batch < 1 || !valid_type(a->in_type) || !(a->eps >= 0.0f))
        return CSA2_ERR_INVALID_ARG;
    if (a->rope_dim < 0 || a->rope_dim > D || a->rope_dim % 2 != 0 || a->idx_rope_dim < 0 || a->idx_rope_dim > IDX_DIM ||
        a->idx_rope_dim % 2 != 0 || (a->weight && !(a->flags & CSA2_ROPE_NORM)))
        return CSA2_ERR_INVALID_ARG;
    if ((a->kv_offsets != nullptr) == (a->page_table != nullptr)) return CSA2_ERR_INVALID_ARG;
    if (a->page_table && (a->page_rows < 128 || a->page_rows % 128 != 0 || a->page_rows > (1 << 24) || a->pages_per_seq < 1))
        return CSA2_ERR_INVALID_ARG;
    if (a->n == 0) return CSA2_OK;
    if (!a->latent || !a->pos || !a->codes || !a->scales || a->total_rows < 1 || (!a->seq && a->n > a->batch))
        return CSA2_ERR_INVALID_ARG;
    if ((a->rope_dim && !a->inv_freq) || (a->idx_proj && (!a->idx_k || !a->idx_kscale)) ||
        (a->idx_proj && a->idx_rope_dim && !a->idx_inv_freq))
        return CSA2_ERR_INVALID_ARG;
    const int li = a->in_type == CSA2_T_F32 ? 4 : 8;
    if (a->latent_stride < D || a->latent_stride % li != 0 ||
        (a->idx_proj && (a->idx_stride < IDX_DIM || a->idx_stride % 2 != 0)))
        return CSA2_ERR_INVALID_ARG;
    if (!aligned(a->latent, 16) || !aligned(a->idx_proj, 8) || !aligned(a->weight, 16) || !aligned(a->pos, 8) ||
        !aligned(a->seq, 4) || !aligned(a->kv_offsets, 8) || !aligned(a->page_table, 4) || !aligned(a->inv_freq, 4) ||
        !aligned(a->idx_inv_freq, 4) || !aligned(a->codes, 8) || !aligned(a->idx_k, 2) || !aligned(a->idx_kscale, 4))
        return CSA2_ERR_INVALID_ARG;
    if (a->workspace && !aligned(a->workspace, 256)) return CSA2_ERR_WORKSPACE;
    AppendParams p;
    p.n = a->n;
    p.batch = a->batch;
    p.rope_dim = a->rope_dim;
    p.idx_rope_dim = a->idx_rope_dim;
    p.norm = (a->flags & CSA2_ROPE_NORM) != 0;
    p.half = (a->flags & CSA2_ROPE_HALF) != 0;
    p.eps = a->eps;
    p.latent_stride = a->latent_stride;
    p.idx_stride = a->idx_stride;
    p.total_rows = a->total_rows;
    p.latent = a->latent;
    p.idx_proj = a->idx_proj;
    p.seq = a->seq;
    p.pos = a->pos;
    p.kv_offsets = a->kv_offsets;
    p.rows = RowMap{a->page_table, a->page_rows, a->pages_per_seq};
    p.inv_freq = a->inv_freq;
    p.idx_inv_freq = a->idx_inv_freq;
    p.weight = a->weight;
    p.codes = a->codes;
    p.scales = a->scales;
    p.idx_k = a->idx_k;
    p.idx_kscale = a->idx_kscale;
    p.err = static_cast<unsigned*>(a->workspace);
    return launch_append_rope(p, a->in_type, static_cast<cudaStream_t>(stream));
}

size_t csa2_cache_workspace_size(const csa2_cache_args* a) {
    if (!a || a->batch < 1 || a->q_per_seq < 1 || a->max_n < 1 || a->window < 0 || a->sinks < 0) return 0;
    if (!cache_sizes_fit(a)) return 0;
    return cache_layout(a).total;
}

csa2_status csa2_attend_cache(const csa2_cache_args* a, void* stream) {
    if (!a) return CSA2_ERR_INVALID_ARG;
    if (a->batch < 1 || a->q_per_seq < 1 || a->q_per_seq > 65536 || (a->ratio != 1 && a->ratio != 2))
        return CSA2_ERR_INVALID_ARG;
    if (a->out_type != CSA2_T_BF16 && a->out_type != CSA2_T_F32)
        return valid_type(a->out_type) ? CSA2_ERR_UNSUPPORTED : CSA2_ERR_INVALID_ARG;
    if (a->reserved0 != 0 || a->max_n < 1 || a->total_n < 1 || a->total_n > INT32_MAX || a->window < 0 || a->sinks < 0)
        return CSA2_ERR_INVALID_ARG;
    if (!cache_sizes_fit(a)) return CSA2_ERR_UNSUPPORTED;
    if (ceil_div(a->max_n, CACHE_TILE) * a->batch * a->q_per_seq > INT32_MAX) return CSA2_ERR_UNSUPPORTED;   // tiles too
    if (!a->kv_offsets || !a->codes || !a->scales || !a->q || !a->out) return CSA2_ERR_INVALID_ARG;
    if (!(a->sm_scale - a->sm_scale == 0.0f)) return CSA2_ERR_INVALID_ARG;          // finite
    if (!aligned(a->codes, 16) || !aligned(a->scales, 16) || !aligned(a->q, 16) || !aligned(a->out, 16) ||
        !aligned(a->lse, 4) || !aligned(a->kv_offsets, 8) || !aligned(a->q_pos, 8) || !aligned(a->page_table, 4))
        return CSA2_ERR_INVALID_ARG;
    if (a->page_table) {
        if (a->page_rows < 128 || a->page_rows % 128 != 0 || a->page_rows > (1 << 24)) return CSA2_ERR_INVALID_ARG;
        if (a->pages_per_seq < ceil_div(a->max_n, a->page_rows)) return CSA2_ERR_INVALID_ARG;
    }
    const CacheLayout L = cache_layout(a);
    if (!a->workspace || !aligned(a->workspace, 256) || a->workspace_bytes < L.total) return CSA2_ERR_WORKSPACE;
    uint8_t* ws = static_cast<uint8_t*>(a->workspace);
    CacheParams p;
    p.batch = a->batch;
    p.q_per_seq = a->q_per_seq;
    p.ratio = a->ratio;
    p.out_f32 = a->out_type == CSA2_T_F32;
    p.max_n = static_cast<int>(a->max_n);
    p.total_n = static_cast<int>(a->total_n);
    p.window = static_cast<int>(std::min<int64_t>(a->window, INT32_MAX));
    p.sinks = static_cast<int>(std::min<int64_t>(a->sinks, INT32_MAX));
    p.kv_offsets = a->kv_offsets;
    p.q_pos = a->q_pos;
    p.q = a->q;
    p.sm_scale = a->sm_scale;
    p.out = a->out;
    p.lse = a->lse;
    p.rows = RowMap{a->page_table, a->page_rows, a->pages_per_seq};
    p.err = reinterpret_cast<unsigned*>(ws);
    p.meta = reinterpret_cast<int32_t*>(ws + L.meta);
    p.part = reinterpret_cast<float*>(ws + L.part);
    p.ranges = L.plan.ranges;
    p.whole_rows = L.plan.whole_rows;
    CUtensorMap codes, scales;
    if (!make_byte_rows_map(a->codes, a->total_n, ROW_CODES, 128, CACHE_TILE, CU_TENSOR_MAP_SWIZZLE_128B, &codes) ||
        !make_byte_rows_map(a->scales, a->total_n, ROW_SCALES, ROW_SCALES, CACHE_TILE, CU_TENSOR_MAP_SWIZZLE_NONE, &scales)) {
        std::snprintf(g_last_error, sizeof(g_last_error), "cuTensorMapEncodeTiled failed (cache)");
        return CSA2_ERR_CUDA;
    }
    return launch_attend_cache(p, codes, scales, static_cast<cudaStream_t>(stream));
}

csa2_status csa2_set_wait_limit(void* workspace, uint32_t polls, void* stream) {
    if (!workspace || !aligned(workspace, 256)) return CSA2_ERR_WORKSPACE;
    // word 1 of the header (word 0 is the error word); a pageable source is staged by the
    // runtime before the call returns, so the local may go out of scope
    const unsigned v = polls;
    const cudaError_t ce = cudaMemcpyAsync(static_cast<unsigned*>(workspace) + 1, &v, sizeof(v),
                                           cudaMemcpyHostToDevice, static_cast<cudaStream_t>(stream));
    return ce == cudaSuccess ? CSA2_OK : fail_cuda("csa2_set_wait_limit", ce);
}

csa2_status csa2_check_device_status(void* workspace, void* stream) {
    if (!workspace || !aligned(workspace, 256)) return CSA2_ERR_WORKSPACE;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    unsigned h = 0;
    cudaError_t ce = cudaMemcpyAsync(&h, workspace, sizeof(h), cudaMemcpyDeviceToHost, s);
    if (ce == cudaSuccess) ce = cudaStreamSynchronize(s);
    if (ce != cudaSuccess) return fail_cuda("csa2_check_device_status", ce);
    if (h != 0 && (ce = cudaMemsetAsync(workspace, 0, sizeof(unsigned), s)) != cudaSuccess)
        return fail_cuda("csa2_check_device_status", ce);
    if (h & ERR_TIMEOUT) return CSA2_ERR_TIMEOUT;
    if (h & ERR_DEVICE) return CSA2_ERR_DEVICE;
    return CSA2_OK;
}

}  // extern "C"
