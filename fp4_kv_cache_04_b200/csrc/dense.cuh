// Launchers of the dense-cache operators: read-back, norm and rotation, append with both,
// attention over the whole cache.
#pragma once

#include <cuda.h>

#include "common.cuh"

namespace csa2 {

// Launch as a programmatic dependent of the kernel before it on the stream: the kernel must
// call griddep_wait() before it touches global memory.
template <typename... Params, typename... Args>
inline void launch_dependent(void (*kernel)(Params...), dim3 grid, int threads, int smem, cudaStream_t stream,
                             const Args&... args) {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    cudaLaunchKernelEx(&cfg, kernel, args...);
}

// FP4 rows back to bf16 (rows outside [0, total_rows) give zeros).
csa2_status launch_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t total_rows, const int64_t* src_row,
                              int64_t n, uint16_t* out, cudaStream_t stream);

// Head norm and rotation of [rows][heads][dim] vectors (csa2_norm_rope).
struct RopeParams {
    int64_t rows;
    int heads, dim, rope_dim;
    int norm, inverse, half;
    int64_t x_row_stride, x_head_stride, out_row_stride, out_head_stride;
    const void* x;
    void* out;
    const int64_t* pos;
    const float* inv_freq;
    const float* weight;
    float eps;
};
csa2_status launch_norm_rope(const RopeParams& p, int in_type, int out_type, cudaStream_t stream);

// Cache append with norm and rotation (csa2_append_rope).
struct AppendParams {
    int64_t n;
    int batch, rope_dim, idx_rope_dim;
    int norm, half;
    float eps;
    int64_t latent_stride, idx_stride, total_rows;
    const void* latent;
    const float* idx_proj;
    const int32_t* seq;
    const int64_t* pos;
    const int64_t* kv_offsets;
    RowMap rows;
    const float* inv_freq;
    const float* idx_inv_freq;
    const float* weight;
    uint8_t* codes;
    uint8_t* scales;
    uint8_t* idx_k;
    float* idx_kscale;
    unsigned* err;            // device error word, or nullptr
};
csa2_status launch_append_rope(const AppendParams& p, int in_type, cudaStream_t stream);

// Attention over the cache without an index (csa2_attend_cache): the visible tiles of all
// rows form one list, cut into at most CACHE_MAX_RANGES equal ranges; a row cut by a range's end
// is joined from the ranges' partials.
struct CacheParams {
    int batch, q_per_seq, ratio, out_f32;
    int max_n, total_n;
    int window, sinks;        // clamped to 2^31 - 1
    const int64_t* kv_offsets;
    const int64_t* q_pos;
    const uint16_t* q;
    float sm_scale;
    void* out;
    float* lse;
    RowMap rows;
    unsigned* err;            // workspace header
    int32_t* meta;            // [ranges][2] rows of a range's two partials (-1: none)
    float* part;              // [ranges][2] partials: m[16], l[16], O[16][512]
    int ranges;
    int whole_rows;           // ranges are whole rows: nothing to join
};
constexpr int CACHE_TILE = 128;                                  // positions per tile
constexpr int CACHE_MAX_RANGES = 148;                            // one CTA per SM
constexpr int CACHE_PART_FLOATS = 2 * HEADS + HEADS * D;
struct CachePlan {
    int ranges;
    bool whole_rows;
    int room;                 // ranges that the workspace has room for: >= ranges, and never less for more work
};
CachePlan cache_plan(int64_t rows, int64_t max_n, int64_t window, int64_t sinks);
// Tensor maps over codes as [total_n][256] bytes (boxes of 128 rows x 128 bytes, 128-byte
// swizzle) and scales as [total_n][32] bytes (boxes of 128 rows, no swizzle).
csa2_status launch_attend_cache(const CacheParams& p, const CUtensorMap& codes, const CUtensorMap& scales,
                                cudaStream_t stream);

}  // namespace csa2
