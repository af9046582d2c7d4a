// FP4 main-KV quantiser: bf16 latent rows -> E2M1 codes + one E4M3 scale per 16 channels
// ("FP4 KV, Bounded Replay, and Other Extensions" section of the thecryptopost.io
// DeepSeek-V4.1-Flash article: E2M1 with one E4M3 scale per 16 channels, NVFP4 without
// its global scale), optionally after ratio-2 merging of adjacent positions (CSA2
// section: the encoder compresses at ratio 2; tldrocket.com: merging of adjacent
// positions).
//
// One warp per output row, one lane per 16-channel group: a warp reads 1 KB (2 KB at
// ratio 2) of contiguous bf16 and writes 256 contiguous code bytes + 32 scale bytes.
// The rounding decisions use IEEE fp32 division (never a reciprocal multiply): both
// operands carry at most 8 significant bits, so the fp32 quotient lands exactly on a
// rounding midpoint iff the exact quotient does, and never crosses one.
#include <cuda_fp4.h>

#include "dense.cuh"
#include "row_formats.cuh"
#include "tc.cuh"

namespace csa2 {

namespace {

// Round-to-nearest-even of a float64 value to bf16, through a round-to-odd float32
// intermediate (16 spare bits make the second rounding exact).
__device__ __forceinline__ uint16_t f64_to_bf16_rne(double m) {
    float f = __double2float_rz(m);
    if (static_cast<double>(f) != m) f = __uint_as_float(__float_as_uint(f) | 1u);
    __nv_bfloat16 h = __float2bfloat16_rn(f);
    return *reinterpret_cast<uint16_t*>(&h);
}

__device__ __forceinline__ void unpack8(const uint4& v, uint16_t (&h)[16], int base) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        h[base + 2 * i] = static_cast<uint16_t>(w[i] & 0xFFFFu);
        h[base + 2 * i + 1] = static_cast<uint16_t>(w[i] >> 16);
    }
}

// One 16-channel group (nvfp4_group): 8 packed code bytes and the scale byte stored.
__device__ __forceinline__ void store_group(const uint16_t (&h)[16], uint8_t* code_dst, uint8_t* scale_dst) {
    uint2 v;
    const uint8_t scale_code = nvfp4_group(h, v);
    *reinterpret_cast<uint2*>(code_dst) = v;
    *scale_dst = scale_code;
}

__global__ void __launch_bounds__(256)
quantize_kernel(const uint16_t* __restrict__ x, int64_t n_out, int ratio,
                const int64_t* __restrict__ dst_row, uint8_t* __restrict__ codes,
                uint8_t* __restrict__ scales) {
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x / 32) + threadIdx.x / 32;
    if (row >= n_out) return;
    const int lane = threadIdx.x & 31;

    uint16_t h[16];                       // the group's 16 bf16 inputs (after merging)
    if (ratio == 1) {
        const uint16_t* src = x + row * D + lane * GROUP;
        unpack8(ldg_stream(src), h, 0);
        unpack8(ldg_stream(src + 8), h, 8);
    } else {
        uint16_t a[16], b[16];
        const uint16_t* s0 = x + (2 * row) * D + lane * GROUP;
        const uint16_t* s1 = s0 + D;
        unpack8(ldg_stream(s0), a, 0);
        unpack8(ldg_stream(s0 + 8), a, 8);
        unpack8(ldg_stream(s1), b, 0);
        unpack8(ldg_stream(s1 + 8), b, 8);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            // the pair sum is exact in float64; halving is exact; one rounding to bf16
            const double m = (static_cast<double>(bf16_bits_to_float(a[i])) +
                              static_cast<double>(bf16_bits_to_float(b[i]))) * 0.5;
            h[i] = f64_to_bf16_rne(m);
        }
    }

    const int64_t out_row = dst_row ? dst_row[row] : row;
    store_group(h, codes + out_row * ROW_CODES + lane * 8, scales + out_row * ROW_SCALES + lane);
}

// Cache append of new positions: warp per row.  Lane l quantises channels 16l..16l+15
// of the main-KV row (as above) and indexer values 2l, 2l+1 (store_idx_row).
__global__ void __launch_bounds__(256)
append_kernel(const uint16_t* __restrict__ latent, const float* __restrict__ proj, int64_t n,
              const int64_t* __restrict__ dst_row, uint8_t* __restrict__ codes,
              uint8_t* __restrict__ scales, uint8_t* __restrict__ idx_k, float* __restrict__ idx_kscale) {
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x / 32) + threadIdx.x / 32;
    if (row >= n) return;
    const int lane = threadIdx.x & 31;
    const int64_t out_row = dst_row[row];

    uint16_t h[16];
    const uint16_t* src = latent + row * D + lane * GROUP;
    unpack8(ldg_stream(src), h, 0);
    unpack8(ldg_stream(src + 8), h, 8);
    store_group(h, codes + out_row * ROW_CODES + lane * 8, scales + out_row * ROW_SCALES + lane);

    const float2 k = __ldg(reinterpret_cast<const float2*>(proj + row * IDX_DIM) + lane);
    store_idx_row(k, lane, idx_k + out_row * IDX_DIM, idx_kscale + out_row);
}

// FP4 rows back to bf16, bound by HBM (131,072 rows in 26 to 29 us, 5.9 to 6.7 TB/s; 39 with 16
// channels a lane, whose stores are not contiguous): a row is 64 pieces of 8 channels; lane l takes pieces l and l + 32,
// so that a warp's loads (4 B) and stores (16 B) are contiguous, four rows in flight.  e2m1 x
// e4m3 has at most 6 significant bits, so the fp32 product and its bf16 rounding are exact.
constexpr int DQ_ROWS = 4;

__global__ void __launch_bounds__(256)
dequantize_kernel(const uint8_t* codes, const uint8_t* scales, int64_t total_rows, const int64_t* src_row, int64_t n,
                  uint16_t* out) {
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t first = (static_cast<int64_t>(blockIdx.x) * (blockDim.x / 32) + threadIdx.x / 32) * DQ_ROWS;
    uint32_t c[DQ_ROWS][2], sc[DQ_ROWS][2];
#pragma unroll
    for (int r = 0; r < DQ_ROWS; ++r) {
        int64_t row = -1;
        if (first + r < n) row = src_row ? src_row[first + r] : first + r;
        const bool ok = row >= 0 && row < total_rows;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            c[r][k] = ok ? reinterpret_cast<const uint32_t*>(codes + row * ROW_CODES)[lane + 32 * k] : 0u;
            sc[r][k] = ok ? scales[row * ROW_SCALES + lane / 2 + 16 * k] : 0u;
        }
    }
#pragma unroll
    for (int r = 0; r < DQ_ROWS; ++r) {
        if (first + r >= n) return;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float s = e4m3_to_float(static_cast<uint8_t>(sc[r][k]));
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __half2_raw hr =
                    __nv_cvt_fp4x2_to_halfraw2(static_cast<__nv_fp4x2_storage_t>((c[r][k] >> (8 * i)) & 0xFFu), __NV_E2M1);
                const float2 f = __half22float2(__half2(hr));
                const __nv_bfloat162 v = __floats2bfloat162_rn(f.x * s, f.y * s);
                w[i] = *reinterpret_cast<const uint32_t*>(&v);
            }
            __stcs(reinterpret_cast<uint4*>(out + (first + r) * D) + lane + 32 * k, make_uint4(w[0], w[1], w[2], w[3]));
        }
    }
}

}  // namespace

csa2_status launch_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t total_rows, const int64_t* src_row,
                              int64_t n, uint16_t* out, cudaStream_t stream) {
    if (n == 0) return CSA2_OK;
    const int rows_per_block = 8 * DQ_ROWS;
    launch_dependent(dequantize_kernel, dim3(static_cast<unsigned>(ceil_div(n, rows_per_block))), 256, 0, stream, codes, scales,
                     total_rows, src_row, n, out);
    return check_launch("dequantize_kernel");
}

csa2_status launch_append(const uint16_t* latent, const float* proj, int64_t n, const int64_t* dst_row,
                          uint8_t* codes, uint8_t* scales, uint8_t* idx_k, float* idx_kscale,
                          cudaStream_t stream) {
    if (n == 0) return CSA2_OK;
    const int rows_per_block = 8;
    append_kernel<<<static_cast<unsigned>(ceil_div(n, rows_per_block)), 32 * rows_per_block, 0, stream>>>(
        latent, proj, n, dst_row, codes, scales, idx_k, idx_kscale);
    return check_launch("append_kernel");
}

csa2_status launch_quantize(const uint16_t* x, int64_t n_in, int ratio, const int64_t* dst_row,
                            uint8_t* codes, uint8_t* scales, cudaStream_t stream) {
    const int64_t n_out = n_in / ratio;
    if (n_out == 0) return CSA2_OK;
    const int rows_per_block = 8;
    const int64_t grid = ceil_div(n_out, rows_per_block);
    quantize_kernel<<<static_cast<unsigned>(grid), 32 * rows_per_block, 0, stream>>>(
        x, n_out, ratio, dst_row, codes, scales);
    return check_launch("quantize_kernel");
}

}  // namespace csa2
