// Conversions of cache rows shared by the quantiser, the plain append and the append with
// norm and rotation.
#pragma once

#include "common.cuh"

namespace csa2 {

// Round-to-nearest-even of a float64 value to bf16, through a round-to-odd float32
// intermediate (16 spare bits make the second rounding exact).
__device__ __forceinline__ uint16_t f64_to_bf16_rne(double m) {
    float f = __double2float_rz(m);
    if (static_cast<double>(f) != m) f = __uint_as_float(__float_as_uint(f) | 1u);
    __nv_bfloat16 h = __float2bfloat16_rn(f);
    return *reinterpret_cast<uint16_t*>(&h);
}

// Indexer-K row of a position, whole warp: lane l holds values 2l, 2l+1.  kscale = amax /
// 448 and code = sign | E4M3 RNE saturating of |k / kscale|, both quotients IEEE fp32; an
// all-zero row gets kscale 0 and zero codes.
__device__ __forceinline__ void store_idx_row(float2 k, int lane, uint8_t* idx_k, float* idx_kscale) {
    float amax = fmaxf(fabsf(k.x), fabsf(k.y));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, off));
    const float ks = amax / 448.0f;
    uint32_t c0 = 0, c1 = 0;
    if (ks > 0.0f) {
        const float q0 = k.x / ks, q1 = k.y / ks;
        c0 = (signbit(q0) ? 0x80u : 0u) | e4m3_encode_rne_sat(fabsf(q0));
        c1 = (signbit(q1) ? 0x80u : 0u) | e4m3_encode_rne_sat(fabsf(q1));
    }
    reinterpret_cast<uint16_t*>(idx_k)[lane] = static_cast<uint16_t>(c0 | (c1 << 8));
    if (lane == 0) *idx_kscale = ks;
}

}  // namespace csa2
