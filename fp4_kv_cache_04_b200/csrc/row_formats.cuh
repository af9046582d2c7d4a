// Conversions of cache rows shared by the quantiser, the plain append and the append with
// norm and rotation.
#pragma once

#include "common.cuh"

namespace csa2 {

// E4M3 codes of lo (bits 0..7) and hi (8..15), to nearest even, saturating at 448.
__device__ __forceinline__ uint32_t e4m3x2_rn(float lo, float hi) {
    uint16_t v;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(v) : "f"(hi), "f"(lo));
    return v;
}

// nvfp4_group with the hardware's E2M1 rounding (to nearest even, saturating, the sign kept
// when the magnitude rounds to 0) and a quotient by reciprocal and one residual step
// (Markstein's correction: the residual x - y s is exact in the fma).  x and s carry at most 8
// and 4 significant bits, so x / s is a rounding midpoint of E2M1 exactly or at least 2^-12
// away from it; the residual brings y to within a unit of the quotient, and to the quotient
// itself where that has 3 bits.
__device__ __forceinline__ uint8_t nvfp4_group_hw(const uint16_t (&h)[16], uint2& codes) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) top = max(top, static_cast<uint32_t>(h[i] & 0x7FFFu));
    if (top >= 0x7F80u) return nvfp4_group(h, codes);      // infinities and NaN as there
    // amax / 6 by the same correction: 8 bits over 2, against E4M3's midpoints of 5
    const float amax = bf16_bits_to_float(static_cast<uint16_t>(top)), q0 = amax * (1.0f / 6.0f);
    const uint32_t scale_code = e4m3x2_rn(fmaf(fmaf(-q0, 6.0f, amax), 1.0f / 6.0f, q0), 0.0f) & 0xFFu;
    const float s = e4m3_to_float(static_cast<uint8_t>(scale_code));
    const float r = scale_code ? __frcp_rn(s) : 0.0f;
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
        float y[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float x = bf16_bits_to_float(h[i + e]), y0 = x * r;
            // (the residual of -0 is +0, which would take its sign)
            y[e] = __uint_as_float(__float_as_uint(fmaf(fmaf(-y0, s, x), r, y0)) | (static_cast<uint32_t>(h[i + e] & 0x8000u) << 16));
        }
        uint32_t b;
        asm("{ .reg .b8 t; cvt.rn.satfinite.e2m1x2.f32 t, %1, %2; cvt.u32.u8 %0, t; }" : "=r"(b) : "f"(y[1]), "f"(y[0]));
        w[i / 8] |= b << (4 * (i & 7));
    }
    codes.x = w[0];
    codes.y = w[1];
    return static_cast<uint8_t>(scale_code);
}

// Indexer-K row of a position, whole warp: lane l holds values 2l, 2l+1.  kscale = amax /
// 448 and code = sign | E4M3 RNE saturating of |k / kscale|, both quotients IEEE fp32; an
// all-zero row gets kscale 0 and zero codes.
__device__ __forceinline__ void store_idx_row(float2 k, int lane, uint8_t* idx_k, float* idx_kscale) {
    float amax = fmaxf(fabsf(k.x), fabsf(k.y));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, off));
    const float ks = amax / 448.0f;
    uint32_t c = 0;
    if (ks > 0.0f) {
        // the minimum takes NaN (a NaN value, or inf / inf) to 448
        const float q0 = k.x / ks, q1 = k.y / ks;
        c = e4m3x2_rn(copysignf(fminf(fabsf(q0), 448.0f), q0), copysignf(fminf(fabsf(q1), 448.0f), q1));
    }
    reinterpret_cast<uint16_t*>(idx_k)[lane] = static_cast<uint16_t>(c);
    if (lane == 0) *idx_kscale = ks;
}

}  // namespace csa2
