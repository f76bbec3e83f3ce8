// q8_codes.cuh -- conversions between INT8 codes and floats shared by the INT8
// quantizers, the W8A16 product and the paged KV-cache kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "q4_device.cuh"

namespace q4dev {

// INT8 code of one value, clamp(rne(fl(v / s)), qmin, 127), through t = v * r
// (r = 1/s correctly rounded, from quot_recip): |t - fl(v/s)| <= |t| (3u + u^2)
// (u = 2^-24), below 3.2e-5 while |t| < 178, and t - rint(t) is exact; so when
// |t - rint(t)| < 0.5 - 3.2e-5 both round to the same integer, and from
// |t| >= 178 on both clamp alike.  Otherwise (near a tie, or a NaN) the exact
// quotient is rounded as the definition states (NaN -> qmin).
__device__ __forceinline__ int int8_code(float v, float s, float r, int qmin) {
    const float t = __fmul_rn(v, r);
    const int q = __float2int_rn(t);
    if (fabsf(__fsub_rn(t, __int2float_rn(q))) < 0.4999679f) return min(max(q, qmin), 127);
    float u = rintf(__fdiv_rn(v, s));
    u = fminf(fmaxf(u, static_cast<float>(qmin)), 127.f);
    return static_cast<int>(u);
}

// Eight codes as two little-endian words (element 0 in byte 0).
__device__ __forceinline__ uint2 pack8_bytes(const int (&q)[8]) {
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t lo = __byte_perm(q[4 * h], q[4 * h + 1], 0x0040);
        const uint32_t hi = __byte_perm(q[4 * h + 2], q[4 * h + 3], 0x0040);
        w[h] = __byte_perm(lo, hi, 0x5410);
    }
    return make_uint2(w[0], w[1]);
}

// The cache's own 16-bit type: bits of a value rounded to nearest even, and back.
template <bool BF16>
__device__ __forceinline__ uint16_t cache_bits(float v) {
    if constexpr (BF16) {
        const __nv_bfloat16 h = __float2bfloat16_rn(v);
        return *reinterpret_cast<const uint16_t*>(&h);
    } else {
        const __half h = __float2half_rn(v);
        return *reinterpret_cast<const uint16_t*>(&h);
    }
}
template <bool BF16>
__device__ __forceinline__ float cache_value(uint16_t b) {
    if constexpr (BF16) {
        return __uint_as_float(static_cast<uint32_t>(b) << 16);
    } else {
        return __half2float(__ushort_as_half(b));
    }
}

// Two codes of a word (bytes selected by `sel`: 0x4140 for bytes 0, 1 and
// 0x4342 for bytes 2, 3) as a pair of exact 16-bit floats.
template <bool BF16>
__device__ __forceinline__ uint32_t q8_pair(uint32_t w, uint32_t sel) {
    if constexpr (BF16) {
        const uint32_t p = prmt(w, 0x43u, sel);  // 0x43 b' 0x43 b
        return sub2<true>(p & 0xFF7FFF7Fu, p & 0xFF80FF80u);
    } else {
        const uint32_t p = prmt(w, 0x64u, sel) ^ 0x00800080u;
        return sub2<false>(p, 0x64806480u);
    }
}

}  // namespace q4dev
