// ep_fp4.cuh -- the MXFP4 codec (OCP Microscaling Formats 1.0): per 32 channels one E8M0 byte
// b = max(floor(log2 amax) - 2 + 127, 0), codes = e2m1 of x * 2^(127 - b), nearest even, 6 the largest.
// The scale is a power of two, so that the division is exact and the code is x's, rounded once.  An
// infinity or a NaN among the 32 makes the byte 255, a NaN for all of them.
#pragma once
#include <cuda_fp4.h>

#include "ep_tcgen05.cuh"

namespace ep {

__host__ __device__ inline int64_t fp4_row_bytes(int H) { return ((int64_t)H / 2 + H / 32 + 15) / 16 * 16; }

// The byte of a block's largest magnitude (max_or_nan's).
__device__ __forceinline__ uint32_t e8m0_of(float amax) {
    const uint32_t e = __float_as_uint(amax) >> 23 & 255u;
    return e == 255u ? 255u : e > 2u ? e - 2u : 0u;
}
// 2^(127 - b), for b up to 252.
__device__ __forceinline__ float e8m0_inverse(uint32_t b) { return __uint_as_float((254u - min(b, 253u)) << 23); }

// Eight codes, the first in the lowest bits.
__device__ __forceinline__ uint32_t e2m1x8(const float* v, float by) {
    uint32_t c = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        c |= (uint32_t)__nv_cvt_float2_to_fp4x2(make_float2(v[2 * i] * by, v[2 * i + 1] * by), __NV_E2M1, cudaRoundNearest) << (8 * i);
    return c;
}

}  // namespace ep
