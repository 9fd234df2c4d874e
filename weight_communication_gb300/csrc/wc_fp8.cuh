// wc_fp8.cuh -- 8-bit (e4m3) codes with one fp32 scale per block of 128 values:
// the rule that makes them and the way back, shared by the kernels that write
// or read such matrices.
//
//   m = max |x| of the block
//   m < 448 * 2^-126 (the scale would not be normal): scale 0, codes 0
//   m infinite or not a number:                       scale NaN, codes 0
//   else scale = m / 448, code = e4m3(x * fl(448 / m)), to nearest, ties to even
//
// 448 is e4m3's largest value, so no code saturates.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "wc_device.cuh"

namespace wc {

constexpr float kFp8Top = 448.0f;

struct Scale8 {
    float scale, inv;
};

__device__ __forceinline__ Scale8 scale_of(float m) {
    Scale8 s;
    if (m < kFp8Top * kMinNormal) {  // exact product
        s.scale = 0.0f;
        s.inv = 0.0f;
    } else if (m <= 3.40282346638528859812e38f) {
        s.scale = __fdiv_rn(m, kFp8Top);
        s.inv = __fdiv_rn(kFp8Top, m);
    } else {
        s.scale = __uint_as_float(0x7FC00000u);
        s.inv = 0.0f;
    }
    return s;
}

// Codes of 8 values of blocks with one inv.  inv 0 gives codes 0 also where
// the product is not a number.
__device__ __forceinline__ uint2 codes_of(const float (&x)[8], float inv) {
    uint32_t h[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        h[j] = __nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(x[2 * j], inv), __fmul_rn(x[2 * j + 1], inv)),
                                        __NV_SATFINITE, __NV_E4M3);
    return inv == 0.0f ? make_uint2(0u, 0u) : make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

// What 8 codes of one block stand for: exact in fp16, then one product.
__device__ __forceinline__ void values_of(uint2 codes, float scale, float (&x)[8]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t w = (j < 2 ? codes.x : codes.y) >> (16 * (j & 1));
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(w & 0xFFFFu), __NV_E4M3);
        const float2 f = __half22float2(__half2(h));
        x[2 * j] = __fmul_rn(f.x, scale);
        x[2 * j + 1] = __fmul_rn(f.y, scale);
    }
}

}  // namespace wc
