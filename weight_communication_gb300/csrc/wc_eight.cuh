// wc_eight.cuh -- a row's block of 128 values over 16 lanes, 8 values each.
//
// VEC: lane l holds columns 8l .. 8l + 7, moved 16 bytes at a time; rows then
// start on 16 bytes and have a multiple of 8 columns.  Otherwise lane l holds
// columns l, l + 16, .., l + 112, moved one at a time, so that rows may start on
// any value and end on any column and neighbouring lanes still touch
// neighbouring values.
#pragma once

#include <stdint.h>

#include "wc_device.cuh"
#include "wc_fp8.cuh"

namespace wc {

constexpr int kBlock8 = 128;  // values per scale

// (Written once and read by a later kernel: first to leave L2.  8192 x 11008 gated
// activation, both ways, 246 -> 234 us; norm of 8192 x 4096, 100 -> 96.)
__device__ __forceinline__ void st_stream_u4(void *p, uint4 v) { __stcs(reinterpret_cast<uint4 *>(p), v); }

template <bool VEC>
__device__ __forceinline__ int column_of(int l, int j) {
    return VEC ? 8 * l + j : l + 16 * j;
}

// Values as they are stored: bf16 two to a word where they come so, else one to a
// word, as a load leaves it, so that nothing waits for it before the value is used.
// `p`: the block's first value, `left`: columns from there to the row's end.  mag():
// the largest magnitude's encoding, in which infinities and NaN are above all finite
// values.
template <typename T, bool VEC>
struct Eight;

template <>
struct Eight<uint16_t, true> {
    uint32_t w[4];
    __device__ __forceinline__ void load(const uint16_t *p, int l, int left) {
        const uint4 q = 8 * l < left ? ld_stream_u4(p + 8 * l) : make_uint4(0u, 0u, 0u, 0u);
        w[0] = q.x;
        w[1] = q.y;
        w[2] = q.z;
        w[3] = q.w;
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = 0u;
    }
    __device__ __forceinline__ float at(int j) const {
        return __uint_as_float((j & 1) ? (w[j / 2] & 0xFFFF0000u) : (w[j / 2] << 16));
    }
    __device__ __forceinline__ uint32_t mag() const {
        uint32_t m = w[0] & 0x7FFF7FFFu;
#pragma unroll
        for (int k = 1; k < 4; ++k) m = __vmaxu2(m, w[k] & 0x7FFF7FFFu);
        return max(m << 16, m & 0xFFFF0000u);
    }
    __device__ __forceinline__ void set(const float (&x)[8]) {
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = f32x2_to_bf16x2_bits(x[2 * k], x[2 * k + 1]);
    }
    __device__ __forceinline__ void store(uint16_t *p, int l, int left) const {
        if (8 * l < left) st_stream_u4(p + 8 * l, make_uint4(w[0], w[1], w[2], w[3]));
    }
};

template <>
struct Eight<uint16_t, false> {
    uint32_t w[8];
    __device__ __forceinline__ void load(const uint16_t *p, int l, int left) {
        if (left >= kBlock8) {  // (most blocks, without comparisons)
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = p[l + 16 * j];
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = l + 16 * j < left ? p[l + 16 * j] : 0u;
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = 0u;
    }
    __device__ __forceinline__ float at(int j) const { return __uint_as_float(w[j] << 16); }
    __device__ __forceinline__ uint32_t mag() const {
        uint32_t m = w[0] & 0x7FFFu;
#pragma unroll
        for (int j = 1; j < 8; ++j) m = max(m, w[j] & 0x7FFFu);
        return m << 16;
    }
    __device__ __forceinline__ void set(const float (&x)[8]) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t both = f32x2_to_bf16x2_bits(x[2 * k], x[2 * k + 1]);
            w[2 * k] = both & 0xFFFFu;
            w[2 * k + 1] = both >> 16;
        }
    }
    __device__ __forceinline__ void store(uint16_t *p, int l, int left) const {
        if (left >= kBlock8) {
#pragma unroll
            for (int j = 0; j < 8; ++j) p[l + 16 * j] = uint16_t(w[j]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (l + 16 * j < left) p[l + 16 * j] = uint16_t(w[j]);
        }
    }
};

template <bool VEC>
struct Eight<float, VEC> {
    uint32_t w[8];
    __device__ __forceinline__ void load(const float *p, int l, int left) {
        if (VEC) {
            uint4 a = make_uint4(0u, 0u, 0u, 0u), b = a;
            if (8 * l < left) {
                a = ld_stream_u4(p + 8 * l);
                b = ld_stream_u4(p + 8 * l + 4);
            }
            w[0] = a.x;
            w[1] = a.y;
            w[2] = a.z;
            w[3] = a.w;
            w[4] = b.x;
            w[5] = b.y;
            w[6] = b.z;
            w[7] = b.w;
        } else if (left >= kBlock8) {
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(p[l + 16 * j]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = l + 16 * j < left ? __float_as_uint(p[l + 16 * j]) : 0u;
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = 0u;
    }
    __device__ __forceinline__ float at(int j) const { return __uint_as_float(w[j]); }
    __device__ __forceinline__ uint32_t mag() const {
        uint32_t m = w[0] & 0x7FFFFFFFu;
#pragma unroll
        for (int j = 1; j < 8; ++j) m = max(m, w[j] & 0x7FFFFFFFu);
        return m;
    }
    __device__ __forceinline__ void set(const float (&x)[8]) {
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(x[j]);
    }
    __device__ __forceinline__ void store(float *p, int l, int left) const {
        if (VEC) {
            if (8 * l < left) {
                st_stream_u4(p + 8 * l, make_uint4(w[0], w[1], w[2], w[3]));
                st_stream_u4(p + 8 * l + 4, make_uint4(w[4], w[5], w[6], w[7]));
            }
        } else if (left >= kBlock8) {
#pragma unroll
            for (int j = 0; j < 8; ++j) p[l + 16 * j] = __uint_as_float(w[j]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (l + 16 * j < left) p[l + 16 * j] = __uint_as_float(w[j]);
        }
    }
};

// The maximum over the 16 lanes of a block.
__device__ __forceinline__ uint32_t block_max(uint32_t m) {
#pragma unroll
    for (int o = 8; o > 0; o /= 2) m = max(m, __shfl_xor_sync(kFull, m, o));
    return m;
}

// Codes of the block's rows at `q`, whose rows go on to the next multiple of 16
// (`left` is of the row's columns; the codes past them are written as 0).
template <bool VEC>
__device__ __forceinline__ void store_codes(uint8_t *q, uint2 codes, int l, int left) {
    const int end = (left + 15) & ~15;
    if (VEC) {
        if (8 * l < end) *reinterpret_cast<uint2 *>(q + 8 * l) = codes;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (l + 16 * j < end) q[l + 16 * j] = uint8_t((j < 4 ? codes.x : codes.y) >> (8 * (j & 3)));
    }
}

template <bool VEC>
__device__ __forceinline__ uint2 load_codes(const uint8_t *q, int l, int left) {
    uint2 codes = make_uint2(0u, 0u);
    if (VEC) {
        if (8 * l < left) codes = ld_stream_u2(q + 8 * l);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (l + 16 * j < left) codes.x |= uint32_t(q[l + 16 * j]) << (8 * j);
            if (l + 64 + 16 * j < left) codes.y |= uint32_t(q[l + 64 + 16 * j]) << (8 * j);
        }
    }
    return codes;
}

}  // namespace wc
