// fp8_quant.cu -- quantization to 8-bit floating point (e4m3) with one fp32
// scale per block of 128 values along the axis that a product sums over.
//
//   m = max |x| of the block
//   m < 448 * 2^-126 (the scale would not be normal): scale 0, codes 0
//   m infinite or not a number:                       scale NaN, codes 0
//   else scale = m / 448, code = e4m3(x * fl(448 / m)), to nearest, ties to even
//
// 448 is e4m3's largest value, so no code saturates.  NaN as the scale of a
// block with a value that is not finite makes every sum it enters NaN, as
// the unquantized product would be.
//
// One CTA per tile of 128 x 128 reads it once and can write both layouts a
// training step needs: the rows' codes (blocks along the columns) and the
// columns' codes (blocks along the rows, stored transposed).  Square blocks,
// for weights, share one scale between the two layouts.  Thread (g, l) holds
// rows 8g..8g+7 and columns 8l..8l+7: rows reduce over 16 lanes, columns over
// the threads' own 8 rows first; the transposed codes go through shared memory
// as 8-byte words of a column's 8 consecutive rows.
// Bound: HBM (2 bytes read and 1 or 2 written per value).
#include <cuda_fp8.h>

#include "wc_device.cuh"
#include "wc_internal.h"

namespace wc {

namespace {

constexpr int kTile = 128;
constexpr int kThreads = 256;
constexpr float kTop = 448.0f;

struct Scale8 {
    float scale, inv;
};

__device__ __forceinline__ Scale8 scale_of(float m) {
    Scale8 s;
    if (m < kTop * kMinNormal) {  // exact product
        s.scale = 0.0f;
        s.inv = 0.0f;
    } else if (m <= 3.40282346638528859812e38f) {
        s.scale = __fdiv_rn(m, kTop);
        s.inv = __fdiv_rn(kTop, m);
    } else {
        s.scale = __uint_as_float(0x7FC00000u);
        s.inv = 0.0f;
    }
    return s;
}

// Codes of 8 values in order, 0 where the block is not finite (inv = 0 times
// an infinity is not a number, so those are set, not computed).
__device__ __forceinline__ uint2 codes_of(const float x[8], const float inv[8]) {
    uint32_t h[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float a = inv[2 * j] == 0.0f ? 0.0f : __fmul_rn(x[2 * j], inv[2 * j]);
        const float b = inv[2 * j + 1] == 0.0f ? 0.0f : __fmul_rn(x[2 * j + 1], inv[2 * j + 1]);
        h[j] = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    }
    return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

// |x| with infinities and NaN ordered above every finite value, for a maximum
// over encodings.
__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// Shared transposed codes: column c's 128 rows as 16 words of 8 bytes, word w
// at slot w ^ (c / 8 % 16) so that the 16 lanes of a store hit 16 banks pairs.
__device__ __forceinline__ int slot_of(int c, int w) { return c * 16 + (w ^ ((c >> 3) & 15)); }

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads)
fp8_quant_kernel(const Fp8Quant a) {
    __shared__ uint2 turned[kTile * 16];
    __shared__ uint32_t col_max[kThreads / 32][kTile];
    __shared__ uint32_t tile_max[kThreads / 32];
    const int l = threadIdx.x & 15, g = threadIdx.x >> 4;  // column group, row group
    const int warp = threadIdx.x >> 5;
    const int64_t r0 = int64_t(blockIdx.y) * kTile, c0 = int64_t(blockIdx.x) * kTile;
    const int64_t c = c0 + 8 * l;
    const T *x = static_cast<const T *>(a.x);

    float v[8][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t r = r0 + 8 * g + i;
        if (VEC && r < a.rows && c + 8 <= a.cols) {
            const T *p = x + r * a.ld + c;
            if constexpr (sizeof(T) == 2) {
                const uint4 w = ld_stream_u4(p);
                const uint32_t h[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    v[i][2 * j] = __uint_as_float(h[j] << 16);
                    v[i][2 * j + 1] = __uint_as_float(h[j] & 0xFFFF0000u);
                }
            } else {
                const float4 w0 = ld_stream_f4(p), w1 = ld_stream_f4(p + 4);
                v[i][0] = w0.x;
                v[i][1] = w0.y;
                v[i][2] = w0.z;
                v[i][3] = w0.w;
                v[i][4] = w1.x;
                v[i][5] = w1.y;
                v[i][6] = w1.z;
                v[i][7] = w1.w;
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[i][j] = 0.0f;
                if (r < a.rows && c + j < a.cols) {
                    if constexpr (sizeof(T) == 2) v[i][j] = bf16_bits_to_f32(x[r * a.ld + c + j]);
                    else v[i][j] = x[r * a.ld + c + j];
                }
            }
        }
    }

    Scale8 square = {0.0f, 0.0f};
    if (a.square) {
        uint32_t m = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) m = max(m, magnitude(v[i][j]));
        m = __reduce_max_sync(kFull, m);
        if ((threadIdx.x & 31) == 0) tile_max[warp] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) m = max(m, tile_max[w]);
        square = scale_of(__uint_as_float(m));
        if (threadIdx.x == 0) {
            if (a.q) a.s[int64_t(blockIdx.x) * a.ld_s + blockIdx.y] = square.scale;
            if (a.qt) a.st[int64_t(blockIdx.y) * a.ld_st + blockIdx.x] = square.scale;
        }
    }

    if (a.q) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t r = r0 + 8 * g + i;
            Scale8 s = square;
            if (!a.square) {
                uint32_t m = 0u;
#pragma unroll
                for (int j = 0; j < 8; ++j) m = max(m, magnitude(v[i][j]));
#pragma unroll
                for (int off = 8; off > 0; off >>= 1) m = max(m, __shfl_xor_sync(kFull, m, off));
                s = scale_of(__uint_as_float(m));
                if (l == 0 && r < a.rows) a.s[int64_t(blockIdx.x) * a.ld_s + r] = s.scale;
            }
            float inv[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) inv[j] = s.inv;
            const uint2 w = codes_of(v[i], inv);
            // a row's padding up to a multiple of 16 bytes is written too, as
            // zeros; ld_q is such a multiple, so the 8 bytes fit
            if (r < a.rows && c < (a.cols + 15) / 16 * 16)
                *reinterpret_cast<uint2 *>(a.q + r * a.ld_q + c) = w;
        }
    }

    if (a.qt) {
        float inv[8];
        if (a.square) {
#pragma unroll
            for (int j = 0; j < 8; ++j) inv[j] = square.inv;
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                uint32_t m = 0u;
#pragma unroll
                for (int i = 0; i < 8; ++i) m = max(m, magnitude(v[i][j]));
                m = max(m, __shfl_xor_sync(kFull, m, 16));
                if ((threadIdx.x & 16) == 0) col_max[warp][8 * l + j] = m;
            }
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                uint32_t m = 0u;
#pragma unroll
                for (int w = 0; w < kThreads / 32; ++w) m = max(m, col_max[w][8 * l + j]);
                const Scale8 s = scale_of(__uint_as_float(m));
                inv[j] = s.inv;
                if (g == 0 && c + j < a.cols) a.st[int64_t(blockIdx.y) * a.ld_st + c + j] = s.scale;
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float t[8], in[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                t[i] = v[i][j];
                in[i] = inv[j];
            }
            turned[slot_of(8 * l + j, g)] = codes_of(t, in);
        }
        __syncthreads();
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            const int cc = p * 16 + g;  // column of the tile; l is its word
            const int64_t r = r0 + 8 * l;
            if (c0 + cc < a.cols && r < (a.rows + 15) / 16 * 16)
                *reinterpret_cast<uint2 *>(a.qt + (c0 + cc) * a.ld_qt + r) = turned[slot_of(cc, l)];
        }
    }
}

}  // namespace

cudaError_t launch_fp8_quant(const Fp8Quant &a, cudaStream_t stream) {
    const dim3 grid(uint32_t((a.cols + kTile - 1) / kTile), uint32_t((a.rows + kTile - 1) / kTile));
    if (a.x_bf16) {
        if (a.ld % 8 == 0) fp8_quant_kernel<uint16_t, true><<<grid, kThreads, 0, stream>>>(a);
        else fp8_quant_kernel<uint16_t, false><<<grid, kThreads, 0, stream>>>(a);
    } else {
        if (a.ld % 4 == 0) fp8_quant_kernel<float, true><<<grid, kThreads, 0, stream>>>(a);
        else fp8_quant_kernel<float, false><<<grid, kThreads, 0, stream>>>(a);
    }
    return cudaPeekAtLastError();
}

}  // namespace wc
