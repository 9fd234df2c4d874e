// fp8_dequant.cu -- a matrix kept in 8 bits (e4m3, one fp32 scale per 128 of a
// row, or per 128 x 128) back to its values: out[r][c] = code * scale, rounded
// once to the output's type.
//
// Bound: HBM (1 byte read, 2 or 4 written per value).  16 lanes have a block of
// 128 (wc_eight.cuh), four blocks of a row in flight per thread.
#include "wc_eight.cuh"
#include "wc_internal.h"

namespace wc {

namespace {

constexpr int kThreads = 256;
constexpr int kRows = kThreads / 16;
constexpr int kAcross = 4;

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) fp8_dequant_kernel(const Fp8Dequant a, int32_t across, int shift) {
    const int64_t down = int64_t(blockIdx.x) / across;
    const int32_t block = int32_t(int64_t(blockIdx.x) - down * across) * kAcross;
    const int64_t row = down * kRows + (threadIdx.x >> 4), col = int64_t(block) * kBlock8;
    const int l = threadIdx.x & 15;
    if (row >= a.rows) return;
    const int left = int(min(a.cols - col, int64_t(kAcross * kBlock8)));
    const uint8_t *q = a.q + row * a.ld_q + col;
    const float *s = a.s + block * a.ld_s + (row >> shift);
    T *out = static_cast<T *>(a.out) + row * a.ld_out + col;
    uint2 codes[kAcross];
    float scale[kAcross];
#pragma unroll
    for (int k = 0; k < kAcross; ++k) {
        const int rest = left - k * kBlock8;
        codes[k] = load_codes<VEC>(q + k * kBlock8, l, rest);
        scale[k] = rest > 0 ? s[k * a.ld_s] : 0.0f;
    }
#pragma unroll
    for (int k = 0; k < kAcross; ++k) {
        float x[8];
        values_of(codes[k], scale[k], x);
        Eight<T, VEC> v;
        v.set(x);
        v.store(out + k * kBlock8, l, left - k * kBlock8);
    }
}

template <typename T>
void launch(const Fp8Dequant &a, cudaStream_t stream) {
    const int32_t across = int32_t((a.cols + kAcross * kBlock8 - 1) / (kAcross * kBlock8));
    const uint32_t grid = uint32_t((a.rows + kRows - 1) / kRows * across);
    const int shift = a.rows_per_scale == 1 ? 0 : 7;
    const bool vec = a.cols % 8 == 0 && reinterpret_cast<uintptr_t>(a.out) % 16 == 0 &&
                     a.ld_out % (16 / int(sizeof(T))) == 0;
    if (vec) fp8_dequant_kernel<T, true><<<grid, kThreads, 0, stream>>>(a, across, shift);
    else fp8_dequant_kernel<T, false><<<grid, kThreads, 0, stream>>>(a, across, shift);
}

}  // namespace

cudaError_t launch_fp8_dequant(const Fp8Dequant &a, cudaStream_t stream) {
    if (a.out_bf16) launch<uint16_t>(a, stream);
    else launch<float>(a, stream);
    return cudaPeekAtLastError();
}

}  // namespace wc
