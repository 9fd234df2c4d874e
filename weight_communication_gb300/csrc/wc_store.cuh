// wc_store.cuh -- a warp's 32 rows of sums from shared memory to rows of a matrix
// that may start on any element.
#pragma once

#include <stdint.h>

#include "wc_device.cuh"

namespace wc {

// Epilogue staging of a warp: 64 bytes (32 bf16 or 16 fp32 columns) of each of
// its 32 rows.  80 bytes from row to row keep 16-byte accesses off one
// another's banks.
constexpr int kStagingPitch = 80;
constexpr int kStagingBytes = 32 * kStagingPitch;

// 32 rows x 32 columns of staged bf16 values to rows that start on any element:
// two rows of 16 lanes at a time, aligned words of two columns, then the columns
// that are half of a word at a row's ends.  Several rows are read before they are
// stored, so that they share one latency (a value per lane and a row at a time:
// 4411 x 9433 x 638 69 us, so 55).
__device__ __forceinline__ void store_pass_bf16(char *base, int64_t ld_out, const uint8_t *staging, int rows, int cols,
                                                int lane) {
    constexpr int U = 8;
    const int half = lane >> 4, h = lane & 15;
    const uint32_t odd0 = uint32_t(reinterpret_cast<uintptr_t>(base) >> 1) & 1u, odd_ld = uint32_t(ld_out) & 1u;
    const uint32_t odd = odd0 ^ (uint32_t(half) & odd_ld);  // of all this lane's rows
    const uint32_t shift = odd * 16;
    const uint8_t *from = staging + half * kStagingPitch + 4 * h;
    char *to = base + (int64_t(half) * ld_out + 2 * h + odd) * 2;
    const int64_t step = 4 * ld_out;
    const bool word = int(2 * h + odd + 1) < cols;
#pragma unroll 1
    for (int r = half; r < 32; r += 2 * U) {
        uint32_t w[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const uint32_t *p = reinterpret_cast<const uint32_t *>(from + 2 * k * kStagingPitch);
            w[k] = __funnelshift_r(p[0], p[1], shift);
        }
        from += 2 * U * kStagingPitch;
#pragma unroll
        for (int k = 0; k < U; ++k) {
            if (word && r + 2 * k < rows) *reinterpret_cast<uint32_t *>(to) = w[k];
            to += step;
        }
    }
    const int odd_row = int(odd0 ^ (uint32_t(lane) & odd_ld));
    uint16_t *row = reinterpret_cast<uint16_t *>(base) + int64_t(lane) * ld_out;
    const uint16_t *of = reinterpret_cast<const uint16_t *>(staging + lane * kStagingPitch);
    if (lane < rows && odd_row) row[0] = of[0];
    if (lane < rows && ((cols - odd_row) & 1) && cols > odd_row) row[cols - 1] = of[cols - 1];
}

// 32 rows x 16 columns of staged fp32 sums, stored or added to what out holds
// (added with several reads of out in flight: 8192 x 11008 x 4096 into fp32 438 us
// with one scale per 128 x 128, 584 with one per row; one by one 1890 and 1420).
template <bool ADD, typename T>
__device__ __forceinline__ void store_pass_f32(T *base, int64_t ld_out, const uint8_t *staging, int rows, int cols,
                                               int lane) {
    constexpr int U = 8;
    const int half = lane >> 4, h = lane & 15;
    if (h >= cols) return;
    const uint8_t *from = staging + half * kStagingPitch + 4 * h;
    T *to = base + int64_t(half) * ld_out + h;
    const int64_t step = 2 * ld_out;
#pragma unroll 1
    for (int r = half; r < 32; r += 2 * U) {
        float old[U];
        if (ADD) {
            const T *p = to;
#pragma unroll
            for (int k = 0; k < U; ++k) {
                old[k] = 0.0f;
                if (r + 2 * k < rows) {
                    if constexpr (sizeof(T) == 2) old[k] = bf16_bits_to_f32(*p);
                    else old[k] = *p;
                }
                p += step;
            }
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            float x = *reinterpret_cast<const float *>(from + 2 * k * kStagingPitch);
            if (ADD) x = __fadd_rn(old[k], x);
            if (r + 2 * k < rows) {
                if constexpr (sizeof(T) == 2) *to = f32_to_bf16_bits(x);
                else *to = x;
            }
            to += step;
        }
        from += 2 * U * kStagingPitch;
    }
}

}  // namespace wc
