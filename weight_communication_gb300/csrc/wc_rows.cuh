// wc_rows.cuh -- rows that start on any element: a run of values is read as the
// aligned chunks of 16 bytes that hold it, and shifted into place.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace wc {

// N words: the chunks from the one that holds *p.  A neighbour's thread reads
// some of them too.
template <int N>
__device__ __forceinline__ void load_chunks(const void *p, uint32_t (&t)[N]) {
    const uint4 *q = reinterpret_cast<const uint4 *>(reinterpret_cast<uintptr_t>(p) & ~uintptr_t(15));
#pragma unroll
    for (int k = 0; k < N / 4; ++k) {
        const uint4 v = __ldg(q + k);
        t[4 * k] = v.x;
        t[4 * k + 1] = v.y;
        t[4 * k + 2] = v.z;
        t[4 * k + 3] = v.w;
    }
}

// Drops the first n < 4 of N words.
template <int N>
__device__ __forceinline__ void drop_words(uint32_t (&t)[N], uint32_t n) {
#pragma unroll
    for (int k = 0; k + 2 < N; ++k) t[k] = (n & 2u) ? t[k + 2] : t[k];
#pragma unroll
    for (int k = 0; k + 1 < N; ++k) t[k] = (n & 1u) ? t[k + 1] : t[k];
}

// The first M words from *p (a 2-byte boundary) of the N > M words that
// load_chunks() gave.
template <int M, int N>
__device__ __forceinline__ void shift_words(const void *p, uint32_t (&t)[N], uint32_t (&out)[M]) {
    const uint32_t at = uint32_t(reinterpret_cast<uintptr_t>(p)) & 15u;
    drop_words(t, at >> 2);
#pragma unroll
    for (int k = 0; k < M; ++k) out[k] = __funnelshift_r(t[k], t[k + 1], (at & 2u) * 8u);
}

}  // namespace wc
