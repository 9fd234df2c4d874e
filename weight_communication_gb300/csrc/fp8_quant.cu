// fp8_quant.cu -- quantization to 8-bit floating point (e4m3) with one fp32
// scale per block of 128 values along the axis that a product sums over.
//
// The rule is in wc_fp8.cuh.  NaN as the scale of a block with a value that is
// not finite makes every sum it enters NaN, as the unquantized product would be.
//
// One CTA per tile of 128 x 128 reads it once and can write both layouts a
// training step needs: the rows' codes (blocks along the columns) and the
// columns' codes (blocks along the rows, stored transposed).  Square blocks,
// for weights, share one scale between the two layouts.  Thread (g, l) holds
// rows 8g..8g+7 and columns 8l..8l+7, bf16 values two to a word, and takes
// maxima of encodings two at a time.  The 16 lanes of a row group reduce
// their 8 rows together (each exchange halves the rows a lane still carries),
// so that a lane divides for one row and not for eight; the columns' scales
// are likewise formed once each, by 128 threads.  The transposed codes go
// through shared memory as 8-byte words of a column's 8 consecutive rows.
// Rows that start anywhere are read in aligned chunks and shifted: 4411 x 9433
// bf16 both ways 49 -> 40 us against value by value.
// Bound: HBM (2 bytes read and 1 or 2 written per value).
#include "wc_device.cuh"
#include "wc_fp8.cuh"
#include "wc_internal.h"
#include "wc_launch.cuh"
#include "wc_rows.cuh"

namespace wc {

namespace {

constexpr int kTile = 128;
constexpr int kThreads = 256;

// The 8 x 8 values of a thread, and the operations on them that depend on the
// type.  An encoding without its sign orders magnitudes, infinities and NaN
// above all finite ones; Max holds such encodings (bf16: of two columns).
template <typename T>
struct Values;

template <>
struct Values<uint16_t> {
    static constexpr int kMaxes = 4;  // words of a row's 8 maxima
    uint32_t w[8][4];
    __device__ __forceinline__ void load(int i, const uint16_t *p) {
        const uint4 q = ld_stream_u4(p);
        w[i][0] = q.x;
        w[i][1] = q.y;
        w[i][2] = q.z;
        w[i][3] = q.w;
    }
    static constexpr int kWords = 8;  // of the chunks of a row
    __device__ __forceinline__ void shift(int i, const uint16_t *p, uint32_t (&t)[kWords]) {
        shift_words(p, t, w[i]);
    }
    __device__ __forceinline__ void load_edge(int i, const uint16_t *p, int64_t left) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t lo = 2 * k < left ? p[2 * k] : 0u;
            const uint32_t hi = 2 * k + 1 < left ? p[2 * k + 1] : 0u;
            w[i][k] = lo | (hi << 16);
        }
    }
    __device__ __forceinline__ float at(int i, int j) const {
        return __uint_as_float((j & 1) ? (w[i][j / 2] & 0xFFFF0000u) : (w[i][j / 2] << 16));
    }
    __device__ __forceinline__ uint32_t mag(int i, int k) const { return w[i][k] & 0x7FFF7FFFu; }
    static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return __vmaxu2(a, b); }
    // the largest of a word's two, as a binary32 encoding
    static __device__ __forceinline__ uint32_t single(uint32_t m) { return max(m << 16, m & 0xFFFF0000u); }
    // column j of a row's maxima, as a binary32 encoding
    static __device__ __forceinline__ uint32_t column(const uint32_t *m, int j) {
        return uint32_t(reinterpret_cast<const uint16_t *>(m)[j]) << 16;
    }
};

template <>
struct Values<float> {
    static constexpr int kMaxes = 8;
    uint32_t w[8][8];
    __device__ __forceinline__ void load(int i, const float *p) {
        const uint4 a = ld_stream_u4(p), b = ld_stream_u4(p + 4);
        w[i][0] = a.x;
        w[i][1] = a.y;
        w[i][2] = a.z;
        w[i][3] = a.w;
        w[i][4] = b.x;
        w[i][5] = b.y;
        w[i][6] = b.z;
        w[i][7] = b.w;
    }
    static constexpr int kWords = 12;
    __device__ __forceinline__ void shift(int i, const float *p, uint32_t (&t)[kWords]) {
        drop_words(t, (uint32_t(reinterpret_cast<uintptr_t>(p)) & 15u) >> 2);
#pragma unroll
        for (int k = 0; k < 8; ++k) w[i][k] = t[k];
    }
    __device__ __forceinline__ void load_edge(int i, const float *p, int64_t left) {
#pragma unroll
        for (int k = 0; k < 8; ++k) w[i][k] = k < left ? __float_as_uint(p[k]) : 0u;
    }
    __device__ __forceinline__ float at(int i, int j) const { return __uint_as_float(w[i][j]); }
    __device__ __forceinline__ uint32_t mag(int i, int k) const { return w[i][k] & 0x7FFFFFFFu; }
    static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return max(a, b); }
    static __device__ __forceinline__ uint32_t single(uint32_t m) { return m; }
    static __device__ __forceinline__ uint32_t column(const uint32_t *m, int j) { return m[j]; }
};

// Shared transposed codes: column c's 128 rows as 16 words of 8 bytes, word w
// at slot w ^ (c / 8 % 16), so that the 16 lanes of a store hit all banks.
__device__ __forceinline__ int slot_of(int c, int w) { return c * 16 + (w ^ ((c >> 3) & 15)); }

template <typename T, bool VEC, bool ROWS, bool COLS, bool SQUARE>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 3 : 2)
fp8_quant_kernel(const Fp8Quant a) {
    using V = Values<T>;
    __shared__ uint2 turned[COLS ? kTile * 16 : 1];
    __shared__ uint32_t col_max[COLS && !SQUARE ? kThreads / 32 : 1][COLS && !SQUARE ? 16 * V::kMaxes : 1];
    __shared__ __align__(16) float col_inv[COLS && !SQUARE ? kTile : 1];
    __shared__ uint32_t tile_max[kThreads / 32];
    const int l = threadIdx.x & 15, g = threadIdx.x >> 4;  // column group, row group
    const int warp = threadIdx.x >> 5;
    const int64_t r0 = int64_t(blockIdx.y) * kTile, c0 = int64_t(blockIdx.x) * kTile;
    const int64_t c = c0 + 8 * l;

    // the product that follows may set itself up; it waits for this kernel's end
    let_successor_start();
    V v;
    constexpr int kShifted = sizeof(T) == 2 ? 4 : 2;  // rows in flight
    const T *x = static_cast<const T *>(a.x) + (r0 + 8 * g) * a.ld + c;
    // (whole chunks are read only where they end inside the matrix)
    const T *const end = static_cast<const T *>(a.x) + (a.rows - 1) * a.ld + a.cols;
    if (!VEC && r0 + 8 * g + 7 < a.rows && a.cols - c >= 8 && end - (x + 7 * a.ld) >= 8 + 16 / int(sizeof(T))) {
#pragma unroll
        for (int i0 = 0; i0 < 8; i0 += kShifted) {
            uint32_t t[kShifted][V::kWords];
#pragma unroll
            for (int i = 0; i < kShifted; ++i) load_chunks(x + (i0 + i) * a.ld, t[i]);
#pragma unroll
            for (int i = 0; i < kShifted; ++i) v.shift(i0 + i, x + (i0 + i) * a.ld, t[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t left = r0 + 8 * g + i < a.rows ? a.cols - c : 0;
            if (VEC && left >= 8) v.load(i, x + i * a.ld);
            else v.load_edge(i, x + i * a.ld, left);
        }
    }

    Scale8 square = {0.0f, 0.0f};
    if (SQUARE) {
        uint32_t m = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int k = 0; k < V::kMaxes; ++k) m = V::larger(m, v.mag(i, k));
        m = __reduce_max_sync(kFull, V::single(m));
        if ((threadIdx.x & 31) == 0) tile_max[warp] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) m = max(m, tile_max[w]);
        square = scale_of(__uint_as_float(m));
        if (threadIdx.x == 0) {
            if (ROWS) a.s[int64_t(blockIdx.x) * a.ld_s + blockIdx.y] = square.scale;
            if (COLS) a.st[int64_t(blockIdx.y) * a.ld_st + blockIdx.x] = square.scale;
        }
    }
    if (COLS && !SQUARE) {  // the columns' maxima over this warp's 16 rows
#pragma unroll
        for (int k = 0; k < V::kMaxes; ++k) {
            uint32_t m = v.mag(0, k);
#pragma unroll
            for (int i = 1; i < 8; ++i) m = V::larger(m, v.mag(i, k));
            m = V::larger(m, __shfl_xor_sync(kFull, m, 16));
            if ((threadIdx.x & 16) == 0) col_max[warp][V::kMaxes * l + k] = m;
        }
    }

    if (ROWS) {
        Scale8 own = square;
        if (!SQUARE) {
            uint32_t m[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                uint32_t n = v.mag(i, 0);
#pragma unroll
                for (int k = 1; k < V::kMaxes; ++k) n = V::larger(n, v.mag(i, k));
                m[i] = V::single(n);
            }
            // lane l ends with the maximum of row l / 2
#pragma unroll
            for (int half = 4; half > 0; half /= 2) {
                const bool upper = (l & (2 * half)) != 0;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (k >= half) continue;
                    const uint32_t give = upper ? m[k] : m[k + half];
                    const uint32_t keep = upper ? m[k + half] : m[k];
                    m[k] = max(keep, __shfl_xor_sync(kFull, give, 2 * half));
                }
            }
            m[0] = max(m[0], __shfl_xor_sync(kFull, m[0], 1));
            own = scale_of(__uint_as_float(m[0]));
            const int64_t r = r0 + 8 * g + l / 2;
            if ((l & 1) == 0 && r < a.rows) a.s[int64_t(blockIdx.x) * a.ld_s + r] = own.scale;
        }
        // a row's padding up to a multiple of 16 bytes is written too, as
        // zeros; ld_q is such a multiple, so the 8 bytes fit
        const bool inside = c < (a.cols + 15) / 16 * 16;
        uint8_t *q = a.q + (r0 + 8 * g) * a.ld_q + c;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float inv = SQUARE ? own.inv : __shfl_sync(kFull, own.inv, 2 * i, 16);
            float t[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) t[j] = v.at(i, j);
            const uint2 w = codes_of(t, inv);
            if (inside && r0 + 8 * g + i < a.rows) *reinterpret_cast<uint2 *>(q + i * a.ld_q) = w;
        }
    }

    if (COLS) {
        if (!SQUARE) {
            __syncthreads();
            if (threadIdx.x < kTile) {
                uint32_t m = V::column(col_max[0], threadIdx.x);
#pragma unroll
                for (int w = 1; w < kThreads / 32; ++w) m = max(m, V::column(col_max[w], threadIdx.x));
                const Scale8 s = scale_of(__uint_as_float(m));
                col_inv[threadIdx.x] = s.inv;
                if (c0 + threadIdx.x < a.cols) a.st[int64_t(blockIdx.y) * a.ld_st + c0 + threadIdx.x] = s.scale;
            }
            __syncthreads();
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float t[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) t[i] = v.at(i, j);
            turned[slot_of(8 * l + j, g)] = codes_of(t, SQUARE ? square.inv : col_inv[SQUARE ? 0 : 8 * l + j]);
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

template <typename T, bool VEC, bool SQUARE>
void launch(const Fp8Quant &a, cudaStream_t stream) {
    const dim3 grid(uint32_t((a.cols + kTile - 1) / kTile), uint32_t((a.rows + kTile - 1) / kTile));
    if (a.q && a.qt) fp8_quant_kernel<T, VEC, true, true, SQUARE><<<grid, kThreads, 0, stream>>>(a);
    else if (a.q) fp8_quant_kernel<T, VEC, true, false, SQUARE><<<grid, kThreads, 0, stream>>>(a);
    else fp8_quant_kernel<T, VEC, false, true, SQUARE><<<grid, kThreads, 0, stream>>>(a);
}

template <typename T>
void launch(const Fp8Quant &a, cudaStream_t stream) {
    const bool vec = a.ld % (16 / sizeof(T)) == 0;  // rows start on 16 bytes
    if (vec && a.square) launch<T, true, true>(a, stream);
    else if (vec) launch<T, true, false>(a, stream);
    else if (a.square) launch<T, false, true>(a, stream);
    else launch<T, false, false>(a, stream);
}

}  // namespace

cudaError_t launch_fp8_quant(const Fp8Quant &a, cudaStream_t stream) {
    if (a.x_bf16) launch<uint16_t>(a, stream);
    else launch<float>(a, stream);
    return cudaPeekAtLastError();
}

}  // namespace wc
