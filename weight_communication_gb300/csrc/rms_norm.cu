// rms_norm.cu -- root-mean-square norm of a residual stream, whose input is kept
// in 8 bits (e4m3, one fp32 scale per 128 of a row) for the backward pass.
//
//   t = x + add (rounded to the type; or t = x),  r = 1 / sqrt(mean of t^2 + eps)
//   y = t * r * w
//   kept: codes and scales of t, and r (fp32)
//   n = t^ * r, with t^ what the codes stand for
//   dx = r * (dy * w - n * mean of (dy * w * n)) (+ what reaches t past the norm)
//   dw = sum over the rows of dy * n
//
// A row is read once: a group of threads holds all of it in registers, two
// pieces of 8 values each (wc_eight.cuh), sums its squares, and writes.
//
// The weight's gradient is summed over rows in registers: a group has the same
// columns in every row it works on.  Each group leaves its sums, which a second
// launch adds in a fixed order.
//
// Bound: HBM.
#include <type_traits>

#include "wc_eight.cuh"
#include "wc_internal.h"
#include "wc_launch.cuh"

namespace wc {

namespace {

constexpr int kSms = 152;

// Threads of a row and pieces of 8 values of each; rows of a CTA.
template <int TPR, int PIECES>
struct Shape {
    static constexpr int kThreads = TPR < 256 ? 256 : TPR;
    static constexpr int kRows = kThreads / TPR;
    static constexpr int kWarps = TPR / 32;  // of a row
    static constexpr int64_t kCols = int64_t(TPR) * PIECES * 8;  // at most
};

// Sum over a row's threads, the same bits in each.  `slots`: one per warp of the CTA,
// not in use by an earlier sum (two sets taken in turn see to that).
template <int WARPS>
__device__ __forceinline__ float row_sum(float x, float *slots) {
#pragma unroll
    for (int o = 16; o > 0; o /= 2) x = __fadd_rn(x, __shfl_xor_sync(kFull, x, o));
    if (WARPS == 1) return x;
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) slots[warp] = x;
    __syncthreads();
    const float *row = slots + warp / WARPS * WARPS;
    x = row[0];
#pragma unroll
    for (int w = 1; w < WARPS; ++w) x = __fadd_rn(x, row[w]);
    return x;
}

__device__ __forceinline__ float weight_at(const void *w, bool bf16, int64_t c) {
    return bf16 ? bf16_bits_to_f32(static_cast<const uint16_t *>(w)[c]) : static_cast<const float *>(w)[c];
}

// The weight's values of one piece (`left` columns from the block's start).
template <bool VEC>
__device__ __forceinline__ void weights(const void *w, bool bf16, int64_t c0, int l, int left, float (&x)[8]) {
    if (VEC && bf16) {
        uint4 q = make_uint4(0u, 0u, 0u, 0u);
        if (8 * l < left) q = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(w) + c0 + 8 * l));
        const uint32_t t[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int j = 0; j < 8; ++j)
            x[j] = __uint_as_float((j & 1) ? (t[j / 2] & 0xFFFF0000u) : (t[j / 2] << 16));
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = column_of<VEC>(l, j);
            x[j] = c < left ? weight_at(w, bf16, c0 + c) : 0.0f;
        }
    }
}

template <typename T, bool VEC, int TPR, int PIECES>
__global__ void __launch_bounds__(Shape<TPR, PIECES>::kThreads) rms_norm_kernel(const RmsNorm a) {
    using S = Shape<TPR, PIECES>;
    __shared__ float slots[S::kThreads / 32];
    const int in_row = threadIdx.x % TPR, l = in_row & 15;
    const int64_t row = int64_t(blockIdx.x) * S::kRows + threadIdx.x / TPR;
    const bool live = row < a.rows;
    const int cols = int(a.cols);
    int col[PIECES], left[PIECES];  // of the piece's block
    Eight<T> t[PIECES];
#pragma unroll
    for (int p = 0; p < PIECES; ++p) {
        col[p] = (p * TPR + in_row) / 16 * kBlock8;
        left[p] = live ? cols - col[p] : 0;
        t[p].template load<VEC>(static_cast<const T *>(a.x) + row * a.ld_x + col[p], l, left[p]);
    }
    if (a.add) {
        Eight<T> o[PIECES];
#pragma unroll
        for (int p = 0; p < PIECES; ++p)
            o[p].template load<VEC>(static_cast<const T *>(a.add) + row * a.ld_add + col[p], l, left[p]);
#pragma unroll
        for (int p = 0; p < PIECES; ++p) {
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = __fadd_rn(t[p].at(j), o[p].at(j));
            t[p].set(x);
            t[p].template store<VEC>(static_cast<T *>(a.total) + row * a.ld_total + col[p], l, left[p]);
        }
    }
    float sum = 0.0f;
#pragma unroll
    for (int p = 0; p < PIECES; ++p)
#pragma unroll
        for (int j = 0; j < 8; ++j) sum = __fmaf_rn(t[p].at(j), t[p].at(j), sum);
    sum = row_sum<S::kWarps>(sum, slots);
    const float r = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(sum, float(cols)), a.eps)));
#pragma unroll
    for (int p = 0; p < PIECES; ++p) {
        float w[8], x[8];
        weights<VEC>(a.weight, a.weight_bf16, col[p], l, left[p], w);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = __fmul_rn(__fmul_rn(t[p].at(j), r), w[j]);
        Eight<T> out;
        out.set(x);
        out.template store<VEC>(static_cast<T *>(a.y) + row * a.ld_y + col[p], l, left[p]);
    }
    if (a.kept.q == nullptr) return;
    if (in_row == 0 && live) a.rstd[row] = r;
#pragma unroll
    for (int p = 0; p < PIECES; ++p) {
        const Scale8 s = scale_of(__uint_as_float(block_max(t[p].mag())));
        if (l == 0 && left[p] > 0) a.kept.s[col[p] / kBlock8 * a.kept.ld_s + row] = s.scale;
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = t[p].at(j);
        store_codes<VEC>(a.kept.q + row * a.kept.ld_q + col[p], codes_of(x, s.inv), l, left[p]);
    }
}

// Row groups of the gradient's grid: what the GPU runs at once, and no more than rows.
template <typename S>
int64_t groups_of(int64_t rows) {
    const int64_t most = int64_t(kSms) * (1024 / S::kThreads) * S::kRows;
    const int64_t ctas = ((rows < most ? rows : most) + S::kRows - 1) / S::kRows;
    return ctas * S::kRows;
}

template <typename T, bool VEC, int TPR, int PIECES>
__global__ void __launch_bounds__(Shape<TPR, PIECES>::kThreads) rms_norm_grad_kernel(const RmsNormGrad a) {
    using S = Shape<TPR, PIECES>;
    __shared__ float slots[2][S::kThreads / 32];
    const int in_row = threadIdx.x % TPR, l = in_row & 15;
    const int64_t group = int64_t(blockIdx.x) * S::kRows + threadIdx.x / TPR;
    const int64_t groups = int64_t(gridDim.x) * S::kRows;
    const int cols = int(a.cols);
    const float each = __fdiv_rn(1.0f, float(cols));
    float dw[PIECES][8];
#pragma unroll
    for (int p = 0; p < PIECES; ++p)
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[p][j] = 0.0f;
    // every group of a CTA takes as many turns, for the CTA's barriers
    const int64_t turns = (a.rows - int64_t(blockIdx.x) * S::kRows + groups - 1) / groups;
    int64_t row = group;
    for (int64_t i = 0; i < turns; ++i, row += groups) {
        const bool live = row < a.rows;
        const float r = live ? a.rstd[row] : 0.0f;
        Eight<T> dy[PIECES];
        uint2 codes[PIECES];
        float scale[PIECES], n[PIECES][8];
#pragma unroll
        for (int p = 0; p < PIECES; ++p) {
            const int col = (p * TPR + in_row) / 16 * kBlock8, left = live ? cols - col : 0;
            dy[p].template load<VEC>(static_cast<const T *>(a.dy) + row * a.ld_dy + col, l, left);
            codes[p] = load_codes<VEC>(a.kept.q + row * a.kept.ld_q + col, l, left);
            scale[p] = left > 0 ? a.kept.s[col / kBlock8 * a.kept.ld_s + row] : 0.0f;
        }
        float sum = 0.0f;
#pragma unroll
        for (int p = 0; p < PIECES; ++p) {
            const int col = (p * TPR + in_row) / 16 * kBlock8;
            float w[8];
            weights<VEC>(a.weight, a.weight_bf16, col, l, cols - col, w);
            values_of(codes[p], scale[p], n[p]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                n[p][j] = __fmul_rn(n[p][j], r);
                sum = __fmaf_rn(__fmul_rn(dy[p].at(j), w[j]), n[p][j], sum);
                dw[p][j] = __fmaf_rn(dy[p].at(j), n[p][j], dw[p][j]);
            }
        }
        const float mean = __fmul_rn(row_sum<S::kWarps>(sum, slots[i & 1]), each);
#pragma unroll
        for (int p = 0; p < PIECES; ++p) {
            const int col = (p * TPR + in_row) / 16 * kBlock8, left = live ? cols - col : 0;
            float w[8], x[8];
            weights<VEC>(a.weight, a.weight_bf16, col, l, cols - col, w);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                x[j] = __fmul_rn(r, __fmaf_rn(-n[p][j], mean, __fmul_rn(dy[p].at(j), w[j])));
            if (a.add) {
                Eight<T> o;
                o.template load<VEC>(static_cast<const T *>(a.add) + row * a.ld_add + col, l, left);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = __fadd_rn(x[j], o.at(j));
            }
            Eight<T> out;
            out.set(x);
            out.template store<VEC>(static_cast<T *>(a.dx) + row * a.ld_dx + col, l, left);
        }
    }
#pragma unroll
    for (int p = 0; p < PIECES; ++p) {
        const int col = (p * TPR + in_row) / 16 * kBlock8;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = col + column_of<VEC>(l, j);
            if (c < cols) a.partials[group * cols + c] = dw[p][j];
        }
    }
    let_successor_start();
}

// dweight = sum of the groups' partials: 32 columns by 32 warps of a CTA, each
// warp every 32nd group, then the warps in turn.
__global__ void __launch_bounds__(1024) dweight_kernel(const float *partials, int64_t groups, int cols,
                                                       void *dweight, int bf16, int accumulate) {
    __shared__ float sums[32][33];
    wait_for_predecessor();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float x = 0.0f;
    if (c < cols)
#pragma unroll 4
        for (int64_t g = warp; g < groups; g += 32) x = __fadd_rn(x, partials[g * cols + c]);
    sums[warp][lane] = x;
    __syncthreads();
    // warp w has column w
    x = sums[lane][warp];
#pragma unroll
    for (int o = 16; o > 0; o /= 2) x = __fadd_rn(x, __shfl_xor_sync(kFull, x, o));
    const int at = blockIdx.x * 32 + warp;
    if (lane != 0 || at >= cols) return;
    if (bf16) {
        uint16_t *p = static_cast<uint16_t *>(dweight) + at;
        if (accumulate) x = __fadd_rn(bf16_bits_to_f32(*p), x);
        *p = f32_to_bf16_bits(x);
    } else {
        float *p = static_cast<float *>(dweight) + at;
        if (accumulate) x = __fadd_rn(*p, x);
        *p = x;
    }
}

// Calls f with the shape of rows of `cols` columns.
template <typename F>
auto with_shape(int64_t cols, F f) {
    if (cols <= Shape<32, 1>::kCols) return f(Shape<32, 1>(), std::integral_constant<int, 32>(), std::integral_constant<int, 1>());
    if (cols <= Shape<32, 2>::kCols) return f(Shape<32, 2>(), std::integral_constant<int, 32>(), std::integral_constant<int, 2>());
    if (cols <= Shape<64, 2>::kCols) return f(Shape<64, 2>(), std::integral_constant<int, 64>(), std::integral_constant<int, 2>());
    if (cols <= Shape<128, 2>::kCols) return f(Shape<128, 2>(), std::integral_constant<int, 128>(), std::integral_constant<int, 2>());
    if (cols <= Shape<256, 2>::kCols) return f(Shape<256, 2>(), std::integral_constant<int, 256>(), std::integral_constant<int, 2>());
    if (cols <= Shape<512, 2>::kCols) return f(Shape<512, 2>(), std::integral_constant<int, 512>(), std::integral_constant<int, 2>());
    static_assert(Shape<1024, 2>::kCols == kNormCols, "the largest shape has the longest row");
    return f(Shape<1024, 2>(), std::integral_constant<int, 1024>(), std::integral_constant<int, 2>());
}

bool vector_rows(const void *p, int64_t ld, bool bf16) {
    return p == nullptr || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % (bf16 ? 8 : 4) == 0);
}

template <typename T, bool VEC>
void launch(const RmsNorm &a, cudaStream_t stream) {
    with_shape(a.cols, [&](auto shape, auto tpr, auto pieces) {
        using S = decltype(shape);
        rms_norm_kernel<T, VEC, decltype(tpr)::value, decltype(pieces)::value>
            <<<uint32_t((a.rows + S::kRows - 1) / S::kRows), S::kThreads, 0, stream>>>(a);
        return 0;
    });
}

template <typename T, bool VEC>
void launch(const RmsNormGrad &a, cudaStream_t stream) {
    with_shape(a.cols, [&](auto shape, auto tpr, auto pieces) {
        using S = decltype(shape);
        rms_norm_grad_kernel<T, VEC, decltype(tpr)::value, decltype(pieces)::value>
            <<<uint32_t(groups_of<S>(a.rows) / S::kRows), S::kThreads, 0, stream>>>(a);
        return 0;
    });
}

}  // namespace

cudaError_t launch_rms_norm(const RmsNorm &a, cudaStream_t stream) {
    const bool vec = a.cols % 8 == 0 && vector_rows(a.x, a.ld_x, a.bf16) && vector_rows(a.add, a.ld_add, a.bf16) &&
                     vector_rows(a.y, a.ld_y, a.bf16) && (!a.add || vector_rows(a.total, a.ld_total, a.bf16)) &&
                     vector_rows(a.weight, 0, a.weight_bf16);
    if (a.bf16 && vec) launch<uint16_t, true>(a, stream);
    else if (a.bf16) launch<uint16_t, false>(a, stream);
    else if (vec) launch<float, true>(a, stream);
    else launch<float, false>(a, stream);
    return cudaPeekAtLastError();
}

int64_t rms_norm_grad_partials(int64_t rows, int64_t cols) {
    return cols * with_shape(cols, [&](auto shape, auto, auto) { return groups_of<decltype(shape)>(rows); });
}

cudaError_t launch_rms_norm_grad(const RmsNormGrad &a, cudaStream_t stream) {
    const bool vec = a.cols % 8 == 0 && vector_rows(a.dy, a.ld_dy, a.bf16) && vector_rows(a.add, a.ld_add, a.bf16) &&
                     vector_rows(a.dx, a.ld_dx, a.bf16) && vector_rows(a.weight, 0, a.weight_bf16);
    if (a.rows > 0) {
        if (a.bf16 && vec) launch<uint16_t, true>(a, stream);
        else if (a.bf16) launch<uint16_t, false>(a, stream);
        else if (vec) launch<float, true>(a, stream);
        else launch<float, false>(a, stream);
        const cudaError_t e = cudaPeekAtLastError();
        if (e != cudaSuccess) return e;
    }
    const int64_t groups = a.rows > 0 ? rms_norm_grad_partials(a.rows, a.cols) / a.cols : 0;
    return launch_after(dweight_kernel, dim3(uint32_t((a.cols + 31) / 32)), dim3(1024), 0, stream, 1,
                        static_cast<const float *>(a.partials), groups, int(a.cols), a.dweight,
                        a.dweight_bf16 ? 1 : 0, a.accumulate ? 1 : 0);
}

}  // namespace wc
