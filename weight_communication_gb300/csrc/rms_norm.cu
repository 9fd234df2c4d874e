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
// A row is read once: a group of threads holds all of it in registers, one or two
// pieces of 8 values each (wc_eight.cuh), sums its squares, and writes.  The grid
// is what the GPU holds, and each group loads its next row before it works on the
// present one: a row's sum and barrier would else leave too little in flight.
//
// The weight's gradient is summed over rows in registers: a group has the same
// columns in every row it works on.  A CTA leaves its groups' sum, and a second
// launch adds those in a fixed order.
//
// Bound: HBM, and the issue of instructions not far below it: products go two at a
// time (fma.f32x2).
#include "wc_eight.cuh"
#include "wc_internal.h"
#include "wc_launch.cuh"

namespace wc {

namespace {

constexpr int kSms = 152;

// Threads of a row (16 to 1024) and pieces of 8 values of each; rows of a CTA.
template <int TPR, int PIECES>
struct Shape {
    static constexpr int kTpr = TPR, kPieces = PIECES;
    static constexpr int kThreads = TPR < 256 ? 256 : TPR;
    static constexpr int kRows = kThreads / TPR;
    static constexpr int kWarps = TPR < 32 ? 1 : TPR / 32;  // of a row
    static constexpr int64_t kCols = int64_t(TPR) * PIECES * 8;  // at most
};

// CTAs of the forward pass that an SM holds at once, as their registers allow.
template <typename T, typename S>
constexpr int per_sm() {
    constexpr bool half = sizeof(T) == 2;
    return S::kThreads == 256 ? (half || S::kPieces == 1 ? 3 : 2) : S::kThreads == 512 && (half || S::kPieces == 1) ? 2 : 1;
}

// Column of the first value of this thread's block of piece p.
template <typename S>
__device__ __forceinline__ int block_column(int in_row, int p) {
    return (p * S::kTpr + in_row) / 16 * kBlock8;
}

// Sum over a row's threads, the same bits in each.  `slots`: one per warp of the CTA,
// not in use by an earlier sum (two sets taken in turn see to that).
template <typename S>
__device__ __forceinline__ float row_sum(float x, float *slots) {
#pragma unroll
    for (int o = S::kTpr < 32 ? S::kTpr / 2 : 16; o > 0; o /= 2) x = __fadd_rn(x, __shfl_xor_sync(kFull, x, o));
    if (S::kWarps == 1) return x;
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) slots[warp] = x;
    __syncthreads();
    const float *row = slots + warp / S::kWarps * S::kWarps;
    x = row[0];
#pragma unroll
    for (int w = 1; w < S::kWarps; ++w) x = __fadd_rn(x, row[w]);
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

// 1 / sqrt(v), within an ulp: the approximation and a step of Newton's iteration.
__device__ __forceinline__ float inverse_root(float v) {
    const float r = rsqrtf(v);
    const float e = __fmaf_rn(-__fmul_rn(v, r), r, 1.0f);
    return v > 0.0f && v < INFINITY ? __fmaf_rn(__fmul_rn(r, 0.5f), e, r) : r;
}

template <typename T, bool VEC>
__device__ __forceinline__ f32x2 pair_of(const Eight<T, VEC> &v, int k) {
    return pack2(v.at(2 * k), v.at(2 * k + 1));
}

template <typename T, bool VEC, typename S>
__global__ void __launch_bounds__(S::kThreads, per_sm<T, S>()) rms_norm_kernel(const RmsNorm a) {
    constexpr int PIECES = S::kPieces;
    __shared__ float slots[2][S::kThreads / 32];
    const int in_row = threadIdx.x % S::kTpr, l = in_row & 15;
    const int64_t step = int64_t(gridDim.x) * S::kRows;
    const int cols = int(a.cols);
    const f32x2 zero = pack2(-0.0f, -0.0f);
    const float each = __fdiv_rn(1.0f, float(cols));
    f32x2 weight[PIECES][4];
#pragma unroll
    for (int p = 0; p < PIECES; ++p) {
        const int col = block_column<S>(in_row, p);
        float w[8];
        weights<VEC>(a.weight, a.weight_bf16, col, l, cols - col, w);
#pragma unroll
        for (int k = 0; k < 4; ++k) weight[p][k] = pack2(w[2 * k], w[2 * k + 1]);
    }
    Eight<T, VEC> x[PIECES], o[PIECES];
    auto fetch = [&](int64_t row) {
#pragma unroll
        for (int p = 0; p < PIECES; ++p) {
            const int col = block_column<S>(in_row, p), left = row < a.rows ? cols - col : 0;
            x[p].load(static_cast<const T *>(a.x) + row * a.ld_x + col, l, left);
            if (a.add) o[p].load(static_cast<const T *>(a.add) + row * a.ld_add + col, l, left);
        }
    };
    // every row group of a CTA takes as many turns, for the CTA's barriers
    const int64_t first = int64_t(blockIdx.x) * S::kRows, turns = (a.rows - first + step - 1) / step;
    int64_t row = first + threadIdx.x / S::kTpr;
    fetch(row);
    for (int64_t i = 0; i < turns; ++i, row += step) {
        const bool live = row < a.rows;
        Eight<T, VEC> t[PIECES];
        f32x2 sum = zero;
#pragma unroll
        for (int p = 0; p < PIECES; ++p) {
            t[p] = x[p];
            if (a.add) {
                const int col = block_column<S>(in_row, p);
                float s[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) s[j] = __fadd_rn(x[p].at(j), o[p].at(j));
                t[p].set(s);
                t[p].store(static_cast<T *>(a.total) + row * a.ld_total + col, l, live ? cols - col : 0);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) sum = fma2_rn(pair_of(t[p], k), pair_of(t[p], k), sum);
        }
        if (i + 1 < turns) fetch(row + step);
        float even, odd;
        unpack2(sum, even, odd);
        const float all = row_sum<S>(__fadd_rn(even, odd), slots[i & 1]);
        const float r = inverse_root(__fmaf_rn(all, each, a.eps));
        const f32x2 rr = pack2(r, r);
#pragma unroll
        for (int p = 0; p < PIECES; ++p) {
            const int col = block_column<S>(in_row, p);
            float y[8];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                unpack2(fma2_rn(fma2_rn(pair_of(t[p], k), rr, zero), weight[p][k], zero), y[2 * k], y[2 * k + 1]);
            Eight<T, VEC> out;
            out.set(y);
            out.store(static_cast<T *>(a.y) + row * a.ld_y + col, l, live ? cols - col : 0);
        }
        if (a.kept.q == nullptr) continue;
        if (in_row == 0 && live) a.rstd[row] = r;
        // a lane divides for one piece: the even ones for the first, the odd ones for the second
        uint32_t mine = block_max(t[0].mag());
        if (PIECES > 1) {
            const uint32_t second = block_max(t[PIECES - 1].mag());
            if (l & 1) mine = second;
        }
        const Scale8 own = scale_of(__uint_as_float(mine));
        if (l < PIECES) {
            const int col = block_column<S>(in_row, l);
            if (live && col < cols) a.kept.s[col / kBlock8 * a.kept.ld_s + row] = own.scale;
        }
#pragma unroll
        for (int p = 0; p < PIECES; ++p) {
            const int col = block_column<S>(in_row, p);
            const float inv = __shfl_sync(kFull, own.inv, p, 16);
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = t[p].at(j);
            store_codes<VEC>(a.kept.q + row * a.kept.ld_q + col, codes_of(v, inv), l, live ? cols - col : 0);
        }
    }
}

// CTAs of the gradient that an SM holds at once.
template <bool VEC, typename S>
struct Plan {
    static constexpr int kCtas = S::kThreads == 256 ? (S::kPieces == 2 ? 2 : VEC ? 3 : 4)
                                 : S::kThreads == 512 && S::kPieces == 1 ? 2 : 1;
    // the groups' sums, where a CTA has several
    static constexpr int kSums = S::kRows > 1 ? S::kThreads * S::kPieces * 8 : 1;
    static int64_t ctas(int64_t rows) {
        const int64_t need = (rows + S::kRows - 1) / S::kRows, most = int64_t(kSms) * kCtas;
        return need < most ? need : most;
    }
};

template <typename T, bool VEC, typename S>
__global__ void __launch_bounds__(S::kThreads, Plan<VEC, S>::kCtas) rms_norm_grad_kernel(const RmsNormGrad a) {
    constexpr int PIECES = S::kPieces;
    __shared__ float slots[2][S::kThreads / 32];
    __shared__ float sums[Plan<VEC, S>::kSums];
    const int me = threadIdx.x, in_row = me % S::kTpr, l = in_row & 15;
    const int64_t first = int64_t(blockIdx.x) * S::kRows, step = int64_t(gridDim.x) * S::kRows;
    const int cols = int(a.cols);
    const float each = __fdiv_rn(1.0f, float(cols));
    const f32x2 zero = pack2(-0.0f, -0.0f);
    f32x2 dw[PIECES][4], weight[PIECES][4];
#pragma unroll
    for (int p = 0; p < PIECES; ++p) {
        const int col = block_column<S>(in_row, p);
        float w[8];
        weights<VEC>(a.weight, a.weight_bf16, col, l, cols - col, w);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            weight[p][k] = pack2(w[2 * k], w[2 * k + 1]);
            dw[p][k] = pack2(0.0f, 0.0f);
        }
    }
    // the next row
    Eight<T, VEC> dy[PIECES], add[PIECES];
    uint2 codes[PIECES];
    float scale[PIECES], r = 0.0f;
    auto fetch = [&](int64_t row) {
        const bool live = row < a.rows;
        if (live) r = a.rstd[row];
#pragma unroll
        for (int p = 0; p < PIECES; ++p) {
            const int col = block_column<S>(in_row, p), left = live ? cols - col : 0;
            dy[p].load(static_cast<const T *>(a.dy) + row * a.ld_dy + col, l, left);
            codes[p] = load_codes<VEC>(a.kept.q + row * a.kept.ld_q + col, l, left);
            scale[p] = left > 0 ? a.kept.s[col / kBlock8 * a.kept.ld_s + row] : 0.0f;
            if (a.add) add[p].load(static_cast<const T *>(a.add) + row * a.ld_add + col, l, left);
            else add[p].zero();
        }
    };
    // every row group of a CTA takes as many turns, for the CTA's barriers
    const int64_t turns = (a.rows - first + step - 1) / step;
    int64_t row = first + me / S::kTpr;
    // (the longest rows leave no registers for it, and short ones that are moved value
    // by value gain more from a fourth CTA: 8192 x 2047 48 -> 44 us)
    constexpr bool kAhead = (VEC || S::kThreads > 256) && S::kThreads * PIECES < 2048;
    if (kAhead) fetch(row);
    for (int64_t i = 0; i < turns; ++i, row += step) {
        if (!kAhead) fetch(row);
        // n, and dy * w
        f32x2 n[PIECES][4], wd[PIECES][4], sum = zero;
        Eight<T, VEC> past[PIECES];
        const f32x2 rr = pack2(r, r);
#pragma unroll
        for (int p = 0; p < PIECES; ++p) {
            float t[8];
            values_of(codes[p], scale[p], t);
            past[p] = add[p];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const f32x2 d = pair_of(dy[p], k);
                n[p][k] = fma2_rn(pack2(t[2 * k], t[2 * k + 1]), rr, zero);
                wd[p][k] = fma2_rn(d, weight[p][k], zero);
                sum = fma2_rn(wd[p][k], n[p][k], sum);
                dw[p][k] = fma2_rn(d, n[p][k], dw[p][k]);
            }
        }
        if (kAhead && i + 1 < turns) fetch(row + step);
        float even, odd;
        unpack2(sum, even, odd);
        const float mean = __fmul_rn(row_sum<S>(__fadd_rn(even, odd), slots[i & 1]), -each);
        const f32x2 mm = pack2(mean, mean);
#pragma unroll
        for (int p = 0; p < PIECES; ++p) {
            const int col = block_column<S>(in_row, p);
            float x[8];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                unpack2(fma2_rn(fma2_rn(n[p][k], mm, wd[p][k]), rr, pair_of(past[p], k)), x[2 * k], x[2 * k + 1]);
            Eight<T, VEC> out;
            out.set(x);
            out.store(static_cast<T *>(a.dx) + row * a.ld_dx + col, l, row < a.rows ? cols - col : 0);
        }
    }
    // the CTA's sum over its groups
#pragma unroll
    for (int p = 0; p < PIECES; ++p) {
        const int col = block_column<S>(in_row, p);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float x[2];
            unpack2(dw[p][k], x[0], x[1]);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int c = col + column_of<VEC>(l, 2 * k + h);
                if (c >= cols) continue;
                if (S::kRows > 1) sums[me / S::kTpr * cols + c] = x[h];
                else a.partials[int64_t(blockIdx.x) * cols + c] = x[h];
            }
        }
    }
    if (S::kRows > 1) {
        __syncthreads();
        for (int c = me; c < cols; c += S::kThreads) {
            float x = sums[c];
#pragma unroll
            for (int g = 1; g < S::kRows; ++g) x = __fadd_rn(x, sums[g * cols + c]);
            a.partials[int64_t(blockIdx.x) * cols + c] = x;
        }
    }
    let_successor_start();
}

// dweight = sum of the CTAs' partials: 32 columns by 32 warps of a CTA, each
// warp every 32nd partial, then the warps in turn.
__global__ void __launch_bounds__(1024) dweight_kernel(const float *partials, int64_t count, int cols,
                                                       void *dweight, int bf16, int accumulate) {
    __shared__ float sums[32][33];
    wait_for_predecessor();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float x = 0.0f;
    if (c < cols)
#pragma unroll 8
        for (int64_t g = warp; g < count; g += 32) x = __fadd_rn(x, partials[g * cols + c]);
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

// f(the shape of rows of `cols` columns).
template <bool VEC, typename F>
auto with_shape(int64_t cols, F f) {
    if (cols <= Shape<16, 1>::kCols) return f(Shape<16, 1>());
    if (cols <= Shape<32, 1>::kCols) return f(Shape<32, 1>());
    if constexpr (VEC) {
        if (cols <= Shape<32, 2>::kCols) return f(Shape<32, 2>());
        if (cols <= Shape<64, 2>::kCols) return f(Shape<64, 2>());
        if (cols <= Shape<128, 2>::kCols) return f(Shape<128, 2>());
        if (cols <= Shape<256, 2>::kCols) return f(Shape<256, 2>());
        if (cols <= Shape<512, 2>::kCols) return f(Shape<512, 2>());
    } else {
        // value by value: more instructions, so more warps to hide their latency
        if (cols <= Shape<64, 1>::kCols) return f(Shape<64, 1>());
        if (cols <= Shape<128, 1>::kCols) return f(Shape<128, 1>());
        if (cols <= Shape<256, 1>::kCols) return f(Shape<256, 1>());
        if (cols <= Shape<512, 1>::kCols) return f(Shape<512, 1>());
        if (cols <= Shape<1024, 1>::kCols) return f(Shape<1024, 1>());
    }
    static_assert(Shape<1024, 2>::kCols == kNormCols, "the largest shape has the longest row");
    return f(Shape<1024, 2>());
}

bool vector_rows(const void *p, int64_t ld, bool bf16) {
    return p == nullptr || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % (bf16 ? 8 : 4) == 0);
}

template <typename T, bool VEC>
void launch(const RmsNorm &a, cudaStream_t stream) {
    with_shape<VEC>(a.cols, [&](auto shape) {
        using S = decltype(shape);
        const int64_t need = (a.rows + S::kRows - 1) / S::kRows, most = int64_t(kSms) * per_sm<T, S>();
        rms_norm_kernel<T, VEC, S><<<uint32_t(need < most ? need : most), S::kThreads, 0, stream>>>(a);
        return 0;
    });
}

template <typename T, bool VEC>
void launch(const RmsNormGrad &a, cudaStream_t stream) {
    with_shape<VEC>(a.cols, [&](auto shape) {
        using S = decltype(shape);
        rms_norm_grad_kernel<T, VEC, S><<<uint32_t(Plan<VEC, S>::ctas(a.rows)), S::kThreads, 0, stream>>>(a);
        return 0;
    });
}

int64_t grad_ctas(int64_t rows, int64_t cols, bool vec) {
    if (vec) return with_shape<true>(cols, [&](auto shape) { return Plan<true, decltype(shape)>::ctas(rows); });
    return with_shape<false>(cols, [&](auto shape) { return Plan<false, decltype(shape)>::ctas(rows); });
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
    const int64_t a = grad_ctas(rows, cols, true), b = grad_ctas(rows, cols, false);
    return cols * (a > b ? a : b);
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
    const int64_t count = a.rows > 0 ? grad_ctas(a.rows, a.cols, vec) : 0;
    return launch_after(dweight_kernel, dim3(uint32_t((a.cols + 31) / 32)), dim3(1024), 0, stream, 1,
                        static_cast<const float *>(a.partials), count, int(a.cols), a.dweight,
                        a.dweight_bf16 ? 1 : 0, a.accumulate ? 1 : 0);
}

}  // namespace wc
