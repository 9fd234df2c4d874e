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
// launch adds in a fixed order.  Those sums leave few registers, so the rows to
// come are brought to shared memory ahead of their turn, each thread's own values
// by cp.async.
//
// Bound: HBM.
#include <atomic>
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

template <int BYTES>
__device__ __forceinline__ void copy_async(void *to, const void *from) {
    const uint32_t at = uint32_t(__cvta_generic_to_shared(to));
    if (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at), "l"(from) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(at), "l"(from), "n"(BYTES) : "memory");
}

// A row's values as one thread takes them: 16-byte words of dy and add, codes and
// scale of each piece, and r.  In shared memory each of them lies by threads.
template <typename T, int THREADS, int PIECES>
struct Stage {
    static constexpr int kWords = sizeof(T) / 2;  // 16-byte words of 8 values
    uint4 dy[PIECES * kWords][THREADS], add[PIECES * kWords][THREADS];
    uint2 codes[PIECES][THREADS];
    float scale[PIECES][THREADS];
    float r[THREADS];
};

// CTAs of the gradient that an SM holds at once, and the stages that then fit
// its shared memory (fewer than two are of no use).
template <typename T, typename S, int PIECES>
struct Plan {
    static constexpr bool kHalf = sizeof(T) == 2;
    static constexpr int kCtas = S::kThreads <= 256 ? (kHalf ? 3 : 2) : S::kThreads <= 512 && kHalf ? 2 : 1;
    // the weight beside them, where there is room: it would come from L2 twice a row
    static constexpr bool kWeight = S::kThreads <= 256;
    static constexpr int kWeightBytes = kWeight ? S::kThreads * PIECES * 32 : 0;
    static constexpr int kFit = (224 * 1024 / kCtas - kWeightBytes) / int(sizeof(Stage<T, S::kThreads, PIECES>));
    static constexpr int kStages = kFit < 2 ? 0 : kFit < 3 ? kFit : 3;
    // Row groups of the grid: what the GPU runs at once, and no more than rows.
    static int64_t groups(int64_t rows) {
        const int64_t most = int64_t(kSms) * kCtas * S::kRows;
        return ((rows < most ? rows : most) + S::kRows - 1) / S::kRows * S::kRows;
    }
};

template <typename T, bool VEC, int TPR, int PIECES>
__global__ void __launch_bounds__(Shape<TPR, PIECES>::kThreads, Plan<T, Shape<TPR, PIECES>, PIECES>::kCtas)
rms_norm_grad_kernel(const RmsNormGrad a) {
    using S = Shape<TPR, PIECES>;
    constexpr int kStages = VEC ? Plan<T, S, PIECES>::kStages : 0, kAhead = kStages - 1;
    constexpr bool kRing = kStages > 0, kWeight = kRing && Plan<T, S, PIECES>::kWeight;
    using Ring = Stage<T, S::kThreads, PIECES>;
    extern __shared__ __align__(16) uint8_t ring_bytes[];
    __shared__ float slots[2][S::kThreads / 32];
    Ring *const ring = reinterpret_cast<Ring *>(ring_bytes);
    const int me = threadIdx.x, in_row = me % TPR, l = in_row & 15;
    const int64_t group = int64_t(blockIdx.x) * S::kRows + me / TPR;
    const int64_t groups = int64_t(gridDim.x) * S::kRows;
    const int cols = int(a.cols);
    const float each = __fdiv_rn(1.0f, float(cols));
    float dw[PIECES][8];
#pragma unroll
    for (int p = 0; p < PIECES; ++p)
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[p][j] = 0.0f;
    // [two words of each piece][threads], each thread's own
    float4 *const own_weight = reinterpret_cast<float4 *>(ring_bytes + kStages * sizeof(Ring)) + me;
    if constexpr (kWeight) {
#pragma unroll
        for (int p = 0; p < PIECES; ++p) {
            const int col = (p * TPR + in_row) / 16 * kBlock8;
            float w[8];
            weights<VEC>(a.weight, a.weight_bf16, col, l, cols - col, w);
            own_weight[2 * p * S::kThreads] = make_float4(w[0], w[1], w[2], w[3]);
            own_weight[(2 * p + 1) * S::kThreads] = make_float4(w[4], w[5], w[6], w[7]);
        }
    }
    auto weight_of = [&](int p, int col, float(&w)[8]) {
        if constexpr (kWeight) {
            const float4 x = own_weight[2 * p * S::kThreads], y = own_weight[(2 * p + 1) * S::kThreads];
            w[0] = x.x;
            w[1] = x.y;
            w[2] = x.z;
            w[3] = x.w;
            w[4] = y.x;
            w[5] = y.y;
            w[6] = y.z;
            w[7] = y.w;
        } else {
            weights<VEC>(a.weight, a.weight_bf16, col, l, cols - col, w);
        }
    };
    // the copies of one row, a group of them even if there is none
    auto fetch = [&](int64_t row, int stage) {
        if (row < a.rows) {
            Ring &s = ring[stage];
            copy_async<4>(&s.r[me], a.rstd + row);
#pragma unroll
            for (int p = 0; p < PIECES; ++p) {
                const int col = (p * TPR + in_row) / 16 * kBlock8;
                if (col + 8 * l < cols) {
                    const T *dy = static_cast<const T *>(a.dy) + row * a.ld_dy + col + 8 * l;
                    const T *add = static_cast<const T *>(a.add) + (a.add ? row * a.ld_add + col + 8 * l : 0);
#pragma unroll
                    for (int k = 0; k < Ring::kWords; ++k) {
                        copy_async<16>(&s.dy[p * Ring::kWords + k][me], dy + k * 4);
                        if (a.add) copy_async<16>(&s.add[p * Ring::kWords + k][me], add + k * 4);
                    }
                    copy_async<8>(&s.codes[p][me], a.kept.q + row * a.kept.ld_q + col + 8 * l);
                    copy_async<4>(&s.scale[p][me], a.kept.s + col / kBlock8 * a.kept.ld_s + row);
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // every group of a CTA takes as many turns, for the CTA's barriers
    const int64_t turns = (a.rows - int64_t(blockIdx.x) * S::kRows + groups - 1) / groups;
    int64_t row = group;
    if constexpr (kRing)
        for (int k = 0; k < kAhead; ++k) fetch(row + k * groups, k);
    int stage = 0;
    for (int64_t i = 0; i < turns; ++i, row += groups) {
        const bool live = row < a.rows;
        float r = 0.0f;
        Eight<T> dy[PIECES];
        float n[PIECES][8];
        if constexpr (kRing) {
            // (the stage that the row before has left)
            fetch(row + kAhead * groups, stage == 0 ? kStages - 1 : stage - 1);
            asm volatile("cp.async.wait_group %0;" ::"n"(kAhead) : "memory");
            const Ring &s = ring[stage];
            if (live) r = s.r[me];
#pragma unroll
            for (int p = 0; p < PIECES; ++p) {
                dy[p].zero();
                uint2 codes = make_uint2(0u, 0u);
                float scale = 0.0f;
                if (live && (p * TPR + in_row) / 16 * kBlock8 + 8 * l < cols) {
#pragma unroll
                    for (int k = 0; k < Ring::kWords; ++k) {
                        const uint4 q = s.dy[p * Ring::kWords + k][me];
                        dy[p].w[4 * k] = q.x;
                        dy[p].w[4 * k + 1] = q.y;
                        dy[p].w[4 * k + 2] = q.z;
                        dy[p].w[4 * k + 3] = q.w;
                    }
                    codes = s.codes[p][me];
                    scale = s.scale[p][me];
                }
                values_of(codes, scale, n[p]);
            }
        } else {
            if (live) r = a.rstd[row];
#pragma unroll
            for (int p = 0; p < PIECES; ++p) {
                const int col = (p * TPR + in_row) / 16 * kBlock8, left = live ? cols - col : 0;
                dy[p].template load<VEC>(static_cast<const T *>(a.dy) + row * a.ld_dy + col, l, left);
                const uint2 codes = load_codes<VEC>(a.kept.q + row * a.kept.ld_q + col, l, left);
                values_of(codes, left > 0 ? a.kept.s[col / kBlock8 * a.kept.ld_s + row] : 0.0f, n[p]);
            }
        }
        float sum = 0.0f;
#pragma unroll
        for (int p = 0; p < PIECES; ++p) {
            const int col = (p * TPR + in_row) / 16 * kBlock8;
            float w[8];
            weight_of(p, col, w);
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
            weight_of(p, col, w);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                x[j] = __fmul_rn(r, __fmaf_rn(-n[p][j], mean, __fmul_rn(dy[p].at(j), w[j])));
            if (a.add) {
                Eight<T> o;
                if constexpr (kRing) {
                    o.zero();
                    if (8 * l < left) {
#pragma unroll
                        for (int k = 0; k < Ring::kWords; ++k) {
                            const uint4 q = ring[stage].add[p * Ring::kWords + k][me];
                            o.w[4 * k] = q.x;
                            o.w[4 * k + 1] = q.y;
                            o.w[4 * k + 2] = q.z;
                            o.w[4 * k + 3] = q.w;
                        }
                    }
                } else {
                    o.template load<VEC>(static_cast<const T *>(a.add) + row * a.ld_add + col, l, left);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = __fadd_rn(x[j], o.at(j));
            }
            Eight<T> out;
            out.set(x);
            out.template store<VEC>(static_cast<T *>(a.dx) + row * a.ld_dx + col, l, left);
        }
        if (++stage == kStages) stage = 0;
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

template <typename T>
int64_t groups_of(int64_t rows, int64_t cols) {
    return with_shape(cols, [&](auto shape, auto, auto pieces) {
        return Plan<T, decltype(shape), decltype(pieces)::value>::groups(rows);
    });
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

template <typename T, bool VEC, int TPR, int PIECES>
cudaError_t launch_grad(const RmsNormGrad &a, cudaStream_t stream) {
    using S = Shape<TPR, PIECES>;
    using P = Plan<T, S, PIECES>;
    constexpr size_t smem = VEC && P::kStages > 0 ? P::kStages * sizeof(Stage<T, S::kThreads, PIECES>) + P::kWeightBytes : 0;
    if constexpr (smem > 48 * 1024) {
        // once for each GPU: the kernel's attribute stays set
        static std::atomic<uint64_t> prepared{0};
        int device = 0;
        cudaError_t e = cudaGetDevice(&device);
        if (e != cudaSuccess) return e;
        const uint64_t bit = uint64_t(1) << (device & 63);
        if (device > 63 || !(prepared.load(std::memory_order_relaxed) & bit)) {
            e = cudaFuncSetAttribute(rms_norm_grad_kernel<T, VEC, TPR, PIECES>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
            if (e != cudaSuccess) return e;
            prepared.fetch_or(bit, std::memory_order_relaxed);
        }
    }
    rms_norm_grad_kernel<T, VEC, TPR, PIECES>
        <<<uint32_t(P::groups(a.rows) / S::kRows), S::kThreads, smem, stream>>>(a);
    return cudaPeekAtLastError();
}

template <typename T, bool VEC>
cudaError_t launch(const RmsNormGrad &a, cudaStream_t stream) {
    return with_shape(a.cols, [&](auto, auto tpr, auto pieces) {
        return launch_grad<T, VEC, decltype(tpr)::value, decltype(pieces)::value>(a, stream);
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
    // (bf16 rows are in no fewer groups than fp32 ones)
    return cols * groups_of<uint16_t>(rows, cols);
}

cudaError_t launch_rms_norm_grad(const RmsNormGrad &a, cudaStream_t stream) {
    const bool vec = a.cols % 8 == 0 && vector_rows(a.dy, a.ld_dy, a.bf16) && vector_rows(a.add, a.ld_add, a.bf16) &&
                     vector_rows(a.dx, a.ld_dx, a.bf16) && vector_rows(a.weight, 0, a.weight_bf16);
    if (a.rows > 0) {
        const cudaError_t e = a.bf16 && vec ? launch<uint16_t, true>(a, stream)
                              : a.bf16      ? launch<uint16_t, false>(a, stream)
                              : vec         ? launch<float, true>(a, stream)
                                            : launch<float, false>(a, stream);
        if (e != cudaSuccess) return e;
    }
    const int64_t groups = a.rows == 0 ? 0 : a.bf16 ? groups_of<uint16_t>(a.rows, a.cols) : groups_of<float>(a.rows, a.cols);
    return launch_after(dweight_kernel, dim3(uint32_t((a.cols + 31) / 32)), dim3(1024), 0, stream, 1,
                        static_cast<const float *>(a.partials), groups, int(a.cols), a.dweight,
                        a.dweight_bf16 ? 1 : 0, a.accumulate ? 1 : 0);
}

}  // namespace wc
