// activation.cu -- a layer's activation, gated or not, whose inputs are kept in
// 8 bits (e4m3, one fp32 scale per 128 of a row) for the backward pass.
//
//   forward : h = act(gate) * up                (or act(gate) alone)
//   kept    : codes and scales of gate and up   (the rule of wc_fp8.cuh)
//   backward: dgate = dh * up^ * act'(gate^),  dup = dh * act(gate^)
//             where ^ is what the kept codes stand for
//
// act is relu, or a * sigmoid(z(a)): silu with z = a, and gelu in its tanh form,
// 0.5 a (1 + tanh(u)) = a * sigmoid(2u), with z = 2u = 2 sqrt(2/pi) (a + 0.044715 a^3).
// So act' = s + a s (1 - s) z'.  All in fp32; h and the gradients are rounded
// once, to their type.
//
// Bound: HBM.  Each value is read once and written once; the codes are made
// from the values that the forward pass holds in registers anyway.  16 lanes
// have a block of 128 (wc_eight.cuh) and a CTA 16 rows by one or four blocks, so that
// the scales, which lie by blocks first and rows second, are written 64 bytes at
// a time.
#include "wc_eight.cuh"
#include "wc_internal.h"

namespace wc {

namespace {

constexpr int kThreads = 256;
constexpr int kRows = kThreads / 16;  // of a CTA
// Blocks of a row that a thread has (ACROSS), all in flight at once: 8192 x 11008 gated,
// both ways, one block 263 us, two 246, four 232.  Where the CTAs would not fill
// the GPU, one (333 x 1003 fp32: four 10.6 us, two 7.1).
constexpr int kMany = 4;

constexpr float kGelu1 = 1.59576912160573071176f;                  // 2 sqrt(2 / pi)
constexpr float kGelu3 = 1.59576912160573071176f * 0.044715f;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 1 / (1 + exp(-z)).  FAST (for 16-bit results): within 2^-20 relative for the
// z where the result is not negligible, in two operations of the special
// functions' unit.
template <bool FAST>
__device__ __forceinline__ float sigmoid(float z) {
    if (FAST) return rcp(__fadd_rn(1.0f, ex2(__fmul_rn(z, -1.44269504088896340736f))));
    return __fdiv_rn(1.0f, __fadd_rn(1.0f, expf(-z)));
}

// Past 100 either way act' is 0 or 1, and nothing below overflows (NaN stays NaN).
__device__ __forceinline__ float within_100(float a) {
    float r;
    asm("{\n.reg .f32 t;\nmin.NaN.f32 t, %1, 0f42C80000;\nmax.NaN.f32 %0, t, 0fC2C80000;\n}\n" : "=f"(r) : "f"(a));
    return r;
}

template <bool FAST>
__device__ __forceinline__ float act(int kind, float a) {
    if (kind == kActRelu) return a < 0.0f ? 0.0f : a;
    float z = a;
    if (kind == kActGelu) z = __fmul_rn(a, __fmaf_rn(__fmul_rn(a, a), kGelu3, kGelu1));
    return __fmul_rn(a, sigmoid<FAST>(z));
}

template <bool FAST>
__device__ __forceinline__ void act_both(int kind, float a, float &f, float &d) {
    if (kind == kActRelu) {
        f = a < 0.0f ? 0.0f : a;
        d = a > 0.0f ? 1.0f : __fmul_rn(0.0f, a);  // NaN for NaN
        return;
    }
    const float b = within_100(a);
    float z = b, dz = 1.0f;
    if (kind == kActGelu) {
        const float sq = __fmul_rn(b, b);
        z = __fmul_rn(b, __fmaf_rn(sq, kGelu3, kGelu1));
        dz = __fmaf_rn(sq, 3.0f * kGelu3, kGelu1);
    }
    const float s = sigmoid<FAST>(z);
    f = __fmul_rn(a, s);
    d = __fmul_rn(s, __fmaf_rn(__fmul_rn(b, __fadd_rn(1.0f, -s)), dz, 1.0f));
}

// The first value of this thread's blocks, and how many columns are left there.
struct Place {
    int64_t row;
    int64_t col;
    int32_t block;
};

template <int ACROSS>
__device__ __forceinline__ Place place(int32_t across) {
    const int64_t tile = blockIdx.x;
    const int64_t down = tile / across;
    const int32_t block = int32_t(tile - down * across) * ACROSS;
    return {down * kRows + (threadIdx.x >> 4), int64_t(block) * kBlock8, block};
}

template <typename T, bool VEC, bool GATED, bool KEEP, int kAcross>
__global__ void __launch_bounds__(kThreads, kAcross == 1 ? 5 : sizeof(T) == 2 ? 4 : 3) act_kernel(const Activation a, int32_t across) {
    constexpr bool kFast = sizeof(T) == 2;
    const Place at = place<kAcross>(across);
    const int l = threadIdx.x & 15;
    const bool live = at.row < a.rows;
    const T *gate = static_cast<const T *>(a.gate) + at.row * a.ld_gate + at.col;
    const T *up = static_cast<const T *>(a.up) + (GATED ? at.row * a.ld_up + at.col : 0);
    T *h = static_cast<T *>(a.h) + at.row * a.ld_h + at.col;
    const int left = live ? int(min(a.cols - at.col, int64_t(kAcross * kBlock8))) : 0;

    Eight<T, VEC> g[kAcross], u[kAcross];
#pragma unroll
    for (int k = 0; k < kAcross; ++k) {
        g[k].load(gate + k * kBlock8, l, left - k * kBlock8);
        if (GATED) u[k].load(up + k * kBlock8, l, left - k * kBlock8);
    }
#pragma unroll
    for (int k = 0; k < kAcross; ++k) {
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            x[j] = act<kFast>(a.kind, g[k].at(j));
            if (GATED) x[j] = __fmul_rn(x[j], u[k].at(j));
        }
        Eight<T, VEC> out;
        out.set(x);
        out.store(h + k * kBlock8, l, left - k * kBlock8);
    }
    if (!KEEP) return;
    // a lane divides for one block, gate's first and then up's
    constexpr int kEach = GATED ? 2 * kAcross : kAcross;
    uint32_t mine = 0u;
#pragma unroll
    for (int k = 0; k < kAcross; ++k) {
        const uint32_t mg = block_max(g[k].mag());
        if ((l & (kEach - 1)) == k) mine = mg;
        if (GATED) {
            const uint32_t mu = block_max(u[k].mag());
            if ((l & (kEach - 1)) == kAcross + k) mine = mu;
        }
    }
    const Scale8 own = scale_of(__uint_as_float(mine));
    if (l < kEach && live) {
        const int k = l & (kAcross - 1);
        if (at.col + k * kBlock8 < a.cols) {
            const Kept8 &to = l < kAcross ? a.kept_gate : a.kept_up;
            to.s[(at.block + k) * to.ld_s + at.row] = own.scale;
        }
    }
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
        const int k = e & (kAcross - 1);
        const float inv = __shfl_sync(kFull, own.inv, e, 16);
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = e < kAcross ? g[k].at(j) : u[k].at(j);
        const Kept8 &to = e < kAcross ? a.kept_gate : a.kept_up;
        store_codes<VEC>(to.q + at.row * to.ld_q + at.col + k * kBlock8, codes_of(x, inv), l, left - k * kBlock8);
    }
}

template <typename T, bool VEC, bool GATED, int kAcross>
__global__ void __launch_bounds__(kThreads, kAcross == 1 ? 5 : sizeof(T) == 2 ? 4 : 3) act_grad_kernel(const ActivationGrad a, int32_t across) {
    constexpr bool kFast = sizeof(T) == 2;
    const Place at = place<kAcross>(across);
    const int l = threadIdx.x & 15;
    if (at.row >= a.rows) return;
    const int left = int(min(a.cols - at.col, int64_t(kAcross * kBlock8)));
    const T *dh = static_cast<const T *>(a.dh) + at.row * a.ld_dh + at.col;
    const uint8_t *qg = a.kept_gate.q + at.row * a.kept_gate.ld_q + at.col;
    const uint8_t *qu = a.kept_up.q + (GATED ? at.row * a.kept_up.ld_q + at.col : 0);
    T *dg = static_cast<T *>(a.dgate) + at.row * a.ld_dgate + at.col;
    T *du = static_cast<T *>(a.dup) + (GATED ? at.row * a.ld_dup + at.col : 0);

    Eight<T, VEC> d[kAcross];
    uint2 cg[kAcross], cu[kAcross];
    float sg[kAcross], su[kAcross];
#pragma unroll
    for (int k = 0; k < kAcross; ++k) {
        const int rest = left - k * kBlock8;
        d[k].load(dh + k * kBlock8, l, rest);
        cg[k] = load_codes<VEC>(qg + k * kBlock8, l, rest);
        sg[k] = rest > 0 ? a.kept_gate.s[(at.block + k) * a.kept_gate.ld_s + at.row] : 0.0f;
        if (GATED) {
            cu[k] = load_codes<VEC>(qu + k * kBlock8, l, rest);
            su[k] = rest > 0 ? a.kept_up.s[(at.block + k) * a.kept_up.ld_s + at.row] : 0.0f;
        }
    }
#pragma unroll
    for (int k = 0; k < kAcross; ++k) {
        const int rest = left - k * kBlock8;
        float g[8], u[8], x[8], y[8];
        values_of(cg[k], sg[k], g);
        if (GATED) values_of(cu[k], su[k], u);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float f, df;
            act_both<kFast>(a.kind, g[j], f, df);
            const float t = d[k].at(j);
            if (GATED) {
                x[j] = __fmul_rn(__fmul_rn(t, u[j]), df);
                y[j] = __fmul_rn(t, f);
            } else {
                x[j] = __fmul_rn(t, df);
            }
        }
        Eight<T, VEC> out;
        out.set(x);
        out.store(dg + k * kBlock8, l, rest);
        if (GATED) {
            out.set(y);
            out.store(du + k * kBlock8, l, rest);
        }
    }
}

// 16 bytes at a time?  (rows, then what is left of each)
template <typename T>
bool vector_rows(const void *p, int64_t ld) {
    return p == nullptr || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % (16 / int(sizeof(T))) == 0);
}

uint32_t tiles(int64_t rows, int64_t cols, int each, int32_t *across) {
    *across = int32_t((cols + each * kBlock8 - 1) / (each * kBlock8));
    return uint32_t((rows + kRows - 1) / kRows * *across);
}

bool many(int64_t rows, int64_t cols) {
    int32_t across;
    return tiles(rows, cols, kMany, &across) >= 4 * 152;
}

template <typename T, bool VEC, int ACROSS>
void launch(const Activation &a, cudaStream_t stream) {
    int32_t across;
    const uint32_t grid = tiles(a.rows, a.cols, ACROSS, &across);
    const bool keep = a.kept_gate.q != nullptr;
    if (a.up && keep) act_kernel<T, VEC, true, true, ACROSS><<<grid, kThreads, 0, stream>>>(a, across);
    else if (a.up) act_kernel<T, VEC, true, false, ACROSS><<<grid, kThreads, 0, stream>>>(a, across);
    else if (keep) act_kernel<T, VEC, false, true, ACROSS><<<grid, kThreads, 0, stream>>>(a, across);
    else act_kernel<T, VEC, false, false, ACROSS><<<grid, kThreads, 0, stream>>>(a, across);
}

template <typename T, bool VEC, int ACROSS>
void launch(const ActivationGrad &a, cudaStream_t stream) {
    int32_t across;
    const uint32_t grid = tiles(a.rows, a.cols, ACROSS, &across);
    if (a.dup) act_grad_kernel<T, VEC, true, ACROSS><<<grid, kThreads, 0, stream>>>(a, across);
    else act_grad_kernel<T, VEC, false, ACROSS><<<grid, kThreads, 0, stream>>>(a, across);
}

template <typename T, typename Call>
void launch(const Call &a, bool vec, cudaStream_t stream) {
    const bool m = many(a.rows, a.cols);
    if (vec && m) launch<T, true, kMany>(a, stream);
    else if (vec) launch<T, true, 1>(a, stream);
    else launch<T, false, 1>(a, stream);  // (many instructions, so rather many warps)
}

template <typename T>
void launch(const Activation &a, cudaStream_t stream) {
    launch<T>(a, a.cols % 8 == 0 && vector_rows<T>(a.gate, a.ld_gate) && vector_rows<T>(a.up, a.ld_up) &&
                     vector_rows<T>(a.h, a.ld_h), stream);
}

template <typename T>
void launch(const ActivationGrad &a, cudaStream_t stream) {
    launch<T>(a, a.cols % 8 == 0 && vector_rows<T>(a.dh, a.ld_dh) && vector_rows<T>(a.dgate, a.ld_dgate) &&
                     vector_rows<T>(a.dup, a.ld_dup), stream);
}

}  // namespace

cudaError_t launch_activation(const Activation &a, cudaStream_t stream) {
    if (a.bf16) launch<uint16_t>(a, stream);
    else launch<float>(a, stream);
    return cudaPeekAtLastError();
}

cudaError_t launch_activation_grad(const ActivationGrad &a, cudaStream_t stream) {
    if (a.bf16) launch<uint16_t>(a, stream);
    else launch<float>(a, stream);
    return cudaPeekAtLastError();
}

}  // namespace wc
