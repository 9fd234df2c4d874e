// grad_clip.cu -- the global norm of a list of gradient tensors, and clipping.
//
//   norm = sqrt(sum over every tensor of x^2)
//   coef = min(1, max_norm / (norm + eps)),   out = coef * x
//
// Two kernels.  The first squares every value once and leaves one fp64 partial
// sum per CTA in the workspace; the second (one CTA for the norm alone, a full
// grid for clipping) adds the partials in their order -- every CTA the same
// additions, so the coefficient is the same bit pattern everywhere and from
// run to run -- and scales.  No atomics, nothing to initialise, nothing kept.
//
// The tensors' addresses and lengths travel as kernel arguments (up to 1024
// per launch, in the constant bank), so a call copies no table to the device.
// Each tensor is cut into tiles of 32 KB that start on its first 16-byte
// boundary; the values before that boundary belong to its first tile.
//
// Range: x^2 leaves binary32 for |x| beyond 2^64 or below 2^-63.  A thread
// sums 32 values at a time in fp32; where that sum is outside
// [2^-90, 2^100) it is taken again in fp64 from the values it still holds, so
// any finite gradient has a finite norm and tiny ones do not vanish.  These
// sums (7 roundings each) are added with their rounding errors kept (TwoSum,
// Knuth), as well as in fp64 and at the cost of fp32 adds: GB300 does two fp64
// fmas per clock and SM.
//
// Bound: HBM.  The norm reads each value once (875 M bf16 values: 0.252 ms in
// all, 6.9 TB/s); clipping has to read it again, and walks the tiles backwards
// so that what the first pass read last is still in L2 (one d = 2048 layer,
// bf16 into fp32: 68 us for 303 MB read once and written, 72 us forwards).  A
// thread has 128 bytes of a tile in flight; half as many left the norm at 6.4
// TB/s.
#include <math.h>

#include "wc_device.cuh"
#include "wc_internal.h"
#include "wc_launch.cuh"

namespace wc {

namespace {

constexpr int kThreads = 256;
constexpr int kLoads = 8;                     // 16-byte loads of a thread per tile
constexpr uint32_t kTileBytes = kThreads * kLoads * 16;  // 32 KB

__host__ __device__ constexpr uint32_t tile_values(bool bf16) { return kTileBytes / (bf16 ? 2 : 4); }

template <int CAP>
struct SpanTable {
    const void *src[CAP];
    void *dst[CAP];
    int64_t n[CAP];
    uint32_t tile_end[CAP];  // tiles of this and all earlier spans
    uint8_t kind[CAP];       // bit 0: src is bf16, bit 1: dst is bf16
    int count;
    uint32_t tiles;
};

struct Tile {
    int span;
    int64_t begin;       // first value of the vector part
    uint32_t len;        // values from begin, at most a tile's
    uint32_t head;       // values before begin that belong to this tile (first tile only)
};

// Values before the first 16-byte boundary of p.
__host__ __device__ __forceinline__ uint32_t head_of(const void *p, bool bf16, int64_t n) {
    const uint32_t size = bf16 ? 2u : 4u;
    const uint32_t h = uint32_t((16u - (reinterpret_cast<uintptr_t>(p) & 15u)) & 15u) / size;
    return int64_t(h) < n ? h : uint32_t(n);
}

template <int CAP>
__device__ __forceinline__ Tile find_tile(const SpanTable<CAP> &t, uint32_t tile) {
    int lo = 0, hi = t.count - 1;  // first span whose tile_end exceeds `tile`
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (t.tile_end[mid] > tile) hi = mid;
        else lo = mid + 1;
    }
    const uint32_t k = tile - (lo == 0 ? 0u : t.tile_end[lo - 1]);
    const bool bf16 = t.kind[lo] & 1;
    const uint32_t head = head_of(t.src[lo], bf16, t.n[lo]), most = tile_values(bf16);
    Tile r;
    r.span = lo;
    r.begin = int64_t(head) + int64_t(k) * most;
    const int64_t left = t.n[lo] - r.begin;
    r.len = left < int64_t(most) ? uint32_t(left) : most;
    r.head = k == 0 ? head : 0u;
    return r;
}

// The values of a tile that thread t holds: 16-byte vectors t, t + 256, ... of
// it.  Past the end they are zero, which adds nothing.
template <bool BF16>
__device__ __forceinline__ void load_tile(const void *src, int64_t begin, uint32_t len,
                                          uint4 (&raw)[kLoads], bool last_use) {
    constexpr uint32_t W = BF16 ? 8 : 4;
    const uint4 *p = reinterpret_cast<const uint4 *>(
        static_cast<const char *>(src) + begin * (BF16 ? 2 : 4));
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
        const uint32_t v = threadIdx.x + kThreads * j;
        raw[j] = make_uint4(0u, 0u, 0u, 0u);
        if ((v + 1) * W <= len) {
            raw[j] = last_use ? __ldcs(p + v) : p[v];
        } else if (v * W < len) {
            uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
            for (uint32_t e = 0; e < W; ++e) {
                if (v * W + e >= len) continue;
                if (BF16) w[e / 2] |= uint32_t(reinterpret_cast<const uint16_t *>(p)[v * W + e])
                                      << (16 * (e & 1));
                else w[e % 4] = reinterpret_cast<const uint32_t *>(p)[v * W + e];
            }
            raw[j] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

// Value j of consecutive vectors.
template <bool BF16>
__device__ __forceinline__ float value_of(const uint4 *raw, int j) {
    if (BF16) {
        const uint4 q = raw[j / 8];
        const uint32_t w = (j % 8) / 2 == 0 ? q.x : (j % 8) / 2 == 1 ? q.y : (j % 8) / 2 == 2 ? q.z : q.w;
        return __uint_as_float((j & 1) ? (w & 0xFFFF0000u) : (w << 16));
    }
    const uint4 q = raw[j / 4];
    return __uint_as_float(j % 4 == 0 ? q.x : j % 4 == 1 ? q.y : j % 4 == 2 ? q.z : q.w);
}

// A sum carried as hi + lo, plus what fp32 could not hold.
struct NormSum {
    float hi = 0.0f, lo = 0.0f;
    double rare = 0.0;
    __device__ __forceinline__ void add(float s) {
        const float t = __fadd_rn(hi, s);
        const float z = __fsub_rn(t, hi);
        lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(t, z)), __fsub_rn(s, z)));
        hi = t;
    }
};

constexpr float kSafeLow = 8.0779356694631608874e-28f;   // 2^-90
constexpr float kSafeHigh = 1.2676506002282294015e30f;   // 2^100

// 32 values: 4 bf16 vectors or 8 fp32 ones.
template <bool BF16>
__device__ __forceinline__ void add_squares(const uint4 *raw, NormSum &sum) {
    f32x2 acc[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] = pack2(0.0f, 0.0f);
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
        const f32x2 x = pack2(value_of<BF16>(raw, j), value_of<BF16>(raw, j + 1));
        acc[(j / 2) % 4] = fma2_rn(x, x, acc[(j / 2) % 4]);
    }
    float p[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) unpack2(acc[j], p[2 * j], p[2 * j + 1]);
    const float s = __fadd_rn(__fadd_rn(__fadd_rn(p[0], p[1]), __fadd_rn(p[2], p[3])),
                              __fadd_rn(__fadd_rn(p[4], p[5]), __fadd_rn(p[6], p[7])));
    if (s >= kSafeLow && s < kSafeHigh) {
        sum.add(s);
    } else {
        uint32_t bits = 0u;
#pragma unroll
        for (int j = 0; j < (BF16 ? 4 : 8); ++j) bits |= raw[j].x | raw[j].y | raw[j].z | raw[j].w;
        if ((bits & (BF16 ? 0x7FFF7FFFu : 0x7FFFFFFFu)) != 0u) {
#pragma unroll
            for (int j = 0; j < 32; ++j) {
                const double x = double(value_of<BF16>(raw, j));
                sum.rare = fma(x, x, sum.rare);
            }
        }
    }
}

// Sum over the CTA, in thread 0.  The same order every time.  Lanes are joined
// in fp32 with the errors kept; fp64 is left for one add per warp (GB300's fp64
// is slow enough that a tree over 256 threads costs microseconds).
__device__ __forceinline__ double block_sum(NormSum sum, double *scratch) {
    if (__any_sync(kFull, sum.rare != 0.0)) {  // (true for a NaN too)
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) sum.rare += __shfl_xor_sync(kFull, sum.rare, off);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        const float hi = __shfl_down_sync(kFull, sum.hi, off), lo = __shfl_down_sync(kFull, sum.lo, off);
        sum.add(hi);
        sum.lo = __fadd_rn(sum.lo, lo);
    }
    if ((threadIdx.x & 31) == 0)
        scratch[threadIdx.x >> 5] = double(sum.hi) + double(sum.lo) + sum.rare;
    __syncthreads();
    double total = 0.0;
    if (threadIdx.x == 0)
        for (int w = 0; w < kThreads / 32; ++w) total += scratch[w];
    return total;
}

template <int CAP>
__global__ void __launch_bounds__(kThreads, 4)
norm_partials_kernel(const __grid_constant__ SpanTable<CAP> t, double *__restrict__ partials) {
    __shared__ double scratch[kThreads / 32];
    // the clipping kernel may be scheduled now; it waits for this one's end
    let_successor_start();
    NormSum sum;
    for (uint32_t i = blockIdx.x; i < t.tiles; i += gridDim.x) {
        const Tile tile = find_tile(t, i);
        const void *src = t.src[tile.span];
        uint4 raw[kLoads];
        if (t.kind[tile.span] & 1) {
            load_tile<true>(src, tile.begin, tile.len, raw, false);
            add_squares<true>(raw, sum);
            add_squares<true>(raw + kLoads / 2, sum);
        } else {
            load_tile<false>(src, tile.begin, tile.len, raw, false);
            add_squares<false>(raw, sum);
        }
        if (threadIdx.x < tile.head) {
            const float x = (t.kind[tile.span] & 1)
                                ? bf16_bits_to_f32(static_cast<const uint16_t *>(src)[threadIdx.x])
                                : static_cast<const float *>(src)[threadIdx.x];
            sum.rare = fma(double(x), double(x), sum.rare);
        }
    }
    const double total = block_sum(sum, scratch);
    if (threadIdx.x == 0) partials[blockIdx.x] = total;
}

struct NormCoef {
    float norm, coef;
};

// The norm and the coefficient from the partials, the same in every CTA: the
// first warp adds them in order of their index modulo 32, then the lanes.
__device__ __forceinline__ NormCoef finish(const double *partials, int count, double max_norm,
                                           double eps, NormCoef *shared) {
    if (threadIdx.x < 32) {
        double v = 0.0;
#pragma unroll 8
        for (int i = threadIdx.x; i < count; i += 32) v += partials[i];
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(kFull, v, off);
        if (threadIdx.x == 0) {
            const double norm = sqrt(v), bound = norm + eps;
            shared->norm = float(norm);
            // (the first two also where the quotient would be inf / inf or 0 / 0; a norm
            // that is not a number stays one)
            shared->coef = norm == HUGE_VAL ? 0.0f : bound <= max_norm ? 1.0f : float(max_norm / bound);
        }
    }
    __syncthreads();
    return *shared;
}

__global__ void __launch_bounds__(kThreads)
norm_finish_kernel(const double *__restrict__ partials, int count, double max_norm, double eps,
                   int with_coef, float *__restrict__ stats) {
    __shared__ NormCoef shared;
    const NormCoef c = finish(partials, count, max_norm, eps, &shared);
    if (threadIdx.x == 0) {
        stats[0] = c.norm;
        if (with_coef) stats[1] = c.coef;
    }
}

__device__ __forceinline__ void store_one(void *dst, bool bf16, int64_t i, float x) {
    if (bf16) static_cast<uint16_t *>(dst)[i] = f32_to_bf16_bits(x);
    else static_cast<float *>(dst)[i] = x;
}

// 32 consecutive bytes in one store: two 16-byte ones would each write half of
// every 32-byte sector they touch.
__device__ __forceinline__ void store_f32x8(float *p, const float x[8]) {
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(x[0]),
                 "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7])
                 : "memory");
}

template <bool BF16>
__device__ __forceinline__ void scale_tile(const uint4 (&raw)[kLoads], const Tile &tile, void *dst,
                                           bool dst_bf16, float coef) {
    constexpr uint32_t W = BF16 ? 8 : 4;
    const uint32_t size = dst_bf16 ? 2u : 4u;
    char *base = static_cast<char *>(dst) + tile.begin * size;
    // one store per W values where the destination starts on a boundary too
    const bool vec = (reinterpret_cast<uintptr_t>(base) & (W * size - 1)) == 0;
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
        const uint32_t v = threadIdx.x + kThreads * j;
        float x[W];
#pragma unroll
        for (uint32_t e = 0; e < W; ++e) x[e] = __fmul_rn(value_of<BF16>(raw + j, e), coef);
        if (vec && (v + 1) * W <= tile.len) {
            if (dst_bf16) {
                uint32_t w[W / 2];
#pragma unroll
                for (uint32_t e = 0; e < W; e += 2) w[e / 2] = f32x2_to_bf16x2_bits(x[e], x[e + 1]);
                if constexpr (BF16)
                    __stcs(reinterpret_cast<uint4 *>(base) + v, make_uint4(w[0], w[1], w[2], w[3]));
                else
                    __stcs(reinterpret_cast<uint2 *>(base) + v, make_uint2(w[0], w[1]));
            } else if constexpr (BF16) {
                store_f32x8(reinterpret_cast<float *>(base) + v * W, x);
            } else {
                __stcs(reinterpret_cast<float4 *>(base) + v, make_float4(x[0], x[1], x[2], x[3]));
            }
        } else {
#pragma unroll
            for (uint32_t e = 0; e < W; ++e)
                if (v * W + e < tile.len) store_one(base, dst_bf16, v * W + e, x[e]);
        }
    }
}

// partials: of every launch of this call; write_stats: the first launch's.
template <int CAP>
__global__ void __launch_bounds__(kThreads, 4)
clip_kernel(const __grid_constant__ SpanTable<CAP> t, const double *__restrict__ partials,
            int count, double max_norm, double eps, float *__restrict__ stats, int in_place,
            int write_stats) {
    __shared__ NormCoef shared;
    // The norm's kernel only reads the gradients, so the first tile may be
    // fetched beside its end.
    Tile tile = find_tile(t, t.tiles - 1u - blockIdx.x);
    uint4 raw[kLoads];
    if (t.kind[tile.span] & 1) load_tile<true>(t.src[tile.span], tile.begin, tile.len, raw, true);
    else load_tile<false>(t.src[tile.span], tile.begin, tile.len, raw, true);
    wait_for_predecessor();
    const NormCoef c = finish(partials, count, max_norm, eps, &shared);
    if (write_stats && blockIdx.x == 0 && threadIdx.x == 0) {
        stats[0] = c.norm;
        stats[1] = c.coef;
    }
    if (in_place && c.coef == 1.0f) return;  // x * 1 = x, and it is there already
    for (uint32_t i = blockIdx.x; i < t.tiles; i += gridDim.x) {
        const void *src = t.src[tile.span];
        void *dst = t.dst[tile.span];
        const bool src_bf16 = t.kind[tile.span] & 1, dst_bf16 = (t.kind[tile.span] & 2) != 0;
        if (src_bf16) scale_tile<true>(raw, tile, dst, dst_bf16, c.coef);
        else scale_tile<false>(raw, tile, dst, dst_bf16, c.coef);
        if (threadIdx.x < tile.head) {
            const float x = src_bf16 ? bf16_bits_to_f32(static_cast<const uint16_t *>(src)[threadIdx.x])
                                     : static_cast<const float *>(src)[threadIdx.x];
            store_one(dst, dst_bf16, threadIdx.x, __fmul_rn(x, c.coef));
        }
        if (i + gridDim.x >= t.tiles) return;
        tile = find_tile(t, t.tiles - 1u - (i + gridDim.x));
        if (t.kind[tile.span] & 1) load_tile<true>(t.src[tile.span], tile.begin, tile.len, raw, true);
        else load_tile<false>(t.src[tile.span], tile.begin, tile.len, raw, true);
    }
}

constexpr int kSmallCap = 64, kLargeCap = kGradSpansPerLaunch;
static_assert(sizeof(SpanTable<kLargeCap>) < 32000, "kernel arguments end at 32764 bytes");

// Spans [first, first + count) with at least one value.
template <int CAP>
void fill(SpanTable<CAP> &t, const GradSpan *spans, int count) {
    t.count = 0;
    t.tiles = 0;
    for (int i = 0; i < count; ++i) {
        const GradSpan &s = spans[i];
        if (s.n == 0) continue;
        const int64_t rest = s.n - head_of(s.src, s.src_bf16, s.n);
        t.src[t.count] = s.src;
        t.dst[t.count] = s.dst;
        t.n[t.count] = s.n;
        t.kind[t.count] = uint8_t((s.src_bf16 ? 1 : 0) | (s.dst_bf16 ? 2 : 0));
        const int64_t most = tile_values(s.src_bf16);
        t.tiles += uint32_t(rest > 0 ? (rest + most - 1) / most : 1);
        t.tile_end[t.count] = t.tiles;
        ++t.count;
    }
}

uint32_t grid_of(uint32_t tiles) {
    return tiles < uint32_t(kGradPartialsPerLaunch) ? tiles : uint32_t(kGradPartialsPerLaunch);
}

template <int CAP>
cudaError_t launch_norm(const GradSpan *spans, int count, double *partials, int *used,
                        cudaStream_t stream) {
    SpanTable<CAP> t;
    fill(t, spans, count);
    if (t.tiles == 0) return cudaSuccess;
    const uint32_t grid = grid_of(t.tiles);
    norm_partials_kernel<CAP><<<grid, kThreads, 0, stream>>>(t, partials + *used);
    *used += int(grid);
    return cudaPeekAtLastError();
}

template <int CAP>
cudaError_t launch_clip(const GradSpan *spans, int count, const double *partials, int used,
                        double max_norm, double eps, float *stats, bool in_place, bool overlap,
                        int *write_stats, cudaStream_t stream) {
    SpanTable<CAP> t;
    fill(t, spans, count);
    if (t.tiles == 0) return cudaSuccess;
    const int first = *write_stats;
    *write_stats = 0;
    const uint32_t grid = grid_of(t.tiles);
    if (overlap)
        return launch_after(clip_kernel<CAP>, dim3(grid), dim3(kThreads), 0, stream, 1, t, partials, used,
                            max_norm, eps, stats, in_place ? 1 : 0, first);
    clip_kernel<CAP><<<grid, kThreads, 0, stream>>>(t, partials, used, max_norm, eps, stats,
                                                    in_place ? 1 : 0, first);
    return cudaPeekAtLastError();
}

}  // namespace

cudaError_t launch_grad_norm(const GradSpan *spans, int count, double *partials, bool clip,
                             bool in_place, double max_norm, double eps, float *stats,
                             cudaStream_t stream) {
    int used = 0;
    for (int at = 0; at < count; at += kLargeCap) {
        const int c = count - at < kLargeCap ? count - at : kLargeCap;
        const cudaError_t e = c <= kSmallCap
                                  ? launch_norm<kSmallCap>(spans + at, c, partials, &used, stream)
                                  : launch_norm<kLargeCap>(spans + at, c, partials, &used, stream);
        if (e != cudaSuccess) return e;
    }
    if (!clip || used == 0) {
        norm_finish_kernel<<<1, kThreads, 0, stream>>>(partials, used, max_norm, eps, clip ? 1 : 0,
                                                       stats);
        return cudaPeekAtLastError();
    }
    // With one launch of each kernel the second may start early; a second pair
    // would have to wait for all first ones.
    const bool overlap = count <= kLargeCap;
    int write_stats = 1;
    for (int at = 0; at < count; at += kLargeCap) {
        const int c = count - at < kLargeCap ? count - at : kLargeCap;
        const cudaError_t e =
            c <= kSmallCap ? launch_clip<kSmallCap>(spans + at, c, partials, used, max_norm, eps,
                                                    stats, in_place, overlap, &write_stats, stream)
                           : launch_clip<kLargeCap>(spans + at, c, partials, used, max_norm, eps,
                                                    stats, in_place, overlap, &write_stats, stream);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace wc
