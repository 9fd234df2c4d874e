// cross_entropy.cu -- softmax cross entropy of a linear output layer over a large
// vocabulary, and its gradient, in pieces of the vocabulary and without keeping
// the logits.
//
//   s[t][v]  = x[t] . w[v],   lse[t] = log sum over v of exp(s[t][v])
//   loss[t]  = lse[t] - s[t][y(t)]
//   d[t][v]  = g[t] (exp(s[t][v] - lse[t]) - [v = y(t)])
//   dx = d w,   dw = d^T x
//
// Forward: tiles of 256 tokens by 256 rows of w on the tensor cores.  A tile's
// epilogue reduces its logits, as they leave the tensor memory, to each token's
// maximum and sum of exponentials over 128 columns, its target left out; a second
// kernel joins those with the target's logit, as log1p(sum over v != y of
// exp(s[t][v] - s[t][y])).
// Backward: for one piece of the vocabulary after the other, the logits once
// more, whose epilogue writes d (bf16, its only rounding) to a buffer, and one
// launch for the two products that read it, dx summed over the pieces in fp32.  A g
// that is the same for all tokens multiplies the products instead: in d it would
// move every target's d, near -1 for all that the model does not know, off a value
// that bf16 holds, in the same direction (up to 2^-8 of the gradient).
// So a pass multiplies four times where one that keeps T x V logits multiplies
// three times.
// Up to four tokens have kernels of their own for the logits of both directions, on the
// ordinary cores with one reading of w.
//
// Both directions sum a logit in the same order, whatever kernel it is: a difference would
// be in d's exponent, and at logits of 1e6 the rounding of a sum is some tenths.  So a column
// that decides a row has d = g there, however large its logit is.  lse is one fp32 number, and
// each d carries its rounding, |lse| 2^-24 of d.
//
// One kernel does all products (bf16 operands, fp32 sums): pairs of SMs
// (cta_group::2) on tiles of 256 x 256, 64 values of K to a stage.  Operands come
// by TMA as they lie: those whose rows run along K are K-major (logits, d in
// dx), the others MN-major (w in dx, d and x in dw), so nothing is transposed.
// Warps 0-7 are the epilogue, 8 brings operands, 9 multiplies; two tiles' sums
// fit the tensor memory, so a tile's epilogue runs beside the next tile's
// products.
//
// The tensor core cuts sums off where fp32 would round them, so logits come out
// nearer to 0 by some 2^-25 of themselves for each 16 values of K (D = 2048: 8e-6
// for a logit of 4).  So it sums 1024 values of K at a time, and the epilogue adds
// those sums up, rounded (losses of 64 x 8000 x 4096: 6.4e-6 off rms without, 1.5e-6
// with it).  What is left largely cancels over the vocabulary; a target's logit
// stands alone, so it is summed by itself in fp32 (warps 10 and 11 of the forward
// pass, the kernel that lays x out in the backward pass), and d of a target
// is expm1(s[t][y] - lse[t]).  (Losses of 8192 x 32000 x 2048: 8.1e-6 off rms with the
// tensor core's target, 1.8e-6 with one chunk, 0.9e-6 with both.)
#include <atomic>
#include <type_traits>

#include "wc_device.cuh"
#include "wc_internal.h"
#include "wc_launch.cuh"
#include "wc_rows.cuh"
#include "wc_store.cuh"
#include "wc_tcgen05.cuh"
#include "wc_wait.cuh"

namespace wc {

namespace {

__device__ unsigned int g_wait_timeouts;

// A warp that gives up takes no further part: it arrives on no barrier and starts
// no copy or product, the others run out in turn, and every output that misses a
// sum is NaN.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity) {
    return wc::mbar_wait(bar, parity, &g_wait_timeouts);
}

constexpr int kSms = 152;
constexpr int kHalf = 128;                  // rows of an operand that a CTA brings
constexpr int kTile = 2 * kHalf;
constexpr int kDepth = 64;                  // values of K in a stage
constexpr int kOperand = kHalf * kDepth * 2;
constexpr int kStageBytes = 2 * kOperand;
constexpr int kStages = 6;
constexpr int kBuffers = 2;                 // tiles of sums in tensor memory
constexpr int kEpilogueWarps = 8, kProducer = 8, kMma = 9, kTargets = 10, kWarps = 12;
constexpr int kThreads = kWarps * 32;
constexpr int kSmem = kStages * kStageBytes + kEpilogueWarps * kStagingBytes + 1024;

constexpr float kLog2E = 1.44269504088896340736f;

// exp(x).  Of a difference of logits: the difference comes first, exact where the two
// are near, and then the factor log2 e.  The other way round, with a rounded product
// log2 e * maximum to subtract, even the maximum's own exponential is off by that
// rounding, however large the logits are (9 % at 1e6, 0 or infinity from 4e9 on).
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float exp_of(float x) { return ex2(__fmul_rn(x, kLog2E)); }

// exp_of(v + add), the same bits, for the two encodings at v (the epilogues' instructions
// show where K is short: losses of 8192 x 32000 x 512 one at a time 257 us, so 247).
__device__ __forceinline__ void exp_of_two(const uint32_t *v, f32x2 add, float &x, float &y) {
    const f32x2 less = fma2_rn(pack2(__uint_as_float(v[0]), __uint_as_float(v[1])), pack2(1.0f, 1.0f), add);
    unpack2(fma2_rn(less, pack2(kLog2E, kLog2E), pack2(-0.0f, -0.0f)), x, y);
    x = ex2(x);
    y = ex2(y);
}
__device__ __forceinline__ float nan32() { return __uint_as_float(0x7FC00000u); }

// One product C[i][j] = sum over k of A[i][k] B[j][k].
struct Job {
    int32_t tiles_i, tiles_j;
    int32_t width;          // columns of a tile: 256, 128 or (K-major B) 192, 64
    int32_t split;          // parts of K with sums of their own
    int32_t blocks;         // of K
    int32_t chunks;         // LONG: of a tile's K, each summed by itself
    int32_t rows_i, rows_j;
    int32_t box_i;          // rows of A in a copy: 128, or fewer if there are fewer
    int32_t mn_i, mn_j;     // MN-major: rows of the operand are contiguous in memory
    int32_t j_at, kj_at;    // where B's rows and its K begin in its matrix
    // what becomes of a product: out [split][rows_i][ld], added to what `add` holds
    void *out;
    const void *add;
    int64_t ld_out, ld_add, split_out, split_add;
    int32_t out_bf16, add_bf16, vec;
    float alpha;            // factor of the product
};

struct Args {
    Job job[2];
    int32_t units[2];       // tiles x split
    int32_t sooner;         // see unit_of
    // of the logits' epilogues
    const void *targets;
    int32_t wide;           // 64-bit targets
    int32_t V;
    float2 *parts;          // [2 tiles_j][rows_i]: maximum, sum of exponentials less it
    float *target_logit;    // [rows_i]
    const uint16_t *x, *w;  // for it, as they were given; x NULL if it is there
    int64_t ld_x, ld_w;
    int32_t D;
    const float *lse, *dlosses;
};

enum Mode { kStats, kGradient, kProducts };

// Row of w that token t is to predict, or -1.
__device__ __forceinline__ int32_t target_of(const void *targets, int wide, int32_t V, int64_t t) {
    const int64_t y = wide ? static_cast<const int64_t *>(targets)[t] : int64_t(static_cast<const int32_t *>(targets)[t]);
    return y >= 0 && y < V ? int32_t(y) : -1;
}

__device__ __forceinline__ float dot8(const uint4 &a, const uint4 &b, float sum) {
    const uint32_t u[4] = {a.x, a.y, a.z, a.w}, v[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        sum = __fmaf_rn(__uint_as_float(u[k] << 16), __uint_as_float(v[k] << 16), sum);
        sum = __fmaf_rn(__uint_as_float(u[k] & 0xFFFF0000u), __uint_as_float(v[k] & 0xFFFF0000u), sum);
    }
    return sum;
}

// A row of a bf16 matrix that starts on any value.
struct Row {
    const uint16_t *p, *end;  // of the row, of the matrix
    int32_t D;
};

__device__ __forceinline__ Row row_of(const uint16_t *p, int64_t ld, int64_t rows, int32_t D, int64_t r) {
    return {p + r * ld, p + (rows - 1) * ld + D, D};
}

// Eight values each from N places of a matrix that ends at `end`, the n[k] first of them
// (the rest 0; none if n[k] <= 0).  All loads are under way at once: one place after
// the other waits for each (1 x 32001 x 2047 81 us, so 40).
template <int N>
__device__ __forceinline__ void values_at(const uint16_t *const (&at)[N], const int32_t (&n)[N], const uint16_t *end,
                                          uint4 (&q)[N]) {
    bool direct = true, inside = true;  // all on 16 bytes; whole chunks end inside the matrix
#pragma unroll
    for (int k = 0; k < N; ++k) {
        direct = direct && (reinterpret_cast<uintptr_t>(at[k]) & 15u) == 0 && n[k] >= 8;
        inside = inside && end - at[k] >= 16;
    }
    if (direct) {
#pragma unroll
        for (int k = 0; k < N; ++k) q[k] = __ldg(reinterpret_cast<const uint4 *>(at[k]));
        return;
    }
    uint32_t w[N][4];
    if (inside) {
        uint32_t t[N][8];
#pragma unroll
        for (int k = 0; k < N; ++k) load_chunks(at[k], t[k]);
#pragma unroll
        for (int k = 0; k < N; ++k) {
            shift_words(at[k], t[k], w[k]);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                w[k][j] = 2 * j + 1 < n[k] ? w[k][j] : 2 * j < n[k] ? w[k][j] & 0xFFFFu : 0u;
        }
    } else {
#pragma unroll
        for (int k = 0; k < N; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t lo = 2 * j < n[k] ? at[k][2 * j] : 0u, hi = 2 * j + 1 < n[k] ? at[k][2 * j + 1] : 0u;
                w[k][j] = lo | hi << 16;
            }
    }
#pragma unroll
    for (int k = 0; k < N; ++k) q[k] = make_uint4(w[k][0], w[k][1], w[k][2], w[k][3]);
}

// The same of row[k] at d + k * step.  (Places past a row's end are read at its start.)
template <int N>
__device__ __forceinline__ void values_at(const Row (&row)[N], int32_t d, int32_t step, uint4 (&q)[N]) {
    const uint16_t *at[N];
    int32_t n[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
        n[k] = row[k].D - (d + k * step);
        at[k] = row[k].p + (n[k] > 0 ? d + k * step : 0);
    }
    values_at(at, n, row[0].end, q);
}

// A warp's sum over D of x[d] w[d], in fp32, the same in every lane.
__device__ __forceinline__ float row_dot(const Row &x, const Row &w, int lane) {
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    const Row xs[4] = {x, x, x, x}, ws[4] = {w, w, w, w};
    int32_t d = 0;
    for (; d + 256 < x.D; d += 1024) {
        uint4 a[4], b[4];
        values_at(xs, d + 8 * lane, 256, a);
        values_at(ws, d + 8 * lane, 256, b);
#pragma unroll
        for (int k = 0; k < 4; ++k) s[k] = dot8(a[k], b[k], s[k]);
    }
    if (d < x.D) {  // (at most 256 values)
        const Row x1[1] = {x}, w1[1] = {w};
        uint4 a[1], b[1];
        values_at(x1, d + 8 * lane, 0, a);
        values_at(w1, d + 8 * lane, 0, b);
        s[0] = dot8(a[0], b[0], s[0]);
    }
    float sum = __fadd_rn(__fadd_rn(s[0], s[1]), __fadd_rn(s[2], s[3]));
#pragma unroll
    for (int o = 16; o > 0; o /= 2) sum = __fadd_rn(sum, __shfl_xor_sync(kFull, sum, o));
    return sum;
}

// Tile order: bands of tiles of i, all of j within a band, so that the CTAs at work
// together share operand rows in L2.  Where j has few tiles a band is no higher than
// that all of them are at work at once (16 tiles high, the gradients' products of
// 8192 x 32000 x 2048 read 1.67 GB from memory for each piece, so 1.40: 585 -> 575 us).
__device__ __forceinline__ void tile_at(const Job &a, int32_t t, int32_t *ti, int32_t *tj) {
    const int32_t height = a.tiles_j >= 16 ? 16 : kSms / 2 / a.tiles_j;
    const int32_t band = t / (height * a.tiles_j);
    const int32_t first = band * height;
    const int32_t high = min(height, a.tiles_i - first);
    const int32_t in = t - band * height * a.tiles_j;
    *ti = first + in % high;
    *tj = in / high;
}

// Number of the unit that a pair of SMs works on as its i-th, of `pairs`; past all
// units there is none.  Job 0's units, which may be much longer, are dealt first.  Some
// pairs then have one less than others; those get the `sooner` units of job 1 that
// take about as long, and the rest is dealt to all.  (8192 x 32000 x 2048: dealing all in
// turn leaves some pairs 5 % more than the mean.)
template <Mode MODE>
__device__ __forceinline__ int32_t unit_of(const Args &a, int32_t pair, int32_t i, int32_t pairs) {
    if (MODE != kProducts) return pair + i * pairs;
    const int32_t more = a.units[0] % pairs, of_0 = a.units[0] / pairs + (pair < more ? 1 : 0);
    if (i < of_0) return pair + i * pairs;
    i -= of_0;
    const int32_t early = more > 0 ? pairs - more : 0;
    if (early > 0 && pair >= more) {
        if (i < a.sooner) return a.units[0] + pair - more + i * early;
        i -= a.sooner;
    }
    return a.units[0] + a.sooner * early + pair + i * pairs;
}

struct Unit {
    int32_t job, ti, tj, part, block0, blocks;
};
template <Mode MODE>
__device__ __forceinline__ Unit unit_at(const Args &a, int32_t u) {
    Unit r;
    r.job = MODE == kProducts && u >= a.units[0] ? 1 : 0;
    const Job &j = a.job[r.job];
    if (r.job) u -= a.units[0];
    const int32_t tile = MODE == kProducts ? u / j.split : u;
    r.part = MODE == kProducts ? u - tile * j.split : 0;
    tile_at(j, tile, &r.ti, &r.tj);
    r.block0 = MODE == kProducts ? int32_t(int64_t(j.blocks) * r.part / j.split) : 0;
    r.blocks = MODE == kProducts ? int32_t(int64_t(j.blocks) * (r.part + 1) / j.split) - r.block0 : j.blocks;
    return r;
}

// `rows` (128, or B's of a narrow tile) x 64 of K of an operand, to up to 16 KB of shared
// memory with 128-byte swizzle: K-major lines of 64 values of K, MN-major 64 lines
// (one per k) of 64 rows, then those of the next 64 rows.
__device__ __forceinline__ void load_operand(uint32_t to, const CUtensorMap *map, uint32_t bar, int mn, int32_t rows,
                                             int32_t row, int32_t k) {
    if (mn) {
        tma_load<true>(to, map, bar, row, k);
        if (rows > 64) tma_load<true>(to + kOperand / 2, map, bar, row + 64, k);
    } else {
        tma_load<true>(to, map, bar, k, row);
    }
}

// Shared-memory operand descriptor (addresses and strides in 16-byte units; bit 46
// is its version, 2 << 61 the 128-byte swizzle).  Groups of 8 lines are 1024 bytes
// apart: K-major of rows, MN-major of k, whose two halves of 64 rows are 8 KB apart.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, int mn) {
    return uint64_t((addr & 0x3FFFFu) >> 4) | (uint64_t(mn ? kOperand / 2 / 16 : 1) << 16) | (uint64_t(64) << 32) |
           (uint64_t(1) << 46) | (uint64_t(2) << 61);
}

// Instruction descriptor: fp32 sums, bf16 x bf16, 256 x width.
__device__ __forceinline__ uint32_t instr_desc(int mn_i, int mn_j, int width) {
    return (1u << 4) | (1u << 7) | (1u << 10) | (uint32_t(mn_i) << 15) | (uint32_t(mn_j) << 16) |
           (uint32_t(width >> 3) << 17) | (uint32_t(kTile >> 4) << 24);
}

__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t add) {
    asm volatile(
        "{\n.reg .pred p;\n"
        "setp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(add)
        : "memory");
}

// ---------------------------------------------------------------------------
// epilogues: a warp's 32 rows x 32 columns, one row per lane
// ---------------------------------------------------------------------------

// The running maximum and sum of a row, of exponentials of the differences to it.  A row
// without columns, or with impossible ones alone, is (-infinity, 0); a sum of NaN stays.
struct Running {
    float top, sum;
};

// What is subtracted: the maximum, or 0 where every exponential is 0.
__device__ __forceinline__ float base_of(float top) { return top == -INFINITY ? 0.0f : top; }

// cols: columns of these that exist (at least 1).
__device__ __forceinline__ void stats(Running &r, uint32_t (&v)[32], int cols) {
    if (cols < 32) {
#pragma unroll
        for (int c = 0; c < 32; ++c)
            if (c >= cols) v[c] = 0xFF800000u;  // -infinity
    }
    float m[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) m[c] = __uint_as_float(v[c]);
#pragma unroll
    for (int c = 4; c < 32; ++c) m[c & 3] = fmaxf(m[c & 3], __uint_as_float(v[c]));
    const float top = fmaxf(r.top, fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])));
    const float from = -base_of(top);
    float s[4] = {__fmul_rn(r.sum, exp_of(__fadd_rn(r.top, from))), 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < 32; c += 2) {
        float x, y;
        exp_of_two(v + c, pack2(from, from), x, y);
        s[c & 3] = __fadd_rn(s[c & 3], x);
        s[(c + 1) & 3] = __fadd_rn(s[(c + 1) & 3], y);
    }
    r.top = top;
    r.sum = __fadd_rn(__fadd_rn(s[0], s[1]), __fadd_rn(s[2], s[3]));
}

// Two parts of a row.
__device__ __forceinline__ float2 joined_stats(float2 a, float2 b) {
    const float top = fmaxf(a.x, b.x);
    const float x = a.x == -INFINITY ? a.y : __fmul_rn(a.y, exp_of(__fadd_rn(a.x, -top)));
    const float y = b.x == -INFINITY ? b.y : __fmul_rn(b.y, exp_of(__fadd_rn(b.x, -top)));
    return make_float2(top, __fadd_rn(x, y));
}

// 32 rows of 64 bytes, staged one per lane, to rows `pitch` bytes apart: 64
// consecutive bytes of 8 rows at a time.
__device__ __forceinline__ void store_staged(const uint8_t *staging, char *base, int64_t pitch, int rows, int lane) {
    const int seg = (lane & 3) * 16;
#pragma unroll
    for (int r = lane >> 2; r < 32; r += 8)
        if (r < rows)
            *reinterpret_cast<uint4 *>(base + r * pitch + seg) =
                *reinterpret_cast<const uint4 *>(staging + r * kStagingPitch + seg);
}

__device__ __forceinline__ void stage_bf16(uint8_t *staging, const float (&x)[32], int lane) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = f32x2_to_bf16x2_bits(x[8 * q + 2 * k], x[8 * q + 2 * k + 1]);
        *reinterpret_cast<uint4 *>(staging + lane * kStagingPitch + q * 16) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// A product's sums.  (row0, col0): the first row of the warp, the first column.
__device__ __forceinline__ void store_sums(const Job &a, int32_t part, const float (&x)[32], uint8_t *staging,
                                           int32_t row0, int32_t col0, int lane) {
    const int rows = a.rows_i - row0, cols = a.rows_j - col0;
    if (rows <= 0 || cols <= 0) return;
    if (a.out_bf16 && a.add == nullptr && a.vec && cols >= 32) {
        stage_bf16(staging, x, lane);
        __syncwarp();
        store_staged(staging, static_cast<char *>(a.out) + (int64_t(row0) * a.ld_out + col0) * 2, a.ld_out * 2, rows, lane);
        __syncwarp();
        return;
    }
    if (a.out_bf16 && a.add == nullptr) {
        stage_bf16(staging, x, lane);
        __syncwarp();
        store_pass_bf16(static_cast<char *>(a.out) + (int64_t(row0) * a.ld_out + col0) * 2, a.ld_out, staging, rows,
                        min(cols, 32), lane);
        __syncwarp();
        return;
    }
    // 16 columns of fp32 at a time
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
            *reinterpret_cast<float4 *>(staging + lane * kStagingPitch + q * 16) =
                make_float4(x[16 * h + 4 * q], x[16 * h + 4 * q + 1], x[16 * h + 4 * q + 2], x[16 * h + 4 * q + 3]);
        __syncwarp();
        const int left = cols - 16 * h;
        const int64_t at = part * a.split_out + int64_t(row0) * a.ld_out + col0 + 16 * h;
        if (!a.out_bf16 && !a.add_bf16 && a.vec && left >= 16) {
            float *out = static_cast<float *>(a.out) + at + 4 * (lane & 3);
            const float *add = static_cast<const float *>(a.add);
            if (add) add += part * a.split_add + int64_t(row0) * a.ld_add + col0 + 16 * h + 4 * (lane & 3);
            float4 old[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int r = (lane >> 2) + 8 * k;
                old[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (add && r < rows) old[k] = *reinterpret_cast<const float4 *>(add + r * a.ld_add);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int r = (lane >> 2) + 8 * k;
                float4 v = *reinterpret_cast<const float4 *>(staging + r * kStagingPitch + (lane & 3) * 16);
                if (add) v = make_float4(__fadd_rn(old[k].x, v.x), __fadd_rn(old[k].y, v.y), __fadd_rn(old[k].z, v.z),
                                         __fadd_rn(old[k].w, v.w));
                if (r < rows) *reinterpret_cast<float4 *>(out + r * a.ld_out) = v;
            }
        } else if (a.add == a.out && a.out_bf16) {
            store_pass_f32<true>(static_cast<uint16_t *>(a.out) + at, a.ld_out, staging, rows, left, lane);
        } else if (a.add == a.out) {
            store_pass_f32<true>(static_cast<float *>(a.out) + at, a.ld_out, staging, rows, left, lane);
        } else if (a.add == nullptr) {
            store_pass_f32<false>(static_cast<float *>(a.out) + at, a.ld_out, staging, rows, left, lane);
        } else {  // fp32 sums of earlier pieces, then to out
            const float *add = static_cast<const float *>(a.add) + part * a.split_add + int64_t(row0) * a.ld_add + col0 + 16 * h;
            const int c = lane & 15;
            if (c < left) {
#pragma unroll 8
                for (int r = lane >> 4; r < 32; r += 2) {
                    if (r >= rows) break;
                    const float y = __fadd_rn(add[r * a.ld_add + c],
                                              *reinterpret_cast<const float *>(staging + r * kStagingPitch + 4 * c));
                    if (a.out_bf16) static_cast<uint16_t *>(a.out)[at + r * a.ld_out + c] = f32_to_bf16_bits(y);
                    else static_cast<float *>(a.out)[at + r * a.ld_out + c] = y;
                }
            }
        }
        __syncwarp();
    }
}

// ---------------------------------------------------------------------------
// kernel
// ---------------------------------------------------------------------------

// LONG: products whose K is summed in several chunks (of all of them, or of one job's).  The tensor core's sums of a chunk
// leave the tensor memory as soon as it is complete and are added up, rounded, in the
// epilogue's registers, so that what is cut off does not grow with K.  For those
// 128 sums of a thread the epilogue takes registers over from the other four warps.
template <Mode MODE, bool LONG>
__global__ void __launch_bounds__(kThreads, 1)
product_kernel(const __grid_constant__ CUtensorMap map_i0, const __grid_constant__ CUtensorMap map_j0,
               const __grid_constant__ CUtensorMap map_i1, const __grid_constant__ CUtensorMap map_j1,
               const __grid_constant__ Args a) {
    // LONG: registers of a thread of the epilogue and of the others, 384 x 168 in all as at
    // the launch (those that neither side spills)
    constexpr int kTaken = MODE == kStats ? 208 : 224, kGiven = 3 * 168 - 2 * kTaken;
    extern __shared__ uint8_t dynamic_smem[];
    // full: a stage's operands are here (both CTAs', counted in the first one).
    // empty: its products have ended.  sums: a tile is complete.  taken: its
    // sums have been read (both CTAs', counted in the first one).
    __shared__ uint64_t full[kStages], empty[kStages], sums[kBuffers], taken[kBuffers], drained;
    __shared__ uint32_t tmem_slot;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t stages = (smem_of(dynamic_smem) + 1023u) & ~1023u;
    const int32_t rank = int32_t(blockIdx.x & 1);
    const int32_t pair = int32_t(blockIdx.x >> 1), pairs = int32_t(gridDim.x >> 1);
    const int32_t units = a.units[0] + (MODE == kProducts ? a.units[1] : 0);

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_of(&full[s]), 1);
            mbar_init(smem_of(&empty[s]), 1);
        }
        for (int b = 0; b < kBuffers; ++b) {
            mbar_init(smem_of(&sums[b]), 1);
            mbar_init(smem_of(&taken[b]), 2 * kEpilogueWarps);
        }
        mbar_init(smem_of(&drained), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    __syncwarp();
    if (warp == kMma) tmem_alloc<true>(smem_of(&tmem_slot), kBuffers * kTile);
    tc_before_sync();
    __syncthreads();
    cluster_sync();  // the other CTA's barriers are ready too
    tc_after_sync();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(&tmem_slot);
    wait_for_predecessor();  // all above is set-up that reads no operand
    let_successor_start();   // (its CTAs find room as these end)

    // The targets' logits: two warps of each CTA, ten of one without tiles.
    auto targets = [&](int32_t of_cta, bool idle) {
        const int32_t busy = min(int32_t(gridDim.x), 2 * units), cta = int32_t(blockIdx.x);
        const int32_t mine = idle ? 2 * busy + 10 * (cta - busy) + of_cta : 2 * cta + of_cta;
        const int32_t all = 2 * busy + 10 * (int32_t(gridDim.x) - busy), T = a.job[0].rows_i;
        for (int32_t t = mine; t < T; t += all) {
            const int32_t y = target_of(a.targets, a.wide, a.V, t);
            if (y < 0) continue;
            const float s = row_dot(row_of(a.x, a.ld_x, T, a.D, t), row_of(a.w, a.ld_w, a.V, a.D, y), lane);
            if (lane == 0) a.target_logit[t] = s;
        }
    };
    const bool has_targets = MODE == kStats && a.x != nullptr, idle = int32_t(blockIdx.x) >= 2 * units;

    if (warp >= kEpilogueWarps) {
        if (LONG) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kGiven));
        if (warp == kProducer) {
            uint32_t stage = 0, phase = 0;
            bool ok = true;
            for (int32_t i = 0, t; ok && (t = unit_of<MODE>(a, pair, i, pairs)) < units; ++i) {
                const Unit u = unit_at<MODE>(a, t);
                const Job &job = a.job[u.job];
                const CUtensorMap *map_i = u.job ? &map_i1 : &map_i0, *map_j = u.job ? &map_j1 : &map_j0;
                const int32_t half = job.width / 2;
                // (rows of A past its box are not brought: what the tensor core makes of those that
                // lie there is not looked at)
                const uint32_t bytes = (2 * job.box_i + job.width) * kDepth * 2;
                const int32_t row_i = u.ti * kTile + rank * kHalf, row_j = job.j_at + u.tj * job.width + rank * half;
                for (int32_t b = 0; b < u.blocks; ++b) {
                    ok = mbar_wait(smem_of(&empty[stage]), phase ^ 1u);
                    if (!ok) break;
                    if (elected()) {
                        const uint32_t local = smem_of(&full[stage]), bar = in_cta(local, 0);
                        const uint32_t base = stages + stage * kStageBytes;
                        const int32_t k = (u.block0 + b) * kDepth;
                        if (rank == 0) mbar_expect(local, bytes);
                        load_operand(base, map_i, bar, job.mn_i, kHalf, row_i, k);
                        load_operand(base + kOperand, map_j, bar, job.mn_j, half, row_j, job.kj_at + k);
                    }
                    __syncwarp();
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (!ok) wait_ms(20);  // for the copies in flight to land before the CTA goes
        } else if (warp == kMma && rank == 0) {
            uint32_t stage = 0, phase = 0, buf = 0, buf_phase = 0;
            bool ok = true;
            const bool lead = elected();
            for (int32_t i = 0, t; ok && (t = unit_of<MODE>(a, pair, i, pairs)) < units; ++i) {
                const Unit u = unit_at<MODE>(a, t);
                const Job &job = a.job[u.job];
                const uint32_t idesc = instr_desc(job.mn_i, job.mn_j, job.width);
                // 16 values of K on: 32 bytes of every line, or 16 lines
                const uint64_t step_i = job.mn_i ? 128 : 2, step_j = job.mn_j ? 128 : 2;
                const int32_t chunks = LONG ? job.chunks : 1;
                for (int32_t part = 0, b = 0; part < chunks; ++part) {
                    const int32_t first = b, end = LONG ? int32_t(int64_t(u.blocks) * (part + 1) / chunks) : u.blocks;
                    ok = mbar_wait(smem_of(&taken[buf]), buf_phase ^ 1u);
                    if (!ok) break;
                    tc_after_sync();
                    for (; b < end; ++b) {
                        ok = mbar_wait(smem_of(&full[stage]), phase);
                        if (!ok) break;
                        tc_after_sync();
                        if (lead) {
                            const uint32_t base = stages + stage * kStageBytes;
                            uint64_t di = smem_desc(base, job.mn_i), dj = smem_desc(base + kOperand, job.mn_j);
#pragma unroll
                            for (int k = 0; k < kDepth / 16; ++k) {
                                mma(tmem + buf * kTile, di, dj, idesc, b > first || k > 0);
                                di += step_i;
                                dj += step_j;
                            }
                            mma_commit<true>(smem_of(&empty[stage]));
                        }
                        __syncwarp();
                        if (++stage == kStages) {
                            stage = 0;
                            phase ^= 1u;
                        }
                    }
                    if (!ok) break;
                    if (lead) mma_commit<true>(smem_of(&sums[buf]));
                    __syncwarp();
                    if (++buf == kBuffers) {
                        buf = 0;
                        buf_phase ^= 1u;
                    }
                }
            }
            // No product may be in flight when the tensor memory is freed.
            if (pair < units) {
                if (lead) mma_commit<true>(smem_of(&drained), 1);
                __syncwarp();
                mbar_wait(smem_of(&drained), 0);
            }
        } else if (warp >= kTargets && has_targets) {
            targets(warp - kTargets, idle);
        }
    } else {
        if (LONG) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kTaken));
        const int group = warp >> 2;
        uint8_t *const staging = dynamic_smem + (stages - smem_of(dynamic_smem)) + kStages * kStageBytes + warp * kStagingBytes;
        const uint32_t taken0 = in_cta(smem_of(&taken[0]), 0);
        uint32_t buf = 0, phase = 0;
        bool ok = true;
        for (int32_t i = 0, t; (t = unit_of<MODE>(a, pair, i, pairs)) < units; ++i) {
            const Unit u = unit_at<MODE>(a, t);
            const Job &job = a.job[u.job];
            const int32_t row0 = u.ti * kTile + rank * kHalf + (warp & 3) * 32, row = row0 + lane;
            const int32_t half = job.width / 2, col0 = u.tj * job.width + group * half;
            const uint32_t of_group = tmem + (uint32_t(warp & 3) << 21) + group * half;
            const bool live = row < job.rows_i;
            // (columns of this group that exist)
            const int32_t cols = max(0, min(job.rows_j - col0, half));
            int32_t target = -1;  // its column in this group, or any number outside
            bool padding = true;
            float lse = 0.0f, g = 0.0f, own = 0.0f;  // own: d of the target
            if (MODE != kProducts && live) {
                const int32_t y = target_of(a.targets, a.wide, a.V, row);
                padding = y < 0;
                if (!padding) target = y - job.j_at - col0;
                if (MODE == kGradient && !padding) {
                    lse = a.lse[row];
                    g = a.dlosses ? a.dlosses[row] : 1.0f;
                    own = __fmul_rn(g, expm1f(__fadd_rn(a.target_logit[row], -lse)));
                }
            }
            const int last = padding ? 0 : cols;  // of the columns with a gradient
            // LONG: the chunks' sums, each of which leaves the tensor memory at once
            float all[LONG ? kHalf : 1];
            auto take = [&](auto first) {
                if (ok) ok = mbar_wait(smem_of(&sums[buf]), phase);
                if (!ok) return;
                tc_after_sync();
#pragma unroll
                for (int c = 0; c < kHalf; c += 32) {
                    if (c >= half) break;
                    uint32_t w[32];
                    tmem_load(of_group + buf * kTile + c, w);
                    tmem_wait(w);
#pragma unroll
                    for (int k = 0; k < 32; ++k) {
                        const float x = __uint_as_float(w[k]);
                        float &sum = all[LONG ? c + k : 0];
                        sum = decltype(first)::value ? x : __fadd_rn(sum, x);
                    }
                }
                tc_before_sync();
                __syncwarp();
                if (elected()) mbar_arrive_cluster(taken0 + buf * 8);
                if (++buf == kBuffers) {
                    buf = 0;
                    phase ^= 1u;
                }
            };
            if (LONG) {
                take(std::true_type());
                for (int32_t part = 1; part < job.chunks; ++part) take(std::false_type());
            }
            const uint32_t from = of_group + buf * kTile;
            if (!LONG && ok) ok = mbar_wait(smem_of(&sums[buf]), phase);
            if (!LONG) tc_after_sync();
            Running run = {-INFINITY, 0.0f};
            uint32_t v[2][32];
            if (!LONG && ok) {
                tmem_load(from, v[0]);
                tmem_wait(v[0]);
            }
#pragma unroll
            for (int c = 0; c < kHalf; c += 32) {
                if (c >= half) break;
                uint32_t(&w)[32] = v[LONG ? 0 : (c / 32) & 1];
                if (!ok) {
#pragma unroll
                    for (int k = 0; k < 32; ++k) w[k] = 0x7FC00000u;
                } else if (LONG) {
#pragma unroll
                    for (int k = 0; k < 32; ++k) w[k] = __float_as_uint(all[LONG ? c + k : 0]);
                } else if (c + 32 < half) {
                    tmem_load(from + c + 32, v[(c / 32 + 1) & 1]);
                } else {
                    tc_before_sync();  // all read: the next tile may have the buffer
                    __syncwarp();
                    if (elected()) mbar_arrive_cluster(taken0 + buf * 8);
                }
                if (MODE == kStats) {
                    if (c < cols) {
                        const int at = target - c;
                        if (__any_sync(kFull, at >= 0 && at < 32)) {
#pragma unroll
                            for (int k = 0; k < 32; ++k) w[k] = at == k ? 0xFF800000u : w[k];  // -infinity
                        }
                        stats(run, w, cols - c);
                    }
                } else if (MODE == kGradient) {
                    float x[32];
#pragma unroll
                    for (int k = 0; k < 32; k += 2) {
                        exp_of_two(w + k, pack2(-lse, -lse), x[k], x[k + 1]);
                        x[k] = __fmul_rn(g, x[k]);
                        x[k + 1] = __fmul_rn(g, x[k + 1]);
                    }
                    if (__any_sync(kFull, padding || (target >= c && target < c + 32) || last < c + 32)) {
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            // (padding tokens have no gradient whatever their logits are)
                            x[k] = c + k >= last ? 0.0f : target - c == k ? own : x[k];
                    }
                    if (col0 + c < job.ld_out) {  // (tiles of 192 columns may go past the buffer's rows)
                        stage_bf16(staging, x, lane);
                        __syncwarp();
                        store_staged(staging, static_cast<char *>(job.out) + (int64_t(row0) * job.ld_out + col0 + c) * 2,
                                     job.ld_out * 2, job.rows_i - row0, lane);
                        __syncwarp();
                    }
                } else {
                    float x[32];
#pragma unroll
                    for (int k = 0; k < 32; ++k) x[k] = __fmul_rn(job.alpha, __uint_as_float(w[k]));
                    store_sums(job, u.part, x, staging, row0, col0 + c, lane);
                }
                if (!LONG && ok && c + 32 < half) tmem_wait(v[(c / 32 + 1) & 1]);
            }
            if (MODE == kStats && live) {
                if (!ok) run = {nan32(), nan32()};
                a.parts[(int64_t(u.tj) * 2 + group) * job.rows_i + row] = make_float2(run.top, run.sum);
            }
            if (!LONG && ++buf == kBuffers) {
                buf = 0;
                phase ^= 1u;
            }
        }
        if (has_targets && idle) targets(warp + 2, idle);
    }

    tc_before_sync();
    __syncthreads();
    // neither CTA's memory goes before the other one is done with it
    cluster_sync();
    tc_after_sync();
    if (warp == kMma) tmem_free<true>(tmem, kBuffers * kTile);
}

// ---------------------------------------------------------------------------
// few tokens
// ---------------------------------------------------------------------------

// Up to four tokens have kernels of their own, on the ordinary cores with one reading of w:
// rows of up to 4096 values few_rows_kernel, longer ones whose tokens fit shared memory
// few_kernel.  Either has both directions, so that both have the same logits, bit for bit.

// Rows of more than 4096 values: a warp has ROWS rows of w at a time, their products with
// all tokens (fp32 in shared memory) in fp32.  GRAD: d (bf16) for the products, instead of the
// tokens' maxima and sums over the warp's rows.
constexpr int kFewThreads = 256, kFewWarps = kFewThreads / 32;

struct Few {
    const uint16_t *x, *w;
    int64_t ld_x, ld_w;
    int32_t V, D;
    const void *targets;
    int32_t wide;
    int32_t tokens;          // at most T
    int32_t first, rows;     // rows of w here, the first of them at w
    float2 *parts;           // [gridDim.x][tokens]
    float *target_logit;
    // GRAD
    const float *lse, *dlosses;
    uint16_t *d;             // [tokens][ld_d], written up to a multiple of 64 columns
    int64_t ld_d;
};

template <int T, bool VEC, int ROWS, bool GRAD>
__global__ void __launch_bounds__(kFewThreads, 2) few_kernel(const Few a) {
    extern __shared__ __align__(16) float tokens[];  // [T][padded D]
    __shared__ float2 joined[kFewWarps][T];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int32_t pitch = (a.D + 7) & ~7;
    wait_for_predecessor();
    let_successor_start();
#pragma unroll
    for (int t = 0; t < T; ++t)
        for (int32_t d = threadIdx.x; d < pitch; d += kFewThreads)
            tokens[t * pitch + d] = d < a.D && t < a.tokens ? bf16_bits_to_f32(a.x[t * a.ld_x + d]) : 0.0f;
    int32_t y[T];
    Running run[T];
#pragma unroll
    for (int t = 0; t < T; ++t) {
        y[t] = t < a.tokens ? target_of(a.targets, a.wide, a.V, t) : -1;
        run[t] = {-INFINITY, 0.0f};
    }
    __syncthreads();
    const int64_t step = int64_t(gridDim.x) * kFewWarps * ROWS, end = GRAD ? (int64_t(a.rows) + 63) / 64 * 64 : a.rows;
    for (int64_t v = (int64_t(blockIdx.x) * kFewWarps + warp) * ROWS; v < end; v += step) {
        float s[ROWS][T];
        Row row[ROWS];
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            // (rows past the last are read as the last, and dropped below)
            row[r] = row_of(a.w, a.ld_w, a.rows, a.D, v + r < a.rows ? v + r : a.rows - 1);
#pragma unroll
            for (int t = 0; t < T; ++t) s[r][t] = 0.0f;
        }
        {
#pragma unroll VEC ? 4 : 2
            for (int32_t d = 8 * lane; d < pitch; d += 256) {
                uint4 q[ROWS];
                if (VEC) {  // (a multiple of 8 columns)
#pragma unroll
                    for (int r = 0; r < ROWS; ++r) q[r] = ld_stream_u4(row[r].p + d);
                } else {
                    values_at(row, d, 0, q);
                }
#pragma unroll
                for (int t = 0; t < T; ++t) {
                    const float4 lo = *reinterpret_cast<const float4 *>(tokens + t * pitch + d);
                    const float4 hi = *reinterpret_cast<const float4 *>(tokens + t * pitch + d + 4);
#pragma unroll
                    for (int r = 0; r < ROWS; ++r) {
                        s[r][t] = __fmaf_rn(__uint_as_float(q[r].x << 16), lo.x, s[r][t]);
                        s[r][t] = __fmaf_rn(__uint_as_float(q[r].x & 0xFFFF0000u), lo.y, s[r][t]);
                        s[r][t] = __fmaf_rn(__uint_as_float(q[r].y << 16), lo.z, s[r][t]);
                        s[r][t] = __fmaf_rn(__uint_as_float(q[r].y & 0xFFFF0000u), lo.w, s[r][t]);
                        s[r][t] = __fmaf_rn(__uint_as_float(q[r].z << 16), hi.x, s[r][t]);
                        s[r][t] = __fmaf_rn(__uint_as_float(q[r].z & 0xFFFF0000u), hi.y, s[r][t]);
                        s[r][t] = __fmaf_rn(__uint_as_float(q[r].w << 16), hi.z, s[r][t]);
                        s[r][t] = __fmaf_rn(__uint_as_float(q[r].w & 0xFFFF0000u), hi.w, s[r][t]);
                    }
                }
            }
        }
#pragma unroll
        for (int t = 0; t < T; ++t) {
            float z[ROWS], top = run[t].top;
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                float sum = s[r][t];
#pragma unroll
                for (int o = 16; o > 0; o /= 2) sum = __fadd_rn(sum, __shfl_xor_sync(kFull, sum, o));
                const bool own = y[t] >= 0 && v + r == y[t] - a.first;
                if (GRAD) {
                    if (lane != 0 || t >= a.tokens) continue;
                    float d = 0.0f;
                    if (y[t] >= 0 && v + r < a.rows) {
                        const float less = __fadd_rn(sum, -a.lse[t]);
                        d = __fmul_rn(a.dlosses ? a.dlosses[t] : 1.0f, own ? expm1f(less) : exp_of(less));
                    }
                    a.d[t * a.ld_d + v + r] = f32_to_bf16_bits(d);
                    continue;
                }
                if (own && lane == 0) a.target_logit[t] = sum;
                z[r] = own || v + r >= a.rows ? -INFINITY : sum;
                top = fmaxf(top, z[r]);
            }
            if (GRAD) continue;
            const float from = -base_of(top);
            float sum = __fmul_rn(run[t].sum, exp_of(__fadd_rn(run[t].top, from)));
#pragma unroll
            for (int r = 0; r < ROWS; ++r) sum = __fadd_rn(sum, exp_of(__fadd_rn(z[r], from)));
            run[t] = {top, sum};
        }
    }
    if constexpr (!GRAD) {
#pragma unroll
        for (int t = 0; t < T; ++t)
            if (lane == 0) joined[warp][t] = make_float2(run[t].top, run[t].sum);
        __syncthreads();
        if (threadIdx.x < a.tokens) {
            float2 r = joined[0][threadIdx.x];
            for (int w = 1; w < kFewWarps; ++w) r = joined_stats(r, joined[w][threadIdx.x]);
            a.parts[int64_t(blockIdx.x) * a.tokens + threadIdx.x] = r;
        }
    }
}

// Rows of up to 4096 values: WARPS warps have R rows of w at a time in registers, a thread
// 8 columns, whose products with the tokens are summed over the row's threads.  Forward:
// each lane then keeps the maximum and sum of the logits that end in it.  GRAD: from the
// logits come d (fp32, not rounded), from those the rows of dw, written at once, and the sums
// of dx, which stay in registers until the CTA's last row; a second kernel adds the CTAs'.
//
// Bound, forward: HBM (32000 x 2048, 19.4 us at the copy rate: one token 24.5 with the join,
// four 33; the tensor cores, with 256 rows for one token, 38).  Rows that start anywhere are
// shifted into place, a third of the instructions (1 x 32001 x 2047: 38).
// Backward: HBM for one token (32000 x 2048: 46 us, 38.7 at the copy rate, 138 by way of the
// tensor cores, which read w three times and d as often), for four the registers that
// hold tokens and dx, which leave a CTA little to have in flight (78 us, so 140); rows that
// start anywhere also leave by way of shared memory (1 x 32001 x 2047: 74, 3 x 5043 x 1995:
// 29, by way of the tensor cores 47).
// R: as many rows as are not spilled (four rows for four tokens' gradients: 32000 x 4096
// 160 us, two 153; eight for one token's log-sums of rows that start anywhere: 41 us, four 38).
template <int T_, int WARPS, bool VEC, bool GRAD>
struct FewShape {
    static constexpr int T = T_, kWarps = WARPS, kLanes = 32 * WARPS;      // of a row
    static constexpr int kThreads = kLanes < 256 ? 256 : kLanes, kGroups = kThreads / kLanes;
    static constexpr int kPerSm = 512 / kThreads;
    static constexpr int R = VEC ? (T == 1 ? 8 : T == 2 ? (GRAD ? 4 : 8) : GRAD ? 2 : 4) : GRAD && T == 4 ? 2 : 4, N = R * T;
    static constexpr int kSums = GRAD && kGroups > 1 ? kThreads * 8 * T : 1;  // the groups' sums of dx
    static int64_t ctas(int64_t V) {
        const int64_t need = (V + kGroups * R - 1) / (kGroups * R), most = int64_t(kSms) * kPerSm;
        return need < most ? need : most;
    }
};

struct FewRows {
    const uint16_t *x, *w;
    int64_t ld_x, ld_w;
    int32_t V, D;
    const void *targets;
    int32_t wide;
    int32_t tokens;          // at most T
    // forward
    float2 *stats;           // [gridDim.x][tokens]
    float *target_logit;
    // GRAD
    const float *lse, *dlosses;
    float dloss;
    void *dw;                // or NULL
    int64_t ld_dw;
    int32_t dw_bf16, accumulate;
    float *parts;            // [gridDim.x][tokens][D], or NULL
};

// Sums over a warp of N values a lane; lane i has that of value i / (32 / N).
template <int N>
__device__ __forceinline__ float sums_over_warp(float (&p)[N], int lane) {
    int bit = 16;
#pragma unroll
    for (int half = N / 2; half > 0; half /= 2) {
        const bool upper = lane & bit;
#pragma unroll
        for (int i = 0; i < half; ++i) {
            const float give = upper ? p[i] : p[i + half], keep = upper ? p[i + half] : p[i];
            p[i] = __fadd_rn(keep, __shfl_xor_sync(kFull, give, bit));
        }
        bit /= 2;
    }
#pragma unroll
    for (; bit > 0; bit /= 2) p[0] = __fadd_rn(p[0], __shfl_xor_sync(kFull, p[0], bit));
    return p[0];
}

// A thread's 8 columns are neighbours.  VEC: rows of w, and of dw, start on 16 bytes and have
// a multiple of 8 columns; else rows of w are shifted into place and those of dw leave by way
// of shared memory, neighbouring values by neighbouring lanes.
template <bool VEC, typename S, bool GRAD>
__global__ void __launch_bounds__(S::kThreads, S::kPerSm) few_rows_kernel(const FewRows a) {
    constexpr int T = S::T, R = S::R, N = S::N;
    __shared__ float slots[2][S::kThreads / 32][N];
    __shared__ float sums[S::kSums];
    __shared__ float2 joined[S::kGroups][T];
    __shared__ __align__(16) float staging[GRAD && !VEC ? S::kThreads * 8 : 4];  // 256 columns of each warp
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = threadIdx.x / S::kLanes, in = threadIdx.x % S::kLanes;
    const int32_t D = a.D;
    auto column = [&](int j) { return 8 * in + j; };
    const f32x2 zero = pack2(0.0f, 0.0f);
    wait_for_predecessor();
    let_successor_start();
    f32x2 x[T][4], dx[T][4];
#pragma unroll
    for (int t = 0; t < T; ++t) {
        const int token = min(t, a.tokens - 1);
        // (a token of padding has a log-sum, and no gradient whatever its row of x holds)
        const bool live = t < a.tokens && (!GRAD || target_of(a.targets, a.wide, a.V, token) >= 0);
        float e[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) e[j] = bf16_bits_to_f32(a.x[token * a.ld_x + min(column(j), D - 1)]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            x[t][k] = pack2(live && column(2 * k) < D ? e[2 * k] : 0.0f, live && column(2 * k + 1) < D ? e[2 * k + 1] : 0.0f);
            dx[t][k] = zero;
        }
    }
    // this lane's logit: of row `of_row` for token `of_token`
    constexpr int kEach = 32 / N;
    const int of_token = lane / kEach % T, of_row = lane / kEach / T;
    const int32_t y = of_token < a.tokens ? target_of(a.targets, a.wide, a.V, of_token) : -1;
    const float lse = GRAD && y >= 0 ? a.lse[of_token] : 0.0f;
    const float g = !GRAD || y < 0 ? 0.0f : a.dlosses ? a.dlosses[of_token] : a.dloss;
    Running run = {-INFINITY, 0.0f};

    const int64_t first = int64_t(blockIdx.x) * S::kGroups * R, step = int64_t(gridDim.x) * S::kGroups * R;
    int64_t v0 = first + group * R;
    // a row's 8 values, or the two chunks of 16 bytes that they lie in
    uint32_t next[R][VEC ? 4 : 8];
    const uint16_t *const end = a.w + (int64_t(a.V) - 1) * a.ld_w + D;
    auto fetch = [&](int64_t v) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const uint16_t *at = a.w + (v + r) * a.ld_w + 8 * in;
            const bool here = v + r < a.V && 8 * in < D;
#pragma unroll
            for (int k = 0; k < (VEC ? 1 : 2); ++k) {
                uint4 q = make_uint4(0u, 0u, 0u, 0u);
                if (VEC) {
                    if (here) q = ld_stream_u4(at);
                } else {  // (of the second one, the matrix may have ended)
                    const uint4 *chunk = reinterpret_cast<const uint4 *>(reinterpret_cast<uintptr_t>(at) & ~uintptr_t(15)) + k;
                    if (here && reinterpret_cast<const uint16_t *>(chunk) < end) q = __ldg(chunk);
                }
                next[r][4 * k] = q.x;
                next[r][4 * k + 1] = q.y;
                next[r][4 * k + 2] = q.z;
                next[r][4 * k + 3] = q.w;
            }
        }
    };
    uint32_t keep[4];  // of a row's last columns
#pragma unroll
    for (int j = 0; j < 4; ++j) keep[j] = column(2 * j + 1) < D ? 0xFFFFFFFFu : column(2 * j) < D ? 0xFFFFu : 0u;
    // every group of a CTA takes as many turns, for the CTA's barriers
    const int64_t turns = (a.V - first + step - 1) / step;
    // the next rows are under way beside these (but where that is spilled: 4 x 32001 x 2047 132
    // us with it, 126 without)
    constexpr bool kAhead = VEC || !GRAD || T < 4 || S::kWarps > 8;
    if (kAhead) fetch(v0);
    for (int64_t i = 0; i < turns; ++i, v0 += step) {
        if (!kAhead) fetch(v0);
        uint32_t cur[R][4];
        float p[N];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (VEC) {
#pragma unroll
                for (int j = 0; j < 4; ++j) cur[r][j] = next[r][j];
            } else {
                const uint32_t at = (uint32_t(reinterpret_cast<uintptr_t>(a.w)) + 2u * uint32_t(v0 + r) * uint32_t(a.ld_w)) & 15u;
                shift_words(at, next[r], cur[r]);
#pragma unroll
                for (int j = 0; j < 4; ++j) cur[r][j] &= keep[j];
            }
        }
        auto pair = [&](int r, int k) { return pack2(__uint_as_float(cur[r][k] << 16), __uint_as_float(cur[r][k] & 0xFFFF0000u)); };
#pragma unroll
        for (int r = 0; r < R; ++r) {
            f32x2 s[T];
#pragma unroll
            for (int t = 0; t < T; ++t) s[t] = zero;
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int t = 0; t < T; ++t) s[t] = fma2_rn(pair(r, k), x[t][k], s[t]);
#pragma unroll
            for (int t = 0; t < T; ++t) {
                float even, odd;
                unpack2(s[t], even, odd);
                p[r * T + t] = __fadd_rn(even, odd);
            }
        }
        if (kAhead && i + 1 < turns) fetch(v0 + step);
        float s = sums_over_warp(p, lane);
        if (S::kWarps > 1) {
            if (lane % kEach == 0) slots[i & 1][warp][lane / kEach] = s;
            __syncthreads();
            s = slots[i & 1][group * S::kWarps][lane / kEach];
#pragma unroll
            for (int k = 1; k < S::kWarps; ++k) s = __fadd_rn(s, slots[i & 1][group * S::kWarps + k][lane / kEach]);
        }
        const int64_t v = v0 + of_row;
        if (!GRAD) {
            if (v == y && lane % kEach == 0 && warp % S::kWarps == 0) a.target_logit[of_token] = s;
            const float z = v == y || v >= a.V ? -INFINITY : s, top = fmaxf(run.top, z), from = -base_of(top);
            run.sum = __fadd_rn(__fmul_rn(run.sum, exp_of(__fadd_rn(run.top, from))), exp_of(__fadd_rn(z, from)));
            run.top = top;
            continue;
        }
        float d = 0.0f;
        if (y >= 0 && v < a.V) d = __fmul_rn(g, v == y ? expm1f(__fadd_rn(s, -lse)) : expf(__fadd_rn(s, -lse)));
#pragma unroll
        for (int r = 0; r < R; ++r) {
            f32x2 out[4] = {zero, zero, zero, zero};
#pragma unroll
            for (int t = 0; t < T; ++t) {
                const float one = __shfl_sync(kFull, d, (r * T + t) * kEach);
                const f32x2 both = pack2(one, one);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    out[k] = fma2_rn(both, x[t][k], out[k]);
                    dx[t][k] = fma2_rn(both, pair(r, k), dx[t][k]);
                }
            }
            if (a.dw == nullptr || v0 + r >= a.V) continue;
            float e[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) unpack2(out[k], e[2 * k], e[2 * k + 1]);
            const int64_t at = (v0 + r) * a.ld_dw;
            if (VEC && 8 * in < D && a.dw_bf16) {
                uint4 *to = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.dw) + at + 8 * in);
                if (a.accumulate) {
                    const uint4 q = *to;
                    const uint32_t old[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        e[j] = __fadd_rn(__uint_as_float(j & 1 ? old[j / 2] & 0xFFFF0000u : old[j / 2] << 16), e[j]);
                }
                __stcs(to, make_uint4(f32x2_to_bf16x2_bits(e[0], e[1]), f32x2_to_bf16x2_bits(e[2], e[3]),
                                      f32x2_to_bf16x2_bits(e[4], e[5]), f32x2_to_bf16x2_bits(e[6], e[7])));
            } else if (VEC && 8 * in < D) {
                float4 *to = reinterpret_cast<float4 *>(static_cast<float *>(a.dw) + at + 8 * in);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float4 old = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    if (a.accumulate) old = to[h];
                    __stcs(to + h, make_float4(__fadd_rn(old.x, e[4 * h]), __fadd_rn(old.y, e[4 * h + 1]),
                                               __fadd_rn(old.z, e[4 * h + 2]), __fadd_rn(old.w, e[4 * h + 3])));
                }
            } else if (!VEC) {
                float4 *const st = reinterpret_cast<float4 *>(staging + warp * 256);
                st[2 * lane] = make_float4(e[0], e[1], e[2], e[3]);
                st[2 * lane + 1] = make_float4(e[4], e[5], e[6], e[7]);
                __syncwarp();
                const int32_t c0 = warp % S::kWarps * 256 + lane;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (c0 + 32 * j >= D) continue;
                    const float one = staging[warp * 256 + lane + 32 * j];
                    if (a.dw_bf16) {
                        uint16_t *to = static_cast<uint16_t *>(a.dw) + at + c0 + 32 * j;
                        *to = f32_to_bf16_bits(a.accumulate ? __fadd_rn(bf16_bits_to_f32(*to), one) : one);
                    } else {
                        float *to = static_cast<float *>(a.dw) + at + c0 + 32 * j;
                        *to = a.accumulate ? __fadd_rn(*to, one) : one;
                    }
                }
                __syncwarp();
            }
        }
    }
    if (!GRAD) {
        // a token's rows of this warp, then the groups' (a group's warps all hold the same)
        float2 r = make_float2(run.top, run.sum);
#pragma unroll
        for (int o = 16; o >= kEach * T; o /= 2)
            r = joined_stats(r, make_float2(__shfl_xor_sync(kFull, r.x, o), __shfl_xor_sync(kFull, r.y, o)));
        if (of_row == 0 && lane % kEach == 0 && warp % S::kWarps == 0) joined[group][of_token] = r;
        __syncthreads();
        if (threadIdx.x < a.tokens) {
            r = joined[0][threadIdx.x];
            for (int k = 1; k < S::kGroups; ++k) r = joined_stats(r, joined[k][threadIdx.x]);
            a.stats[int64_t(blockIdx.x) * a.tokens + threadIdx.x] = r;
        }
        return;
    }
    if (a.parts == nullptr) return;
#pragma unroll
    for (int t = 0; t < T; ++t) {
        if (t >= a.tokens) break;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float e[2];
            unpack2(dx[t][k], e[0], e[1]);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int32_t c = column(2 * k + h);
                if (c >= D) continue;
                if (S::kGroups > 1) sums[(group * T + t) * D + c] = e[h];
                else a.parts[(int64_t(blockIdx.x) * a.tokens + t) * D + c] = e[h];
            }
        }
    }
    if (S::kGroups == 1) return;
    __syncthreads();
    for (int32_t c = threadIdx.x; c < a.tokens * D; c += S::kThreads) {
        float e = sums[c];
#pragma unroll
        for (int k = 1; k < S::kGroups; ++k) e = __fadd_rn(e, sums[k * T * D + c]);
        a.parts[int64_t(blockIdx.x) * a.tokens * D + c] = e;
    }
}

// dx of few tokens: the CTAs' sums, 32 values by 32 warps of a CTA, each warp every 32nd
// sum, then the warps in turn.
__global__ void __launch_bounds__(1024) join_few_kernel(const float *parts, int32_t count, int32_t tokens, int32_t D,
                                                        void *dx, int bf16, int64_t ld_dx) {
    __shared__ float sums[32][33];
    wait_for_predecessor();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int32_t n = tokens * D, c = blockIdx.x * 32 + lane;
    float x = 0.0f;
    if (c < n)
#pragma unroll 8
        for (int32_t g = warp; g < count; g += 32) x = __fadd_rn(x, parts[int64_t(g) * n + c]);
    sums[warp][lane] = x;
    __syncthreads();
    x = sums[lane][warp];  // warp w has value w
#pragma unroll
    for (int o = 16; o > 0; o /= 2) x = __fadd_rn(x, __shfl_xor_sync(kFull, x, o));
    const int32_t at = blockIdx.x * 32 + warp;
    if (lane != 0 || at >= n) return;
    const int32_t t = at / D;
    if (bf16) static_cast<uint16_t *>(dx)[t * ld_dx + at - t * D] = f32_to_bf16_bits(x);
    else static_cast<float *>(dx)[t * ld_dx + at - t * D] = x;
}

// ---------------------------------------------------------------------------
// small kernels
// ---------------------------------------------------------------------------

// lse and loss of each token from the parts of its row: 32 tokens by 32 warps of
// a CTA, each warp every 32nd part, then the warps in turn.
__global__ void __launch_bounds__(1024) join_stats_kernel(const float2 *parts, int32_t count, int32_t T,
                                                          const float *target_logit, const void *targets, int wide,
                                                          int32_t V, float *losses, float *lse) {
    __shared__ float2 row[32][33];
    wait_for_predecessor();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int32_t t = blockIdx.x * 32 + lane;
    float2 r = make_float2(-INFINITY, 0.0f);
    if (t < T)
#pragma unroll 4
        for (int32_t p = warp; p < count; p += 32) r = joined_stats(r, parts[int64_t(p) * T + t]);
    row[warp][lane] = r;
    __syncthreads();
    r = row[lane][warp];  // warp w has token w
#pragma unroll
    for (int o = 16; o > 0; o /= 2) {
        const float2 other = make_float2(__shfl_xor_sync(kFull, r.x, o), __shfl_xor_sync(kFull, r.y, o));
        r = lane & o ? joined_stats(other, r) : joined_stats(r, other);
    }
    const int32_t at = blockIdx.x * 32 + warp;
    if (lane != 0 || at >= T) return;
    if (target_of(targets, wide, V, at) < 0) {
        if (lse) lse[at] = __fadd_rn(r.x, logf(r.y));
        if (losses) losses[at] = 0.0f;
        return;
    }
    // the log of the others' sum over the target's exponential (-infinity if there are none)
    const float s = target_logit[at];
    const float more = r.y == 0.0f ? -INFINITY : __fadd_rn(__fadd_rn(r.x, -s), logf(r.y));
    const float rest = log1pf(expf(-fabsf(more)));
    const float loss = __fadd_rn(more > 0.0f ? more : 0.0f, rest);
    // from the larger of the two (a target may be impossible, its logit -infinity)
    if (lse) lse[at] = more > 0.0f ? __fadd_rn(__fadd_rn(r.x, logf(r.y)), rest) : __fadd_rn(s, loss);
    if (losses) losses[at] = loss;
}

// A matrix [rows][D] with rows that start on 16 bytes, from one whose rows may
// start anywhere.
struct LayOut {
    const uint16_t *src;     // NULL: nothing to do
    int64_t ld, rows;
    uint16_t *dst;
};

// x and w laid out, x a warp per row; x may have no place to go.  With target_logit, the
// products of x's rows with their target's row of w go there, and with `mask` rows
// whose target is padding become 0.
struct LayOuts {
    LayOut x, w;
    int32_t D, ctas_x, mask; // CTAs at work on x
    const void *targets;
    const uint16_t *given_w;
    int64_t ld_w;
    int32_t wide, V;
    float *target_logit;     // or NULL
};

__global__ void __launch_bounds__(256) lay_out_kernel(const LayOuts a) {
    wait_for_predecessor();
    let_successor_start();
    const int lane = threadIdx.x & 31;
    const bool of_x = int32_t(blockIdx.x) < a.ctas_x;
    const LayOut &m = of_x ? a.x : a.w;
    const int64_t cta = of_x ? blockIdx.x : blockIdx.x - a.ctas_x, ctas = of_x ? a.ctas_x : gridDim.x - a.ctas_x;
    const int32_t ld = (a.D + 7) & ~7;
    if (!of_x) {
        // four places of 8 values per thread, a grid's width apart
        const int64_t chunks = ld / 8, n = m.rows * chunks, step = ctas * 256;
        const uint16_t *const end = row_of(m.src, m.ld, m.rows, a.D, 0).end;
        for (int64_t i = cta * 256 + threadIdx.x; i < n; i += 4 * step) {
            const uint16_t *at[4];
            int32_t left[4];
            int64_t to[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int64_t j = i + k * step < n ? i + k * step : i, r = j / chunks;
                const int32_t c = int32_t(j - r * chunks) * 8;
                at[k] = m.src + r * m.ld + c;
                left[k] = a.D - c;
                to[k] = 8 * j;
            }
            uint4 q[4];
            values_at(at, left, end, q);
#pragma unroll
            for (int k = 0; k < 4; ++k) *reinterpret_cast<uint4 *>(m.dst + to[k]) = q[k];
        }
        return;
    }
    for (int64_t r = cta * 8 + (threadIdx.x >> 5); r < m.rows; r += ctas * 8) {
        const int32_t y = a.target_logit ? target_of(a.targets, a.wide, a.V, r) : 0;
        const Row row = row_of(m.src, m.ld, m.rows, a.D, r), rows[4] = {row, row, row, row};
        uint16_t *to = m.dst + r * ld;
        const bool zero = y < 0 && a.mask;
        int32_t d = m.dst ? 0 : ld;
        for (; d + 256 < ld; d += 1024) {
            const int32_t c = d + 8 * lane;
            uint4 q[4];
            values_at(rows, c, 256, q);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (c + 256 * k < ld)
                    *reinterpret_cast<uint4 *>(to + c + 256 * k) = zero ? make_uint4(0u, 0u, 0u, 0u) : q[k];
        }
        if (d + 8 * lane < ld) {
            const Row one[1] = {row};
            uint4 q[1];
            values_at(one, d + 8 * lane, 0, q);
            *reinterpret_cast<uint4 *>(to + d + 8 * lane) = zero ? make_uint4(0u, 0u, 0u, 0u) : q[0];
        }
        if (a.target_logit == nullptr || y < 0) continue;
        const float s = row_dot(row, row_of(a.given_w, a.ld_w, a.V, a.D, y), lane);
        if (lane == 0) a.target_logit[r] = s;
    }
}

// out = the sum of `count` matrices [rows][ld_part] of fp32, in order; ld_part is a
// multiple of 4, and a thread has 4 columns.
__global__ void __launch_bounds__(256) join_sums_kernel(const float *parts, int32_t count, int64_t rows, int32_t cols,
                                                        int32_t ld_part, void *out, int bf16, int64_t ld_out, int vec) {
    wait_for_predecessor();
    const int32_t quads = ld_part / 4;
    const int64_t stride = rows * ld_part;
    for (int64_t r = blockIdx.y; r < rows; r += gridDim.y) {
        const int32_t q = int32_t(blockIdx.x) * 256 + threadIdx.x;
        if (q >= quads) continue;
        const float4 *p = reinterpret_cast<const float4 *>(parts + r * ld_part) + q;
        float4 x = *p;
#pragma unroll 4
        for (int32_t k = 1; k < count; ++k) {
            const float4 y = *reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(p) + k * stride);
            x = make_float4(__fadd_rn(x.x, y.x), __fadd_rn(x.y, y.y), __fadd_rn(x.z, y.z), __fadd_rn(x.w, y.w));
        }
        const int64_t at = r * ld_out + 4 * q;
        const float e[4] = {x.x, x.y, x.z, x.w};
        if (vec && bf16 && 4 * q + 4 <= cols) {
            *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(out) + at) =
                make_uint2(f32x2_to_bf16x2_bits(x.x, x.y), f32x2_to_bf16x2_bits(x.z, x.w));
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (4 * q + k >= cols) break;
                if (bf16) static_cast<uint16_t *>(out)[at + k] = f32_to_bf16_bits(e[k]);
                else static_cast<float *>(out)[at + k] = e[k];
            }
        }
    }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t up256(int64_t bytes) { return ceil_div(bytes, 256) * 256; }

struct Bf16Matrix {
    const uint16_t *p;
    int64_t ld, rows, cols;
};

// Boxes of `rows` rows x 64 of K, or MN-major of 64 rows x 64 of K.
cudaError_t describe(CUtensorMap *map, const Bf16Matrix &m, bool mn, int rows = kHalf) {
    EncodeTiled encode;
    const cudaError_t e = encoder(&encode);
    if (e != cudaSuccess) return e;
    const cuuint64_t dims[2] = {cuuint64_t(m.cols), cuuint64_t(m.rows)};
    // (a single row is apart from none)
    const cuuint64_t strides[1] = {cuuint64_t(m.rows > 1 ? m.ld : ceil_div(m.cols, 8) * 8) * 2};
    const cuuint32_t box[2] = {64, cuuint32_t(mn ? 64 : rows)};
    const cuuint32_t step[2] = {1, 1};
    const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<uint16_t *>(m.p), dims, strides,
                              box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Rows of a copy of tokens (a multiple of 8, as the swizzle repeats): with 128 the copies of
// rows that do not exist take as long as those of w (5 x 32000 x 2048: 39.5 us, so 32.5).
int box_of(int64_t T) { return T < kHalf ? int(ceil_div(T, 8) * 8) : kHalf; }

template <Mode MODE, bool LONG>
cudaError_t run(const CUtensorMap (&maps)[4], Args &a, cudaStream_t stream) {
    // once for each GPU: the kernel's attribute stays set
    static std::atomic<uint64_t> prepared{0};
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    const uint64_t bit = uint64_t(1) << (device & 63);
    if (device > 63 || !(prepared.load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute(product_kernel<MODE, LONG>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
        prepared.fetch_or(bit, std::memory_order_relaxed);
    }
    for (int k = 0; k < 2; ++k) a.units[k] = a.job[k].tiles_i * a.job[k].tiles_j * a.job[k].split;
    const int64_t units = int64_t(a.units[0]) + (MODE == kProducts ? a.units[1] : 0);
    a.sooner = 0;
    if (MODE == kProducts && a.units[0] > 0 && a.units[1] > 0) {
        auto cycles = [](const Job &j) { return int64_t(j.blocks) / j.split * (j.width + 256) + 1500; };
        const int64_t each = cycles(a.job[1]);
        a.sooner = int32_t((cycles(a.job[0]) + each / 2) / each);
    }
    // (CTAs without tiles sum targets' logits, ten warps with one token at a time)
    const int64_t more = MODE == kStats && a.x ? units + ceil_div(a.job[0].rows_i, 20) : 0, pairs = units > more ? units : more;
    const uint32_t grid = 2 * uint32_t(pairs < kSms / 2 ? pairs : kSms / 2);
    return launch_after(product_kernel<MODE, LONG>, dim3(grid), dim3(kThreads), kSmem, stream, 2, maps[0], maps[1],
                        maps[2], maps[3], a);
}

// Stages of K whose products the tensor core sums by itself: 1024 values.  They take little
// longer for it, as the sums leave beside the next chunk's products (8192 x 32000 x 2048:
// losses 528 us either way; both gradients, with the chunks of their products, 1711 instead
// of 1692).  Both directions have the same chunks, so that they have the same logits, bit for
// bit: the log-sum is one of the forward pass's logits where one decides a row, and what
// another order of the sums would be off by, some 2^-22 of a logit, is in the exponent.
template <Mode MODE>
cudaError_t run_logits(const CUtensorMap (&maps)[4], Args &a, cudaStream_t stream) {
    constexpr int32_t chunk = 1024 / kDepth;
    a.job[0].chunks = (a.job[0].blocks + chunk - 1) / chunk;
    return a.job[0].chunks > 1 ? run<MODE, true>(maps, a, stream) : run<MODE, false>(maps, a, stream);
}

// The same of dx's and dw's products, whose K are the vocabulary and the tokens: 8192 values,
// so that what is cut off, some 2^-16 of a sum at most, does not grow with them (dw of a million
// tokens, terms of one sign: 3.7e-3 without).  (8192 x 32000 x 2048, dx in two chunks 2510 us, in
// one 2500; both in chunks of 4096 2590.)
cudaError_t run_products(const CUtensorMap (&maps)[4], Args &a, cudaStream_t stream) {
    constexpr int32_t chunk = 8192 / kDepth;
    bool several = false;
    for (Job &j : a.job) {
        j.chunks = j.split > 0 ? (j.blocks + j.split * chunk - 1) / (j.split * chunk) : 0;
        several = several || j.chunks > 1;
    }
    return several ? run<kProducts, true>(maps, a, stream) : run<kProducts, false>(maps, a, stream);
}

bool aligned(const uint16_t *p, int64_t ld) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 8 == 0; }

// Columns of a tile of logits.  A stage of a narrow tile takes not much less time than
// of a wide one, as it brings x all the same (16 stages of 64 in one wave: 256 columns
// 12.8 us, 128 10.8; 1024 x 32000 x 2048, many waves: 74 us, 117), so narrow ones serve
// where the wide ones leave SMs without work.
int width_of(int64_t T, int64_t V) {
    const int64_t tiles = ceil_div(T, kTile);
    int best = kTile;
    int64_t least = 0;
    for (int w = kTile; w >= 64; w -= 64) {
        const int64_t cost = ceil_div(tiles * ceil_div(V, w), kSms / 2) * (w + 256);
        if (w == kTile || cost < least) {
            best = w;
            least = cost;
        }
    }
    return best;
}

// Tokens of one forward launch: it leaves 16 bytes per token and 256 rows of w.
constexpr int64_t kTokens = 65536;

// The workspace's parts, one after another.
struct Layout {
    int64_t bytes = 0;
    int64_t take(int64_t n) {
        const int64_t at = bytes;
        bytes += up256(n);
        return at;
    }
};

// Few tokens with rows of up to 4096 values?  A thread has 8 columns, a CTA at most 512 threads.
bool few_short(const CrossEntropy &c) { return c.T <= 4 && c.D <= 4096; }

// Few tokens with longer rows?  Their fp32 values fit shared memory twice per SM.
constexpr int kFewBytes = 112 * 1024;
int64_t few_tokens_held(const CrossEntropy &c) { return c.T <= 2 ? c.T : 4; }
bool few_long(const CrossEntropy &c) {
    return c.T <= 4 && c.D > 4096 && few_tokens_held(c) * (c.D + 7) * 4 <= kFewBytes;
}

// f(the shape for c's tokens and columns).
template <bool VEC, bool GRAD, typename F>
auto with_few_shape(const CrossEntropy &c, F f) {
    auto of = [&](auto warps) {
        constexpr int W = decltype(warps)::value;
        if (c.T == 1) return f(FewShape<1, W, VEC, GRAD>());
        if (c.T == 2) return f(FewShape<2, W, VEC, GRAD>());
        return f(FewShape<4, W, VEC, GRAD>());
    };
    if (c.D <= 256) return of(std::integral_constant<int, 1>());
    if (c.D <= 512) return of(std::integral_constant<int, 2>());
    if (c.D <= 1024) return of(std::integral_constant<int, 4>());
    if (c.D <= 2048) return of(std::integral_constant<int, 8>());
    return of(std::integral_constant<int, 16>());
}

// vec: of what is written.
template <bool GRAD>
int64_t few_ctas(const CrossEntropy &c, bool vec) {
    auto ctas = [&](auto shape) { return decltype(shape)::ctas(c.V); };
    return vec && c.D % 8 == 0 && aligned(c.w, c.ld_w) ? with_few_shape<true, GRAD>(c, ctas) : with_few_shape<false, GRAD>(c, ctas);
}

// Rows of w that a warp of few_kernel has at a time: four share a token's values, and one
// keeps more of the GPU busy where rows are few (4 x 1043 x 3009: 24 us with four, 14 with one).
int64_t few_rows(int64_t V) { return V <= 4 * kSms * kFewWarps ? 1 : 4; }

int64_t few_grid(int64_t V) {
    const int64_t ctas = ceil_div(V, kFewWarps * few_rows(V));
    return ctas < 2 * kSms ? ctas : 2 * kSms;
}

struct FewLayout {
    int64_t ctas, parts, target_logit, bytes;
    explicit FewLayout(const CrossEntropy &c) {
        Layout l;
        ctas = few_short(c) ? few_ctas<false>(c, true) : few_grid(c.V);
        parts = l.take(ctas * c.T * int64_t(sizeof(float2)));
        target_logit = l.take(c.T * 4);
        bytes = l.bytes;
    }
};

struct Forward {
    int64_t parts, target_logit, x, w, bytes;
    explicit Forward(const CrossEntropy &c) {
        Layout l;
        const int64_t T = c.T < kTokens ? c.T : kTokens;
        parts = l.take(ceil_div(c.V, width_of(T, c.V)) * 2 * T * int64_t(sizeof(float2)));
        target_logit = l.take(c.T * 4);
        x = aligned(c.x, c.ld_x) ? -1 : l.take(c.T * ceil_div(c.D, 8) * 16);
        w = aligned(c.w, c.ld_w) ? -1 : l.take(c.V * ceil_div(c.D, 8) * 16);
        bytes = l.bytes;
    }
};

// Columns of a piece: its gradients of the logits (bf16) take 256 MB, or as much
// as dx's sums where that is more, so that those are not moved more often than
// the pieces themselves.
int64_t piece_of(const CrossEntropy &c) {
    const int64_t budget = int64_t(1) << 28, sums = 4 * c.T * c.D;
    int64_t cols = (budget > sums ? budget : sums) / (2 * c.T) / kTile * kTile;
    if (cols < kTile) cols = kTile;
    const int64_t pieces = ceil_div(c.V, cols);
    return ceil_div(ceil_div(c.V, pieces), kTile) * kTile;
}

struct Backward {
    int64_t x, w, target_logit, d, dx, bytes;
    int64_t piece, split, ld_dx;
    int width;  // of a tile of the products
    // dx's K is the vocabulary, so where tokens are few its tiles are few and long.
    // How many parts each is split into, and the tiles' width: the least of an
    // estimate of the launch in cycles -- a stage takes w + 256, a tile 1500 beside its
    // stages, the parts' join 5000 and their memory traffic.
    // (1024 x 32000 x 2048: dx whole 204 us, in four parts 161 and 10 for the join.)
    void plan(const CrossEntropy &c) {
        const int64_t blocks = ceil_div(piece, kDepth), rows = ceil_div(c.T, kTile);
        int64_t least = 0;
        for (int w = kTile; w >= kTile / 2; w /= 2)
            for (int64_t s = 1; s <= 32 && (s == 1 || blocks / s >= 4); s += s < 4 ? 1 : s / 2) {
                const int64_t across = ceil_div(c.D, w), stage = w + 256;
                const int64_t unit_dx = ceil_div(blocks, s) * stage + 1500, unit_dw = ceil_div(c.T, kDepth) * stage + 1500;
                const int64_t all = rows * across * s * unit_dx + ceil_div(piece, kTile) * across * unit_dw;
                const int64_t longest = unit_dx > unit_dw ? unit_dx : unit_dw, even = all / (kSms / 2) + longest / 2;
                const int64_t cost = (even > longest ? even : longest) + (s > 1 ? 5000 + s * c.T * c.D / 300 : 0);
                if (least == 0 || cost < least) {
                    least = cost;
                    split = s;
                    width = w;
                }
            }
    }
    explicit Backward(const CrossEntropy &c) {
        Layout l;
        const int64_t ld = ceil_div(c.D, 8) * 16;
        x = l.take(c.T * ld);
        w = aligned(c.w, c.ld_w) ? -1 : l.take(c.V * ld);
        target_logit = l.take(c.T * 4);
        piece = piece_of(c);
        d = l.take(c.T * piece * 2);
        ld_dx = ceil_div(c.D, 4) * 4;
        plan(c);
        dx = split > 1 || piece < c.V ? l.take(split * c.T * ld_dx * 4) : -1;
        bytes = l.bytes;
    }
};

// x and w to the places given, each if it is not NULL; target_logit and mask as above.
cudaError_t lay_out(const CrossEntropy &c, uint16_t *x, uint16_t *w, float *target_logit, bool mask,
                    cudaStream_t stream) {
    auto ctas = [](int64_t rows) { return int32_t(rows < 128 * kSms ? ceil_div(rows, 8) : 16 * kSms); };
    LayOuts a = {};
    if (x || target_logit) a.x = {c.x, c.ld_x, c.T, x};
    if (w) a.w = {c.w, c.ld_w, c.V, w};
    a.D = int32_t(c.D);
    a.ctas_x = ctas(a.x.rows);
    a.mask = mask;
    a.targets = c.targets;
    a.given_w = c.w;
    a.ld_w = c.ld_w;
    a.wide = c.wide;
    a.V = int32_t(c.V);
    a.target_logit = target_logit;
    // (1024 places of w per CTA and turn)
    const int64_t places = ceil_div(a.w.rows * ceil_div(c.D, 8), 1024);
    const int32_t ctas_w = int32_t(places < 32 * kSms ? places : 32 * kSms);
    return launch_after(lay_out_kernel, dim3(uint32_t(a.ctas_x + ctas_w)), dim3(256), 0, stream, 1, a);
}

Job job_of(int64_t rows_i, int64_t rows_j, int64_t K, int width) {
    Job j = {};
    j.tiles_i = int32_t(ceil_div(rows_i, kTile));
    j.tiles_j = int32_t(ceil_div(rows_j, width));
    j.width = width;
    j.split = 1;
    j.blocks = int32_t(ceil_div(K, kDepth));
    j.rows_i = int32_t(rows_i);
    j.rows_j = int32_t(rows_j);
    j.box_i = kHalf;
    return j;
}

template <int T, bool VEC, int ROWS, bool GRAD>
cudaError_t run_few(const Few &a, uint32_t grid, size_t smem, cudaStream_t stream) {
    // once for each GPU: the kernel's attribute stays set
    static std::atomic<uint64_t> prepared{0};
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    const uint64_t bit = uint64_t(1) << (device & 63);
    if (device > 63 || !(prepared.load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute(few_kernel<T, VEC, ROWS, GRAD>, cudaFuncAttributeMaxDynamicSharedMemorySize, kFewBytes);
        if (e != cudaSuccess) return e;
        prepared.fetch_or(bit, std::memory_order_relaxed);
    }
    return launch_after(few_kernel<T, VEC, ROWS, GRAD>, dim3(grid), dim3(kFewThreads), smem, stream, 1, a);
}

template <int T, bool GRAD>
cudaError_t run_few(const Few &a, bool vec, int64_t rows, uint32_t grid, size_t smem, cudaStream_t stream) {
    if (rows == 1)
        return vec ? run_few<T, true, 1, GRAD>(a, grid, smem, stream) : run_few<T, false, 1, GRAD>(a, grid, smem, stream);
    return vec ? run_few<T, true, 4, GRAD>(a, grid, smem, stream) : run_few<T, false, 4, GRAD>(a, grid, smem, stream);
}

// The rows first .. first + rows - 1 of w, whose results `a` says where to leave.
template <bool GRAD>
cudaError_t run_few(const CrossEntropy &c, Few a, int64_t first, int64_t rows, cudaStream_t stream) {
    a.x = c.x;
    a.w = c.w + first * c.ld_w;
    a.ld_x = c.ld_x;
    a.ld_w = c.ld_w;
    a.V = int32_t(c.V);
    a.D = int32_t(c.D);
    a.targets = c.targets;
    a.wide = c.wide;
    a.tokens = int32_t(c.T);
    a.first = int32_t(first);
    a.rows = int32_t(rows);
    const int64_t padded = GRAD ? ceil_div(rows, kDepth) * kDepth : rows;
    const uint32_t grid = uint32_t(few_grid(padded));
    const int held = int(few_tokens_held(c));
    const size_t smem = size_t(held) * ((c.D + 7) / 8 * 8) * 4;
    const bool vec = aligned(c.w, c.ld_w) && c.D % 8 == 0;
    const int64_t each = few_rows(padded);
    return held == 1   ? run_few<1, GRAD>(a, vec, each, grid, smem, stream)
           : held == 2 ? run_few<2, GRAD>(a, vec, each, grid, smem, stream)
                       : run_few<4, GRAD>(a, vec, each, grid, smem, stream);
}

cudaError_t join_stats(const CrossEntropy &c, const float2 *parts, int32_t count, int64_t t0, int64_t tokens,
                       const float *target_logit, cudaStream_t stream) {
    return launch_after(join_stats_kernel, dim3(uint32_t(ceil_div(tokens, 32))), dim3(1024), 0, stream, 1, parts, count,
                        int32_t(tokens), target_logit,
                        static_cast<const void *>(static_cast<const char *>(c.targets) + t0 * (c.wide ? 8 : 4)),
                        c.wide ? 1 : 0, int32_t(c.V), c.losses ? c.losses + t0 : nullptr, c.lse ? c.lse + t0 : nullptr);
}

template <bool GRAD>
cudaError_t run_few_rows(const CrossEntropy &c, FewRows a, bool vec, cudaStream_t stream) {
    a.x = c.x;
    a.w = c.w;
    a.ld_x = c.ld_x;
    a.ld_w = c.ld_w;
    a.V = int32_t(c.V);
    a.D = int32_t(c.D);
    a.targets = c.targets;
    a.wide = c.wide;
    a.tokens = int32_t(c.T);
    auto launch = [&](auto kernel, auto shape) {
        using S = decltype(shape);
        return launch_after(kernel, dim3(uint32_t(S::ctas(c.V))), dim3(S::kThreads), 0, stream, 1, a);
    };
    if (vec && c.D % 8 == 0 && aligned(c.w, c.ld_w))
        return with_few_shape<true, GRAD>(c, [&](auto shape) { return launch(few_rows_kernel<true, decltype(shape), GRAD>, shape); });
    return with_few_shape<false, GRAD>(c, [&](auto shape) { return launch(few_rows_kernel<false, decltype(shape), GRAD>, shape); });
}

cudaError_t launch_few(const CrossEntropy &c, cudaStream_t stream) {
    const FewLayout f(c);
    char *const ws = static_cast<char *>(c.workspace);
    float2 *const parts = reinterpret_cast<float2 *>(ws + f.parts);
    float *const target_logit = reinterpret_cast<float *>(ws + f.target_logit);
    cudaError_t e;
    if (few_short(c)) {
        FewRows a = {};
        a.stats = parts;
        a.target_logit = target_logit;
        e = run_few_rows<false>(c, a, true, stream);
    } else {
        Few a = {};
        a.parts = parts;
        a.target_logit = target_logit;
        e = run_few<false>(c, a, 0, c.V, stream);
    }
    if (e != cudaSuccess) return e;
    return join_stats(c, parts, int32_t(f.ctas), 0, c.T, target_logit, stream);
}

cudaError_t launch_few_grad(const CrossEntropyGrad &c, cudaStream_t stream) {
    const bool vec = !c.dw || aligned(static_cast<const uint16_t *>(c.dw), c.ld_dw);
    const int64_t ctas = few_ctas<true>(c, vec);
    float *const parts = c.dx ? static_cast<float *>(c.workspace) : nullptr;
    FewRows a = {};
    a.lse = c.lse_in;
    a.dlosses = c.dlosses;
    a.dloss = c.dloss;
    a.dw = c.dw;
    a.ld_dw = c.ld_dw;
    a.dw_bf16 = c.dw_bf16;
    a.accumulate = c.accumulate;
    a.parts = parts;
    const cudaError_t e = run_few_rows<true>(c, a, vec, stream);
    if (e != cudaSuccess || !c.dx) return e;
    return launch_after(join_few_kernel, dim3(uint32_t(ceil_div(c.T * c.D, 32))), dim3(1024), 0, stream, 1,
                        static_cast<const float *>(parts), int32_t(ctas), int32_t(c.T), int32_t(c.D), c.dx, c.dx_bf16 ? 1 : 0, c.ld_dx);
}

}  // namespace

int64_t cross_entropy_workspace(const CrossEntropy &c) {
    return few_short(c) || few_long(c) ? FewLayout(c).bytes : Forward(c).bytes;
}

cudaError_t launch_cross_entropy(const CrossEntropy &c, cudaStream_t stream) {
    if (few_short(c) || few_long(c)) return launch_few(c, stream);
    const Forward f(c);
    char *const ws = static_cast<char *>(c.workspace);
    Bf16Matrix x = {c.x, c.ld_x, c.T, c.D}, w = {c.w, c.ld_w, c.V, c.D};
    cudaError_t e = cudaSuccess;
    if (f.x >= 0) x = {reinterpret_cast<uint16_t *>(ws + f.x), ceil_div(c.D, 8) * 8, c.T, c.D};
    if (f.w >= 0) w = {reinterpret_cast<uint16_t *>(ws + f.w), ceil_div(c.D, 8) * 8, c.V, c.D};
    // The targets' logits: beside the rows that are laid out anyway, in the products'
    // spare warps, or, where those would take longer than the products, by themselves
    // (a warp takes some 2 us for each 1024 of D, a stage of a tile 0.3 us; 6614 x 627 x
    // 2274: 148 us in the spare warps).
    const int width = width_of(c.T < kTokens ? c.T : kTokens, c.V);
    const int64_t tiles = ceil_div(c.T, kTile) * ceil_div(c.V, width);
    const bool apart = f.x >= 0 || f.w >= 0 ||
                       ceil_div(c.T, 2 * kSms) * ceil_div(c.D, 1024) * 7 > ceil_div(tiles, kSms / 2) * ceil_div(c.D, kDepth);
    float *const target_logit = reinterpret_cast<float *>(ws + f.target_logit);
    if (apart) {
        e = lay_out(c, f.x >= 0 ? const_cast<uint16_t *>(x.p) : nullptr, f.w >= 0 ? const_cast<uint16_t *>(w.p) : nullptr,
                    target_logit, false, stream);
        if (e != cudaSuccess) return e;
    }
    CUtensorMap maps[4];
    if ((e = describe(&maps[1], w, false, width / 2)) != cudaSuccess) return e;
    const int64_t id = c.wide ? 8 : 4;
    for (int64_t t0 = 0; t0 < c.T; t0 += kTokens) {
        Bf16Matrix some = x;
        some.p += t0 * x.ld;
        some.rows = c.T - t0 < kTokens ? c.T - t0 : kTokens;
        if ((e = describe(&maps[0], some, false, box_of(some.rows))) != cudaSuccess) return e;
        maps[2] = maps[0];
        maps[3] = maps[1];
        Args a = {};
        a.job[0] = job_of(some.rows, c.V, c.D, width);
        a.job[0].box_i = box_of(some.rows);
        a.targets = static_cast<const char *>(c.targets) + t0 * id;
        a.wide = c.wide;
        a.V = int32_t(c.V);
        a.parts = reinterpret_cast<float2 *>(ws + f.parts);
        a.target_logit = target_logit + t0;
        a.x = apart ? nullptr : c.x + t0 * c.ld_x;
        a.w = c.w;
        a.ld_x = c.ld_x;
        a.ld_w = c.ld_w;
        a.D = int32_t(c.D);
        if ((e = run_logits<kStats>(maps, a, stream)) != cudaSuccess) return e;
        e = join_stats(c, a.parts, 2 * a.job[0].tiles_j, t0, some.rows, a.target_logit, stream);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

int64_t cross_entropy_grad_workspace(const CrossEntropy &c) {
    if (!few_short(c)) return Backward(c).bytes;
    const int64_t a = few_ctas<true>(c, true), b = few_ctas<true>(c, false);
    return up256((a > b ? a : b) * c.T * c.D * 4);
}

cudaError_t launch_cross_entropy_grad(const CrossEntropyGrad &c, cudaStream_t stream) {
    if (few_short(c)) return launch_few_grad(c, stream);
    const Backward f(c);
    char *const ws = static_cast<char *>(c.workspace);
    // x with its padding tokens 0, so that nothing that they hold reaches dw
    const Bf16Matrix x = {reinterpret_cast<uint16_t *>(ws + f.x), ceil_div(c.D, 8) * 8, c.T, c.D};
    float *const target_logit = reinterpret_cast<float *>(ws + f.target_logit);
    Bf16Matrix w = {c.w, c.ld_w, c.V, c.D};
    if (f.w >= 0) w = {reinterpret_cast<uint16_t *>(ws + f.w), x.ld, c.V, c.D};
    cudaError_t e = lay_out(c, const_cast<uint16_t *>(x.p), f.w >= 0 ? const_cast<uint16_t *>(w.p) : nullptr,
                            target_logit, true, stream);
    if (e != cudaSuccess) return e;
    const Bf16Matrix d = {reinterpret_cast<uint16_t *>(ws + f.d), f.piece, c.T, f.piece};
    CUtensorMap logits[4], products[4];
    if ((e = describe(&logits[0], x, false, box_of(c.T))) != cudaSuccess) return e;
    const int width = width_of(c.T, f.piece < c.V ? f.piece : c.V);
    if ((e = describe(&logits[1], w, false, width / 2)) != cudaSuccess) return e;
    logits[2] = logits[0];
    logits[3] = logits[1];
    if ((e = describe(&products[0], d, false)) != cudaSuccess) return e;
    if ((e = describe(&products[1], w, true)) != cudaSuccess) return e;
    if ((e = describe(&products[2], d, true)) != cudaSuccess) return e;
    if ((e = describe(&products[3], x, true)) != cudaSuccess) return e;
    float *const sums = f.dx >= 0 ? reinterpret_cast<float *>(ws + f.dx) : nullptr;
    const int64_t size = c.dw_bf16 ? 2 : 4;
    // one gradient for all losses is applied to the products, after d's rounding
    const float alpha = c.dlosses ? 1.0f : c.dloss;

    for (int64_t v0 = 0; v0 < c.V; v0 += f.piece) {
        const int64_t cols = c.V - v0 < f.piece ? c.V - v0 : f.piece;
        const bool last = v0 + cols == c.V;
        if (few_long(c)) {
            Few a = {};
            a.lse = c.lse_in;
            a.dlosses = c.dlosses;
            a.d = reinterpret_cast<uint16_t *>(ws + f.d);
            a.ld_d = f.piece;
            e = run_few<true>(c, a, v0, cols, stream);
        } else {
            Args a = {};
            a.job[0] = job_of(c.T, cols, c.D, width);
            a.job[0].box_i = box_of(c.T);
            a.job[0].j_at = int32_t(v0);
            a.job[0].out = ws + f.d;
            a.job[0].ld_out = f.piece;
            a.targets = c.targets;
            a.wide = c.wide;
            a.V = int32_t(c.V);
            a.target_logit = target_logit;
            a.lse = c.lse_in;
            a.dlosses = c.dlosses;
            e = run_logits<kGradient>(logits, a, stream);
        }
        if (e != cudaSuccess) return e;

        Args p = {};
        if (c.dx) {
            Job &j = p.job[0] = job_of(c.T, c.D, cols, f.width);
            j.mn_j = 1;
            j.alpha = alpha;
            j.kj_at = int32_t(v0);
            j.split = int32_t(f.split < j.blocks ? f.split : j.blocks);
            if (sums && !(last && f.split == 1)) {
                j.out = sums;
                j.ld_out = f.ld_dx;
                j.split_out = c.T * f.ld_dx;
                j.vec = 1;
            } else {
                j.out = c.dx;
                j.out_bf16 = c.dx_bf16;
                j.ld_out = c.ld_dx;
                j.vec = aligned(static_cast<const uint16_t *>(c.dx), c.ld_dx);
            }
            if (v0 > 0) {
                j.add = sums;
                j.ld_add = f.ld_dx;
                j.split_add = c.T * f.ld_dx;
            }
        }
        if (c.dw) {
            Job &j = p.job[1] = job_of(cols, c.D, c.T, f.width);
            j.mn_i = j.mn_j = 1;
            j.alpha = alpha;
            j.out = static_cast<char *>(c.dw) + v0 * c.ld_dw * size;
            j.out_bf16 = c.dw_bf16;
            j.ld_out = c.ld_dw;
            j.vec = aligned(static_cast<const uint16_t *>(c.dw), c.ld_dw);
            if (c.accumulate) {
                j.add = j.out;
                j.add_bf16 = c.dw_bf16;
                j.ld_add = c.ld_dw;
            }
        }
        if ((e = run_products(products, p, stream)) != cudaSuccess) return e;
    }
    if (c.dx && f.split > 1) {
        const uint32_t across = uint32_t(ceil_div(f.ld_dx / 4, 256)), down = uint32_t(c.T < 65535 ? c.T : 65535);
        return launch_after(join_sums_kernel, dim3(across, down), dim3(256), 0, stream, 1,
                            static_cast<const float *>(sums), int32_t(f.split), c.T, int32_t(c.D), int32_t(f.ld_dx),
                            c.dx, c.dx_bf16 ? 1 : 0, c.ld_dx, aligned(static_cast<const uint16_t *>(c.dx), c.ld_dx) ? 1 : 0);
    }
    return cudaSuccess;
}

cudaError_t cross_entropy_wait_timeouts(unsigned int *count, bool reset) {
    cudaError_t e = cudaMemcpyFromSymbol(count, g_wait_timeouts, sizeof(*count));
    if (e == cudaSuccess && reset) {
        const unsigned int zero = 0u;
        e = cudaMemcpyToSymbol(g_wait_timeouts, &zero, sizeof(zero));
    }
    return e;
}

}  // namespace wc
