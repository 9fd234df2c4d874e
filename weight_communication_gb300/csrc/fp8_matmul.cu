// fp8_matmul.cu -- matrix product of two 8-bit (e4m3) operands with one fp32
// scale per block of 128 along the summed axis, on the tcgen05 tensor cores.
//
//   C[m][n] = sum over blocks kb of
//             sa[m][kb] * sb[n][kb] * (sum over the block's 128 k of a[m][k] * b[n][k])
//
// The scales are fp32 and not powers of two, so a block's sum has to leave the
// tensor core before it is scaled.  It is scaled by the two scales' product, taken
// in fp32: one operation per sum where a side has one scale per 128 rows.  The
// product of any two blocks' scales should be a normal number (the largest
// magnitudes of the blocks, multiplied, between 2.4e-33 and 6.8e43); a subnormal
// one costs up to 2^-125 per block, one that overflows makes the output infinite
// or not a number, even where the block's sum is 0.  One block is one step of the pipeline: TMA
// brings 128 bytes of 128 rows of one operand and of NT rows of the other
// (128-byte swizzle, zero fill at every edge), four tcgen05.mma of K = 32 put
// the block's sum into a TMEM buffer, and the epilogue warps read that buffer
// and add it, scaled, to fp32 sums in registers while the tensor core works
// on the next buffers.  The inner sum of 128 products is the tensor core's
// fp32 accumulation; every sum beyond it is an fp32 fma.
//
// Where the tiles are too few for the GPU, a cluster of up to eight CTAs shares
// each tile's blocks of K and adds its sums through shared memory.
//
// A persistent CTA has a TMA warp, an MMA warp, a warp that brings scales, and
// one or two warpgroups of epilogue; they run ahead of one another across
// tiles.  The operand with its rows on the MMA's 128 rows is called i, the one
// on its NT columns j.  Few rows of `a` (decoding, short batches) go on j, with
// the weights on i, so the tensor core's rows are full either way.
//
// What bounds it: a step keeps half of the TMEM from its products' issue until
// its epilogue has read it -- 512 cycles of products, 190 until their end is
// seen, 380 of reading, 280 until the MMA warp has seen that and issued again --
// so two steps in flight fill the tensor core for 1024 cycles of every 1400.
// 8192 x 11008 x 4096 (weights, one scale per 128 x 128): 0.28 ms, 2.6 PFLOP/s.
// A scale per row on both sides (a weight's gradient) is bound by the fp32 units,
// which have two operations per sum and block there: 5504 x 2048 x 4096 into fp32
// 79 us, 52 with one scale per 128 x 128 on one side.
#include <atomic>

#include "wc_device.cuh"
#include "wc_internal.h"
#include "wc_launch.cuh"
#include "wc_store.cuh"
#include "wc_tcgen05.cuh"
#include "wc_wait.cuh"

namespace wc {

namespace {

// ---------------------------------------------------------------------------
// PTX
// ---------------------------------------------------------------------------

__device__ unsigned int g_wait_timeouts;

// A warp that gives up a wait takes no further part: it arrives on no barrier and
// starts no copy or product, so what the others still complete is complete, and
// they run out in turn.  Every output that misses a sum is NaN, and the waits are
// counted for the host.  (The loops of the TMA and MMA warps are run by all lanes
// alike, so their counters and descriptors are uniform registers.)
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity) {
    return wc::mbar_wait(bar, parity, &g_wait_timeouts);
}

// 16 bytes, those past `bytes` zero.
__device__ __forceinline__ void copy16(uint32_t dst, const float *src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

__device__ __forceinline__ void copy4(uint32_t dst, const float *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

template <bool PAIR>
__device__ __forceinline__ void buffer_free(uint32_t bar) {
    if (PAIR) mbar_arrive_cluster(bar);
    else mbar_arrive(bar);
}

template <bool PAIR>
__device__ __forceinline__ void mma_fp8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                        uint32_t add) {
    if (PAIR)
        asm volatile(
            "{\n.reg .pred p;\n"
            "setp.ne.b32 p, %4, 0;\n"
            "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(add)
            : "memory");
    else
        asm volatile(
            "{\n.reg .pred p;\n"
            "setp.ne.b32 p, %4, 0;\n"
            "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(add)
            : "memory");
}

// 16 lanes x 32 columns: registers 4g .. 4g + 3 of lane l hold row l / 4, columns
// 8g + 2 (l % 4) and the next one, and the same columns of row l / 4 + 8.
__device__ __forceinline__ void tmem_load_fragment(uint32_t addr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
}

// Shared-memory operand descriptor: rows of 128 bytes, 128-byte swizzle,
// groups of 8 rows 1024 bytes apart.  Addresses and strides in 16-byte units;
// bit 46 is the descriptor's version, 2 << 61 the swizzle.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr) {
    return uint64_t((addr & 0x3FFFFu) >> 4) | (uint64_t(1) << 16) | (uint64_t(64) << 32) |
           (uint64_t(1) << 46) | (uint64_t(2) << 61);
}

// Instruction descriptor: fp32 accumulators, e4m3 x e4m3, both K-major.
__host__ __device__ constexpr uint32_t instr_desc(int m, int nt) {
    return (1u << 4) | (uint32_t(nt >> 3) << 17) | (uint32_t(m >> 4) << 24);
}

// ---------------------------------------------------------------------------
// kernel
// ---------------------------------------------------------------------------

constexpr int kRows = 128;   // rows of a tile on i
constexpr int kBlock = 128;  // values per scale: one pipeline step

template <int NT>
struct Shape {
    static constexpr int kGroups = NT >= 128 ? 2 : 1;  // epilogue warpgroups
    static constexpr int kCols = NT / kGroups;         // columns of one
    static constexpr int kBuffers = NT == 256 ? 2 : 4;
    static constexpr int kTmemCols = kBuffers * NT;
    static constexpr int kChunk = kCols < 32 ? 16 : 32;  // columns of one TMEM load
    // NT = 256: two CTAs on neighbouring SMs share a tile of 256 x 256.  Each
    // holds the sums of its own 128 rows of i and brings half the rows of j;
    // the first one's MMA thread multiplies for both.  A lone CTA would need
    // 48 KB per step where each of the pair needs 32 KB, and L2 to shared
    // memory, with the copies and the products sharing shared memory's port,
    // has less to do.  (Alone, 128 x 256 tiles: 8192 x 11008 x 4096 in 0.283 ms
    // at best without any epilogue work; pairs with it: 0.28 ms.)
    static constexpr bool kPair = NT == 256;
    static constexpr int kRowsJ = kPair ? NT / 2 : NT;  // rows of j that this CTA brings
    static constexpr int kStageBytes = (kRows + kRowsJ) * kBlock;
    static constexpr int kStages = NT >= 128 ? 6 : 8;
    // two epilogue warpgroups need more than a third of the registers each, so
    // the TMA and MMA warps are part of a full warpgroup that gives its up
    static constexpr bool kSplitRegs = NT == 256;
    static constexpr int kThreads = kGroups * 128 + 128;
    // Scales of a step (i's rows, then j's columns) come to shared memory three
    // steps ahead, a latency from L2 that one step does not cover.  Copies for
    // step c wait for the product of step c - kScaleSlots + kBuffers + 1, which
    // began after every warp had left the scales of step c - kScaleSlots.
    static constexpr int kScales = kRows + NT;
    static constexpr int kAhead = 3;
    static constexpr int kScaleSlots = kAhead + kBuffers + 3;
    // stages, one staging buffer per epilogue warp, scales, and room to align
    static constexpr int kScalesAt = kStages * kStageBytes + kGroups * 4 * kStagingBytes;
    static constexpr int kSmem = kScalesAt + kScaleSlots * kScales * 4 + 1024;
};

struct Side {
    const float *s;
    int64_t ld_s;
    int shift;      // rows per scale: 1 << shift
    int quads;      // four rows' scales are 16 aligned bytes
    int32_t rows;
};

struct Args {
    Side i, j;
    int32_t blocks;          // ceil(K / 128)
    int32_t tiles_i, tiles_j;
    void *out;
    int64_t ld_out;
    int out_bf16, accumulate, vector_out;
    int32_t split;           // CTAs (one cluster) that share a tile's blocks
};

// A warp's part in copying the scales of ROWS rows of a tile, block after block:
// four consecutive rows per lane where the layout allows, else one by one.
// Rows past the operand's end get a scale that no stored output uses.
template <int ROWS>
struct ScaleRows {
    static constexpr int kSingles = (ROWS + 31) / 32, kQuads = (ROWS + 127) / 128;
    const float *p[kSingles];
    uint32_t bytes[kQuads];
    __device__ __forceinline__ void start(const Side &s, int32_t row0, int step, int32_t block0, int lane) {
        const float *from = s.s + block0 * s.ld_s;
        if (ROWS >= 16 && s.quads) {
#pragma unroll
            for (int r = 0; r < kQuads; ++r) {
                const int32_t row = row0 + 128 * r + 4 * lane, left = s.rows - row;
                p[r] = from + (left > 0 ? row : 0);
                bytes[r] = left >= 4 ? 16u : left > 0 ? 4u * left : 0u;
            }
        } else {
#pragma unroll
            for (int r = 0; r < kSingles; ++r)
                p[r] = from + (min(row0 + (32 * r + lane) * step, s.rows - 1) >> s.shift);
        }
    }
    __device__ __forceinline__ void copy(const Side &s, uint32_t to, int lane) {
        if (ROWS >= 16 && s.quads) {
#pragma unroll
            for (int r = 0; r < kQuads; ++r) {
                if (ROWS >= 128 || lane < ROWS / 4) copy16(to + r * 512 + lane * 16, p[r], bytes[r]);
                p[r] += s.ld_s;
            }
        } else {
#pragma unroll
            for (int r = 0; r < kSingles; ++r) {
                if (ROWS >= 32 || lane < ROWS) copy4(to + r * 128 + lane * 4, p[r]);
                p[r] += s.ld_s;
            }
        }
    }
};

// Tile order: bands of 16 tiles of i, all of j within a band, so that the CTAs
// at work together share operand rows in L2.
__device__ __forceinline__ void tile_at(const Args &a, int32_t t, int32_t *ti, int32_t *tj) {
    const int32_t band = t / (16 * a.tiles_j);
    const int32_t first = band * 16;
    const int32_t high = min(16, a.tiles_i - first);
    const int32_t in = t - band * 16 * a.tiles_j;
    *ti = first + in % high;
    *tj = in / high;
}

__device__ __forceinline__ void put(const Args &a, int64_t at, float x) {
    if (a.out_bf16) {
        uint16_t *p = static_cast<uint16_t *>(a.out) + at;
        if (a.accumulate) x = __fadd_rn(bf16_bits_to_f32(*p), x);
        *p = f32_to_bf16_bits(x);
    } else {
        float *p = static_cast<float *>(a.out) + at;
        if (a.accumulate) x = __fadd_rn(*p, x);
        *p = x;
    }
}

// NaN for a warp's 32 rows x cols columns of a tile, where its sums are missing.
template <bool TRANS>
__device__ __forceinline__ void put_nan(const Args &a, int32_t i0, int32_t j0, int cols, int lane) {
#pragma unroll 1
    for (int r = 0; r < 32 && i0 + r < a.i.rows; ++r)
#pragma unroll 1
        for (int c = lane; c < cols && j0 + c < a.j.rows; c += 32)
            put(a, TRANS ? int64_t(j0 + c) * a.ld_out + i0 + r : int64_t(i0 + r) * a.ld_out + j0 + c,
                __uint_as_float(0x7FC00000u));
}

// What a kernel can do with out: its rows start on 16 bytes and are written; they
// start on any element; out is added to.
enum Rows { kAligned, kAnywhere, kAdded };

// A warp's 32 rows x COLS columns of a tile (one row per lane) to out [i][j],
// through shared memory: a lane's row is 64 bytes wide there, and the warp
// writes 64 consecutive bytes of 8 rows at a time, where a store straight from
// the registers would touch 32 rows (8192 x 11008 x 4096, with the chunked
// TMEM reads: 0.337 -> 0.306 ms).
template <int COLS, bool BF16, bool FRAGMENT, Rows ROWS, bool LAST>
__device__ __forceinline__ void store_rows(const Args &a, const f32x2 (&acc)[COLS / 2],
                                           uint8_t *staging, int32_t row0, int32_t j0, int lane) {
    constexpr int W = BF16 ? 32 : 16;  // columns of a pass
    constexpr int SIZE = BF16 ? 2 : 4;
    const int32_t rows = a.i.rows - row0;
#pragma unroll
    for (int c0 = 0; c0 < COLS; c0 += W) {
        const int32_t cols = a.j.rows - (j0 + c0);  // of this pass and later ones
        if (cols <= 0 || rows <= 0) break;
        if (FRAGMENT) {
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int g = 0; g < W / 8; ++g) {
                    float x, y;
                    unpack2(acc[r * (COLS / 8) + c0 / 8 + g], x, y);
                    uint8_t *to = staging + (8 * r + lane / 4) * kStagingPitch + (8 * g + 2 * (lane & 3)) * SIZE;
                    if (BF16) *reinterpret_cast<uint32_t *>(to) = f32x2_to_bf16x2_bits(x, y);
                    else *reinterpret_cast<float2 *>(to) = make_float2(x, y);
                }
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float x, y;
                    if (BF16) {
                        unpack2(acc[(c0 + q * 8) / 2 + k], x, y);
                        w[k] = f32x2_to_bf16x2_bits(x, y);
                    } else if (k % 2 == 0) {
                        unpack2(acc[(c0 + q * 4 + k) / 2], x, y);
                        w[k] = __float_as_uint(x);
                        w[k + 1] = __float_as_uint(y);
                    }
                }
                *reinterpret_cast<uint4 *>(staging + lane * kStagingPitch + q * 16) =
                    make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
        __syncwarp();
        char *base = static_cast<char *>(a.out) + (int64_t(row0) * a.ld_out + j0 + c0) * (ROWS == kAdded && a.out_bf16 ? 2 : SIZE);
        if (ROWS == kAligned && cols >= W) {
            const int r0 = lane >> 2, seg = (lane & 3) * 16;
#pragma unroll
            for (int r = r0; r < 32; r += 8)
                if (r < rows)
                    *reinterpret_cast<uint4 *>(base + int64_t(r) * a.ld_out * SIZE + seg) =
                        *reinterpret_cast<const uint4 *>(staging + r * kStagingPitch + seg);
        } else if (ROWS == kAdded && a.vector_out && !a.out_bf16 && cols >= W) {
            constexpr int U = FRAGMENT ? 4 : 2;  // accesses of out in flight
            const int seg = (lane & 3) * 16;
            const uint8_t *from = staging + (lane >> 2) * kStagingPitch + seg;
            char *to = base + int64_t(lane >> 2) * a.ld_out * SIZE + seg;
            const int64_t step = 8 * a.ld_out * SIZE;
#pragma unroll 1
            for (int r = lane >> 2; r < 32; r += 8 * U) {
                float4 old[U];
                {
                    const char *p = to;
#pragma unroll
                    for (int k = 0; k < U; ++k) {
                        if (r + 8 * k < rows) old[k] = *reinterpret_cast<const float4 *>(p);
                        p += step;
                    }
                }
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    uint4 v = *reinterpret_cast<const uint4 *>(from);
                    v = make_uint4(__float_as_uint(__fadd_rn(old[k].x, __uint_as_float(v.x))),
                                       __float_as_uint(__fadd_rn(old[k].y, __uint_as_float(v.y))),
                                       __float_as_uint(__fadd_rn(old[k].z, __uint_as_float(v.z))),
                                       __float_as_uint(__fadd_rn(old[k].w, __uint_as_float(v.w))));
                    if (r + 8 * k < rows) *reinterpret_cast<uint4 *>(to) = v;
                    from += 8 * kStagingPitch;
                    to += step;
                }
            }
        } else if (ROWS == kAligned && LAST) {  // the last columns
            const int c = lane % W;
            for (int r = lane / W; r < 32 && r < rows; r += 32 / W) {
                if (c >= cols) break;
                const uint8_t *p = staging + r * kStagingPitch + c * SIZE;
                char *o = base + (int64_t(r) * a.ld_out + c) * SIZE;
                if (BF16) *reinterpret_cast<uint16_t *>(o) = *reinterpret_cast<const uint16_t *>(p);
                else *reinterpret_cast<uint32_t *>(o) = *reinterpret_cast<const uint32_t *>(p);
            }
        } else if (ROWS == kAnywhere && BF16) {
            store_pass_bf16(base, a.ld_out, staging, rows, min(cols, W), lane);
        } else if (ROWS == kAdded && a.out_bf16) {
            store_pass_f32<ROWS == kAdded>(reinterpret_cast<uint16_t *>(base), a.ld_out, staging, rows, cols, lane);
        } else if (ROWS != kAligned) {
            store_pass_f32<ROWS == kAdded>(reinterpret_cast<float *>(base), a.ld_out, staging, rows, cols, lane);
        }
        __syncwarp();
    }
}

// The columns past the last whole pass, straight from the registers.
template <int COLS>
__device__ __forceinline__ void store_last_columns(const Args &a, const f32x2 (&acc)[COLS / 2], int32_t i,
                                                   int32_t j0) {
    const int32_t left = a.j.rows - j0, first = a.out_bf16 ? left & ~31 : left & ~15;
    if (i >= a.i.rows || first >= COLS || first == left) return;
#pragma unroll
    for (int c = 0; c < COLS; c += 2) {
        float x, y;
        unpack2(acc[c / 2], x, y);
        if (c >= first && c < left) put(a, int64_t(i) * a.ld_out + j0 + c, x);
        if (c >= first && c + 1 < left) put(a, int64_t(i) * a.ld_out + j0 + c + 1, y);
    }
}

// (Sums to be added to out stay fp32 until then.)  LAST: the columns past the last
// whole pass go through shared memory too.  Straight from the registers they take
// longer (777 x 1112 x 555: 8.7 us instead of 6.2), but large tiles with one scale
// for their columns have no registers left for that loop, and few such ends.
template <int COLS, bool FRAGMENT, Rows ROWS, bool LAST>
__device__ __forceinline__ void store_tile(const Args &a, const f32x2 (&acc)[COLS / 2], uint8_t *staging,
                                           int32_t row0, int32_t i, int32_t j0, int lane) {
    if (a.out_bf16 && ROWS != kAdded)
        store_rows<COLS, true, FRAGMENT, ROWS, LAST>(a, acc, staging, row0, j0, lane);
    else
        store_rows<COLS, false, FRAGMENT, ROWS, LAST>(a, acc, staging, row0, j0, lane);
    if (ROWS == kAligned && !LAST) store_last_columns<COLS>(a, acc, i, j0);
}

// Sums of a tile over the CTAs that share its blocks.  Each has left its own in
// shared memory as lines of 128 consecutive outputs (TRANS: columns of the tile,
// else rows), kPartialPitch values apart; each adds every split-th line over the
// cluster and stores it.  It begins with its own part and goes round, so the
// order is fixed for each line and no CTA is read by all others at once (all from
// the first one on: 128 x 1003 x 11008 with eight CTAs 15 us, so 10.3).
// missing: a CTA of the cluster gave up, so every line is NaN.
constexpr int kPartialPitch = 132;

__device__ __forceinline__ void st_cluster_u32(uint32_t addr, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

template <bool TRANS, int NT, int WARPS>
__device__ __forceinline__ void add_partials(const Args &a, int32_t tile, int32_t part, uint32_t partial,
                                             bool missing, int warp, int lane) {
    int32_t ti, tj;
    tile_at(a, tile, &ti, &tj);
    const int32_t line0 = TRANS ? tj * NT : ti * kRows, at0 = (TRANS ? ti * kRows : tj * NT) + 4 * lane;
    const int32_t lines = min(TRANS ? NT : kRows, (TRANS ? a.j.rows : a.i.rows) - line0);
    const int32_t left = (TRANS ? a.i.rows : a.j.rows) - at0;
    for (int32_t line = part + a.split * warp; line < lines; line += a.split * WARPS) {
        const uint32_t addr = partial + (line * kPartialPitch + 4 * lane) * 4;
        float4 x = ld_cluster_f4(in_cta(addr, part));
#pragma unroll 2
        for (int32_t p = 1, from = part; p < a.split; ++p) {
            if (++from == a.split) from = 0;
            const float4 y = ld_cluster_f4(in_cta(addr, from));
            x.x = __fadd_rn(x.x, y.x);
            x.y = __fadd_rn(x.y, y.y);
            x.z = __fadd_rn(x.z, y.z);
            x.w = __fadd_rn(x.w, y.w);
        }
        if (missing) {
            const float nan = __uint_as_float(0x7FC00000u);
            x = make_float4(nan, nan, nan, nan);
        }
        if (left <= 0) continue;
        const int64_t at = int64_t(line0 + line) * a.ld_out + at0;
        if (a.vector_out && !a.accumulate && left >= 4) {
            if (a.out_bf16)
                *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + at) =
                    make_uint2(f32x2_to_bf16x2_bits(x.x, x.y), f32x2_to_bf16x2_bits(x.z, x.w));
            else
                *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + at) = x;
        } else {
            put(a, at, x.x);
            if (left > 1) put(a, at + 1, x.y);
            if (left > 2) put(a, at + 2, x.z);
            if (left > 3) put(a, at + 3, x.w);
        }
    }
}

// VECJ: j has a scale per row (one per column of the tile), else one per 128.
// TRANS: out is [j][i], else [i][j].  ROWS: for the large tiles, whose sums leave
// few registers (the other cases' code in the same kernel: 8192 x 11008 x 4096
// 329 us instead of 279); the others choose as they store.
template <int NT, bool VECJ, bool TRANS, Rows ROWS>
__global__ void __launch_bounds__(Shape<NT>::kThreads, 1)
fp8_matmul_kernel(const __grid_constant__ CUtensorMap map_i, const __grid_constant__ CUtensorMap map_j,
                  const Args a) {
    using S = Shape<NT>;
    constexpr bool kPair = S::kPair;
    constexpr int kTileRows = kPair ? 2 * kRows : kRows;
    constexpr int kChunk = NT == 256 && ROWS != kAligned ? 16 : S::kChunk;
    constexpr bool kFragment = VECJ && NT == 256;  // TMEM is read in fragments
    constexpr int kProducer = S::kGroups * 4, kMma = kProducer + 1, kScaler = kProducer + 2;
    extern __shared__ uint8_t dynamic_smem[];
    // full[stage]: the step's operands are here, and the TMEM buffer it goes to
    // is free.  done[stage]: its product is complete, and its scales are here.
    // (One barrier to wait for and one to arrive on keep the MMA thread's work
    // beside the products short: the queue of products is two deep.)
    __shared__ uint64_t full[S::kStages], done[S::kStages], drained;
    __shared__ uint32_t tmem_slot, gave_up;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t stages = (smem_of(dynamic_smem) + 1023u) & ~1023u;
    uint8_t *const aligned_smem = dynamic_smem + (stages - smem_of(dynamic_smem));
    float *const scales = reinterpret_cast<float *>(aligned_smem + S::kScalesAt);
    float *const partial = reinterpret_cast<float *>(aligned_smem);
    const int32_t tiles = a.tiles_i * a.tiles_j;
    // the CTAs of a pair are neighbours in the grid and work on one tile
    const int32_t rank = kPair ? int32_t(blockIdx.x & 1) : 0;
    const uint32_t sharing = kPair ? 2u : uint32_t(a.split);  // CTAs of a tile
    const int32_t first_tile = int32_t(blockIdx.x / sharing), tile_step = int32_t(gridDim.x / sharing);
    // this CTA's blocks of K
    const int32_t part = kPair ? 0 : int32_t(blockIdx.x % sharing);
    const int32_t block0 = kPair ? 0 : a.blocks * part / a.split;
    const int32_t blocks = kPair ? a.blocks : a.blocks * (part + 1) / a.split - block0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S::kStages; ++s) {
            mbar_init(smem_of(&full[s]), 1 + S::kGroups * 4 * (kPair ? 2 : 1));
            mbar_init(smem_of(&done[s]), 2);
        }
        mbar_init(smem_of(&drained), 1);
        gave_up = 0u;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    __syncwarp();
    if (warp == kMma) tmem_alloc<kPair>(smem_of(&tmem_slot), S::kTmemCols);
    tc_before_sync();
    __syncthreads();
    if (kPair) cluster_sync();  // the other CTA's barriers are ready too
    tc_after_sync();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(&tmem_slot);
    wait_for_predecessor();  // all above is set-up that reads no operand

    // 384 threads start with 168 registers each: 2 x 128 x 224 + 128 x 56 =
    // 64512 = 384 x 168
    if (warp >= kProducer) {
        if (S::kSplitRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp == kProducer) {
            uint32_t stage = 0, phase = 0;
            bool ok = true;
            for (int32_t t = first_tile; ok && t < tiles; t += tile_step) {
                int32_t ti, tj;
                tile_at(a, t, &ti, &tj);
                for (int32_t kb = 0; kb < blocks; ++kb) {
                    ok = mbar_wait(smem_of(&done[stage]), phase ^ 1u);
                    if (!ok) break;
                    if (elected()) {
                        // the first CTA's barrier counts the bytes of both
                        const uint32_t local = smem_of(&full[stage]);
                        const uint32_t bar = kPair ? in_cta(local, 0) : local;
                        const uint32_t base = stages + stage * S::kStageBytes;
                        if (rank == 0) mbar_expect(local, S::kStageBytes * (kPair ? 2 : 1));
                        tma_load<kPair>(base, &map_i, bar, (block0 + kb) * kBlock,
                                        ti * kTileRows + rank * kRows);
                        tma_load<kPair>(base + kRows * kBlock, &map_j, bar, (block0 + kb) * kBlock,
                                        tj * NT + rank * S::kRowsJ);
                    }
                    __syncwarp();
                    if (++stage == S::kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (!ok) wait_ms(20);  // for the copies in flight to land before the CTA goes
        } else if (warp == kMma && rank == 0) {
            uint32_t stage = 0, phase = 0, buf = 0;
            bool ok = true;
            const bool lead = elected();
            for (int32_t t = first_tile; ok && t < tiles; t += tile_step) {
                for (int32_t kb = 0; kb < blocks; ++kb) {
                    ok = mbar_wait(smem_of(&full[stage]), phase);
                    if (!ok) break;
                    tc_after_sync();
                    if (lead) {
                        const uint32_t base = stages + stage * S::kStageBytes;
                        const uint64_t di = smem_desc(base), dj = smem_desc(base + kRows * kBlock);
#pragma unroll
                        for (int k = 0; k < kBlock / 32; ++k)  // 32 bytes on, in 16-byte units
                            mma_fp8<kPair>(tmem + buf * NT, di + 2 * k, dj + 2 * k,
                                           instr_desc(kTileRows, NT), k > 0);
                        mma_commit<kPair>(smem_of(&done[stage]));
                    }
                    __syncwarp();
                    if (++stage == S::kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                    if (++buf == S::kBuffers) buf = 0;
                }
            }
            // No product may be in flight when the TMEM is freed.  (The epilogue has
            // waited for the last one too, unless it gave up.)
            if (lead) mma_commit<kPair>(smem_of(&drained), 1);
            __syncwarp();
            mbar_wait(smem_of(&drained), 0);
        } else if (warp == kScaler) {
            const int32_t mine = first_tile < tiles ? (tiles - 1 - first_tile) / tile_step + 1 : 0;
            const int64_t steps = int64_t(mine) * blocks;
            int32_t t = first_tile, kb = 0;  // of the next step to copy
            uint32_t slot = 0, stage = 0, seen = 0, seen_phase = 0;
            ScaleRows<kRows> si;
            ScaleRows<VECJ ? NT : S::kGroups> sj;
            for (int64_t g = -S::kAhead; g < steps; ++g) {
                if (g + S::kAhead - S::kScaleSlots + S::kBuffers + 1 >= 0) {
                    if (!mbar_wait(smem_of(&done[seen]), seen_phase)) break;
                    if (++seen == S::kStages) {
                        seen = 0;
                        seen_phase ^= 1u;
                    }
                }
                if (t < tiles) {  // (blocks > 0)
                    if (kb == 0) {
                        int32_t ti, tj;
                        tile_at(a, t, &ti, &tj);
                        si.start(a.i, ti * kTileRows + rank * kRows, 1, block0, lane);
                        sj.start(a.j, tj * NT, VECJ ? 1 : S::kCols, block0, lane);
                    }
                    const uint32_t to = smem_of(scales + slot * S::kScales);
                    si.copy(a.i, to, lane);
                    sj.copy(a.j, to + kRows * 4, lane);
                    if (++slot == S::kScaleSlots) slot = 0;
                    if (++kb == blocks) {
                        kb = 0;
                        t += tile_step;
                    }
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
                if (g < 0) continue;
                // all but the last kAhead steps' copies have landed
                asm volatile("cp.async.wait_group %0;" ::"n"(S::kAhead) : "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_of(&done[stage]));
                __syncwarp();
                if (++stage == S::kStages) stage = 0;
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
        }
    } else {
        if (S::kSplitRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
        const int group = warp >> 2, in_group = threadIdx.x & 127;
        const uint32_t from0 = tmem + (uint32_t(warp & 3) << 21) + group * S::kCols;
        uint32_t stage = 0, phase = 0, buf = 0, slot = 0;
        bool ok = true;
        // The buffer of step g is free for step g + kBuffers: an arrival on that
        // step's barrier in the first CTA.  All buffers are free at the start.
        const bool lead = elected();
        const uint32_t full0 = kPair ? in_cta(smem_of(&full[0]), 0) : smem_of(&full[0]);
        uint32_t freed = S::kBuffers;
        for (int b = 0; b < S::kBuffers; ++b)
            if (lead) buffer_free<kPair>(full0 + b * 8);
        for (int32_t t = first_tile; t < tiles; t += tile_step) {
            int32_t ti, tj;
            tile_at(a, t, &ti, &tj);
            const int32_t i = ti * kTileRows + rank * kRows + in_group;
            const int32_t j0 = tj * NT + group * S::kCols;
            f32x2 acc[S::kCols / 2];
#pragma unroll
            for (int c = 0; c < S::kCols / 2; ++c) acc[c] = pack2(0.0f, 0.0f);
            for (int32_t kb = 0; ok && kb < blocks; ++kb) {
                ok = mbar_wait(smem_of(&done[stage]), phase);
                if (!ok) break;
                tc_after_sync();
                const uint32_t from = from0 + buf * NT;
                const float *sc = scales + slot * S::kScales;
                if (++slot == S::kScaleSlots) slot = 0;
                if (++buf == S::kBuffers) buf = 0;
                if (++stage == S::kStages) {
                    stage = 0;
                    phase ^= 1u;
                }
                const float *sj = sc + kRows + group * S::kCols;
                if (kFragment) {
                    // rows 16 h + l / 4 + 8 q, columns 8 k + 2 (l % 4): a lane meets a
                    // quarter of the columns, so their scales cost a quarter of the
                    // shared-memory reads of one row per lane
                    f32x2 si[2][2];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float x = sc[(warp & 3) * 32 + 8 * r + lane / 4];
                        si[r / 2][r % 2] = pack2(x, x);
                    }
                    const f32x2 zero = pack2(-0.0f, -0.0f);
                    uint32_t p[2][16];
                    tmem_load_fragment(from, p[0]);
                    tmem_wait(p[0]);
                    f32x2 wj[4];
#pragma unroll
                    for (int u = 0; u < S::kCols / 16; ++u) {
                        const int c0 = u / 2 * 32, h = u % 2;
                        if (u + 1 < S::kCols / 16) {
                            tmem_load_fragment(from + (u + 1) / 2 * 32 + (((u + 1) % 2) << 20), p[(u + 1) & 1]);
                        } else {
                            tc_before_sync();  // all read: the tensor core may have the buffer
                            __syncwarp();
                            if (lead) buffer_free<kPair>(full0 + freed * 8);
                            if (++freed == S::kStages) freed = 0;
                        }
#pragma unroll
                        for (int g = 0; g < 4; ++g) {
                            if (h == 0) {
                                const float2 x = *reinterpret_cast<const float2 *>(sj + c0 + 8 * g + 2 * (lane & 3));
                                wj[g] = pack2(x.x, x.y);
                            }
#pragma unroll
                            for (int q = 0; q < 2; ++q) {
                                const uint32_t *v = &p[u & 1][4 * g + 2 * q];
                                const int at = (h * 2 + q) * (S::kCols / 8) + c0 / 8 + g;
                                acc[at] = fma2_rn(pack2(__uint_as_float(v[0]), __uint_as_float(v[1])),
                                                  fma2_rn(si[h][q], wj[g], zero), acc[at]);
                            }
                        }
                        if (u + 1 < S::kCols / 16) tmem_wait(p[(u + 1) & 1]);
                    }
                    continue;
                }
                uint32_t p[2][kChunk];
                tmem_load(from, p[0]);
                const float s = VECJ ? sc[in_group] : __fmul_rn(sc[in_group], sc[kRows + group]);
                const f32x2 s2 = pack2(s, s);
                tmem_wait(p[0]);
                // one chunk's columns load while the previous chunk's are added
#pragma unroll
                for (int k = 0; k < S::kCols / kChunk; ++k) {
                    const int c0 = k * kChunk;
                    const bool more = c0 + kChunk < S::kCols;
                    if (more) {
                        tmem_load(from + c0 + kChunk, p[(k + 1) & 1]);
                    } else {  // all read: the tensor core may have the buffer
                        tc_before_sync();
                        __syncwarp();
                        if (lead) buffer_free<kPair>(full0 + freed * 8);
                        if (++freed == S::kStages) freed = 0;
                    }
#pragma unroll
                    for (int c = 0; c < kChunk; c += 4) {
                        const uint32_t *q = &p[k & 1][c];
                        const f32x2 v0 = pack2(__uint_as_float(q[0]), __uint_as_float(q[1]));
                        const f32x2 v1 = pack2(__uint_as_float(q[2]), __uint_as_float(q[3]));
                        const int at = (c0 + c) / 2;
                        if (VECJ) {
                            const float4 w = *reinterpret_cast<const float4 *>(sj + c0 + c);
                            const f32x2 zero = pack2(-0.0f, -0.0f);
                            acc[at] = fma2_rn(v0, fma2_rn(s2, pack2(w.x, w.y), zero), acc[at]);
                            acc[at + 1] = fma2_rn(v1, fma2_rn(s2, pack2(w.z, w.w), zero), acc[at + 1]);
                        } else {
                            acc[at] = fma2_rn(v0, s2, acc[at]);
                            acc[at + 1] = fma2_rn(v1, s2, acc[at + 1]);
                        }
                    }
                    if (more) tmem_wait(p[(k + 1) & 1]);
                }
            }
            if (!ok) {  // this tile and all later ones of this warp
                if (!kPair && a.split > 1) {  // its part is missing in every CTA of the cluster
                    if (lane < a.split) st_cluster_u32(in_cta(smem_of(&gave_up), lane), 1u);
                    break;
                }
                put_nan<TRANS>(a, i - lane, j0, S::kCols, lane);
                continue;
            }
            if (!kPair && a.split > 1) {
                // the last product is complete, so the stages are free
#pragma unroll
                for (int c = 0; c < S::kCols; c += 4) {
                    float x[4];
                    unpack2(acc[c / 2], x[0], x[1]);
                    unpack2(acc[c / 2 + 1], x[2], x[3]);
                    const int at = group * S::kCols + c;
                    if (TRANS) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) partial[(at + k) * kPartialPitch + in_group] = x[k];
                    } else {
                        *reinterpret_cast<float4 *>(partial + in_group * kPartialPitch + at) =
                            make_float4(x[0], x[1], x[2], x[3]);
                    }
                }
            } else if (TRANS) {
                if (i < a.i.rows) {
#pragma unroll
                    for (int c = 0; c < S::kCols; c += 2) {
                        float x, y;
                        unpack2(acc[c / 2], x, y);
                        if (j0 + c < a.j.rows) put(a, int64_t(j0 + c) * a.ld_out + i, x);
                        if (j0 + c + 1 < a.j.rows) put(a, int64_t(j0 + c + 1) * a.ld_out + i, y);
                    }
                }
            } else {
                uint8_t *staging = aligned_smem + S::kStages * S::kStageBytes + warp * kStagingBytes;
                const int32_t row0 = ti * kTileRows + rank * kRows + (warp & 3) * 32;
                if (NT == 256)
                    store_tile<S::kCols, kFragment, ROWS, kFragment>(a, acc, staging, row0, i, j0, lane);
                else if (a.accumulate)
                    store_tile<S::kCols, kFragment, kAdded, true>(a, acc, staging, row0, i, j0, lane);
                else if (a.vector_out)
                    store_tile<S::kCols, kFragment, kAligned, true>(a, acc, staging, row0, i, j0, lane);
                else
                    store_tile<S::kCols, kFragment, kAnywhere, true>(a, acc, staging, row0, i, j0, lane);
            }
        }
    }

    if (!kPair && a.split > 1) {
        __syncwarp();
        cluster_sync();
        if (warp < kProducer && first_tile < tiles)
            add_partials<TRANS, NT, S::kGroups * 4>(a, first_tile, part, smem_of(partial),
                                                    *reinterpret_cast<volatile uint32_t *>(&gave_up) != 0u,
                                                    warp, lane);
        cluster_sync();
    }
    tc_before_sync();
    __syncthreads();
    // neither CTA's memory goes before the other one is done with it
    if (kPair) cluster_sync();
    tc_after_sync();
    if (warp == kMma) tmem_free<kPair>(tmem, S::kTmemCols);
}

// out = 0 (or unchanged) where there is nothing to sum.
__global__ void __launch_bounds__(256) zero_kernel(void *out, int bf16, int64_t M, int64_t N, int64_t ld) {
    for (int64_t at = int64_t(blockIdx.x) * 256 + threadIdx.x; at < M * N; at += int64_t(gridDim.x) * 256) {
        const int64_t m = at / N, n = at - m * N;
        if (bf16) static_cast<uint16_t *>(out)[m * ld + n] = 0;
        else static_cast<float *>(out)[m * ld + n] = 0.0f;
    }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------

cudaError_t operand_map(CUtensorMap *map, const Fp8Operand &op, int64_t rows, int64_t K, int box_rows) {
    EncodeTiled encode;
    const cudaError_t e = encoder(&encode);
    if (e != cudaSuccess) return e;
    const cuuint64_t dims[2] = {cuuint64_t(K), cuuint64_t(rows)};
    const cuuint64_t strides[1] = {cuuint64_t(op.ld)};
    const cuuint32_t box[2] = {kBlock, cuuint32_t(box_rows)};
    const cuuint32_t step[2] = {1, 1};
    const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t *>(op.q), dims,
                              strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

constexpr int kSms = 152;

bool vector_out(const Fp8Matmul &m) { return m.ld_out % (m.out_bf16 ? 8 : 4) == 0; }

Side side_of(const Fp8Operand &op, int64_t rows) {
    const bool each = op.rows_per_scale == 1;
    return {op.s, op.ld_s, each ? 0 : 7, each && op.ld_s % 4 == 0, int32_t(rows)};
}

// Clusters of `size` CTAs that run at once, as CUDA counts them (GB300: 76,
// 46, 36, 28, 23, 15, 15 of 2 to 8 -- the SMs of a GPC do not divide evenly).
// Every shape of the kernel has an SM to itself, so the count is the GPU's alone
// and is asked for once.
template <typename Kernel>
int clusters_of(Kernel kernel, int threads, int smem, int device, int size) {
    static std::atomic<int> known[64][9];
    if (device < 64 && known[device][size].load(std::memory_order_relaxed) > 0)
        return known[device][size].load(std::memory_order_relaxed);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(size) * kSms);
    cfg.blockDim = dim3(unsigned(threads));
    cfg.dynamicSmemBytes = size_t(smem);
    cudaLaunchAttribute attr[1] = {};
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = unsigned(size);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
        (void)cudaGetLastError();
        n = 0;  // no split
    }
    if (device < 64) known[device][size].store(n, std::memory_order_relaxed);
    return n;
}

// CTAs that share a tile's blocks of K: as many as run at once, three blocks or
// more each, and none where that saves less than adding the sums costs (a block
// takes 0.3 us; the exchange 2.5 us for 128 x 128 sums, 1 us for fewer columns).
// One token, 4096 x 11008: 28.9 -> 10.8 us; 128 x 1003 x 11008: 32.9 -> 10.3;
// 5 blocks on 63 tiles of 128 x 128 would take 8.7 us instead of 7.4.
template <typename Kernel>
int32_t split_of(Kernel kernel, int threads, int smem, int device, int64_t tiles, int32_t blocks,
                 int32_t worth) {
    if (tiles > kSms / 2) return 1;
    for (int32_t s = 8; s > 1; --s)
        if (blocks >= 3 * s && blocks - (blocks + s - 1) / s >= worth &&
            tiles <= clusters_of(kernel, threads, smem, device, s))
            return s;
    return 1;
}

template <int NT, bool VECJ, bool TRANS, Rows ROWS>
cudaError_t run(const Fp8Matmul &m, const Fp8Operand &oi, const Fp8Operand &oj, int64_t rows_i,
                int64_t rows_j, cudaStream_t stream) {
    using S = Shape<NT>;
    CUtensorMap map_i, map_j;
    cudaError_t e = operand_map(&map_i, oi, rows_i, m.K, kRows);
    if (e == cudaSuccess) e = operand_map(&map_j, oj, rows_j, m.K, S::kRowsJ);
    if (e != cudaSuccess) return e;
    // once for each GPU: the kernel's attribute stays set
    static std::atomic<uint64_t> prepared{0};
    int device = 0;
    if ((e = cudaGetDevice(&device)) != cudaSuccess) return e;
    const uint64_t bit = uint64_t(1) << (device & 63);
    if (device > 63 || !(prepared.load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute(fp8_matmul_kernel<NT, VECJ, TRANS, ROWS>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
        if (e != cudaSuccess) return e;
        prepared.fetch_or(bit, std::memory_order_relaxed);
    }
    Args a;
    a.i = side_of(oi, rows_i);
    a.j = side_of(oj, rows_j);
    a.blocks = int32_t((m.K + kBlock - 1) / kBlock);
    const int tile_rows = S::kPair ? 2 * kRows : kRows;
    a.tiles_i = int32_t((rows_i + tile_rows - 1) / tile_rows);
    a.tiles_j = int32_t((rows_j + NT - 1) / NT);
    a.out = m.out;
    a.ld_out = m.ld_out;
    a.out_bf16 = m.out_bf16;
    a.accumulate = m.accumulate;
    a.vector_out = vector_out(m);
    const int64_t tiles = int64_t(a.tiles_i) * a.tiles_j;
    const int64_t places = S::kPair ? kSms / 2 : kSms;
    a.split = 1;
    if constexpr (!S::kPair)
        a.split = split_of(fp8_matmul_kernel<NT, VECJ, TRANS, ROWS>, S::kThreads, S::kSmem, device, tiles,
                           a.blocks, NT >= 128 ? 8 : 4);
    const uint32_t cluster = S::kPair ? 2 : uint32_t(a.split);
    const uint32_t grid = uint32_t(tiles < places ? tiles : places) * cluster;
    return launch_after(fp8_matmul_kernel<NT, VECJ, TRANS, ROWS>, dim3(grid), dim3(S::kThreads), S::kSmem,
                        stream, cluster, map_i, map_j, a);
}

template <int NT, bool TRANS, Rows ROWS = kAligned>
cudaError_t run(const Fp8Matmul &m, const Fp8Operand &oi, const Fp8Operand &oj, int64_t rows_i,
                int64_t rows_j, cudaStream_t stream) {
    return oj.rows_per_scale == 1 ? run<NT, true, TRANS, ROWS>(m, oi, oj, rows_i, rows_j, stream)
                                  : run<NT, false, TRANS, ROWS>(m, oi, oj, rows_i, rows_j, stream);
}

}  // namespace

cudaError_t launch_fp8_matmul(const Fp8Matmul &m, cudaStream_t stream) {
    if (m.K == 0) {
        if (m.accumulate) return cudaSuccess;
        const int64_t ctas = (m.M * m.N + 255) / 256;
        const uint32_t grid = uint32_t(ctas < 8 * kSms ? ctas : 8 * kSms);
        zero_kernel<<<grid, 256, 0, stream>>>(m.out, m.out_bf16 ? 1 : 0, m.M, m.N, m.ld_out);
        return cudaPeekAtLastError();
    }
    if (m.M <= 16) return run<16, true>(m, m.b, m.a, m.N, m.M, stream);
    if (m.M <= 32) return run<32, true>(m, m.b, m.a, m.N, m.M, stream);
    if (m.M <= 64) return run<64, true>(m, m.b, m.a, m.N, m.M, stream);
    // a block takes a CTA of 128 x 128 as long as a pair of 256 x 256, so the small
    // tiles serve where one wave of them is enough (4411 x 638 x 9433: 175 small
    // tiles in two waves 55 us, 54 large ones 34)
    const int64_t small = ((m.M + 127) / 128) * ((m.N + 127) / 128);
    if (small <= kSms) return run<128, false>(m, m.a, m.b, m.M, m.N, stream);
    if (m.accumulate) return run<256, false, kAdded>(m, m.a, m.b, m.M, m.N, stream);
    if (!vector_out(m)) return run<256, false, kAnywhere>(m, m.a, m.b, m.M, m.N, stream);
    return run<256, false, kAligned>(m, m.a, m.b, m.M, m.N, stream);
}

cudaError_t fp8_wait_timeouts(unsigned int *count, bool reset) {
    cudaError_t e = cudaMemcpyFromSymbol(count, g_wait_timeouts, sizeof(*count));
    if (e == cudaSuccess && reset) {
        const unsigned int zero = 0u;
        e = cudaMemcpyToSymbol(g_wait_timeouts, &zero, sizeof(zero));
    }
    return e;
}

}  // namespace wc
