// fp8_matmul.cu -- matrix product of two 8-bit (e4m3) operands with one fp32
// scale per block of 128 along the summed axis, on the tcgen05 tensor cores.
//
//   C[m][n] = sum over blocks kb of
//             sa[m][kb] * sb[n][kb] * (sum over the block's 128 k of a[m][k] * b[n][k])
//
// The scales are any fp32 values, so a block's sum has to leave the tensor
// core before it is scaled.  One block is one step of the pipeline: TMA
// brings 128 bytes of 128 rows of one operand and of NT rows of the other
// (128-byte swizzle, zero fill at every edge), four tcgen05.mma of K = 32 put
// the block's sum into a TMEM buffer, and the epilogue warps read that buffer
// and add it, scaled, to fp32 sums in registers while the tensor core works
// on the next buffers.  The inner sum of 128 products is the tensor core's
// fp32 accumulation; every sum beyond it is an fp32 fma.
//
// A persistent CTA has one TMA thread, one MMA thread and one or two
// warpgroups of epilogue; the three run ahead of one another across tiles.
// The operand with its rows on the MMA's 128 rows is called i, the one on its
// NT columns j.  Few rows of `a` (decoding, short batches) go on j, with the
// weights on i, so the tensor core's 128 rows are full either way.
#include <cuda.h>

#include "wc_device.cuh"
#include "wc_internal.h"

namespace wc {

namespace {

// ---------------------------------------------------------------------------
// PTX
// ---------------------------------------------------------------------------

__device__ unsigned int g_wait_timeouts;

__device__ __forceinline__ uint32_t smem_of(const void *p) {
    return uint32_t(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n.reg .pred p;\n"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        "selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done != 0;
}

// Waits for the phase of that parity to end.  A wait that does not end within
// about two seconds is given up: the role that sees it returns, the others
// run out in turn, and the count of such waits is left for the host.
__device__ __forceinline__ bool mbar_wait_slow(uint32_t bar, uint32_t parity) {
    unsigned long long start, now;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(start));
    for (uint32_t i = 0; i < (1u << 28); ++i) {
        if (mbar_try(bar, parity)) return true;
        if ((i & 63u) == 63u) {
            asm volatile("mov.u64 %0, %globaltimer;" : "=l"(now));
            if (now - start > 2000000000ull) break;
        }
    }
    atomicAdd(&g_wait_timeouts, 1u);
    return false;
}

__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity) {
    if (mbar_try(bar, parity)) return true;
    return mbar_wait_slow(bar, parity);
}

__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// x: byte of the row (a multiple of 128 here), y: row.
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap *map, uint32_t bar,
                                         int32_t x, int32_t y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(map), "r"(bar), "r"(x), "r"(y)
        : "memory");
}

__device__ __forceinline__ void mma_fp8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                        uint32_t add) {
    asm volatile(
        "{\n.reg .pred p;\n"
        "setp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(add)
        : "memory");
}

__device__ __forceinline__ void mma_commit(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
        : "memory");
}

__device__ __forceinline__ void tc_before_sync() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_after_sync() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// Loads N columns of this warp's 32 lanes; the registers hold them only after
// tmem_wait on the same registers.  (The wait takes them as operands, so no
// use of a value can be moved before it.)
__device__ __forceinline__ void tmem_load(uint32_t addr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
}
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}
__device__ __forceinline__ void tmem_load(uint32_t addr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
}
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
}

// Shared-memory operand descriptor: rows of 128 bytes, 128-byte swizzle,
// groups of 8 rows 1024 bytes apart.  Addresses and strides in 16-byte units;
// bit 46 is the descriptor's version, 2 << 61 the swizzle.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr) {
    return uint64_t((addr & 0x3FFFFu) >> 4) | (uint64_t(1) << 16) | (uint64_t(64) << 32) |
           (uint64_t(1) << 46) | (uint64_t(2) << 61);
}

// Instruction descriptor: fp32 accumulators, e4m3 x e4m3, both K-major,
// M = 128, N = nt.
__host__ __device__ constexpr uint32_t instr_desc(int nt) {
    return (1u << 4) | (uint32_t(nt >> 3) << 17) | (uint32_t(128 >> 4) << 24);
}

// ---------------------------------------------------------------------------
// kernel
// ---------------------------------------------------------------------------

constexpr int kRows = 128;   // rows of a tile on i
constexpr int kBlock = 128;  // values per scale: one pipeline step

// Epilogue staging of a warp: 64 bytes (32 bf16 or 16 fp32 columns) of each of
// its 32 rows.  80 bytes from row to row keep 16-byte accesses off one
// another's banks.
constexpr int kStagingPitch = 80;
constexpr int kStagingBytes = 32 * kStagingPitch;

template <int NT>
struct Shape {
    static constexpr int kGroups = NT == 256 ? 2 : 1;  // epilogue warpgroups
    static constexpr int kCols = NT / kGroups;         // columns of one
    static constexpr int kBuffers = NT == 256 ? 2 : 4;
    static constexpr int kTmemCols = kBuffers * NT;
    static constexpr int kChunk = kCols < 32 ? 16 : 32;  // columns of one TMEM load
    static constexpr int kStageBytes = (kRows + NT) * kBlock;
    static constexpr int kStages = NT == 256 ? 4 : NT == 128 ? 6 : 8;
    // two epilogue warpgroups need more than a third of the registers each, so
    // the TMA and MMA warps are part of a full warpgroup that gives its up
    static constexpr bool kSplitRegs = kGroups == 2;
    static constexpr int kThreads = kGroups * 128 + (kSplitRegs ? 128 : 64);
    // stages, one staging buffer per epilogue warp, and room to align
    static constexpr int kSmem = kStages * kStageBytes + kGroups * 4 * kStagingBytes + 1024;
};

struct Side {
    const float *s;
    int64_t ld_s;
    int shift;      // rows per scale: 1 << shift
    int32_t rows;
};

struct Args {
    Side i, j;
    int32_t blocks;          // ceil(K / 128)
    int32_t tiles_i, tiles_j;
    void *out;
    int64_t ld_out;
    int out_bf16, accumulate, vector_out;
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

// A warp's 32 rows x COLS columns of a tile (one row per lane) to out [i][j],
// through shared memory: a lane's row is 64 bytes wide there, and the warp
// writes 64 consecutive bytes of 8 rows at a time, where a store straight from
// the registers would touch 32 rows (measured on 8192 x 11008 x 4096 together
// with the chunked TMEM reads: 0.337 -> 0.306 ms).
template <int COLS, bool BF16>
__device__ __forceinline__ void store_rows(const Args &a, const f32x2 (&acc)[COLS / 2],
                                           uint8_t *staging, int32_t row0, int32_t j0, int lane) {
    constexpr int W = BF16 ? 32 : 16;  // columns of a pass
    constexpr int SIZE = BF16 ? 2 : 4;
    const int32_t rows = a.i.rows - row0;
#pragma unroll
    for (int c0 = 0; c0 < COLS; c0 += W) {
        const int32_t cols = a.j.rows - (j0 + c0);  // of this pass and later ones
        if (cols <= 0 || rows <= 0) break;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (BF16) {
                    float x, y;
                    unpack2(acc[(c0 + q * 8) / 2 + k], x, y);
                    w[k] = f32x2_to_bf16x2_bits(x, y);
                } else if (k % 2 == 0) {
                    float x, y;
                    unpack2(acc[(c0 + q * 4 + k) / 2], x, y);
                    w[k] = __float_as_uint(x);
                    w[k + 1] = __float_as_uint(y);
                }
            }
            *reinterpret_cast<uint4 *>(staging + lane * kStagingPitch + q * 16) =
                make_uint4(w[0], w[1], w[2], w[3]);
        }
        __syncwarp();
        char *base = static_cast<char *>(a.out) + (int64_t(row0) * a.ld_out + j0 + c0) * SIZE;
        if (a.vector_out && cols >= W) {
            const int r0 = lane >> 2, seg = (lane & 3) * 16;
#pragma unroll
            for (int r = r0; r < 32; r += 8)
                if (r < rows)
                    *reinterpret_cast<uint4 *>(base + int64_t(r) * a.ld_out * SIZE + seg) =
                        *reinterpret_cast<const uint4 *>(staging + r * kStagingPitch + seg);
        } else {
            const int c = lane % W;
            for (int r = lane / W; r < 32 && r < rows; r += 32 / W) {
                if (c >= cols) break;
                const uint8_t *p = staging + r * kStagingPitch + c * SIZE;
                char *o = base + (int64_t(r) * a.ld_out + c) * SIZE;
                if (BF16) *reinterpret_cast<uint16_t *>(o) = *reinterpret_cast<const uint16_t *>(p);
                else *reinterpret_cast<uint32_t *>(o) = *reinterpret_cast<const uint32_t *>(p);
            }
        }
        __syncwarp();
    }
}

// The same added to what out holds, straight from the registers.
template <int COLS>
__device__ __forceinline__ void add_row(const Args &a, const f32x2 (&acc)[COLS / 2], int32_t i,
                                        int32_t j0) {
    if (i >= a.i.rows) return;
#pragma unroll
    for (int c = 0; c < COLS; c += 2) {
        float x, y;
        unpack2(acc[c / 2], x, y);
        if (j0 + c < a.j.rows) put(a, int64_t(i) * a.ld_out + j0 + c, x);
        if (j0 + c + 1 < a.j.rows) put(a, int64_t(i) * a.ld_out + j0 + c + 1, y);
    }
}

// VECJ: j has a scale per row (one per column of the tile), else one per 128.
// TRANS: out is [j][i], else [i][j].
template <int NT, bool VECJ, bool TRANS>
__global__ void __launch_bounds__(Shape<NT>::kThreads, 1)
fp8_matmul_kernel(const __grid_constant__ CUtensorMap map_i, const __grid_constant__ CUtensorMap map_j,
                  const Args a) {
    using S = Shape<NT>;
    extern __shared__ uint8_t dynamic_smem[];
    __shared__ uint64_t full[S::kStages], empty[S::kStages], acc_full[S::kBuffers],
        acc_empty[S::kBuffers], drained;
    __shared__ uint32_t tmem_slot;
    __shared__ __align__(16) float sj_smem[VECJ ? S::kGroups : 1][2][VECJ ? S::kCols : 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int kProducer = S::kGroups * 4, kMma = kProducer + 1;
    const uint32_t stages = (smem_of(dynamic_smem) + 1023u) & ~1023u;
    const int32_t tiles = a.tiles_i * a.tiles_j;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S::kStages; ++s) {
            mbar_init(smem_of(&full[s]), 1);
            mbar_init(smem_of(&empty[s]), 1);
        }
        for (int b = 0; b < S::kBuffers; ++b) {
            mbar_init(smem_of(&acc_full[b]), 1);
            mbar_init(smem_of(&acc_empty[b]), S::kGroups * 4);
        }
        mbar_init(smem_of(&drained), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == kMma) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_of(&tmem_slot)),
                     "r"(uint32_t(S::kTmemCols))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(&tmem_slot);
    wait_for_predecessor();  // all above is set-up that reads no operand

    // 384 threads start with 168 registers each: 2 x 128 x 224 + 128 x 56 =
    // 64512 = 384 x 168
    if (warp >= kProducer) {
        if (S::kSplitRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp == kProducer && lane == 0) {
            uint32_t stage = 0, phase = 0, issued = 0;
            bool ok = true;
            for (int32_t t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
                int32_t ti, tj;
                tile_at(a, t, &ti, &tj);
                for (int32_t kb = 0; kb < a.blocks; ++kb) {
                    if (!mbar_wait(smem_of(&empty[stage]), phase ^ 1u)) {
                        ok = false;
                        break;
                    }
                    const uint32_t bar = smem_of(&full[stage]);
                    const uint32_t base = stages + stage * S::kStageBytes;
                    mbar_expect(bar, S::kStageBytes);
                    tma_load(base, &map_i, bar, kb * kBlock, ti * kRows);
                    tma_load(base + kRows * kBlock, &map_j, bar, kb * kBlock, tj * NT);
                    ++issued;
                    if (++stage == S::kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (!ok) {  // let the copies in flight land before the CTA goes
                const uint32_t pending = issued < uint32_t(S::kStages) ? issued : S::kStages;
                for (uint32_t back = pending; back > 0; --back) {
                    const uint32_t n = issued - back;
                    mbar_wait(smem_of(&full[n % S::kStages]), (n / S::kStages) & 1u);
                }
            }
        } else if (warp == kMma && lane == 0) {
            uint32_t stage = 0, phase = 0, buf = 0, buf_phase = 0;
            bool ok = true;
            for (int32_t t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
                for (int32_t kb = 0; kb < a.blocks; ++kb) {
                    if (!mbar_wait(smem_of(&acc_empty[buf]), buf_phase ^ 1u) ||
                        !mbar_wait(smem_of(&full[stage]), phase)) {
                        ok = false;
                        break;
                    }
                    tc_after_sync();
                    const uint32_t base = stages + stage * S::kStageBytes;
                    const uint64_t di = smem_desc(base), dj = smem_desc(base + kRows * kBlock);
#pragma unroll
                    for (int k = 0; k < kBlock / 32; ++k)  // 32 bytes on, in 16-byte units
                        mma_fp8(tmem + buf * NT, di + 2 * k, dj + 2 * k, instr_desc(NT), k > 0);
                    mma_commit(smem_of(&empty[stage]));
                    mma_commit(smem_of(&acc_full[buf]));
                    if (++stage == S::kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                    if (++buf == S::kBuffers) {
                        buf = 0;
                        buf_phase ^= 1u;
                    }
                }
            }
            if (!ok) {  // no product may be in flight when the TMEM is freed
                mma_commit(smem_of(&drained));
                mbar_wait(smem_of(&drained), 0);
            }
        }
    } else {
        if (S::kSplitRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
        const int group = warp >> 2, in_group = threadIdx.x & 127;
        const uint32_t lane_base = tmem + (uint32_t(warp & 3) << 21);
        uint32_t buf = 0, buf_phase = 0;
        bool ok = true;
        // After a wait that ran out the warps go through the rest without
        // waiting or storing, so the barriers below still meet.
        for (int32_t t = blockIdx.x; t < tiles; t += gridDim.x) {
            int32_t ti, tj;
            tile_at(a, t, &ti, &tj);
            const int32_t i = ti * kRows + in_group;
            const int32_t j0 = tj * NT + group * S::kCols;
            const int32_t row_i = min(i, a.i.rows - 1) >> a.i.shift;
            const int32_t row_j = VECJ ? min(j0 + in_group, a.j.rows - 1)
                                       : min(j0, a.j.rows - 1) >> a.j.shift;
            f32x2 acc[S::kCols / 2];
#pragma unroll
            for (int c = 0; c < S::kCols / 2; ++c) acc[c] = pack2(0.0f, 0.0f);
            float si = __ldg(a.i.s + row_i), sj = __ldg(a.j.s + row_j);
            for (int32_t kb = 0; kb < a.blocks; ++kb) {
                float si_next = 0.0f, sj_next = 0.0f;
                if (kb + 1 < a.blocks) {
                    si_next = __ldg(a.i.s + (kb + 1) * a.i.ld_s + row_i);
                    sj_next = __ldg(a.j.s + (kb + 1) * a.j.ld_s + row_j);
                }
                if (VECJ) {
                    if (in_group < S::kCols) sj_smem[group][kb & 1][in_group] = sj;
                    asm volatile("bar.sync %0, 128;" ::"r"(1 + group) : "memory");
                }
                ok = __all_sync(kFull, ok && mbar_wait(smem_of(&acc_full[buf]), buf_phase));
                tc_after_sync();
                const float s = VECJ ? si : __fmul_rn(si, sj);
                const f32x2 s2 = pack2(s, s);
// one chunk's columns load while the previous chunk's are added
                const uint32_t from = lane_base + buf * NT + group * S::kCols;
                uint32_t p[2][S::kChunk];
                tmem_load(from, p[0]);
                tmem_wait(p[0]);
#pragma unroll
                for (int k = 0; k < S::kCols / S::kChunk; ++k) {
                    const int c0 = k * S::kChunk;
                    const bool more = c0 + S::kChunk < S::kCols;
                    if (more) {
                        tmem_load(from + c0 + S::kChunk, p[(k + 1) & 1]);
                    } else {  // all read: the tensor core may have the buffer
                        tc_before_sync();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(smem_of(&acc_empty[buf]));
                    }
#pragma unroll
                    for (int c = 0; c < S::kChunk; c += 4) {
                        const uint32_t *q = &p[k & 1][c];
                        const f32x2 v0 = pack2(__uint_as_float(q[0]), __uint_as_float(q[1]));
                        const f32x2 v1 = pack2(__uint_as_float(q[2]), __uint_as_float(q[3]));
                        const int at = (c0 + c) / 2;
                        if (VECJ) {
                            const float4 w = *reinterpret_cast<const float4 *>(
                                &sj_smem[group][kb & 1][VECJ ? c0 + c : 0]);
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
                if (++buf == S::kBuffers) {
                    buf = 0;
                    buf_phase ^= 1u;
                }
                si = si_next;
                sj = sj_next;
            }
            if (!ok) continue;
            if (TRANS) {
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
                uint8_t *staging = dynamic_smem + (stages - smem_of(dynamic_smem)) +
                                   S::kStages * S::kStageBytes + warp * kStagingBytes;
                const int32_t row0 = ti * kRows + (warp & 3) * 32;
                if (a.accumulate) add_row<S::kCols>(a, acc, i, j0);
                else if (a.out_bf16) store_rows<S::kCols, true>(a, acc, staging, row0, j0, lane);
                else store_rows<S::kCols, false>(a, acc, staging, row0, j0, lane);
            }
        }
    }

    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    if (warp == kMma)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                     "r"(uint32_t(S::kTmemCols)));
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

typedef CUresult (*EncodeTiled)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

cudaError_t encoder(EncodeTiled *out) {
    static EncodeTiled fn = nullptr;  // the driver's function, the same for every call
    if (fn == nullptr) {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        const cudaError_t e =
            cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q);
        if (e != cudaSuccess) return e;
        if (q != cudaDriverEntryPointSuccess || p == nullptr) return cudaErrorNotSupported;
        fn = reinterpret_cast<EncodeTiled>(p);
    }
    *out = fn;
    return cudaSuccess;
}

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

template <int NT, bool VECJ, bool TRANS>
cudaError_t run(const Fp8Matmul &m, const Fp8Operand &oi, const Fp8Operand &oj, int64_t rows_i,
                int64_t rows_j, cudaStream_t stream) {
    using S = Shape<NT>;
    CUtensorMap map_i, map_j;
    cudaError_t e = operand_map(&map_i, oi, rows_i, m.K, kRows);
    if (e == cudaSuccess) e = operand_map(&map_j, oj, rows_j, m.K, NT);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(fp8_matmul_kernel<NT, VECJ, TRANS>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e != cudaSuccess) return e;
    Args a;
    a.i = {oi.s, oi.ld_s, oi.rows_per_scale == 128 ? 7 : 0, int32_t(rows_i)};
    a.j = {oj.s, oj.ld_s, oj.rows_per_scale == 128 ? 7 : 0, int32_t(rows_j)};
    a.blocks = int32_t((m.K + kBlock - 1) / kBlock);
    a.tiles_i = int32_t((rows_i + kRows - 1) / kRows);
    a.tiles_j = int32_t((rows_j + NT - 1) / NT);
    a.out = m.out;
    a.ld_out = m.ld_out;
    a.out_bf16 = m.out_bf16;
    a.accumulate = m.accumulate;
    a.vector_out = !m.accumulate && m.ld_out % (m.out_bf16 ? 8 : 4) == 0;
    const int64_t tiles = int64_t(a.tiles_i) * a.tiles_j;
    const uint32_t grid = uint32_t(tiles < kSms ? tiles : kSms);
    return launch_after(fp8_matmul_kernel<NT, VECJ, TRANS>, dim3(grid), dim3(S::kThreads), S::kSmem,
                        stream, map_i, map_j, a);
}

template <int NT, bool TRANS>
cudaError_t run(const Fp8Matmul &m, const Fp8Operand &oi, const Fp8Operand &oj, int64_t rows_i,
                int64_t rows_j, cudaStream_t stream) {
    return oj.rows_per_scale == 1 ? run<NT, true, TRANS>(m, oi, oj, rows_i, rows_j, stream)
                                  : run<NT, false, TRANS>(m, oi, oj, rows_i, rows_j, stream);
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
    const int64_t wide = ((m.M + 127) / 128) * ((m.N + 255) / 256);
    if (wide < kSms) return run<128, false>(m, m.a, m.b, m.M, m.N, stream);
    return run<256, false>(m, m.a, m.b, m.M, m.N, stream);
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
