// wc_internal.h -- launchers shared between the kernel files and the C ABI.
// Arguments reaching these have been validated by the ABI layer.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace wc {

// Sizes of one qgZ problem.  All element indices fit in 32 bits: the ABI
// rejects R*N >= 2^32.
struct QgzGeometry {
    uint32_t N;                // elements per rank
    uint32_t S;                // slice (shard) length, N / R
    uint32_t R;                // ranks
    uint32_t G;                // groups
    uint32_t L;                // ranks per group, R / G
    uint32_t blocks_per_rank;  // N / B
    uint32_t total;            // R * N
};

// ef: NULL, or the error buffer [R][N] in the form ef_mode names: 1 fp32,
// 2 bf16, 3 int8 codes with ef_scales [R][N/B] fp32 (gradient order).
constexpr int kEfModeF32 = 1, kEfModeBf16 = 2, kEfModeInt8 = 3;
cudaError_t launch_ef_quant_int4(const uint16_t *g, void *ef, int ef_mode, float *ef_scales,
                                 uint8_t *codes, float *scales, const QgzGeometry &geo, int B,
                                 float s, float beta, cudaStream_t stream);
cudaError_t launch_dequant_reduce(const uint8_t *codes, const float *scales,
                                  const QgzGeometry &geo, int B, float out_scale, void *out,
                                  bool out_bf16, cudaStream_t stream);
// ef1: fp32 [G*N] error of every requantized value (unit order), or NULL.
cudaError_t launch_dequant_reduce_requant(const uint8_t *codes, const float *scales,
                                          uint8_t *out_codes, float *out_scales,
                                          const QgzGeometry &geo, int B, float *ef1, float s,
                                          float beta, cudaStream_t stream);
// ef, ef_mode, ef_scales as in launch_ef_quant_int4; codes/scales: the
// ranks' send buffers, or both NULL.
cudaError_t launch_qgz_fused_step(const uint16_t *g, void *ef, int ef_mode, float *ef_scales,
                                  uint8_t *codes, float *scales, const QgzGeometry &geo, int B,
                                  float s, float beta, float out_scale, void *out, bool out_bf16,
                                  cudaStream_t stream);
// The same, with out_codes/out_scales the first hop's output as
// launch_dequant_reduce_requant writes it and ef1 its error buffer or NULL.
cudaError_t launch_qgz_first_hop_fused(const uint16_t *g, void *ef, int ef_mode,
                                       float *ef_scales, uint8_t *codes, float *scales,
                                       const QgzGeometry &geo, int B, float s, float beta,
                                       uint8_t *out_codes, float *out_scales, float *ef1,
                                       cudaStream_t stream);
// replica: bf16 [n] written with the dequantized weights, or NULL.
cudaError_t launch_qwz_quant_int8(const uint16_t *w, int8_t *codes, float *scales,
                                  uint16_t *replica, uint32_t n, int B, cudaStream_t stream);
cudaError_t launch_qwz_dequant_int8(const int8_t *codes, const float *scales, uint16_t *w_out,
                                    uint32_t n, int B, cudaStream_t stream);
cudaError_t launch_sr_accumulate(uint16_t *dst, uint16_t *src, uint32_t n, uint32_t seed,
                                 uint32_t step, cudaStream_t stream);
uint32_t sr_key(uint32_t seed, uint32_t step);

// One gradient tensor: n values at src, and where its clipped values go.
struct GradSpan {
    const void *src;
    void *dst;
    int64_t n;
    bool src_bf16, dst_bf16;
};
// Tensors whose addresses fit one launch's arguments, and the partial sums
// (fp64) that a launch leaves.
constexpr int kGradSpansPerLaunch = 1024, kGradPartialsPerLaunch = 608;
// stats: [0] norm and, with clip, [1] coefficient.
cudaError_t launch_grad_norm(const GradSpan *spans, int count, double *partials, bool clip,
                             bool in_place, double max_norm, double eps, float *stats,
                             cudaStream_t stream);

cudaError_t launch_embedding(const void *table, bool bf16, int64_t ld_table, const void *ids,
                             bool wide, int64_t n, int64_t first, int64_t V, int64_t D,
                             float scale, void *out, int64_t ld_out, cudaStream_t stream);
struct EmbeddingGrad {
    const void *dy;
    bool dy_bf16;
    int64_t ld_dy;
    const void *ids;
    bool wide;  // 64-bit ids
    int64_t n, first, V, D;
    float scale;
    bool accumulate;
    void *dtable;
    bool out_bf16;
    int64_t ld_out;
    void *workspace;
};
// Bytes of workspace; reads n, V and D alone.
int64_t embedding_grad_workspace(const EmbeddingGrad &a);
cudaError_t launch_embedding_grad(const EmbeddingGrad &a, cudaStream_t stream);

// 8-bit floating point (e4m3) with one fp32 scale per block of 128.
struct Fp8Quant {
    const void *x;
    bool x_bf16;
    int64_t rows, cols, ld;
    bool square;               // one scale per 128 x 128 instead of 1 x 128
    uint8_t *q;                // [rows][ld_q], or NULL
    int64_t ld_q;
    float *s;                  // [ceil(cols/128)][ld_s]
    int64_t ld_s;
    uint8_t *qt;               // [cols][ld_qt], or NULL
    int64_t ld_qt;
    float *st;                 // [ceil(rows/128)][ld_st]
    int64_t ld_st;
};
cudaError_t launch_fp8_quant(const Fp8Quant &a, cudaStream_t stream);
struct Fp8Operand {
    const uint8_t *q;          // [rows][ld]
    int64_t ld;
    const float *s;            // [ceil(K/128)][ld_s]
    int64_t ld_s;
    int rows_per_scale;        // 1 or 128
};
struct Fp8Matmul {
    Fp8Operand a, b;
    int64_t M, N, K;
    void *out;                 // [M][ld_out]
    bool out_bf16;
    int64_t ld_out;
    bool accumulate;
};
cudaError_t launch_fp8_matmul(const Fp8Matmul &a, cudaStream_t stream);
// Waits of the product's kernels that ran out (0 unless a launch went wrong).
cudaError_t fp8_wait_timeouts(unsigned int *count, bool reset);

// Violation record of one source file's kernels in a checked build (see
// WC_IN_BOUNDS in wc_device.cuh).  sr_accumulate.cu has none: its kernel
// tests every access against the element count as part of its own logic.
struct CheckRecord {
    unsigned int count;       // accesses skipped since the last reset
    unsigned int first_line;  // source line of the first one (0: none)
};

#if defined(WC_CHECKED) && WC_CHECKED
cudaError_t check_record_qgz_quant(CheckRecord *out, bool reset, bool probe);
cudaError_t check_record_qgz_reduce(CheckRecord *out, bool reset, bool probe);
cudaError_t check_record_qgz_hop1(CheckRecord *out, bool reset, bool probe);
cudaError_t check_record_qgz_fused(CheckRecord *out, bool reset, bool probe);
cudaError_t check_record_qwz(CheckRecord *out, bool reset, bool probe);
#endif

}  // namespace wc
