// abi.cu -- the extern "C" entry points declared in include/wc.h: argument
// validation on the host, then one kernel launch per call (the gradient norm,
// clipping and the embedding's gradient: two or three, back to back).
#include <math.h>
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include <algorithm>
#include <new>
#include <vector>

#include "../../include/wc.h"
#include "wc_internal.h"

namespace {

thread_local char g_last_error[512] = "";

int fail(int code, const char *fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_last_error, sizeof(g_last_error), fmt, ap);
    va_end(ap);
    return code;
}

int from_cuda(cudaError_t err, const char *what) {
    if (err == cudaSuccess) return WC_OK;
    // Reported here, so cleared: the launches ask for the last error, and a later
    // call would find this one again.  (One that ended the context stays.)
    (void)cudaGetLastError();
    return fail(WC_ECUDA, "%s: %s (%s)", what, cudaGetErrorName(err), cudaGetErrorString(err));
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool pow2_in(int64_t b, int64_t lo, int64_t hi) {
    return b >= lo && b <= hi && (b & (b - 1)) == 0;
}

// Validates the sizes shared by the qgZ entry points and fills `geo`.
// Returns WC_OK, or an error code with the message set.
int qgz_geometry(const char *fn, int64_t N, int R, int G, int B, wc::QgzGeometry *geo) {
    if (N < 0) return fail(WC_EINVAL, "%s: N = %lld is negative", fn, (long long)N);
    if (R < 1 || G < 1) return fail(WC_EINVAL, "%s: need R >= 1 and G >= 1 (R=%d, G=%d)", fn, R, G);
    if (R % G) return fail(WC_EINVAL, "%s: G=%d does not divide R=%d", fn, G, R);
    if (!pow2_in(B, 32, 1024))
        return fail(WC_EINVAL, "%s: block B=%d must be a power of two in [32, 1024]", fn, B);
    if (N % R) return fail(WC_EINVAL, "%s: R=%d does not divide N=%lld", fn, R, (long long)N);
    const int64_t S = N / R;
    if (S % B) return fail(WC_EINVAL, "%s: B=%d does not divide the shard N/R=%lld", fn, B, (long long)S);
    // (R*N < 2^32 with B >= 32 dividing N/R also keeps R below 65536, the
    // grid's y limit that the reduce uses for destinations.)
    if (N >= (int64_t(1) << 32) || N * (int64_t)R >= (int64_t(1) << 32))
        return fail(WC_ERANGE, "%s: R*N = %lld must be below 2^32", fn, (long long)(N * R));
    geo->N = uint32_t(N);
    geo->S = uint32_t(S);
    geo->R = uint32_t(R);
    geo->G = uint32_t(G);
    geo->L = uint32_t(R / G);
    geo->blocks_per_rank = uint32_t(N / B);
    geo->total = uint32_t(N * R);
    return WC_OK;
}

#define WC_REQUIRE_PTR(fn, p)                                                        \
    do {                                                                             \
        if ((p) == nullptr) return fail(WC_EINVAL, "%s: %s is NULL", fn, #p);        \
        if (!aligned16(p)) return fail(WC_EALIGN, "%s: %s is not 16-byte aligned", fn, #p); \
    } while (0)

}  // namespace

extern "C" {

WC_API const char *wc_last_error(void) { return g_last_error; }

WC_API int wc_version(void) { return 1 * 10000 + 0 * 100 + 0; }

WC_API int wc_ef_quant_int4(const uint16_t *g, float *ef, uint8_t *codes, float *scales,
                            int64_t N, int R, int G, int B, float err_scale, float err_beta,
                            void *stream) {
    static const char *fn = "wc_ef_quant_int4";
    wc::QgzGeometry geo;
    int rc = qgz_geometry(fn, N, R, G, B, &geo);
    if (rc != WC_OK) return rc;
    if (N == 0) return WC_OK;
    WC_REQUIRE_PTR(fn, g);
    WC_REQUIRE_PTR(fn, codes);
    WC_REQUIRE_PTR(fn, scales);
    if (ef != nullptr && !aligned16(ef)) return fail(WC_EALIGN, "%s: ef is not 16-byte aligned", fn);
    return from_cuda(wc::launch_ef_quant_int4(g, ef, wc::kEfModeF32, nullptr, codes, scales, geo,
                                              B, err_scale, err_beta,
                                              static_cast<cudaStream_t>(stream)),
                     fn);
}

WC_API int wc_ef_quant_int4_bf16ef(const uint16_t *g, uint16_t *ef16, uint8_t *codes,
                                   float *scales, int64_t N, int R, int G, int B,
                                   float err_scale, float err_beta, void *stream) {
    static const char *fn = "wc_ef_quant_int4_bf16ef";
    wc::QgzGeometry geo;
    int rc = qgz_geometry(fn, N, R, G, B, &geo);
    if (rc != WC_OK) return rc;
    if (N == 0) return WC_OK;
    WC_REQUIRE_PTR(fn, g);
    WC_REQUIRE_PTR(fn, ef16);
    WC_REQUIRE_PTR(fn, codes);
    WC_REQUIRE_PTR(fn, scales);
    return from_cuda(wc::launch_ef_quant_int4(g, ef16, wc::kEfModeBf16, nullptr, codes, scales,
                                              geo, B, err_scale, err_beta,
                                              static_cast<cudaStream_t>(stream)),
                     fn);
}

WC_API int wc_ef_quant_int4_int8ef(const uint16_t *g, int8_t *ef8, float *ef8_scales,
                                   uint8_t *codes, float *scales, int64_t N, int R, int G,
                                   int B, float err_scale, float err_beta, void *stream) {
    static const char *fn = "wc_ef_quant_int4_int8ef";
    wc::QgzGeometry geo;
    int rc = qgz_geometry(fn, N, R, G, B, &geo);
    if (rc != WC_OK) return rc;
    if (N == 0) return WC_OK;
    WC_REQUIRE_PTR(fn, g);
    WC_REQUIRE_PTR(fn, ef8);
    WC_REQUIRE_PTR(fn, ef8_scales);
    WC_REQUIRE_PTR(fn, codes);
    WC_REQUIRE_PTR(fn, scales);
    return from_cuda(wc::launch_ef_quant_int4(g, ef8, wc::kEfModeInt8, ef8_scales, codes, scales,
                                              geo, B, err_scale, err_beta,
                                              static_cast<cudaStream_t>(stream)),
                     fn);
}

WC_API int wc_dequant_reduce(const uint8_t *codes, const float *scales, int64_t N, int R,
                             int G, int B, float out_scale, void *out, int out_dtype,
                             void *stream) {
    static const char *fn = "wc_dequant_reduce";
    wc::QgzGeometry geo;
    int rc = qgz_geometry(fn, N, R, G, B, &geo);
    if (rc != WC_OK) return rc;
    if (out_dtype != WC_F32 && out_dtype != WC_BF16)
        return fail(WC_EINVAL, "%s: out_dtype %d is neither WC_F32 nor WC_BF16", fn, out_dtype);
    if (N == 0) return WC_OK;
    WC_REQUIRE_PTR(fn, codes);
    WC_REQUIRE_PTR(fn, scales);
    WC_REQUIRE_PTR(fn, out);
    return from_cuda(wc::launch_dequant_reduce(codes, scales, geo, B, out_scale, out,
                                               out_dtype == WC_BF16,
                                               static_cast<cudaStream_t>(stream)),
                     fn);
}

WC_API int wc_dequant_reduce_requant(const uint8_t *codes, const float *scales, int64_t N,
                                     int R, int G, int B, uint8_t *out_codes,
                                     float *out_scales, void *stream) {
    static const char *fn = "wc_dequant_reduce_requant";
    wc::QgzGeometry geo;
    int rc = qgz_geometry(fn, N, R, G, B, &geo);
    if (rc != WC_OK) return rc;
    if (N * (int64_t)G >= (int64_t(1) << 32))
        return fail(WC_ERANGE, "%s: G*N must be below 2^32", fn);
    if (N == 0) return WC_OK;
    WC_REQUIRE_PTR(fn, codes);
    WC_REQUIRE_PTR(fn, scales);
    WC_REQUIRE_PTR(fn, out_codes);
    WC_REQUIRE_PTR(fn, out_scales);
    return from_cuda(wc::launch_dequant_reduce_requant(codes, scales, out_codes, out_scales, geo,
                                                       B, nullptr, 0.0f, 0.0f,
                                                       static_cast<cudaStream_t>(stream)),
                     fn);
}

WC_API int wc_dequant_reduce_requant_ef(const uint8_t *codes, const float *scales, int64_t N,
                                        int R, int G, int B, uint8_t *out_codes,
                                        float *out_scales, float *ef1, float err_scale,
                                        float err_beta, void *stream) {
    static const char *fn = "wc_dequant_reduce_requant_ef";
    wc::QgzGeometry geo;
    int rc = qgz_geometry(fn, N, R, G, B, &geo);
    if (rc != WC_OK) return rc;
    if (N * (int64_t)G >= (int64_t(1) << 32))
        return fail(WC_ERANGE, "%s: G*N must be below 2^32", fn);
    if (N == 0) return WC_OK;
    WC_REQUIRE_PTR(fn, codes);
    WC_REQUIRE_PTR(fn, scales);
    WC_REQUIRE_PTR(fn, out_codes);
    WC_REQUIRE_PTR(fn, out_scales);
    WC_REQUIRE_PTR(fn, ef1);
    return from_cuda(wc::launch_dequant_reduce_requant(codes, scales, out_codes, out_scales, geo,
                                                       B, ef1, err_scale, err_beta,
                                                       static_cast<cudaStream_t>(stream)),
                     fn);
}

// The fused step's checks and launch for every error-buffer form (ef_mode:
// the buffer's form; ef_needed: the entry point takes no NULL buffer).
static int fused_step(const char *fn, const uint16_t *g, void *ef, int ef_mode, bool ef_needed,
                      float *ef_scales, uint8_t *codes, float *scales, int64_t N, int R, int B,
                      float err_scale, float err_beta, float out_scale, void *out, int out_dtype,
                      void *stream) {
    wc::QgzGeometry geo;
    int rc = qgz_geometry(fn, N, R, 1, B, &geo);
    if (rc != WC_OK) return rc;
    if (B < 128) return fail(WC_EINVAL, "%s: block B=%d must be at least 128", fn, B);
    if (out_dtype != WC_F32 && out_dtype != WC_BF16)
        return fail(WC_EINVAL, "%s: out_dtype %d is neither WC_F32 nor WC_BF16", fn, out_dtype);
    if ((codes == nullptr) != (scales == nullptr))
        return fail(WC_EINVAL, "%s: codes and scales must both be given or both be NULL", fn);
    if (N == 0) return WC_OK;
    WC_REQUIRE_PTR(fn, g);
    WC_REQUIRE_PTR(fn, out);
    if (ef_needed) WC_REQUIRE_PTR(fn, ef);
    if (ef != nullptr && !aligned16(ef)) return fail(WC_EALIGN, "%s: ef is not 16-byte aligned", fn);
    if (ef_mode == wc::kEfModeInt8) WC_REQUIRE_PTR(fn, ef_scales);
    if (codes != nullptr && (!aligned16(codes) || !aligned16(scales)))
        return fail(WC_EALIGN, "%s: codes or scales is not 16-byte aligned", fn);
    return from_cuda(wc::launch_qgz_fused_step(g, ef, ef_mode, ef_scales, codes, scales, geo, B,
                                               err_scale, err_beta, out_scale, out,
                                               out_dtype == WC_BF16,
                                               static_cast<cudaStream_t>(stream)),
                     fn);
}

WC_API int wc_qgz_step_fused(const uint16_t *g, float *ef, uint8_t *codes, float *scales,
                             int64_t N, int R, int B, float err_scale, float err_beta,
                             float out_scale, void *out, int out_dtype, void *stream) {
    return fused_step("wc_qgz_step_fused", g, ef, wc::kEfModeF32, false, nullptr, codes, scales,
                      N, R, B, err_scale, err_beta, out_scale, out, out_dtype, stream);
}

WC_API int wc_qgz_step_fused_bf16ef(const uint16_t *g, uint16_t *ef16, uint8_t *codes,
                                    float *scales, int64_t N, int R, int B, float err_scale,
                                    float err_beta, float out_scale, void *out, int out_dtype,
                                    void *stream) {
    return fused_step("wc_qgz_step_fused_bf16ef", g, ef16, wc::kEfModeBf16, true, nullptr, codes,
                      scales, N, R, B, err_scale, err_beta, out_scale, out, out_dtype, stream);
}

WC_API int wc_qgz_step_fused_int8ef(const uint16_t *g, int8_t *ef8, float *ef8_scales,
                                    uint8_t *codes, float *scales, int64_t N, int R, int B,
                                    float err_scale, float err_beta, float out_scale, void *out,
                                    int out_dtype, void *stream) {
    return fused_step("wc_qgz_step_fused_int8ef", g, ef8, wc::kEfModeInt8, true, ef8_scales,
                      codes, scales, N, R, B, err_scale, err_beta, out_scale, out, out_dtype,
                      stream);
}

// The fused first stage's checks and launch for every error-buffer form.
static int first_hop_fused(const char *fn, const uint16_t *g, void *ef, int ef_mode,
                           bool ef_needed, float *ef_scales, uint8_t *codes, float *scales,
                           int64_t N, int R, int G, int B, float err_scale, float err_beta,
                           uint8_t *out_codes, float *out_scales, float *ef1, void *stream) {
    wc::QgzGeometry geo;
    int rc = qgz_geometry(fn, N, R, G, B, &geo);
    if (rc != WC_OK) return rc;
    if (B < 128) return fail(WC_EINVAL, "%s: block B=%d must be at least 128", fn, B);
    if (N * (int64_t)G >= (int64_t(1) << 32))
        return fail(WC_ERANGE, "%s: G*N must be below 2^32", fn);
    if ((codes == nullptr) != (scales == nullptr))
        return fail(WC_EINVAL, "%s: codes and scales must both be given or both be NULL", fn);
    if (N == 0) return WC_OK;
    WC_REQUIRE_PTR(fn, g);
    WC_REQUIRE_PTR(fn, out_codes);
    WC_REQUIRE_PTR(fn, out_scales);
    if (ef_needed) WC_REQUIRE_PTR(fn, ef);
    if (ef != nullptr && !aligned16(ef)) return fail(WC_EALIGN, "%s: ef is not 16-byte aligned", fn);
    if (ef_mode == wc::kEfModeInt8) WC_REQUIRE_PTR(fn, ef_scales);
    if (codes != nullptr && (!aligned16(codes) || !aligned16(scales)))
        return fail(WC_EALIGN, "%s: codes or scales is not 16-byte aligned", fn);
    if (!aligned16(out_codes) || !aligned16(out_scales))
        return fail(WC_EALIGN, "%s: out_codes or out_scales is not 16-byte aligned", fn);
    if (ef1 != nullptr && !aligned16(ef1)) return fail(WC_EALIGN, "%s: ef1 is not 16-byte aligned", fn);
    return from_cuda(wc::launch_qgz_first_hop_fused(g, ef, ef_mode, ef_scales, codes, scales, geo,
                                                    B, err_scale, err_beta, out_codes, out_scales,
                                                    ef1, static_cast<cudaStream_t>(stream)),
                     fn);
}

WC_API int wc_qgz_first_hop_fused(const uint16_t *g, float *ef, uint8_t *codes, float *scales,
                                  int64_t N, int R, int G, int B, float err_scale,
                                  float err_beta, uint8_t *out_codes, float *out_scales,
                                  float *ef1, void *stream) {
    return first_hop_fused("wc_qgz_first_hop_fused", g, ef, wc::kEfModeF32, false, nullptr, codes,
                           scales, N, R, G, B, err_scale, err_beta, out_codes, out_scales, ef1,
                           stream);
}

WC_API int wc_qgz_first_hop_fused_bf16ef(const uint16_t *g, uint16_t *ef16, uint8_t *codes,
                                         float *scales, int64_t N, int R, int G, int B,
                                         float err_scale, float err_beta, uint8_t *out_codes,
                                         float *out_scales, float *ef1, void *stream) {
    return first_hop_fused("wc_qgz_first_hop_fused_bf16ef", g, ef16, wc::kEfModeBf16, true,
                           nullptr, codes, scales, N, R, G, B, err_scale, err_beta, out_codes,
                           out_scales, ef1, stream);
}

WC_API int wc_qgz_first_hop_fused_int8ef(const uint16_t *g, int8_t *ef8, float *ef8_scales,
                                         uint8_t *codes, float *scales, int64_t N, int R, int G,
                                         int B, float err_scale, float err_beta,
                                         uint8_t *out_codes, float *out_scales, float *ef1,
                                         void *stream) {
    return first_hop_fused("wc_qgz_first_hop_fused_int8ef", g, ef8, wc::kEfModeInt8, true,
                           ef8_scales, codes, scales, N, R, G, B, err_scale, err_beta, out_codes,
                           out_scales, ef1, stream);
}

static int qwz_sizes(const char *fn, int64_t n, int B) {
    if (n < 0) return fail(WC_EINVAL, "%s: n = %lld is negative", fn, (long long)n);
    if (!pow2_in(B, 32, 4096))
        return fail(WC_EINVAL, "%s: block B=%d must be a power of two in [32, 4096]", fn, B);
    if (n % B) return fail(WC_EINVAL, "%s: B=%d does not divide n=%lld", fn, B, (long long)n);
    if (n >= (int64_t(1) << 32)) return fail(WC_ERANGE, "%s: n must be below 2^32", fn);
    return WC_OK;
}

WC_API int wc_qwz_quant_int8(const uint16_t *w, int8_t *codes, float *scales, int64_t n, int B,
                             void *stream) {
    static const char *fn = "wc_qwz_quant_int8";
    int rc = qwz_sizes(fn, n, B);
    if (rc != WC_OK) return rc;
    if (n == 0) return WC_OK;
    WC_REQUIRE_PTR(fn, w);
    WC_REQUIRE_PTR(fn, codes);
    WC_REQUIRE_PTR(fn, scales);
    return from_cuda(wc::launch_qwz_quant_int8(w, codes, scales, nullptr, uint32_t(n), B,
                                               static_cast<cudaStream_t>(stream)),
                     fn);
}

WC_API int wc_qwz_quant_replica_int8(const uint16_t *w, int8_t *codes, float *scales,
                                     uint16_t *replica, int64_t n, int B, void *stream) {
    static const char *fn = "wc_qwz_quant_replica_int8";
    int rc = qwz_sizes(fn, n, B);
    if (rc != WC_OK) return rc;
    if (n == 0) return WC_OK;
    WC_REQUIRE_PTR(fn, w);
    WC_REQUIRE_PTR(fn, codes);
    WC_REQUIRE_PTR(fn, scales);
    WC_REQUIRE_PTR(fn, replica);
    return from_cuda(wc::launch_qwz_quant_int8(w, codes, scales, replica, uint32_t(n), B,
                                               static_cast<cudaStream_t>(stream)),
                     fn);
}

WC_API int wc_qwz_dequant_int8(const int8_t *codes, const float *scales, uint16_t *w_out,
                               int64_t n, int B, void *stream) {
    static const char *fn = "wc_qwz_dequant_int8";
    int rc = qwz_sizes(fn, n, B);
    if (rc != WC_OK) return rc;
    if (n == 0) return WC_OK;
    WC_REQUIRE_PTR(fn, codes);
    WC_REQUIRE_PTR(fn, scales);
    WC_REQUIRE_PTR(fn, w_out);
    return from_cuda(wc::launch_qwz_dequant_int8(codes, scales, w_out, uint32_t(n), B,
                                                 static_cast<cudaStream_t>(stream)),
                     fn);
}

WC_API int wc_sr_accumulate_bf16(uint16_t *dst, uint16_t *src, int64_t n, uint32_t seed,
                                 uint32_t step, void *stream) {
    static const char *fn = "wc_sr_accumulate_bf16";
    if (n < 0) return fail(WC_EINVAL, "%s: n = %lld is negative", fn, (long long)n);
    if (n >= (int64_t(1) << 32)) return fail(WC_ERANGE, "%s: n must be below 2^32", fn);
    if (n == 0) return WC_OK;
    WC_REQUIRE_PTR(fn, dst);
    WC_REQUIRE_PTR(fn, src);
    const uintptr_t a = reinterpret_cast<uintptr_t>(dst), b = reinterpret_cast<uintptr_t>(src);
    const uintptr_t bytes = uintptr_t(n) * 2u;
    if (a < b + bytes && b < a + bytes) return fail(WC_EINVAL, "%s: dst and src overlap", fn);
    return from_cuda(wc::launch_sr_accumulate(dst, src, uint32_t(n), seed, step,
                                              static_cast<cudaStream_t>(stream)),
                     fn);
}

namespace {

bool float_type(int t) { return t == WC_F32 || t == WC_BF16; }

struct Extent {
    uintptr_t begin, end;
    bool written;
};

// Checks one list of tensors and appends them (dst: where the values go).
int span_list(const char *fn, const char *name, const wc_span *spans, int count) {
    for (int i = 0; i < count; ++i) {
        const wc_span &s = spans[i];
        if (!float_type(s.dtype))
            return fail(WC_EINVAL, "%s: %s[%d] has dtype %d, neither WC_F32 nor WC_BF16", fn, name, i,
                        s.dtype);
        if (s.n < 0) return fail(WC_EINVAL, "%s: %s[%d] has n = %lld", fn, name, i, (long long)s.n);
        if (s.n >= (int64_t(1) << 40)) return fail(WC_ERANGE, "%s: %s[%d] has 2^40 values or more", fn, name, i);
        if (s.n > 0 && s.data == nullptr) return fail(WC_EINVAL, "%s: %s[%d] is NULL", fn, name, i);
        const uintptr_t size = s.dtype == WC_BF16 ? 2 : 4;
        if (reinterpret_cast<uintptr_t>(s.data) % size)
            return fail(WC_EALIGN, "%s: %s[%d] is not aligned to its %d-byte values", fn, name, i, int(size));
    }
    return WC_OK;
}

// No written tensor may share memory with another tensor of the call.
int disjoint(const char *fn, const std::vector<Extent> &extents) {
    bool ordered = true;  // usually the list is in address order already
    for (size_t i = 1; ordered && i < extents.size(); ++i)
        ordered = extents[i - 1].begin <= extents[i].begin;
    const std::vector<Extent> *v = &extents;
    std::vector<Extent> sorted;
    if (!ordered) {
        sorted = extents;
        std::sort(sorted.begin(), sorted.end(),
                  [](const Extent &a, const Extent &b) { return a.begin < b.begin; });
        v = &sorted;
    }
    uintptr_t read_end = 0, write_end = 0;
    for (const Extent &e : *v) {
        if (e.begin < write_end || (e.written && e.begin < read_end))
            return fail(WC_EINVAL, "%s: a written tensor overlaps another one", fn);
        uintptr_t &end = e.written ? write_end : read_end;
        end = std::max(end, e.end);
    }
    return WC_OK;
}

int grad_call(const char *fn, const wc_span *spans, const wc_span *dst, int count, bool clip,
              double max_norm, double eps, float *stats, void *workspace, int64_t workspace_bytes,
              void *stream) {
    if (count < 0) return fail(WC_EINVAL, "%s: count = %d is negative", fn, count);
    if (count > 0 && spans == nullptr) return fail(WC_EINVAL, "%s: spans is NULL", fn);
    if (clip && !(max_norm >= 0.0)) return fail(WC_EINVAL, "%s: max_norm = %g must be at least 0", fn, max_norm);
    if (clip && !(eps >= 0.0 && eps < HUGE_VAL))
        return fail(WC_EINVAL, "%s: eps = %g must be finite and at least 0", fn, eps);
    int rc = span_list(fn, "spans", spans, count);
    if (rc == WC_OK && dst != nullptr) rc = span_list(fn, "dst", dst, count);
    if (rc != WC_OK) return rc;
    WC_REQUIRE_PTR(fn, stats);
    WC_REQUIRE_PTR(fn, workspace);
    if (workspace_bytes < wc_grad_norm_workspace(count))
        return fail(WC_EINVAL, "%s: workspace of %lld bytes, %lld are needed", fn,
                    (long long)workspace_bytes, (long long)wc_grad_norm_workspace(count));
    try {
        std::vector<wc::GradSpan> list;
        list.reserve(size_t(count));
        std::vector<Extent> extents;
        if (clip) extents.reserve(size_t(count) * (dst ? 2 : 1));
        int64_t total = 0;
        for (int i = 0; i < count; ++i) {
            const wc_span &s = spans[i];
            const wc_span &d = dst ? dst[i] : s;
            if (d.n != s.n)
                return fail(WC_EINVAL, "%s: dst[%d] has %lld values, spans[%d] %lld", fn, i,
                            (long long)d.n, i, (long long)s.n);
            list.push_back({s.data, d.data, s.n, s.dtype == WC_BF16, d.dtype == WC_BF16});
            total += s.n;
            if (total >= (int64_t(1) << 40)) return fail(WC_ERANGE, "%s: 2^40 values or more in all", fn);
            if (!clip || s.n == 0) continue;
            const uintptr_t a = reinterpret_cast<uintptr_t>(s.data), b = reinterpret_cast<uintptr_t>(d.data);
            extents.push_back({a, a + uintptr_t(s.n) * (s.dtype == WC_BF16 ? 2 : 4), dst == nullptr});
            if (dst) extents.push_back({b, b + uintptr_t(s.n) * (d.dtype == WC_BF16 ? 2 : 4), true});
        }
        if (clip && (rc = disjoint(fn, extents)) != WC_OK) return rc;
        return from_cuda(wc::launch_grad_norm(list.data(), count, static_cast<double *>(workspace),
                                              clip, dst == nullptr, max_norm, eps, stats,
                                              static_cast<cudaStream_t>(stream)),
                         fn);
    } catch (const std::bad_alloc &) {
        return fail(WC_EINVAL, "%s: no host memory for a list of %d tensors", fn, count);
    }
}

// Sizes shared by the embedding's two directions.
int embedding_sizes(const char *fn, int id_type, int64_t n, int64_t first, int64_t V, int64_t D) {
    if (id_type != WC_I32 && id_type != WC_I64)
        return fail(WC_EINVAL, "%s: id_type %d is neither WC_I32 nor WC_I64", fn, id_type);
    if (n < 0 || V < 0 || D < 0)
        return fail(WC_EINVAL, "%s: n = %lld, V = %lld, D = %lld must not be negative", fn, (long long)n,
                    (long long)V, (long long)D);
    if (first < 0 || first >= (int64_t(1) << 62))
        return fail(WC_EINVAL, "%s: first = %lld must be in [0, 2^62)", fn, (long long)first);
    // (the kernels step past the last token or row in 32 bits)
    const int64_t limit = (int64_t(1) << 31) - 4096;
    if (n > limit || V > limit) return fail(WC_ERANGE, "%s: n or V exceeds 2^31 - 4096", fn);
    if (D > (int64_t(1) << 22)) return fail(WC_ERANGE, "%s: D exceeds 2^22", fn);
    if (D > 0 && n >= (int64_t(1) << 40) / D) return fail(WC_ERANGE, "%s: n * D reaches 2^40", fn);
    return WC_OK;
}

// Ids are read one at a time, so they start on any id.
int ids_pointer(const char *fn, const void *ids, int id_type) {
    const uintptr_t size = id_type == WC_I64 ? 8 : 4;
    if (ids == nullptr) return fail(WC_EINVAL, "%s: ids is NULL", fn);
    if (reinterpret_cast<uintptr_t>(ids) % size)
        return fail(WC_EALIGN, "%s: ids is not aligned to its %d-byte values", fn, int(size));
    return WC_OK;
}

int64_t blocks128(int64_t n) { return (n + 127) / 128; }

}  // namespace

WC_API int64_t wc_grad_norm_workspace(int count) {
    const int64_t launches = count > 0 ? (int64_t(count) + wc::kGradSpansPerLaunch - 1) / wc::kGradSpansPerLaunch : 1;
    return launches * wc::kGradPartialsPerLaunch * int64_t(sizeof(double));
}

WC_API int wc_grad_norm(const wc_span *spans, int count, float *stats, void *workspace,
                        int64_t workspace_bytes, void *stream) {
    return grad_call("wc_grad_norm", spans, nullptr, count, false, 0.0, 0.0, stats, workspace,
                     workspace_bytes, stream);
}

WC_API int wc_grad_clip(const wc_span *spans, const wc_span *dst, int count, double max_norm,
                        double eps, float *stats, void *workspace, int64_t workspace_bytes,
                        void *stream) {
    return grad_call("wc_grad_clip", spans, dst, count, true, max_norm, eps, stats, workspace,
                     workspace_bytes, stream);
}

WC_API int wc_embedding(const void *table, int dtype, int64_t ld_table, const void *ids,
                        int id_type, int64_t n, int64_t first, int64_t V, int64_t D, float scale,
                        void *out, int64_t ld_out, void *stream) {
    static const char *fn = "wc_embedding";
    int rc = embedding_sizes(fn, id_type, n, first, V, D);
    if (rc != WC_OK) return rc;
    if (!float_type(dtype)) return fail(WC_EINVAL, "%s: dtype %d is neither WC_F32 nor WC_BF16", fn, dtype);
    if (ld_table < D || ld_out < D)
        return fail(WC_EINVAL, "%s: ld_table = %lld, ld_out = %lld are below D = %lld", fn,
                    (long long)ld_table, (long long)ld_out, (long long)D);
    if (n == 0 || D == 0) return WC_OK;
    if (V > 0) WC_REQUIRE_PTR(fn, table);
    if ((rc = ids_pointer(fn, ids, id_type)) != WC_OK) return rc;
    WC_REQUIRE_PTR(fn, out);
    return from_cuda(wc::launch_embedding(table, dtype == WC_BF16, ld_table, ids, id_type == WC_I64,
                                          n, first, V, D, scale, out, ld_out,
                                          static_cast<cudaStream_t>(stream)),
                     fn);
}

WC_API int64_t wc_embedding_grad_workspace(int64_t n, int64_t V, int64_t D) {
    static const char *fn = "wc_embedding_grad_workspace";
    const int rc = embedding_sizes(fn, WC_I32, n, 0, V, D);
    if (rc != WC_OK) return rc;
    if (D == 0) return 0;
    wc::EmbeddingGrad a = {};
    a.n = n;
    a.V = V;
    a.D = D;
    return wc::embedding_grad_workspace(a);
}

WC_API int wc_embedding_grad(const void *dy, int dy_dtype, int64_t ld_dy, const void *ids,
                             int id_type, int64_t n, int64_t first, int64_t V, int64_t D,
                             float scale, int accumulate, void *dtable, int out_dtype,
                             int64_t ld_out, void *workspace, int64_t workspace_bytes,
                             void *stream) {
    static const char *fn = "wc_embedding_grad";
    int rc = embedding_sizes(fn, id_type, n, first, V, D);
    if (rc != WC_OK) return rc;
    if (!float_type(dy_dtype) || !float_type(out_dtype))
        return fail(WC_EINVAL, "%s: dy_dtype %d or out_dtype %d is neither WC_F32 nor WC_BF16", fn,
                    dy_dtype, out_dtype);
    if (ld_dy < D || ld_out < D)
        return fail(WC_EINVAL, "%s: ld_dy = %lld, ld_out = %lld are below D = %lld", fn,
                    (long long)ld_dy, (long long)ld_out, (long long)D);
    if (V == 0 || D == 0 || (n == 0 && accumulate)) return WC_OK;
    if (n > 0) {
        WC_REQUIRE_PTR(fn, dy);
        if ((rc = ids_pointer(fn, ids, id_type)) != WC_OK) return rc;
    }
    WC_REQUIRE_PTR(fn, dtable);
    WC_REQUIRE_PTR(fn, workspace);
    const int64_t need = wc_embedding_grad_workspace(n, V, D);
    if (workspace_bytes < need)
        return fail(WC_EINVAL, "%s: workspace of %lld bytes, %lld are needed", fn,
                    (long long)workspace_bytes, (long long)need);
    wc::EmbeddingGrad a;
    a.dy = dy;
    a.dy_bf16 = dy_dtype == WC_BF16;
    a.ld_dy = ld_dy;
    a.ids = ids;
    a.wide = id_type == WC_I64;
    a.n = n;
    a.first = first;
    a.V = V;
    a.D = D;
    a.scale = scale;
    a.accumulate = accumulate != 0;
    a.dtable = dtable;
    a.out_bf16 = out_dtype == WC_BF16;
    a.ld_out = ld_out;
    a.workspace = workspace;
    return from_cuda(wc::launch_embedding_grad(a, static_cast<cudaStream_t>(stream)), fn);
}

WC_API int wc_fp8_quant(const void *x, int dtype, int64_t rows, int64_t cols, int64_t ld,
                        int square, uint8_t *q, int64_t ld_q, float *s, int64_t ld_s, uint8_t *qt,
                        int64_t ld_qt, float *st, int64_t ld_st, void *stream) {
    static const char *fn = "wc_fp8_quant";
    if (!float_type(dtype)) return fail(WC_EINVAL, "%s: dtype %d is neither WC_F32 nor WC_BF16", fn, dtype);
    if (rows < 0 || cols < 0)
        return fail(WC_EINVAL, "%s: rows = %lld, cols = %lld must not be negative", fn, (long long)rows, (long long)cols);
    if (rows > 65535 * 128 || cols > 65535 * 128)
        return fail(WC_ERANGE, "%s: rows or cols exceeds 8388480", fn);
    if (ld < cols) return fail(WC_EINVAL, "%s: ld = %lld is below cols = %lld", fn, (long long)ld, (long long)cols);
    if ((q == nullptr) != (s == nullptr) || (qt == nullptr) != (st == nullptr))
        return fail(WC_EINVAL, "%s: codes and scales must both be given or both be NULL", fn);
    if (q != nullptr && (ld_q % 16 || ld_q < cols))
        return fail(WC_EINVAL, "%s: ld_q = %lld must be a multiple of 16 and at least cols", fn, (long long)ld_q);
    if (qt != nullptr && (ld_qt % 16 || ld_qt < rows))
        return fail(WC_EINVAL, "%s: ld_qt = %lld must be a multiple of 16 and at least rows", fn, (long long)ld_qt);
    if (q != nullptr && ld_s < (square ? blocks128(rows) : rows))
        return fail(WC_EINVAL, "%s: ld_s = %lld does not hold a block's scales", fn, (long long)ld_s);
    if (qt != nullptr && ld_st < (square ? blocks128(cols) : cols))
        return fail(WC_EINVAL, "%s: ld_st = %lld does not hold a block's scales", fn, (long long)ld_st);
    if (rows == 0 || cols == 0) return WC_OK;
    if (q == nullptr && qt == nullptr) return fail(WC_EINVAL, "%s: q and qt are both NULL", fn);
    WC_REQUIRE_PTR(fn, x);
    if (q != nullptr && (!aligned16(q) || !aligned16(s)))
        return fail(WC_EALIGN, "%s: q or s is not 16-byte aligned", fn);
    if (qt != nullptr && (!aligned16(qt) || !aligned16(st)))
        return fail(WC_EALIGN, "%s: qt or st is not 16-byte aligned", fn);
    wc::Fp8Quant a;
    a.x = x;
    a.x_bf16 = dtype == WC_BF16;
    a.rows = rows;
    a.cols = cols;
    a.ld = ld;
    a.square = square != 0;
    a.q = q;
    a.ld_q = ld_q;
    a.s = s;
    a.ld_s = ld_s;
    a.qt = qt;
    a.ld_qt = ld_qt;
    a.st = st;
    a.ld_st = ld_st;
    return from_cuda(wc::launch_fp8_quant(a, static_cast<cudaStream_t>(stream)), fn);
}

WC_API int wc_fp8_matmul(const uint8_t *a, int64_t lda, const float *sa, int64_t ldsa,
                         int a_rows_per_scale, const uint8_t *b, int64_t ldb, const float *sb,
                         int64_t ldsb, int b_rows_per_scale, int64_t M, int64_t N, int64_t K,
                         void *out, int out_dtype, int64_t ld_out, int accumulate, void *stream) {
    static const char *fn = "wc_fp8_matmul";
    if (M < 0 || N < 0 || K < 0)
        return fail(WC_EINVAL, "%s: M = %lld, N = %lld, K = %lld must not be negative", fn, (long long)M,
                    (long long)N, (long long)K);
    const int64_t limit = int64_t(1) << 31;
    // (2^31 - 256: the tiles' coordinates are 32-bit and go up to the next 256)
    if (M > limit - 256 || N > limit - 256 || K > limit - 256)
        return fail(WC_ERANGE, "%s: M, N or K exceeds 2^31 - 256", fn);
    if (N > 0 && M >= (int64_t(1) << 44) / N) return fail(WC_ERANGE, "%s: M * N reaches 2^44", fn);
    if (!float_type(out_dtype))
        return fail(WC_EINVAL, "%s: out_dtype %d is neither WC_F32 nor WC_BF16", fn, out_dtype);
    if ((a_rows_per_scale != 1 && a_rows_per_scale != 128) || (b_rows_per_scale != 1 && b_rows_per_scale != 128))
        return fail(WC_EINVAL, "%s: rows per scale (%d and %d) must be 1 or 128", fn, a_rows_per_scale,
                    b_rows_per_scale);
    if (lda % 16 || ldb % 16 || lda < K || ldb < K)
        return fail(WC_EINVAL, "%s: lda = %lld, ldb = %lld must be multiples of 16 and at least K", fn,
                    (long long)lda, (long long)ldb);
    if (ldsa < (a_rows_per_scale == 128 ? blocks128(M) : M) || ldsb < (b_rows_per_scale == 128 ? blocks128(N) : N))
        return fail(WC_EINVAL, "%s: ldsa = %lld or ldsb = %lld does not hold a block's scales", fn,
                    (long long)ldsa, (long long)ldsb);
    if (ld_out < N) return fail(WC_EINVAL, "%s: ld_out = %lld is below N = %lld", fn, (long long)ld_out, (long long)N);
    if (M == 0 || N == 0) return WC_OK;
    if (K > 0) {
        WC_REQUIRE_PTR(fn, a);
        WC_REQUIRE_PTR(fn, sa);
        WC_REQUIRE_PTR(fn, b);
        WC_REQUIRE_PTR(fn, sb);
    }
    WC_REQUIRE_PTR(fn, out);
    wc::Fp8Matmul m;
    m.a = {a, lda, sa, ldsa, a_rows_per_scale};
    m.b = {b, ldb, sb, ldsb, b_rows_per_scale};
    m.M = M;
    m.N = N;
    m.K = K;
    m.out = out;
    m.out_bf16 = out_dtype == WC_BF16;
    m.ld_out = ld_out;
    m.accumulate = accumulate != 0;
    return from_cuda(wc::launch_fp8_matmul(m, static_cast<cudaStream_t>(stream)), fn);
}

WC_API int wc_wait_timeouts(int reset) {
    static const char *fn = "wc_wait_timeouts";
    unsigned int n = 0;
    const cudaError_t e = wc::fp8_wait_timeouts(&n, reset != 0);
    if (e != cudaSuccess) return from_cuda(e, fn);
    return n > 0x7FFFFFFFu ? 0x7FFFFFFF : int(n);
}

WC_API int wc_checked_violations(int flags) {
    static const char *fn = "wc_checked_violations";
    if (flags & ~(WC_CHECK_RESET | WC_CHECK_PROBE))
        return fail(WC_EINVAL, "%s: unknown flags 0x%x", fn, unsigned(flags));
#if defined(WC_CHECKED) && WC_CHECKED
    struct Reader {
        const char *file;
        cudaError_t (*read)(wc::CheckRecord *, bool, bool);
    };
    static const Reader readers[] = {
        {"qgz_quant.cu", wc::check_record_qgz_quant}, {"qgz_reduce.cu", wc::check_record_qgz_reduce},
        {"qgz_hop1.cu", wc::check_record_qgz_hop1},   {"qgz_fused.cu", wc::check_record_qgz_fused},
        {"qwz.cu", wc::check_record_qwz},
    };
    uint64_t total = 0;
    const char *first_file = nullptr;
    unsigned int first_line = 0;
    for (const Reader &r : readers) {
        wc::CheckRecord rec = {0u, 0u};
        const cudaError_t e = r.read(&rec, (flags & WC_CHECK_RESET) != 0,
                                     (flags & WC_CHECK_PROBE) != 0);
        if (e != cudaSuccess) return from_cuda(e, fn);
        if (rec.count != 0 && first_file == nullptr) {
            first_file = r.file;
            first_line = rec.first_line;
        }
        total += rec.count;
    }
    if (total == 0) return 0;
    fail(WC_OK, "%s: %llu accesses skipped, one of them in %s line %u", fn,
         (unsigned long long)total, first_file, first_line);
    return total > 0x7FFFFFFFull ? 0x7FFFFFFF : int(total);
#else
    return fail(WC_EINVAL, "%s: this library was built without checks (WC_CHECKED=1)", fn);
#endif
}

}  // extern "C"
