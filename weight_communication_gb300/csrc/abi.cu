// abi.cu -- the extern "C" entry points declared in include/wc.h: argument
// validation on the host, then one kernel launch per call (the gradient norm,
// clipping, the gradients of embedding and norm: two or three, back to back; the
// cross entropy: two or three per piece of its work).
#include <math.h>
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include <algorithm>
#include <initializer_list>
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

// Rows of values may start on any value.
int values_pointer(const char *fn, const char *name, const void *p, int dtype) {
    const uintptr_t size = dtype == WC_BF16 ? 2 : 4;
    if (p == nullptr) return fail(WC_EINVAL, "%s: %s is NULL", fn, name);
    if (reinterpret_cast<uintptr_t>(p) % size)
        return fail(WC_EALIGN, "%s: %s is not aligned to its %d-byte values", fn, name, int(size));
    return WC_OK;
}

// Rows at most 2^38 values apart (what a TMA descriptor takes), and offsets of 2^60
// values at most.
int row_pitch(const char *fn, const char *name, int64_t ld, int64_t rows, int64_t cols) {
    if (ld < cols)
        return fail(WC_EINVAL, "%s: ld_%s = %lld is below %lld columns", fn, name, (long long)ld, (long long)cols);
    if (ld >= (int64_t(1) << 38) || (rows > 0 && ld >= (int64_t(1) << 60) / rows))
        return fail(WC_ERANGE, "%s: ld_%s = %lld is too large", fn, name, (long long)ld);
    return WC_OK;
}

// Memory that a call reads or writes: rows of `width` bytes, `pitch` bytes apart.
struct Region {
    const char *name;
    const void *p;  // NULL: none
    int64_t rows, width, pitch;
};
Region matrix(const char *name, const void *p, int64_t rows, int64_t cols, int64_t ld, int64_t size) {
    return {name, p, rows, cols * size, ld * size};
}
Region bytes(const char *name, const void *p, int64_t n) { return {name, p, 1, n, n}; }

int64_t floor_div(int64_t a, int64_t b) { return a / b - (a % b < 0 ? 1 : 0); }  // b > 0

// A byte of both?  (Matrices that lie between one another's rows have none.)
bool overlap(Region a, Region b) {
    if (a.p == nullptr || b.p == nullptr || a.rows == 0 || b.rows == 0 || a.width == 0 || b.width == 0) return false;
    const int64_t at_a = int64_t(reinterpret_cast<uintptr_t>(a.p)), at_b = int64_t(reinterpret_cast<uintptr_t>(b.p));
    const int64_t end_a = at_a + (a.rows - 1) * a.pitch + a.width, end_b = at_b + (b.rows - 1) * b.pitch + b.width;
    if (end_a <= at_b || end_b <= at_a) return false;
    if (a.rows == 1) a.pitch = b.pitch;
    if (b.rows == 1) b.pitch = a.pitch;
    if (a.pitch == b.pitch) {
        // rows i and i + k, whose starts are apart + k pitch bytes from one another
        const int64_t apart = at_b - at_a, first = floor_div(-b.width - apart, a.pitch) + 1;
        const int64_t k = first > 1 - a.rows ? first : 1 - a.rows;
        return k < b.rows && apart + k * a.pitch < a.width;
    }
    if (a.rows > b.rows) return overlap(b, a);
    for (int64_t i = 0; i < a.rows; ++i) {
        const int64_t start = at_a + i * a.pitch, first = floor_div(start - b.width - at_b, b.pitch) + 1;
        const int64_t j = first > 0 ? first : 0;
        if (j < b.rows && at_b + j * b.pitch < start + a.width) return true;
    }
    return false;
}

// What is written overlaps neither what is read nor what else is written.
int written_apart(const char *fn, std::initializer_list<Region> written, std::initializer_list<Region> read) {
    for (const Region *w = written.begin(); w < written.end(); ++w) {
        for (const Region *other = w + 1; other < written.end(); ++other)
            if (overlap(*w, *other)) return fail(WC_EINVAL, "%s: %s overlaps %s", fn, w->name, other->name);
        for (const Region &r : read)
            if (overlap(*w, r)) return fail(WC_EINVAL, "%s: %s overlaps %s", fn, w->name, r.name);
    }
    return WC_OK;
}

// What is read, unless it is the very rows that are written, which a call may allow.
Region unless_same(const Region &read, const Region &written) {
    Region r = read;
    if (r.p == written.p && r.width == written.width && (r.pitch == written.pitch || r.rows == 1)) r.p = nullptr;
    return r;
}

int block_sizes(const char *fn, int64_t rows, int64_t cols) {
    if (rows < 0 || cols < 0)
        return fail(WC_EINVAL, "%s: rows = %lld, cols = %lld must not be negative", fn, (long long)rows, (long long)cols);
    if (rows > 65535 * 128 || cols > 65535 * 128)
        return fail(WC_ERANGE, "%s: rows or cols exceeds 8388480", fn);
    if (cols > 0 && rows >= (int64_t(1) << 40) / cols) return fail(WC_ERANGE, "%s: rows * cols reaches 2^40", fn);
    return WC_OK;
}

int activation_kind(const char *fn, int dtype, int kind) {
    if (!float_type(dtype)) return fail(WC_EINVAL, "%s: dtype %d is neither WC_F32 nor WC_BF16", fn, dtype);
    if (kind != WC_RELU && kind != WC_SILU && kind != WC_GELU)
        return fail(WC_EINVAL, "%s: kind %d is none of WC_RELU, WC_SILU, WC_GELU", fn, kind);
    return WC_OK;
}

// `k` as the kernels take it; NULL is an empty one.
int kept_matrix(const char *fn, const char *name, const wc_kept *k, int64_t rows, int64_t cols, wc::Kept8 *to) {
    if (k == nullptr) return WC_OK;
    if (k->codes == nullptr || k->scales == nullptr)
        return fail(WC_EINVAL, "%s: %s has no codes or no scales", fn, name);
    if (!aligned16(k->codes) || !aligned16(k->scales))
        return fail(WC_EALIGN, "%s: codes or scales of %s are not 16-byte aligned", fn, name);
    if (k->ld_codes % 16 || k->ld_codes < cols)
        return fail(WC_EINVAL, "%s: ld_codes = %lld of %s must be a multiple of 16 and at least cols", fn,
                    (long long)k->ld_codes, name);
    if (k->ld_codes >= (int64_t(1) << 38) || k->ld_scales >= (int64_t(1) << 38))
        return fail(WC_ERANGE, "%s: ld_codes or ld_scales of %s reaches 2^38", fn, name);
    if (k->ld_scales < rows)
        return fail(WC_EINVAL, "%s: ld_scales = %lld of %s does not hold a block's scales", fn,
                    (long long)k->ld_scales, name);
    *to = {k->codes, k->ld_codes, k->scales, k->ld_scales};
    return WC_OK;
}

Region codes_of(const char *name, const wc::Kept8 &k, int64_t rows, int64_t cols) {
    return {name, k.q, rows, (cols + 15) / 16 * 16, k.ld_q};
}
Region scales_of(const char *name, const wc::Kept8 &k, int64_t rows, int64_t cols) {
    return matrix(name, k.s, blocks128(cols), rows, k.ld_s, 4);
}

int norm_sizes(const char *fn, int64_t rows, int64_t cols, int dtype, int weight_dtype) {
    if (!float_type(dtype) || !float_type(weight_dtype))
        return fail(WC_EINVAL, "%s: dtype %d or weight_dtype %d is neither WC_F32 nor WC_BF16", fn, dtype, weight_dtype);
    if (rows < 0 || cols < 1)
        return fail(WC_EINVAL, "%s: rows = %lld must not be negative, cols = %lld must be at least 1", fn,
                    (long long)rows, (long long)cols);
    if (rows > 65535 * 128) return fail(WC_ERANGE, "%s: rows exceeds 8388480", fn);
    if (cols > wc::kNormCols) return fail(WC_ERANGE, "%s: cols exceeds %lld", fn, (long long)wc::kNormCols);
    return WC_OK;
}

int cross_entropy_sizes(const char *fn, const uint16_t *x, int64_t ld_x, const uint16_t *w, int64_t ld_w,
                        int64_t T, int64_t V, int64_t D, wc::CrossEntropy *c) {
    if (T < 0 || V < 1 || D < 1)
        return fail(WC_EINVAL, "%s: T = %lld must not be negative, V = %lld and D = %lld must be at least 1", fn,
                    (long long)T, (long long)V, (long long)D);
    // (the kernels step past the last token or row in 32 bits)
    const int64_t limit = (int64_t(1) << 31) - 4096;
    if (T > limit || V > limit) return fail(WC_ERANGE, "%s: T or V exceeds 2^31 - 4096", fn);
    if (D > (int64_t(1) << 22)) return fail(WC_ERANGE, "%s: D exceeds 2^22", fn);
    if (T >= (int64_t(1) << 44) / V) return fail(WC_ERANGE, "%s: T * V reaches 2^44", fn);
    if (T >= (int64_t(1) << 40) / D || V >= (int64_t(1) << 40) / D)
        return fail(WC_ERANGE, "%s: T * D or V * D reaches 2^40", fn);
    int rc = row_pitch(fn, "x", ld_x, T, D);
    if (rc == WC_OK) rc = row_pitch(fn, "w", ld_w, V, D);
    if (rc != WC_OK) return rc;
    c->x = x;
    c->w = w;
    c->ld_x = ld_x;
    c->ld_w = ld_w;
    c->T = T;
    c->V = V;
    c->D = D;
    return WC_OK;
}

int cross_entropy_inputs(const char *fn, wc::CrossEntropy *c, const void *targets, int id_type) {
    if (id_type != WC_I32 && id_type != WC_I64)
        return fail(WC_EINVAL, "%s: id_type %d is neither WC_I32 nor WC_I64", fn, id_type);
    if (c->T == 0) return WC_OK;
    int rc = values_pointer(fn, "x", c->x, WC_BF16);
    if (rc == WC_OK) rc = values_pointer(fn, "w", c->w, WC_BF16);
    if (rc != WC_OK) return rc;
    const uintptr_t size = id_type == WC_I64 ? 8 : 4;
    if (targets == nullptr) return fail(WC_EINVAL, "%s: targets is NULL", fn);
    if (reinterpret_cast<uintptr_t>(targets) % size)
        return fail(WC_EALIGN, "%s: targets is not aligned to its %d-byte values", fn, int(size));
    c->targets = targets;
    c->wide = id_type == WC_I64;
    return WC_OK;
}

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

WC_API int wc_fp8_dequant(const uint8_t *q, int64_t ld_q, const float *s, int64_t ld_s,
                          int rows_per_scale, int64_t rows, int64_t cols, void *out, int out_dtype,
                          int64_t ld_out, void *stream) {
    static const char *fn = "wc_fp8_dequant";
    int rc = block_sizes(fn, rows, cols);
    if (rc != WC_OK) return rc;
    if (!float_type(out_dtype))
        return fail(WC_EINVAL, "%s: out_dtype %d is neither WC_F32 nor WC_BF16", fn, out_dtype);
    if (rows_per_scale != 1 && rows_per_scale != 128)
        return fail(WC_EINVAL, "%s: rows per scale (%d) must be 1 or 128", fn, rows_per_scale);
    if (ld_q % 16 || ld_q < cols)
        return fail(WC_EINVAL, "%s: ld_q = %lld must be a multiple of 16 and at least cols", fn, (long long)ld_q);
    if (ld_s < (rows_per_scale == 128 ? blocks128(rows) : rows))
        return fail(WC_EINVAL, "%s: ld_s = %lld does not hold a block's scales", fn, (long long)ld_s);
    if ((rc = row_pitch(fn, "out", ld_out, rows, cols)) != WC_OK) return rc;
    if (ld_q >= (int64_t(1) << 38) || ld_s >= (int64_t(1) << 38))
        return fail(WC_ERANGE, "%s: ld_q or ld_s reaches 2^38", fn);
    if (rows == 0 || cols == 0) return WC_OK;
    WC_REQUIRE_PTR(fn, q);
    WC_REQUIRE_PTR(fn, s);
    if ((rc = values_pointer(fn, "out", out, out_dtype)) != WC_OK) return rc;
    const bool per_row = rows_per_scale == 1;
    rc = written_apart(fn, {matrix("out", out, rows, cols, ld_out, out_dtype == WC_BF16 ? 2 : 4)},
                       {{"q", q, rows, cols, ld_q}, matrix("s", s, blocks128(cols), per_row ? rows : blocks128(rows), ld_s, 4)});
    if (rc != WC_OK) return rc;
    const wc::Fp8Dequant a = {q, ld_q, s, ld_s, rows_per_scale, rows, cols, out, out_dtype == WC_BF16, ld_out};
    return from_cuda(wc::launch_fp8_dequant(a, static_cast<cudaStream_t>(stream)), fn);
}

WC_API int wc_activation(const void *gate, int64_t ld_gate, const void *up, int64_t ld_up, int dtype,
                         int kind, int64_t rows, int64_t cols, void *h, int64_t ld_h,
                         const wc_kept *kept_gate, const wc_kept *kept_up, void *stream) {
    static const char *fn = "wc_activation";
    int rc = block_sizes(fn, rows, cols);
    if (rc == WC_OK) rc = activation_kind(fn, dtype, kind);
    if (rc == WC_OK) rc = row_pitch(fn, "gate", ld_gate, rows, cols);
    if (rc == WC_OK && up) rc = row_pitch(fn, "up", ld_up, rows, cols);
    if (rc == WC_OK) rc = row_pitch(fn, "h", ld_h, rows, cols);
    if (rc != WC_OK) return rc;
    if (rows == 0 || cols == 0) return WC_OK;
    if ((kept_up != nullptr) != (up != nullptr && kept_gate != nullptr))
        return fail(WC_EINVAL, "%s: kept_up must be given if and only if up and kept_gate are", fn);
    if ((rc = values_pointer(fn, "gate", gate, dtype)) != WC_OK) return rc;
    if (up && (rc = values_pointer(fn, "up", up, dtype)) != WC_OK) return rc;
    if ((rc = values_pointer(fn, "h", h, dtype)) != WC_OK) return rc;
    wc::Activation a = {};
    if ((rc = kept_matrix(fn, "kept_gate", kept_gate, rows, cols, &a.kept_gate)) != WC_OK) return rc;
    if ((rc = kept_matrix(fn, "kept_up", kept_up, rows, cols, &a.kept_up)) != WC_OK) return rc;
    const int64_t size = dtype == WC_BF16 ? 2 : 4;
    const Region in_gate = matrix("gate", gate, rows, cols, ld_gate, size), in_up = matrix("up", up, rows, cols, ld_up, size);
    const Region out = matrix("h", h, rows, cols, ld_h, size);
    const Region qg = codes_of("codes of kept_gate", a.kept_gate, rows, cols), qu = codes_of("codes of kept_up", a.kept_up, rows, cols);
    const Region sg = scales_of("scales of kept_gate", a.kept_gate, rows, cols), su = scales_of("scales of kept_up", a.kept_up, rows, cols);
    if ((rc = written_apart(fn, {out}, {unless_same(in_gate, out), unless_same(in_up, out)})) != WC_OK) return rc;
    if (kept_gate && (rc = written_apart(fn, {qg, sg, qu, su}, {in_gate, in_up, out})) != WC_OK) return rc;
    a.gate = gate;
    a.up = up;
    a.ld_gate = ld_gate;
    a.ld_up = ld_up;
    a.bf16 = dtype == WC_BF16;
    a.kind = kind;
    a.rows = rows;
    a.cols = cols;
    a.h = h;
    a.ld_h = ld_h;
    return from_cuda(wc::launch_activation(a, static_cast<cudaStream_t>(stream)), fn);
}

WC_API int wc_activation_grad(const void *dh, int64_t ld_dh, int dtype, int kind, int64_t rows,
                              int64_t cols, const wc_kept *kept_gate, const wc_kept *kept_up,
                              void *dgate, int64_t ld_dgate, void *dup, int64_t ld_dup, void *stream) {
    static const char *fn = "wc_activation_grad";
    int rc = block_sizes(fn, rows, cols);
    if (rc == WC_OK) rc = activation_kind(fn, dtype, kind);
    if (rc == WC_OK) rc = row_pitch(fn, "dh", ld_dh, rows, cols);
    if (rc == WC_OK) rc = row_pitch(fn, "dgate", ld_dgate, rows, cols);
    if (rc == WC_OK && dup) rc = row_pitch(fn, "dup", ld_dup, rows, cols);
    if (rc != WC_OK) return rc;
    if (rows == 0 || cols == 0) return WC_OK;
    if (kept_gate == nullptr) return fail(WC_EINVAL, "%s: kept_gate is NULL", fn);
    if ((kept_up != nullptr) != (dup != nullptr))
        return fail(WC_EINVAL, "%s: kept_up must be given if and only if dup is", fn);
    if ((rc = values_pointer(fn, "dh", dh, dtype)) != WC_OK) return rc;
    if ((rc = values_pointer(fn, "dgate", dgate, dtype)) != WC_OK) return rc;
    if (dup && (rc = values_pointer(fn, "dup", dup, dtype)) != WC_OK) return rc;
    wc::ActivationGrad a = {};
    if ((rc = kept_matrix(fn, "kept_gate", kept_gate, rows, cols, &a.kept_gate)) != WC_OK) return rc;
    if ((rc = kept_matrix(fn, "kept_up", kept_up, rows, cols, &a.kept_up)) != WC_OK) return rc;
    const int64_t size = dtype == WC_BF16 ? 2 : 4;
    const Region in = matrix("dh", dh, rows, cols, ld_dh, size);
    const Region og = matrix("dgate", dgate, rows, cols, ld_dgate, size), ou = matrix("dup", dup, rows, cols, ld_dup, size);
    rc = written_apart(fn, {og, ou}, {codes_of("codes of kept_gate", a.kept_gate, rows, cols),
                                      scales_of("scales of kept_gate", a.kept_gate, rows, cols),
                                      codes_of("codes of kept_up", a.kept_up, rows, cols),
                                      scales_of("scales of kept_up", a.kept_up, rows, cols)});
    for (const Region &out : {og, ou})
        if (rc == WC_OK) rc = written_apart(fn, {out}, {unless_same(in, out)});
    if (rc != WC_OK) return rc;
    a.dh = dh;
    a.ld_dh = ld_dh;
    a.bf16 = dtype == WC_BF16;
    a.kind = kind;
    a.rows = rows;
    a.cols = cols;
    a.dgate = dgate;
    a.dup = dup;
    a.ld_dgate = ld_dgate;
    a.ld_dup = ld_dup;
    return from_cuda(wc::launch_activation_grad(a, static_cast<cudaStream_t>(stream)), fn);
}

WC_API int wc_rms_norm(const void *x, int64_t ld_x, const void *add, int64_t ld_add, int dtype,
                       int64_t rows, int64_t cols, const void *weight, int weight_dtype, double eps,
                       void *y, int64_t ld_y, void *total, int64_t ld_total, float *rstd,
                       const wc_kept *kept, void *stream) {
    static const char *fn = "wc_rms_norm";
    int rc = norm_sizes(fn, rows, cols, dtype, weight_dtype);
    if (rc == WC_OK) rc = row_pitch(fn, "x", ld_x, rows, cols);
    if (rc == WC_OK && add) rc = row_pitch(fn, "add", ld_add, rows, cols);
    if (rc == WC_OK) rc = row_pitch(fn, "y", ld_y, rows, cols);
    if (rc == WC_OK && add) rc = row_pitch(fn, "total", ld_total, rows, cols);
    if (rc != WC_OK) return rc;
    if (!(eps >= 0.0 && eps < HUGE_VAL)) return fail(WC_EINVAL, "%s: eps = %g must be finite and at least 0", fn, eps);
    if (rows == 0) return WC_OK;
    if ((rstd != nullptr) != (kept != nullptr))
        return fail(WC_EINVAL, "%s: rstd and kept must both be given or both be NULL", fn);
    if ((total != nullptr) != (add != nullptr))
        return fail(WC_EINVAL, "%s: total must be given if and only if add is", fn);
    if ((rc = values_pointer(fn, "x", x, dtype)) != WC_OK) return rc;
    if (add && (rc = values_pointer(fn, "add", add, dtype)) != WC_OK) return rc;
    if ((rc = values_pointer(fn, "weight", weight, weight_dtype)) != WC_OK) return rc;
    if ((rc = values_pointer(fn, "y", y, dtype)) != WC_OK) return rc;
    if (total && (rc = values_pointer(fn, "total", total, dtype)) != WC_OK) return rc;
    if (rstd && (rc = values_pointer(fn, "rstd", rstd, WC_F32)) != WC_OK) return rc;
    wc::RmsNorm a = {};
    if ((rc = kept_matrix(fn, "kept", kept, rows, cols, &a.kept)) != WC_OK) return rc;
    const int64_t size = dtype == WC_BF16 ? 2 : 4;
    const Region in = matrix("x", x, rows, cols, ld_x, size), in_add = matrix("add", add, rows, cols, ld_add, size);
    const Region out = matrix("y", y, rows, cols, ld_y, size), sum = matrix("total", total, rows, cols, ld_total, size);
    const Region w = bytes("weight", weight, cols * (weight_dtype == WC_BF16 ? 2 : 4));
    rc = written_apart(fn, {out, sum, bytes("rstd", rstd, 4 * rows), codes_of("codes of kept", a.kept, rows, cols),
                            scales_of("scales of kept", a.kept, rows, cols)}, {w});
    for (const Region &o : {out, sum})
        if (rc == WC_OK) rc = written_apart(fn, {o}, {unless_same(in, o), unless_same(in_add, o)});
    if (rc == WC_OK && kept)
        rc = written_apart(fn, {bytes("rstd", rstd, 4 * rows), codes_of("codes of kept", a.kept, rows, cols),
                                scales_of("scales of kept", a.kept, rows, cols)}, {in, in_add});
    if (rc != WC_OK) return rc;
    a.x = x;
    a.add = add;
    a.ld_x = ld_x;
    a.ld_add = ld_add;
    a.bf16 = dtype == WC_BF16;
    a.rows = rows;
    a.cols = cols;
    a.weight = weight;
    a.weight_bf16 = weight_dtype == WC_BF16;
    a.eps = float(eps);
    a.y = y;
    a.total = total;
    a.ld_y = ld_y;
    a.ld_total = ld_total;
    a.rstd = rstd;
    return from_cuda(wc::launch_rms_norm(a, static_cast<cudaStream_t>(stream)), fn);
}

WC_API int64_t wc_rms_norm_grad_workspace(int64_t rows, int64_t cols) {
    static const char *fn = "wc_rms_norm_grad_workspace";
    const int rc = norm_sizes(fn, rows, cols, WC_F32, WC_F32);
    if (rc != WC_OK) return rc;
    return rows > 0 ? 4 * wc::rms_norm_grad_partials(rows, cols) : 0;
}

WC_API int wc_rms_norm_grad(const void *dy, int64_t ld_dy, const void *add, int64_t ld_add, int dtype,
                            int64_t rows, int64_t cols, const void *weight, int weight_dtype,
                            const float *rstd, const wc_kept *kept, void *dx, int64_t ld_dx,
                            void *dweight, int dweight_dtype, int accumulate, void *workspace,
                            int64_t workspace_bytes, void *stream) {
    static const char *fn = "wc_rms_norm_grad";
    int rc = norm_sizes(fn, rows, cols, dtype, weight_dtype);
    if (rc != WC_OK) return rc;
    if (!float_type(dweight_dtype))
        return fail(WC_EINVAL, "%s: dweight_dtype %d is neither WC_F32 nor WC_BF16", fn, dweight_dtype);
    if ((rc = row_pitch(fn, "dy", ld_dy, rows, cols)) != WC_OK) return rc;
    if (add && (rc = row_pitch(fn, "add", ld_add, rows, cols)) != WC_OK) return rc;
    if ((rc = row_pitch(fn, "dx", ld_dx, rows, cols)) != WC_OK) return rc;
    if ((rc = values_pointer(fn, "dweight", dweight, dweight_dtype)) != WC_OK) return rc;
    wc::RmsNormGrad a = {};
    if (rows > 0) {
        if (kept == nullptr) return fail(WC_EINVAL, "%s: kept is NULL", fn);
        if ((rc = values_pointer(fn, "dy", dy, dtype)) != WC_OK) return rc;
        if (add && (rc = values_pointer(fn, "add", add, dtype)) != WC_OK) return rc;
        if ((rc = values_pointer(fn, "weight", weight, weight_dtype)) != WC_OK) return rc;
        if ((rc = values_pointer(fn, "rstd", rstd, WC_F32)) != WC_OK) return rc;
        if ((rc = values_pointer(fn, "dx", dx, dtype)) != WC_OK) return rc;
        if ((rc = kept_matrix(fn, "kept", kept, rows, cols, &a.kept)) != WC_OK) return rc;
        WC_REQUIRE_PTR(fn, workspace);
        const int64_t need = wc_rms_norm_grad_workspace(rows, cols);
        if (workspace_bytes < need)
            return fail(WC_EINVAL, "%s: workspace of %lld bytes, %lld are needed", fn, (long long)workspace_bytes,
                        (long long)need);
        // (dweight may be weight: it is written when all rows are done)
        const int64_t size = dtype == WC_BF16 ? 2 : 4;
        const Region in = matrix("dy", dy, rows, cols, ld_dy, size), in_add = matrix("add", add, rows, cols, ld_add, size);
        const Region out = matrix("dx", dx, rows, cols, ld_dx, size);
        const Region w = bytes("weight", weight, cols * (weight_dtype == WC_BF16 ? 2 : 4));
        const Region sums = bytes("dweight", dweight, cols * (dweight_dtype == WC_BF16 ? 2 : 4)), ws = bytes("workspace", workspace, need);
        const Region r = bytes("rstd", rstd, 4 * rows), q = codes_of("codes of kept", a.kept, rows, cols),
                     s = scales_of("scales of kept", a.kept, rows, cols);
        rc = written_apart(fn, {out, sums, ws}, {r, q, s});
        if (rc == WC_OK) rc = written_apart(fn, {out}, {w, unless_same(in, out), unless_same(in_add, out)});
        if (rc == WC_OK) rc = written_apart(fn, {sums}, {unless_same(w, sums), in, in_add});
        if (rc == WC_OK) rc = written_apart(fn, {ws}, {w, in, in_add});
        if (rc != WC_OK) return rc;
    } else if (accumulate) {
        return WC_OK;
    }
    a.dy = dy;
    a.add = add;
    a.ld_dy = ld_dy;
    a.ld_add = ld_add;
    a.bf16 = dtype == WC_BF16;
    a.rows = rows;
    a.cols = cols;
    a.weight = weight;
    a.weight_bf16 = weight_dtype == WC_BF16;
    a.rstd = rstd;
    a.dx = dx;
    a.ld_dx = ld_dx;
    a.dweight = dweight;
    a.dweight_bf16 = dweight_dtype == WC_BF16;
    a.accumulate = accumulate != 0;
    a.partials = static_cast<float *>(workspace);
    return from_cuda(wc::launch_rms_norm_grad(a, static_cast<cudaStream_t>(stream)), fn);
}

WC_API int64_t wc_cross_entropy_workspace(const uint16_t *x, int64_t ld_x, const uint16_t *w,
                                          int64_t ld_w, int64_t T, int64_t V, int64_t D) {
    wc::CrossEntropy c = {};
    const int rc = cross_entropy_sizes("wc_cross_entropy_workspace", x, ld_x, w, ld_w, T, V, D, &c);
    if (rc != WC_OK) return rc;
    return T > 0 ? wc::cross_entropy_workspace(c) : 0;
}

WC_API int wc_cross_entropy(const uint16_t *x, int64_t ld_x, const uint16_t *w, int64_t ld_w,
                            const void *targets, int id_type, int64_t T, int64_t V, int64_t D,
                            float *losses, float *lse, void *workspace, int64_t workspace_bytes,
                            void *stream) {
    static const char *fn = "wc_cross_entropy";
    wc::CrossEntropy c = {};
    int rc = cross_entropy_sizes(fn, x, ld_x, w, ld_w, T, V, D, &c);
    if (rc != WC_OK) return rc;
    if ((rc = cross_entropy_inputs(fn, &c, targets, id_type)) != WC_OK) return rc;
    if (T == 0) return WC_OK;
    if (losses == nullptr && lse == nullptr) return fail(WC_EINVAL, "%s: losses and lse are both NULL", fn);
    if (losses && (rc = values_pointer(fn, "losses", losses, WC_F32)) != WC_OK) return rc;
    if (lse && (rc = values_pointer(fn, "lse", lse, WC_F32)) != WC_OK) return rc;
    WC_REQUIRE_PTR(fn, workspace);
    const int64_t need = wc::cross_entropy_workspace(c);
    if (workspace_bytes < need)
        return fail(WC_EINVAL, "%s: workspace of %lld bytes, %lld are needed", fn, (long long)workspace_bytes,
                    (long long)need);
    rc = written_apart(fn, {bytes("losses", losses, 4 * T), bytes("lse", lse, 4 * T), bytes("workspace", workspace, need)},
                       {matrix("x", x, T, D, ld_x, 2), matrix("w", w, V, D, ld_w, 2),
                        bytes("targets", targets, T * (id_type == WC_I64 ? 8 : 4))});
    if (rc != WC_OK) return rc;
    c.workspace = workspace;
    c.losses = losses;
    c.lse = lse;
    return from_cuda(wc::launch_cross_entropy(c, static_cast<cudaStream_t>(stream)), fn);
}

WC_API int64_t wc_cross_entropy_grad_workspace(const uint16_t *x, int64_t ld_x, const uint16_t *w,
                                               int64_t ld_w, int64_t T, int64_t V, int64_t D) {
    wc::CrossEntropyGrad c = {};
    const int rc = cross_entropy_sizes("wc_cross_entropy_grad_workspace", x, ld_x, w, ld_w, T, V, D, &c);
    if (rc != WC_OK) return rc;
    return T > 0 ? wc::cross_entropy_grad_workspace(c) : 0;
}

WC_API int wc_cross_entropy_grad(const uint16_t *x, int64_t ld_x, const uint16_t *w, int64_t ld_w,
                                 const void *targets, int id_type, int64_t T, int64_t V, int64_t D,
                                 const float *lse, const float *dlosses, double dloss, void *dx,
                                 int dx_dtype, int64_t ld_dx, void *dw, int dw_dtype, int64_t ld_dw,
                                 int accumulate, void *workspace, int64_t workspace_bytes,
                                 void *stream) {
    static const char *fn = "wc_cross_entropy_grad";
    wc::CrossEntropyGrad c = {};
    int rc = cross_entropy_sizes(fn, x, ld_x, w, ld_w, T, V, D, &c);
    if (rc != WC_OK) return rc;
    if (dx == nullptr && dw == nullptr) return fail(WC_EINVAL, "%s: dx and dw are both NULL", fn);
    if ((dx && !float_type(dx_dtype)) || (dw && !float_type(dw_dtype)))
        return fail(WC_EINVAL, "%s: dx_dtype %d or dw_dtype %d is neither WC_F32 nor WC_BF16", fn, dx_dtype, dw_dtype);
    if (dx && (rc = row_pitch(fn, "dx", ld_dx, T, D)) != WC_OK) return rc;
    if (dw && (rc = row_pitch(fn, "dw", ld_dw, V, D)) != WC_OK) return rc;
    if ((rc = cross_entropy_inputs(fn, &c, targets, id_type)) != WC_OK) return rc;
    if (dw && (rc = values_pointer(fn, "dw", dw, dw_dtype)) != WC_OK) return rc;
    if (T == 0) {
        if (dw == nullptr || accumulate) return WC_OK;
        const size_t size = dw_dtype == WC_BF16 ? 2 : 4;
        return from_cuda(cudaMemset2DAsync(dw, size_t(ld_dw) * size, 0, size_t(D) * size, size_t(V),
                                           static_cast<cudaStream_t>(stream)),
                         fn);
    }
    if (dx && (rc = values_pointer(fn, "dx", dx, dx_dtype)) != WC_OK) return rc;
    if ((rc = values_pointer(fn, "lse", lse, WC_F32)) != WC_OK) return rc;
    if (dlosses && (rc = values_pointer(fn, "dlosses", dlosses, WC_F32)) != WC_OK) return rc;
    WC_REQUIRE_PTR(fn, workspace);
    const int64_t need = wc::cross_entropy_grad_workspace(c);
    if (workspace_bytes < need)
        return fail(WC_EINVAL, "%s: workspace of %lld bytes, %lld are needed", fn, (long long)workspace_bytes,
                    (long long)need);
    rc = written_apart(fn, {matrix("dx", dx, T, D, ld_dx, dx_dtype == WC_BF16 ? 2 : 4),
                            matrix("dw", dw, V, D, ld_dw, dw_dtype == WC_BF16 ? 2 : 4), bytes("workspace", workspace, need)},
                       {matrix("x", x, T, D, ld_x, 2), matrix("w", w, V, D, ld_w, 2),
                        bytes("targets", targets, T * (id_type == WC_I64 ? 8 : 4)), bytes("lse", lse, 4 * T),
                        bytes("dlosses", dlosses, 4 * T)});
    if (rc != WC_OK) return rc;
    c.workspace = workspace;
    c.lse_in = lse;
    c.dlosses = dlosses;
    c.dloss = float(dloss);
    c.dx = dx;
    c.dx_bf16 = dx_dtype == WC_BF16;
    c.ld_dx = ld_dx;
    c.dw = dw;
    c.dw_bf16 = dw_dtype == WC_BF16;
    c.ld_dw = ld_dw;
    c.accumulate = accumulate != 0;
    return from_cuda(wc::launch_cross_entropy_grad(c, static_cast<cudaStream_t>(stream)), fn);
}

WC_API int wc_wait_timeouts(int reset) {
    static const char *fn = "wc_wait_timeouts";
    unsigned int n = 0, m = 0;
    cudaError_t e = wc::fp8_wait_timeouts(&n, reset != 0);
    if (e == cudaSuccess) e = wc::cross_entropy_wait_timeouts(&m, reset != 0);
    if (e != cudaSuccess) return from_cuda(e, fn);
    const uint64_t all = uint64_t(n) + m;
    return all > 0x7FFFFFFFu ? 0x7FFFFFFF : int(all);
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
