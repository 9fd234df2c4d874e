// embedding.cu -- embedding lookup with scaling, and its gradient.
//
//   out[t]    = scale * table[ids[t] - first]        (zero for ids outside)
//   dtable[v] = scale * sum over t with ids[t] - first = v, t ascending, of dy[t]
//
// ids outside [first, first + V) -- padding, or rows of another rank's shard --
// read as zero and receive nothing.
//
// Lookup: one 16-byte vector per thread and step, four in flight; HBM-bound
// (16384 x 2048 bf16 15 us with the table's rows in L2).
//
// Gradient: three kernels, no atomics on global memory, the same bits every
// run.  (1) sort: each CTA owns a run of table rows, reads every id (they sit
// in L2) and writes the positions of its rows' tokens, in token order, at
// their sorted places -- a stable counting sort in one launch, because a CTA
// learns its place in the output by counting the ids below its rows.  It also
// writes the zeros of its rows without a token: the sort waits on latencies,
// and leaves the memory idle for them.
// (2) sum: the sorted tokens are cut into equal runs, one per worker, so that
// a row with many tokens (Zipf's law) is spread over many workers; a worker
// writes the rows that lie inside its run and leaves fp32 partial sums of the
// at most two rows that cross its ends.  (3) join: adds those partial sums in
// order.  Bound: HBM, reading dy once and writing the table's gradient once:
// 16384 tokens into 32000 x 2048 bf16 take 45.5 us (197 MB, 4.3 TB/s), of which
// the sort waits on latencies for about 8 and the zero rows are written in the
// next 16.  (Zeros for every row at the start of the sort: 52.5 us, its reads
// queue behind them.)  Few tokens are bound by latencies: 3001 x 1002 into
// 50021 fp32 rows 14.6 us.  Every CTA of the sort reads every id, twice beyond 8192
// tokens, so tokens x max(152, rows / 1024) ids come from L2: little at these
// sizes, most of the time with many of both (64 columns added to fp32 rows, 2^20
// tokens: 0.37 ms into 2^15 rows, 0.65 into 2^18, 2.0 into 2^20).
#include "wc_device.cuh"
#include "wc_internal.h"
#include "wc_launch.cuh"
#include "wc_rows.cuh"

namespace wc {

namespace {

// ---------------------------------------------------------------------------
// element access: E values of bf16 or fp32 as one vector
// ---------------------------------------------------------------------------

template <typename T, int E>
struct Pack {
    static constexpr int kBytes = E * int(sizeof(T));
    static constexpr int kWords = kBytes < 4 ? 1 : kBytes / 4;
    uint32_t w[kWords];
};

template <typename T, int E, bool STREAM>
__device__ __forceinline__ Pack<T, E> load_pack(const T *p) {
    Pack<T, E> r;
    constexpr int B = Pack<T, E>::kBytes;
    if constexpr (B >= 16) {
#pragma unroll
        for (int i = 0; i < B / 16; ++i) {
            const uint4 *q = reinterpret_cast<const uint4 *>(p) + i;
            const uint4 v = STREAM ? __ldcs(q) : *q;
            r.w[4 * i] = v.x;
            r.w[4 * i + 1] = v.y;
            r.w[4 * i + 2] = v.z;
            r.w[4 * i + 3] = v.w;
        }
    } else if constexpr (B == 8) {
        const uint2 *q = reinterpret_cast<const uint2 *>(p);
        const uint2 v = STREAM ? __ldcs(q) : *q;
        r.w[0] = v.x;
        r.w[1] = v.y;
    } else if constexpr (B == 4) {
        const uint32_t *q = reinterpret_cast<const uint32_t *>(p);
        r.w[0] = STREAM ? __ldcs(q) : *q;
    } else {
        const uint16_t *q = reinterpret_cast<const uint16_t *>(p);
        r.w[0] = STREAM ? __ldcs(q) : *q;
    }
    return r;
}

template <typename T, int E>
__device__ __forceinline__ void store_pack(T *p, const Pack<T, E> &v) {
    constexpr int B = Pack<T, E>::kBytes;
    if constexpr (B >= 16) {
#pragma unroll
        for (int i = 0; i < B / 16; ++i)
            __stcs(reinterpret_cast<uint4 *>(p) + i,
                   make_uint4(v.w[4 * i], v.w[4 * i + 1], v.w[4 * i + 2], v.w[4 * i + 3]));
    } else if constexpr (B == 8) {
        __stcs(reinterpret_cast<uint2 *>(p), make_uint2(v.w[0], v.w[1]));
    } else if constexpr (B == 4) {
        __stcs(reinterpret_cast<uint32_t *>(p), v.w[0]);
    } else {
        __stcs(reinterpret_cast<uint16_t *>(p), uint16_t(v.w[0]));
    }
}

template <typename T, int E>
__device__ __forceinline__ float pack_value(const Pack<T, E> &v, int e) {
    if constexpr (sizeof(T) == 4) return __uint_as_float(v.w[e]);
    return __uint_as_float((e & 1) ? (v.w[e / 2] & 0xFFFF0000u) : (v.w[e / 2] << 16));
}

template <typename T, int E>
__device__ __forceinline__ Pack<T, E> pack_of(const float x[E]) {
    Pack<T, E> r;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int e = 0; e < E; ++e) r.w[e] = __float_as_uint(x[e]);
    } else if constexpr (E == 1) {
        r.w[0] = f32_to_bf16_bits(x[0]);
    } else {
#pragma unroll
        for (int e = 0; e < E; e += 2) r.w[e / 2] = f32x2_to_bf16x2_bits(x[e], x[e + 1]);
    }
    return r;
}

// id - first; ids at the far negative end wrap to a row beyond any table.
__device__ __forceinline__ int64_t relative(int64_t id, int64_t first) {
    return int64_t(uint64_t(id) - uint64_t(first));
}

template <typename I>
__device__ __forceinline__ int64_t row_of(const I *ids, int64_t t, int64_t first, int64_t V) {
    const int64_t r = relative(ids[t], first);
    return r >= 0 && r < V ? r : -1;
}

// ---------------------------------------------------------------------------
// lookup
// ---------------------------------------------------------------------------

constexpr int kLookupThreads = 256;
constexpr int kLookupUnroll = 4;

// vecs: vectors of E values in a row; a CTA covers kLookupThreads *
// kLookupUnroll consecutive vectors of the [n][vecs] output.
template <typename T, typename I, int E>
__global__ void __launch_bounds__(kLookupThreads)
lookup_kernel(const T *__restrict__ table, int64_t ld_table, const I *__restrict__ ids, int64_t n,
              int64_t first, int64_t V, uint32_t vecs, float scale, T *__restrict__ out,
              int64_t ld_out) {
    const int64_t base = int64_t(blockIdx.x) * (kLookupThreads * kLookupUnroll);
    const int64_t t0 = base / vecs;
    const uint32_t v0 = uint32_t(base - t0 * vecs);
    Pack<T, E> r[kLookupUnroll];
    int64_t tok[kLookupUnroll], row[kLookupUnroll];
    uint32_t vec[kLookupUnroll];
#pragma unroll
    for (int j = 0; j < kLookupUnroll; ++j) {
        const uint32_t at = v0 + threadIdx.x + j * kLookupThreads;  // < vecs + 1024
        const uint32_t dt = at / vecs;
        tok[j] = t0 + dt;
        vec[j] = at - dt * vecs;
        row[j] = tok[j] < n ? row_of(ids, tok[j], first, V) : -1;
    }
#pragma unroll
    for (int j = 0; j < kLookupUnroll; ++j) {
        if (row[j] >= 0) {
            r[j] = load_pack<T, E, false>(table + row[j] * ld_table + int64_t(vec[j]) * E);
        } else {
#pragma unroll
            for (int w = 0; w < Pack<T, E>::kWords; ++w) r[j].w[w] = 0u;
        }
    }
#pragma unroll
    for (int j = 0; j < kLookupUnroll; ++j) {
        if (tok[j] >= n) continue;
        if (scale != 1.0f && row[j] >= 0) {
            float x[E];
#pragma unroll
            for (int e = 0; e < E; ++e) x[e] = __fmul_rn(pack_value<T, E>(r[j], e), scale);
            r[j] = pack_of<T, E>(x);
        }
        store_pack<T, E>(out + tok[j] * ld_out + int64_t(vec[j]) * E, r[j]);
    }
}

// The same where rows start on any element: a thread has one aligned chunk of 16
// bytes of an output row (chunks: of a row at most), and shifts the values that
// belong there into place; the ends of a row go value by value.
template <typename T, typename I>
__global__ void __launch_bounds__(kLookupThreads)
lookup_any_kernel(const T *__restrict__ table, int64_t ld_table, const I *__restrict__ ids, int64_t n,
                  int64_t first, int64_t V, int32_t D, uint32_t chunks, float scale, T *__restrict__ out,
                  int64_t ld_out) {
    constexpr int W = 16 / int(sizeof(T));  // values of a chunk
    const int64_t base = int64_t(blockIdx.x) * (kLookupThreads * kLookupUnroll);
    const int64_t t0 = base / chunks;
    const uint32_t v0 = uint32_t(base - t0 * chunks);
    const T *const end = table + (V - 1) * ld_table + D;
    uint32_t t[kLookupUnroll][8];
    const T *from[kLookupUnroll];  // of the chunk's first value
    T *to[kLookupUnroll];
    int32_t lo[kLookupUnroll], hi[kLookupUnroll];  // values of the chunk that belong to the row
    bool zero[kLookupUnroll], whole[kLookupUnroll];
#pragma unroll
    for (int j = 0; j < kLookupUnroll; ++j) {
        const uint32_t at = v0 + threadIdx.x + j * kLookupThreads;
        const uint32_t dt = at / chunks;
        const int64_t token = t0 + dt;
        const int64_t row = token < n ? row_of(ids, token, first, V) : -1;
        T *const dst = out + token * ld_out;
        const int32_t lead = int32_t(reinterpret_cast<uintptr_t>(dst) & 15u) / int32_t(sizeof(T));
        const int32_t c = int32_t(at - dt * chunks) * W - lead;  // column of the chunk's first value
        to[j] = dst + c;
        lo[j] = max(0, -c);
        hi[j] = token < n ? min(W, D - c) : 0;
        zero[j] = row < 0;
        from[j] = table + row * ld_table + c;
        whole[j] = !zero[j] && lo[j] == 0 && hi[j] == W && end - from[j] >= 2 * W;
        if (whole[j]) load_chunks(from[j], t[j]);
    }
#pragma unroll
    for (int j = 0; j < kLookupUnroll; ++j) {
        if (whole[j] || (zero[j] && lo[j] == 0 && hi[j] == W)) {
            Pack<T, W> r;
#pragma unroll
            for (int k = 0; k < 4; ++k) r.w[k] = 0u;
            if (whole[j]) {
                shift_words(from[j], t[j], r.w);
                if (scale != 1.0f) {
                    float x[W];
#pragma unroll
                    for (int e = 0; e < W; ++e) x[e] = __fmul_rn(pack_value<T, W>(r, e), scale);
                    r = pack_of<T, W>(x);
                }
            }
            store_pack<T, W>(to[j], r);
        } else {
            for (int32_t e = lo[j]; e < hi[j]; ++e) {
                Pack<T, 1> r;
                r.w[0] = 0u;
                if (!zero[j]) {
                    r = load_pack<T, 1, false>(from[j] + e);
                    if (scale != 1.0f) {
                        const float x[1] = {__fmul_rn(pack_value<T, 1>(r, 0), scale)};
                        r = pack_of<T, 1>(x);
                    }
                }
                store_pack<T, 1>(to[j] + e, r);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// gradient (1): stable counting sort of the tokens by row, and zero rows
// ---------------------------------------------------------------------------

constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortUnroll = 8;
constexpr int kSortPitch = kSortWarps + 1;  // counters of a row; odd, so that a warp's
                                            // counters of different rows are in different banks

// Zeros for the rows without a token: bytes of a row and distance of rows, both
// even.  base NULL: none are written.
struct ZeroRows {
    char *base;
    int64_t pitch, bytes;
};

// A warp's zeros: 16 bytes at a time, and what lies before the first and after
// the last 16-byte boundary two by two (two by two alone, a gradient of
// 32000 x 2047 bf16 takes 131 us instead of 104).
__device__ __forceinline__ void zero_row(char *p, int64_t bytes, int lane) {
    const int64_t lead = int64_t(16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15;
    const int64_t head = lead < bytes ? lead : bytes;
    const int64_t body = (bytes - head) / 16, tail = bytes - head - 16 * body;
    if (2 * lane < head) __stcs(reinterpret_cast<uint16_t *>(p) + lane, uint16_t(0));
    for (int64_t i = lane; i < body; i += 32)
        __stcs(reinterpret_cast<uint4 *>(p + head) + i, make_uint4(0u, 0u, 0u, 0u));
    if (2 * lane < tail) __stcs(reinterpret_cast<uint16_t *>(p + head + 16 * body) + lane, uint16_t(0));
}

// Rows of tokens t, t + 32, ..., as places in [lo, hi), -1 outside; counts the
// ones below.
template <typename I>
__device__ __forceinline__ void load_rows(const I *ids, int64_t t, int64_t end, int64_t first,
                                          int32_t lo, int32_t hi, int32_t (&k)[kSortUnroll],
                                          int32_t &below) {
    int64_t r[kSortUnroll];
#pragma unroll
    for (int u = 0; u < kSortUnroll; ++u) r[u] = t + 32 * u < end ? relative(ids[t + 32 * u], first) : -1;
#pragma unroll
    for (int u = 0; u < kSortUnroll; ++u) {
        if (r[u] >= 0 && r[u] < lo) ++below;
        k[u] = r[u] >= lo && r[u] < hi ? int32_t(r[u] - lo) : -1;
    }
}

// order[p], rows[p]: token and row at sorted place p.  row_start[v]: first
// place of row v; row_start[V]: tokens with a row.  CTA b owns rows
// [b * per_cta, (b + 1) * per_cta).  All of its shared memory is dynamic,
// sort_smem(per_cta) bytes: what a launch asks for is then what the 48 KB that
// need no opt-in are compared with.
__host__ __device__ constexpr size_t sort_smem(int32_t per_cta) {
    return (size_t(per_cta) * (kSortPitch + 1) + kSortWarps + 1) * 4;
}

template <typename I>
__global__ void __launch_bounds__(kSortThreads)
sort_kernel(const I *__restrict__ ids, int32_t n, int64_t first, int32_t V, int32_t per_cta,
            int32_t *__restrict__ order, int32_t *__restrict__ rows,
            int32_t *__restrict__ row_start, const ZeroRows zeros) {
    extern __shared__ int32_t counters[];
    let_successor_start();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int32_t lo = int32_t(blockIdx.x) * per_cta;
    const int32_t hi = min(V, lo + per_cta);
    const int32_t own = hi - lo;
    int32_t *base = counters + per_cta * kSortPitch;  // first place of each row
    int32_t *warp_total = base + per_cta;
    int32_t &below_total = warp_total[kSortWarps];
    for (int i = threadIdx.x; i < per_cta * (kSortPitch + 1); i += kSortThreads) counters[i] = 0;
    if (threadIdx.x == 0) below_total = 0;
    __syncthreads();

    // each warp counts its own consecutive stretch of tokens; one that fits is
    // kept for the second pass
    const int32_t stretch = int32_t((int64_t(n) + kSortWarps - 1) / kSortWarps + 31) / 32 * 32;
    const int64_t begin = int64_t(stretch) * warp;
    const int64_t end = begin + stretch < int64_t(n) ? begin + stretch : int64_t(n);
    const bool kept = stretch <= 32 * kSortUnroll;
    int32_t below = 0, k[kSortUnroll];
    for (int64_t t0 = begin; t0 < end; t0 += 32 * kSortUnroll) {
        load_rows(ids, t0 + lane, end, first, lo, hi, k, below);
#pragma unroll
        for (int u = 0; u < kSortUnroll; ++u)
            if (k[u] >= 0) atomicAdd(&counters[k[u] * kSortPitch + warp], 1);
    }
    below = __reduce_add_sync(kFull, below);
    if (lane == 0) atomicAdd(&below_total, below);
    __syncthreads();

    // places: rows in order, and within a row the warps in order
    int32_t carry = below_total;
    for (int32_t r0 = 0; r0 < own; r0 += kSortThreads) {
        const int32_t r = r0 + int32_t(threadIdx.x);
        int32_t c = 0;
        if (r < own) {
            int32_t *of = counters + r * kSortPitch;
#pragma unroll 8
            for (int w = 0; w < kSortWarps; ++w) {
                const int32_t x = of[w];
                of[w] = c;
                c += x;
            }
        }
        int32_t inc = c;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int32_t u = __shfl_up_sync(kFull, inc, off);
            if (lane >= off) inc += u;
        }
        if (lane == 31) warp_total[warp] = inc;
        __syncthreads();
        int32_t before = 0, all = 0;
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w) {
            if (w < warp) before += warp_total[w];
            all += warp_total[w];
        }
        const int32_t at = carry + before + inc - c;
        if (r < own) {
            base[r] = at;
            row_start[lo + r] = at;
        }
        carry += all;
        __syncthreads();
    }
    if (hi == V && threadIdx.x == 0) row_start[V] = carry;

    if (zeros.base != nullptr) {  // drained by the memory system while the rest runs
        for (int32_t r = warp; r < own; r += kSortWarps) {
            if (base[r] != (r + 1 < own ? base[r + 1] : carry)) continue;
            zero_row(zeros.base + int64_t(lo + r) * zeros.pitch, zeros.bytes, lane);
        }
    }

    // the same stretch again, in order: equal rows of a step keep lane order
    for (int64_t t0 = begin; t0 < end; t0 += 32 * kSortUnroll) {
        int32_t unused = 0;
        if (!kept) load_rows(ids, t0 + lane, end, first, lo, hi, k, unused);
#pragma unroll
        for (int u = 0; u < kSortUnroll; ++u) {
            const unsigned live = __ballot_sync(kFull, k[u] >= 0);
            if (k[u] >= 0) {
                const unsigned peers = __match_any_sync(live, k[u]);
                int32_t *counter = &counters[k[u] * kSortPitch + warp];
                const int32_t at = base[k[u]] + *counter + __popc(peers & ((1u << lane) - 1u));
                order[at] = int32_t(t0 + 32 * u + lane);
                rows[at] = lo + k[u];
                __syncwarp(live);
                if ((peers & ((1u << lane) - 1u)) == 0u) *counter += __popc(peers);
            }
            __syncwarp();
        }
    }
}

// ---------------------------------------------------------------------------
// gradient (2): sums over equal runs of sorted tokens
// ---------------------------------------------------------------------------

constexpr int kSumThreads = 256;
// Tokens of a step: narrow packs leave registers for more of them in flight, but
// not beside old values (12103 tokens of 1091 bf16 values, the whole gradient:
// 36.0 us with four, 32.4 with eight; 3001 of 1002 added to fp32: 14.3 and 15.9).
__host__ __device__ constexpr int sum_unroll(int e, bool acc) { return e <= 2 && !acc ? 8 : 4; }

struct SumPlan {
    int32_t n;        // tokens
    int32_t V;        // rows
    uint32_t D;       // columns
    uint32_t vecs;    // vectors of E columns
    uint32_t lanes;   // threads of a worker along the columns (power of two <= 256)
    uint32_t workers;
};

// Sorted places [begin, end) of a worker; returns the length of a run.
__device__ __forceinline__ uint32_t run_of(const int32_t *row_start, const SumPlan &p, uint32_t w,
                                       int32_t *begin, int32_t *end) {
    const uint32_t live = uint32_t(row_start[p.V]);
    const uint32_t per = (live + p.workers - 1) / p.workers;
    const uint64_t b = uint64_t(per) * w, e = b + per;
    *begin = int32_t(b < live ? b : live);
    *end = int32_t(e < live ? e : live);
    return per;
}

// scale * acc, added to `old` if ACC.
template <bool ACC, typename TO, int E>
__device__ __forceinline__ void write_row(TO *p, const float acc[E], float scale, const Pack<TO, E> &old) {
    float x[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        x[e] = __fmul_rn(acc[e], scale);
        if (ACC) x[e] = __fadd_rn(pack_value<TO, E>(old, e), x[e]);
    }
    store_pack<TO, E>(p, pack_of<TO, E>(x));
}

// heads, tails: [workers][D] fp32.  heads[w]: the part in run w of a row that
// began in an earlier run and ends in this one.  tails[w]: the part in run w
// of a row that goes on in the next run.  joins[w]: the row that heads[w] is a
// part of (-1: none) and the run it begins in.
// The places of the next step are read during this one, and with ACC the old
// values of every row that ends in a step beside its tokens: a worker has few
// tokens, and what it waits for is one memory latency after another (3001
// tokens added to fp32 rows: 11.3 -> 7.6 us).
template <typename TI, typename TO, int E, bool ACC>
__global__ void __launch_bounds__(kSumThreads)
sum_kernel(const TI *__restrict__ dy, int64_t ld_dy, const int32_t *__restrict__ order,
           const int32_t *__restrict__ rows, const int32_t *__restrict__ row_start, SumPlan p,
           float scale, TO *__restrict__ dtable, int64_t ld_out,
           float *__restrict__ heads, float *__restrict__ tails, int2 *__restrict__ joins) {
    constexpr int kUnroll = sum_unroll(E, ACC);
    const uint32_t lane = threadIdx.x & (p.lanes - 1);
    const uint32_t w = blockIdx.x * (kSumThreads / p.lanes) + threadIdx.x / p.lanes;
    const uint32_t v = blockIdx.y * p.lanes + lane;
    if (w >= p.workers || v >= p.vecs) return;
    const int64_t col = int64_t(v) * E;
    let_successor_start();
    wait_for_predecessor();
    int32_t begin, end;
    const uint32_t per = run_of(row_start, p, w, &begin, &end);
    int2 join = make_int2(-1, 0);
    if (begin < end) {
        const int32_t live = row_start[p.V];
        const int32_t prior = begin > 0 ? rows[begin - 1] : -1;
        const int32_t next = end < live ? rows[end] : -1;
        float acc[E];
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = 0.0f;
        // rows of places j .. j + kUnroll, `next` at `end`; tokens of all but the last
        int32_t r[kUnroll + 1], token[kUnroll];
        auto places = [&](int32_t j) {
#pragma unroll
            for (int u = 0; u <= kUnroll; ++u) {
                r[u] = j + u < end ? rows[j + u] : next;
                if (u < kUnroll && j + u < end) token[u] = order[j + u];
            }
        };
        places(begin);
        for (int32_t j = begin; j < end; j += kUnroll) {
            Pack<TI, E> g[kUnroll];
            Pack<TO, E> old[kUnroll] = {};
            int32_t row[kUnroll + 1];
#pragma unroll
            for (int u = 0; u <= kUnroll; ++u) row[u] = r[u];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                if (j + u >= end) continue;
                g[u] = load_pack<TI, E, true>(dy + int64_t(token[u]) * ld_dy + col);
                if (ACC && row[u] != row[u + 1] && row[u] != prior)
                    old[u] = load_pack<TO, E, true>(dtable + int64_t(row[u]) * ld_out + col);
            }
            if (j + kUnroll < end) places(j + kUnroll);
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                if (j + u >= end) break;
#pragma unroll
                for (int e = 0; e < E; ++e) acc[e] = __fadd_rn(acc[e], pack_value<TI, E>(g[u], e));
                if (row[u] == row[u + 1]) continue;  // goes on, maybe in the next run
                if (row[u] == prior) {
                    join = make_int2(row[u], int32_t(uint32_t(row_start[row[u]]) / per));
#pragma unroll
                    for (int e = 0; e < E; ++e) heads[int64_t(w) * p.D + col + e] = acc[e];
                } else {
                    write_row<ACC, TO, E>(dtable + int64_t(row[u]) * ld_out + col, acc, scale, old[u]);
                }
#pragma unroll
                for (int e = 0; e < E; ++e) acc[e] = 0.0f;
            }
        }
        if (rows[end - 1] == next) {
#pragma unroll
            for (int e = 0; e < E; ++e) tails[int64_t(w) * p.D + col + e] = acc[e];
        }
    }
    if (blockIdx.y == 0 && lane == 0) joins[w] = join;
}

// ---------------------------------------------------------------------------
// gradient (3): rows that cross runs
// ---------------------------------------------------------------------------

constexpr int kJoinLanes = 64;   // threads along the columns, E columns each
constexpr int kJoinParts = 4;    // threads that share a row's runs
constexpr int kJoinThreads = kJoinLanes * kJoinParts;
constexpr int kJoinUnroll = 4;

// CTA (y, w): if a row that began earlier ends in run w, adds its parts over
// the runs, split in four consecutive shares that are added in order.  Up to
// four parts -- all but the rows with many tokens -- are a share each; a thread
// adds its columns' alone then, and fewer CTAs have work.  (A CTA per 256
// columns: with two CTAs for all of a run's columns the row of the most
// frequent token took 11.5 us instead of 6.9; with eight shares the start of
// the idle CTAs cost as much.)
template <typename TO, int E, bool ACC>
__global__ void __launch_bounds__(kJoinThreads)
join_kernel(SumPlan p, float scale, TO *__restrict__ dtable, int64_t ld_out,
            const float *__restrict__ heads, const float *__restrict__ tails,
            const int2 *__restrict__ joins) {
    __shared__ float part[kJoinParts][kJoinLanes * E];
    const uint32_t w = blockIdx.y, y = blockIdx.x;
    wait_for_predecessor();
    const int2 join = joins[w];
    if (join.x < 0) return;
    const uint32_t first = uint32_t(join.y);
    TO *row = dtable + int64_t(join.x) * ld_out;
    // parts first .. w - 1 are tails, part w is a head
    const uint32_t count = w - first;
    auto tail = [&](uint32_t i, uint32_t col) {
        return load_pack<float, E, true>(tails + int64_t(i) * p.D + col);
    };
    auto finish = [&](float (&sum)[E], const Pack<float, E> &head, const Pack<TO, E> &old, uint32_t col) {
#pragma unroll
        for (int k = 0; k < E; ++k) sum[k] = __fadd_rn(sum[k], pack_value<float, E>(head, k));
        write_row<ACC, TO, E>(row + col, sum, scale, old);
    };
    if (count <= uint32_t(kJoinParts)) {
        const uint32_t col = (y * kJoinThreads + threadIdx.x) * E;
        if (col < p.D) {
            Pack<float, E> x[kJoinParts];
#pragma unroll
            for (uint32_t u = 0; u < kJoinParts; ++u)
                if (u < count) x[u] = tail(first + u, col);
            const Pack<float, E> head = load_pack<float, E, true>(heads + int64_t(w) * p.D + col);
            Pack<TO, E> old = {};
            if (ACC) old = load_pack<TO, E, true>(row + col);
            float sum[E];
#pragma unroll
            for (int k = 0; k < E; ++k) sum[k] = 0.0f;
#pragma unroll
            for (uint32_t u = 0; u < kJoinParts; ++u)
                if (u < count) {
#pragma unroll
                    for (int k = 0; k < E; ++k) sum[k] = __fadd_rn(sum[k], pack_value<float, E>(x[u], k));
                }
            finish(sum, head, old, col);
        }
        return;
    }
    const uint32_t c = threadIdx.x % kJoinLanes, s = threadIdx.x / kJoinLanes;
    const uint32_t share = (count + kJoinParts - 1) / kJoinParts;
    const uint32_t b = first + s * share < w ? first + s * share : w;
    const uint32_t e = b + share < w ? b + share : w;
    const uint32_t col = (y * kJoinLanes + c) * E;
    float sum[E];
#pragma unroll
    for (int k = 0; k < E; ++k) sum[k] = 0.0f;
    if (col < p.D) {
        for (uint32_t i = b; i < e; i += kJoinUnroll) {
            Pack<float, E> x[kJoinUnroll];
#pragma unroll
            for (int u = 0; u < kJoinUnroll; ++u)
                if (i + u < e) x[u] = tail(i + u, col);
#pragma unroll
            for (int u = 0; u < kJoinUnroll; ++u)
                if (i + u < e) {
#pragma unroll
                    for (int k = 0; k < E; ++k) sum[k] = __fadd_rn(sum[k], pack_value<float, E>(x[u], k));
                }
        }
    }
#pragma unroll
    for (int k = 0; k < E; ++k) part[s][c * E + k] = sum[k];
    __syncthreads();
    if (s != 0 || col >= p.D) return;
    const Pack<float, E> head = load_pack<float, E, true>(heads + int64_t(w) * p.D + col);
    Pack<TO, E> old = {};
    if (ACC) old = load_pack<TO, E, true>(row + col);
#pragma unroll
    for (int k = 0; k < E; ++k)
#pragma unroll
        for (int i = 1; i < kJoinParts; ++i) sum[k] = __fadd_rn(sum[k], part[i][c * E + k]);
    finish(sum, head, old, col);
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------

constexpr int kSms = 152;
// The sort fills at most 137 KB of shared memory (larger tables
// take more CTAs than SMs).
constexpr int32_t kSortRowsMax = 1024;
constexpr int kSumCtas = 4 * kSms;

// Widest vector (in values) that every row of both buffers starts on.
int vector_width(uint32_t D, int64_t ld_a, int size_a, int64_t ld_b, int size_b) {
    int e = 8;
    while (e > 1 && (D % e || (ld_a * size_a) % (e * size_a > 16 ? 16 : e * size_a) ||
                     (ld_b * size_b) % (e * size_b > 16 ? 16 : e * size_b)))
        e /= 2;
    return e;
}

SumPlan plan_of(const EmbeddingGrad &a, int e) {
    SumPlan p;
    p.n = int32_t(a.n);
    p.V = int32_t(a.V);
    p.D = uint32_t(a.D);
    p.vecs = p.D / e;
    p.lanes = 8;
    while (p.lanes < p.vecs && p.lanes < uint32_t(kSumThreads)) p.lanes *= 2;
    // fewer lanes where that leaves fewer idle (331 vectors in 3 x 128 lanes and not
    // 2 x 256: 14427 tokens added to bf16 rows 38.4 -> 34.1 us)
    auto padded = [&](uint32_t lanes) { return (p.vecs + lanes - 1) / lanes * lanes; };
    while (p.lanes > 64 && padded(p.lanes / 2) < padded(p.lanes)) p.lanes /= 2;
    const uint32_t slices = (p.vecs + p.lanes - 1) / p.lanes;
    const uint32_t ctas = (kSumCtas + slices - 1) / slices;
    p.workers = ctas * (kSumThreads / p.lanes);
    return p;
}

int grad_width(const EmbeddingGrad &a) {
    return vector_width(uint32_t(a.D), a.ld_dy, a.dy_bf16 ? 2 : 4, a.ld_out, a.out_bf16 ? 2 : 4);
}

int64_t align16(int64_t bytes) { return (bytes + 15) / 16 * 16; }

template <typename T, typename I>
cudaError_t lookup(const void *table, int64_t ld_table, const void *ids, int64_t n, int64_t first,
                   int64_t V, int64_t D, float scale, void *out, int64_t ld_out,
                   cudaStream_t stream) {
    int e = vector_width(uint32_t(D), ld_table, int(sizeof(T)), ld_out, int(sizeof(T)));
    if (sizeof(T) == 4 && e > 4) e = 4;
    // Rows on no more than 4 bytes, unless they are short: 16384 of 2047 bf16 values
    // 79 us by single values and 31 in chunks, of 151 7.6 and 6.6, of 71 4.7 and 5.8;
    // by pairs of 2046 43 us and 30, of 502 12.2 and 12.4.  Few values are bound by
    // latency, which is longer in chunks (37 tokens of 1001 fp32 values 2.0 and 3.1).
    if (e * int(sizeof(T)) <= 4 && D * int(sizeof(T)) >= (e == 1 ? 256 : 2048) && n * D >= (1 << 18)) {
        const uint32_t chunks = uint32_t((D * int64_t(sizeof(T)) + 14) / 16 + 1);
        const int64_t per_cta = kLookupThreads * kLookupUnroll;
        lookup_any_kernel<T, I><<<uint32_t((n * chunks + per_cta - 1) / per_cta), kLookupThreads, 0, stream>>>(
            static_cast<const T *>(table), ld_table, static_cast<const I *>(ids), n, first, V, int32_t(D),
            chunks, scale, static_cast<T *>(out), ld_out);
        return cudaPeekAtLastError();
    }
    const uint32_t vecs = uint32_t(D / e);
    const int64_t per = kLookupThreads * kLookupUnroll;
    const uint32_t grid = uint32_t((n * vecs + per - 1) / per);
#define WC_LOOKUP(E)                                                                          \
    lookup_kernel<T, I, E><<<grid, kLookupThreads, 0, stream>>>(                              \
        static_cast<const T *>(table), ld_table, static_cast<const I *>(ids), n, first, V,    \
        vecs, scale, static_cast<T *>(out), ld_out)
    if constexpr (sizeof(T) == 2) {
        if (e == 8) {
            WC_LOOKUP(8);
            return cudaPeekAtLastError();
        }
    }
    if (e >= 4) WC_LOOKUP(4);
    else if (e == 2) WC_LOOKUP(2);
    else WC_LOOKUP(1);
#undef WC_LOOKUP
    return cudaPeekAtLastError();
}

template <typename TI, typename TO, bool ACC>
cudaError_t launch_sum(const EmbeddingGrad &a, const SumPlan &p, int e, const int32_t *order,
                       const int32_t *rows, const int32_t *row_start, float *heads, float *tails,
                       int2 *joins, cudaStream_t stream) {
    const dim3 grid((p.workers + kSumThreads / p.lanes - 1) / (kSumThreads / p.lanes),
                    (p.vecs + p.lanes - 1) / p.lanes);
    TO *dtable = static_cast<TO *>(a.dtable);
#define WC_SUM(E)                                                                             \
    launch_after(sum_kernel<TI, TO, E, ACC>, grid, dim3(kSumThreads), 0, stream, 1,           \
                 static_cast<const TI *>(a.dy), a.ld_dy, order, rows, row_start, p, a.scale,  \
                 dtable, a.ld_out, heads, tails, joins)
    cudaError_t err = e == 8 ? WC_SUM(8) : e == 4 ? WC_SUM(4) : e == 2 ? WC_SUM(2) : WC_SUM(1);
#undef WC_SUM
    if (err != cudaSuccess || a.n < 2) return err;  // one token crosses no run
#define WC_JOIN(E)                                                                            \
    launch_after(join_kernel<TO, E, ACC>,                                                     \
                 dim3((p.D + kJoinLanes * E - 1) / (kJoinLanes * E), p.workers),              \
                 dim3(kJoinThreads), 0, stream, 1, p, a.scale, dtable, a.ld_out, heads, tails, joins)
    return e >= 4 ? WC_JOIN(4) : e == 2 ? WC_JOIN(2) : WC_JOIN(1);
#undef WC_JOIN
}

template <typename TI, typename TO>
cudaError_t launch_sum(const EmbeddingGrad &a, const SumPlan &p, int e, const int32_t *order,
                       const int32_t *rows, const int32_t *row_start, float *heads, float *tails,
                       int2 *joins, cudaStream_t stream) {
    return a.accumulate ? launch_sum<TI, TO, true>(a, p, e, order, rows, row_start, heads, tails, joins, stream)
                        : launch_sum<TI, TO, false>(a, p, e, order, rows, row_start, heads, tails, joins, stream);
}

}  // namespace

cudaError_t launch_embedding(const void *table, bool bf16, int64_t ld_table, const void *ids,
                             bool wide, int64_t n, int64_t first, int64_t V, int64_t D,
                             float scale, void *out, int64_t ld_out, cudaStream_t stream) {
    if (bf16)
        return wide ? lookup<uint16_t, int64_t>(table, ld_table, ids, n, first, V, D, scale, out, ld_out, stream)
                    : lookup<uint16_t, int32_t>(table, ld_table, ids, n, first, V, D, scale, out, ld_out, stream);
    return wide ? lookup<float, int64_t>(table, ld_table, ids, n, first, V, D, scale, out, ld_out, stream)
                : lookup<float, int32_t>(table, ld_table, ids, n, first, V, D, scale, out, ld_out, stream);
}

int64_t embedding_grad_workspace(const EmbeddingGrad &a) {
    // the plan with the fewest columns per vector has the most workers x D
    int64_t most = 0;
    for (int e = 1; e <= 8; e *= 2) {
        if (a.D % e) continue;
        const SumPlan p = plan_of(a, e);
        const int64_t bytes = 2 * align16(int64_t(p.workers) * p.D * 4) + align16(int64_t(p.workers) * 8);
        if (bytes > most) most = bytes;
    }
    return 2 * align16(a.n * 4) + align16((a.V + 1) * 4) + most;
}

cudaError_t launch_embedding_grad(const EmbeddingGrad &a, cudaStream_t stream) {
    const int e = grad_width(a);
    const SumPlan p = plan_of(a, e);
    char *ws = static_cast<char *>(a.workspace);
    int32_t *order = reinterpret_cast<int32_t *>(ws);
    ws += align16(a.n * 4);
    int32_t *rows = reinterpret_cast<int32_t *>(ws);
    ws += align16(a.n * 4);
    int32_t *row_start = reinterpret_cast<int32_t *>(ws);
    ws += align16((a.V + 1) * 4);
    float *heads = reinterpret_cast<float *>(ws);
    ws += align16(int64_t(p.workers) * p.D * 4);
    float *tails = reinterpret_cast<float *>(ws);
    ws += align16(int64_t(p.workers) * p.D * 4);
    int2 *joins = reinterpret_cast<int2 *>(ws);

    int32_t per_cta = int32_t((a.V + kSms - 1) / kSms);
    if (per_cta > kSortRowsMax) per_cta = kSortRowsMax;
    const uint32_t sort_grid = uint32_t((a.V + per_cta - 1) / per_cta);
    const size_t smem = sort_smem(per_cta);
    cudaError_t err = cudaSuccess;
    if (smem > 48 * 1024)
        err = a.wide ? cudaFuncSetAttribute(sort_kernel<int64_t>,
                                            cudaFuncAttributeMaxDynamicSharedMemorySize,
                                            int(sort_smem(kSortRowsMax)))
                     : cudaFuncSetAttribute(sort_kernel<int32_t>,
                                            cudaFuncAttributeMaxDynamicSharedMemorySize,
                                            int(sort_smem(kSortRowsMax)));
    if (err != cudaSuccess) return err;
    ZeroRows zeros = {};
    if (!a.accumulate) {
        const int64_t size = a.out_bf16 ? 2 : 4;
        zeros.base = static_cast<char *>(a.dtable);
        zeros.pitch = a.ld_out * size;
        zeros.bytes = a.D * size;
    }
    if (a.wide)
        sort_kernel<int64_t><<<sort_grid, kSortThreads, smem, stream>>>(
            static_cast<const int64_t *>(a.ids), p.n, a.first, p.V, per_cta, order, rows, row_start, zeros);
    else
        sort_kernel<int32_t><<<sort_grid, kSortThreads, smem, stream>>>(
            static_cast<const int32_t *>(a.ids), p.n, a.first, p.V, per_cta, order, rows, row_start, zeros);
    err = cudaPeekAtLastError();
    if (err != cudaSuccess || a.n == 0) return err;
    if (a.dy_bf16)
        return a.out_bf16 ? launch_sum<uint16_t, uint16_t>(a, p, e, order, rows, row_start, heads, tails, joins, stream)
                          : launch_sum<uint16_t, float>(a, p, e, order, rows, row_start, heads, tails, joins, stream);
    return a.out_bf16 ? launch_sum<float, uint16_t>(a, p, e, order, rows, row_start, heads, tails, joins, stream)
                      : launch_sum<float, float>(a, p, e, order, rows, row_start, heads, tails, joins, stream);
}

}  // namespace wc
