// kq_kv_plan.cuh -- what the kernels of the attention over the INT4 key / value cache
// share: which keys and rows a sequence has, the workspace's parts, small arithmetic.
#pragma once

#include <limits.h>

#include "kq_common.cuh"
#include "kq_internal.h"
#include "kq_wait.cuh"

namespace kq {
namespace kv {

constexpr int CH = 128;         // keys per chunk
constexpr int kTileRows = 256;  // rows of a block of the tile kernel
enum : unsigned { kSiteKvWait = 262144u };
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Pairs of fp32 values.
__device__ __forceinline__ uint64_t pair2(float a, float b) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ uint64_t pair2u(uint32_t a, uint32_t b) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ void split2(uint64_t d, float &a, float &b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(d));
}
__device__ __forceinline__ void split2u(uint64_t d, uint32_t &a, uint32_t &b) {
    asm("mov.b64 {%0, %1}, %2;" : "=r"(a), "=r"(b) : "l"(d));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// The tanh of a cap.  Its error has to be relative: a cap far above the scores multiplies it, and scores far below
// the cap are to stay as they are.
//
// tanh within +-1/2: z q(z^2), q of degree 5 fitted to tanh there by least squares with weights that level the error
// (under 1e-10; fp32's own rounding is 3e-8).
__device__ __forceinline__ uint64_t tanh_small(uint64_t z) {
    using tc::f32x2_mul;
    const uint64_t u = f32x2_mul(z, z);
    uint64_t q = pair2(-0.00646002684f, -0.00646002684f);
    q = fma2(q, u, pair2(0.0211690962f, 0.0211690962f));
    q = fma2(q, u, pair2(-0.0538669676f, -0.0538669676f));
    q = fma2(q, u, pair2(0.133326113f, 0.133326113f));
    q = fma2(q, u, pair2(-0.333333105f, -0.333333105f));
    q = fma2(q, u, pair2(1.0f, 1.0f));
    return f32x2_mul(q, z);
}
// tanh of any numbers: z p(z^2) / q(z^2) within +-9, past which tanh is 1 to fp32; p and q of degree 4, fitted to
// tanh there by least squares on q's multiple, with weights that level the relative error (2e-8).  No coefficient is
// negative, so that fp32 loses two bits at most.  z p and q of a pair; a NaN stays one.
__device__ __forceinline__ void tanh_parts(uint64_t &z, uint64_t &q) {
    using tc::f32x2_mul;
    auto within = [](float x) {
        float y;
        asm("{\n\t.reg .f32 t;\n\tmax.NaN.f32 t, %1, 0fC1100000;\n\tmin.NaN.f32 %0, t, 0f41100000;\n\t}" : "=f"(y) : "f"(x));
        return y;
    };
    float a, b;
    split2(z, a, b);
    z = pair2(within(a), within(b));
    const uint64_t u = f32x2_mul(z, z);
    uint64_t p = pair2(1.33545539e-08f, 1.33545539e-08f);
    p = fma2(p, u, pair2(2.06090008e-05f, 2.06090008e-05f));
    p = fma2(p, u, pair2(0.00349558308f, 0.00349558308f));
    p = fma2(p, u, pair2(0.133810207f, 0.133810207f));
    p = fma2(p, u, pair2(1.0f, 1.0f));
    z = f32x2_mul(z, p);
    q = pair2(7.77651337e-07f, 7.77651337e-07f);
    q = fma2(q, u, pair2(0.000328562659f, 0.000328562659f));
    q = fma2(q, u, pair2(0.0258769635f, 0.0258769635f));
    q = fma2(q, u, pair2(0.467143357f, 0.467143357f));
    q = fma2(q, u, pair2(1.0f, 1.0f));
}
// Of two pairs, with one reciprocal (q is under 2^9 each).
__device__ __forceinline__ void tanh_pairs(uint64_t &a, uint64_t &b) {
    using tc::f32x2_mul;
    uint64_t qa, qb;
    tanh_parts(a, qa);
    tanh_parts(b, qb);
    float x0, x1;
    const uint64_t ab = f32x2_mul(qa, qb);  // the first of both, the second of both
    split2(ab, x0, x1);
    const float r = __fdividef(1.0f, x0 * x1);
    const uint64_t rab = pair2(r * x1, r * x0);
    a = f32x2_mul(a, f32x2_mul(rab, qb));
    b = f32x2_mul(b, f32x2_mul(rab, qa));
}
__device__ __forceinline__ float tanh_any(float z) {
    uint64_t p = pair2(z, z), q;
    tanh_parts(p, q);
    float n, d, same;
    split2(p, n, same);
    split2(q, d, same);
    return __fdividef(n, d);
}
// Wait for a phase; gives up as wait_bounded_err does.
__device__ __forceinline__ bool wait_all(uint32_t bar, uint32_t parity, volatile int *abort, unsigned int *err) {
    return __all_sync(0xffffffffu,
                      tc::wait_bounded_err(bar, parity, abort, kSiteKvWait, tc::kWaitLimitNs, false, err));
}

// ---- which keys and rows a unit has ---------------------------------------------

// The launch as its kernels see it.  "Sequence" B, where there is a shared prefix,
// is the prefix with the queries of all sequences.  Own keys and the prefix's are each
// the row kernel's or the tile kernel's; own keys of a batch whose sequences differ much in
// their queries (prompts and single tokens at once) are both's: a sequence with up to `few`
// rows per key head is the row kernel's.
struct Plan {
    KvAttnArgs a;
    int G;             // query heads per key head
    int partial;       // a prefix is there: every kernel's rows are parts, joined at the end
    int rows_own, rows_prefix;   // the row kernel has own keys, the prefix's
    int few;           // where both kernels have own keys: the most rows of a sequence of the row kernel; else 0
    int own_splits, pre_splits;  // the tile kernel's parts of a row, of own keys and of the prefix's (0: not its)
    int ctas;          // blocks of the row kernel
    int later;         // this launch follows another of the same call (see begin_launch)
    int2 *parts;       // [2][T * H] for every row of the row kernel: the first block that has keys of it, and how
                       // many have; with `few`, -1 and own_splits for one of the tile kernel
    float *slot_o;     // [ctas][2][R][D] partial rows: a block's first unit, its last unit
    float *slot_l;     // [ctas][2][R]
    float *whole_o;    // [2][T * H][D] rows whose keys lay in one block (own keys; the prefix's)
    float *whole_l;    // [2][T * H]
    float *tile_o;     // [own_splits + pre_splits][T * H][D] parts of rows
    float *tile_l;     // [own_splits + pre_splits][T * H]
};

struct Seq {
    int n;         // keys
    int m;         // queries that are computed
    int q0;        // first query token
    int shift;     // query i sees the keys t <= shift + i
    int lo;        // no query sees a key below
    int c0, N;     // first chunk, chunks
    int tiles;     // row tiles
    const int32_t *pages;
};

// The row and tile kernels of one call need nothing of one another, so a later one of them does not wait for the
// one before but for its end: its blocks start as the other's give up their SMs.  What they both read was complete
// when the first one's blocks passed their wait, and they let a later launch begin only after it.  The last
// one's end is then the end of all.  (A prefix of 6007 keys behind the own keys of 200 sequences: 90 -> 85 us.)
__device__ __forceinline__ void begin_launch(const Plan &p) {
    if (p.later) __threadfence();
    else griddep_wait();
}
__device__ __forceinline__ void end_launch(const Plan &p) {
    if (p.later) griddep_wait();
}

// First query token and number of queries of sequence b, within the T tokens whatever q_start holds.
__device__ __forceinline__ void queries_of(const KvAttnArgs &a, int64_t b, int &q0, int &m) {
    q0 = int(b);
    m = 1;
    if (a.q_start) {
        const int T = int(a.T);
        q0 = min(max(a.q_start[b], 0), T);
        m = max(min(a.q_start[b + 1], T) - q0, 0);
    }
}
__device__ __forceinline__ int all_queries(const KvAttnArgs &a) {
    return a.q_start ? min(max(a.q_start[a.B], 0), int(a.T)) : int(a.T);
}

template <int R>
__device__ __forceinline__ Seq load_seq(const Plan &p, int64_t b, bool report) {
    const KvAttnArgs &a = p.a;
    Seq s;
    int lo = 0;
    if (b == a.B) {  // the shared prefix: every row sees all of it, but for a window
        s.n = int(a.prefix_len);
        s.q0 = 0;
        s.m = all_queries(a);
        s.shift = s.n;
        s.pages = a.prefix_pages;
    } else {
        int m;
        queries_of(a, b, s.q0, m);
        const int given = max(a.kv_len[b], 0);
        const int most = int(a.max_pages) << a.c.page_shift;
        s.n = min(given, most);
        s.m = min(m, a.max_q);
        if (report && (given > most || m > a.max_q)) {
            atomicOr(a.err, kSiteKvAttention);
            for (int64_t r = int64_t(s.q0 + s.m) * a.q_heads; r < int64_t(s.q0 + m) * a.q_heads; ++r)
                p.parts[r] = make_int2(0, 0);  // rows past the bound
        }
        s.shift = given - m;
        s.pages = a.page_table + b * a.max_pages;
        if (a.window) lo = int(max(int64_t(0), int64_t(s.shift) - a.window + 1));
    }
    // the other kernel's: no rows here
    if (p.few && b != a.B && (s.m * p.G > p.few) != (R == kTileRows)) s.m = 0;
    const int hi = min(s.n, max(0, s.shift + s.m));
    s.lo = lo;
    s.c0 = min(lo, max(hi - 1, 0)) / CH;
    s.N = max(1, (hi + CH - 1) / CH - s.c0);  // a unit without keys still has its rows to write
    s.tiles = (s.m * p.G + R - 1) / R;
    return s;
}

// The sequence of token t (the last that begins at or before it), by a warp: 32 looked at in a step.
__device__ __forceinline__ int seq_of(const KvAttnArgs &a, int t) {
    int lo = 0, hi = int(a.B);
    const int lane = threadIdx.x & 31;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32, k = lo + lane * step;
        const int n = max(1, __popc(__ballot_sync(0xffffffffu, k < hi && a.q_start[k] <= t)));
        lo += (n - 1) * step;
        hi = min(hi, lo + step);
    }
    return lo;
}

// Position of token t's queries among the keys of its sequence (for windows over a prefix).
__device__ __forceinline__ int query_shift(const KvAttnArgs &a, int t) {
    if (!a.q_start) return a.kv_len[t] > 0 ? a.kv_len[t] - 1 : -1;
    int lo = 0, hi = int(a.B);
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (a.q_start[mid + 1] <= t) lo = mid + 1;
        else hi = mid;
    }
    if (lo == int(a.B)) return -1;
    return max(a.kv_len[lo], 0) - (a.q_start[lo + 1] - a.q_start[lo]) + t - a.q_start[lo];
}

}  // namespace kv

// Row tiles (256 rows of a key head) of m queries with G heads each.
inline int64_t kv_tiles(int64_t m, int G) { return (m * G + kv::kTileRows - 1) / kv::kTileRows; }
// The own keys' row tiles have places, per key head, of which a sequence's first lies at own_place of its first
// query: no two sequences' meet, as a part of r rows has at most r / 256 + 1 tiles and, beside a row kernel, more
// than `few` rows.  T tokens have own_place(T, B) at most.
__host__ __device__ inline int64_t own_place(int64_t q, int64_t b, int G, int few) {
    return q * G / kv::kTileRows + (G <= few ? q * G / (few + 1) : b);
}
// Places to launch: those, or what all sequences have at the bound of queries.
inline int64_t kv_own_tiles(int64_t T, int64_t B, int max_q, int G, int few) {
    const int64_t full = kv_tiles(max_q, G) * B, any = own_place(T, B, G, few);
    return full < any ? full : any;
}
// The tile kernel over the own keys of all sequences, or over the prefix.
cudaError_t launch_kv_tile(const kv::Plan &p, bool prefix, int splits, int device, cudaStream_t stream);

}  // namespace kq
