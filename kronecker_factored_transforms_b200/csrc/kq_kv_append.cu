// kq_kv_append.cu -- new tokens into the pages of the INT4 key / value cache, and
// their rows back out.
//
//     q_out = R(pos) q Pq,   y = R(pos) k Pk  or  v Pv,
//     s = alpha max|y| / 7,  code = clamp(round_half_even(y / s), -8, 7)
//
// All rows of one kind (queries, keys, values) are one [rows x D] [D x D] product:
// tiles of 128 rows, a thread and a TMEM lane per row, D its head_dim.  The bytes of
// the rows bound it (2 D in, and 2 D or D / 2 + 4 out), so a row moves once each way:
//   - a warp fetches its 32 rows by cp.async, two rows a step, into padded rows of
//     shared memory (a thread then reads its row 16 bytes at a time without conflicts),
//     the rows of the tile after next as soon as their place is free; query rows leave
//     through the same place, again two whole rows a store.
//   - the thread rotates its row in fp32 and splits each value into bf16 terms by
//     truncation, which go to TMEM as the A operand: two terms for queries (16 bits;
//     the result is rounded to bf16), three for keys (all 24 bits of the fp32 value),
//     one for values (they are bf16).  The factor is the B operand in shared memory,
//     as it lies in memory (N contiguous).
//   - two teams, each with 256 TMEM columns: eight warps turn rows into terms (128
//     columns; two warps share the rows of a TMEM quarter, every second 16 bytes each),
//     four take the fp32 rows (128 columns) while the eight are at their next tile.
//     The keys' largest term waits, in the row's place, for the products of the other two
//     and takes their columns (smallest first: the tensor core truncates the sum at every
//     addition).
//   - one block an SM, all its tiles of one kind, so that it needs one factor.
//
// Codes of exact arithmetic: where y / s lies nearer to a rounding border than fp32 can
// tell, the code is computed again by its warp in fp64.  How near that is follows from
// the row and the factor: |x| |P_j| (of two-norms, the largest column's) is the most
// that products add up to on the way to a sum that cancels (see error_of).  The warps
// that make terms sum a row's squares on the way, the block its factor's columns'.
// A row in ten has such a value, three of the 32 of a warp, so they are done four at a
// time, eight lanes each, with the row and its row of the table brought to shared memory
// (5000 clocks; one after another, from L2, they took 6000 each).
//
// Measured: 129-133 us for 8192 tokens of 64 query and 8 key heads of 128 with a rotary
// table (2.7 TB/s of 6.55), with the read-back of their keys and values, 13 us of that;
// 116 us when a border of 2^-19 of max|y| sent one row in 250 back, which a factor that
// cancels does not keep to.  Both teams' chains (rows, rotation, terms, product, codes)
// are waiting most of the time, and 24 warps at 80 registers (head_dim 128: with 80 bytes
// of spills) are all that an SM holds.
#include <mutex>

#include "kq_common.cuh"
#include "kq_internal.h"
#include "kq_tc05_ptx.cuh"
#include "kq_wait.cuh"

namespace kq {
namespace {

using namespace tc;

constexpr int A_THREADS = 768;     // per team eight warps that make terms and four that take rows
// What a row's fp32 values may be off by, from the two-norms of the rotated row and of the factor's largest column.
// A step of 16 products cuts them and the sum so far at 2^-25 of the largest (2^-25 is kept, 2^-26 lost, as measured),
// and the new sum is truncated to fp32: 16 times 2^-25 and 2^-23 of at most |x||P_j| in each of D / 16 steps, 5/8 D
// 2^-24; the smaller terms of keys and the rotation add less than 6 2^-24.  0.7 D covers both and the norms' own
// rounding.  The small parts stand for squares and sums that underflow.
template <int D>
__device__ __forceinline__ float error_of(float squares, float column) {
    return 0.7f * D * 0x1p-24f * (sqrtf(squares) + 0x1p-59f) * (column + 0x1p-59f) + 0x1p-118f;
}
enum : unsigned { kSiteKvAppendWait = 524288u };

template <int D>
struct ACfg {
    static constexpr int ROW = D * 2 + 16;            // a row's place in shared memory, padded
    static constexpr int STAGE = 128 * ROW;
    static constexpr int OFF_X = D * D * 2;           // after the factor
    // an undecided row: its fp32 values, the row itself, the table's row; padded, so that four rows lie in different banks
    static constexpr int ROW_X = D * 4, ROW_CS = ROW_X + D * 2, ROW_PLACE = ROW_CS + D * 4 + 32;
    static constexpr int OWN = 4 * ROW_PLACE > 4096 ? 4 * ROW_PLACE : 4096;
    static constexpr int OFF_Y = OFF_X + 4 * STAGE;   // OWN bytes for each warp that takes rows
    static constexpr int OFF_NORM = OFF_Y + 8 * OWN;  // [pair][turn][half of the pieces][row]: sums of squares
    static constexpr int OFF_COL = OFF_NORM + 2 * 2 * 2 * 128 * 4;  // [warp][column]: the same of the factor's rows
    static constexpr int OFF_BAR = OFF_COL + (A_THREADS / 32) * D * 4;
    static constexpr int OFF_MISC = OFF_BAR + 8 * 6;  // of each pair: products done, rows and their norms ready, rows taken
    static constexpr int SMEM = OFF_MISC + 16 + 1024;
    static_assert(SMEM <= 227 * 1024, "shared memory");
};

// 16 bytes to shared memory, of which the first `size` come from `src` and the rest are zeros.
__device__ __forceinline__ void cp_async16(uint32_t dst, uint64_t src, uint32_t size) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(size) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// round_half_even(y * inv) as an int for |y * inv| < 2^22 (alpha >= 2^-19): the low mantissa bits
// after adding 1.5 * 2^23; `off` keeps the largest distance to the rounded value.
__device__ __forceinline__ int round_off(uint32_t ybits, float inv, float &off) {
    const float y = __uint_as_float(ybits), b = fmaf(y, inv, 12582912.0f);
    off = fmaxf(off, fabsf(fmaf(y, inv, -(b - 12582912.0f))));
    return int(__float_as_uint(b)) - 0x4B400000;
}

__device__ __forceinline__ void unpack8(const uint4 &u, float (&v)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

// ---- rows that fp32 does not decide, in fp64 ----
// Shared memory by its 32-bit address, as these are out of line (and all that they read there is written before the
// call): a row, its row of the table, the factor.
struct ExactRow {
    uint32_t x, cs, factor;
    int rope_dim;
    bool inter;
};
__device__ __forceinline__ float shared_f32(uint32_t at) {
    float v;
    asm("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at));
    return v;
}
__device__ __forceinline__ double shared_bf16(uint32_t at) {
    uint16_t w;
    asm("ld.shared.u16 %0, [%1];" : "=h"(w) : "r"(at));
    return double(bf16_bits_to_float(w));
}
// Where the factor's element (k, n) lies: (row_place(k) ^ column n's swizzle) + column n's place.
__device__ __forceinline__ uint32_t row_place(int k) { return uint32_t(k * 128 + ((k & 7) << 4)); }
template <int D>
struct Column {
    uint32_t at, swizzle;
    __device__ __forceinline__ Column(uint32_t factor, int n)
        : at(factor + uint32_t((n >> 6) * D * 128 + 2 * (n & 7))), swizzle(uint32_t(((n & 63) >> 3) << 4)) {}
    __device__ __forceinline__ double operator()(uint32_t row) const { return shared_bf16(at + (row ^ swizzle)); }
};
__device__ __forceinline__ int exact_code(double y, double s) {
    return s > 0.0 ? int(rint(fmin(fmax(y / s, -8.0), 7.0))) : 0;
}
// The elements of the rotated row from the sub-th of each eight pairs, and of each eight that do not turn, on: calls
// use(value, place of its row of the factor), for eight lanes from 0 on as often.  Their rows lie in different banks.
template <int D, typename F>
__device__ __forceinline__ void exact_elements(const ExactRow &a, int sub, F use) {
    const int half = a.rope_dim >> 1, i0 = a.inter ? 2 * sub : sub, i1 = a.inter ? i0 + 1 : sub + half;
    const int step = a.inter ? 16 : 8;  // a multiple of eight rows: row_place goes on evenly
    uint32_t x0 = a.x + 2 * i0, x1 = a.x + 2 * i1, c = a.cs + 4 * sub, k0 = row_place(i0), k1 = row_place(i1);
#pragma unroll 1
    for (int p = 0; p < half; p += 8) {
        const double u = shared_bf16(x0), w = shared_bf16(x1), cc = double(shared_f32(c)), ss = double(shared_f32(c + 4 * half));
        use(fma(u, cc, -(w * ss)), k0);
        use(fma(w, cc, u * ss), k1);
        x0 += 2 * step, x1 += 2 * step, c += 32;
        k0 += 128 * step, k1 += 128 * step;
    }
    uint32_t x = a.x + 2 * (a.rope_dim + sub), k = row_place(a.rope_dim + sub);
#pragma unroll 2
    for (int i = a.rope_dim; i < D; i += 8) {
        use(shared_bf16(x), k);
        x += 16, k += 1024;
    }
}

// Four rows (`there`: this lane's is one) of which fp32 leaves few codes open, eight lanes a row.  `y32`: its fp32 values
// in shared memory, off by at most `err`, the largest `m`; the codes that they gave are stored already.  A value y_n lies
// over the border b, b + 1/2 whole, where 7 y_n - b alpha |y_t| > 0, y_t the largest: one sum over the row.  Returns
// false where the largest is not sure.
template <int D>
__device__ __noinline__ bool border_rows(ExactRow a, uint8_t *codes, float alpha, bool there, uint32_t y32, float m,
                                         float err, float inv, float limit) {
    auto value = [&](int n) { return shared_f32(y32 + 4 * n); };
    const int sub = threadIdx.x & 7;
    uint32_t may = 0, near = 0;  // of this lane's columns, sub + 8 i
    const float large = m - 2.5f * err, past = __fdividef(8.0f, inv);
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
        const float y = value(sub + 8 * i);
        float off = 0.0f;
        round_off(__float_as_uint(y), inv, off);
        if (fabsf(y) >= large) may |= 1u << i;
        if (off > limit && fabsf(y) < past) near |= 1u << i;
    }
    constexpr int NONE = 1 << 20;
    auto next = [&](uint32_t &mask) -> int {  // the row's next column
        const int n = mask ? sub + 8 * (__ffs(mask) - 1) : NONE;
        int least = n;
#pragma unroll
        for (int o = 4; o; o >>= 1) least = min(least, __shfl_xor_sync(0xffffffffu, least, o));
        if (n == least) mask &= mask - 1;
        return least;
    };
    if (!there) may = near = 0;
    // (indexes are columns of the row whatever there is: a load may be done ahead of the test that it hangs on)
    const int first = next(may), top = first & (D - 1);
    const bool sure = next(may) == NONE;
    if (!sure) near = 0;
    for (;;) {
        const int found = next(near), n = found & (D - 1);
        if (!__any_sync(0xffffffffu, found != NONE)) break;
        double d = 0.0;
        const float border = floorf(value(n) * inv) + 0.5f;
        if (found != NONE) {
            const double share = -double(copysignf(border, value(top) * border)) * double(alpha);
            const Column<D> largest(a.factor, top), column(a.factor, n);
            exact_elements<D>(a, sub, [&](double v, uint32_t k) { d = fma(v, fma(share, largest(k), 7.0 * column(k)), d); });
        }
#pragma unroll
        for (int o = 4; o; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
        if (sub == 0 && found != NONE) {
            const int under = int(border - 0.5f), code = under + (d > 0.0 || (d == 0.0 && (under & 1)));
            float off = 0.0f;
            if (code != round_off(__float_as_uint(value(n)), inv, off)) {
                const int shift = 4 * (n & 1), c = min(max(code, -8), 7);
                codes[n >> 1] = uint8_t((codes[n >> 1] & ~(15 << shift)) | (c & 15) << shift);
            }
        }
    }
    __syncwarp();
    return sure;
}

// A row of which every column may matter: the products cancel, or the scale is very small.
template <int D>
__device__ __noinline__ void whole_row(ExactRow a, uint8_t *codes, float *scale, float alpha) {
    constexpr int N = D / 32;  // columns of a lane, side by side
    const int lane = threadIdx.x & 31;
    double y[N] = {}, top = 0.0;
    exact_elements<D>(a, lane & 7, [&](double v, uint32_t k) {
#pragma unroll 2
        for (int l = 0; l < 8; ++l) {
            const double x = __shfl_sync(0xffffffffu, v, l);
            const uint32_t row = __shfl_sync(0xffffffffu, k, l);
#pragma unroll
            for (int e = 0; e < N; ++e) y[e] = fma(x, Column<D>(a.factor, N * lane + e)(row), y[e]);
        }
    });
#pragma unroll
    for (int e = 0; e < N; ++e) top = fmax(top, fabs(y[e]));
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmax(top, __shfl_xor_sync(0xffffffffu, top, o));
    const double s = double(alpha) * top / 7.0;
    uint32_t word = 0;
#pragma unroll
    for (int e = 0; e < N; ++e) word |= uint32_t(exact_code(y[e], s) & 15) << (4 * e);
    __syncwarp();
    if constexpr (N == 4) reinterpret_cast<uint16_t *>(codes)[lane] = uint16_t(word);
    else codes[lane] = uint8_t(word);
    if (lane == 0) *scale = float(s);
    __syncwarp();
}

template <typename T>
__device__ __forceinline__ T *from_lane(T *p, int lane) {
    return reinterpret_cast<T *>(__shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(p), lane));
}
__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ void unpack2(uint64_t d, float &a, float &b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(d));
}
__device__ __forceinline__ uint64_t f32x2_fma(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

// Four consecutive pairs of fp32 values -> words of their leading bf16 terms (truncated), the
// values less those terms left behind; exact.
__device__ __forceinline__ void take_term(float (&v)[8], uint32_t (&w)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t a = __float_as_uint(v[2 * i]), b = __float_as_uint(v[2 * i + 1]);
        w[i] = __byte_perm(a, b, 0x7632);
        unpack2(f32x2_sub(pack2(v[2 * i], v[2 * i + 1]),
                          pack2(__uint_as_float(a & 0xffff0000u), __uint_as_float(b & 0xffff0000u))),
                v[2 * i], v[2 * i + 1]);
    }
}
// Squares of eight bf16 values, added to eight sums.
__device__ __forceinline__ void add_squares(const uint4 &u, uint64_t (&s)[4]) {
    float v[8];
    unpack8(u, v);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint64_t p = pack2(v[2 * e], v[2 * e + 1]);
        s[e] = f32x2_fma(p, p, s[e]);
    }
}

// Every second eight (`which`: the even or the odd ones) of the row's values, rotated, or pair
// of eights that turn together: calls put(first element, values).
template <int D, typename F>
__device__ __forceinline__ void rotated_row(const unsigned char *xrow, const float *cs, int rope_dim, bool inter,
                                            int which, F put) {
    const uint4 *x = reinterpret_cast<const uint4 *>(xrow);
    const int half = rope_dim >> 1;
    if (inter) {
        auto eight = [&](int i) {
            float v[8];
            unpack8(x[i >> 3], v);
            const float4 c = __ldg(reinterpret_cast<const float4 *>(cs + (i >> 1)));
            const float4 s = __ldg(reinterpret_cast<const float4 *>(cs + half + (i >> 1)));
            const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float a = v[2 * e], b = v[2 * e + 1];
                v[2 * e] = fmaf(a, cc[e], -(b * ss[e]));
                v[2 * e + 1] = fmaf(b, cc[e], a * ss[e]);
            }
            put(i, v);
        };
        if (rope_dim == D) {  // the usual case, unrolled so that the table's loads run ahead
#pragma unroll
            for (int i = 0; i < D; i += 16) eight(i + 8 * which);
            return;
        }
        for (int i = 8 * which; i < rope_dim; i += 16) eight(i);
    } else {
        auto eight = [&](int i) {
            float a[8], b[8];
            unpack8(x[i >> 3], a);
            unpack8(x[(i + half) >> 3], b);
            float c[8], s[8];
#pragma unroll
            for (int e = 0; e < 8; e += 4) {
                const float4 u = __ldg(reinterpret_cast<const float4 *>(cs + i + e));
                const float4 w = __ldg(reinterpret_cast<const float4 *>(cs + half + i + e));
                c[e] = u.x, c[e + 1] = u.y, c[e + 2] = u.z, c[e + 3] = u.w;
                s[e] = w.x, s[e + 1] = w.y, s[e + 2] = w.z, s[e + 3] = w.w;
            }
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                const uint64_t p = pack2(a[e], a[e + 1]), q = pack2(b[e], b[e + 1]);
                const uint64_t cc = pack2(c[e], c[e + 1]), ss = pack2(s[e], s[e + 1]);
                const uint64_t minus = pack2(-b[e], -b[e + 1]);
                unpack2(f32x2_fma(p, cc, f32x2_mul(minus, ss)), a[e], a[e + 1]);
                unpack2(f32x2_fma(q, cc, f32x2_mul(p, ss)), b[e], b[e + 1]);
            }
            put(i, a);
            put(i + half, b);
        };
        if (rope_dim == D) {
#pragma unroll
            for (int i = 0; i < D / 2; i += 16) eight(i + 8 * which);
            return;
        }
        for (int i = 8 * which; i < half; i += 16) eight(i);
    }
    for (int i = rope_dim + 8 * which; i < D; i += 16) {
        float v[8];
        unpack8(x[i >> 3], v);
        put(i, v);
    }
}

template <int D>
__global__ void __launch_bounds__(A_THREADS, 1)
    kq_kv_append_kernel(const __grid_constant__ KvAppendArgs a, int blocks_q, int blocks_k, int blocks_v) {
    using C = ACfg<D>;
    extern __shared__ __align__(1024) unsigned char a_raw[];
    const uint32_t raw_addr = smem_u32(a_raw), sbase = (raw_addr + 1023u) & ~1023u;
    unsigned char *smem = a_raw + (sbase - raw_addr);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int pair = warp < 16 ? warp >> 3 : (warp - 16) >> 2, r = tid & 127;  // the team; this thread's row of a tile
    auto bar = [&](int i) -> uint32_t { return sbase + uint32_t(C::OFF_BAR + 8 * i); };
    const uint32_t done = bar(pair), ready = bar(2 + pair), taken = bar(4 + pair);
    volatile int *s_abort = reinterpret_cast<volatile int *>(smem + C::OFF_MISC + 4);
    if (tid == 0) {
        for (int i = 0; i < 4; ++i) mbar_init(bar(i), i < 2 ? 1 : 2);
        mbar_init(bar(4), 4);
        mbar_init(bar(5), 4);
        *s_abort = 0;
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(sbase + C::OFF_MISC, 512);
        tmem_relinquish();
    }
    const int H = a.q_heads, Hk = a.c.heads, psh = a.c.page_shift;
    // the block's kind, and its tiles: every blocks_*-th of the kind; the teams take turns
    const int bid = blockIdx.x, kind = bid < blocks_q ? 0 : bid < blocks_q + blocks_k ? 1 : 2;
    const int64_t rows = a.T * (kind == 0 ? H : Hk), tiles = (rows + 127) / 128;
    const int64_t step = kind == 0 ? blocks_q : kind == 1 ? blocks_k : blocks_v;
    const uint32_t heads = kind == 0 ? H : Hk;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem0 = *reinterpret_cast<volatile uint32_t *>(smem + C::OFF_MISC);
    const uint32_t tmem = tmem0 + uint32_t(256 * pair), lanes = uint32_t(32 * (warp & 3)) << 16;
    griddep_wait();
    griddep_launch_dependents();

    // A wait that gives up raises the block's abort flag: no product is issued after it and no row stored.  The warps
    // that make terms go through their tiles all the same, as they meet at barriers, but wait for nothing more.
    auto wait = [&](uint32_t b, uint32_t parity, bool ignore_abort) -> bool {
        // looks 60 ns apart at first, which leave the issue slots to the other warps
        bool ok = mbar_try_wait(b, parity);
        for (int i = 0; i < 200 && !ok && !*s_abort; ++i) {
            __nanosleep(60);
            ok = mbar_try_wait(b, parity);
        }
        if (!ok) ok = wait_bounded_err(b, parity, s_abort, kSiteKvAppendWait, kWaitLimitNs, ignore_abort, a.err);
        return __all_sync(0xffffffffu, ok);
    };
    // This thread's row of a tile: token and head; false past the last row.
    auto row_of = [&](int64_t tile, int &t, int &h) -> bool {
        const int64_t row = tile * 128 + r;
        t = int(uint32_t(row) / heads);
        h = int(uint32_t(row) - uint32_t(t) * heads);
        return row < rows;
    };
    const uint16_t *const rows_from = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
    const int64_t stride = kind == 0 ? a.q_stride : kind == 1 ? a.k_stride : a.v_stride;
    auto source = [&](int t, int h) { return rows_from + int64_t(t) * stride + int64_t(h) * D; };
    {  // the factor
        const uint16_t *P = kind == 0 ? a.Pq : kind == 1 ? a.Pk : a.Pv;
        uint64_t col[4] = {0, 0, 0, 0};  // squares of the eight columns that this thread has
        static_assert(A_THREADS % (D / 8) == 0, "a thread's columns");
#pragma unroll
        for (int u = tid; u < D * D / 8; u += A_THREADS) {
            const int k = u / (D / 8), n = 8 * (u % (D / 8));
            const uint4 p = __ldg(reinterpret_cast<const uint4 *>(P + k * D + n));
            *reinterpret_cast<uint4 *>(smem + (n >> 6) * D * 128 + k * 128 + ((((n & 63) >> 3) ^ (k & 7)) << 4)) = p;
            add_squares(p, col);
        }
        if (kind != 0) {
            float c[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) unpack2(col[e], c[2 * e], c[2 * e + 1]);
#pragma unroll
            for (int e = 0; e < 8; ++e)
#pragma unroll
                for (int o = D / 8; o < 32; o <<= 1) c[e] += __shfl_xor_sync(0xffffffffu, c[e], o);
            if (lane < D / 8) {
                float4 *to = reinterpret_cast<float4 *>(smem + C::OFF_COL + (warp * D + 8 * lane) * 4);
                to[0] = make_float4(c[0], c[1], c[2], c[3]);
                to[1] = make_float4(c[4], c[5], c[6], c[7]);
            }
        }
        fence_proxy_async_smem();
    }

    int64_t tile = (bid - (kind == 0 ? 0 : kind == 1 ? blocks_q : blocks_q + blocks_k)) + pair * step;
    uint32_t turns = 0;
    if (warp < 16) {
        // ---------------- rows into terms, terms times the factor ----------------
        const int which = (warp >> 2) & 1;  // of the two warps of a TMEM quarter
        unsigned char *const place0 = smem + C::OFF_X + 2 * pair * C::STAGE + r * C::ROW;
        // The quarter's 32 rows of a tile, half of their pieces: a step takes PER rows, a lane 16 bytes.
        constexpr int PIECES = D / 16, PER = 32 / PIECES;
        const int sub = lane / PIECES, piece = lane % PIECES + which * PIECES;
        // This thread's row of a tile (null past the last), and its position: both an iteration ahead of their use.
        auto look = [&](int64_t tile, const uint16_t *&x, int &pos) {
            x = nullptr;
            pos = 0;
            int t, h;
            if (tile < tiles && row_of(tile, t, h)) {
                x = source(t, h);
                if (kind < 2 && a.rope_dim) pos = a.positions[t];
            }
        };
        auto fetch = [&](const uint16_t *x, int stage) {
            const uint32_t dst =
                smem_u32(place0 + stage * C::STAGE - lane * C::ROW) + uint32_t(sub * C::ROW + 16 * piece);
#pragma unroll
            for (int i = 0; i < 32 / PER; ++i) {
                const uint64_t src = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(x), i * PER + sub);
                cp_async16(dst + uint32_t(i * PER * C::ROW), src ? src + 16 * piece : reinterpret_cast<uint64_t>(a.Pk),
                           src ? 16u : 0u);  // rows past the last are zeros
            }
            cp_async_commit();
        };
        const uint16_t *x2;
        int pos0, pos1, pos2;
        look(tile, x2, pos0);
        fetch(x2, 0);
        look(tile + 2 * step, x2, pos1);
        fetch(x2, 1);
        __syncthreads();  // the factor
        const uint32_t ta = tmem + lanes;
        constexpr uint32_t idesc = idesc_bf16_f32_bn(128, D);
        uint32_t products = 0;
        // Rows (+)= the terms times the factor, by one thread of the warpgroup.
        auto multiply = [&](int terms, bool accumulate, bool last) {
            tmem_wait_st();
            tc_fence_before();
            named_barrier_sync(1 + pair, 256);
            if ((warp & 7) == 0) {
                const bool ok = accumulate || wait(taken, (turns & 1u) ^ 1u, false);  // the last tile's rows
                tc_fence_after();
                if (elect_one() && ok && !*s_abort) {
                    // the smallest term first: the sum is truncated at every addition
                    for (int term = terms - 1; term >= 0; --term)
#pragma unroll
                        for (int k = 0; k < D / 16; ++k)
                            mma_ts(tmem + 128, tmem + uint32_t(64 * term + 8 * k),
                                   sdesc_nmajor_sw128(sbase + uint32_t(2048 * k), D * 128), idesc,
                                   accumulate || term + 1 < terms || k);
                    tc_commit(done);
                    if (last) {
                        tc_commit(ready);
                        mbar_arrive(ready);  // the rows' norms, written before the barrier
                    }
                }
                __syncwarp();
            }
            ++products;
        };
        // the terms' columns are free once the last product is done
        // (where they are not in time the abort flag is up, and the next product is not issued)
        auto multiplied = [&](bool ignore_abort) {
            if (products) (void)wait(done, (products - 1) & 1u, ignore_abort);
            tc_fence_after();
        };
        const bool inter = a.rope_interleaved != 0;
        for (; tile < tiles; tile += 2 * step, ++turns) {
            const int stage = int(turns & 1u);
            unsigned char *x = place0 + stage * C::STAGE;
            auto one_term = [&] {  // what lies in the row's place
#pragma unroll 1
                for (int i = 0; i < D / 16; ++i) {
                    const uint4 u = reinterpret_cast<const uint4 *>(x)[2 * i + which];
                    tmem_st_32x32b_x4(ta + uint32_t(4 * (2 * i + which)), u.x, u.y, u.z, u.w);
                }
            };
            const float *cs = a.rope + int64_t(uint32_t(pos0) < uint32_t(a.rope_positions) ? pos0 : 0) * a.rope_dim;
            look(tile + 4 * step, x2, pos2);
            cp_async_wait<1>();
            named_barrier_sync(3 + pair, 256);  // the other warp's pieces
            multiplied(false);
            float *norm = reinterpret_cast<float *>(smem + C::OFF_NORM) + ((2 * pair + stage) * 2 + which) * 128 + r;
            if (kind == 2) {
                uint64_t sq[4] = {0, 0, 0, 0};
#pragma unroll 1
                for (int i = 0; i < D / 16; ++i) {
                    const uint4 u = reinterpret_cast<const uint4 *>(x)[2 * i + which];
                    tmem_st_32x32b_x4(ta + uint32_t(4 * (2 * i + which)), u.x, u.y, u.z, u.w);
                    add_squares(u, sq);
                }
                float s[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) unpack2(sq[e], s[2 * e], s[2 * e + 1]);
                *norm = ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
                multiply(1, false, true);
            } else {
                uint64_t sq = 0;
                // queries: both terms; keys: the second and third, and then the first, which waits in the row's place
                rotated_row<D>(x, cs, a.rope_dim, inter, which, [&](int i, float (&v)[8]) {
                    uint32_t w[4];
                    if (kind == 1)
#pragma unroll
                        for (int e = 0; e < 8; e += 2) {
                            const uint64_t p = pack2(v[e], v[e + 1]);
                            sq = f32x2_fma(p, p, sq);
                        }
                    take_term(v, w);
                    if (kind == 1) {
                        *reinterpret_cast<uint4 *>(x + 2 * i) = make_uint4(w[0], w[1], w[2], w[3]);
                        take_term(v, w);
                    }
                    tmem_st_32x32b_x4(ta + uint32_t(i >> 1), w[0], w[1], w[2], w[3]);
                    tmem_st_32x32b_x4(ta + 64 + uint32_t(i >> 1), pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                      pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
                });
                if (kind == 1) {
                    float even, odd;
                    unpack2(sq, even, odd);
                    *norm = even + odd;
                }
                multiply(2, false, kind == 0);
                if (kind == 1) {
                    multiplied(false);
                    one_term();
                    multiply(1, true, true);
                }
            }
            fetch(x2, stage);  // all warps have read the tile's rows: they were at multiply's barrier
            pos0 = pos1;
            pos1 = pos2;
        }
        cp_async_wait<0>();
        // the products in flight end before their TMEM is given back
        multiplied(true);
    } else {
        // ---------------- rows out ----------------
        const uint32_t td = tmem + lanes + 128;
        unsigned char *const own = smem + C::OFF_Y + (warp - 16) * C::OWN;
        __syncthreads();  // the factor
        float column = 0.0f;  // the two-norm of its largest column
        if (kind != 0) {
            constexpr int N = D / 32;  // columns of a lane
            float c[N] = {};
            for (int w = 0; w < A_THREADS / 32; ++w)
#pragma unroll
                for (int e = 0; e < N; ++e)
                    c[e] += reinterpret_cast<const float *>(smem + C::OFF_COL)[w * D + N * lane + e];
#pragma unroll
            for (int e = 0; e < N; ++e) column = fmaxf(column, c[e]);
            column = sqrtf(__uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(column))));
        }
        // This thread's row of a tile, its slot and position, loaded a tile ahead of their use.
        struct Row {
            int t, h, pos;
            bool real;
            int64_t slot;
        };
        auto look = [&](int64_t tile) {
            Row w;
            w.pos = 0;
            w.slot = -1;
            w.real = row_of(tile, w.t, w.h) && tile < tiles;
            if (w.real) {
                if (kind != 0) w.slot = a.slots[w.t];
                if (a.rope_dim) w.pos = a.positions[w.t];
            }
            return w;
        };
        Row next = look(tile);
        {
            for (; tile < tiles; tile += 2 * step, ++turns) {
                const Row now = next;
                next = look(tile + 2 * step);
                const int t = now.t, h = now.h;
                const bool real = now.real;
                const bool pos_ok = !a.rope_dim || uint32_t(now.pos) < uint32_t(a.rope_positions);
                int64_t slot = now.slot;
                const float *cs = a.rope + int64_t(pos_ok ? now.pos : 0) * a.rope_dim;
                if (!pos_ok || (slot >= a.c.pages << psh)) {
                    atomicOr(a.err, kSiteKvAppend);
                    slot = -1;
                }
                if (!wait(ready, turns & 1u, false) || __any_sync(0xffffffffu, *s_abort != 0)) break;
                tc_fence_after();
                if (kind == 0) {
                    // ---- queries: bf16, 64 columns at a time through the warp's 4 KB (32 rows of 128 bytes,
                    // their pieces exchanged by row), so that whole rows are stored; q_out is dense ----
                    const int64_t row0 = tile * 128 + 32 * (warp & 3);
#pragma unroll
                    for (int c = 0; c < D / 64; ++c) {
#pragma unroll
                        for (int b = 0; b < 2; ++b) {
                            uint32_t v[32];
                            tmem_ld_32x32b_x32(td + uint32_t(64 * c + 32 * b), v);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                uint32_t w[4];
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    w[k] = pos_ok ? pack_bf16x2(__uint_as_float(v[8 * e + 2 * k]),
                                                                __uint_as_float(v[8 * e + 2 * k + 1]))
                                                  : 0u;
                                *reinterpret_cast<uint4 *>(own + 128 * lane + (((4 * b + e) ^ (lane & 7)) << 4)) =
                                    make_uint4(w[0], w[1], w[2], w[3]);
                            }
                        }
                        if (c == D / 64 - 1) tc_fence_before();
                        __syncwarp();
                        if (c == D / 64 - 1 && lane == 0) mbar_arrive(taken);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int row = 4 * i + (lane >> 3);
                            if (row0 + row < rows)
                                *reinterpret_cast<uint4 *>(a.q_out + (row0 + row) * D + 64 * c + 8 * (lane & 7)) =
                                    *reinterpret_cast<const uint4 *>(own + 128 * row + (((lane ^ row) & 7) << 4));
                        }
                        __syncwarp();
                    }
                } else {
                    // ---- a row of the cache ----
                    float m = 0.0f;
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t v[32];
                        tmem_ld_32x32b_x32(td + uint32_t(32 * c), v);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; e += 2)
                            m = fmax3(m, fabsf(__uint_as_float(v[e])), fabsf(__uint_as_float(v[e + 1])));
                    }
                    const float alpha = kind == 1 ? a.alpha_k : a.alpha_v;
                    const float sc = __fdiv_rn(alpha * m, 7.0f);
                    const float inv = sc > 0.0f ? fminf(__frcp_rn(sc), 3.0e38f) : 0.0f;
                    const bool store = real && slot >= 0 && pos_ok;
                    const int64_t row =
                        store ? (((slot >> psh) * Hk + h) << psh) + (slot & ((int64_t(1) << psh) - 1)) : 0;
                    uint8_t *codes = (kind == 1 ? a.c.k_codes : a.c.v_codes) + row * (D / 2);
                    float *scale = (kind == 1 ? a.c.k_scale : a.c.v_scale) + row;
                    float off = 0.0f;
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t v[32], w[4];
                        tmem_ld_32x32b_x32(td + uint32_t(32 * c), v);
                        tmem_wait_ld();
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const uint32_t *y = v + 8 * k;
                            uint32_t p = 0;
#pragma unroll
                            for (int e = 6; e >= 0; e -= 2)
                                p = pack_s4x2(round_off(y[e + 1], inv, off), round_off(y[e], inv, off), p);
                            w[k] = p;
                        }
                        if (store) reinterpret_cast<uint4 *>(codes)[c] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                    if (store) *scale = sc;
                    // ---- rows with a value too near a border for fp32, again in fp64 ----
                    // (scales that leave fp32's normal range, or would keep under 12 bits, are among them; a NaN or
                    // an infinity is not).  y is off by err, and so is m: y / s by 7 / alpha + |y / s| times err / m,
                    // and by three roundings; past 8 no border matters.
                    const float *norms = reinterpret_cast<const float *>(smem + C::OFF_NORM) +
                                         (2 * pair + int(turns & 1u)) * 256 + r;
                    const float squares = norms[0] + norms[128], err = error_of<D>(squares, column);
                    const float limit = 0.5f - 0x1p-19f - (7.0f / alpha + fminf(7.0f / alpha, 8.5f)) * __fdividef(err, m);
                    const bool open = store && m < 3.0e38f && (m > 0.0f ? off > limit || sc < 1e-30f || err > m * 0x1p-12f
                                                                         : squares > 0.0f);
                    const bool few = m > 0.0f && sc >= 1e-30f && err <= m * 0x1p-12f && limit > 0.25f;
                    uint32_t again = __ballot_sync(0xffffffffu, open && few);
                    uint32_t wholes = __ballot_sync(0xffffffffu, open && !few);
                    const uint16_t *x = source(t, h);
                    const int rope_dim = kind == 1 ? a.rope_dim : 0;
                    // Lane group `at` of 8 or 32 lanes brings the row of lane `src`, and the table's.
                    auto bring = [&](int at, int src, int from, int lanes) {
                        const uint32_t to = smem_u32(own) + uint32_t(at * C::ROW_PLACE);
                        const uint64_t px = reinterpret_cast<uint64_t>(from_lane(x, src));
                        const uint64_t pc = reinterpret_cast<uint64_t>(from_lane(cs, src));
                        for (int u = from; u < D / 8; u += lanes) cp_async16(to + C::ROW_X + 16 * u, px + 16 * u, 16u);
                        for (int u = from; u < rope_dim / 4; u += lanes) cp_async16(to + C::ROW_CS + 16 * u, pc + 16 * u, 16u);
                        cp_async_commit();
                        return ExactRow{to + C::ROW_X, to + C::ROW_CS, sbase, rope_dim, a.rope_interleaved != 0};
                    };
                    while (again) {  // four at a time: a lane's row is the (lane / 8)th of them
                        const int rank = __popc(again & ((1u << lane) - 1)), rows4 = min(4, __popc(again));
                        const bool mine = (again >> lane & 1u) && rank < 4;
                        int src = 0;
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (k < rows4) {
                                if (k == 0 || k == lane >> 3) src = __ffs(again) - 1;
                                again &= again - 1;
                            }
                        const ExactRow row = bring(lane >> 3, src, lane & 7, 8);
#pragma unroll
                        for (int c = 0; c < D / 32; ++c) {
                            uint32_t v[32];
                            tmem_ld_32x32b_x32(td + uint32_t(32 * c), v);
                            tmem_wait_ld();
                            if (mine)
#pragma unroll
                                for (int e = 0; e < 8; ++e)
                                    *reinterpret_cast<uint4 *>(own + rank * C::ROW_PLACE + 128 * c + 16 * e) =
                                        make_uint4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
                        }
                        cp_async_wait<0>();
                        __syncwarp();
                        const bool sure =
                            border_rows<D>(row, from_lane(codes, src), alpha, lane >> 3 < rows4,
                                           row.x - C::ROW_X,
                                           __shfl_sync(0xffffffffu, m, src), __shfl_sync(0xffffffffu, err, src),
                                           __shfl_sync(0xffffffffu, inv, src), __shfl_sync(0xffffffffu, limit, src));
                        __syncwarp();
                        wholes |= __reduce_or_sync(0xffffffffu, lane >> 3 < rows4 && !sure ? 1u << src : 0u);
                    }
                    for (; wholes; wholes &= wholes - 1) {
                        const int src = __ffs(wholes) - 1;
                        const ExactRow row = bring(0, src, lane, 32);
                        cp_async_wait<0>();
                        __syncwarp();
                        whole_row<D>(row, from_lane(codes, src), from_lane(scale, src), alpha);
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(taken);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem0, 512);
    }
}

// Rows back out: a thread turns 16 codes (8 bytes) into 32 bytes of bf16.
template <int D>
__global__ void __launch_bounds__(256)
    kq_kv_gather_kernel(const __grid_constant__ KvCache c, const int64_t *__restrict__ slots,
                        uint16_t *__restrict__ k_out, uint16_t *__restrict__ v_out, int64_t T, unsigned int *err) {
    constexpr int PER = D / 16;  // threads per row
    griddep_wait();
    griddep_launch_dependents();
    const int64_t n = T * c.heads * PER, psize = int64_t(1) << c.page_shift;
    const bool val = blockIdx.y != 0;
    const uint8_t *codes = val ? c.v_codes : c.k_codes;
    const float *scales = val ? c.v_scale : c.k_scale;
    uint16_t *out = val ? v_out : k_out;
    for (int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; i < n; i += int64_t(gridDim.x) * blockDim.x) {
        const int64_t r = i / PER, t = r / c.heads;
        const int part = int(i % PER), h = int(r % c.heads);
        const int64_t slot = slots[t];
        uint32_t w[2] = {0u, 0u};
        float s = 0.0f;
        if (slot >= 0 && slot < c.pages * psize) {
            const int64_t row = ((slot >> c.page_shift) * c.heads + h) * psize + (slot & (psize - 1));
            const uint2 v = *reinterpret_cast<const uint2 *>(codes + row * (D / 2) + 8 * part);
            w[0] = v.x;
            w[1] = v.y;
            s = scales[row];
        } else if (slot >= 0 && part == 0 && h == 0) {
            atomicOr(err, kSiteKvAppend);
        }
        uint32_t o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t b = w[e >> 2] >> (8 * (e & 3));
            const int lo = int(b << 28) >> 28, hi = int(b << 24) >> 28;
            o[e] = pack_bf16x2(float(lo) * s, float(hi) * s);
        }
        uint4 *dst = reinterpret_cast<uint4 *>(out + r * D + 16 * part);
        dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
        dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
}

}  // namespace

template <int D>
static cudaError_t launch_append_inst(const KvAppendArgs &a, int num_sms, int device, cudaStream_t stream) {
    using C = ACfg<D>;
    auto kern = kq_kv_append_kernel<D>;
    static std::once_flag once[64];
    static cudaError_t attr_err[64];
    if (device < 0 || device >= 64) return cudaErrorInvalidDevice;
    std::call_once(once[device], [&] {
        attr_err[device] = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    });
    if (attr_err[device] != cudaSuccess) return attr_err[device];
    // Blocks for each kind: one more at a time to the kind whose blocks have the most to do.  A tile of keys
    // takes about 2.1 times, one of values 1.7 times what one of queries does (1.8 and 1.4 at head_dim 64), with the
    // rows that are computed again, and the rotation more the fewer heads there are: a warp's rows then read as many
    // rows of the table.  (16 heads of each kind, 8192 tokens: 125 us at 2.1 and 1.7, 137 at 1.9 and 1.35; at
    // head_dim 64 61 and 56; 65536 tokens of 8 query heads on one key head: 149 us without the terms for the rotation,
    // 112 with them, before rows were computed again as often.)
    const int64_t tiles[3] = {(a.T * a.q_heads + 127) / 128, (a.T * a.c.heads + 127) / 128,
                              (a.T * a.c.heads + 127) / 128};
    const double turn = double(a.rope_dim) / D;
    const double cost[3] = {1.0 + (a.q_heads ? 0.5 * turn / a.q_heads : 0.0),
                            (D == 128 ? 2.1 : 1.8) + 1.5 * turn / a.c.heads, D == 128 ? 1.7 : 1.4};
    int blocks[3] = {tiles[0] > 0, 1, 1};
    for (int n = blocks[0] + 2; n < num_sms; ++n) {
        int most = -1;
        double load = 0.0;
        for (int k = 0; k < 3; ++k) {
            if (blocks[k] >= tiles[k]) continue;
            const double l = cost[k] * double((tiles[k] + blocks[k] - 1) / blocks[k]);
            if (l > load) most = k, load = l;
        }
        if (most < 0) break;
        ++blocks[most];
    }
    return launch_overlapped(kern, unsigned(blocks[0] + blocks[1] + blocks[2]), A_THREADS, C::SMEM, stream, a, blocks[0],
                             blocks[1], blocks[2]);
}

cudaError_t launch_kv_append(const KvAppendArgs &a, int num_sms, int device, cudaStream_t stream) {
    return a.c.D == 128 ? launch_append_inst<128>(a, num_sms, device, stream)
                        : launch_append_inst<64>(a, num_sms, device, stream);
}

cudaError_t launch_kv_gather(const KvCache &c, const int64_t *slots, uint16_t *k_out, uint16_t *v_out, int64_t T,
                             unsigned int *err, cudaStream_t stream) {
    const int64_t blocks = (T * c.heads * (c.D / 16) + 255) / 256;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(blocks < 1184 ? blocks : 1184), 2);
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = c.D == 128
                              ? cudaLaunchKernelEx(&cfg, kq_kv_gather_kernel<128>, c, slots, k_out, v_out, T, err)
                              : cudaLaunchKernelEx(&cfg, kq_kv_gather_kernel<64>, c, slots, k_out, v_out, T, err);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace kq
