// kq_kv_tile.cu -- attention over the INT4 key / value cache for many query rows per
// key head: chunks of prompts, and the queries of a whole batch against the prefix that
// its sequences share.
//
// There the products bound it, 4 head_dim flops per row and key on the tensor cores,
// and beside them the exponentials: 16 a clock and SM, so that 256 rows x 128 keys take
// 2048 clocks in either.  A block has 256 rows of one key head, as two tiles of 128
// (MMA's M, one row per TMEM lane), and walks 128 keys at a time:
//   - one warpgroup brings the codes: a thread reads the 64 or 32 bytes of its key's row
//     and of its value's row a tile ahead, turns them into bf16 integers (exact) and
//     lays them out as operands: K with head_dim contiguous, V with the keys as MMA's K
//     and head_dim as N.  Both row tiles multiply by them.  A word's nibbles come out in
//     the order 0 4 1 5 2 6 3 7; queries are laid in the same order, and the output is
//     put right where it leaves.
//   - scores S = Q K^T into TMEM, one warpgroup per row tile for the softmax, a thread
//     per row: x = S ks with the key's scale (times the softmax scale), p = 2^(x - m);
//     p times the value's scale goes back over S as bf16, O += P V.  The scales never
//     meet the codes, and the sum of p is fp32 with unrounded terms.  A weight's rounding
//     to bf16 (2^-9 at most) is of the size of the output's own.
//   - one pass over the scores: m is the maximum of the row's first chunk, and a weight
//     may pass 1, as fp32 and bf16 have the range (up to 2^60 here).  When a chunk's
//     largest passed 2^8, m is raised before the next one, which rescales O: rare.
//     A chunk with a value scale over 2^40, whose product with 2^60 would leave the
//     range, is looked at first as a masked one is, and its weights stay under 2^8.
//   - the two row tiles are half a step apart: while one warpgroup is at its softmax
//     the tensor core works for the other.
// Keys that a row does not see, past its place or out of its window, are looked at only
// in the chunks where a warp's rows have any; those scores go through TMEM once more.
//
// The grid has a place for every tile that the tokens could have; a sequence's tiles are found in the block.
// One unit = 256 rows of a key head and sequence, cut over `splits` blocks along its keys
// where there are fewer units than SMs; partial rows then go to the workspace for
// kq_kv_combine_kernel.
//
// Measured, head_dim 128: two chunks of 1024 and fewer queries on 2500 to 6000 keys, 32 heads
// on 8 key heads, 199 us (690 TFLOP/s; tensor pipe and exponentials both 40 % busy): a step
// of 256 rows x 128 keys takes 4500 clocks, in which a row tile's softmax (2400 to 2850) and
// its products (1600) wait for one another; a second set of scores has no place in TMEM
// there (at head_dim 64, where 128 columns are free, the order is the same).
// A prefix of 16384 keys for 64 sequences of 8 heads a key head: 68 us with the own keys.
#include <mutex>

#include "kq_kv_plan.cuh"

namespace kq {
namespace {

using namespace kv;
using namespace tc;

constexpr int T_THREADS = 416;  // two warpgroups of softmax, one of codes, a warp of MMAs

template <int D>
struct TCfg {
    static constexpr int HALF = 128 * 128;           // 128 rows of 64 bf16 values
    static constexpr int OPERAND = HALF * (D / 64);  // 128 rows of D values
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_K = 2 * OPERAND;
    static constexpr int OFF_V = OFF_K + 2 * OPERAND;
    static constexpr int OFF_SC = OFF_V + 2 * OPERAND;  // per stage 128 key scales, 128 value scales
    static constexpr int OFF_BAR = OFF_SC + 2 * 1024;
    enum { KFULL = 0, KFREE = 2, VFULL = 4, VFREE = 6, SREADY = 8, PREADY = 10, ODONE = 12, SCFREE = 14, DONE = 16, QREADY = 17, NBAR = 18 };
    static constexpr int OFF_MISC = OFF_BAR + 8 * NBAR;
    static constexpr int SMEM = OFF_MISC + 16 + 1024;  // TMEM base, abort flag, per stage whether it is special
    static constexpr int COL_S = 0, COL_O = 256;  // TMEM columns: S of tile q at 128 q, O at 256 + D q
    static_assert(SMEM <= 227 * 1024, "shared memory");
};

template <bool B>
struct Is {
    static constexpr bool value = B;
};

// Eight codes as bf16 integers, pairs (0, 4), (1, 5), (2, 6), (3, 7): (code + 8) | 0x4300 is 136 + code.
__device__ __forceinline__ uint4 codes_bf16(uint32_t w) {
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t t;
        // (x & 0xf) ^ (0x4300 | 8)
        asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(t) : "r"(w >> (4 * i)), "r"(0x000f000fu), "r"(0x43084308u));
        asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(o[i]) : "r"(t), "r"(0x43084308u));
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}
// Eight consecutive bf16 values in that order.
__device__ __forceinline__ uint4 order_bf16(const uint4 &u) {
    return make_uint4(__byte_perm(u.x, u.z, 0x5410), __byte_perm(u.x, u.z, 0x7632), __byte_perm(u.y, u.w, 0x5410),
                      __byte_perm(u.y, u.w, 0x7632));
}
// Place of 16-byte piece u of row r in an operand of D values a row (128-byte swizzle).
__device__ __forceinline__ uint32_t operand_place(int r, int u) {
    return uint32_t((u >> 3) * (128 * 128) + r * 128 + (((u ^ r) & 7) << 4));
}

template <int D, bool CAP>
__global__ void __launch_bounds__(T_THREADS, 1)
    kq_kv_tile_kernel(const __grid_constant__ Plan p, int prefix, int splits, int own_tiles) {
    using C = TCfg<D>;
    extern __shared__ __align__(1024) unsigned char t_raw[];
    const uint32_t raw_addr = smem_u32(t_raw), sbase = (raw_addr + 1023u) & ~1023u;
    unsigned char *smem = t_raw + (sbase - raw_addr);
    const KvAttnArgs &a = p.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, wg = warp >> 2;
    const int Hk = a.c.heads, H = a.q_heads, psh = a.c.page_shift;
    auto bar = [&](int i) -> uint32_t { return sbase + uint32_t(C::OFF_BAR + 8 * i); };
    volatile int *s_abort = reinterpret_cast<volatile int *>(smem + C::OFF_MISC + 4);
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(C::KFULL + i), 128);
            mbar_init(bar(C::VFULL + i), 128);
            mbar_init(bar(C::KFREE + i), 1);
            mbar_init(bar(C::VFREE + i), 1);
            mbar_init(bar(C::SREADY + i), 1);
            mbar_init(bar(C::PREADY + i), 4);
            mbar_init(bar(C::ODONE + i), 1);
            mbar_init(bar(C::SCFREE + i), 8);
        }
        mbar_init(bar(C::DONE), 1);
        mbar_init(bar(C::QREADY), 256);
        *s_abort = 0;
        fence_mbar_init();
    }
    if (warp == 12) {
        tmem_alloc(sbase + C::OFF_MISC, 512);
        tmem_relinquish();
    }
    begin_launch(p);

    // ---- the block's unit: rows, and its part of their keys ----
    const int id = int(blockIdx.x), split = id % splits;
    int u = id / splits;
    const int h = u % Hk;
    u /= Hk;
    int64_t b = a.B;
    bool none = false;
    if (!prefix && a.B <= 32) {
        // The longest units first: sequences by falling length, each with the tiles that it has.
        int len = INT_MIN, has = 0;
        if (lane < a.B) {
            len = a.kv_len[lane];
            has = load_seq<kTileRows>(p, lane, false).tiles;
        }
        int before = 0;
        for (int k = 0; k < int(a.B); ++k) {
            const int other = __shfl_sync(0xffffffffu, len, k), its = __shfl_sync(0xffffffffu, has, k);
            if (other > len || (other == len && k < lane)) before += its;
        }
        const uint32_t at = __ballot_sync(0xffffffffu, before <= u && u < before + has);
        none = at == 0;
        b = none ? 0 : __ffs(at) - 1;
        u -= __shfl_sync(0xffffffffu, before, int(b));
    } else if (!prefix && own_tiles) {
        b = u / own_tiles;
        u -= int(b) * own_tiles;
    } else if (!prefix) {
        // the last sequence whose place is at or before u, 32 looked at in a step
        auto begin = [&](int64_t k) {
            int q0, m;
            queries_of(a, k, q0, m);
            return own_place(q0, k, p.G, p.few);
        };
        int64_t lo = 0, hi = a.B;
        while (hi - lo > 1) {
            const int64_t step = (hi - lo + 31) / 32, k = lo + lane * step;
            const int n = max(1, __popc(__ballot_sync(0xffffffffu, k < hi && begin(k) <= u)));
            lo += (n - 1) * step;
            hi = min(hi, lo + step);
        }
        b = lo;
        u = int(max(int64_t(0), u - begin(b)));
    }
    const Seq s = load_seq<kTileRows>(p, b, u == 0 && h == 0 && split == 0 && tid == 0 && !prefix);
    none |= u >= s.tiles;
    const int tile = none ? 0 : s.tiles - 1 - u;  // the last rows of a chunk, which see the most keys, before its first
    const int rows = none ? 0 : min(kTileRows, s.m * p.G - tile * kTileRows);
    const int first = tile * kTileRows / p.G, last = (tile * kTileRows + max(rows, 1) - 1) / p.G;  // queries
    // keys that some row of the tile sees
    int hi = min(s.n, max(0, s.shift + last + 1)), lo = 0;
    if (a.window && !prefix) lo = int(min(int64_t(hi), max(int64_t(0), int64_t(s.shift) + first - a.window + 1)));
    const int c0 = lo / CH, chunks = (hi + CH - 1) / CH - c0;
    const int j0 = c0 + int(int64_t(chunks) * split / splits), j1 = c0 + int(int64_t(chunks) * (split + 1) / splits);
    const int N = j1 - j0;  // chunks of this block
    const bool two = rows > 128;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + C::OFF_MISC);
    griddep_launch_dependents();

    // ---- queries: bf16 rows as operands; rows past the last are zeros ----
    if (wg < 2) {
        // a warp brings 32 rows, whole rows side by side: a lane 16 bytes of 256 / D rows a step
        const int r = tid & 127, j = tile * kTileRows + 128 * wg + r;
        const bool real = 128 * wg + r < rows;
        const int i = real ? j / p.G : 0;
        const uint16_t *mine = real ? a.q + (int64_t(s.q0 + i) * H + h * p.G + (j - i * p.G)) * D : nullptr;
        constexpr int PIECES = D / 8, PER = 32 / PIECES;
        uint4 q[32 / PER];
#pragma unroll
        for (int k = 0; k < 32 / PER; ++k) {
            const uint64_t from = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(mine), k * PER + lane / PIECES);
            q[k] = make_uint4(0, 0, 0, 0);
            if (from) q[k] = reinterpret_cast<const uint4 *>(from)[lane % PIECES];
        }
#pragma unroll
        for (int k = 0; k < 32 / PER; ++k)
            *reinterpret_cast<uint4 *>(smem + C::OFF_Q + wg * C::OPERAND +
                                       operand_place((r & ~31) + k * PER + lane / PIECES, lane % PIECES)) = order_bf16(q[k]);
        fence_proxy_async_smem();
        mbar_arrive(bar(C::QREADY));
    }

    auto wait = [&](int i, uint32_t parity) -> bool { return wait_all(bar(i), parity & 1u, s_abort, a.err); };

    if (rows <= 0) {
        // no such rows (a bound on them sized the grid)
    } else if (wg < 2) {
        // ---------------- softmax: a row per thread ----------------
        const int r = tid & 127, jr = 128 * wg + r, j = tile * kTileRows + jr;
        const bool real = jr < rows;
        const int i = real ? j / p.G : 0;
        int row_lo = 0, row_hi = 0;  // keys that the row sees
        if (real) {
            row_hi = min(s.n, max(0, s.shift + i + 1));
            if (a.window) {
                const int64_t pos = prefix ? a.prefix_len + query_shift(a, s.q0 + i) : int64_t(s.shift) + i;
                row_lo = int(min(int64_t(row_hi), max(int64_t(0), pos - a.window + 1)));
            }
        }
        const uint32_t lanes = uint32_t(32 * (warp & 3)) << 16;
        const uint32_t ts = tmem + lanes + uint32_t(C::COL_S + 128 * wg), to = tmem + lanes + uint32_t(C::COL_O + D * wg);
        float m = 0.0f, l0 = 0.0f, l1 = 0.0f;  // the reference, and the sum of the weights in two parts
        bool seen = !real;                     // the reference is set: some chunk had a key that the row sees
        bool ok = true;
        const int steps = wg == 0 || two ? N : 0;
        if (wg == 1 && !two) {  // no rows: only the scales' stages are given back
            for (int n = 0; n < N; ++n) {
                ok = wait(C::VFULL + (n & 1), uint32_t(n >> 1));
                if (!ok) break;
                if (lane == 0) mbar_arrive(bar(C::SCFREE + (n & 1)));
            }
        }
        // all rows of the warp see all keys of [all_lo, all_hi) (rows past the last are not looked at)
        const bool no_rows = !__any_sync(0xffffffffu, real);
        const int all_lo = __reduce_max_sync(0xffffffffu, real ? row_lo : 0);
        const int all_hi = __reduce_min_sync(0xffffffffu, real ? row_hi : INT_MAX);
        float rise = 0.0f;  // how far the last chunk's largest score was over the reference
        for (int n = 0; n < steps; ++n) {
            const int t0 = (j0 + n) * CH;
            const float4 *ks = reinterpret_cast<const float4 *>(smem + C::OFF_SC + 1024 * (n & 1));
            const float4 *vs = ks + 32;
            ok = wait(C::KFULL + (n & 1), uint32_t(n >> 1)) && wait(C::SREADY + wg, uint32_t(n));
            if (!ok) break;
            tc_fence_after();
            if (no_rows) {  // this warp's weights are never read
                if (lane == 0) {
                    mbar_arrive(bar(C::PREADY + wg));
                    mbar_arrive(bar(C::SCFREE + (n & 1)));
                }
                continue;
            }
            // a key without a page, or a value scale over 2^40
            const bool special = *reinterpret_cast<volatile int *>(smem + C::OFF_MISC + 8 + 4 * (n & 1)) != 0;
            const bool slow = special || t0 < all_lo || t0 + CH > all_hi;
            // The reference rises by `up`: O, whose last product has ended with S's, and the sums follow.
            auto raise = [&](float up) {
                const float f = ex2(-up);
                m += up;
                l0 *= f;
                l1 *= f;
                if (n > 0) {
#pragma unroll 1
                    for (int c = 0; c < D; c += 16) {
                        uint32_t v[16];
                        tmem_ld_32x32b_x16(to + uint32_t(c), v);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * f);
                        tmem_st_32x32b_x16(to + uint32_t(c), v);
                    }
                    tmem_wait_st();
                }
            };
            if (__any_sync(0xffffffffu, rise > 8.0f)) raise(rise > 8.0f ? rise : 0.0f);
            rise = 0.0f;
            const bool first_keys = __any_sync(0xffffffffu, !seen);
            if (slow || first_keys) {
                // ---- the row's largest score; where some keys are not seen, the scores with -inf for those
                // go back to their place ----
                float top = -INFINITY;
                if (!slow) {
#pragma unroll 1
                    for (int c = 0; c < CH; c += 32) {
                        uint32_t v[32];
                        tmem_ld_32x32b_x32(ts + uint32_t(c), v);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; e += 4) {
                            const float4 k = ks[(c + e) >> 2];
                            top = fmax3(top, __uint_as_float(v[e]) * k.x, __uint_as_float(v[e + 1]) * k.y);
                            top = fmax3(top, __uint_as_float(v[e + 2]) * k.z, __uint_as_float(v[e + 3]) * k.w);
                        }
                    }
                    if (CAP) top = a.softcap * kLog2e * tanh_any(top);  // which rises with its argument
                } else
#pragma unroll 1
                for (int c = 0; c < CH; c += 32) {
                    uint32_t v[32];
                    tmem_ld_32x32b_x32(ts + uint32_t(c), v);
                    tmem_wait_ld();
                    if constexpr (CAP) {
                        float far = 0.0f;
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            v[e] = __float_as_uint(__uint_as_float(v[e]) * reinterpret_cast<const float *>(ks)[c + e]);
                            far = fmaxf(far, fabsf(__uint_as_float(v[e])));
                        }
                        const bool small = __all_sync(0xffffffffu, far <= 0.5f);
#pragma unroll
                        for (int e = 0; e < 32; e += 4) {
                            uint64_t a0 = pair2u(v[e], v[e + 1]), a1 = pair2u(v[e + 2], v[e + 3]);
                            if (small) a0 = tanh_small(a0), a1 = tanh_small(a1);
                            else tanh_pairs(a0, a1);
                            split2u(a0, v[e], v[e + 1]);
                            split2u(a1, v[e + 2], v[e + 3]);
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const float k = reinterpret_cast<const float *>(ks)[c + e];
                        float x = __uint_as_float(v[e]) * (CAP ? a.softcap * kLog2e : k);
                        const int t = t0 + c + e;
                        if (t < row_lo || t >= row_hi || (special && k == -INFINITY)) x = -INFINITY;
                        v[e] = __float_as_uint(x);
                        top = fmaxf(top, x);
                    }
                    tmem_st_32x32b_x16(ts + uint32_t(c), reinterpret_cast<const uint32_t(&)[16]>(v[0]));
                    tmem_st_32x32b_x16(ts + uint32_t(c + 16), reinterpret_cast<const uint32_t(&)[16]>(v[16]));
                }
                tmem_wait_st();
                if (!seen && top > -INFINITY) {  // nothing has been summed yet: the reference may be anywhere
                    seen = true;
                    m = top;
                }
                if (__any_sync(0xffffffffu, top > m + 8.0f)) raise(top > m + 8.0f ? top - m : 0.0f);
            }
            // ---- weights, over the scores ----
            uint64_t sum = pair2(l0, l1);
            auto weights = [&](auto raw) {
#pragma unroll 1
                for (int c = 0; c < CH; c += 32) {
                    uint32_t v[32], w[16];
                    tmem_ld_32x32b_x32(ts + uint32_t(c), v);
                    tmem_wait_ld();
                    // x = S ks - m (capped: cap tanh(S ks) - m), or the prepared scores less m; p = 2^x
                    uint64_t more;  // what the block adds to the sum
                    float most[4];
                    auto block = [&](auto small) {
                        const uint64_t minus = pair2(-m, -m);
                        more = pair2(0.0f, 0.0f);
#pragma unroll
                        for (int k = 0; k < 4; ++k) most[k] = -INFINITY;
#pragma unroll
                        for (int e = 0; e < 32; e += 4) {
                            uint64_t a0 = pair2u(v[e], v[e + 1]), a1 = pair2u(v[e + 2], v[e + 3]);
                            float x0, x1, x2, x3;
                            if constexpr (decltype(raw)::value) {
                                const float4 k = ks[(c + e) >> 2];
                                if constexpr (CAP) {
                                    a0 = f32x2_mul(a0, pair2(k.x, k.y));
                                    a1 = f32x2_mul(a1, pair2(k.z, k.w));
                                    if constexpr (decltype(small)::value) {
                                        a0 = tanh_small(a0);
                                        a1 = tanh_small(a1);
                                    } else {
                                        tanh_pairs(a0, a1);
                                    }
                                    const uint64_t cap = pair2(a.softcap * kLog2e, a.softcap * kLog2e);
                                    a0 = fma2(a0, cap, minus);
                                    a1 = fma2(a1, cap, minus);
                                } else {
                                    a0 = fma2(a0, pair2(k.x, k.y), minus);
                                    a1 = fma2(a1, pair2(k.z, k.w), minus);
                                }
                                split2(a0, x0, x1);
                                split2(a1, x2, x3);
                                most[(e >> 1) & 2] = fmax3(most[(e >> 1) & 2], x0, x1);
                                most[((e >> 1) & 2) + 1] = fmax3(most[((e >> 1) & 2) + 1], x2, x3);
                            } else {
                                split2(add2(a0, minus), x0, x1);
                                split2(add2(a1, minus), x2, x3);
                            }
                            const float4 z = vs[(c + e) >> 2];
                            const uint64_t p0 = pair2(ex2(x0), ex2(x1)), p1 = pair2(ex2(x2), ex2(x3));
                            more = add2(more, add2(p0, p1));
                            float y0, y1, y2, y3;
                            split2(f32x2_mul(p0, pair2(z.x, z.y)), y0, y1);
                            split2(f32x2_mul(p1, pair2(z.z, z.w)), y2, y3);
                            w[e >> 1] = pack_bf16x2(y0, y1);
                            w[(e >> 1) + 1] = pack_bf16x2(y2, y3);
                        }
                    };
                    auto choose = [&] {
                        if constexpr (CAP && decltype(raw)::value) {
                            // the tanh: a polynomial where all its arguments are small, as they mostly are, for
                            // the exponentials bound this kernel
                            float far[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                            for (int e = 0; e < 32; e += 4) {
                                const float4 k = ks[(c + e) >> 2];
                                far[0] = fmaxf(far[0], fabsf(__uint_as_float(v[e]) * k.x));
                                far[1] = fmaxf(far[1], fabsf(__uint_as_float(v[e + 1]) * k.y));
                                far[2] = fmaxf(far[2], fabsf(__uint_as_float(v[e + 2]) * k.z));
                                far[3] = fmaxf(far[3], fabsf(__uint_as_float(v[e + 3]) * k.w));
                            }
                            if (__all_sync(0xffffffffu, fmaxf(fmaxf(far[0], far[1]), fmaxf(far[2], far[3])) <= 0.5f)) {
                                block(Is<true>{});
                                return;
                            }
                        }
                        block(Is<false>{});
                    };
                    choose();
                    if constexpr (decltype(raw)::value) {
                        const float top = fmaxf(fmaxf(most[0], most[1]), fmaxf(most[2], most[3]));
                        if (__any_sync(0xffffffffu, top > 60.0f)) {
                            // out of a weight's range: raise the reference here, and what the chunk has so far,
                            // and do the block again
                            const float up = top > 60.0f ? top : 0.0f, f = ex2(-up);
                            split2(sum, l0, l1);
                            raise(up);
                            sum = pair2(l0, l1);
                            rise = fmaxf(rise - up, 0.0f);
#pragma unroll 1
                            for (int d = 0; d < (c >> 1); d += 16) {
                                tmem_ld_32x32b_x16(ts + uint32_t(d), w);
                                tmem_wait_ld();
#pragma unroll
                                for (int e = 0; e < 16; ++e)
                                    w[e] = pack_bf16x2(__uint_as_float(w[e] << 16) * f,
                                                       __uint_as_float(w[e] & 0xffff0000u) * f);
                                tmem_st_32x32b_x16(ts + uint32_t(d), w);
                            }
                            tmem_wait_st();
                            choose();
                        }
                        rise = fmaxf(rise, fmaxf(fmaxf(most[0], most[1]), fmaxf(most[2], most[3])));
                    }
                    sum = add2(sum, more);
                    tmem_st_32x32b_x16(ts + uint32_t(c >> 1), w);
                }
            };
            if (slow) weights(Is<false>{});
            else weights(Is<true>{});
            split2(sum, l0, l1);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bar(C::PREADY + wg));
                mbar_arrive(bar(C::SCFREE + (n & 1)));
            }
        }
        // ---- the rows ----
        if (steps > 0 && ok) ok = wait(C::ODONE + wg, uint32_t(N - 1));
        if ((wg == 0 || two) && ok) {
            tc_fence_after();
            const float l = l0 + l1;
            const float inv = l > 0.0f ? 1.0f / l : l == 0.0f ? 0.0f : l;
            const float lse = l == 0.0f ? -INFINITY : m + lg2(l);  // in powers of two
            const int64_t at = int64_t(s.q0 + i) * H + h * p.G + (real ? j - i * p.G : 0);
            const bool final = splits == 1 && !p.partial;
            float *po = p.tile_o + (int64_t(prefix ? p.own_splits : 0) + split) * a.T * H * D;
            // 32 columns at a time through the warp's 4 KB of the queries' place (its products have ended), a
            // row's 16-byte pieces exchanged by row, so that a store takes 128 bytes of 4 rows
            unsigned char *own = smem + C::OFF_Q + wg * C::OPERAND + (warp & 3) * 4096;
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                uint32_t v[32];
                if (N > 0) {
                    tmem_ld_32x32b_x32(to + uint32_t(c), v);
                    tmem_wait_ld();
                }
#pragma unroll
                for (int e = 0; e < 32; e += 8) {
                    // columns 2 i, 2 i + 1 of eight are the elements i, i + 4
                    float o[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        o[(k >> 1) + 4 * (k & 1)] = N > 0 && l != 0.0f ? __uint_as_float(v[e + k]) * inv : 0.0f;
                    *reinterpret_cast<float4 *>(own + 128 * lane + (((e / 4) ^ (lane & 7)) << 4)) =
                        make_float4(o[0], o[1], o[2], o[3]);
                    *reinterpret_cast<float4 *>(own + 128 * lane + (((e / 4 + 1) ^ (lane & 7)) << 4)) =
                        make_float4(o[4], o[5], o[6], o[7]);
                }
                __syncwarp();
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int row = 4 * k + (lane >> 3);
                    const int64_t to_row = __shfl_sync(0xffffffffu, real ? at : int64_t(-1), row);
                    const float4 o = *reinterpret_cast<const float4 *>(own + 128 * row + (((lane ^ row) & 7) << 4));
                    if (to_row >= 0) {
                        if (final)
                            *reinterpret_cast<uint2 *>(a.out + to_row * D + c + 4 * (lane & 7)) =
                                make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
                        else
                            *reinterpret_cast<float4 *>(po + to_row * D + c + 4 * (lane & 7)) = o;
                    }
                }
                __syncwarp();
            }
            if (real) {
                if (p.few && !prefix && split == 0) p.parts[at] = make_int2(-1, splits);
                if (!final) p.tile_l[(int64_t(prefix ? p.own_splits : 0) + split) * a.T * H + at] = lse;
                else if (a.lse) a.lse[at] = lse * 0.6931471805599453f;
            }
        }
        tc_fence_before();
    } else if (wg == 2) {
        // ---------------- codes into operands: a key per thread ----------------
        const int r = tid & 127;
        const float factor = CAP ? a.scale / a.softcap : a.scale * kLog2e;
        // of a key's scale times that: finite, so that a zero score stays one; a tanh is 1 long before
        constexpr float kMost = CAP ? 0x1p100f : 0x1.fffffep127f;
        constexpr int W = D / 32;  // 16-byte pieces of a row of codes
        struct Row {
            uint4 k[W], v[W];
            float ks, vs;
        };
        auto page_of = [&](int n) -> int {
            const int t = (j0 + n) * CH + r;
            return n < N && t < s.n && t >= lo ? s.pages[t >> psh] : -1;
        };
        auto load = [&](int n, int page) {
            Row w;
            const int t = (j0 + n) * CH + r;
            w.ks = w.vs = 0.0f;
#pragma unroll
            for (int i = 0; i < W; ++i) w.k[i] = w.v[i] = make_uint4(0, 0, 0, 0);
            if (n < N && t < s.n && t >= lo) {
                if (uint32_t(page) < uint32_t(a.c.pages)) {
                    const int64_t row = ((int64_t(page) * Hk + h) << psh) + (t & ((1 << psh) - 1));
                    const uint4 *k = reinterpret_cast<const uint4 *>(a.c.k_codes + row * (D / 2));
                    const uint4 *v = reinterpret_cast<const uint4 *>(a.c.v_codes + row * (D / 2));
#pragma unroll
                    for (int i = 0; i < W; ++i) w.k[i] = k[i], w.v[i] = v[i];
                    w.ks = fminf(fmaxf(a.c.k_scale[row] * factor, -kMost), kMost);
                    w.vs = fminf(a.c.v_scale[row], 0x1.fffffep127f);  // a weight of 0 leaves any row out
                } else {
                    w.ks = -INFINITY;  // no such page: the mark by which the softmax leaves the key out
                    atomicOr(a.err, kSiteKvAttention);
                }
            }
            return w;
        };
        auto lay = [&](int off, const uint4 (&c)[W]) {
#pragma unroll
            for (int i = 0; i < W; ++i) {
                const uint32_t x[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    *reinterpret_cast<uint4 *>(smem + off + operand_place(r, 4 * i + k)) = codes_bf16(x[k]);
            }
        };
        bool ok = true;
        Row now = load(0, page_of(0));
        int page = page_of(1);
        for (int n = 0; n < N; ++n) {
            const int st = n & 1;
            const uint32_t ph = uint32_t(n >> 1) ^ 1u;
            const Row next = load(n + 1, page);
            page = page_of(n + 2);
            const bool special = named_barrier_any(1, 128, (now.ks == -INFINITY && now.vs == 0.0f) || now.vs > 0x1p40f);
            ok = ok && wait(C::KFREE + st, ph) && wait(C::SCFREE + st, ph);
            if (!ok) continue;  // the warpgroup's barrier wants every warp, also one that has given up
            if (r == 0) *reinterpret_cast<volatile int *>(smem + C::OFF_MISC + 8 + 4 * st) = special;
            lay(C::OFF_K + st * C::OPERAND, now.k);
            float *sc = reinterpret_cast<float *>(smem + C::OFF_SC + 1024 * st);
            sc[r] = now.ks;
            sc[128 + r] = now.vs;
            fence_proxy_async_smem();
            mbar_arrive(bar(C::KFULL + st));
            ok = wait(C::VFREE + st, ph);
            if (!ok) continue;
            lay(C::OFF_V + st * C::OPERAND, now.v);
            fence_proxy_async_smem();
            mbar_arrive(bar(C::VFULL + st));
            now = next;
        }
    } else {
        // ---------------- products ----------------
        constexpr uint32_t idesc_s = idesc_bf16_f32(128, 128), idesc_o = idesc_bf16_f32_bn(128, D);
        const int nq = two ? 2 : 1;
        auto scores = [&](int n, int q) {  // S(q) = Q(q) K(n)^T
            if (elect_one()) {
                const uint32_t qa = sbase + uint32_t(C::OFF_Q + q * C::OPERAND);
                const uint32_t ka = sbase + uint32_t(C::OFF_K + (n & 1) * C::OPERAND);
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t off = uint32_t((k >> 2) * C::HALF + 32 * (k & 3));
                    mma_ss(tmem + uint32_t(C::COL_S + 128 * q), sdesc_kmajor_sw128(qa + off), sdesc_kmajor_sw128(ka + off),
                           idesc_s, k != 0);
                }
                tc_commit(bar(C::SREADY + q));
            }
            __syncwarp();
        };
        bool ok = N > 0 && wait(C::QREADY, 0u) && wait(C::KFULL, 0u);
        if (ok) {
            tc_fence_after();
            for (int q = 0; q < nq; ++q) scores(0, q);
            if (elect_one()) tc_commit(bar(C::KFREE));
            __syncwarp();
        }
        for (int n = 0; n < N && ok; ++n) {
            ok = wait(C::VFULL + (n & 1), uint32_t(n >> 1));
            if (ok && n + 1 < N) ok = wait(C::KFULL + ((n + 1) & 1), uint32_t((n + 1) >> 1));
            for (int q = 0; q < nq && ok; ++q) {
                ok = wait(C::PREADY + q, uint32_t(n));
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {  // O(q) += P(q) V(n)
                    const uint32_t va = sbase + uint32_t(C::OFF_V + (n & 1) * C::OPERAND);
#pragma unroll
                    for (int k = 0; k < CH / 16; ++k)
                        mma_ts(tmem + uint32_t(C::COL_O + D * q), tmem + uint32_t(C::COL_S + 128 * q + 8 * k),
                               sdesc_nmajor_sw128(va + uint32_t(2048 * k), C::HALF), idesc_o, n != 0 || k != 0);
                    tc_commit(bar(C::ODONE + q));
                }
                __syncwarp();
                if (n + 1 < N) scores(n + 1, q);
            }
            if (ok && elect_one()) {
                tc_commit(bar(C::VFREE + (n & 1)));
                if (n + 1 < N) tc_commit(bar(C::KFREE + ((n + 1) & 1)));
            }
            __syncwarp();
        }
        // every product has ended before the block's TMEM is given back
        if (elect_one()) tc_commit(bar(C::DONE));
        __syncwarp();
        (void)wait_bounded_err(bar(C::DONE), 0u, s_abort, kSiteKvWait, kWaitLimitNs, true, a.err);
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 12) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    end_launch(p);
}

template <int D, bool CAP>
cudaError_t launch_inst(const Plan &p, bool prefix, int splits, int device, cudaStream_t stream) {
    using C = TCfg<D>;
    auto kern = kq_kv_tile_kernel<D, CAP>;
    static std::once_flag once[64];
    static cudaError_t attr_err[64];
    if (device < 0 || device >= 64) return cudaErrorInvalidDevice;
    std::call_once(once[device], [&] {
        attr_err[device] = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    });
    if (attr_err[device] != cudaSuccess) return attr_err[device];
    // where that is no more, every sequence has the places of one at the bound of queries: own_tiles
    const int64_t full = kv_tiles(p.a.max_q, p.G);
    const int64_t tiles = prefix ? kv_tiles(p.a.T, p.G) : kv_own_tiles(p.a.T, p.a.B, p.a.max_q, p.G, p.few);
    const int64_t grid = tiles * p.a.c.heads * splits;
    if (grid >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
    return launch_overlapped(kern, unsigned(grid), T_THREADS, C::SMEM, stream, p, int(prefix), splits,
                             int(tiles == full * p.a.B ? full : 0));
}

}  // namespace

cudaError_t launch_kv_tile(const kv::Plan &p, bool prefix, int splits, int device, cudaStream_t stream) {
    if (p.a.c.D == 128)
        return p.a.softcap > 0.0f ? launch_inst<128, true>(p, prefix, splits, device, stream)
                                  : launch_inst<128, false>(p, prefix, splits, device, stream);
    return p.a.softcap > 0.0f ? launch_inst<64, true>(p, prefix, splits, device, stream)
                              : launch_inst<64, false>(p, prefix, splits, device, stream);
}

}  // namespace kq
