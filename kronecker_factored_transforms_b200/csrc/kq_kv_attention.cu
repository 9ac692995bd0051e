// kq_kv_attention.cu -- softmax attention over the pages of the INT4 key / value
// cache (kq_kv_attention, kq_kv_attention_shared).
//
// For a query row q (one token, one head) and the keys t that it sees, with c_t
// and s_t the codes and scales of the cache's rows:
//
//     x_t = scale s_t (q . c_t), capped by a tanh where asked,
//     out = sum_t exp(x_t) s'_t c'_t / sum_t exp(x_t),   lse = log sum_t exp(x_t)
//
// The scales never meet the codes: s_t multiplies a score, s'_t a weight.  So the
// matrix products run on the codes themselves, which 16-bit floats hold exactly.
//
// The row kernel (kq_kv_rows_kernel) serves few query rows per key head (one token
// of each sequence, with its group of heads; a few drafted tokens).  There the
// bytes of the cache bound it: head_dim / 2 + 4 for 4 head_dim flops per row of
// queries.  Its products run in the warps' own mma (m16n8k16): 16 keys are the M
// side, 8 rows of queries the N side, so that one group of heads fills the tile,
// which a 128-row tcgen05 tile would leave 15/16 empty, and the codes go from
// shared memory straight into the registers of the A operand:
//   - a 16-bit word (w ^ 0x8) & 0xf is code + 8 as a subnormal fp16 (times 2^-24),
//     so two codes cost one LOP3; codes in the next nibble come out times 16.
//   - scores: the + 8 is taken back by starting the accumulator at -8 sum(q), the
//     factors 16 and 2^24 by the query operand and the score's multiplier.  The query
//     row is brought to fp16 by a power of two: exact, as bf16 has 8 bits.
//   - values: here the + 8 is taken off every code (one HFMA2 for two), because
//     weights all have one sign: 8 sum(p) would outgrow sum(p c) in the sum.
//   - the order of head_dim within the products is free, so a lane takes 16
//     consecutive bytes of a key row, and 8 of a value row, as they lie.
// Weights go to fp16 as 2^(x + log2 s' - r): relative to a running reference r that
// follows the maximum of x + log2 s', so they keep 11 bits whatever the scales'
// size, with r moved only when a weight would pass 2^14 (rounded to 2^6 under it).
// The sum of exp(x) is fp32 with unrounded terms.
//
// Work is split evenly: the (sequence, key head, row tile) units are laid in a row,
// 128 keys a chunk, and every block takes the same number of chunks wherever that
// cuts; a warp of its own loads them into a ring of stages, four warps take 32 keys
// of each chunk, with their own softmax states, joined at a unit's end.  A unit cut
// by block borders leaves partial rows in the workspace, at most two per block,
// which kq_kv_combine_kernel joins in a fixed order.
//
// Measured, head_dim 128 and 8 key heads: 4 sequences of 65 to 131 thousand keys, 4 query
// heads a key head, 97-104 us (4.2-4.4 TB/s of 6.55; issue slots 56 % busy, ALU 52 %: some 500
// instructions for 32 keys and warp); 64 sequences of 60 to 8192 keys, 8 query heads a key
// head, 37-39 us; one token on 1531 keys 10 us.  With capped scores 42 us for 40 without.
#include <cuda_fp16.h>

#include <mutex>

#include "kq_kv_plan.cuh"

namespace kq {
namespace {

using namespace kv;

constexpr float kNone = -1e30f;  // reference of a row that has seen no key
constexpr int WARPS = 4;        // multiplying warps per block
constexpr int MT = 2;           // tiles of 16 keys that each takes of a chunk
static_assert(CH == 16 * MT * WARPS, "keys per chunk");
constexpr int R_THREADS = 32 * (WARPS + 1);
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&v);
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
// Codes of nibbles 0 and 4 (lo) and 1 and 5 (hi, times 16) of a word, plus 8, times 2^-24, as fp16 pairs.
// (w & mask) ^ eight, one LOP3 with the second constant in a register.
__device__ __forceinline__ uint32_t and_xor(uint32_t w, uint32_t mask, uint32_t eight) {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(d) : "r"(w), "r"(mask), "r"(eight));
    return d;
}
__device__ __forceinline__ uint32_t nib_lo(uint32_t w) { return and_xor(w, 0x000f000fu, 0x00080008u); }
__device__ __forceinline__ uint32_t nib_hi(uint32_t w) { return and_xor(w, 0x00f000f0u, 0x00800080u); }

// The work of all units, dealt to the blocks: n places each, and one more to the first `more`.  A unit
// is as many places as it has chunks, behind kUnitCost empty ones that stand for its start and end (its
// queries made operands, its warps' rows joined: some 5000 clocks, where a chunk takes 1900).  A block
// works on the chunks at its places; the blocks of a unit are consecutive.
constexpr int kUnitCost = 3;
struct Shares {
    int64_t n, more;
    __device__ __forceinline__ Shares(int64_t total, int ctas) {
        n = total < (int64_t(1) << 31) ? int64_t(uint32_t(total) / uint32_t(ctas)) : total / ctas;
        more = total - n * ctas;
    }
    __device__ __forceinline__ int64_t begin(int64_t block) const { return n * block + min(block, more); }
    __device__ __forceinline__ int block_of(int64_t place) const {
        const int64_t big = (n + 1) * more;
        return int(place < big ? place / (n + 1) : more + (place - big) / n);
    }
};

// A walk over the chunks of a block: sequence, head, row tile, chunk.
template <int R>
struct Walk {
    int64_t b;
    int h, tile, c;
    Seq s;
    __device__ __forceinline__ void next(const Plan &p, int64_t seqs) {
        if (++c < s.c0 + s.N) return;
        if (++tile == s.tiles) {
            tile = 0;
            if (++h == p.a.c.heads) {
                h = 0;
                do {
                    if (++b >= seqs) return;
                    s = load_seq<R>(p, b, false);
                } while (s.tiles == 0);
            }
        }
        c = s.c0;
    }
};

// ---- the row kernel ----------------------------------------------------------------

template <int D, int NT>
struct RCfg {
    static constexpr int R = 8 * NT;               // query rows per tile
    static constexpr int STAGES = 3;
    static constexpr int CODES = CH * D / 2;       // a chunk's codes, of keys or of values
    static constexpr int Q = 2 * CODES + 2 * CH * 4;  // the unit's query rows, where one begins
    static constexpr int STAGE = Q + R * D * 2;
    static constexpr int PROW = D + 8;              // floats of a row of a part
    static constexpr int PART = R * (PROW + 2) * 4;  // a warp's rows when a unit ends: values, reference, sum
    static constexpr int OFF_PART = STAGES * STAGE;
    static constexpr int OFF_DESC = OFF_PART + WARPS * PART;      // a Desc per stage
    static constexpr int OFF_BAR = OFF_DESC + STAGES * 64;
    static constexpr int FULL = 0, EMPTY = STAGES, JOIN = 2 * STAGES, NBAR = JOIN + 2;
    static constexpr int OFF_MISC = OFF_BAR + 8 * NBAR;           // abort flag
    static constexpr int OFF_SCAN = (OFF_MISC + 4 + 15) & ~15;
    static constexpr int SMEM = OFF_SCAN + 8 * (WARPS + 1) + 16;
    // blocks per SM, as registers and shared memory allow (head_dim 64, 64 sequences of 4000 keys, 8 key heads of 4:
    // 82 us with three, 54 with four, 59 with five and 72 registers)
    static constexpr int OCC = NT == 1 ? (D == 64 ? 4 : 3) : 2;
    static_assert((SMEM + 1024) * OCC <= 227 * 1024, "shared memory of the resident blocks");
    static_assert(STAGE % 128 == 0 && OFF_PART % 16 == 0 && OFF_BAR % 8 == 0, "alignment");
};

// What the loading warp says of a stage's chunk to those that multiply.
struct Desc {
    int t0, n;        // first key, keys of the sequence
    uint32_t flags;   // bit s: the 16 keys from t0 + 16 s are there; and those below
    int shift;
    int q0, m, h, tile;
    int place;        // of partial rows: kWhole, or the slot's number
    int prefix;       // whether this is the shared prefix
    int parts;        // blocks that have keys of the unit (0: this is not the first of them)
    int pad[5];
};
static_assert(sizeof(Desc) == 64, "a stage's description");
enum : uint32_t { kUnitBegins = 1u << 16, kUnitEnds = 1u << 17, kShareEnds = 1u << 18 };  // unit: or its part here
constexpr int kWhole = -1;

template <int D, int NT, bool CAP>
__global__ void __launch_bounds__(R_THREADS, RCfg<D, NT>::OCC) kq_kv_rows_kernel(const __grid_constant__ Plan p) {
    using C = RCfg<D, NT>;
    using namespace tc;
    constexpr int R = C::R, KS = D / 16, W = D / 32;  // k steps; words of a lane's part of a key row
    extern __shared__ __align__(128) unsigned char smem[];
    const KvAttnArgs &a = p.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    const int Hk = a.c.heads, H = a.q_heads, psh = a.c.page_shift;
    // sequences of the walk: the own keys', and the prefix last
    const int64_t seqs = a.B + p.rows_prefix;
    const uint32_t sbase = smem_u32(smem);
    auto bar = [&](int i) -> uint32_t { return sbase + uint32_t(C::OFF_BAR + 8 * i); };
    volatile int *s_abort = reinterpret_cast<volatile int *>(smem + C::OFF_MISC);
    int64_t *scan = reinterpret_cast<int64_t *>(smem + C::OFF_SCAN);  // warp sums; then the block's first chunk
    if (tid == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(bar(C::FULL + s), 33);  // the loading warp's lanes once their copies have landed, and one more
            mbar_init(bar(C::EMPTY + s), WARPS);
        }
        mbar_init(bar(C::JOIN), WARPS);
        mbar_init(bar(C::JOIN + 1), WARPS);
        *s_abort = 0;
        fence_mbar_init();
    }
    begin_launch(p);
    griddep_launch_dependents();

    // ---- the block's share: chunks [w0, w1) of all ----
    const int64_t per = (seqs + R_THREADS - 1) / R_THREADS, s0 = min(per * tid, seqs), s1 = min(s0 + per, seqs);
    int64_t mine = 0;
    for (int64_t b = s0; b < s1; ++b) {
        const Seq s = load_seq<R>(p, b, blockIdx.x == 0);
        mine += int64_t(s.tiles) * (s.N + kUnitCost);
    }
    mine *= Hk;
    int64_t before = mine;
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += v;
    }
    if (lane == 31) scan[warp] = before;
    __syncthreads();
    int64_t total = 0;
    before -= mine;
    for (int w = 0; w <= WARPS; ++w) {
        if (w < warp) before += scan[w];
        total += scan[w];
    }
    if (blockIdx.x >= total) return end_launch(p);
    const Shares sh(total, p.ctas);
    const int64_t w0 = sh.begin(blockIdx.x), w1 = sh.begin(blockIdx.x + 1);
    __syncthreads();
    if (before <= w0 && w0 < before + mine) {
        int64_t at = before, b = s0;
        Seq s = load_seq<R>(p, b, false);
        while (at + int64_t(s.tiles) * (s.N + kUnitCost) * Hk <= w0) {
            at += int64_t(s.tiles) * (s.N + kUnitCost) * Hk;
            s = load_seq<R>(p, ++b, false);
        }
        // the unit of place w0, and the first chunk from there on: this unit's, as its chunks come last
        const int64_t r = w0 - at, u = r / (s.N + kUnitCost), c = r - u * (s.N + kUnitCost) - kUnitCost;
        scan[0] = b;
        scan[1] = u;
        scan[2] = c > 0 ? c : 0;
        scan[3] = w0 + (c < 0 ? -c : 0);
    }
    __syncthreads();
    if (scan[3] >= w1) return end_launch(p);  // places of a unit's start alone

    if (warp == WARPS) {
        // ---------------- the loading warp: one chunk per stage, 16 bytes a lane and copy ----------------
        // (Bulk copies of a page's part would be fewer, but a lane's own takes its own pass through the
        // instruction: 100 clocks for each, 3000 for a chunk of 16-key pages.)
        Walk<R> w;
        w.b = scan[0];
        w.s = load_seq<R>(p, w.b, false);
        w.c = w.s.c0 + int(scan[2]);
        w.tile = int(scan[1] % w.s.tiles);
        w.h = int(scan[1] / w.s.tiles);
        int64_t place = scan[3];  // of the chunk
        bool entire = w.c == w.s.c0;  // whether this block has had the unit from its first chunk on
        bool begins = true, first = true;
        constexpr int SUBS = CH / 16;
        // lane i looks up the page of the chunk's keys 16 i .. 16 i + 15; -1: not wanted
        auto page_of = [&](const Walk<R> &v) -> int {
            const int t = v.c * CH + 16 * lane;
            return lane < SUBS && t < v.s.n && t + 16 > v.s.lo ? v.s.pages[t >> psh] : -1;
        };
        int page = page_of(w);
        const uint8_t *const kc = a.c.k_codes + 16 * lane, *const vc = a.c.v_codes + 16 * lane;
        Ring rg;
        for (bool more = true; more; rg.next(C::STAGES)) {
            // the next chunk's pages are looked up while this one is copied
            Walk<R> ahead = w;
            int next_page = -1;
            const int last = w.s.c0 + w.s.N - 1;
            const int64_t next_place = place + 1 + (w.c == last ? kUnitCost : 0);
            more = next_place < w1;
            if (more) {
                ahead.next(p, seqs);
                next_page = page_of(ahead);
            }
            if (!wait_all(bar(C::EMPTY + rg.idx), rg.phase ^ 1u, s_abort, a.err)) break;
            const int t = w.c * CH + 16 * lane;
            const bool wanted = lane < SUBS && t < w.s.n && t + 16 > w.s.lo;
            const bool there = wanted && uint32_t(page) < uint32_t(a.c.pages);
            if (wanted && !there) atomicOr(a.err, kSiteKvAttention);
            const uint32_t ok = __ballot_sync(0xffffffffu, there);
            const int64_t row = there ? ((int64_t(page) * Hk + w.h) << psh) + (t & ((1 << psh) - 1)) : 0;
            const uint32_t dst = sbase + uint32_t(rg.idx * C::STAGE) + uint32_t(16 * lane);
#pragma unroll
            for (int s = 0; s < SUBS; ++s) {
                const int64_t at = __shfl_sync(0xffffffffu, row, s) * (D / 2);
                if (ok >> s & 1u) {
#pragma unroll
                    for (int k = 0; k < D / 64; ++k) {  // 16 rows of D / 2 bytes are D / 64 times 512
                        cp_async16(dst + uint32_t(s * 8 * D + 512 * k), kc + at + 512 * k);
                        cp_async16(dst + uint32_t(C::CODES + s * 8 * D + 512 * k), vc + at + 512 * k);
                    }
                }
            }
            const int64_t mine = __shfl_sync(0xffffffffu, row, lane >> 2) + 4 * (lane & 3);  // 4 keys' scales
            if (ok >> (lane >> 2) & 1u) {
                cp_async16(dst + uint32_t(2 * C::CODES), a.c.k_scale + mine);
                cp_async16(dst + uint32_t(2 * C::CODES + 4 * CH), a.c.v_scale + mine);
            }
            if (begins) {
                const int rows = min(R, w.s.m * p.G - w.tile * R), j = w.tile * R + lane, i0 = j / p.G;
                const int64_t from = (int64_t(w.s.q0 + i0) * H + w.h * p.G + (j - i0 * p.G)) * D;
                constexpr int PIECES = D / 8;  // 16-byte pieces of a query row
#pragma unroll
                for (int k = 0; k < R * PIECES / 32; ++k) {
                    const int r = (32 * k + lane) / PIECES;
                    const int64_t at = __shfl_sync(0xffffffffu, from, r);
                    if (r < rows)
                        cp_async16(dst + uint32_t(C::Q + 512 * k), a.q + at + 8 * (lane % PIECES));
                }
            }
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar(C::FULL + rg.idx)) : "memory");
            const bool ends = w.c == last || !more;
            if (lane == 0) {
                Desc *d = reinterpret_cast<Desc *>(smem + C::OFF_DESC + 64 * rg.idx);
                const uint32_t flags = ok | (begins ? uint32_t(kUnitBegins) : 0u) | (ends ? uint32_t(kUnitEnds) : 0u) |
                                       (more ? 0u : uint32_t(kShareEnds));
                *reinterpret_cast<int4 *>(d) = make_int4(w.c * CH, w.s.n, int(flags), w.s.shift);
                if (begins || ends) {
                    *reinterpret_cast<int4 *>(&d->q0) = make_int4(w.s.q0, w.s.m, w.h, w.tile);
                    d->place = entire && w.c == last ? kWhole : int(blockIdx.x) * 2 + (first && !entire ? 0 : 1);
                    d->prefix = w.b == a.B;
                    d->parts =
                        !entire ? 0 : w.c == last ? 1 : ends ? sh.block_of(place + last - w.c) - int(blockIdx.x) + 1 : 0;
                }
                mbar_arrive(bar(C::FULL + rg.idx));
            }
            w = ahead;
            page = next_page;
            place = next_place;
            begins = w.c == w.s.c0;
            if (begins) {
                entire = true;
                first = false;
            }
        }
        cp_async_wait_all();  // every copy in flight lands before the block may end
        return;
    }

    // ---------------- the multiplying warps: 16 MT keys of every chunk each ----------------
    // Row r of a tile is key order(r) of its 16: so that a lane's key rows, and the
    // rows 2c, 2c + 1 of values, start in different banks (rows are 64 or 32 bytes).
    auto order = [](int r) { return r ^ ((r >> 1) & 1); };
    float o[NT][D / 16][4];
    uint32_t qf[NT][KS][2];
    float mult[NT][2], start[NT][2], ref[NT][2], sum[NT][2];
    int lo[NT][2], hi[NT][2];    // keys that the rows of this lane's columns see: [lo, hi)
    int lo_all = 0, hi_all = 0;  // keys that all rows see
    uint32_t seen = 0;           // columns whose reference is set, one bit each; all once
    constexpr uint32_t kAllSeen = (1u << 2 * NT) - 1;
    Ring rg;
    uint32_t joins = 0;
    const int og = order(g);
    for (bool more = true; more; rg.next(C::STAGES)) {
        if (!wait_all(bar(C::FULL + rg.idx), rg.phase, s_abort, a.err)) break;
        const Desc *desc = reinterpret_cast<const Desc *>(smem + C::OFF_DESC + 64 * rg.idx);
        const uint32_t flags = desc->flags;
        more = (flags & kShareEnds) == 0;
        if (flags & kUnitBegins) {
            // ---- a unit begins: its queries ----
            const int q0 = desc->q0, m = desc->m, tile = desc->tile, shift = desc->shift, n = desc->n;
            lo_all = 0;
            hi_all = INT_MAX;
            seen = 0;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int j = tile * R + 8 * nt + g;
                const bool real = j < m * p.G;
                const int i = real ? j / p.G : 0;
                const unsigned char *qr = smem + rg.idx * C::STAGE + C::Q + (8 * nt + g) * D * 2 + c * (D / 2);
                uint4 v[W];
                float big = 0.0f;
#pragma unroll
                for (int w = 0; w < W; ++w) {  // eight consecutive elements per word of codes
                    v[w] = real ? *reinterpret_cast<const uint4 *>(qr + 16 * w) : make_uint4(0, 0, 0, 0);
                    const uint32_t u[4] = {v[w].x, v[w].y, v[w].z, v[w].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        big = fmaxf(big, fmaxf(fabsf(__uint_as_float(u[e] << 16)), fabsf(__uint_as_float(u[e] & 0xffff0000u))));
                }
                big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
                big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
                // 2^(14 - e) for a largest element in [2^e, 2^(e + 1)): it stays under 2^15
                const int e = int(__float_as_uint(big) >> 23) - 127;
                const int up = big > 0.0f && e < 128 ? min(14 - e, 120) : 0;
                const float f = __uint_as_float(uint32_t(up + 127) << 23);
                float tot = 0.0f;
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    const uint32_t u[4] = {v[w].x, v[w].y, v[w].z, v[w].w};
                    float x[8];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        x[2 * k] = __uint_as_float(u[k] << 16) * f;
                        x[2 * k + 1] = __uint_as_float(u[k] & 0xffff0000u) * f;
                    }
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const uint32_t b0 = pack_f16x2(x[2 * k], x[2 * k + 4]);
                        const uint32_t b1 = pack_f16x2(x[2 * k + 1] * 0.0625f, x[2 * k + 5] * 0.0625f);
                        qf[nt][2 * w + k][0] = b0;
                        qf[nt][2 * w + k][1] = b1;
                        const float2 y0 = __half22float2(*reinterpret_cast<const __half2 *>(&b0));
                        const float2 y1 = __half22float2(*reinterpret_cast<const __half2 *>(&b1));
                        tot += (y0.x + y0.y) + 16.0f * (y1.x + y1.y);
                    }
                }
                tot += __shfl_xor_sync(0xffffffffu, tot, 1);
                tot += __shfl_xor_sync(0xffffffffu, tot, 2);
                // The score's multiplier: the softmax scale, and what the operands were scaled by.
                const float back = __uint_as_float(uint32_t(127 - up) << 23);  // 1 / f
                float mul = (CAP ? a.scale / a.softcap : a.scale * kLog2e) * back * 0x1p24f;
                // a zero score is one under any scale; a cap far under the scores is passed at 2^100 as anywhere
                if (big == 0.0f) mul = 0.0f;
                if (CAP) mul = fminf(fmaxf(mul, -0x1p100f), 0x1p100f);
                int rl = 0, rh = 0;
                if (real) {
                    rh = min(n, max(0, shift + i + 1));
                    if (a.window) {
                        const int64_t pos =
                            desc->prefix ? a.prefix_len + query_shift(a, q0 + i) : int64_t(shift) + i;
                        rl = int(min(int64_t(rh), max(int64_t(0), pos - a.window + 1)));
                    }
                }
                // rows lie in the lanes of group g; the scores' columns in those of c
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int src = 4 * (2 * c + k);
                    mult[nt][k] = __shfl_sync(0xffffffffu, mul, src);
                    start[nt][k] = __shfl_sync(0xffffffffu, tot, src) * (-8.0f * 0x1p-24f);
                    lo[nt][k] = __shfl_sync(0xffffffffu, rl, src);
                    hi[nt][k] = __shfl_sync(0xffffffffu, rh, src);
                    ref[nt][k] = 0.0f;
                    sum[nt][k] = 0.0f;
                    if (lo[nt][k] >= hi[nt][k]) seen |= 1u << (2 * nt + k);  // nothing to see
                }
                // rows past the last one see nothing, and are not looked at
                lo_all = max(lo_all, __reduce_max_sync(0xffffffffu, real ? rl : 0));
                hi_all = min(hi_all, __reduce_min_sync(0xffffffffu, real ? rh : INT_MAX));
#pragma unroll
                for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
                    for (int k = 0; k < 4; ++k) o[nt][mt][k] = 0.0f;
            }
        }
        constexpr uint32_t kMine = (1u << MT) - 1;
        const uint32_t mine_ok = flags >> (MT * warp) & kMine;
        if (mine_ok) {
            const int t0 = desc->t0 + 16 * MT * warp;
            const unsigned char *st = smem + rg.idx * C::STAGE + 16 * MT * warp * (D / 2);
            const float *sc = reinterpret_cast<const float *>(smem + rg.idx * C::STAGE + 2 * C::CODES) + 16 * MT * warp;
            // ---- scores: S^T[key][row] ----
            float x[MT][NT][4], ks[MT][2], lv[MT][2];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    x[mt][nt][0] = x[mt][nt][2] = start[nt][0];
                    x[mt][nt][1] = x[mt][nt][3] = start[nt][1];
                }
                uint32_t k0[W], k1[W];  // this lane's parts of the key rows g and g + 8
                const unsigned char *kt = st + 16 * mt * (D / 2);
                if constexpr (D == 128) {
                    const uint4 u = *reinterpret_cast<const uint4 *>(kt + 64 * og + 16 * c);
                    const uint4 v = *reinterpret_cast<const uint4 *>(kt + 64 * (og + 8) + 16 * c);
                    k0[0] = u.x, k0[1] = u.y, k0[2] = u.z, k0[3] = u.w;
                    k1[0] = v.x, k1[1] = v.y, k1[2] = v.z, k1[3] = v.w;
                } else {
                    const uint2 u = *reinterpret_cast<const uint2 *>(kt + 32 * og + 8 * c);
                    const uint2 v = *reinterpret_cast<const uint2 *>(kt + 32 * (og + 8) + 8 * c);
                    k0[0] = u.x, k0[1] = u.y;
                    k1[0] = v.x, k1[1] = v.y;
                }
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    ks[mt][k] = sc[16 * mt + og + 8 * k];
                    // an infinite scale as 2^128, so that a score of -inf leaves that key out too
                    lv[mt][k] = fminf(lg2(sc[CH + 16 * mt + og + 8 * k]), 128.0f);
                }
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    const uint32_t u = k0[w], v = k1[w], u8 = u >> 8, v8 = v >> 8;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma_f16(x[mt][nt], nib_lo(u), nib_lo(v), nib_hi(u), nib_hi(v), qf[nt][2 * w][0], qf[nt][2 * w][1]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma_f16(x[mt][nt], nib_lo(u8), nib_lo(v8), nib_hi(u8), nib_hi(v8), qf[nt][2 * w + 1][0],
                                qf[nt][2 * w + 1][1]);
                }
            }
            // ---- weights ----
            const bool inner = mine_ok == kMine && t0 >= lo_all && t0 + 16 * MT <= hi_all;
            if (!inner) {  // past the last key a page may hold anything
                const int n = desc->n;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    const int left = mine_ok >> mt & 1u ? n - t0 - 16 * mt : 0;
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        if (og + 8 * k >= left) ks[mt][k] = lv[mt][k] = 0.0f;
                }
            }
            // For the reference a scale under 2^-100, or of 0 (a row of zeros), counts as 2^-100: the sum of exp(x)
            // is relative to the same reference and must not pass fp32's range.
            auto floored = [](float l) { return fmaxf(l, -100.0f); };
            float top = -INFINITY;  // of a weight's exponent
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float f = ks[mt][k >> 1] * mult[nt][k & 1];
                        if (CAP) x[mt][nt][k] *= f;
                        else x[mt][nt][k] = fmaf(x[mt][nt][k], f, -ref[nt][k & 1]);
                    }
            if constexpr (CAP) {
                const uint64_t cap = pair2(a.softcap * kLog2e, a.softcap * kLog2e);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float(&y)[4] = x[mt][nt];
                        uint64_t z0 = pair2(y[0], y[1]), z1 = pair2(y[2], y[3]);
                        tanh_pairs(z0, z1);
                        const uint64_t minus = pair2(-ref[nt][0], -ref[nt][1]);
                        split2(fma2(z0, cap, minus), y[0], y[1]);
                        split2(fma2(z1, cap, minus), y[2], y[3]);
                    }
            }
            if (!inner) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int t = mine_ok >> mt & 1u ? t0 + 16 * mt + og + 8 * k : INT_MAX;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int j = 0; j < 2; ++j)
                                if (t < lo[nt][j] || t >= hi[nt][j]) x[mt][nt][2 * k + j] = -INFINITY;
                    }
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    top = fmax3(top, fmaxf(x[mt][nt][0], x[mt][nt][1]) + floored(lv[mt][0]),
                                fmaxf(x[mt][nt][2], x[mt][nt][3]) + floored(lv[mt][1]));
            if (__any_sync(0xffffffffu, top > 14.0f || seen != kAllSeen)) {
                // move the references to 6 under the maxima so far
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        float up = -INFINITY;
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt)
                            up = fmax3(up, x[mt][nt][k] + floored(lv[mt][0]), x[mt][nt][k + 2] + floored(lv[mt][1]));
                        up = fmaxf(up, __shfl_xor_sync(0xffffffffu, up, 4));
                        up = fmaxf(up, __shfl_xor_sync(0xffffffffu, up, 8));
                        up = fmaxf(up, __shfl_xor_sync(0xffffffffu, up, 16));
                        const bool was = seen >> (2 * nt + k) & 1u;
                        // a row's first keys set its reference, later ones may only raise it
                        if (up > -INFINITY) seen |= 1u << (2 * nt + k);
                        up = was ? fmaxf(up - 6.0f, 0.0f) : up > -INFINITY ? up - 6.0f : 0.0f;
                        const float f = was ? ex2(-up) : 1.0f;
                        ref[nt][k] += up;
                        sum[nt][k] *= f;
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) {
                            x[mt][nt][k] -= up;
                            x[mt][nt][k + 2] -= up;
                        }
#pragma unroll
                        for (int e = 0; e < D / 16; ++e) {
                            o[nt][e][k] *= f;
                            o[nt][e][k + 2] *= f;
                        }
                    }
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                uint32_t pf[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float w[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        sum[nt][k & 1] += ex2(x[mt][nt][k]);
                        w[k] = ex2(x[mt][nt][k] + lv[mt][k >> 1]);
                    }
                    pf[nt][0] = transpose8x8(pack_f16x2(w[0], w[1]));
                    pf[nt][1] = transpose8x8(pack_f16x2(w[2], w[3]));
                }
                // ---- values: O^T[element][row] += codes^T weights ----
                // this lane's elements: D / 8 from g D / 8 on, of the tile's rows 2c, 2c + 1 and 2c + 8, 2c + 9
                const unsigned char *vt = st + C::CODES + 16 * mt * (D / 2);
                uint32_t v[4][D / 64];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int r = order(2 * c + (k & 1)) + 8 * (k >> 1);
                    if constexpr (D == 128) {
                        const uint2 u = *reinterpret_cast<const uint2 *>(vt + 64 * r + 8 * g);
                        v[k][0] = u.x, v[k][1] = u.y;
                    } else {
                        v[k][0] = *reinterpret_cast<const uint32_t *>(vt + 32 * r + 4 * g);
                    }
                }
#pragma unroll
                for (int w = 0; w < D / 64; ++w)
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        // nibbles 4 half .. 4 half + 3 of the word, of a pair of keys
                        const uint32_t sel = half ? 0x7632u : 0x5410u;
                        const uint32_t u = __byte_perm(v[0][w], v[1][w], sel), y = __byte_perm(v[2][w], v[3][w], sel);
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            const uint32_t us = q ? u >> 8 : u, ys = q ? y >> 8 : y;
                            constexpr uint32_t kEight = 0x80088008u, kOne = 0x3c003c00u, kSixteenth = 0x2c002c00u;
                            const uint32_t a0 = hfma2(nib_lo(us), kOne, kEight);
                            const uint32_t a1 = hfma2(nib_hi(us), kSixteenth, kEight);
                            const uint32_t a2 = hfma2(nib_lo(ys), kOne, kEight);
                            const uint32_t a3 = hfma2(nib_hi(ys), kSixteenth, kEight);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                mma_f16(o[nt][4 * w + 2 * half + q], a0, a1, a2, a3, pf[nt][0], pf[nt][1]);
                        }
                    }
            }
        }

        // ---- the unit's end, or the share's: join the warps ----
        if (flags & kUnitEnds) {
            // the parts are free once all warps have read the last unit's
            if (joins && !wait_all(bar(C::JOIN + 1), (joins - 1) & 1u, s_abort, a.err)) break;
            float *part = reinterpret_cast<float *>(smem + C::OFF_PART + warp * C::PART);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int row = 8 * nt + 2 * c + k;
                    float l = sum[nt][k];
                    l += __shfl_xor_sync(0xffffffffu, l, 4);
                    l += __shfl_xor_sync(0xffffffffu, l, 8);
                    l += __shfl_xor_sync(0xffffffffu, l, 16);
                    if (g == 0) {
                        part[R * C::PROW + row] = l == 0.0f ? kNone : ref[nt][k];
                        part[R * C::PROW + R + row] = l;
                    }
#pragma unroll
                    for (int mt = 0; mt < D / 16; ++mt) {
                        // elements g D / 8 + 2 mt, + 1, where lanes write without conflicts
                        *reinterpret_cast<float2 *>(part + row * C::PROW + 16 * mt + 2 * g) =
                            make_float2(o[nt][mt][k], o[nt][mt][k + 2]);
                    }
                }
            }
            const int q0 = desc->q0, h = desc->h, tile = desc->tile, place = desc->place;
            const int rows = min(R, desc->m * p.G - tile * R);
            const int64_t whole_at = desc->prefix ? a.T * H : 0;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::JOIN));
            const int parts = desc->parts;
            int2 *rec = p.parts + whole_at;
            if (!wait_all(bar(C::JOIN), joins & 1u, s_abort, a.err)) break;
            const float *all = reinterpret_cast<const float *>(smem + C::OFF_PART);
            for (int u = tid; u < rows * (D / 4); u += 32 * WARPS) {
                const int row = u / (D / 4), d = 4 * (u % (D / 4));
                float top = kNone;
#pragma unroll
                for (int w = 0; w < WARPS; ++w) top = fmaxf(top, all[w * (C::PART / 4) + R * C::PROW + row]);
                float l = 0.0f;
                float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                for (int w = 0; w < WARPS; ++w) {
                    const float *q = all + w * (C::PART / 4);
                    const float f = ex2(q[R * C::PROW + row] - top);
                    const int at = row * C::PROW + 8 * (d % (D / 8)) + 2 * (d / (D / 8));
                    const float2 y = *reinterpret_cast<const float2 *>(q + at);
                    const float2 z = *reinterpret_cast<const float2 *>(q + at + 16);
                    l += q[R * C::PROW + R + row] * f;
                    v.x += y.x * f, v.y += y.y * f, v.z += z.x * f, v.w += z.y * f;
                }
                const float inv = l > 0.0f ? 0x1p24f / l : l == 0.0f ? 0.0f : l;
                const float lse = l == 0.0f ? -INFINITY : top + lg2(l);  // in powers of two
                const int j = tile * R + row, i = j / p.G;
                const int64_t at = int64_t(q0 + i) * H + h * p.G + (j - i * p.G);
                v.x *= inv, v.y *= inv, v.z *= inv, v.w *= inv;
                if (d == 0 && parts) rec[at] = make_int2(blockIdx.x, parts);
                if (place == kWhole && !p.partial) {
                    *reinterpret_cast<uint2 *>(a.out + at * D + d) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
                    if (a.lse && d == 0) a.lse[at] = lse * 0.6931471805599453f;
                } else {
                    const int64_t k = place == kWhole ? whole_at + at : int64_t(place) * R + row;
                    *reinterpret_cast<float4 *>((place == kWhole ? p.whole_o : p.slot_o) + k * D + d) = v;
                    if (d == 0) (place == kWhole ? p.whole_l : p.slot_l)[k] = lse;
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::JOIN + 1));
            ++joins;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::EMPTY + rg.idx));
    }
    end_launch(p);
}

// ---- joining partial rows ---------------------------------------------------------
// A row's parts are the slots of the blocks that its unit was cut over, in order; behind a
// prefix, those of both units.  WARPS_PER_ROW = 1: four rows per block, or 4: one, its warps
// taking every fourth part (few rows, each cut over many blocks).  A warp's lanes first read
// the parts' sums, 32 at a time, then add up the parts' values with the weights that result.
template <int D, int R, int WARPS_PER_ROW>
__global__ void __launch_bounds__(128) kq_kv_combine_kernel(const __grid_constant__ Plan p) {
    __shared__ float so[4][D], sl[4], sw[4];
    const KvAttnArgs &a = p.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, H = a.q_heads;
    griddep_wait();
    griddep_launch_dependents();
    const int64_t rows = a.T * H;
    const int64_t at = WARPS_PER_ROW == 4 ? blockIdx.x : int64_t(blockIdx.x) * 4 + warp;
    const bool real = at < rows && at < int64_t(all_queries(a)) * H;  // not padding behind the last sequence
    if (!real) return;
    const int t = int(at / H), g = int(at - int64_t(t) * H) % p.G;
    // own keys: parts of the row kernel (as its records say) or of the tile kernel, and so for the prefix's
    int2 rec0 = make_int2(0, p.own_splits), rec1 = make_int2(0, p.pre_splits);
    int row0 = 0, row1 = 0;
    if (p.rows_own) rec0 = p.parts[at];
    if (p.rows_prefix) rec1 = p.parts[rows + at];
    auto sound = [&](const int2 &r) { return r.y >= 1 && r.y <= p.ctas && r.x >= 0 && r.x <= p.ctas - r.y; };
    const bool tiled = p.few && rec0.x == -1 && rec0.y == p.own_splits, rows_own = p.rows_own && !tiled;
    if ((rows_own && !sound(rec0)) || (p.rows_prefix && !sound(rec1))) return;  // a row past the bound on queries
    if (!p.partial && p.rows_own && rec0.y == 1) return;  // written by its block
    const int n = rec0.y + rec1.y;
    const bool cut0 = rows_own && rec0.y > 1, cut1 = p.rows_prefix && rec1.y > 1;
    if (cut0 || cut1 || !rows_own) {  // the row's place in its unit's tile; whether it is bounded away
        const int i = a.q_start ? t - a.q_start[seq_of(a, t)] : 0;  // the query's number in its sequence
        if (i < 0 || i >= a.max_q) return;
        row0 = (i * p.G + g) % R;
        row1 = (t * p.G + g) % R;
    }
    // Where part k lies: the rows and sums that it is among, and its index there.
    auto place = [&](int k, const float *&o, const float *&l) -> int64_t {
        const int u = k >= rec0.y;
        const int i = u ? k - rec0.y : k;
        if (u ? !p.rows_prefix : !rows_own) {
            o = p.tile_o, l = p.tile_l;
            return int64_t((u ? p.own_splits : 0) + i) * rows + at;
        }
        const int2 rec = u ? rec1 : rec0;
        if (rec.y == 1) {
            o = p.whole_o, l = p.whole_l;
            return u * rows + at;
        }
        o = p.slot_o, l = p.slot_l;
        // a unit's first block holds it as its last unit, the others as their first
        return (int64_t(rec.x + i) * 2 + (i == 0 ? 1 : 0)) * R + (u ? row1 : row0);
    };
    float top = -INFINITY, wsum = 0.0f;
    float v[D / 32];
#pragma unroll
    for (int e = 0; e < D / 32; ++e) v[e] = 0.0f;
    const int first = WARPS_PER_ROW == 4 ? warp : 0;
    for (int k0 = first; k0 < n; k0 += 32 * WARPS_PER_ROW) {
        const int mine = k0 + lane * WARPS_PER_ROW;
        float l = -INFINITY;
        const float *src = p.slot_o;
        if (mine < n) {
            const float *sums;
            const int64_t from = place(mine, src, sums);
            src += from * D;
            l = sums[from];
        }
        // the first parts' values are on their way before the sums are known
        constexpr int AHEAD = 4;
        const int cnt = min(32, (n - k0 + WARPS_PER_ROW - 1) / WARPS_PER_ROW);
        auto value = [&](int k) {
            const float *sk = reinterpret_cast<const float *>(
                __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(src), k));
            if constexpr (D == 128) return reinterpret_cast<const float4 *>(sk)[lane];
            else return reinterpret_cast<const float2 *>(sk)[lane];
        };
        decltype(value(0)) z[AHEAD];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k)
            if (k < cnt) z[k] = value(k);
        float m = l;
#pragma unroll
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float nt = fmaxf(top, m);
        float w = l == -INFINITY ? 0.0f : ex2(l - nt);
        const float f = top == -INFINITY ? 0.0f : ex2(top - nt);
        top = nt;
        float s = w;
#pragma unroll
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        wsum = wsum * f + s;
#pragma unroll
        for (int e = 0; e < D / 32; ++e) v[e] *= f;
        auto add = [&](int k, const auto &y) {
            const float wk = __shfl_sync(0xffffffffu, w, k);  // 0 for a part without keys, whose values may be anything
            if (wk == 0.0f) return;
            v[0] = fmaf(y.x, wk, v[0]), v[1] = fmaf(y.y, wk, v[1]);
            if constexpr (D == 128) v[2] = fmaf(y.z, wk, v[2]), v[3] = fmaf(y.w, wk, v[3]);
        };
#pragma unroll
        for (int k = 0; k < AHEAD; ++k)
            if (k < cnt) add(k, z[k]);
#pragma unroll 4
        for (int k = AHEAD; k < cnt; ++k) add(k, value(k));
    }
    if constexpr (WARPS_PER_ROW == 4) {
#pragma unroll
        for (int e = 0; e < D / 32; ++e) so[warp][lane * (D / 32) + e] = v[e];
        if (lane == 0) sl[warp] = top, sw[warp] = wsum;
        __syncthreads();
        if (warp) return;
        top = fmaxf(fmaxf(sl[0], sl[1]), fmaxf(sl[2], sl[3]));
        wsum = 0.0f;
#pragma unroll
        for (int e = 0; e < D / 32; ++e) v[e] = 0.0f;
        for (int k = 0; k < 4; ++k) {
            if (sw[k] == 0.0f) continue;  // no part with a key
            const float f = ex2(sl[k] - top);
            wsum += sw[k] * f;
#pragma unroll
            for (int e = 0; e < D / 32; ++e) v[e] += so[k][lane * (D / 32) + e] * f;
        }
    }
    const float inv = wsum == 0.0f ? 0.0f : 1.0f / wsum;
    uint32_t *out = reinterpret_cast<uint32_t *>(a.out + at * D) + lane * (D / 64);
#pragma unroll
    for (int e = 0; e < D / 64; ++e) out[e] = pack_bf16x2(v[2 * e] * inv, v[2 * e + 1] * inv);
    if (lane == 0 && a.lse) a.lse[at] = wsum == 0.0f ? -INFINITY : (top + lg2(wsum)) * 0.6931471805599453f;
}

// ---- host side ------------------------------------------------------------------------

constexpr int kMaxCtas = 4 * 160;  // blocks of the row kernel, at most
constexpr int kSms = 148;          // of a B200; the tile kernel has one block on each

int row_tile(int64_t rows) { return rows <= 8 ? 8 : 16; }

// Whether the rows of a key head and sequence, or of a key head and the prefix, are the tile kernel's.  The
// row kernel reads the codes again (from L2) for every 8 or 16 rows; the tile kernel works on up to 256 at
// once but has one block an SM and a longer way to its first product.  Measured in us, row against tile
// kernel, head_dim 128, 24 sequences of 100 to 4100 keys on 4 key heads: 20 rows 28 against 41, 40 rows 35
// against 42, 64 rows 50 against 46.  A prefix on 8 key heads: 32 rows 17 against 19 (1000 keys) and 28
// against 29 (8000), 64 rows 20 against 21 (1000) but 70 against 37 (16000).
// (All at head_dim 128; at 64 nothing was measured, and the prefix's length is not asked.)
constexpr int kManyRows = 48;
bool many_rows(int64_t rows) { return rows > kManyRows; }
bool many_prefix_rows(int64_t rows) { return rows > 32; }

// Blocks to cut a unit's keys over, where there are too few units for all SMs, up to two rounds of blocks:
// the number that ends first, a block being as long as its chunks and four more (its start and its rows'
// end: some 17000 clocks, where a chunk takes 4500), and a part to join a third of one.
int most_splits(int64_t units) { return units < 2 * kSms ? int(2 * kSms / units < 32 ? 2 * kSms / units : 32) : 1; }
int tile_splits(int64_t units, int64_t chunks) {
    int best = 1;
    double least = 0.0;
    for (int s = 1; s <= most_splits(units) && s <= chunks; ++s) {
        const double rounds = double((units * s + kSms - 1) / kSms);
        const double cost = rounds * (4.0 + double((chunks + s - 1) / s)) + 0.33 * s;
        if (s == 1 || cost < least) best = s, least = cost;
    }
    return best;
}

uint64_t align256(uint64_t x) { return (x + 255) & ~uint64_t(255); }

// Who does what, and the workspace's parts from `base`; returns the bytes.  `own_most`, `pre_most`: chunks
// that a sequence, the prefix have at most (parts are no more; the sizes are laid out for any number).
uint64_t lay_out(Plan &p, unsigned char *base, int64_t T, int64_t B, int H, int Hk, int D, int max_q, int64_t own_most,
                 int64_t pre_most) {
    const int G = H / Hk;
    p.G = G;
    const bool own_tile = many_rows(int64_t(max_q) * G), pre_tile = own_tile || many_prefix_rows(T * G);
    // Sequences that are far from even, as prompts and single tokens at once: those with few rows are the row
    // kernel's.  (8 key heads of 4, us with both kernels against the tile kernel alone: 1024 queries of one
    // sequence and 63 single ones on 2000 keys each 129 against 203, 512 and 255 on 1000 155 against 368, 1024
    // and 15 on 2000 86 against 84.)  Of the others, the units to expect:
    p.few = own_tile && T * 5 < B * max_q * 3 ? kManyRows : 0;
    const int64_t places = kv_own_tiles(T, B, max_q, G, p.few);
    const int64_t expect = kv_tiles(max_q, G) + kv_own_tiles(T - max_q, B - 1, max_q, G, p.few);
    const int64_t own_units = (expect < places ? expect : places) * Hk;
    const int own = own_tile ? most_splits(own_units) : 0;
    const int pre = pre_tile ? most_splits(kv_tiles(T, G) * Hk) : 0;
    p.own_splits = own_tile ? tile_splits(own_units, own_most) : 0;
    p.pre_splits = pre_most && pre_tile ? tile_splits(kv_tiles(T, G) * Hk, pre_most) : 0;
    p.rows_own = !own_tile || p.few;
    p.rows_prefix = pre_most && !pre_tile;
    p.partial = pre_most > 0;
    const int R = row_tile(int64_t(max_q) * G);
    const uint64_t rows = uint64_t(T) * H;
    uint64_t at = 0;
    auto take = [&](uint64_t bytes) {
        unsigned char *r = base + at;
        at += align256(bytes);
        return r;
    };
    p.parts = reinterpret_cast<int2 *>(take(rows * 2 * 8));
    p.slot_o = reinterpret_cast<float *>(take(!p.rows_own ? 0 : uint64_t(kMaxCtas) * 2 * R * D * 4));
    p.slot_l = reinterpret_cast<float *>(take(!p.rows_own ? 0 : uint64_t(kMaxCtas) * 2 * R * 4));
    p.whole_o = reinterpret_cast<float *>(take(!p.rows_own ? 0 : rows * 2 * D * 4));
    p.whole_l = reinterpret_cast<float *>(take(!p.rows_own ? 0 : rows * 2 * 4));
    p.tile_o = reinterpret_cast<float *>(take(uint64_t(own + pre) * rows * D * 4));
    p.tile_l = reinterpret_cast<float *>(take(uint64_t(own + pre) * rows * 4));
    return at;
}

template <int D, int R>
cudaError_t launch_combine(const Plan &p, cudaStream_t stream) {
    const int64_t rows = p.a.T * p.a.q_heads;
    return rows <= 2048 ? launch_overlapped(kq_kv_combine_kernel<D, R, 4>, unsigned(rows), 128, 0, stream, p)
                        : launch_overlapped(kq_kv_combine_kernel<D, R, 1>, unsigned((rows + 3) / 4), 128, 0, stream, p);
}

template <int D, int NT, bool CAP>
cudaError_t launch_rows(Plan &p, int num_sms, int device, cudaStream_t stream) {
    using C = RCfg<D, NT>;
    auto kern = kq_kv_rows_kernel<D, NT, CAP>;
    static std::once_flag once[64];
    static cudaError_t attr_err[64];
    if (device < 0 || device >= 64) return cudaErrorInvalidDevice;
    std::call_once(once[device], [&] {
        attr_err[device] = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    });
    if (attr_err[device] != cudaSuccess) return attr_err[device];
    p.ctas = num_sms * C::OCC < kMaxCtas ? num_sms * C::OCC : kMaxCtas;
    return launch_overlapped(kern, unsigned(p.ctas), R_THREADS, C::SMEM, stream, p);
}

template <int D, int NT>
cudaError_t launch_all(Plan &p, int num_sms, int device, cudaStream_t stream) {
    cudaError_t e = cudaSuccess;
    p.ctas = 0;
    p.later = 0;
    if (p.own_splits) {
        e = launch_kv_tile(p, false, p.own_splits, device, stream);
        p.later = 1;
    }
    if (e == cudaSuccess && p.rows_own) {
        e = p.a.softcap > 0.0f ? launch_rows<D, NT, true>(p, num_sms, device, stream)
                               : launch_rows<D, NT, false>(p, num_sms, device, stream);
        p.later = 1;
    }
    if (e == cudaSuccess && p.pre_splits) e = launch_kv_tile(p, true, p.pre_splits, device, stream);
    if (e != cudaSuccess || (!p.rows_own && !p.partial && p.own_splits == 1)) return e;
    return launch_combine<D, 8 * NT>(p, stream);
}

}  // namespace

uint64_t kv_attention_workspace_bytes(int64_t T, int64_t B, int q_heads, int kv_heads, int head_dim, int max_q) {
    Plan p;
    return lay_out(p, nullptr, T, B, q_heads, kv_heads, head_dim, max_q, 1, 1);
}

cudaError_t launch_kv_attention(const KvAttnArgs &a, int num_sms, int device, cudaStream_t stream) {
    Plan p;
    p.a = a;
    const int64_t own_most = ((a.max_pages << a.c.page_shift) + CH - 1) / CH;
    const int64_t pre_most = a.prefix_pages ? (a.prefix_len + CH - 1) / CH : 0;
    lay_out(p, a.workspace, a.T, a.B, a.q_heads, a.c.heads, a.c.D, a.max_q, own_most, pre_most);
    const bool one = row_tile(int64_t(a.max_q) * p.G) == 8;
    if (a.c.D == 128)
        return one ? launch_all<128, 1>(p, num_sms, device, stream) : launch_all<128, 2>(p, num_sms, device, stream);
    return one ? launch_all<64, 1>(p, num_sms, device, stream) : launch_all<64, 2>(p, num_sms, device, stream);
}

}  // namespace kq
