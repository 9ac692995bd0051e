// kq_kv_attention.cu -- softmax attention over the pages of the INT4 key / value
// cache, behind a prefix that all sequences share or none.
#include "kq_common.cuh"
#include "kq_internal.h"

namespace kq {
namespace {

constexpr int S_THREADS = 128;

// One query row and head per block: a thread per key for the scores, a thread per
// output element for the values, 128 keys at a time with a running maximum and sum.
template <int D>
__global__ void __launch_bounds__(S_THREADS) kq_kv_attention_kernel(const __grid_constant__ KvAttnArgs a) {
    __shared__ float qs[D], ps[S_THREADS], red[8];
    __shared__ int64_t row_of[S_THREADS];
    const int tid = threadIdx.x, H = a.q_heads, Hk = a.c.heads;
    griddep_wait();
    griddep_launch_dependents();
    const int h = int(blockIdx.x % H), kh = h / (H / Hk);
    const int64_t t = blockIdx.x / H;
    int64_t b = t;
    int m = 1, i = 0;
    if (a.q_start) {
        int64_t lo = 0, hi = a.B;  // the sequence whose rows hold t
        while (lo < hi) {
            const int64_t mid = (lo + hi) / 2;
            if (a.q_start[mid + 1] <= t) lo = mid + 1;
            else hi = mid;
        }
        if (lo == a.B) return;
        b = lo;
        m = a.q_start[b + 1] - a.q_start[b];
        i = int(t - a.q_start[b]);
    }
    if (i >= a.max_q) {
        if (tid == 0) atomicOr(a.err, kSiteKvAttention);
        return;
    }
    const int psize = 1 << a.c.page_shift;
    int64_t n = a.kv_len[b] > 0 ? a.kv_len[b] : 0;
    if (n > a.max_pages * psize) {
        if (tid == 0) atomicOr(a.err, kSiteKvAttention);
        n = a.max_pages * psize;
    }
    const int64_t n_given = a.kv_len[b] > 0 ? a.kv_len[b] : 0;
    if (tid < D) qs[tid] = bf16_bits_to_float(a.q[(t * H + h) * D + tid]);
    const int64_t pos = a.prefix_len + n_given - m + i;
    const int64_t low = a.window ? pos - a.window + 1 : 0;
    float top = -INFINITY, sum = 0.0f, acc = 0.0f;
    const int64_t total = a.prefix_len + n;
    for (int64_t k0 = 0; k0 < total; k0 += S_THREADS) {
        __syncthreads();
        const int64_t k = k0 + tid;
        bool see = k < total && k >= low && (k < a.prefix_len || k <= pos);
        int64_t row = 0;
        if (see) {
            const bool pre = k < a.prefix_len;
            const int64_t kk = pre ? k : k - a.prefix_len;
            const int64_t page = pre ? a.prefix_pages[kk >> a.c.page_shift]
                                     : a.page_table[b * a.max_pages + (kk >> a.c.page_shift)];
            if (page < 0 || page >= a.c.pages) {
                see = false;
                atomicOr(a.err, kSiteKvAttention);
            } else {
                row = (page * Hk + kh) * psize + (kk & (psize - 1));
            }
        }
        float x = -INFINITY;
        if (see) {
            float d = 0.0f;
            for (int e = 0; e < D / 2; ++e) {
                const int c = a.c.k_codes[row * (D / 2) + e];
                d += qs[2 * e] * float(int(uint32_t(c) << 28) >> 28) + qs[2 * e + 1] * float(int(uint32_t(c) << 24) >> 28);
            }
            x = d * a.c.k_scale[row] * a.scale;
            if (a.softcap > 0.0f) x = a.softcap * tanhf(x / a.softcap);
        }
        float mx = x;
        for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        if ((tid & 31) == 0) red[tid >> 5] = mx;
        __syncthreads();
        mx = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
        const float nt = fmaxf(top, mx);
        if (nt == -INFINITY) continue;
        const float fix = expf(top - nt), p = expf(x - nt);
        top = nt;
        ps[tid] = see ? p * a.c.v_scale[row] : 0.0f;
        row_of[tid] = row;
        float sm = p;
        for (int o = 16; o; o >>= 1) sm += __shfl_xor_sync(0xffffffffu, sm, o);
        if ((tid & 31) == 0) red[4 + (tid >> 5)] = sm;
        __syncthreads();
        sum = sum * fix + red[4] + red[5] + red[6] + red[7];
        if (tid < D) {
            acc *= fix;
            for (int j = 0; j < S_THREADS && k0 + j < total; ++j)
                if (ps[j] != 0.0f) {
                    const int c = a.c.v_codes[row_of[j] * (D / 2) + (tid >> 1)] >> (4 * (tid & 1));
                    acc += ps[j] * float(int(uint32_t(c) << 28) >> 28);
                }
        }
    }
    if (tid < D) a.out[(t * H + h) * D + tid] = float_to_bf16_bits(sum > 0.0f ? acc / sum : 0.0f);
    if (tid == 0 && a.lse) a.lse[t * H + h] = sum > 0.0f ? top + logf(sum) : -INFINITY;
}

}  // namespace

uint64_t kv_attention_workspace_bytes(int64_t, int64_t, int, int, int, int) { return 16; }

cudaError_t launch_kv_attention(const KvAttnArgs &a, int, int, cudaStream_t stream) {
    const unsigned grid = unsigned(a.T * a.q_heads);
    return a.c.D == 128 ? launch_overlapped(kq_kv_attention_kernel<128>, grid, S_THREADS, 0, stream, a)
                        : launch_overlapped(kq_kv_attention_kernel<64>, grid, S_THREADS, 0, stream, a);
}

}  // namespace kq
