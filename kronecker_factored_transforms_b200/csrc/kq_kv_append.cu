// kq_kv_append.cu -- new tokens into the pages of the INT4 key / value cache, and
// their rows back out.
//
//     q_out = R(pos) q Pq,   y = R(pos) k Pk  or  v Pv,
//     s = alpha max|y| / 7,  code = clamp(round_half_even(y / s), -8, 7)
#include "kq_common.cuh"
#include "kq_internal.h"

namespace kq {
namespace {

constexpr int A_THREADS = 128;

// Element i of a row rotated by its token's angles; exact products in fp64.
__device__ __forceinline__ double rotated(const uint16_t *x, int i, const float *cs, int rope_dim, bool inter) {
    const double xi = double(bf16_bits_to_float(x[i]));
    if (i >= rope_dim) return xi;
    const int half = rope_dim >> 1;
    const int a = inter ? i >> 1 : (i < half ? i : i - half);  // the pair's angle
    const bool first = inter ? (i & 1) == 0 : i < half;
    const int j = inter ? i ^ 1 : (first ? i + half : i - half);
    const double xj = double(bf16_bits_to_float(x[j]));
    const double c = double(cs[a]), s = double(cs[half + a]);
    return first ? xi * c - xj * s : xj * s + xi * c;
}

template <int D>
__global__ void __launch_bounds__(A_THREADS) kq_kv_append_kernel(const __grid_constant__ KvAppendArgs a) {
    __shared__ double xs[D];
    __shared__ double red[4];
    __shared__ uint8_t cs[D];
    const int H = a.q_heads, Hk = a.c.heads, tid = threadIdx.x;
    const int rows = H + 2 * Hk;
    griddep_wait();
    griddep_launch_dependents();
    for (int64_t u = blockIdx.x; u < a.T * rows; u += gridDim.x) {
        const int64_t t = u / rows;
        const int r = int(u % rows);
        const int kind = r < H ? 0 : r < H + Hk ? 1 : 2;
        const int h = kind == 0 ? r : kind == 1 ? r - H : r - H - Hk;
        const uint16_t *x = kind == 0 ? a.q + t * a.q_stride : kind == 1 ? a.k + t * a.k_stride : a.v + t * a.v_stride;
        const uint16_t *P = kind == 0 ? a.Pq : kind == 1 ? a.Pk : a.Pv;
        x += int64_t(h) * D;
        bool pos_ok = true;
        const float *table = nullptr;
        if (a.rope) {
            const int64_t pos = a.positions[t];
            pos_ok = pos >= 0 && pos < a.rope_positions;
            table = a.rope + (pos_ok ? pos : 0) * a.rope_dim;
        }
        __syncthreads();
        if (tid < D)
            xs[tid] = rotated(x, tid, table, kind < 2 && a.rope ? a.rope_dim : 0, a.rope_interleaved != 0);
        __syncthreads();
        double y = 0.0;
        if (tid < D)
            for (int i = 0; i < D; ++i) y += xs[i] * double(bf16_bits_to_float(P[i * D + tid]));
        if (kind == 0) {
            if (tid < D) a.q_out[(t * H + h) * D + tid] = pos_ok ? float_to_bf16_bits(float(y)) : 0;
            if (!pos_ok && tid == 0) atomicOr(a.err, kSiteKvAppend);
            continue;
        }
        double m = fabs(y);
        for (int o = 16; o; o >>= 1) m = fmax(m, __shfl_xor_sync(0xffffffffu, m, o));
        if ((tid & 31) == 0) red[tid >> 5] = m;
        __syncthreads();
        m = fmax(fmax(red[0], red[1]), fmax(red[2], red[3]));
        const double s = double(kind == 1 ? a.alpha_k : a.alpha_v) * m / 7.0;
        if (tid < D) cs[tid] = uint8_t(int(s > 0.0 ? rint(fmin(fmax(y / s, -8.0), 7.0)) : 0.0) & 15);
        __syncthreads();
        const int64_t slot = a.slots[t], psize = int64_t(1) << a.c.page_shift;
        if (slot < 0) continue;
        if (slot >= a.c.pages * psize || !pos_ok) {
            if (tid == 0) atomicOr(a.err, kSiteKvAppend);
            continue;
        }
        const int64_t row = ((slot >> a.c.page_shift) * Hk + h) * psize + (slot & (psize - 1));
        uint8_t *codes = kind == 1 ? a.c.k_codes : a.c.v_codes;
        if (tid < D / 2) codes[row * (D / 2) + tid] = uint8_t(cs[2 * tid] | (cs[2 * tid + 1] << 4));
        if (tid == 0) (kind == 1 ? a.c.k_scale : a.c.v_scale)[row] = float(s);
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

cudaError_t launch_kv_append(const KvAppendArgs &a, int num_sms, int device, cudaStream_t stream) {
    const int64_t units = a.T * (a.q_heads + 2 * a.c.heads);
    const unsigned grid = unsigned(units < 16 * num_sms ? units : 16 * num_sms);
    return a.c.D == 128 ? launch_overlapped(kq_kv_append_kernel<128>, grid, A_THREADS, 0, stream, a)
                        : launch_overlapped(kq_kv_append_kernel<64>, grid, A_THREADS, 0, stream, a);
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
