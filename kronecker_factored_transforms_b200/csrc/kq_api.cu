// kq_api.cu -- the extern "C" boundary of libkq (declared in include/kq.h).
//
// Every entry point validates its arguments on the host before anything is
// launched, then picks a kernel for the shape and launches it on the
// caller's stream.  Nothing is allocated and no per-call state is kept.
#include <cmath>
#include <cstdint>
#include <mutex>

#include "../../include/kq.h"
#include "kq_internal.h"

namespace {

constexpr int kVersion = 1 * 10000 + 0 * 100 + 0;

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

struct Range {
    uintptr_t lo, hi;  // [lo, hi)
};
Range range_of(const void *p, uint64_t bytes) {
    uintptr_t b = reinterpret_cast<uintptr_t>(p);
    return Range{b, b + static_cast<uintptr_t>(bytes)};
}
bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi && a.hi > a.lo && b.hi > b.lo; }

bool supported_factor(int k) { return k >= 16 && k <= 128 && k % 16 == 0; }

// Shape checks shared by all entries: SHAPE, then UNSUPPORTED, then overflow.
kq_status check_shape(int64_t T, int n1, int n2) {
    if (T < 0 || n1 <= 0 || n2 <= 0) return KQ_ERR_SHAPE;
    if (!supported_factor(n1) || !supported_factor(n2)) return KQ_ERR_UNSUPPORTED;
    const int64_t n = int64_t(n1) * n2;
    if (T > INT64_MAX / (n * 4)) return KQ_ERR_SHAPE;  // largest buffer is T*n*4 bytes
    return KQ_OK;
}

kq_status check_alpha(float alpha) {
    if (!std::isfinite(alpha) || !(alpha > 0.0f) || alpha > 1.0f) return KQ_ERR_ARG;
    return KQ_OK;
}

struct DeviceInfo {
    int device = -1;
    int num_sms = 0;
};

// SM count per device, queried once per device.
kq_status device_info(DeviceInfo &info) {
    static std::mutex mu;
    static int sms_cache[64] = {0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return KQ_ERR_CUDA;
    std::lock_guard<std::mutex> lock(mu);
    if (dev < 0 || dev >= 64) return KQ_ERR_CUDA;
    if (sms_cache[dev] == 0) {
        int sms = 0;
        if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return KQ_ERR_CUDA;
        sms_cache[dev] = sms;
    }
    info.device = dev;
    info.num_sms = sms_cache[dev];
    return KQ_OK;
}

// Which transform kernel a quantising call of this size runs.  The pair-pipelined
// kernel (n1 = 64) wins on short launches, where its short start-up and per-group
// pipeline matter most, and the batch-pipelined tcgen05 kernel on long ones.  The
// crossover, measured on B200: without cinv about 56 groups of 128 / n2 tokens per
// SM (64x64: 25.2 against 25.8 us at T = 10000, 39.4 against 39.9 at 16384, 152
// against 148 at 65536); with cinv about 4 (64x128: 6.6 against 6.7 us at T = 256,
// 8.0 both at 512, 11.8 against 11.1 at 1024, 19.5 against 15.3 at 2048).
enum class Kern { Fused, Tc05, WarpMma };
Kern choose_kernel(int64_t T, int n1, int n2, bool scaled, float alpha, bool quant, int num_sms) {
    if (!quant || !(alpha >= 0x1p-19f)) return Kern::WarpMma;  // fp32 y out, or the rounding's range
    // tokens per group: 128 / (n2 padded to 64 or 128)
    const int64_t h = n2 <= 64 ? 2 : 1, groups = (T + h - 1) / h;
    // TMA row coordinates are 32-bit: past 2^31 rows of x both tensor-core kernels give way
    if (T * int64_t(n1) >= (int64_t(1) << 31)) return Kern::WarpMma;
    const int64_t per_sm = scaled ? 4 : 56;
    if (kq::fused_supports(n1, n2, scaled) && groups <= per_sm * num_sms) return Kern::Fused;
    if (kq::tc05_supports(n1, n2, scaled)) return Kern::Tc05;
    return Kern::WarpMma;
}

const char *kernel_name_of(Kern k) {
    switch (k) {
    case Kern::Fused: return "kq_fused_kernel";
    case Kern::Tc05: return "kq_tc05_fused_kernel";
    default: return "kq_warp_mma_kernel";
    }
}

kq_status run_transform(const uint16_t *x, const uint16_t *P1, const uint16_t *P2, const float *cinv,
                        float alpha, uint8_t *q_out, float *scale_out, float *y_out, int64_t T,
                        int n1, int n2, kq_stream_t stream) {
    DeviceInfo info;
    kq_status st = device_info(info);
    if (st != KQ_OK) return st;
    kq::LaunchArgs a;
    a.x = x;
    a.P1 = P1;
    a.P2 = P2;
    a.cinv = cinv;
    a.alpha = alpha;
    a.q_out = q_out;
    a.scale_out = scale_out;
    a.y_out = y_out;
    a.T = T;
    a.n1 = n1;
    a.n2 = n2;
    a.num_sms = info.num_sms;
    a.device = info.device;
    a.stream = reinterpret_cast<cudaStream_t>(stream);
    // The tcgen05 kernels round with a 1.5 * 2^23 shift, exact while |y / s| = 7 / alpha < 2^22.
    cudaError_t err;
    switch (choose_kernel(T, n1, n2, cinv != nullptr, alpha, y_out == nullptr, info.num_sms)) {
    case Kern::Fused: err = kq::launch_fused(a); break;
    case Kern::Tc05: err = kq::launch_tc05(a); break;
    default: err = kq::launch_warp_mma(a); break;
    }
    return err == cudaSuccess ? KQ_OK : KQ_ERR_CUDA;
}

}  // namespace

extern "C" {

kq_status kq_transform_quant(const uint16_t *x, const uint16_t *P1, const uint16_t *P2,
                             const float *cinv, float alpha, uint8_t *q_out, float *scale_out,
                             int64_t T, int n1, int n2, kq_stream_t stream) {
    kq_status st = check_shape(T, n1, n2);
    if (st != KQ_OK) return st;
    if ((st = check_alpha(alpha)) != KQ_OK) return st;
    if (T == 0) return KQ_OK;
    if (!x || !P1 || !P2 || !q_out || !scale_out) return KQ_ERR_NULL;
    if (!aligned(x, 16) || !aligned(P1, 16) || !aligned(P2, 16) || !aligned(q_out, 16) ||
        !aligned(scale_out, 4) || (cinv && !aligned(cinv, 16)))
        return KQ_ERR_ALIGN;
    const uint64_t n = uint64_t(n1) * n2;
    const Range in[4] = {range_of(x, uint64_t(T) * n * 2), range_of(P1, uint64_t(n1) * n1 * 2),
                         range_of(P2, uint64_t(n2) * n2 * 2), range_of(cinv, cinv ? n * 4 : 0)};
    const Range rq = range_of(q_out, uint64_t(T) * n / 2), rs = range_of(scale_out, uint64_t(T) * 4);
    for (const Range &r : in)
        if (overlap(r, rq) || overlap(r, rs)) return KQ_ERR_ARG;
    if (overlap(rq, rs)) return KQ_ERR_ARG;
    return run_transform(x, P1, P2, cinv, alpha, q_out, scale_out, nullptr, T, n1, n2, stream);
}

kq_status kq_transform(const uint16_t *x, const uint16_t *P1, const uint16_t *P2, const float *cinv,
                       float *y_out, int64_t T, int n1, int n2, kq_stream_t stream) {
    kq_status st = check_shape(T, n1, n2);
    if (st != KQ_OK) return st;
    if (T == 0) return KQ_OK;
    if (!x || !P1 || !P2 || !y_out) return KQ_ERR_NULL;
    if (!aligned(x, 16) || !aligned(P1, 16) || !aligned(P2, 16) || !aligned(y_out, 16) ||
        (cinv && !aligned(cinv, 16)))
        return KQ_ERR_ALIGN;
    const uint64_t n = uint64_t(n1) * n2;
    const Range in[4] = {range_of(x, uint64_t(T) * n * 2), range_of(P1, uint64_t(n1) * n1 * 2),
                         range_of(P2, uint64_t(n2) * n2 * 2), range_of(cinv, cinv ? n * 4 : 0)};
    const Range ry = range_of(y_out, uint64_t(T) * n * 4);
    for (const Range &r : in)
        if (overlap(r, ry)) return KQ_ERR_ARG;
    return run_transform(x, P1, P2, cinv, 1.0f, nullptr, nullptr, y_out, T, n1, n2, stream);
}

kq_status kq_dequant_inverse(const uint8_t *q, const float *scale, const float *P1inv,
                             const float *P2inv, const float *c, float *x_hat, int64_t T, int n1,
                             int n2, kq_stream_t stream) {
    kq_status st = check_shape(T, n1, n2);
    if (st != KQ_OK) return st;
    if (T == 0) return KQ_OK;
    if (!q || !scale || !P1inv || !P2inv || !x_hat) return KQ_ERR_NULL;
    if (!aligned(q, 16) || !aligned(scale, 4) || !aligned(P1inv, 4) || !aligned(P2inv, 4) ||
        !aligned(x_hat, 16) || (c && !aligned(c, 4)))
        return KQ_ERR_ALIGN;
    const uint64_t n = uint64_t(n1) * n2;
    const Range in[5] = {range_of(q, uint64_t(T) * n / 2), range_of(scale, uint64_t(T) * 4),
                         range_of(P1inv, uint64_t(n1) * n1 * 4), range_of(P2inv, uint64_t(n2) * n2 * 4),
                         range_of(c, c ? n * 4 : 0)};
    const Range rx = range_of(x_hat, uint64_t(T) * n * 4);
    for (const Range &r : in)
        if (overlap(r, rx)) return KQ_ERR_ARG;
    cudaError_t err = kq::launch_dequant_inverse(q, scale, P1inv, P2inv, c, x_hat, T, n1, n2,
                                                 reinterpret_cast<cudaStream_t>(stream));
    return err == cudaSuccess ? KQ_OK : KQ_ERR_CUDA;
}

namespace {
// The checks and the launch of both W4A4 entries; `ob` = output bytes per element.
kq_status w4a4_gemm(const uint8_t *qx, const float *sx, const uint8_t *qw, const float *sw, void *y, int ob,
                    int64_t M, int64_t N, int64_t K, kq_stream_t stream) {
    if (M < 0 || N < 0 || K < 128 || K > 262144 || K % 128 != 0) return KQ_ERR_SHAPE;
    if (M > int64_t(65535) * 128) return KQ_ERR_SHAPE;  // grid rows
    if (M == 0 || N == 0) return KQ_OK;
    if (M > INT64_MAX / N / 4) return KQ_ERR_SHAPE;
    if (!qx || !sx || !qw || !sw || !y) return KQ_ERR_NULL;
    if (!aligned(qx, 16) || !aligned(qw, 16) || !aligned(sx, 4) || !aligned(sw, 4) || !aligned(y, uintptr_t(ob)))
        return KQ_ERR_ALIGN;
    const Range in[4] = {range_of(qx, uint64_t(M) * uint64_t(K) / 2), range_of(sx, uint64_t(M) * 4),
                         range_of(qw, uint64_t(N) * uint64_t(K) / 2), range_of(sw, uint64_t(N) * 4)};
    const Range ry = range_of(y, uint64_t(M) * uint64_t(N) * uint64_t(ob));
    for (const Range &r : in)
        if (overlap(r, ry)) return KQ_ERR_ARG;
    DeviceInfo info;
    kq_status st = device_info(info);
    if (st != KQ_OK) return st;
    cudaError_t err = kq::launch_w4a4_gemm(qx, sx, qw, sw, y, ob == 2, M, N, K, info.device,
                                           reinterpret_cast<cudaStream_t>(stream));
    return err == cudaSuccess ? KQ_OK : KQ_ERR_CUDA;
}
}  // namespace

kq_status kq_w4a4_gemm(const uint8_t *qx, const float *sx, const uint8_t *qw, const float *sw, float *y,
                       int64_t M, int64_t N, int64_t K, kq_stream_t stream) {
    return w4a4_gemm(qx, sx, qw, sw, y, 4, M, N, K, stream);
}

kq_status kq_w4a4_gemm_bf16(const uint8_t *qx, const float *sx, const uint8_t *qw, const float *sw, uint16_t *y,
                            int64_t M, int64_t N, int64_t K, kq_stream_t stream) {
    return w4a4_gemm(qx, sx, qw, sw, y, 2, M, N, K, stream);
}

kq_status kq_headwise_transform_quant(const uint16_t *x, const uint16_t *Ph, float alpha, uint8_t *q_out,
                                      float *scale_out, int64_t T, int heads, int head_dim, kq_stream_t stream) {
    if (T < 0 || heads <= 0 || head_dim <= 0) return KQ_ERR_SHAPE;
    if (head_dim != 64 && head_dim != 128) return KQ_ERR_UNSUPPORTED;
    if (T > (int64_t(1) << 31) / heads) return KQ_ERR_SHAPE;  // rows are TMA coordinates
    kq_status st = check_alpha(alpha);
    if (st != KQ_OK) return st;
    if (!(alpha >= 0x1p-19f)) return KQ_ERR_UNSUPPORTED;  // the code rounding's range
    if (T == 0) return KQ_OK;
    if (!x || !Ph || !q_out || !scale_out) return KQ_ERR_NULL;
    if (!aligned(x, 16) || !aligned(Ph, 16) || !aligned(q_out, 16) || !aligned(scale_out, 4)) return KQ_ERR_ALIGN;
    const int64_t R = T * heads;
    const Range in[2] = {range_of(x, uint64_t(R) * head_dim * 2), range_of(Ph, uint64_t(head_dim) * head_dim * 2)};
    const Range out[2] = {range_of(q_out, uint64_t(R) * head_dim / 2), range_of(scale_out, uint64_t(R) * 4)};
    for (const Range &o : out)
        for (const Range &i : in)
            if (overlap(o, i)) return KQ_ERR_ARG;
    if (overlap(out[0], out[1])) return KQ_ERR_ARG;
    DeviceInfo info;
    if ((st = device_info(info)) != KQ_OK) return st;
    cudaError_t err = kq::launch_rowwise(x, Ph, alpha, q_out, scale_out, R, head_dim, info.num_sms, info.device,
                                         reinterpret_cast<cudaStream_t>(stream));
    return err == cudaSuccess ? KQ_OK : KQ_ERR_CUDA;
}

kq_status kq_headwise_transform_quant_nvfp4(const uint16_t *x, const uint16_t *Ph, uint8_t *q_out,
                                            uint8_t *block_scale_out, float *scale_out, int64_t T, int heads,
                                            int head_dim, kq_stream_t stream) {
    if (T < 0 || heads <= 0 || head_dim <= 0) return KQ_ERR_SHAPE;
    if (head_dim != 64 && head_dim != 128) return KQ_ERR_UNSUPPORTED;
    if (T > (int64_t(1) << 31) / heads) return KQ_ERR_SHAPE;  // rows are TMA coordinates
    if (T == 0) return KQ_OK;
    if (!x || !Ph || !q_out || !block_scale_out || !scale_out) return KQ_ERR_NULL;
    if (!aligned(x, 16) || !aligned(Ph, 16) || !aligned(q_out, 16) || !aligned(block_scale_out, 8) ||
        !aligned(scale_out, 4))
        return KQ_ERR_ALIGN;
    const int64_t R = T * heads;
    const Range in[2] = {range_of(x, uint64_t(R) * head_dim * 2), range_of(Ph, uint64_t(head_dim) * head_dim * 2)};
    const Range out[3] = {range_of(q_out, uint64_t(R) * head_dim / 2), range_of(block_scale_out, uint64_t(R) * head_dim / 16),
                          range_of(scale_out, uint64_t(R) * 4)};
    for (const Range &o : out)
        for (const Range &i : in)
            if (overlap(o, i)) return KQ_ERR_ARG;
    if (overlap(out[0], out[1]) || overlap(out[0], out[2]) || overlap(out[1], out[2])) return KQ_ERR_ARG;
    DeviceInfo info;
    kq_status st = device_info(info);
    if (st != KQ_OK) return st;
    cudaError_t err = kq::launch_rowwise_nvfp4(x, Ph, q_out, block_scale_out, scale_out, R, head_dim, info.num_sms,
                                               info.device, reinterpret_cast<cudaStream_t>(stream));
    return err == cudaSuccess ? KQ_OK : KQ_ERR_CUDA;
}

kq_status kq_transform_quant_two_stage(const uint16_t *x, const uint16_t *P1, const uint16_t *P2,
                                       const float *cinv, float alpha, uint8_t *q_out, float *scale_out,
                                       void *workspace, uint64_t workspace_bytes, int64_t T, int n1, int n2,
                                       kq_stream_t stream) {
    if (T < 0 || n1 <= 0 || n2 <= 0) return KQ_ERR_SHAPE;
    if (!kq::two_stage_supports(n1, n2)) return KQ_ERR_UNSUPPORTED;
    const int64_t n = int64_t(n1) * n2;
    if (T >= (int64_t(1) << 31) / n) return KQ_ERR_SHAPE;  // rows and offsets are 32-bit
    kq_status st = check_alpha(alpha);
    if (st != KQ_OK) return st;
    if (!(alpha >= 0x1p-19f)) return KQ_ERR_UNSUPPORTED;  // the code rounding's range
    if (T == 0) return KQ_OK;
    if (!x || !P1 || !P2 || !q_out || !scale_out || !workspace) return KQ_ERR_NULL;
    if (!aligned(x, 16) || !aligned(P1, 16) || !aligned(P2, 16) || !aligned(q_out, 16) ||
        !aligned(workspace, 16) || !aligned(scale_out, 4) || (cinv && !aligned(cinv, 16)))
        return KQ_ERR_ALIGN;
    const uint64_t need = kq::two_stage_workspace_bytes(T, n1, n2);
    if (workspace_bytes < need) return KQ_ERR_ARG;
    const Range in[4] = {range_of(x, uint64_t(T) * n * 2), range_of(P1, uint64_t(n1) * n1 * 2),
                         range_of(P2, uint64_t(n2) * n2 * 2), range_of(cinv, cinv ? uint64_t(n) * 4 : 0)};
    const Range out[3] = {range_of(q_out, uint64_t(T) * n / 2), range_of(scale_out, uint64_t(T) * 4),
                          range_of(workspace, need)};
    for (const Range &o : out)
        for (const Range &i : in)
            if (overlap(o, i)) return KQ_ERR_ARG;
    if (overlap(out[0], out[1]) || overlap(out[0], out[2]) || overlap(out[1], out[2])) return KQ_ERR_ARG;
    DeviceInfo info;
    if ((st = device_info(info)) != KQ_OK) return st;
    kq::LaunchArgs a;
    a.x = x;
    a.P1 = P1;
    a.P2 = P2;
    a.cinv = cinv;
    a.alpha = alpha;
    a.q_out = q_out;
    a.scale_out = scale_out;
    a.y_out = nullptr;
    a.T = T;
    a.n1 = n1;
    a.n2 = n2;
    a.num_sms = info.num_sms;
    a.device = info.device;
    a.stream = reinterpret_cast<cudaStream_t>(stream);
    return kq::launch_two_stage(a, workspace) == cudaSuccess ? KQ_OK : KQ_ERR_CUDA;
}

uint64_t kq_two_stage_workspace_bytes(int64_t T, int n1, int n2) {
    if (T <= 0 || n1 <= 0 || n2 <= 0) return 0;
    return kq::two_stage_workspace_bytes(T, n1, n2);
}

kq_status kq_transform_quant_two_stage_static(const uint16_t *x, const uint16_t *P1, const uint16_t *P2,
                                              const float *cinv, float alpha, uint8_t *q_out, float *scale_out,
                                              int64_t T, int n1, int n2, kq_stream_t stream) {
    static_assert(KQ_STATIC_WORKSPACE_BYTES == kq::kStaticScratchBytes, "static workspace size");
    if (T < 0 || n1 <= 0 || n2 <= 0) return KQ_ERR_SHAPE;
    if (!kq::two_stage_supports(n1, n2)) return KQ_ERR_UNSUPPORTED;
    if (T > int64_t(kq::kStaticScratchBytes / kq::two_stage_workspace_bytes(1, n1, n2))) return KQ_ERR_ARG;
    void *scratch = nullptr;
    if (T > 0) {
        DeviceInfo info;
        kq_status st = device_info(info);
        if (st != KQ_OK) return st;
        if (kq::static_scratch(info.device, &scratch) != cudaSuccess) return KQ_ERR_CUDA;
    }
    return kq_transform_quant_two_stage(x, P1, P2, cinv, alpha, q_out, scale_out, scratch, kq::kStaticScratchBytes, T,
                                        n1, n2, stream);
}

// ---- the quantised key / value cache --------------------------------------------
namespace {

int log2_page(int page_size) {
    for (int s = 4; s <= 8; ++s)
        if (page_size == 1 << s) return s;
    return -1;
}

// The cache's description, checked: sizes, then support, then pointers.
kq_status check_cache(const kq_kv_cache *c) {
    if (!c) return KQ_ERR_NULL;
    if (c->num_pages < 1 || c->num_pages > INT32_MAX || c->kv_heads < 1 || c->kv_heads > 1024 || c->head_dim < 1 ||
        c->page_size < 1)
        return KQ_ERR_SHAPE;
    if ((c->head_dim != 64 && c->head_dim != 128) || log2_page(c->page_size) < 0) return KQ_ERR_UNSUPPORTED;
    if (!c->k_codes || !c->k_scale || !c->v_codes || !c->v_scale) return KQ_ERR_NULL;
    if (!aligned(c->k_codes, 16) || !aligned(c->k_scale, 16) || !aligned(c->v_codes, 16) || !aligned(c->v_scale, 16))
        return KQ_ERR_ALIGN;
    return KQ_OK;
}

struct CacheRanges {
    Range r[4];
};
CacheRanges cache_ranges(const kq_kv_cache *c) {
    const uint64_t rows = uint64_t(c->num_pages) * uint64_t(c->kv_heads) * uint64_t(c->page_size);
    const uint64_t codes = rows * uint64_t(c->head_dim / 2);
    return CacheRanges{{range_of(c->k_codes, codes), range_of(c->k_scale, rows * 4), range_of(c->v_codes, codes),
                        range_of(c->v_scale, rows * 4)}};
}

kq::KvCache cache_view(const kq_kv_cache *c) {
    return kq::KvCache{c->k_codes, c->k_scale, c->v_codes, c->v_scale, c->num_pages, log2_page(c->page_size),
                       c->kv_heads, c->head_dim};
}

bool any_overlap(const Range *a, int na, const Range *b, int nb) {
    for (int i = 0; i < na; ++i)
        for (int j = 0; j < nb; ++j)
            if (overlap(a[i], b[j])) return true;
    return false;
}

// [T] rows of `width` elements, `stride` elements apart.
Range rows_range(const void *p, int64_t T, int64_t stride, int64_t width) {
    return range_of(p, p ? (uint64_t(T - 1) * uint64_t(stride) + uint64_t(width)) * 2 : 0);
}

}  // namespace

kq_status kq_kv_append(const kq_kv_cache *cache, const kq_kv_transform *tf, const uint16_t *q, int64_t q_stride,
                       const uint16_t *k, int64_t k_stride, const uint16_t *v, int64_t v_stride,
                       const int32_t *positions, const int64_t *slots, uint16_t *q_out, int64_t T, int q_heads,
                       kq_stream_t stream) {
    if (T < 0 || q_heads < 0 || q_heads > 1024) return KQ_ERR_SHAPE;
    if (T == 0) return KQ_OK;
    kq_status st = check_cache(cache);
    if (st != KQ_OK) return st;
    if (!tf) return KQ_ERR_NULL;
    const int D = cache->head_dim, Hk = cache->kv_heads;
    if (T >= (int64_t(1) << 31) / (q_heads + Hk)) return KQ_ERR_SHAPE;
    if (check_alpha(tf->alpha_k) != KQ_OK || check_alpha(tf->alpha_v) != KQ_OK) return KQ_ERR_ARG;
    if (!(tf->alpha_k >= 0x1p-19f) || !(tf->alpha_v >= 0x1p-19f)) return KQ_ERR_UNSUPPORTED;
    if (tf->rope) {
        if (tf->rope_positions < 1 || tf->rope_positions > INT32_MAX || tf->rope_dim < 1 || tf->rope_dim > D)
            return KQ_ERR_SHAPE;
        if (tf->rope_dim % 16 != 0) return KQ_ERR_UNSUPPORTED;
    }
    if (!k || !v || !slots || !tf->Pk || !tf->Pv || (tf->rope && !positions)) return KQ_ERR_NULL;
    if (q_heads > 0 && (!q || !q_out || !tf->Pq)) return KQ_ERR_NULL;
    const int64_t wq = int64_t(q_heads) * D, wk = int64_t(Hk) * D, kMaxStride = int64_t(1) << 31;
    if (k_stride < wk || v_stride < wk || k_stride > kMaxStride || v_stride > kMaxStride) return KQ_ERR_ARG;
    if (q_heads > 0 && (q_stride < wq || q_stride > kMaxStride)) return KQ_ERR_ARG;
    if (!aligned(k, 16) || !aligned(v, 16) || k_stride % 8 != 0 || v_stride % 8 != 0 || !aligned(tf->Pk, 16) ||
        !aligned(tf->Pv, 16) || !aligned(slots, 8) || (tf->rope && (!aligned(tf->rope, 16) || !aligned(positions, 4))))
        return KQ_ERR_ALIGN;
    if (q_heads > 0 && (!aligned(q, 16) || !aligned(q_out, 16) || q_stride % 8 != 0 || !aligned(tf->Pq, 16)))
        return KQ_ERR_ALIGN;
    const uint64_t DD = uint64_t(D) * D * 2;
    const Range in[9] = {rows_range(q_heads > 0 ? q : nullptr, T, q_stride, wq),
                         rows_range(k, T, k_stride, wk),
                         rows_range(v, T, v_stride, wk),
                         range_of(tf->Pk, DD),
                         range_of(tf->Pv, DD),
                         range_of(q_heads > 0 ? tf->Pq : nullptr, q_heads > 0 ? DD : 0),
                         range_of(tf->rope, tf->rope ? uint64_t(tf->rope_positions) * uint64_t(tf->rope_dim) * 4 : 0),
                         range_of(positions, tf->rope ? uint64_t(T) * 4 : 0),
                         range_of(slots, uint64_t(T) * 8)};
    const CacheRanges cr = cache_ranges(cache);
    const Range out[5] = {cr.r[0], cr.r[1], cr.r[2], cr.r[3],
                          range_of(q_heads > 0 ? q_out : nullptr, q_heads > 0 ? uint64_t(T) * uint64_t(wq) * 2 : 0)};
    if (any_overlap(in, 9, out, 5)) return KQ_ERR_ARG;
    for (int i = 0; i < 5; ++i)
        if (any_overlap(out + i, 1, out + i + 1, 4 - i)) return KQ_ERR_ARG;
    DeviceInfo info;
    if ((st = device_info(info)) != KQ_OK) return st;
    kq::KvAppendArgs a;
    a.c = cache_view(cache);
    a.Pq = tf->Pq;
    a.Pk = tf->Pk;
    a.Pv = tf->Pv;
    a.alpha_k = tf->alpha_k;
    a.alpha_v = tf->alpha_v;
    a.rope = tf->rope;
    a.rope_positions = tf->rope_positions;
    a.rope_dim = tf->rope ? tf->rope_dim : 0;
    a.rope_interleaved = tf->rope_interleaved != 0;
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.positions = positions;
    a.slots = slots;
    a.q_out = q_out;
    a.T = T;
    a.q_heads = q_heads;
    if (kq::device_error_word(info.device, &a.err) != cudaSuccess) return KQ_ERR_CUDA;
    cudaError_t err = kq::launch_kv_append(a, info.num_sms, info.device, reinterpret_cast<cudaStream_t>(stream));
    return err == cudaSuccess ? KQ_OK : KQ_ERR_CUDA;
}

kq_status kq_kv_gather(const kq_kv_cache *cache, const int64_t *slots, uint16_t *k_out, uint16_t *v_out, int64_t T,
                       kq_stream_t stream) {
    if (T < 0) return KQ_ERR_SHAPE;
    if (T == 0) return KQ_OK;
    kq_status st = check_cache(cache);
    if (st != KQ_OK) return st;
    if (T >= (int64_t(1) << 31) / cache->kv_heads) return KQ_ERR_SHAPE;
    if (!slots || !k_out || !v_out) return KQ_ERR_NULL;
    if (!aligned(slots, 8) || !aligned(k_out, 16) || !aligned(v_out, 16)) return KQ_ERR_ALIGN;
    const CacheRanges cr = cache_ranges(cache);
    const Range in[5] = {cr.r[0], cr.r[1], cr.r[2], cr.r[3], range_of(slots, uint64_t(T) * 8)};
    const uint64_t bytes = uint64_t(T) * uint64_t(cache->kv_heads) * uint64_t(cache->head_dim) * 2;
    const Range out[2] = {range_of(k_out, bytes), range_of(v_out, bytes)};
    if (any_overlap(in, 5, out, 2) || overlap(out[0], out[1])) return KQ_ERR_ARG;
    DeviceInfo info;
    if ((st = device_info(info)) != KQ_OK) return st;
    unsigned int *err_word = nullptr;
    if (kq::device_error_word(info.device, &err_word) != cudaSuccess) return KQ_ERR_CUDA;
    cudaError_t err = kq::launch_kv_gather(cache_view(cache), slots, k_out, v_out, T, err_word,
                                           reinterpret_cast<cudaStream_t>(stream));
    return err == cudaSuccess ? KQ_OK : KQ_ERR_CUDA;
}

namespace {
constexpr int64_t kMaxSequences = 65535, kMaxKeys = int64_t(1) << 30;

kq_status kv_attention(const kq_kv_cache *cache, const uint16_t *q, const int32_t *q_start,
                       const int32_t *prefix_pages, int64_t prefix_len, const int32_t *page_table, int64_t max_pages,
                       const int32_t *kv_len, float scale, float softcap, int window, uint16_t *out, float *lse,
                       void *workspace, uint64_t workspace_bytes, int64_t T, int64_t B, int q_heads, int max_q,
                       kq_stream_t stream) {
    if (T < 0 || B < 0 || q_heads < 1 || q_heads > 1024 || prefix_len < 0 || max_pages < 1) return KQ_ERR_SHAPE;
    if (T == 0 || B == 0) return KQ_OK;
    kq_status st = check_cache(cache);
    if (st != KQ_OK) return st;
    if (q_heads % cache->kv_heads != 0 || T >= (int64_t(1) << 31) / q_heads || B > kMaxSequences ||
        (!q_start && T != B) || max_pages >= kMaxKeys / cache->page_size || prefix_len >= kMaxKeys)
        return KQ_ERR_SHAPE;
    if (!std::isfinite(scale) || !std::isfinite(softcap) || softcap < 0.0f || window < 0 || max_q < 1)
        return KQ_ERR_ARG;
    // what the kernels multiply by: scale log2(e), scale / softcap and softcap log2(e)
    if (!std::isfinite(scale * 1.5f) || !std::isfinite(softcap * 1.5f) ||
        (softcap > 0.0f && !std::isfinite(scale / softcap)))
        return KQ_ERR_ARG;
    if (!q || !page_table || !kv_len || !out || !workspace || (prefix_len > 0 && !prefix_pages)) return KQ_ERR_NULL;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(workspace, 16) || !aligned(page_table, 4) ||
        !aligned(kv_len, 4) || (q_start && !aligned(q_start, 4)) || (lse && !aligned(lse, 4)) ||
        (prefix_len > 0 && !aligned(prefix_pages, 4)))
        return KQ_ERR_ALIGN;
    if (!q_start) max_q = 1;
    if (max_q > T) max_q = int(T);
    const uint64_t need =
        kq::kv_attention_workspace_bytes(T, B, q_heads, cache->kv_heads, cache->head_dim, max_q);
    if (workspace_bytes < need) return KQ_ERR_ARG;
    const uint64_t rows = uint64_t(T) * uint64_t(q_heads);
    const CacheRanges cr = cache_ranges(cache);
    const uint64_t ppages = (uint64_t(prefix_len) + uint64_t(cache->page_size) - 1) / uint64_t(cache->page_size);
    const Range in[9] = {cr.r[0], cr.r[1], cr.r[2], cr.r[3], range_of(q, rows * uint64_t(cache->head_dim) * 2),
                         range_of(page_table, uint64_t(B) * uint64_t(max_pages) * 4),
                         range_of(kv_len, uint64_t(B) * 4),
                         range_of(q_start, q_start ? (uint64_t(B) + 1) * 4 : 0),
                         range_of(prefix_pages, ppages * 4)};
    const Range res[3] = {range_of(out, rows * uint64_t(cache->head_dim) * 2), range_of(lse, lse ? rows * 4 : 0),
                          range_of(workspace, need)};
    if (any_overlap(in, 9, res, 3) || any_overlap(res, 1, res + 1, 2) || overlap(res[1], res[2])) return KQ_ERR_ARG;
    DeviceInfo info;
    if ((st = device_info(info)) != KQ_OK) return st;
    kq::KvAttnArgs a;
    a.c = cache_view(cache);
    a.q = q;
    a.q_start = q_start;
    a.prefix_pages = prefix_len > 0 ? prefix_pages : nullptr;
    a.prefix_len = prefix_len;
    a.page_table = page_table;
    a.max_pages = max_pages;
    a.kv_len = kv_len;
    a.scale = scale;
    a.softcap = softcap;
    a.window = window;
    a.out = out;
    a.lse = lse;
    a.workspace = static_cast<unsigned char *>(workspace);
    a.T = T;
    a.B = B;
    a.q_heads = q_heads;
    a.max_q = max_q;
    if (kq::device_error_word(info.device, &a.err) != cudaSuccess) return KQ_ERR_CUDA;
    cudaError_t err = kq::launch_kv_attention(a, info.num_sms, info.device, reinterpret_cast<cudaStream_t>(stream));
    return err == cudaSuccess ? KQ_OK : KQ_ERR_CUDA;
}
}  // namespace

kq_status kq_kv_attention(const kq_kv_cache *cache, const uint16_t *q, const int32_t *q_start,
                          const int32_t *page_table, int64_t max_pages, const int32_t *kv_len, float scale,
                          float softcap, int window, uint16_t *out, float *lse, void *workspace,
                          uint64_t workspace_bytes, int64_t T, int64_t B, int q_heads, int max_q,
                          kq_stream_t stream) {
    return kv_attention(cache, q, q_start, nullptr, 0, page_table, max_pages, kv_len, scale, softcap, window, out, lse,
                        workspace, workspace_bytes, T, B, q_heads, max_q, stream);
}

kq_status kq_kv_attention_shared(const kq_kv_cache *cache, const uint16_t *q, const int32_t *q_start,
                                 const int32_t *prefix_pages, int64_t prefix_len, const int32_t *page_table,
                                 int64_t max_pages, const int32_t *kv_len, float scale, float softcap, int window,
                                 uint16_t *out, float *lse, void *workspace, uint64_t workspace_bytes, int64_t T,
                                 int64_t B, int q_heads, int max_q, kq_stream_t stream) {
    return kv_attention(cache, q, q_start, prefix_pages, prefix_len, page_table, max_pages, kv_len, scale, softcap,
                        window, out, lse, workspace, workspace_bytes, T, B, q_heads, max_q, stream);
}

uint64_t kq_kv_attention_workspace_bytes(int64_t T, int64_t B, int q_heads, int kv_heads, int head_dim, int max_q) {
    if (T <= 0 || B <= 0 || q_heads < 1 || q_heads > 1024 || kv_heads < 1 || q_heads % kv_heads != 0 || max_q < 1 ||
        (head_dim != 64 && head_dim != 128) || T >= (int64_t(1) << 31) / q_heads || B > kMaxSequences)
        return 0;
    return kq::kv_attention_workspace_bytes(T, B, q_heads, kv_heads, head_dim, int(max_q > T ? T : max_q));
}

kq_status kq_device_error(kq_stream_t stream, int *code) {
    if (!code) return KQ_ERR_NULL;
    unsigned int v = 0;
    if (kq::read_and_clear_device_error(reinterpret_cast<cudaStream_t>(stream), &v) != cudaSuccess)
        return KQ_ERR_CUDA;
    *code = static_cast<int>(v);
    return KQ_OK;
}

kq_status kq_selftest_bounded_wait(int64_t limit_us, kq_stream_t stream) {
    if (limit_us < 1 || limit_us > 10000000) return KQ_ERR_ARG;
    cudaError_t err = kq::launch_selftest_wait(uint64_t(limit_us) * 1000u,
                                               reinterpret_cast<cudaStream_t>(stream));
    return err == cudaSuccess ? KQ_OK : KQ_ERR_CUDA;
}

const char *kq_status_string(int status) {
    switch (status) {
    case KQ_OK: return "ok";
    case KQ_ERR_NULL: return "a required pointer is NULL";
    case KQ_ERR_SHAPE: return "bad shape (T < 0, n1 <= 0, n2 <= 0 or size overflow)";
    case KQ_ERR_UNSUPPORTED:
        return "unsupported size or parameter for this entry (factors: multiples of 16 up to 128, or up to 256 for "
               "the two-stage entries; head_dim 64 or 128; pages of 16 to 256 rows; rotated elements a multiple of 16; alpha of at least 2^-19 where the entry requires it)";
    case KQ_ERR_ALIGN: return "misaligned pointer";
    case KQ_ERR_ARG: return "bad argument (alpha outside (0, 1], a scale, bound or stride out of range, a workspace too small, or "
                            "outputs overlap inputs)";
    case KQ_ERR_CUDA: return "CUDA runtime error";
    case KQ_ERR_TIMEOUT: return "a bounded wait inside a kernel timed out";
    default: return "unknown status";
    }
}

const char *kq_kernel_name(int n1, int n2, int has_cinv) {
    if (!supported_factor(n1) || !supported_factor(n2)) return "unsupported";
    return kq::tc05_supports(n1, n2, has_cinv != 0) ? "kq_tc05_fused_kernel" : "kq_warp_mma_kernel";
}

const char *kq_kernel_for(int64_t T, int n1, int n2, int has_cinv, float alpha) {
    if (T < 0 || !supported_factor(n1) || !supported_factor(n2)) return "unsupported";
    int sms = 148;
    DeviceInfo info;
    if (device_info(info) == KQ_OK) sms = info.num_sms;
    return kernel_name_of(choose_kernel(T, n1, n2, has_cinv != 0, alpha, true, sms));
}

int kq_version(void) { return kVersion; }

}  // extern "C"
