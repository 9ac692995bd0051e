// kq_internal.h -- launch plumbing shared between the C ABI and the kernels.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace kq {

struct LaunchArgs {
    const uint16_t *x;
    const uint16_t *P1;
    const uint16_t *P2;
    const float *cinv;   // nullptr: c = 1
    float alpha;
    uint8_t *q_out;      // quantise mode
    float *scale_out;
    float *y_out;        // transform-only mode when non-null
    int64_t T;
    int n1, n2;
    int num_sms;
    int device;
    cudaStream_t stream;
};

// General warp-level MMA kernel: every supported shape.
cudaError_t launch_warp_mma(const LaunchArgs &a);

// Persistent tcgen05/TMEM kernel for the shapes it covers (alpha >= 2^-19).
bool tc05_supports(int n1, int n2, bool scaled);
cudaError_t launch_tc05(const LaunchArgs &a);

// Group-pipelined tcgen05/TMEM kernel (n1 = 64, n2 in {64, 128}; alpha >= 2^-19).
bool fused_supports(int n1, int n2, bool scaled);
cudaError_t launch_fused(const LaunchArgs &a);

// Diagnostic: a kernel whose bounded wait on a never-signalled barrier gives up.
cudaError_t launch_selftest_wait(uint64_t limit_ns, cudaStream_t stream);

// cuTensorMapEncodeTiled from the driver (null if unavailable).
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

// Device address of the status word (for kernels in other translation units).
cudaError_t device_error_word(int device, unsigned int **word);

// Read and clear the device status word set by bounded waits that gave up.
cudaError_t read_and_clear_device_error(cudaStream_t stream, unsigned int *code);

// Check entry: q * s -> P1inv^T Y P2inv -> * c, fp32 on CUDA cores.
cudaError_t launch_dequant_inverse(const uint8_t *q, const float *scale, const float *P1inv,
                                   const float *P2inv, const float *c, float *x_hat, int64_t T,
                                   int n1, int n2, cudaStream_t stream);

// W4A4 product of packed INT4 codes: y = sx[m] sw[o] sum_k qx[m][k] qw[o][k].
cudaError_t launch_w4a4_gemm(const uint8_t *qx, const float *sx, const uint8_t *qw, const float *sw, void *y,
                             bool bf16_out, int64_t M, int64_t N, int64_t K, int device, cudaStream_t stream);

// Per-head transform + INT4 per row: rows of head_dim (64 or 128) values.
cudaError_t launch_rowwise(const uint16_t *x, const uint16_t *Ph, float alpha, uint8_t *q_out, float *scale_out,
                           int64_t R, int head_dim, int num_sms, int device, cudaStream_t stream);
// The same transform with NVFP4 rows: E2M1 codes, an E4M3 scale per 16 values,
// an fp32 scale per row.
cudaError_t launch_rowwise_nvfp4(const uint16_t *x, const uint16_t *Ph, uint8_t *q_out, uint8_t *bscale_out,
                                 float *scale_out, int64_t R, int head_dim, int num_sms, int device,
                                 cudaStream_t stream);

// Two-stage transform + INT4 for factors up to 256 through a workspace of
// two_stage_workspace_bytes(T, n1, n2) bytes (Z^T hi then lo, bf16).
bool two_stage_supports(int n1, int n2);
uint64_t two_stage_workspace_bytes(int64_t T, int n1, int n2);
cudaError_t launch_two_stage(const LaunchArgs &a, void *workspace);

// The static workspace of kq_transform_quant_two_stage_static (one per device).
constexpr uint64_t kStaticScratchBytes = uint64_t(64) << 20;
cudaError_t static_scratch(int device, void **ptr);

// ---- the quantised key / value cache ------------------------------------------

// Pages of INT4 rows (see kq_kv_cache in kq.h), as the kernels take them.
struct KvCache {
    uint8_t *k_codes;
    float *k_scale;
    uint8_t *v_codes;
    float *v_scale;
    int64_t pages;
    int page_shift;  // log2 of the page size
    int heads;
    int D;
};

struct KvAppendArgs {
    KvCache c;
    const uint16_t *Pq, *Pk, *Pv;
    float alpha_k, alpha_v;
    const float *rope;  // nullptr: no rotation
    int64_t rope_positions;
    int rope_dim;
    int rope_interleaved;
    const uint16_t *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;
    const int32_t *positions;
    const int64_t *slots;
    uint16_t *q_out;
    int64_t T;
    int q_heads;
    unsigned int *err;  // device status word
};
cudaError_t launch_kv_append(const KvAppendArgs &a, int num_sms, int device, cudaStream_t stream);
cudaError_t launch_kv_gather(const KvCache &c, const int64_t *slots, uint16_t *k_out, uint16_t *v_out, int64_t T,
                             unsigned int *err, cudaStream_t stream);

struct KvAttnArgs {
    KvCache c;
    const uint16_t *q;
    const int32_t *q_start;       // nullptr: one query per sequence
    const int32_t *prefix_pages;  // nullptr: no shared prefix
    int64_t prefix_len;
    const int32_t *page_table;
    int64_t max_pages;
    const int32_t *kv_len;
    float scale, softcap;
    int window;  // 0: none
    uint16_t *out;
    float *lse;  // may be nullptr
    unsigned char *workspace;
    int64_t T, B;
    int q_heads, max_q;
    unsigned int *err;
};
uint64_t kv_attention_workspace_bytes(int64_t T, int64_t B, int q_heads, int kv_heads, int head_dim, int max_q);
cudaError_t launch_kv_attention(const KvAttnArgs &a, int num_sms, int device, cudaStream_t stream);

// Site codes of the status word for indexes that are not followed.
enum : unsigned { kSiteKvAppend = 65536u, kSiteKvAttention = 131072u };

}  // namespace kq
