// Host-side launchers behind the C ABI in include/oss.h. Arguments are
// already validated by api.cu when these run.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/oss.h"
#include "paged.h"

namespace oss {

// Kernel ids stored in bits 0..7 of the device error word.
enum KernelId : unsigned int {
  kKernelAttnFwd = 1, kKernelSoftmaxRows = 2, kKernelPaged = 3, kKernelAttnPacked = 4
};

// Test hook for the bounded wait of the cluster-resident row kernel (see
// os_debug_inject_fault): extra_tx > 0 makes each CTA expect that many bytes
// more than its first row's copies deliver; timeout_ns > 0 replaces the
// default wait limit.
struct RowsFault {
  uint32_t extra_tx = 0;
  int64_t timeout_ns = 0;
};

// err_word: the device error word (the cluster-resident kernel records a
// give-up on its bounded wait there); may be null.
// ws (may be null, ws_bytes 0): a workspace of softmax_workspace_bytes()
// bytes; with it, rows beyond the cluster path's 1.6 MB are read once from
// HBM instead of twice.
cudaError_t launch_softmax_rows(const float* x, float* y, float* m, float* l,
                                int64_t rows, int64_t cols, int64_t ld_x, int64_t ld_y,
                                float scale, unsigned int* err_word, const RowsFault& fault,
                                void* ws, int64_t ws_bytes, cudaStream_t stream);

// 16-bit rows: dtype 1 = bf16, 2 = fp16 (x and y); m, l fp32 or null.
cudaError_t launch_softmax_rows16(const uint16_t* x, uint16_t* y, float* m, float* l,
                                  int64_t rows, int64_t cols, int64_t ld_x, int64_t ld_y,
                                  float scale, int dtype, unsigned int* err_word,
                                  const RowsFault& fault, void* ws, int64_t ws_bytes,
                                  cudaStream_t stream);

// Workspace the row softmax of rows of `row_bytes` bytes uses on the current
// device (0: none; -1: the device could not be queried).
int64_t softmax_workspace_bytes(int64_t row_bytes);

// Comparators: passes = 2 (online (m, l) pass, then a write pass) or 3 (max
// pass, sum pass, write pass); each pass re-reads x from HBM. m, l required.
cudaError_t launch_softmax_rows_multipass(const float* x, float* y, float* m, float* l,
                                          int64_t rows, int64_t cols, int64_t ld_x, int64_t ld_y,
                                          float scale, int passes, cudaStream_t stream);

cudaError_t launch_decode_splitkv(const uint16_t* q, const uint16_t* k, const uint16_t* v,
                                  const int32_t* kv_len, int B, int H, int Lmax, int D,
                                  int num_splits, float scale, float* part_m, float* part_l,
                                  float* part_o, cudaStream_t stream);

cudaError_t launch_merge_partials(const float* part_m, const float* part_l, const float* part_o,
                                  int64_t groups, int num_splits, int D, int finalize,
                                  void* o_out, float* m_out, float* l_out, float* lse_out,
                                  cudaStream_t stream);

// Test hook for the bounded waits of the attention kernel (see
// os_debug_inject_fault): skip_v_step >= 0 makes the producer skip that V
// load; timeout_ns > 0 replaces the default wait limit.
struct AttnFault {
  int skip_v_step = -1;
  int64_t timeout_ns = 0;
};

// Partial-state output of the attention forward: row r's (m, l, O) go to
// slot r * stride + index of m, l [rows * stride] and o [rows * stride, D].
struct AttnPartialOut {
  float* m;
  float* l;
  float* o;
  int stride;
  int index;
};

// Returns cudaErrorNotSupported for shapes the kernel does not cover. With
// partial != nullptr the kernel writes partial states instead of o and lse.
// rescale_policy: an os_rescale_policy value (0 threshold, 1 on rise, 2
// every tile). workspace (may be null): at least attention_workspace_bytes
// bytes, counters zero; with it, a non-causal launch whose query tiles do not
// fill the last round splits that round's tiles along the keys.
cudaError_t launch_attention_fwd(const uint16_t* q, const uint16_t* k, const uint16_t* v,
                                 uint16_t* o, float* lse, int B, int H, int Sq, int Sk, int D,
                                 float scale, bool causal, unsigned int* err_word,
                                 const AttnFault& fault, const AttnPartialOut* partial,
                                 int rescale_policy, void* workspace, int64_t workspace_bytes,
                                 cudaStream_t stream);

// Workspace the attention forward of this shape uses on the current device
// (0: none; -1: the device could not be queried).
int64_t attention_workspace_bytes(int B, int H, int Sq, int Sk, bool causal);

// Bytes of per-tile counters at the end of that workspace (*bytes; 0 when it
// uses none). Returns -1 when the device could not be queried, else 0.
int64_t attention_workspace_counters(int B, int H, int Sq, int Sk, bool causal, int64_t* bytes);

// SMs of the current device (0: it could not be queried).
int device_sms();

// The pools and tables of a validated os_paged_cache, for kernels.
PagedCache paged_cache(const os_paged_cache& c);

cudaError_t launch_kv_append(const uint16_t* k, const uint16_t* v, int64_t ld_token, int64_t ld_head,
                             int64_t tokens, const int32_t* cu, const os_paged_cache& cache,
                             unsigned int* err, cudaStream_t stream);

cudaError_t launch_kv_evict(const os_paged_cache& cache, const float* weights, int64_t ld_w_batch,
                            int64_t ld_w_head, const int32_t* new_table, int64_t ld_new_table,
                            int32_t new_max_pages, int32_t budget, int32_t recent, int32_t* kept,
                            int32_t* new_len, float* new_weights, unsigned int* err,
                            cudaStream_t stream);

// Workspace of the paged decode on the current device (-1: it could not be
// queried).
int64_t decode_paged_workspace_bytes(int H, const os_paged_cache& cache, bool weights);

cudaError_t launch_decode_paged(const uint16_t* q, int64_t ld_q_batch, int64_t ld_q_head, int H,
                                const os_paged_cache& cache, float scale, uint16_t* o, float* lse,
                                float* weights, int64_t ld_w_batch, int64_t ld_w_head,
                                void* workspace, unsigned int* err, cudaStream_t stream);

// The pools of a validated os_paged_cache_fp8, for kernels.
struct Fp8Pools;
Fp8Pools fp8_pools(const os_paged_cache_fp8& c);

cudaError_t launch_kv_append_fp8(const uint16_t* k, const uint16_t* v, int64_t ld_token, int64_t ld_head, int64_t tokens,
                                 const int32_t* cu, const os_paged_cache_fp8& cache, unsigned int* err,
                                 cudaStream_t stream);

cudaError_t launch_kv_read_fp8(const os_paged_cache_fp8& cache, const int32_t* cu, int64_t tokens, uint16_t* k,
                               uint16_t* v, int64_t ld_token, int64_t ld_head, unsigned int* err, cudaStream_t stream);

// Workspace of the 8-bit paged decode on the current device (-1: it could not be queried).
int64_t decode_paged_fp8_workspace_bytes(int H, const os_paged_cache& pages);

cudaError_t launch_decode_paged_fp8(const uint16_t* q, int64_t ld_q_batch, int64_t ld_q_head, int H,
                                    const os_paged_cache_fp8& cache, float scale, uint16_t* o, float* lse,
                                    void* workspace, unsigned int* err, cudaStream_t stream);

// Workspace of the decode behind shared prefixes on the current device (-1: it could not be
// queried).
int64_t decode_shared_workspace_bytes(int H, const os_paged_cache& cache, int groups, int prefix_max_pages);

cudaError_t launch_decode_shared(const uint16_t* q, int64_t ld_q_batch, int64_t ld_q_head, int H,
                                 const os_paged_cache& cache, const PrefixTables& prefix, float scale, uint16_t* o,
                                 float* lse, void* workspace, unsigned int* err, const AttnFault& fault,
                                 cudaStream_t stream);

// Arguments of the packed attention forward, as os_attention_fwd_packed's.
struct PackedArgs {
  const uint16_t *q, *k, *v;
  int64_t ld_q_token, ld_q_head, ld_kv_token, ld_kv_head;
  uint16_t* o;
  float* lse;
  const int32_t *cu_q, *cu_k;
  int32_t batch;
  int64_t tokens_q, tokens_k;
  int32_t Hq, Hkv, D;
  bool f16;
  float scale;
  bool causal;
};

// Workspace of the packed attention forward on the current device (-1: it
// could not be queried).
int64_t attn_packed_workspace_bytes(int64_t tokens_k, int Hkv, int D);

cudaError_t launch_attn_packed(const PackedArgs& args, void* workspace, unsigned int* err,
                               const AttnFault& fault, cudaStream_t stream);

// Layout of the workspace of the prefixes' part of os_attention_decode_shared: offsets, then
// the size.
struct PrefixPlan {
  int shares, packs, head_shift;  // 2^head_shift query heads of a key head side by side in a tile
  int64_t part_o, part_ml, where, state_o, state_ml, bytes;
};

PrefixPlan prefix_plan(int H, const os_paged_cache& cache);

struct PrefixLaunch;

// Attention of every sequence's token over its group's prefix, ending in states (m, l, O).
cudaError_t launch_attn_prefix(const uint16_t* q, int64_t ld_q_batch, int64_t ld_q_head, int H, const os_paged_cache& cache,
                               const PrefixLaunch& launch, float scale, const PrefixPlan& plan, void* workspace,
                               unsigned int* err, const AttnFault& fault, cudaStream_t stream);

// log2(e) split into a float and the float nearest to the remainder, so that
// hi + lo carries about 48 bits of it.
void split_constant(double c, float* hi, float* lo);

}  // namespace oss
