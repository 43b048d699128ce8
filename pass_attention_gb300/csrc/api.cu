// The C ABI of liboss (include/oss.h): host-side validation, then launch.
// Nothing here synchronises, allocates device memory or prints.
// os_softmax_rows_from_host creates four CUDA events per call (released at
// its end) and, once per device, two copy streams.

#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>

#include <cuda_runtime.h>

#include "../../include/oss.h"
#include "oss_internal.h"

// One error word per device, written by kernels that give up on a bounded
// wait (first code wins) and read back by os_check_device_error.
__device__ unsigned int g_oss_error_word;

namespace {

constexpr int kMaxDevices = 64;
// Device address of g_oss_error_word, per device, filled on first use. Host
// threads may race to fill a slot; they store the same address, and the
// atomic makes that race well defined.
std::atomic<unsigned int*> g_err_ptr[kMaxDevices];

unsigned int* error_word() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
  unsigned int* cached = g_err_ptr[dev].load(std::memory_order_acquire);
  if (!cached) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_oss_error_word) != cudaSuccess) return nullptr;
    cached = static_cast<unsigned int*>(p);
    g_err_ptr[dev].store(cached, std::memory_order_release);
  }
  return cached;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

os_status from_cuda(cudaError_t e) {
  if (e == cudaSuccess) return OS_OK;
  if (e == cudaErrorNotSupported) return OS_ERR_UNSUPPORTED;
  return OS_ERR_CUDA;
}

bool valid_scale(float s) { return std::isfinite(s) && s > 0.f; }

// Armed by os_debug_inject_fault, consumed by the next os_attention_fwd on
// the same host thread.
thread_local oss::AttnFault t_fault;
// Armed by os_debug_inject_fault (kind 2), consumed by the next
// os_softmax_rows or os_softmax_rows_16bit on the same host thread.
thread_local oss::RowsFault t_rows_fault;

// Whether two runs of 4-byte elements share one.
bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y ? y - x < static_cast<uintptr_t>(na) * 4 : x - y < static_cast<uintptr_t>(nb) * 4;
}

// What every call on a paged cache asks of it. The pools themselves are
// checked by the calls that follow them.
os_status check_cache(const os_paged_cache* c) {
  if (!c || !c->page_table || !c->kv_len || !c->k_pages || !c->v_pages) return OS_ERR_INVALID_ARGUMENT;
  if (c->num_pages <= 0 || c->heads <= 0 || c->page_size <= 0 || c->head_dim <= 0 || c->batch <= 0 ||
      c->max_pages <= 0)
    return OS_ERR_INVALID_ARGUMENT;
  if (c->dtype != OS_DTYPE_BF16 && c->dtype != OS_DTYPE_F16) return OS_ERR_INVALID_ARGUMENT;
  // a stride of 0 would put several rows of a pool in one place
  if (c->ld_page < (c->num_pages > 1) || c->ld_head < (c->heads > 1) || c->ld_slot < 1 || c->ld_table < 0)
    return OS_ERR_INVALID_ARGUMENT;
  if (!aligned16(c->k_pages) || !aligned16(c->v_pages) || ((c->ld_page | c->ld_head | c->ld_slot) & 7))
    return OS_ERR_MISALIGNED;
  if ((reinterpret_cast<uintptr_t>(c->page_table) | reinterpret_cast<uintptr_t>(c->kv_len)) & 3u)
    return OS_ERR_MISALIGNED;
  if (c->page_size < 16 || c->page_size > 1024 || (c->page_size & (c->page_size - 1)))
    return OS_ERR_UNSUPPORTED;
  if (c->head_dim != 64 && c->head_dim != 128) return OS_ERR_UNSUPPORTED;
  if (c->batch > 65535 || c->heads > 65535 || static_cast<int64_t>(c->max_pages) * c->page_size > (int64_t(1) << 30))
    return OS_ERR_UNSUPPORTED;
  return OS_OK;
}

// The same for a cache in 8 bits.
os_status check_cache_fp8(const os_paged_cache_fp8* c) {
  if (!c || !c->k_scales || !c->v_scales) return OS_ERR_INVALID_ARGUMENT;
  const os_status st = check_cache(&c->pages);
  if (st != OS_OK) return st;
  if (c->ld_scale_page < (c->pages.num_pages > 1) || c->ld_scale_head < (c->pages.heads > 1)) return OS_ERR_INVALID_ARGUMENT;
  if (!aligned16(c->k_scales) || !aligned16(c->v_scales) ||
      ((c->pages.ld_page | c->pages.ld_head | c->pages.ld_slot | c->ld_scale_page | c->ld_scale_head) & 15))
    return OS_ERR_MISALIGNED;
  return OS_OK;
}

// What the appending calls ask of the new rows, and the reading one of where they go.
os_status check_rows(const void* k, const void* v, int64_t ld_token, int64_t ld_head, int64_t tokens, const int32_t* cu) {
  if (!k || !v) return OS_ERR_INVALID_ARGUMENT;
  if (tokens > 0x7fffffff) return OS_ERR_UNSUPPORTED;
  if (!aligned16(k) || !aligned16(v) || ((ld_token | ld_head) & 7)) return OS_ERR_MISALIGNED;
  if (reinterpret_cast<uintptr_t>(cu) & 3u) return OS_ERR_MISALIGNED;
  return OS_OK;
}

// Whether a workspace size may be asked for H query heads over this cache.
bool sized_cache(int32_t H, const os_paged_cache& c) {
  if (c.heads <= 0 || H <= 0 || H % c.heads) return false;
  if (c.batch <= 0 || c.batch > 65535 || c.max_pages <= 0 || c.page_size <= 0 ||
      static_cast<int64_t>(c.max_pages) * c.page_size > (int64_t(1) << 30))
    return false;
  return c.head_dim == 64 || c.head_dim == 128;
}

// Set by os_attention_set_rescale_policy; kept for the host thread's later
// attention calls.
thread_local int t_rescale_policy = OS_RESCALE_THRESHOLD;

// The two copy streams of os_softmax_rows_from_host on the current device
// (non-blocking, made on first use and kept for the process).
cudaError_t copy_streams(cudaStream_t* up, cudaStream_t* down) {
  static std::mutex mu;
  static cudaStream_t streams[kMaxDevices][2];
  static bool made[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(mu);
  if (!made[dev]) {
    if ((e = cudaStreamCreateWithFlags(&streams[dev][0], cudaStreamNonBlocking)) != cudaSuccess) return e;
    if ((e = cudaStreamCreateWithFlags(&streams[dev][1], cudaStreamNonBlocking)) != cudaSuccess) {
      cudaStreamDestroy(streams[dev][0]);
      return e;
    }
    made[dev] = true;
  }
  *up = streams[dev][0];
  *down = streams[dev][1];
  return cudaSuccess;
}

// The pipeline of os_softmax_rows_from_host over blocks of chunk_rows rows:
// a block's upload on `up`, its kernel on `main` once the upload landed, its
// downloads on `down` once the kernel ended. `up` and `down` start after the
// work already on `main`, and `main` ends after the last download. A wait
// enqueued on an event keeps the record it saw, so each event is recorded
// again for the next block.
cudaError_t from_host_pipeline(const float* x_host, float* y_host, float* m_host, float* l_host,
                               float* x_dev, float* y_dev, float* m_dev, float* l_dev, int64_t rows,
                               int64_t cols, float scale, int64_t chunk_rows, cudaStream_t main,
                               cudaStream_t up, cudaStream_t down, const cudaEvent_t* ev) {
  cudaError_t e;
  if ((e = cudaEventRecord(ev[0], main)) != cudaSuccess) return e;
  if ((e = cudaStreamWaitEvent(up, ev[0], 0)) != cudaSuccess) return e;
  if ((e = cudaStreamWaitEvent(down, ev[0], 0)) != cudaSuccess) return e;
  for (int64_t r0 = 0; r0 < rows; r0 += chunk_rows) {
    const int64_t n = (rows - r0 < chunk_rows) ? rows - r0 : chunk_rows;
    const int64_t off = r0 * cols;
    const size_t bytes = static_cast<size_t>(n * cols) * sizeof(float);
    const size_t vb = static_cast<size_t>(n) * sizeof(float);
    if ((e = cudaMemcpyAsync(x_dev + off, x_host + off, bytes, cudaMemcpyHostToDevice, up)) != cudaSuccess)
      return e;
    if ((e = cudaEventRecord(ev[1], up)) != cudaSuccess) return e;
    if ((e = cudaStreamWaitEvent(main, ev[1], 0)) != cudaSuccess) return e;
    if ((e = oss::launch_softmax_rows(x_dev + off, y_dev + off, m_dev ? m_dev + r0 : nullptr,
                                      l_dev ? l_dev + r0 : nullptr, n, cols, cols, cols, scale,
                                      error_word(), oss::RowsFault(), nullptr, 0, main)) != cudaSuccess)
      return e;
    if ((e = cudaEventRecord(ev[2], main)) != cudaSuccess) return e;
    if ((e = cudaStreamWaitEvent(down, ev[2], 0)) != cudaSuccess) return e;
    if ((e = cudaMemcpyAsync(y_host + off, y_dev + off, bytes, cudaMemcpyDeviceToHost, down)) != cudaSuccess)
      return e;
    if (m_host && (e = cudaMemcpyAsync(m_host + r0, m_dev + r0, vb, cudaMemcpyDeviceToHost, down)) != cudaSuccess)
      return e;
    if (l_host && (e = cudaMemcpyAsync(l_host + r0, l_dev + r0, vb, cudaMemcpyDeviceToHost, down)) != cudaSuccess)
      return e;
  }
  if ((e = cudaEventRecord(ev[3], down)) != cudaSuccess) return e;
  return cudaStreamWaitEvent(main, ev[3], 0);
}

}  // namespace

extern "C" {

int32_t os_abi_version(void) { return OSS_ABI_VERSION; }

const char* os_status_string(os_status status) {
  switch (status) {
    case OS_OK: return "OS_OK";
    case OS_ERR_INVALID_ARGUMENT: return "OS_ERR_INVALID_ARGUMENT";
    case OS_ERR_MISALIGNED: return "OS_ERR_MISALIGNED";
    case OS_ERR_UNSUPPORTED: return "OS_ERR_UNSUPPORTED";
    case OS_ERR_CUDA: return "OS_ERR_CUDA";
    case OS_ERR_TIMEOUT: return "OS_ERR_TIMEOUT";
    case OS_ERR_BAD_INDEX: return "OS_ERR_BAD_INDEX";
  }
  return "OS_ERR_UNKNOWN";
}

os_status os_softmax_rows_ws(const float* x, float* y, float* m, float* l, int64_t rows,
                             int64_t cols, int64_t ld_x, int64_t ld_y, float scale, void* workspace,
                             int64_t workspace_bytes, void* stream) {
  if (!x || !y) return OS_ERR_INVALID_ARGUMENT;
  if (rows <= 0 || cols <= 0 || ld_x < cols || ld_y < cols) return OS_ERR_INVALID_ARGUMENT;
  if (cols > (int64_t(1) << 30) || rows > (int64_t(1) << 40)) return OS_ERR_INVALID_ARGUMENT;
  if (!valid_scale(scale)) return OS_ERR_INVALID_ARGUMENT;
  if (workspace_bytes < 0 || (!workspace && workspace_bytes != 0)) return OS_ERR_INVALID_ARGUMENT;
  if ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(y) |
       reinterpret_cast<uintptr_t>(m) | reinterpret_cast<uintptr_t>(l)) & 3u)
    return OS_ERR_MISALIGNED;
  if (!aligned16(workspace)) return OS_ERR_MISALIGNED;
  const oss::RowsFault fault = t_rows_fault;
  t_rows_fault = oss::RowsFault();
  return from_cuda(oss::launch_softmax_rows(x, y, m, l, rows, cols, ld_x, ld_y, scale,
                                            error_word(), fault, workspace, workspace_bytes,
                                            static_cast<cudaStream_t>(stream)));
}

os_status os_softmax_rows(const float* x, float* y, float* m, float* l, int64_t rows,
                          int64_t cols, int64_t ld_x, int64_t ld_y, float scale, void* stream) {
  return os_softmax_rows_ws(x, y, m, l, rows, cols, ld_x, ld_y, scale, nullptr, 0, stream);
}

os_status os_softmax_rows_16bit_ws(const void* x, void* y, float* m, float* l, int64_t rows,
                                   int64_t cols, int64_t ld_x, int64_t ld_y, float scale,
                                   int32_t dtype, void* workspace, int64_t workspace_bytes,
                                   void* stream) {
  if (!x || !y) return OS_ERR_INVALID_ARGUMENT;
  if (rows <= 0 || cols <= 0 || ld_x < cols || ld_y < cols) return OS_ERR_INVALID_ARGUMENT;
  if (cols > (int64_t(1) << 30) || rows > (int64_t(1) << 40)) return OS_ERR_INVALID_ARGUMENT;
  if (!valid_scale(scale) || (dtype != OS_DTYPE_BF16 && dtype != OS_DTYPE_F16))
    return OS_ERR_INVALID_ARGUMENT;
  if (workspace_bytes < 0 || (!workspace && workspace_bytes != 0)) return OS_ERR_INVALID_ARGUMENT;
  if ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(y)) & 1u) return OS_ERR_MISALIGNED;
  if ((reinterpret_cast<uintptr_t>(m) | reinterpret_cast<uintptr_t>(l)) & 3u) return OS_ERR_MISALIGNED;
  if (!aligned16(workspace)) return OS_ERR_MISALIGNED;
  const oss::RowsFault fault = t_rows_fault;
  t_rows_fault = oss::RowsFault();
  return from_cuda(oss::launch_softmax_rows16(static_cast<const uint16_t*>(x),
                                              static_cast<uint16_t*>(y), m, l, rows, cols, ld_x,
                                              ld_y, scale, dtype, error_word(), fault, workspace,
                                              workspace_bytes, static_cast<cudaStream_t>(stream)));
}

os_status os_softmax_rows_16bit(const void* x, void* y, float* m, float* l, int64_t rows,
                                int64_t cols, int64_t ld_x, int64_t ld_y, float scale,
                                int32_t dtype, void* stream) {
  return os_softmax_rows_16bit_ws(x, y, m, l, rows, cols, ld_x, ld_y, scale, dtype, nullptr, 0,
                                  stream);
}

int64_t os_softmax_rows_workspace_bytes(int64_t rows, int64_t cols, int32_t dtype) {
  if (rows <= 0 || cols <= 0) return 0;
  if (dtype != 0 && dtype != OS_DTYPE_BF16 && dtype != OS_DTYPE_F16) return 0;
  return oss::softmax_workspace_bytes(cols * (dtype == 0 ? 4 : 2));
}

os_status os_softmax_rows_from_host(const float* x_host, float* y_host, float* m_host, float* l_host,
                                    float* x_dev, float* y_dev, float* m_dev, float* l_dev,
                                    int64_t rows, int64_t cols, float scale, int64_t chunk_rows,
                                    void* stream) {
  if (!x_host || !y_host || !x_dev || !y_dev) return OS_ERR_INVALID_ARGUMENT;
  if ((m_host && !m_dev) || (l_host && !l_dev)) return OS_ERR_INVALID_ARGUMENT;
  if (rows <= 0 || cols <= 0 || chunk_rows < 0) return OS_ERR_INVALID_ARGUMENT;
  if (cols > (int64_t(1) << 30) || rows > (int64_t(1) << 40)) return OS_ERR_INVALID_ARGUMENT;
  if (!valid_scale(scale)) return OS_ERR_INVALID_ARGUMENT;
  if ((reinterpret_cast<uintptr_t>(x_dev) | reinterpret_cast<uintptr_t>(y_dev) |
       reinterpret_cast<uintptr_t>(m_dev) | reinterpret_cast<uintptr_t>(l_dev)) & 3u)
    return OS_ERR_MISALIGNED;
  if (chunk_rows == 0) {  // about 64 MiB of x a block
    chunk_rows = (int64_t(64) << 20) / (cols * 4);
    if (chunk_rows < 1) chunk_rows = 1;
  }
  cudaStream_t up = nullptr, down = nullptr;
  cudaError_t e = copy_streams(&up, &down);
  if (e != cudaSuccess) return from_cuda(e);
  cudaEvent_t ev[4] = {nullptr, nullptr, nullptr, nullptr};
  for (int i = 0; i < 4 && e == cudaSuccess; ++i) e = cudaEventCreateWithFlags(&ev[i], cudaEventDisableTiming);
  if (e == cudaSuccess)
    e = from_host_pipeline(x_host, y_host, m_host, l_host, x_dev, y_dev, m_dev, l_dev, rows, cols, scale,
                           chunk_rows, static_cast<cudaStream_t>(stream), up, down, ev);
  // an event destroyed while work it was recorded on is pending is released
  // once that work completes: this does not wait
  for (int i = 0; i < 4; ++i)
    if (ev[i]) cudaEventDestroy(ev[i]);
  return from_cuda(e);
}

os_status os_softmax_rows_multipass(const float* x, float* y, float* m, float* l, int64_t rows,
                                    int64_t cols, int64_t ld_x, int64_t ld_y, float scale,
                                    int32_t passes, void* stream) {
  if (!x || !y || !m || !l) return OS_ERR_INVALID_ARGUMENT;
  if (rows <= 0 || cols <= 0 || ld_x < cols || ld_y < cols) return OS_ERR_INVALID_ARGUMENT;
  if (cols > (int64_t(1) << 30) || rows > (int64_t(1) << 40)) return OS_ERR_INVALID_ARGUMENT;
  if (!valid_scale(scale) || (passes != 2 && passes != 3)) return OS_ERR_INVALID_ARGUMENT;
  if ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(y) |
       reinterpret_cast<uintptr_t>(m) | reinterpret_cast<uintptr_t>(l)) & 3u)
    return OS_ERR_MISALIGNED;
  return from_cuda(oss::launch_softmax_rows_multipass(x, y, m, l, rows, cols, ld_x, ld_y, scale,
                                                      passes, static_cast<cudaStream_t>(stream)));
}

os_status os_attention_fwd(const os_bf16* q, const os_bf16* k, const os_bf16* v, os_bf16* o,
                           float* lse, int32_t B, int32_t H, int32_t Sq, int32_t Sk, int32_t D,
                           float scale, int causal, void* stream) {
  if (!q || !k || !v || !o) return OS_ERR_INVALID_ARGUMENT;
  if (B <= 0 || H <= 0 || Sq <= 0 || Sk <= 0 || D <= 0) return OS_ERR_INVALID_ARGUMENT;
  if (!valid_scale(scale)) return OS_ERR_INVALID_ARGUMENT;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o)) return OS_ERR_MISALIGNED;
  if (D != 128) return OS_ERR_UNSUPPORTED;
  if (causal && Sq != Sk) return OS_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(B) * H > 65535 * 64) return OS_ERR_UNSUPPORTED;
  unsigned int* err = error_word();
  if (!err) return OS_ERR_CUDA;
  const oss::AttnFault fault = t_fault;
  t_fault = oss::AttnFault();
  return from_cuda(oss::launch_attention_fwd(q, k, v, o, lse, B, H, Sq, Sk, D, scale,
                                             causal != 0, err, fault, nullptr, t_rescale_policy,
                                             nullptr, 0, static_cast<cudaStream_t>(stream)));
}

int64_t os_attention_fwd_workspace_bytes(int32_t B, int32_t H, int32_t Sq, int32_t Sk, int32_t D,
                                         int causal) {
  if (B <= 0 || H <= 0 || Sq <= 0 || Sk <= 0 || D != 128) return 0;
  if (static_cast<int64_t>(B) * H > 65535 * 64) return 0;
  return oss::attention_workspace_bytes(B, H, Sq, Sk, causal != 0);
}

os_status os_attention_fwd_ws(const os_bf16* q, const os_bf16* k, const os_bf16* v, os_bf16* o,
                              float* lse, int32_t B, int32_t H, int32_t Sq, int32_t Sk, int32_t D,
                              float scale, int causal, void* workspace, int64_t workspace_bytes,
                              void* stream) {
  if (!q || !k || !v || !o) return OS_ERR_INVALID_ARGUMENT;
  if (B <= 0 || H <= 0 || Sq <= 0 || Sk <= 0 || D <= 0) return OS_ERR_INVALID_ARGUMENT;
  if (!valid_scale(scale)) return OS_ERR_INVALID_ARGUMENT;
  if (workspace_bytes < 0 || (!workspace && workspace_bytes != 0)) return OS_ERR_INVALID_ARGUMENT;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(workspace))
    return OS_ERR_MISALIGNED;
  if (D != 128) return OS_ERR_UNSUPPORTED;
  if (causal && Sq != Sk) return OS_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(B) * H > 65535 * 64) return OS_ERR_UNSUPPORTED;
  const int64_t need = oss::attention_workspace_bytes(B, H, Sq, Sk, causal != 0);
  if (need < 0) return OS_ERR_CUDA;
  if (need > 0 && workspace && workspace_bytes < need) return OS_ERR_INVALID_ARGUMENT;
  unsigned int* err = error_word();
  if (!err) return OS_ERR_CUDA;
  const oss::AttnFault fault = t_fault;
  t_fault = oss::AttnFault();
  return from_cuda(oss::launch_attention_fwd(q, k, v, o, lse, B, H, Sq, Sk, D, scale,
                                             causal != 0, err, fault, nullptr, t_rescale_policy,
                                             workspace, workspace_bytes,
                                             static_cast<cudaStream_t>(stream)));
}

os_status os_attention_fwd_partial(const os_bf16* q, const os_bf16* k, const os_bf16* v,
                                   int32_t B, int32_t H, int32_t Sq, int32_t Sk, int32_t D,
                                   float scale, int causal, float* part_m, float* part_l,
                                   float* part_o, int32_t part_stride, int32_t part_index,
                                   void* stream) {
  if (!q || !k || !v || !part_m || !part_l || !part_o) return OS_ERR_INVALID_ARGUMENT;
  if (B <= 0 || H <= 0 || Sq <= 0 || Sk <= 0 || D <= 0) return OS_ERR_INVALID_ARGUMENT;
  if (part_stride <= 0 || part_index < 0 || part_index >= part_stride) return OS_ERR_INVALID_ARGUMENT;
  if (!valid_scale(scale)) return OS_ERR_INVALID_ARGUMENT;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(part_o)) return OS_ERR_MISALIGNED;
  if (D != 128) return OS_ERR_UNSUPPORTED;
  if (causal && Sq != Sk) return OS_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(B) * H > 65535 * 64) return OS_ERR_UNSUPPORTED;
  unsigned int* err = error_word();
  if (!err) return OS_ERR_CUDA;
  const oss::AttnFault fault = t_fault;
  t_fault = oss::AttnFault();
  const oss::AttnPartialOut out{part_m, part_l, part_o, part_stride, part_index};
  return from_cuda(oss::launch_attention_fwd(q, k, v, nullptr, nullptr, B, H, Sq, Sk, D, scale,
                                             causal != 0, err, fault, &out, t_rescale_policy,
                                             nullptr, 0, static_cast<cudaStream_t>(stream)));
}

os_status os_attention_decode_splitkv(const os_bf16* q, const os_bf16* k, const os_bf16* v,
                                      const int32_t* kv_len, int32_t B, int32_t H, int32_t Lmax,
                                      int32_t D, int32_t num_splits, float scale, float* part_m,
                                      float* part_l, float* part_o, void* stream) {
  if (!q || !k || !v || !kv_len || !part_m || !part_l || !part_o) return OS_ERR_INVALID_ARGUMENT;
  if (B <= 0 || H <= 0 || Lmax <= 0 || D <= 0 || num_splits <= 0) return OS_ERR_INVALID_ARGUMENT;
  if (!valid_scale(scale)) return OS_ERR_INVALID_ARGUMENT;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(part_o))
    return OS_ERR_MISALIGNED;
  if (D != 128 || num_splits > 64 || B > 65535 || H > 65535) return OS_ERR_UNSUPPORTED;
  return from_cuda(oss::launch_decode_splitkv(q, k, v, kv_len, B, H, Lmax, D, num_splits, scale,
                                              part_m, part_l, part_o,
                                              static_cast<cudaStream_t>(stream)));
}

os_status os_merge_partials(const float* part_m, const float* part_l, const float* part_o,
                            int64_t groups, int32_t num_splits, int32_t D, int finalize,
                            void* o_out, float* m_out, float* l_out, float* lse_out,
                            void* stream) {
  if (!part_m || !part_l || !part_o || !o_out) return OS_ERR_INVALID_ARGUMENT;
  if (groups <= 0 || num_splits <= 0 || D <= 0) return OS_ERR_INVALID_ARGUMENT;
  if (!aligned16(part_o) || !aligned16(o_out)) return OS_ERR_MISALIGNED;
  if (num_splits > 64 || D > 256 || (D & 3)) return OS_ERR_UNSUPPORTED;
  return from_cuda(oss::launch_merge_partials(part_m, part_l, part_o, groups, num_splits, D,
                                              finalize, o_out, m_out, l_out, lse_out,
                                              static_cast<cudaStream_t>(stream)));
}

os_status os_kv_cache_append(const void* k, const void* v, int64_t ld_token, int64_t ld_head,
                             int64_t tokens, const int32_t* cu_seqlens, const os_paged_cache* cache,
                             void* stream) {
  const os_status st = check_cache(cache);
  if (st != OS_OK) return st;
  if (tokens < 0 || ld_token < 0 || ld_head < 0 || (!cu_seqlens && tokens != cache->batch))
    return OS_ERR_INVALID_ARGUMENT;
  if (tokens == 0) return OS_OK;
  if (!k || !v) return OS_ERR_INVALID_ARGUMENT;
  if (tokens > 0x7fffffff) return OS_ERR_UNSUPPORTED;
  if (!aligned16(k) || !aligned16(v) || ((ld_token | ld_head) & 7)) return OS_ERR_MISALIGNED;
  if (reinterpret_cast<uintptr_t>(cu_seqlens) & 3u) return OS_ERR_MISALIGNED;
  unsigned int* err = error_word();
  if (!err) return OS_ERR_CUDA;
  return from_cuda(oss::launch_kv_append(static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v),
                                         ld_token, ld_head, tokens, cu_seqlens, *cache, err,
                                         static_cast<cudaStream_t>(stream)));
}

int64_t os_attention_decode_paged_workspace_bytes(int32_t H, const os_paged_cache* cache, int weights) {
  if (!cache || cache->heads <= 0 || H <= 0 || H % cache->heads) return 0;
  if (cache->batch <= 0 || cache->batch > 65535 || cache->max_pages <= 0 || cache->page_size <= 0 ||
      static_cast<int64_t>(cache->max_pages) * cache->page_size > (int64_t(1) << 30))
    return 0;
  if (cache->head_dim != 64 && cache->head_dim != 128) return 0;
  return oss::decode_paged_workspace_bytes(H, *cache, weights != 0);
}

os_status os_attention_decode_paged(const void* q, int64_t ld_q_batch, int64_t ld_q_head, int32_t H,
                                    const os_paged_cache* cache, float scale, void* o, float* lse,
                                    float* weights, int64_t ld_w_batch, int64_t ld_w_head,
                                    void* workspace, int64_t workspace_bytes, void* stream) {
  const os_status st = check_cache(cache);
  if (st != OS_OK) return st;
  if (!q || !o || !workspace || H <= 0 || H % cache->heads || !valid_scale(scale)) return OS_ERR_INVALID_ARGUMENT;
  if (ld_q_batch < 0 || ld_q_head < 0) return OS_ERR_INVALID_ARGUMENT;
  if (weights && (ld_w_batch < (cache->batch > 1) || ld_w_head < (cache->heads > 1))) return OS_ERR_INVALID_ARGUMENT;
  if (!aligned16(q) || !aligned16(o) || !aligned16(workspace) || ((ld_q_batch | ld_q_head) & 7))
    return OS_ERR_MISALIGNED;
  if ((reinterpret_cast<uintptr_t>(lse) | reinterpret_cast<uintptr_t>(weights)) & 3u) return OS_ERR_MISALIGNED;
  if (H > 65535) return OS_ERR_UNSUPPORTED;
  const int64_t need = oss::decode_paged_workspace_bytes(H, *cache, weights != nullptr);
  if (need < 0) return OS_ERR_CUDA;
  if (workspace_bytes < need) return OS_ERR_INVALID_ARGUMENT;
  unsigned int* err = error_word();
  if (!err) return OS_ERR_CUDA;
  return from_cuda(oss::launch_decode_paged(static_cast<const uint16_t*>(q), ld_q_batch, ld_q_head, H, *cache,
                                            scale, static_cast<uint16_t*>(o), lse, weights, ld_w_batch,
                                            ld_w_head, workspace, err, static_cast<cudaStream_t>(stream)));
}

os_status os_kv_cache_append_fp8(const void* k, const void* v, int64_t ld_token, int64_t ld_head, int64_t tokens,
                                 const int32_t* cu_seqlens, const os_paged_cache_fp8* cache, void* stream) {
  os_status st = check_cache_fp8(cache);
  if (st != OS_OK) return st;
  if (tokens < 0 || ld_token < 0 || ld_head < 0 || (!cu_seqlens && tokens != cache->pages.batch))
    return OS_ERR_INVALID_ARGUMENT;
  if (tokens == 0) return OS_OK;
  if ((st = check_rows(k, v, ld_token, ld_head, tokens, cu_seqlens)) != OS_OK) return st;
  unsigned int* err = error_word();
  if (!err) return OS_ERR_CUDA;
  return from_cuda(oss::launch_kv_append_fp8(static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v), ld_token,
                                             ld_head, tokens, cu_seqlens, *cache, err,
                                             static_cast<cudaStream_t>(stream)));
}

os_status os_kv_cache_read_fp8(const os_paged_cache_fp8* cache, const int32_t* cu_seqlens, int64_t tokens, void* k,
                               void* v, int64_t ld_token, int64_t ld_head, void* stream) {
  os_status st = check_cache_fp8(cache);
  if (st != OS_OK) return st;
  if (tokens < 0 || !cu_seqlens) return OS_ERR_INVALID_ARGUMENT;
  // a stride of 0 would put several rows in one place
  if (ld_token < (tokens > 1) || ld_head < (cache->pages.heads > 1)) return OS_ERR_INVALID_ARGUMENT;
  if (tokens == 0) return OS_OK;
  if ((st = check_rows(k, v, ld_token, ld_head, tokens, cu_seqlens)) != OS_OK) return st;
  unsigned int* err = error_word();
  if (!err) return OS_ERR_CUDA;
  return from_cuda(oss::launch_kv_read_fp8(*cache, cu_seqlens, tokens, static_cast<uint16_t*>(k),
                                           static_cast<uint16_t*>(v), ld_token, ld_head, err,
                                           static_cast<cudaStream_t>(stream)));
}

int64_t os_attention_decode_paged_fp8_workspace_bytes(int32_t H, const os_paged_cache_fp8* cache) {
  if (!cache || !sized_cache(H, cache->pages)) return 0;
  return oss::decode_paged_fp8_workspace_bytes(H, cache->pages);
}

os_status os_attention_decode_paged_fp8(const void* q, int64_t ld_q_batch, int64_t ld_q_head, int32_t H,
                                        const os_paged_cache_fp8* cache, float scale, void* o, float* lse,
                                        void* workspace, int64_t workspace_bytes, void* stream) {
  const os_status st = check_cache_fp8(cache);
  if (st != OS_OK) return st;
  if (!q || !o || !workspace || H <= 0 || H % cache->pages.heads || !valid_scale(scale)) return OS_ERR_INVALID_ARGUMENT;
  if (ld_q_batch < 0 || ld_q_head < 0) return OS_ERR_INVALID_ARGUMENT;
  if (!aligned16(q) || !aligned16(o) || !aligned16(workspace) || ((ld_q_batch | ld_q_head) & 7))
    return OS_ERR_MISALIGNED;
  if (reinterpret_cast<uintptr_t>(lse) & 3u) return OS_ERR_MISALIGNED;
  if (H > 65535) return OS_ERR_UNSUPPORTED;
  const int64_t need = oss::decode_paged_fp8_workspace_bytes(H, cache->pages);
  if (need < 0) return OS_ERR_CUDA;
  if (workspace_bytes < need) return OS_ERR_INVALID_ARGUMENT;
  unsigned int* err = error_word();
  if (!err) return OS_ERR_CUDA;
  return from_cuda(oss::launch_decode_paged_fp8(static_cast<const uint16_t*>(q), ld_q_batch, ld_q_head, H, *cache, scale,
                                                static_cast<uint16_t*>(o), lse, workspace, err,
                                                static_cast<cudaStream_t>(stream)));
}

int64_t os_attention_decode_shared_workspace_bytes(int32_t H, const os_paged_cache* cache, int32_t prefix_max_pages,
                                                   int32_t groups) {
  if (!cache || !sized_cache(H, *cache) || groups <= 0 || groups > 65535 || prefix_max_pages <= 0 ||
      static_cast<int64_t>(prefix_max_pages) * cache->page_size > (int64_t(1) << 30))
    return 0;
  return oss::decode_shared_workspace_bytes(H, *cache, groups, prefix_max_pages);
}

os_status os_attention_decode_shared(const void* q, int64_t ld_q_batch, int64_t ld_q_head, int32_t H,
                                     const os_paged_cache* cache, const int32_t* prefix_table, int64_t ld_prefix_table,
                                     const int32_t* prefix_len, int32_t prefix_max_pages, const int32_t* cu_groups,
                                     int32_t groups, float scale, void* o, float* lse, void* workspace,
                                     int64_t workspace_bytes, void* stream) {
  const os_status st = check_cache(cache);
  if (st != OS_OK) return st;
  if (!q || !o || !workspace || H <= 0 || H % cache->heads || !valid_scale(scale)) return OS_ERR_INVALID_ARGUMENT;
  if (!prefix_table || !prefix_len || ld_prefix_table < 0 || prefix_max_pages <= 0 || groups <= 0 ||
      (!cu_groups && groups != 1))
    return OS_ERR_INVALID_ARGUMENT;
  // a tensor map wants a positive stride for a dimension that is walked
  if (ld_q_batch < (cache->batch > 1) || ld_q_head < (H > 1)) return OS_ERR_INVALID_ARGUMENT;
  if (!aligned16(q) || !aligned16(o) || !aligned16(workspace) || ((ld_q_batch | ld_q_head) & 7))
    return OS_ERR_MISALIGNED;
  if ((reinterpret_cast<uintptr_t>(lse) | reinterpret_cast<uintptr_t>(prefix_table) |
       reinterpret_cast<uintptr_t>(prefix_len) | reinterpret_cast<uintptr_t>(cu_groups)) & 3u)
    return OS_ERR_MISALIGNED;
  if (H > 65535 || groups > 65535 || static_cast<int64_t>(prefix_max_pages) * cache->page_size > (int64_t(1) << 30))
    return OS_ERR_UNSUPPORTED;
  const int64_t need = oss::decode_shared_workspace_bytes(H, *cache, groups, prefix_max_pages);
  if (need < 0) return OS_ERR_CUDA;
  if (workspace_bytes < need) return OS_ERR_INVALID_ARGUMENT;
  unsigned int* err = error_word();
  if (!err) return OS_ERR_CUDA;
  const oss::PrefixTables prefix{prefix_table, ld_prefix_table, prefix_len, cu_groups, groups, prefix_max_pages};
  const oss::AttnFault fault = t_fault;
  t_fault = oss::AttnFault();
  return from_cuda(oss::launch_decode_shared(static_cast<const uint16_t*>(q), ld_q_batch, ld_q_head, H, *cache, prefix,
                                             scale, static_cast<uint16_t*>(o), lse, workspace, err, fault,
                                             static_cast<cudaStream_t>(stream)));
}

int64_t os_attention_fwd_packed_workspace_bytes(int64_t tokens_k, int32_t Hkv, int32_t D) {
  if (tokens_k < 0 || tokens_k > 0x7fffffff || Hkv <= 0 || Hkv > 65535 || (D != 64 && D != 128)) return 0;
  return oss::attn_packed_workspace_bytes(tokens_k, Hkv, D);
}

os_status os_attention_fwd_packed(const void* q, int64_t ld_q_token, int64_t ld_q_head, const void* k,
                                  const void* v, int64_t ld_kv_token, int64_t ld_kv_head, void* o,
                                  float* lse, const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k,
                                  int32_t batch, int64_t tokens_q, int64_t tokens_k, int32_t Hq, int32_t Hkv,
                                  int32_t D, int32_t dtype, float scale, int causal, void* workspace,
                                  int64_t workspace_bytes, void* stream) {
  if (!cu_seqlens_q || !cu_seqlens_k || batch <= 0 || tokens_q < 0 || tokens_k < 0 || Hq <= 0 || Hkv <= 0 ||
      Hq % Hkv || D <= 0 || !valid_scale(scale))
    return OS_ERR_INVALID_ARGUMENT;
  if (dtype != OS_DTYPE_BF16 && dtype != OS_DTYPE_F16) return OS_ERR_INVALID_ARGUMENT;
  // a tensor map wants a positive stride for a dimension that is walked
  if (ld_q_token < (tokens_q > 1) || ld_q_head < (Hq > 1) || ld_kv_token < (tokens_k > 1) || ld_kv_head < (Hkv > 1))
    return OS_ERR_INVALID_ARGUMENT;
  if (D != 64 && D != 128) return OS_ERR_UNSUPPORTED;
  if (batch > 65535 || Hq > 65535 || tokens_q > 0x7fffffff || tokens_k > 0x7fffffff) return OS_ERR_UNSUPPORTED;
  if (tokens_q == 0) return OS_OK;
  if (!q || !o || !workspace || (tokens_k > 0 && (!k || !v))) return OS_ERR_INVALID_ARGUMENT;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(workspace) ||
      ((ld_q_token | ld_q_head | ld_kv_token | ld_kv_head) & 7))
    return OS_ERR_MISALIGNED;
  if ((reinterpret_cast<uintptr_t>(lse) | reinterpret_cast<uintptr_t>(cu_seqlens_q) |
       reinterpret_cast<uintptr_t>(cu_seqlens_k)) & 3u)
    return OS_ERR_MISALIGNED;
  const int64_t need = oss::attn_packed_workspace_bytes(tokens_k, Hkv, D);
  if (need < 0) return OS_ERR_CUDA;
  if (workspace_bytes < need) return OS_ERR_INVALID_ARGUMENT;
  unsigned int* err = error_word();
  if (!err) return OS_ERR_CUDA;
  const oss::PackedArgs a{static_cast<const uint16_t*>(q), static_cast<const uint16_t*>(k),
                          static_cast<const uint16_t*>(v), ld_q_token, ld_q_head, ld_kv_token, ld_kv_head,
                          static_cast<uint16_t*>(o), lse, cu_seqlens_q, cu_seqlens_k, batch, tokens_q,
                          tokens_k, Hq, Hkv, D, dtype == OS_DTYPE_F16, scale, causal != 0};
  const oss::AttnFault fault = t_fault;
  t_fault = oss::AttnFault();
  return from_cuda(oss::launch_attn_packed(a, workspace, err, fault, static_cast<cudaStream_t>(stream)));
}

os_status os_kv_cache_evict(const os_paged_cache* cache, const float* weights, int64_t ld_w_batch,
                            int64_t ld_w_head, const int32_t* new_table, int64_t ld_new_table,
                            int32_t new_max_pages, int32_t budget, int32_t recent, int32_t* kept,
                            int32_t* new_len, float* new_weights, void* stream) {
  const os_status st = check_cache(cache);
  if (st != OS_OK) return st;
  if (!weights || !new_table || !kept || !new_len || !new_weights) return OS_ERR_INVALID_ARGUMENT;
  if (ld_w_batch < 0 || ld_w_head < 0 || ld_new_table < 0 || new_max_pages <= 0) return OS_ERR_INVALID_ARGUMENT;
  if (budget <= 0 || recent < 0 || recent > budget) return OS_ERR_INVALID_ARGUMENT;
  const int64_t room = static_cast<int64_t>(new_max_pages) * cache->page_size;
  if (budget > room) return OS_ERR_INVALID_ARGUMENT;
  if ((reinterpret_cast<uintptr_t>(weights) | reinterpret_cast<uintptr_t>(new_table) |
       reinterpret_cast<uintptr_t>(kept) | reinterpret_cast<uintptr_t>(new_len) |
       reinterpret_cast<uintptr_t>(new_weights)) & 3u)
    return OS_ERR_MISALIGNED;
  if (room > (int64_t(1) << 30)) return OS_ERR_UNSUPPORTED;
  // an output must not lie in what other CTAs still read, nor in another output
  const int64_t rows = static_cast<int64_t>(cache->batch) * cache->heads;
  const struct {
    const void* at;
    int64_t n;
  } spans[] = {{kept, rows * budget},
               {new_len, cache->batch},
               {new_weights, rows * room},
               {weights, (cache->batch - 1) * ld_w_batch + (cache->heads - 1) * ld_w_head +
                             static_cast<int64_t>(cache->max_pages) * cache->page_size},
               {cache->kv_len, cache->batch},
               {cache->page_table, (cache->batch - 1) * cache->ld_table + cache->max_pages},
               {new_table, (cache->batch - 1) * ld_new_table + new_max_pages}};
  if (new_table == cache->page_table) return OS_ERR_INVALID_ARGUMENT;
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 7; ++j)
      if (overlap(spans[i].at, spans[i].n, spans[j].at, spans[j].n)) return OS_ERR_INVALID_ARGUMENT;
  unsigned int* err = error_word();
  if (!err) return OS_ERR_CUDA;
  return from_cuda(oss::launch_kv_evict(*cache, weights, ld_w_batch, ld_w_head, new_table, ld_new_table,
                                        new_max_pages, budget, recent, kept, new_len, new_weights, err,
                                        static_cast<cudaStream_t>(stream)));
}

os_status os_attention_set_rescale_policy(int32_t policy) {
  if (policy != OS_RESCALE_THRESHOLD && policy != OS_RESCALE_ON_RISE && policy != OS_RESCALE_ALWAYS)
    return OS_ERR_INVALID_ARGUMENT;
  t_rescale_policy = policy;
  return OS_OK;
}

int32_t os_attention_rescale_policy(void) { return t_rescale_policy; }

os_status os_debug_inject_fault(int32_t kind, int32_t step, int64_t timeout_ns) {
  if (kind < 0 || kind > 2 || step < 0 || timeout_ns < 0) return OS_ERR_INVALID_ARGUMENT;
  t_fault = oss::AttnFault();
  t_rows_fault = oss::RowsFault();
  if (kind == 1) {
    t_fault.skip_v_step = step;
    t_fault.timeout_ns = timeout_ns;
  } else if (kind == 2) {
    t_rows_fault.extra_tx = 16;
    t_rows_fault.timeout_ns = timeout_ns;
  }
  return OS_OK;
}

os_status os_check_device_error(void* stream, int32_t* code) {
  if (code) *code = 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cudaStreamSynchronize(s) != cudaSuccess) return OS_ERR_CUDA;
  unsigned int* err = error_word();
  if (!err) return OS_ERR_CUDA;
  unsigned int word = 0;
  if (cudaMemcpyAsync(&word, err, sizeof(word), cudaMemcpyDeviceToHost, s) != cudaSuccess)
    return OS_ERR_CUDA;
  if (cudaMemsetAsync(err, 0, sizeof(word), s) != cudaSuccess) return OS_ERR_CUDA;
  if (cudaStreamSynchronize(s) != cudaSuccess) return OS_ERR_CUDA;
  if (code) *code = static_cast<int32_t>(word);
  if (!word) return OS_OK;
  return (word & 0xffu) == oss::kKernelPaged ? OS_ERR_BAD_INDEX : OS_ERR_TIMEOUT;
}

}  // extern "C"
