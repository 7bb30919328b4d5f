// around.cuh -- declarations shared by the operators around the packed cache
// (norm and rotation, paged append, shared-history and cross attention).
#pragma once
#include <atomic>

#include "common.cuh"

namespace qwm {

// Whether an offset, length or page number read from a device array had to be
// clamped since the last call (1 or 0; -1: CUDA error).
int read_and_clear_append_fault();
int read_and_clear_flash_fault();
int read_and_clear_flash_timeout();

// Attention of few rows per head over the packed tokens (attention_rows.cu): one
// fp32 partial per row, query head and slot; empty slots get a log-sum-exp of -inf.
struct RowsPlan {
  int grid, slots;
};
bool rows_supported(const Dims& D, int64_t T, int64_t rows, int sms);  // rows: query rows per key head
// K' and V' of `heads` heads from h0 on, [head][T][d] bf16.
cudaError_t launch_unpack(const Dims& D, const CacheView& v, int64_t T, int h0, int heads,
                          uint16_t* K, uint16_t* V, int sms, cudaStream_t s);
RowsPlan rows_plan(const Dims& D, int64_t T, int sms, int most);  // at most `most` >= 3 slots
cudaError_t launch_rows(const Dims& D, const CacheView& v, int64_t T, const uint16_t* Q, int64_t ldq,
                        int64_t nq, int Hq, float scale_log2, const RowsPlan& plan, float* ws_o,
                        float* ws_l, cudaStream_t s);

// Raise a kernel's dynamic shared memory limit to the most it may use, once per
// device (the attribute costs a call about a microsecond).  `done`: one per kernel.
template <class Kernel>
cudaError_t allow_smem(Kernel kern, std::atomic<uint64_t>& done, int bytes) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

inline bool aligned_to(const void* p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }

inline int page_shift(const qwm_pages* p) {
  int s = 0;
  while ((1 << s) < p->page_size) ++s;
  return s;
}

inline bool pages_ok(const qwm_pages* p) {
  if (!p || !p->K || !p->V || p->n_pages < 1 || p->n_pages > (int64_t(1) << 31) - 1) return false;
  if (p->heads < 1 || p->heads > 4096 || (p->head_dim != 64 && p->head_dim != 128)) return false;
  if (p->page_size < 16 || p->page_size > 256 || (p->page_size & (p->page_size - 1))) return false;
  return p->reserved == 0;
}

}  // namespace qwm
