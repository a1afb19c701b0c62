// Host side of serving many requests: the row kernels of a step over a block-paged cache, and the message of the calls
// that need no context.  (Apart from k2_kernels.h, whose contents date the measured traffic of the decode step.)
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace k2 {

// ---- a step over a block-paged cache (k2_prefill.cu)
// split-half RoPE of packed QKV rows at positions[t]: q [n][nq * D] as fp16 (a value beyond its range raises
// GUARD_RANGE), k | v [n][2 nkv * D] fp32; a position outside [0, cap) raises GUARD_POS and counts as 0
cudaError_t launch_rope_rows(const float* qkv, __half* q, float* kv, const float2* rope, const int* positions, int n,
                             int nq, int nkv, int D, int cap, unsigned* guard, cudaStream_t s);
// fp16 values as bf16 hi + lo (exact)
cudaError_t launch_half_hilo(const __half* x, __nv_bfloat16* oh, __nv_bfloat16* ol, size_t n, cudaStream_t s);
// row r of out = row cu[r + 1] - 1 of X (n rows), zeros for a request without rows
cudaError_t launch_last_rows(const float* X, const int* cu, int requests, int n, float* out, int H, cudaStream_t s);
// next[r] = arg[r] for the requests with rows
cudaError_t launch_active_next(const int* arg, const int* cu, int requests, int* next, cudaStream_t s);

// Whether two sets of n rows of `row` bytes, each `stride` >= row bytes apart, share a byte (slices of the same wider
// rows need not).  Sets of different strides are compared by their first rows alone.
inline bool rows_meet(const void* a, int64_t a_stride, const void* b, int64_t b_stride, int64_t row, int64_t n) {
  const int64_t d = static_cast<int64_t>(reinterpret_cast<uintptr_t>(b) - reinterpret_cast<uintptr_t>(a));
  if (n < 2 || a_stride != b_stride || a_stride < 1) return d > -row && d < row;
  int64_t k = d / a_stride, m = d % a_stride;  // b's row 0 lies m bytes behind the start of a's row k
  if (m < 0) m += a_stride, --k;
  return (m < row && k > -n && k < n) || (a_stride - m < row && k + 1 > -n && k + 1 < n);
}

// The message of k2_last_error(NULL): why this thread's last call without a context was refused.
void set_error(const char* fmt, ...);

}  // namespace k2
