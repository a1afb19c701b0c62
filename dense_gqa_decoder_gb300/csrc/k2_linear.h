// Rows as E4M3 codes, and the matrix product that reads them: what the entry points and the model's layers share.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/k2.h"

namespace k2 {

// What k2_quantize_rows and k2_norm_quantize take: rows of up to kMaxRowCols values (as fp32 in shared memory: 192 KB), and
// for the norm an eps that is a normal number.
constexpr int kMaxRowCols = 49152;
constexpr float kMinEps = 0x1p-126f;

// A product as the kernels see it (k2_linear_args, checked).
struct LinearArgs {
  const float* w_scale;  // null: none
  const float* x_scale;
  const float* bias;
  const void* residual;
  long long residual_stride;
  void* out;
  long long out_stride;
  int tokens, rows, cols;  // rows: of the weight matrix
  int dtype, out_dtype, act;
  unsigned* flags;         // nullable; raised with `bit` when a wait runs out
  unsigned bit;
  unsigned long long limit_ns;
};

// The weights [rows][cols] of a product: rows `stride` elements apart, or (packed) pairs of rows in 512-byte chunks, as
// the decode step streams them.
struct LinearWeights {
  const void* base;
  long long stride;
  bool packed;
};

// `n` rows of `row` bytes, `stride` bytes apart
struct RowSet {
  const void* p;
  int64_t stride, row, n;
};
// Whether two sets share a byte.  Sets of the same stride may be slices of the same wider rows; others are compared by the
// memory from their first byte to their last.
inline bool sets_meet(const RowSet& a, const RowSet& b) {
  if (!a.p || !b.p || a.n < 1 || b.n < 1) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  const uintptr_t a1 = a0 + (a.n - 1) * a.stride + a.row, b1 = b0 + (b.n - 1) * b.stride + b.row;
  if (a1 <= b0 || b1 <= a0) return false;
  if (a.n < 2 || b.n < 2 || a.stride != b.stride) return true;
  const int64_t d = b0 >= a0 ? static_cast<int64_t>((b0 - a0) % a.stride)  // from a row of a to the next start of a row of b
                             : (a.stride - static_cast<int64_t>((a0 - b0) % a.stride)) % a.stride;
  return d < a.row || a.stride - d < b.row;
}

// fp8 codes [N][K] in the decode step's tile units as packed pairs (k2_gemv_packed.cu)
cudaError_t launch_f8_pairs(uint8_t* dst, const uint8_t* src, int N, int K, cudaStream_t s);

// launch_prefill_attn with fp32 rows in place of bf16 halves (k2_prefill.cu)
cudaError_t launch_prefill_attn_f32(const float* Q, int kv_dtype, const void* kc, const void* vc, const void* ks, const void* vs,
                                    float* out, int n, int nq, int nkv, int D, int pos0, size_t head_row0, int cap, float scale,
                                    cudaStream_t s);

k2_status launch_linear(const LinearWeights& w, const void* x, long long x_stride, const LinearArgs& a, cudaStream_t s);

}  // namespace k2
