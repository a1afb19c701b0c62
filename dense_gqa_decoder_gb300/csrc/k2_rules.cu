// Per-row rules on logits (k2_adjust_logits): penalties for ids that a row
// already holds, biases, grammar masks, in one pass over the logits.  The
// rules and their order are stated in include/k2.h.
//
// A CTA takes a slice of one row's vocabulary.  The row's token history is
// read once per slice and counted into shared memory (one word per id: bit 31
// says "seen", the rest counts the answer's occurrences), so the counts are
// exact whatever the order of the atomics; the biases of the slice are added
// by one warp in list order, so that an id listed twice gives the same sum
// every time.  Then one pass reads the logits and writes the result.
#include <math.h>

#include <algorithm>

#include "k2_kernels.h"
#include "k2_common.cuh"
#include "../../include/k2.h"

namespace k2 {

namespace {

constexpr int kRuleThreads = 512;
constexpr int kRuleSlice = 8192;  // ids of one CTA: 64 KB of shared memory
constexpr unsigned kSeen = 0x80000000u;

__global__ void __launch_bounds__(kRuleThreads) rules_kernel(const k2_logit_rules u, const float* in, long long ld,
                                                             float* out, long long ld_out, int vocab) {
  extern __shared__ unsigned smem[];
  unsigned* cnt = smem;
  float* val = reinterpret_cast<float*>(smem + kRuleSlice);
  const int r = blockIdx.y, tid = threadIdx.x;
  const int v0 = blockIdx.x * kRuleSlice, n = min(kRuleSlice, vocab - v0);
  const float* x = in + r * ld + v0;
  float* y = out + r * ld_out + v0;
  for (int i = tid; i < n; i += kRuleThreads) {
    cnt[i] = 0;
    val[i] = x[i];
  }
  __syncthreads();
  if (u.ids != nullptr) {
    const int* ids = u.ids + r * u.ids_stride;
    const int len = static_cast<int>(min(static_cast<long long>(u.ids_len[r]), static_cast<long long>(u.ids_stride)));
    const int prompt = u.prompt_len != nullptr ? u.prompt_len[r] : 0;
    for (int i = tid; i < len; i += kRuleThreads) {
      const unsigned d = static_cast<unsigned>(ids[i] - v0);
      if (d < static_cast<unsigned>(n)) {
        atomicOr(&cnt[d], kSeen);
        if (i >= prompt) atomicAdd(&cnt[d], 1u);
      }
    }
    __syncthreads();
    const float rep = u.repetition != nullptr ? u.repetition[r] : 1.f;
    const float freq = u.frequency != nullptr ? u.frequency[r] : 0.f, pres = u.presence != nullptr ? u.presence[r] : 0.f;
    for (int i = tid; i < n; i += kRuleThreads) {
      const unsigned c = cnt[i];
      if (c == 0) continue;
      float l = val[i];
      if (u.repetition != nullptr) l = l > 0.f ? __fdiv_rn(l, rep) : __fmul_rn(l, rep);
      if (c != kSeen) l = __fsub_rn(__fsub_rn(l, __fmul_rn(freq, static_cast<float>(c & ~kSeen))), pres);
      val[i] = l;
    }
    __syncthreads();
  }
  if (u.bias_offset != nullptr) {
    if (tid == 0) {
      for (int j = max(u.bias_offset[r], 0); j < min(u.bias_offset[r + 1], u.n_bias); ++j) {
        const unsigned d = static_cast<unsigned>(u.bias_ids[j] - v0);
        if (d < static_cast<unsigned>(n)) val[d] += u.bias[j];
      }
    }
    __syncthreads();
  }
  const int mr = u.mask == nullptr ? -1 : u.mask_row != nullptr ? u.mask_row[r] : r;
  const bool masked = mr >= 0 && mr < u.n_masks;
  const unsigned* words = masked ? u.mask + mr * u.mask_stride : nullptr;
  for (int i = tid; i < n; i += kRuleThreads) {
    const int id = v0 + i;
    y[i] = masked && !((words[id >> 5] >> (id & 31)) & 1u) ? -INFINITY : val[i];
  }
}

}  // namespace

}  // namespace k2

using namespace k2;

extern "C" k2_status k2_adjust_logits(const k2_logit_rules* u, const float* d_logits, int64_t ld, float* d_out,
                                      int64_t ld_out, int32_t rows, int32_t vocab, void* stream) {
  if (!u || rows < 0 || vocab < 1) {
    set_error("rules must be non-null, rows >= 0 and vocab >= 1");
    return K2_ERR_ARG;
  }
  if (rows == 0) return K2_OK;
  if (!d_logits || !d_out || reinterpret_cast<uintptr_t>(d_logits) % 4 || reinterpret_cast<uintptr_t>(d_out) % 4) {
    set_error("d_logits and d_out must be non-null float pointers");
    return K2_ERR_ARG;
  }
  if (rows > 65535 || (rows > 1 && (ld < vocab || ld_out < vocab))) {
    set_error("rows of at least vocab elements, at most 65535 of them (got %d rows, ld %lld and %lld)", rows,
              static_cast<long long>(ld), static_cast<long long>(ld_out));
    return K2_ERR_SHAPE;
  }
  if (d_logits == d_out && rows > 1 && ld != ld_out) {
    set_error("in place, both leading dimensions must be the same");
    return K2_ERR_ARG;
  }
  if ((u->repetition || u->presence || u->frequency) && !u->ids) {
    set_error("penalties need the rows' token ids");
    return K2_ERR_ARG;
  }
  if (u->ids && (!u->ids_len || u->ids_stride < 0)) {
    set_error("ids need ids_len and ids_stride >= 0");
    return K2_ERR_ARG;
  }
  if (u->bias_offset && (!u->bias_ids || !u->bias || u->n_bias < 0)) {
    set_error("biases need bias_ids, bias and n_bias >= 0");
    return K2_ERR_ARG;
  }
  if (u->mask && (u->n_masks < 1 || (u->n_masks > 1 && u->mask_stride < (static_cast<int64_t>(vocab) + 31) / 32))) {
    set_error("masks need n_masks >= 1 and rows of at least ceil(vocab / 32) words");
    return K2_ERR_ARG;
  }
  const int smem = 8 * kRuleSlice;
  cudaError_t e = cudaFuncSetAttribute(rules_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess) {
    const dim3 grid((vocab + kRuleSlice - 1) / kRuleSlice, rows);
    rules_kernel<<<grid, kRuleThreads, smem, static_cast<cudaStream_t>(stream)>>>(*u, d_logits, ld, d_out, ld_out, vocab);
    e = cudaGetLastError();
  }
  if (e == cudaSuccess) return K2_OK;
  set_error("logit rules launch: %s", cudaGetErrorString(e));
  return K2_ERR_CUDA;
}
