// Per-row rules on logits (k2_adjust_logits): penalties for ids that a row
// already holds, biases, grammar masks, in one pass over the logits.  The
// rules and their order are stated in include/k2.h.
//
// Bound by the logits' bytes, read and written once: a thread keeps 16 of them in
// registers while the row's token history is counted into shared memory (one word
// per id of the CTA's slice: bit 31 says "seen", bit 30 "has a bias", the rest
// counts the answer's occurrences), so the counts are exact whatever the order of
// the atomics.  Biases are few: those of the slice are gathered in list order, and
// the thread that holds such an id adds its entries in that order, so that an id
// listed twice gives the same sum every time.
#include <math.h>

#include <algorithm>

#include "k2_kernels.h"
#include "k2_common.cuh"
#include "../../include/k2.h"

namespace k2 {

namespace {

constexpr unsigned kSeen = 0x80000000u, kBiased = 0x40000000u, kCount = 0x3FFFFFFFu;

// VEC: every row of logits and output is 16-byte aligned
template <int THREADS, int kPerThread, bool VEC>
__global__ void __launch_bounds__(THREADS, (kPerThread == 8 ? 2048 : 1536) / THREADS) rules_kernel(const k2_logit_rules u, const float* in, long long ld, float* out,
                                                                        long long ld_out, int vocab) {
  constexpr int SLICE = THREADS * kPerThread;
  __shared__ __align__(16) unsigned cnt[SLICE];
  __shared__ int b_id[THREADS];
  __shared__ float b_val[THREADS];
  __shared__ int w_sum[THREADS / 32];
  const int r = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int v0 = blockIdx.x * SLICE, n = min(SLICE, vocab - v0);
  const float* x = in + r * ld + v0;
  float* y = out + r * ld_out + v0;
  // element j of this thread: four neighbours at a time (VEC), else strided
  auto place = [&](int j) { return VEC ? 4 * (tid + THREADS * (j >> 2)) + (j & 3) : tid + THREADS * j; };
  const bool counted = u.repetition != nullptr || u.presence != nullptr || u.frequency != nullptr;
  const int j0 = u.bias_offset != nullptr ? max(__ldg(u.bias_offset + r), 0) : 0;
  const int j1 = u.bias_offset != nullptr ? min(__ldg(u.bias_offset + r + 1), u.n_bias) : 0;
  const int len = counted ? static_cast<int>(min(static_cast<long long>(__ldg(u.ids_len + r)), static_cast<long long>(u.ids_stride))) : 0;
  const int prompt = counted && u.prompt_len != nullptr ? __ldg(u.prompt_len + r) : 0;
  const float rep = u.repetition != nullptr ? __ldg(u.repetition + r) : 1.f;
  const float freq = u.frequency != nullptr ? __ldg(u.frequency + r) : 0.f, pres = u.presence != nullptr ? __ldg(u.presence + r) : 0.f;
  const int mr = u.mask == nullptr ? -1 : u.mask_row != nullptr ? __ldg(u.mask_row + r) : r;
  float l[kPerThread];
  if constexpr (VEC) {
#pragma unroll
    for (int j = 0; j < kPerThread; j += 4) {
      const int at = place(j);
      if (at + 4 <= n) {
        const float4 f = *reinterpret_cast<const float4*>(x + at);
        l[j] = f.x;
        l[j + 1] = f.y;
        l[j + 2] = f.z;
        l[j + 3] = f.w;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) l[j + e] = at + e < n ? x[at + e] : 0.f;
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < kPerThread; ++j) l[j] = place(j) < n ? x[place(j)] : 0.f;
  }
  if (counted || j0 < j1) {
#pragma unroll
    for (int j = 0; j < kPerThread; j += 4) *reinterpret_cast<uint4*>(cnt + 4 * (tid + THREADS * (j >> 2))) = make_uint4(0, 0, 0, 0);
    // the first THREADS biases of the row: which of them lie in the slice
    unsigned d = ~0u;
    float value = 0.f;
    if (j0 + tid < j1) {
      d = static_cast<unsigned>(__ldg(u.bias_ids + j0 + tid) - v0);
      value = __ldg(u.bias + j0 + tid);
    }
    unsigned m = __ballot_sync(0xffffffffu, d < static_cast<unsigned>(n));
    if (lane == 0) w_sum[warp] = __popc(m);
    __syncthreads();
    int listed = 0;
    if (j0 < j1) {  // listed in order
      int before = 0;
#pragma unroll
      for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) before += w_sum[w];
        listed += w_sum[w];
      }
      if (d < static_cast<unsigned>(n)) {
        const int at = before + __popc(m & ((1u << lane) - 1));
        b_id[at] = static_cast<int>(d);
        b_val[at] = value;
        atomicOr(&cnt[d], kBiased);
      }
    }
    if (counted) {
      const int* ids = u.ids + r * u.ids_stride;
      auto count = [&](int id, int i) {
        const unsigned e = static_cast<unsigned>(id - v0);
        if (e < static_cast<unsigned>(n)) {
          if (i >= prompt) atomicAdd(&cnt[e], 1u);
          atomicOr(&cnt[e], kSeen);
        }
      };
      int i = 0;
      if ((reinterpret_cast<uintptr_t>(ids) & 15) == 0) {  // four ids at a time, four such loads on their way
        const int4* ids4 = reinterpret_cast<const int4*>(ids);
        const int quads = len > 0 ? len >> 2 : 0;
#pragma unroll 1
        for (int q0 = tid; q0 < quads; q0 += 4 * THREADS) {
          int4 v[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (q0 + j * THREADS < quads) v[j] = __ldg(ids4 + q0 + j * THREADS);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int q = q0 + j * THREADS;
            if (q >= quads) break;
            count(v[j].x, 4 * q);
            count(v[j].y, 4 * q + 1);
            count(v[j].z, 4 * q + 2);
            count(v[j].w, 4 * q + 3);
          }
        }
        i = 4 * quads;
      }
#pragma unroll 1
      for (i += tid; i < len; i += THREADS) count(__ldg(ids + i), i);
    }
    // a quotient as a product with the reciprocal, one rounding more: it decides nothing but a few logits' last bits
    const float inv = 1.f / rep;
    __syncthreads();
    auto touched = [&](unsigned c, float v, int at) {
      if (c & (kSeen | kCount)) {
        if (u.repetition != nullptr) v *= v > 0.f ? inv : rep;
        if (c & kCount) v = __fsub_rn(__fsub_rn(v, __fmul_rn(freq, static_cast<float>(c & kCount))), pres);
      }
      if (c & kBiased)
        for (int i = 0; i < listed; ++i)
          if (b_id[i] == at) v = __fadd_rn(v, b_val[i]);
      return v;
    };
    if constexpr (VEC) {
#pragma unroll
      for (int j = 0; j < kPerThread; j += 4) {
        const uint4 c = *reinterpret_cast<const uint4*>(cnt + place(j));
        if ((c.x | c.y | c.z | c.w) == 0) continue;
        if (c.x) l[j] = touched(c.x, l[j], place(j));
        if (c.y) l[j + 1] = touched(c.y, l[j + 1], place(j + 1));
        if (c.z) l[j + 2] = touched(c.z, l[j + 2], place(j + 2));
        if (c.w) l[j + 3] = touched(c.w, l[j + 3], place(j + 3));
      }
    } else {
#pragma unroll
      for (int j = 0; j < kPerThread; ++j) {
        const unsigned c = cnt[place(j)];
        if (c) l[j] = touched(c, l[j], place(j));
      }
    }
    // further biases, THREADS at a time
#pragma unroll 1
    for (int k = j0 + THREADS; k < j1; k += THREADS) {
      __syncthreads();
      for (int i = tid; i < listed; i += THREADS) cnt[b_id[i]] &= ~kBiased;  // (an id listed twice: the same store)
      d = k + tid < j1 ? static_cast<unsigned>(__ldg(u.bias_ids + k + tid) - v0) : ~0u;
      const bool take = d < static_cast<unsigned>(n);
      m = __ballot_sync(0xffffffffu, take);
      if (lane == 0) w_sum[warp] = __popc(m);
      __syncthreads();
      int before = 0;
      listed = 0;
#pragma unroll 1
      for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) before += w_sum[w];
        listed += w_sum[w];
      }
      if (take) {
        const int at = before + __popc(m & ((1u << lane) - 1));
        b_id[at] = static_cast<int>(d);
        b_val[at] = __ldg(u.bias + k + tid);
        atomicOr(&cnt[d], kBiased);
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < kPerThread; ++j) {
        const int at = place(j);
        if (cnt[at] & kBiased) l[j] = touched(kBiased, l[j], at);
      }
    }
  }
  const bool masked = mr >= 0 && mr < u.n_masks;
  const unsigned* words = masked ? u.mask + mr * u.mask_stride : nullptr;
  if constexpr (VEC) {
#pragma unroll
    for (int j = 0; j < kPerThread; j += 4) {
      const int at = place(j);
      if (at >= n) break;
      if (masked) {  // four neighbours lie in one word
        const unsigned bits = __ldg(words + ((v0 + at) >> 5)) >> ((v0 + at) & 31);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (!((bits >> e) & 1u)) l[j + e] = -INFINITY;
      }
      if (at + 4 <= n) {
        *reinterpret_cast<float4*>(y + at) = make_float4(l[j], l[j + 1], l[j + 2], l[j + 3]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (at + e < n) y[at + e] = l[j + e];
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < kPerThread; ++j) {
      const int at = place(j);
      if (at >= n) break;
      if (masked && !((__ldg(words + ((v0 + at) >> 5)) >> ((v0 + at) & 31)) & 1u)) l[j] = -INFINITY;
      y[at] = l[j];
    }
  }
}

template <int THREADS, int kPerThread>
cudaError_t launch_rules(const k2_logit_rules& u, const float* in, long long ld, float* out, long long ld_out, int rows, int vocab,
                         cudaStream_t s) {
  const bool vec = ((reinterpret_cast<uintptr_t>(in) | reinterpret_cast<uintptr_t>(out)) & 15) == 0 &&
                   (rows == 1 || ((ld | ld_out) & 3) == 0);
  const dim3 grid((vocab + THREADS * kPerThread - 1) / (THREADS * kPerThread), rows);
  if (vec) rules_kernel<THREADS, kPerThread, true><<<grid, THREADS, 0, s>>>(u, in, ld, out, ld_out, vocab);
  else rules_kernel<THREADS, kPerThread, false><<<grid, THREADS, 0, s>>>(u, in, ld, out, ld_out, vocab);
  return cudaGetLastError();
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
  // each slice reads its row's whole history: large slices (64 rows of 250624: 44 us, against 48 with slices of half the
  // size), unless they leave SMs idle and the history is short (one row: 3.9 us, against 4.9)
  const long long large = static_cast<long long>(rows) * ((vocab + 8191) / 8192);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = large >= 152 || (u->ids && u->ids_stride > 4096) ? launch_rules<512, 16>(*u, d_logits, ld, d_out, ld_out, rows, vocab, st)
                                                                         : launch_rules<256, 8>(*u, d_logits, ld, d_out, ld_out, rows, vocab, st);
  if (e == cudaSuccess) return K2_OK;
  set_error("logit rules launch: %s", cudaGetErrorString(e));
  return K2_ERR_CUDA;
}
