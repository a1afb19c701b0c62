// Per-row rules on logits (k2_adjust_logits): penalties for ids that a row
// already holds, biases, grammar masks, in one pass over the logits.  The
// rules and their order are stated in include/k2.h.
//
// Bound by the logits' bytes, read and written once.  A CTA takes a slice of a row's vocabulary and counts the row's
// token history into shared memory, a cell per id: the answer's occurrences, and a top bit for ids of the prompt; so the
// counts are exact whatever the order of the atomics, and a cell of zero means that no penalty touches the id.  Then the
// slice streams through registers.  Every slice reads its row's whole history, so slices are as large as still gives
// every SM three of them.  64 rows of 250624 with up to 8192 tokens and 300 biases each take 33 us, 4.0 TB/s (44 with
// slices of 8192 held in registers, 52 with those staged in shared memory by bulk copies; a prefetch of the slice to L2
// changes nothing); 256 rows 116 us, 4.5 TB/s; one row, where every step of the way there is a latency, 4.1 us.
//
// Biases are few.  The thread that finds the first entry of an id in the slice works that id out by itself, all its
// entries in list order, so that an id listed twice gives the same sum every time; it stores the result after the slice.
#include <limits.h>
#include <math.h>

#include <algorithm>
#include <atomic>

#include "k2_serve.h"
#include "k2_common.cuh"
#include "../../include/k2.h"

namespace k2 {

namespace {

constexpr int kThreads = 512, kCtas = 3;  // per SM
constexpr int kCellBytes = 71680;         // of a CTA, at most: three CTAs fill an SM's shared memory
constexpr int kMinSlice = 2048;

// A slice's cells: 16 bits for histories of up to 32767 tokens, else 32 bits.
template <typename Cell>
struct Cells {
  static constexpr int kPerWord = 4 / sizeof(Cell), kBits = 8 * sizeof(Cell);
  static constexpr unsigned kPrompt = 1u << (kBits - 1), kCount = kPrompt - 1u;
  __device__ static void add(unsigned* words, unsigned e, bool prompt) {
    const unsigned shift = kPerWord == 1 ? 0 : (e & 1u) * 16u;
    if (prompt) atomicOr(words + e / kPerWord, kPrompt << shift);
    else atomicAdd(words + e / kPerWord, 1u << shift);
  }
  __device__ static unsigned get(const unsigned* words, int e) { return reinterpret_cast<const Cell*>(words)[e]; }
};

// What the rules say about one row
struct Row {
  int j0, j1;        // its biases
  int len, prompt;   // its tokens, and how many of them are the prompt
  float rep, freq, pres;
  const unsigned* mask;
};
__device__ __forceinline__ Row row_of(const k2_logit_rules& u, int r, bool counted) {
  Row w;
  w.j0 = u.bias_offset != nullptr ? min(max(__ldg(u.bias_offset + r), 0), u.n_bias) : 0;
  w.j1 = u.bias_offset != nullptr ? min(__ldg(u.bias_offset + r + 1), u.n_bias) : 0;
  w.len = counted ? static_cast<int>(min(static_cast<long long>(__ldg(u.ids_len + r)), static_cast<long long>(u.ids_stride))) : 0;
  w.prompt = counted && u.prompt_len != nullptr ? __ldg(u.prompt_len + r) : 0;
  w.rep = u.repetition != nullptr ? __ldg(u.repetition + r) : 1.f;
  w.freq = u.frequency != nullptr ? __ldg(u.frequency + r) : 0.f;
  w.pres = u.presence != nullptr ? __ldg(u.presence + r) : 0.f;
  const int m = u.mask == nullptr ? -1 : u.mask_row != nullptr ? __ldg(u.mask_row + r) : r;
  w.mask = m >= 0 && m < u.n_masks ? u.mask + m * u.mask_stride : nullptr;
  return w;
}

// counts the row's tokens that lie in the slice [v0, v0 + n)
template <typename Cell>
__device__ __forceinline__ void count_ids(unsigned* words, const int* ids, const Row& w, int v0, int n) {
  auto count = [&](int id, int i) {
    const unsigned e = static_cast<unsigned>(id) - static_cast<unsigned>(v0);
    if (e < static_cast<unsigned>(n)) Cells<Cell>::add(words, e, i < w.prompt);
  };
  int i = 0;
  if ((reinterpret_cast<uintptr_t>(ids) & 15) == 0) {  // four ids at a time, four such loads on their way
    const int4* ids4 = reinterpret_cast<const int4*>(ids);
    const int quads = w.len > 0 ? w.len >> 2 : 0;
#pragma unroll 1
    for (int q0 = threadIdx.x; q0 < quads; q0 += 4 * kThreads) {
      int4 v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (q0 + j * kThreads < quads) v[j] = __ldg(ids4 + q0 + j * kThreads);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int q = q0 + j * kThreads;
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
  for (i += threadIdx.x; i < w.len; i += kThreads) count(__ldg(ids + i), i);
}

// The penalties of an id whose cell is c (not zero).
template <typename Cell>
__device__ __forceinline__ float penalised(const Row& w, bool repeats, unsigned c, float v) {
  if (repeats) v = v > 0.f ? __fdiv_rn(v, w.rep) : v * w.rep;
  const unsigned times = c & Cells<Cell>::kCount;
  if (times) v = __fsub_rn(__fsub_rn(v, __fmul_rn(w.freq, static_cast<float>(times))), w.pres);
  return v;
}

// The biases j .. j + 511 that lie in the slice, in order, in b_id and b_val; how many.  All threads; ends with a barrier.
__device__ __forceinline__ int list_biases(const k2_logit_rules& u, int j, int j1, int v0, int n, int* b_id, float* b_val, int* w_sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned d = ~0u;
  float value = 0.f;
  if (static_cast<int>(threadIdx.x) < j1 - j) {
    d = static_cast<unsigned>(__ldg(u.bias_ids + j + threadIdx.x)) - static_cast<unsigned>(v0);
    value = __ldg(u.bias + j + threadIdx.x);
  }
  const unsigned m = __ballot_sync(0xffffffffu, d < static_cast<unsigned>(n));
  if (lane == 0) w_sum[warp] = __popc(m);
  __syncthreads();
  int before = 0, listed = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += w_sum[w];
    listed += w_sum[w];
  }
  if (d < static_cast<unsigned>(n)) {
    const int at = before + __popc(m & ((1u << lane) - 1));
    b_id[at] = static_cast<int>(d);
    b_val[at] = value;
  }
  __syncthreads();
  return listed;
}
// Adds to v the listed biases of the id of entry i, in order; whether entry i is its first.  The loop is the same for all
// lanes of a warp (with bounds of their own, the lanes ran one after another: 57 us for the 64 rows above).
__device__ __forceinline__ bool add_biases(const int* b_id, const float* b_val, int i, int listed, float& v) {
  const int id = b_id[i];
  bool first = true;
#pragma unroll 4
  for (int k = 0; k < listed; ++k) {
    const bool same = b_id[k] == id;
    first = first && !(same && k < i);
    v = same ? __fadd_rn(v, b_val[k]) : v;
  }
  return first;
}

// VEC: every row of logits and output is 16-byte aligned.
template <typename Cell, bool VEC>
__global__ void __launch_bounds__(kThreads, kCtas)
    rules_kernel(const k2_logit_rules u, const float* in, long long ld, float* out, long long ld_out, int vocab, int slice) {
  extern __shared__ __align__(16) unsigned words[];
  __shared__ int b_id[kThreads];
  __shared__ float b_val[kThreads];
  __shared__ int w_sum[kThreads / 32];
  using C = Cells<Cell>;
  constexpr int U = VEC ? 2 : 8, W = VEC ? 4 : 1;  // steps at a time, logits of a step
  const int r = blockIdx.y, tid = threadIdx.x;
  const int v0 = blockIdx.x * slice, n = min(slice, vocab - v0);
  const float* x = in + r * ld + v0;
  float* y = out + r * ld_out + v0;
  const bool counted = u.repetition != nullptr || u.presence != nullptr || u.frequency != nullptr;
  const bool repeats = u.repetition != nullptr;
  const Row w = row_of(u, r, counted);
  auto allowed = [&](int at) { return w.mask == nullptr || ((__ldg(w.mask + ((v0 + at) >> 5)) >> ((v0 + at) & 31)) & 1u); };

  if (counted) {
    for (int i = 4 * tid; i < (n + C::kPerWord - 1) / C::kPerWord; i += 4 * kThreads) *reinterpret_cast<uint4*>(words + i) = make_uint4(0, 0, 0, 0);
    __syncthreads();
    count_ids<Cell>(words, u.ids + r * u.ids_stride, w, v0, n);
    __syncthreads();
  }
  bool mine = false;  // an id with biases is this thread's
  int my_at = 0;
  float my_value = 0.f;
  if (w.j0 < w.j1) {
    const int listed = list_biases(u, w.j0, w.j1, v0, n, b_id, b_val, w_sum);
    if (tid < listed) {
      my_at = b_id[tid];
      mine = allowed(my_at);
      my_value = x[my_at];
      const unsigned c = counted ? C::get(words, my_at) : 0u;
      if (c) my_value = penalised<Cell>(w, repeats, c, my_value);
      mine = add_biases(b_id, b_val, tid, listed, my_value) && mine;
    }
    __syncthreads();  // in place, x before the slice's stores
  }

#pragma unroll 1
  for (int base = W * tid; base < n; base += U * W * kThreads) {
    if constexpr (VEC) {
      float4 f[U];
      unsigned bits[U];
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int at = base + j * 4 * kThreads;
        bits[j] = w.mask != nullptr && at < n ? __ldg(w.mask + ((v0 + at) >> 5)) >> ((v0 + at) & 31) : 0xFu;
        if (at + 4 <= n) f[j] = *reinterpret_cast<const float4*>(x + at);
        else f[j] = make_float4(at < n ? x[at] : 0.f, at + 1 < n ? x[at + 1] : 0.f, at + 2 < n ? x[at + 2] : 0.f, 0.f);
      }
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int at = base + j * 4 * kThreads;
        if (at >= n) break;
        if (counted) {
          unsigned c0, c1, c2, c3;
          if constexpr (C::kPerWord == 2) {
            const uint2 c = *reinterpret_cast<const uint2*>(words + at / 2);
            c0 = c.x & 0xFFFFu, c1 = c.x >> 16, c2 = c.y & 0xFFFFu, c3 = c.y >> 16;
          } else {
            const uint4 c = *reinterpret_cast<const uint4*>(words + at);
            c0 = c.x, c1 = c.y, c2 = c.z, c3 = c.w;
          }
          if (c0 | c1 | c2 | c3) {
            if (c0) f[j].x = penalised<Cell>(w, repeats, c0, f[j].x);
            if (c1) f[j].y = penalised<Cell>(w, repeats, c1, f[j].y);
            if (c2) f[j].z = penalised<Cell>(w, repeats, c2, f[j].z);
            if (c3) f[j].w = penalised<Cell>(w, repeats, c3, f[j].w);
          }
        }
        if (!(bits[j] & 1u)) f[j].x = -INFINITY;
        if (!(bits[j] & 2u)) f[j].y = -INFINITY;
        if (!(bits[j] & 4u)) f[j].z = -INFINITY;
        if (!(bits[j] & 8u)) f[j].w = -INFINITY;
        if (at + 4 <= n) {
          *reinterpret_cast<float4*>(y + at) = f[j];
        } else {
          y[at] = f[j].x;
          if (at + 1 < n) y[at + 1] = f[j].y;
          if (at + 2 < n) y[at + 2] = f[j].z;
        }
      }
    } else {
      float f[U];
#pragma unroll
      for (int j = 0; j < U; ++j) f[j] = base + j * kThreads < n ? x[base + j * kThreads] : 0.f;
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int at = base + j * kThreads;
        if (at >= n) break;
        const unsigned c = counted ? C::get(words, at) : 0u;
        if (c) f[j] = penalised<Cell>(w, repeats, c, f[j]);
        y[at] = allowed(at) ? f[j] : -INFINITY;
      }
    }
  }

  if (w.j0 < w.j1) {
    __syncthreads();
    if (mine) y[my_at] = my_value;
#pragma unroll 1
    for (int j = w.j0 + kThreads; j < w.j1; j += kThreads) {  // long lists: on what the entries before have left
      __syncthreads();
      const int listed = list_biases(u, j, w.j1, v0, n, b_id, b_val, w_sum);
      if (tid < listed) {
        float v = y[b_id[tid]];
        const bool first = add_biases(b_id, b_val, tid, listed, v);
        if (first && allowed(b_id[tid])) y[b_id[tid]] = v;
      }
    }
  }
}

template <typename Cell, bool VEC>
cudaError_t launch_rules(const k2_logit_rules& u, const float* in, long long ld, float* out, long long ld_out, int rows, int vocab,
                         cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (!e) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e) return e;
  if (dev >= 64) return cudaErrorInvalidDevice;
  static std::atomic<uint64_t> ready{0};
  const uint64_t bit = 1ull << dev;
  if (!(ready.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(rules_kernel<Cell, VEC>, cudaFuncAttributeMaxDynamicSharedMemorySize, kCellBytes);
    if (e) return e;
    ready.fetch_or(bit, std::memory_order_release);
  }
  // as many slices as the SMs take at once, if none gets too small or too large for that
  constexpr int kMaxSlice = kCellBytes / static_cast<int>(sizeof(Cell));
  int per_row = std::min(kCtas * sms / rows, (vocab + kMinSlice - 1) / kMinSlice);
  per_row = std::max(per_row, (vocab + kMaxSlice - 1) / kMaxSlice);
  const int slice = ((vocab + per_row - 1) / per_row + 31) & ~31;
  const dim3 grid((vocab + slice - 1) / slice, rows);
  const bool counted = u.repetition || u.presence || u.frequency;
  rules_kernel<Cell, VEC><<<grid, kThreads, counted ? slice * sizeof(Cell) : 0, s>>>(u, in, ld, out, ld_out, vocab, slice);
  return cudaGetLastError();
}

}  // namespace

}  // namespace k2

using namespace k2;

extern "C" k2_status k2_adjust_logits(const k2_logit_rules* u, const float* d_logits, int64_t ld, float* d_out,
                                      int64_t ld_out, int32_t rows, int32_t vocab, void* stream) {
  if (!u || rows < 0 || vocab < 1 || vocab > 1 << 30) {
    set_error("rules must be non-null, rows >= 0 and vocab 1 .. 2^30");
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
  if (d_logits != d_out && rows_meet(d_logits, 4 * ld, d_out, 4 * ld_out, 4ll * vocab, rows)) {
    set_error("the output may be the logits, but not lie over a part of them");
    return K2_ERR_ARG;
  }
  if ((u->repetition || u->presence || u->frequency) && !u->ids) {
    set_error("penalties need the rows' token ids");
    return K2_ERR_ARG;
  }
  if (u->ids && (!u->ids_len || u->ids_stride < 0 || u->ids_stride > 1 << 30)) {
    set_error("ids need ids_len and ids_stride 0 .. 2^30");
    return K2_ERR_ARG;
  }
  if (u->bias_offset && (!u->bias_ids || !u->bias || u->n_bias < 0 || u->n_bias > 1 << 30)) {
    set_error("biases need bias_ids, bias and n_bias 0 .. 2^30");
    return K2_ERR_ARG;
  }
  if (u->mask && (u->n_masks < 1 || (u->n_masks > 1 && u->mask_stride < (static_cast<int64_t>(vocab) + 31) / 32))) {
    set_error("masks need n_masks >= 1 and rows of at least ceil(vocab / 32) words");
    return K2_ERR_ARG;
  }
  const bool vec = ((reinterpret_cast<uintptr_t>(d_logits) | reinterpret_cast<uintptr_t>(d_out)) & 15) == 0 &&
                   (rows == 1 || ((ld | ld_out) & 3) == 0);
  const bool small = !u->ids || u->ids_stride <= 32767;
  const auto launch = small ? (vec ? launch_rules<uint16_t, true> : launch_rules<uint16_t, false>)
                            : (vec ? launch_rules<uint32_t, true> : launch_rules<uint32_t, false>);
  const cudaError_t e = launch(*u, d_logits, ld, d_out, ld_out, rows, vocab, static_cast<cudaStream_t>(stream));
  if (e == cudaSuccess) return K2_OK;
  set_error("logit rules launch: %s", cudaGetErrorString(e));
  return K2_ERR_CUDA;
}
