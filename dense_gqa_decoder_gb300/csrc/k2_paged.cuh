// What the operators over a block-paged 8-bit cache share: their checks of the
// pool's descriptor, the two code formats, and the arguments of the kernels.
#pragma once

#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "../../include/k2.h"
#include "k2_common.cuh"
#include "k2_serve.h"

namespace k2 {

inline bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// K2_OK, or why the pool of a call cannot be used (set_error says it in words)
inline k2_status check_paged_kv(const k2_paged_kv* kv) {
  if (!kv || !kv->k || !kv->v || !kv->k_scale || !kv->v_scale) {
    set_error("the pool's k, v, k_scale and v_scale must be non-null");
    return K2_ERR_ARG;
  }
  if (!aligned16(kv->k) || !aligned16(kv->v)) {
    set_error("the pool's k and v must be 16-byte aligned");
    return K2_ERR_ARG;
  }
  if (kv->dtype != K2_I8 && kv->dtype != K2_F8) {
    set_error("a paged cache holds K2_I8 or K2_F8 codes (got dtype %d)", kv->dtype);
    return K2_ERR_UNSUPPORTED;
  }
  if (kv->block_tokens != 16 && kv->block_tokens != 32 && kv->block_tokens != 64 && kv->block_tokens != 128) {
    set_error("block_tokens must be 16, 32, 64 or 128 (got %d)", kv->block_tokens);
    return K2_ERR_UNSUPPORTED;
  }
  if (kv->head_dim != 64 && kv->head_dim != 128) {
    set_error("head_dim must be 64 or 128 (got %d)", kv->head_dim);
    return K2_ERR_UNSUPPORTED;
  }
  if (kv->n_kv_heads < 1 || kv->n_kv_heads > 128 || kv->n_blocks < 1) {
    set_error("n_kv_heads must be in [1, 128] and n_blocks >= 1 (got %d, %d)", kv->n_kv_heads, kv->n_blocks);
    return K2_ERR_SHAPE;
  }
  if (kv->wait_limit_us < 0) {
    set_error("wait_limit_us must be >= 0 (got %d)", kv->wait_limit_us);
    return K2_ERR_ARG;
  }
  // slots are 32-bit numbers, and so are the kernels' places in units of 16 rows of all heads
  if (static_cast<int64_t>(kv->n_blocks) * kv->block_tokens > INT32_MAX ||
      static_cast<int64_t>(kv->n_blocks) * kv->block_tokens / 16 * kv->n_kv_heads >= UINT32_MAX) {
    set_error("n_blocks * block_tokens must stay below 2^31, and times n_kv_heads below 2^36");
    return K2_ERR_SHAPE;
  }
  return K2_OK;
}

// A pool as the kernels see it; row r of KV head g of block b starts at code
// ((b * n_kv + g) * block + r) * head_dim (a 64-bit offset).
struct PagedPool {
  uint8_t* k;
  uint8_t* v;
  float* ks;
  float* vs;
  int n_blocks, n_kv;
  int block_log2;
  unsigned* flags;

  explicit PagedPool(const k2_paged_kv& kv)
      : k(static_cast<uint8_t*>(kv.k)), v(static_cast<uint8_t*>(kv.v)), ks(kv.k_scale), vs(kv.v_scale),
        n_blocks(kv.n_blocks), n_kv(kv.n_kv_heads),
        block_log2(kv.block_tokens == 16 ? 4 : kv.block_tokens == 32 ? 5 : kv.block_tokens == 64 ? 6 : 7),
        flags(kv.flags) {}
};

__device__ __forceinline__ void raise_flag(unsigned* flags, unsigned bit) {
  if (flags != nullptr) atomicOr(flags, bit);
}

// The two code formats.  code(x, s): x / s rounded to a code (nearest, ties to
// even; NaN and everything under s = 0 give 0, what lies beyond is clamped);
// value(c): the code's value in units of the scale.
struct CodeI8 {
  static constexpr float kMax = 127.0f;
  __device__ __forceinline__ static uint32_t round(float y) {
    return static_cast<uint32_t>(__float2int_rn(fminf(fmaxf(y, -127.f), 127.f))) & 0xFFu;
  }
  __device__ __forceinline__ static float value(uint32_t c) { return static_cast<float>(static_cast<int8_t>(c)); }
};
struct CodeF8 {
  static constexpr float kMax = 448.0f;
  __device__ __forceinline__ static uint32_t round(float y) {
    return __nv_cvt_float_to_fp8(y, __NV_SATFINITE, __NV_E4M3);
  }
  __device__ __forceinline__ static float value(uint32_t c) {
    const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(c), __NV_E4M3);
    return __half2float(__half(h));
  }
};
template <typename C>
__device__ __forceinline__ uint32_t quantize(float x, float s) {
  const float y = __fdiv_rn(x, s);
  return s > 0.f && y == y ? C::round(y) : 0u;
}

// ---- attention: what its two kernels share ---------------------------------------------------

struct PagedAttnArgs {
  const void* q;
  long long q_stride;
  const int* cu_q;
  const int* kv_len;
  const int* table;
  int table_stride, requests, tokens, n_heads, max_q;
  float scale;
  void* out;
  long long out_stride;
  uint64_t wait_ns;  // the longest wait for another role of a CTA
};

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }


constexpr int kMaxRep = 16;  // query heads per KV head
constexpr int kMaxKeys = 1 << 30;

// ---- what both kernels need to know about a request -----------------------------------------
struct Req {
  int q0, nq, len;  // first query row, queries, keys
  bool ok;          // consistent lengths
};
__device__ __forceinline__ Req request(const PagedAttnArgs& a, int block_log2, int r) {
  Req x;
  x.q0 = a.cu_q[r];
  const int q1 = a.cu_q[r + 1];
  x.len = a.kv_len[r];
  x.ok = x.q0 >= 0 && q1 >= x.q0 && q1 <= a.tokens;
  x.nq = x.ok ? q1 - x.q0 : 0;
  if (x.nq > 0)
    x.ok = x.nq <= a.max_q && x.nq <= x.len && x.len <= kMaxKeys &&
           x.len <= (static_cast<long long>(a.table_stride) << block_log2);
  return x;
}

__device__ __forceinline__ float exp2_approx(float x) {  // 2^x (2^-inf = 0), relative error about 2^-22
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kLog2e = 1.4426950408889634f;

// Codes to fp16, exactly.  int8: with its sign bit flipped a code is u = c + 128,
// and the fp16 number with the bits 0x6400 | u is 1024 + u, so one subtraction of
// 1152 gives c.  (Left out, with 1152 times a query row's sum taken off its scores instead, it made their fp32
// accumulators nine times as large as a full-scale score, and was no faster.)  E4M3 values are fp16 values.
template <typename C>
struct Widen;
template <>
struct Widen<CodeI8> {
  // the word's codes as the bytes that pair() takes
  __device__ __forceinline__ static uint32_t prep(uint32_t w) { return w ^ 0x80808080u; }
  // bytes 0 and 1 (HI: 2 and 3) of a prepared word
  template <bool HI>
  __device__ __forceinline__ static uint32_t pair(uint32_t w) {
    const uint32_t m = __byte_perm(w, 0x64646464u, HI ? 0x4342 : 0x4140);
    const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&m), __half2half2(__ushort_as_half(0x6480)));
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};
template <>
struct Widen<CodeF8> {
  __device__ __forceinline__ static uint32_t prep(uint32_t w) { return w; }
  template <bool HI>
  __device__ __forceinline__ static uint32_t pair(uint32_t w) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(HI ? w >> 16 : w & 0xFFFFu), __NV_E4M3);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};

__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void* src, bool take) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(take ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async16_to(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// Eight neighbouring query elements as fp32
template <typename T>
__device__ __forceinline__ void load8(const T* p, float* f) {
  const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
  Unpack<T>::run(v, f);
}
// four outputs
template <typename T>
__device__ __forceinline__ void store4(T* p, float a, float b, float c, float d) {
  T v[4] = {from_f32<T>(a), from_f32<T>(b), from_f32<T>(c), from_f32<T>(d)};
  *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(v);
}

// a / b for a >= 0, b > 0: a division of 32 bits where that holds both
__device__ __forceinline__ long long quotient(long long a, long long b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}
// Equal shares of `total` units of work for n CTAs, the first `more` of them one longer: the first unit of CTA c, and
// the CTA of unit x.
struct Share {
  long long each;
  int more;
  __device__ __forceinline__ Share(long long total, int n) {
    each = quotient(total, n);
    more = static_cast<int>(total - each * n);
  }
  __device__ __forceinline__ long long first(int c) const { return each * c + min(c, more); }
  __device__ __forceinline__ int cta_of(long long x) const {
    const long long longer = (each + 1) * more;
    return static_cast<int>(x < longer ? quotient(x, each + 1) : more + quotient(x - longer, each));
  }
};

constexpr int kAttnMaxCtas = 1024;

// opts a kernel in to its shared memory, once per device (bit `dev` of `ready`)
inline cudaError_t allow_smem(const void* kernel, int bytes, int dev, std::atomic<uint64_t>& ready) {
  const uint64_t bit = 1ull << dev;
  if (ready.load(std::memory_order_acquire) & bit) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) ready.fetch_or(bit, std::memory_order_release);
  return e;
}

// Prompt chunks (k2_paged_chunk.cu): the requests with more than small_rows query rows.
//
// The kernels of a call let their successor start before they have waited themselves (elsewhere a kernel does so only after
// its own wait, so that whatever starts finds all but its predecessor completed).  The same holds here at the call's end:
// the kernel for few rows is launched in plain stream order, the one for chunks and the one that joins its parts are its
// dependents and wait for their predecessor before every exit, and the last lets nobody start early.  Between the kernel for
// few rows and the one for chunks there is nothing to wait for: they share no output and no part of the workspace.  A plan's
// two launches follow the same pattern.
size_t paged_chunk_part_bytes();  // of one CTA's two parts
cudaError_t launch_paged_chunk(const PagedPool& p, const PagedAttnArgs& a, int head_dim, int kv_dtype, int q_dtype,
                               int small_rows, float* parts, int sms, int dev, cudaStream_t s);

}  // namespace k2
