// What the operators over a block-paged 8-bit cache share: their checks of the
// pool's descriptor, the two code formats, and the arguments of the kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/k2.h"
#include "k2_common.cuh"
#include "k2_kernels.h"

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

}  // namespace k2
