// Rows as E4M3 codes with one scale per row: plain (k2_quantize_rows), or of the normalised sum of a layer's output and
// the residual stream (k2_norm_quantize).
//
//   h = x + residual;  y = h * rsqrt(mean_g(h^2) + eps) * gain  (or y = x)
//   s = max|y| / 448;  code = E4M3(y / s)
//
// Every row is read once and held (in registers, or as fp32 in shared memory) until its sums and its maximum are known, so
// the bytes bound a large call: 8192 rows of 10240 bf16 values are 252 MB, 37 us at the copy rate.  A small call is bounded
// by its chain: load, sum, maximum, codes.
#include <math.h>

#include <algorithm>

#include "k2_common.cuh"
#include "k2_linear.h"
#include "k2_paged.cuh"

namespace k2 {

namespace {

constexpr int kMaxCols = 49152;   // a row in shared memory as fp32: 192 KB
constexpr float kTop = 448.0f;    // the largest finite E4M3 value
constexpr uint8_t kCodeNaN = 0x7F;

struct RowArgs {
  const void* x;
  long long x_stride;
  const void* res;
  long long res_stride;
  void* res_out;
  long long res_out_stride;
  const void* gain;
  int gain_dtype;
  int cols, groups;
  float eps;
  uint8_t* codes;
  long long codes_stride;
  float* scales;
};

struct None {};

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

__device__ __forceinline__ float load_gain(const void* g, int dtype, int i) {
  if (dtype == K2_F32) return __ldg(static_cast<const float*>(g) + i);
  if (dtype == K2_BF16) return __bfloat162float(__ldg(static_cast<const __nv_bfloat16*>(g) + i));
  return __half2float(__ldg(static_cast<const __half*>(g) + i));
}

// |v| as a number that grows with it and is largest for a NaN
__device__ __forceinline__ unsigned magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

__device__ __forceinline__ uint32_t code_of(float y, float s) {
  return __nv_cvt_float_to_fp8(__fdiv_rn(y, s), __NV_SATFINITE, __NV_E4M3);
}

// A block's sum and maximum: every thread gets the same value (`part`: a word per warp)
__device__ __forceinline__ float block_sum(float v, float* part) {
  v = warp_sum(v);
  __syncthreads();  // the last reduction's words have been read
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  float sum = 0.f;
  for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) sum += part[w];
  return sum;
}
__device__ __forceinline__ unsigned block_max(unsigned v, unsigned* part) {
  v = __reduce_max_sync(0xffffffffu, v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  unsigned m = 0;
  for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) m = max(m, part[w]);
  return m;
}

// A finite row whose squares overflow is summed in units of 2^80, where 49152 of the largest squares stay below 2^112.
constexpr float kUnit = 0x1p-80f;

// Any row: one CTA, the values as fp32 in shared memory, element by element.
template <typename XT, typename RT, bool NORM>
__global__ void __launch_bounds__(256) rows_kernel(RowArgs a) {
  extern __shared__ float row[];
  __shared__ float part[8];
  __shared__ unsigned mpart[8];
  const int t = blockIdx.x, tid = threadIdx.x, n = a.cols;
  const XT* x = static_cast<const XT*>(a.x) + a.x_stride * t;
  uint8_t* codes = a.codes + a.codes_stride * t;
  unsigned top = 0;
  for (int i = tid; i < n; i += 256) {
    float h = to_f32(x[i]);
    if constexpr (!std::is_same<RT, None>::value) {
      h += to_f32(static_cast<const RT*>(a.res)[a.res_stride * t + i]);
      static_cast<RT*>(a.res_out)[a.res_out_stride * t + i] = from_f32<RT>(h);
    }
    row[i] = h;
    if (!NORM) top = max(top, magnitude(h));
  }
  if constexpr (NORM) {
    const int size = n / a.groups;
    __syncthreads();
    for (int g = 0; g < a.groups; ++g) {
      float* part_of = row + g * size;
      float ss = 0.f, unit = 1.f;
      for (int i = tid; i < size; i += 256) ss += part_of[i] * part_of[i];
      float mean = block_sum(ss, part) / static_cast<float>(size) + a.eps;
      if (!(mean <= 3.4028235e38f)) {
        unit = kUnit;
        ss = 0.f;
        for (int i = tid; i < size; i += 256) ss += (part_of[i] * unit) * (part_of[i] * unit);
        mean = block_sum(ss, part) / static_cast<float>(size) + a.eps * unit * unit;
      }
      const float r = 1.0f / sqrtf(mean);
      for (int i = tid; i < size; i += 256) {
        const float y = part_of[i] * unit * r * load_gain(a.gain, a.gain_dtype, g * size + i);
        part_of[i] = y;
        top = max(top, magnitude(y));
      }
    }
  }
  top = block_max(top, mpart);
  const bool fine = top < 0x7F800000u;
  const float s = fine ? __uint_as_float(top) / kTop : __uint_as_float(0x7FC00000u);
  for (int i = tid; i < n; i += 256)
    codes[i] = fine ? (s > 0.f ? static_cast<uint8_t>(code_of(row[i], s)) : static_cast<uint8_t>(0)) : kCodeNaN;
  if (tid == 0) a.scales[t] = s;
}

template <typename XT, typename RT, bool NORM>
cudaError_t launch_rows(const RowArgs& a, int tokens, cudaStream_t s) {
  auto kernel = rows_kernel<XT, RT, NORM>;
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = allow_smem(reinterpret_cast<const void*>(kernel), kMaxCols * static_cast<int>(sizeof(float)), dev, ready);
  if (e != cudaSuccess) return e;
  kernel<<<tokens, 256, a.cols * sizeof(float), s>>>(a);
  return cudaGetLastError();
}

template <typename XT>
cudaError_t launch_norm(const RowArgs& a, int res_dtype, int tokens, cudaStream_t s) {
  if (!a.res) return launch_rows<XT, None, true>(a, tokens, s);
  if (res_dtype == K2_F32) return launch_rows<XT, float, true>(a, tokens, s);
  if (res_dtype == K2_BF16) return launch_rows<XT, __nv_bfloat16, true>(a, tokens, s);
  return launch_rows<XT, __half, true>(a, tokens, s);
}

int row_type_bytes(int dtype) { return dtype == K2_F32 ? 4 : dtype == K2_BF16 || dtype == K2_F16 ? 2 : 0; }
bool off_type(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes != 0; }

// What both calls refuse of their input rows, codes and scales
k2_status check_rows(const char* what, const void* d_x, int dtype, int64_t x_stride, int tokens, int cols,
                     const uint8_t* d_codes, int64_t codes_stride, const float* d_scales) {
  const int b = row_type_bytes(dtype);
  if (!b) {
    set_error("%s must be K2_F32, K2_BF16 or K2_F16 (got dtype %d)", what, dtype);
    return K2_ERR_UNSUPPORTED;
  }
  if (tokens < 0 || tokens > 1 << 30 || cols < 1 || cols > kMaxCols) {
    set_error("tokens in [0, 2^30] and rows of 1 .. %d values (got %d, %d)", kMaxCols, tokens, cols);
    return K2_ERR_SHAPE;
  }
  if (tokens == 0) return K2_OK;
  if (!d_x || !d_codes || !d_scales) {
    set_error("the input rows, d_codes and d_scales must be non-null");
    return K2_ERR_ARG;
  }
  if (off_type(d_x, b) || off_type(d_scales, 4)) {
    set_error("%s and d_scales must be aligned to their types", what);
    return K2_ERR_ARG;
  }
  const int64_t most = INT64_MAX / 8 / (tokens + 1);  // so that no offset overflows
  if (tokens > 1 && (x_stride < cols || codes_stride < cols || x_stride > most || codes_stride > most)) {
    set_error("rows must be at least as far apart as they are long (%d; got %lld, codes %lld)", cols,
              static_cast<long long>(x_stride), static_cast<long long>(codes_stride));
    return K2_ERR_ARG;
  }
  const RowSet x = {d_x, b * x_stride, static_cast<int64_t>(b) * cols, tokens}, codes = {d_codes, codes_stride, cols, tokens},
               scales = {d_scales, 4, 4, tokens};
  if (sets_meet(x, codes) || sets_meet(x, scales) || sets_meet(codes, scales)) {
    set_error("the codes and scales may not lie over the input or each other");
    return K2_ERR_ARG;
  }
  return K2_OK;
}

}  // namespace

}  // namespace k2

using namespace k2;

extern "C" {

k2_status k2_quantize_rows(const void* d_x, int32_t dtype, int64_t x_stride, int32_t tokens, int32_t cols,
                           uint8_t* d_codes, int64_t codes_stride, float* d_scales, void* stream) {
  const k2_status st = check_rows("d_x", d_x, dtype, x_stride, tokens, cols, d_codes, codes_stride, d_scales);
  if (st != K2_OK || tokens == 0) return st;
  RowArgs a = {};
  a.x = d_x;
  a.x_stride = tokens > 1 ? x_stride : 0;
  a.cols = cols;
  a.groups = 1;
  a.codes = d_codes;
  a.codes_stride = tokens > 1 ? codes_stride : 0;
  a.scales = d_scales;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == K2_F32    ? launch_rows<float, None, false>(a, tokens, s)
                        : dtype == K2_BF16 ? launch_rows<__nv_bfloat16, None, false>(a, tokens, s)
                                           : launch_rows<__half, None, false>(a, tokens, s);
  if (e == cudaSuccess) return K2_OK;
  set_error("quantize launch: %s", cudaGetErrorString(e));
  return K2_ERR_CUDA;
}

k2_status k2_norm_quantize(const void* d_x, int32_t x_dtype, int64_t x_stride, const void* d_residual,
                           int64_t residual_stride, void* d_residual_out, int64_t residual_out_stride,
                           int32_t residual_dtype, const void* d_gain, int32_t gain_dtype, int32_t tokens,
                           int32_t hidden, int32_t groups, float eps, uint8_t* d_codes, int64_t codes_stride,
                           float* d_scales, void* stream) {
  const k2_status st = check_rows("d_x", d_x, x_dtype, x_stride, tokens, hidden, d_codes, codes_stride, d_scales);
  if (st != K2_OK) return st;
  const int gb = row_type_bytes(gain_dtype), rb = d_residual || d_residual_out ? row_type_bytes(residual_dtype) : 4;
  if (!gb || !rb) {
    set_error("gain and residual must be K2_F32, K2_BF16 or K2_F16 (got dtypes %d, %d)", gain_dtype, residual_dtype);
    return K2_ERR_UNSUPPORTED;
  }
  if (groups < 1 || hidden % groups) {
    set_error("hidden %d must be a multiple of groups (got %d)", hidden, groups);
    return K2_ERR_SHAPE;
  }
  if (!(eps >= 0x1p-126f) || isinf(eps)) {
    set_error("eps must be finite and at least 2^-126 (got %g)", eps);
    return K2_ERR_ARG;
  }
  if (tokens == 0) return K2_OK;
  if (!d_gain || !d_residual != !d_residual_out) {
    set_error("d_gain must be non-null, d_residual and d_residual_out both given or both NULL");
    return K2_ERR_ARG;
  }
  if (off_type(d_gain, gb) || off_type(d_residual, rb) || off_type(d_residual_out, rb)) {
    set_error("gain and residual must be aligned to their types");
    return K2_ERR_ARG;
  }
  const int64_t most = INT64_MAX / 8 / (tokens + 1);
  if (d_residual && tokens > 1 &&
      (residual_stride < hidden || residual_out_stride < hidden || residual_stride > most || residual_out_stride > most)) {
    set_error("residual rows must be at least hidden = %d elements apart (got %lld, %lld)", hidden,
              static_cast<long long>(residual_stride), static_cast<long long>(residual_out_stride));
    return K2_ERR_ARG;
  }
  const int64_t xb = row_type_bytes(x_dtype);
  const RowSet x = {d_x, xb * x_stride, xb * hidden, tokens}, codes = {d_codes, codes_stride, hidden, tokens},
               scales = {d_scales, 4, 4, tokens}, gain = {d_gain, 0, static_cast<int64_t>(gb) * hidden, 1},
               res = {d_residual, rb * residual_stride, static_cast<int64_t>(rb) * hidden, tokens},
               out = {d_residual_out, rb * residual_out_stride, static_cast<int64_t>(rb) * hidden, tokens};
  const bool same = d_residual == d_residual_out && (tokens == 1 || residual_stride == residual_out_stride);
  if ((!same && sets_meet(res, out)) || sets_meet(out, x) || sets_meet(out, codes) || sets_meet(out, scales) ||
      sets_meet(out, gain) || sets_meet(codes, res) || sets_meet(codes, gain) || sets_meet(scales, res) ||
      sets_meet(scales, gain)) {
    set_error("outputs may not lie over inputs or each other (d_residual_out may be d_residual, with its stride)");
    return K2_ERR_ARG;
  }
  RowArgs a = {d_x, tokens > 1 ? x_stride : 0, d_residual, tokens > 1 ? residual_stride : 0, d_residual_out,
               tokens > 1 ? residual_out_stride : 0, d_gain, gain_dtype, hidden, groups, eps, d_codes,
               tokens > 1 ? codes_stride : 0, d_scales};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = x_dtype == K2_F32    ? launch_norm<float>(a, residual_dtype, tokens, s)
                        : x_dtype == K2_BF16 ? launch_norm<__nv_bfloat16>(a, residual_dtype, tokens, s)
                                             : launch_norm<__half>(a, residual_dtype, tokens, s);
  if (e == cudaSuccess) return K2_OK;
  set_error("norm launch: %s", cudaGetErrorString(e));
  return K2_ERR_CUDA;
}

}  // extern "C"
