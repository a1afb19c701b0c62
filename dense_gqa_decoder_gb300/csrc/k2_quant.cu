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

int row_type_bytes(int dtype) { return dtype == K2_F32 ? 4 : dtype == K2_BF16 || dtype == K2_F16 ? 2 : 0; }

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
// the largest of |m|, |a| and |b|; a NaN wins
__device__ __forceinline__ float max_magnitude(float m, float a, float b) {
  asm("max.NaN.abs.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(a), "f"(b));
  return m;
}
// pairs of fp32 numbers, each product and sum rounded as by itself
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float2 two(f32x2 v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}

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

// ---- rows of whole 8-value vectors at aligned places ------------------------------------------------------------------
//
// A CTA per row, V vectors of 8 values per thread in registers.  The norm's groups hold whole vectors and are at most kGroups,
// so that a thread adds its squares into one of as many sums.
constexpr int kGroups = 4;

// 8 values as they are held until their row's maximum is known: fp32, or the 16-bit values themselves
template <typename T>
struct Held {
  uint4 bits = {0, 0, 0, 0};
  __device__ __forceinline__ void load(const T* p) { bits = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void values(f32x2 (&f)[4]) const {
    float v[8];
    Unpack<T>::run(bits, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = pk2(v[2 * i], v[2 * i + 1]);
  }
  // the largest magnitude so far: as pairs of 15-bit numbers, among which a NaN's is larger than all others
  using Top = uint32_t;
  __device__ __forceinline__ void raise(Top& top) const {
    const uint32_t w[4] = {bits.x, bits.y, bits.z, bits.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) top = __vmaxu2(top, w[i] & 0x7FFF7FFFu);
  }
  __device__ __forceinline__ static float top(Top t) {
    const uint32_t m = max(t >> 16, t & 0xFFFFu);
    if (std::is_same<T, __nv_bfloat16>::value) return __uint_as_float(m << 16);
    return __half2float(__ushort_as_half(static_cast<unsigned short>(m)));
  }
};
template <>
struct Held<float> {
  ulonglong2 bits[2] = {{0, 0}, {0, 0}};
  __device__ __forceinline__ void load(const float* p) {
    bits[0] = reinterpret_cast<const ulonglong2*>(p)[0];
    bits[1] = reinterpret_cast<const ulonglong2*>(p)[1];
  }
  __device__ __forceinline__ void values(f32x2 (&f)[4]) const { f[0] = bits[0].x, f[1] = bits[0].y, f[2] = bits[1].x, f[3] = bits[1].y; }
  using Top = float;
  __device__ __forceinline__ void raise(Top& top) const {
    f32x2 f[4];
    values(f);
#pragma unroll
    for (int i = 0; i < 4; ++i) top = max_magnitude(top, two(f[i]).x, two(f[i]).y);
  }
  __device__ __forceinline__ static float top(Top t) { return t; }
};
__device__ __forceinline__ void store8(float* p, const f32x2 (&f)[4]) {
  reinterpret_cast<ulonglong2*>(p)[0] = make_ulonglong2(f[0], f[1]);
  reinterpret_cast<ulonglong2*>(p)[1] = make_ulonglong2(f[2], f[3]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const f32x2 (&f)[4]) {
  uint4 v;
  __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&v);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(two(f[i]).x, two(f[i]).y);
  *reinterpret_cast<uint4*>(p) = v;
}
__device__ __forceinline__ void store8(__half* p, const f32x2 (&f)[4]) {
  uint4 v;
  __half2* h = reinterpret_cast<__half2*>(&v);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2half2_rn(two(f[i]).x, two(f[i]).y);
  *reinterpret_cast<uint4*>(p) = v;
}
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3) |
         static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3)) << 16;
}
// A row's scale, and the codes of its values.  The quotients y / s are correctly rounded without a division each: with r the
// rounded reciprocal of s, a quotient q that is close is improved by q + (y - q s) r, whose remainder is exact; from within one
// step of the quotient this gives the rounded quotient itself (P. Markstein, Computation of elementary functions on the IBM RISC
// System/6000 processor, IBM J. Res. Dev. 34, 1990), and one improvement of y r leads there.  s is far enough from the ends of
// fp32 (`plain`) that no remainder of a quotient above 2^-11 is lost; what lies below gets the code 0 anyhow.  All with the
// quotients' signs turned, which keeps the sign of a zero, and turned back in the codes.  (With a division
// per value 8192 x 10240 took 59.5 us.  Two products that bound the quotient, and a division where they give two codes: 49 us,
// because quotients of bf16 rows lie half way between two codes so often that every third row needed divisions.)
struct RowScale {
  float s;
  f32x2 s2, minus_r2;
  bool fine, plain;  // all values finite; the codes can be had so
  __device__ __forceinline__ explicit RowScale(unsigned top) {
    fine = top < 0x7F800000u;
    s = fine ? __uint_as_float(top) / kTop : __uint_as_float(0x7FC00000u);
    const float r = __frcp_rn(s);
    s2 = pk2(s, s);
    minus_r2 = pk2(-r, -r);
    plain = s >= 0x1p-80f && s <= 0x1p110f;  // (not where it is NaN)
  }
  __device__ __forceinline__ f32x2 minus_quotients(f32x2 y) const {
    f32x2 q = mul2(y, minus_r2);
    q = fma2(fma2(q, s2, y), minus_r2, q);
    return fma2(fma2(q, s2, y), minus_r2, q);
  }
  __device__ __forceinline__ uint2 codes(const f32x2 (&y)[4]) const {
    const float2 a = two(minus_quotients(y[0])), b = two(minus_quotients(y[1])), c = two(minus_quotients(y[2])),
                 d = two(minus_quotients(y[3]));
    return make_uint2(codes4(a.x, a.y, b.x, b.y) ^ 0x80808080u, codes4(c.x, c.y, d.x, d.y) ^ 0x80808080u);
  }
  __device__ __noinline__ static uint2 divided(const float4 a, const float4 b, float s, bool fine) {
    if (!fine) return make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
    if (s == 0.f) return make_uint2(0u, 0u);
    return make_uint2(codes4(__fdiv_rn(a.x, s), __fdiv_rn(a.y, s), __fdiv_rn(a.z, s), __fdiv_rn(a.w, s)),
                      codes4(__fdiv_rn(b.x, s), __fdiv_rn(b.y, s), __fdiv_rn(b.z, s), __fdiv_rn(b.w, s)));
  }
  __device__ __forceinline__ uint2 divided(const f32x2 (&y)[4]) const {
    const float2 a = two(y[0]), b = two(y[1]), c = two(y[2]), d = two(y[3]);
    return divided(make_float4(a.x, a.y, b.x, b.y), make_float4(c.x, c.y, d.x, d.y), s, fine);
  }
};

constexpr int kRowThreads = 320, kVectorThreads = 512, kWideThreads = 1024;

// what the warps of a CTA tell each other
struct RowShared {
  float sums[32][kGroups];
  unsigned tops[32];
};

// One row, spread over the CTA: thread i holds vectors i, i + threads, ...
template <typename XT, typename RT, bool NORM, int V>
struct Row {
  static constexpr bool kAdds = !std::is_same<RT, None>::value;
  using Added = typename std::conditional<kAdds, RT, float>::type;
  Held<XT> x[V];
  Held<Added> r[kAdds ? V : 1];

  __device__ __forceinline__ void load(const XT* from, const Added* added, int n8) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v < n8) x[i].load(from + 8 * v);
    }
    if constexpr (kAdds) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        if (v < n8) r[i].load(added + 8 * v);
      }
    }
  }

  // the largest of the CTA's values, as a magnitude, in every thread
  __device__ __forceinline__ static unsigned top_of(float top, unsigned* tops) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const unsigned m = __reduce_max_sync(0xffffffffu, magnitude(top));
    if (lane == 0) tops[warp] = m;
    __syncthreads();
    return __reduce_max_sync(0xffffffffu, lane < warps ? tops[lane] : 0u);
  }
  // the codes of row t, whose vector i is value(i, .), and its scale; again(.) stores them by divisions
  template <typename F, typename G>
  __device__ __forceinline__ static void store_codes(const RowArgs& a, long long t, int n8, const RowScale& scale, F value, G again) {
    uint2* codes = reinterpret_cast<uint2*>(a.codes + a.codes_stride * t);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      f32x2 f[4];
      value(i, f);
      const uint2 w = scale.codes(f);
      if (v < n8) codes[v] = w;
    }
    if (!scale.plain) again(codes);
    if (threadIdx.x == 0) a.scales[t] = scale.s;
  }

  // what is stored of row t
  __device__ __forceinline__ void finish(const RowArgs& a, long long t, RowShared& sh) {
    const int n8 = a.cols >> 3;
    if constexpr (NORM) {
      normalise(a, t, n8, sh);
    } else {
      typename Held<XT>::Top top = 0;
#pragma unroll
      for (int i = 0; i < V; ++i) x[i].raise(top);
      const RowScale scale(top_of(Held<XT>::top(top), sh.tops));
      store_codes(a, t, n8, scale, [&](int i, f32x2 (&f)[4]) { x[i].values(f); },
                  [&](uint2* codes) {  // read again: the values need not stay in registers
                    const XT* from = static_cast<const XT*>(a.x) + a.x_stride * t;
#pragma unroll 1
                    for (int v = threadIdx.x; v < n8; v += blockDim.x) {
                      Held<XT> h;
                      f32x2 f[4];
                      h.load(from + 8 * v);
                      h.values(f);
                      codes[v] = scale.divided(f);
                    }
                  });
    }
  }

  __device__ __forceinline__ void normalise(const RowArgs& a, long long t, int n8, RowShared& sh) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5, size8 = n8 / a.groups;
    int group[V];
    f32x2 h[V][4];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      group[i] = v < size8 ? 0 : v < 2 * size8 ? 1 : v < 3 * size8 ? 2 : 3;  // (what lies behind the row is 0)
      x[i].values(h[i]);
      if constexpr (kAdds) {
        f32x2 f[4];
        r[i].values(f);
#pragma unroll
        for (int j = 0; j < 4; ++j) h[i][j] = add2(h[i][j], f[j]);
        if (v < n8) store8(static_cast<RT*>(a.res_out) + a.res_out_stride * t + 8 * v, h[i]);
      }
    }
    // the sum of each group's squares over the CTA, lanes g, g + 4, ... of every warp taking the last steps of group g; `unit`:
    // what the values are multiplied with first
    const float count = static_cast<float>(8 * size8);
    auto mean_of_lane = [&](float unit) {
      float ss[kGroups] = {};
#pragma unroll
      for (int i = 0; i < V; ++i) {
        f32x2 sq2 = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const f32x2 e = unit == 1.f ? h[i][j] : mul2(h[i][j], pk2(unit, unit));
          sq2 = fma2(e, e, sq2);
        }
        const float sq = sum2(sq2);
#pragma unroll
        for (int g = 0; g < kGroups; ++g) ss[g] += group[i] == g ? sq : 0.f;
      }
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        if (g >= a.groups) break;
        const float w = warp_sum(ss[g]);
        if (lane == 0) sh.sums[warp][g] = w;
      }
      __syncthreads();
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < kWideThreads / 32; w += 8) {
        if (w >= warps) break;
        if (w + (lane >> 2) < warps) sum += sh.sums[w + (lane >> 2)][lane & 3];
      }
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      return sum / count + a.eps * unit * unit;
    };
    float mean = mean_of_lane(1.f);
    // a finite row's squares overflow (or a value is not finite): those groups in other units
    const bool over = (lane & 3) < a.groups && !(mean <= 3.4028235e38f);
    const unsigned overs = __ballot_sync(0xffffffffu, over);
    if (overs != 0) {
      __syncthreads();  // the sums have been read
      const float again = mean_of_lane(kUnit);
      if (over) mean = again;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if ((overs >> group[i] & 1u) != 0)
#pragma unroll
          for (int j = 0; j < 4; ++j) h[i][j] = mul2(h[i][j], pk2(kUnit, kUnit));
    }
    const float mine = __frsqrt_rn(mean);
    float top = 0.f, factor[kGroups];
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      factor[g] = 0.f;
      if (g < a.groups) factor[g] = __shfl_sync(0xffffffffu, mine, g);
    }
    if (a.gain_dtype == K2_F32) apply<float>(a, n8, group, factor, h, top);
    else if (a.gain_dtype == K2_BF16) apply<__nv_bfloat16>(a, n8, group, factor, h, top);
    else apply<__half>(a, n8, group, factor, h, top);
    const RowScale scale(top_of(top, sh.tops));
    store_codes(a, t, n8, scale, [&](int i, f32x2 (&f)[4]) {
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = h[i][j];
    }, [&](uint2* codes) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        if (v < n8) codes[v] = scale.divided(h[i]);
      }
    });
  }

  // the factors of the groups and the gain
  template <typename GT>
  __device__ __forceinline__ static void apply(const RowArgs& a, int n8, const int (&group)[V], const float (&factor)[kGroups],
                                               f32x2 (&h)[V][4], float& top) {
    Held<GT> gain[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v < n8) gain[i].load(static_cast<const GT*>(a.gain) + 8 * v);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float f = factor[0];
#pragma unroll
      for (int g = 1; g < kGroups; ++g) f = group[i] == g ? factor[g] : f;
      f32x2 g8[4];
      gain[i].values(g8);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        h[i][j] = mul2(mul2(h[i][j], pk2(f, f)), g8[j]);
        top = max_magnitude(top, two(h[i][j]).x, two(h[i][j]).y);
      }
    }
  }
};

// A CTA per row.  Many rows, the usual case: up to 320 threads (512 with 4 and more vectors each), so few registers that 1280
// threads (1536) fit an SM and their rows are on their way while others are worked on (without these limits 8192 x 10240 bf16
// values 57.8 us, 40.4 with them; norm of 8192 x 2560 in bf16 30.0 and 27.1, in fp32, where two vectors a thread spill eight bytes
// for it, 41.7 and 42.4).  WIDE: up to 1024 threads.
// (Rows copied ahead into shared memory by CTAs that stay were slower: 8192 x 10240 values 58 us, when this form took 49.)
template <typename XT, typename RT, bool NORM, int V, bool WIDE>
__global__ void __launch_bounds__(WIDE ? kWideThreads : V <= 2 ? kRowThreads : kVectorThreads,
                                  WIDE ? 1 : V <= 2 ? 1280 / kRowThreads : V == 4 && !NORM && sizeof(XT) == 2 ? 1536 / kVectorThreads : 1)
    vector_rows_kernel(const RowArgs a) {
  using R = Row<XT, RT, NORM, V>;
  __shared__ RowShared sh;
  const long long t = blockIdx.x;
  pdl_wait();  // the rows may be the previous kernel's
  pdl_trigger();
  R row;
  row.load(static_cast<const XT*>(a.x) + a.x_stride * t, static_cast<const typename R::Added*>(a.res) + a.res_stride * t, a.cols >> 3);
  row.finish(a, t, sh);
}

bool at8(const void* p, long long stride, int bytes) {  // 8 values of `bytes` (at most 16 bytes at once) can be taken together
  const int step = std::min(16, 8 * bytes);
  return reinterpret_cast<uintptr_t>(p) % step == 0 && stride * bytes % step == 0;
}

// ---- any row ----------------------------------------------------------------------------------------------------------
//
// One CTA, the values as fp32 in shared memory, element by element.
template <typename XT, typename RT, bool NORM>
__global__ void __launch_bounds__(256) rows_kernel(RowArgs a) {
  extern __shared__ float row[];
  __shared__ float part[8];
  __shared__ unsigned mpart[8];
  const int t = blockIdx.x, tid = threadIdx.x, n = a.cols;
  const XT* x = static_cast<const XT*>(a.x) + a.x_stride * t;
  uint8_t* codes = a.codes + a.codes_stride * t;
  unsigned top = 0;
  pdl_wait();
  pdl_trigger();
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
      const float r = __frsqrt_rn(mean);
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

template <typename K, typename... Args>
cudaError_t launch_early(K kernel, int ctas, int threads, size_t smem, cudaStream_t s, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // the start overlaps the end of the kernel before it
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename XT, typename RT, bool NORM>
cudaError_t launch_rows(const RowArgs& a, int tokens, cudaStream_t s) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && (dev < 0 || dev >= 64)) e = cudaErrorInvalidDevice;
  if (e != cudaSuccess) return e;
  constexpr int rb = std::is_same<RT, None>::value ? 4 : sizeof(RT);
  const int n8 = a.cols / 8;
  const bool whole = a.cols % 8 == 0 && n8 <= (NORM ? 4 : 8) * kVectorThreads && at8(a.x, a.x_stride, sizeof(XT)) && at8(a.codes, a.codes_stride, 1) &&
                     at8(a.res, a.res_stride, rb) && at8(a.res_out, a.res_out_stride, rb);
  if (whole && (!NORM || (a.groups <= kGroups && n8 % a.groups == 0 && at8(a.gain, 0, row_type_bytes(a.gain_dtype))))) {
    // Few rows, fewer than SMs: many threads, few vectors each (norm of 64 x 2560 2.6 us with 320 threads, 2.8 with 160; of 16 x 10240
    // 4.5 with 640 and 4.2 with 320; conversions the same either way); many: fewer threads, so that more rows are on their way at
    // once (8192 x 10240 values 40.4 us, wide 57.1; norm of 8192 x 2560 in bf16 27.1 and 36.2, in fp32 42.4 and 45.0).
    constexpr std::integral_constant<int, 1> one;
    constexpr std::integral_constant<int, 2> both;
    constexpr std::integral_constant<int, 4> four;
    constexpr std::integral_constant<int, 8> eight;
    auto threads = [&](int v) { return ((n8 + v - 1) / v + 31) / 32 * 32; };
    int sms = 0;
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    constexpr std::integral_constant<bool, true> wide;
    constexpr std::integral_constant<bool, false> narrow;
    auto go = [&](auto v, auto w) {
      return launch_early(vector_rows_kernel<XT, RT, NORM, decltype(v)::value, decltype(w)::value>, tokens, threads(v), 0, s, a);
    };
    if (tokens <= sms && n8 <= 640) return go(one, wide);
    if (tokens <= sms && n8 <= 2 * kWideThreads) return go(both, wide);
    if (n8 <= 96) return go(one, narrow);
    if (n8 <= 2 * kRowThreads) return go(both, narrow);
    if (n8 <= 4 * kVectorThreads) return go(four, narrow);
    if constexpr (!NORM) return go(eight, narrow);
  }
  static std::atomic<uint64_t> ready{0};
  auto kernel = rows_kernel<XT, RT, NORM>;
  e = allow_smem(reinterpret_cast<const void*>(kernel), kMaxRowCols * static_cast<int>(sizeof(float)), dev, ready);
  if (e != cudaSuccess) return e;
  return launch_early(kernel, tokens, 256, a.cols * sizeof(float), s, a);
}

template <typename XT>
cudaError_t launch_norm(const RowArgs& a, int res_dtype, int tokens, cudaStream_t s) {
  if (!a.res) return launch_rows<XT, None, true>(a, tokens, s);
  if (res_dtype == K2_F32) return launch_rows<XT, float, true>(a, tokens, s);
  if (res_dtype == K2_BF16) return launch_rows<XT, __nv_bfloat16, true>(a, tokens, s);
  return launch_rows<XT, __half, true>(a, tokens, s);
}

bool off_type(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes != 0; }

// What both calls refuse of their input rows, codes and scales
k2_status check_rows(const k2_row_args* p) {
  if (!p) {
    set_error("the arguments must be non-null");
    return K2_ERR_ARG;
  }
  const int b = row_type_bytes(p->x_dtype);
  if (!b) {
    set_error("rows must be K2_F32, K2_BF16 or K2_F16 (got dtype %d)", p->x_dtype);
    return K2_ERR_UNSUPPORTED;
  }
  if (p->tokens < 0 || p->tokens > 1 << 30 || p->cols < 1 || p->cols > kMaxRowCols) {
    set_error("tokens in [0, 2^30] and rows of 1 .. %d values (got %d, %d)", kMaxRowCols, p->tokens, p->cols);
    return K2_ERR_SHAPE;
  }
  if (p->tokens == 0) return K2_OK;
  if (!p->x || !p->codes || !p->scales) {
    set_error("x, codes and scales must be non-null");
    return K2_ERR_ARG;
  }
  if (off_type(p->x, b) || off_type(p->scales, 4)) {
    set_error("x and scales must be aligned to their types");
    return K2_ERR_ARG;
  }
  const int64_t most = INT64_MAX / 8 / (p->tokens + 1);  // so that no offset overflows
  if (p->tokens > 1 && (p->x_stride < p->cols || p->codes_stride < p->cols || p->x_stride > most || p->codes_stride > most)) {
    set_error("rows must be at least as far apart as they are long (%d; got %lld, codes %lld)", p->cols,
              static_cast<long long>(p->x_stride), static_cast<long long>(p->codes_stride));
    return K2_ERR_ARG;
  }
  const RowSet x = {p->x, b * p->x_stride, static_cast<int64_t>(b) * p->cols, p->tokens},
               codes = {p->codes, p->codes_stride, p->cols, p->tokens}, scales = {p->scales, 4, 4, p->tokens};
  if (sets_meet(x, codes) || sets_meet(x, scales) || sets_meet(codes, scales)) {
    set_error("the codes and scales may not lie over the input or each other");
    return K2_ERR_ARG;
  }
  return K2_OK;
}

// (the distance of the one row of a single token is not read)
RowArgs row_args(const k2_row_args& p) {
  const long long many = p.tokens > 1;
  return {p.x, many * p.x_stride, p.residual, many * p.residual_stride, p.residual_out, many * p.residual_out_stride, p.gain,
          p.gain_dtype, p.cols, p.groups, p.eps, p.codes, many * p.codes_stride, p.scales};
}

}  // namespace

}  // namespace k2

using namespace k2;

extern "C" {

k2_status k2_quantize_rows(const k2_row_args* p, void* stream) {
  const k2_status st = check_rows(p);
  if (st != K2_OK) return st;
  if (p->residual || p->residual_out || p->gain) {
    set_error("residual, residual_out and gain belong to k2_norm_quantize");
    return K2_ERR_ARG;
  }
  if (p->tokens == 0) return K2_OK;
  const RowArgs a = row_args(*p);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = p->x_dtype == K2_F32    ? launch_rows<float, None, false>(a, p->tokens, s)
                        : p->x_dtype == K2_BF16 ? launch_rows<__nv_bfloat16, None, false>(a, p->tokens, s)
                                                : launch_rows<__half, None, false>(a, p->tokens, s);
  if (e == cudaSuccess) return K2_OK;
  set_error("quantize launch: %s", cudaGetErrorString(e));
  return K2_ERR_CUDA;
}

k2_status k2_norm_quantize(const k2_row_args* p, void* stream) {
  const k2_status st = check_rows(p);
  if (st != K2_OK) return st;
  const bool adds = p->residual || p->residual_out;
  const int gb = row_type_bytes(p->gain_dtype), rb = adds ? row_type_bytes(p->residual_dtype) : 4;
  if (!gb || !rb) {
    set_error("gain and residual must be K2_F32, K2_BF16 or K2_F16 (got dtypes %d, %d)", p->gain_dtype, p->residual_dtype);
    return K2_ERR_UNSUPPORTED;
  }
  if (p->groups < 1 || p->cols % p->groups) {
    set_error("cols %d must be a multiple of groups (got %d)", p->cols, p->groups);
    return K2_ERR_SHAPE;
  }
  if (!(p->eps >= kMinEps) || isinf(p->eps)) {
    set_error("eps must be finite and at least 2^-126 (got %g)", p->eps);
    return K2_ERR_ARG;
  }
  if (p->tokens == 0) return K2_OK;
  if (!p->gain || !p->residual != !p->residual_out) {
    set_error("gain must be non-null, residual and residual_out both given or both NULL");
    return K2_ERR_ARG;
  }
  if (off_type(p->gain, gb) || off_type(p->residual, rb) || off_type(p->residual_out, rb)) {
    set_error("gain and residual must be aligned to their types");
    return K2_ERR_ARG;
  }
  const int64_t most = INT64_MAX / 8 / (p->tokens + 1), rs = p->residual_stride, os = p->residual_out_stride;
  if (adds && p->tokens > 1 && (rs < p->cols || os < p->cols || rs > most || os > most)) {
    set_error("residual rows must be at least cols = %d elements apart (got %lld, %lld)", p->cols, static_cast<long long>(rs),
              static_cast<long long>(os));
    return K2_ERR_ARG;
  }
  const int64_t xb = row_type_bytes(p->x_dtype), n = p->cols, t = p->tokens;
  const RowSet x = {p->x, xb * p->x_stride, xb * n, t}, codes = {p->codes, p->codes_stride, n, t}, scales = {p->scales, 4, 4, t},
               gain = {p->gain, 0, gb * n, 1}, res = {p->residual, rb * rs, rb * n, t}, out = {p->residual_out, rb * os, rb * n, t};
  const bool same = p->residual == p->residual_out && (t == 1 || rs == os);
  if ((!same && sets_meet(res, out)) || sets_meet(out, x) || sets_meet(out, codes) || sets_meet(out, scales) ||
      sets_meet(out, gain) || sets_meet(codes, res) || sets_meet(codes, gain) || sets_meet(scales, res) ||
      sets_meet(scales, gain)) {
    set_error("outputs may not lie over inputs or each other (residual_out may be residual, with its stride)");
    return K2_ERR_ARG;
  }
  const RowArgs a = row_args(*p);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = p->x_dtype == K2_F32    ? launch_norm<float>(a, p->residual_dtype, p->tokens, s)
                        : p->x_dtype == K2_BF16 ? launch_norm<__nv_bfloat16>(a, p->residual_dtype, p->tokens, s)
                                                : launch_norm<__half>(a, p->residual_dtype, p->tokens, s);
  if (e == cudaSuccess) return K2_OK;
  set_error("norm launch: %s", cudaGetErrorString(e));
  return K2_ERR_CUDA;
}

}  // extern "C"
