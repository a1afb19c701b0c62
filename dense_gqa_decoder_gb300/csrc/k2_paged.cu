// The host-side bookkeeping of a block-paged cache, on the GPU: the tables of
// the next step (k2_paged_plan) and the quantizing append (k2_paged_append).
// What they compute is stated in include/k2.h.
#include <algorithm>
#include <type_traits>

#include "k2_paged.cuh"

namespace k2 {

namespace {

// ---- tables, slots and positions from request lengths -----------------------------------------
//
// A step's plan is three prefix sums over the requests (new tokens, blocks
// taken, blocks given back), after which every token, new block and returned
// block finds its request by binary search and its block by arithmetic on the
// state before the step: the x-th entry of the free stack with the returned
// blocks on top is d_free[x] below the old count F, else the (x - F)-th
// returned block.  What the kernel writes (table entries of new blocks, stack
// entries at or above F) is nothing that it reads, and the words that it may
// write over its own inputs (count, lengths) are written once all have read them.
//
// Bound by latency, not by bytes.  One CTA does a decode step in one launch (64 requests: 4.9 us); the tokens of a large
// step are spread over a CTA per 1024, each of which sums the lengths up for itself, and a second launch, which has
// done the same meanwhile, writes what may lie over the inputs (1024 requests and 34000 tokens: 7.5 us, 13.0 in one
// launch of a cluster of eight CTAs, whose instructions took the time).
constexpr int kPlanThreads = 1024, kPlanPer = K2_PAGED_MAX_REQUESTS / kPlanThreads;
constexpr int kPlanCtas = 256;  // of a large step, at most
constexpr int kPlanCap = 1 << 30;  // sums saturate here: min(a + b, cap) is associative for a, b >= 0
static_assert(kPlanPer * kPlanThreads == K2_PAGED_MAX_REQUESTS, "whole requests per thread");

struct PlanArgs {
  const int* cached;
  const int* fresh;
  int requests, block_log2;
  int* table;
  int table_stride;
  int* free_ids;
  int free_capacity;
  const int* free_count;
  int* free_count_out;
  int* kv_len;
  int* cu_new;
  int* slots;
  int* positions;
  int max_tokens;
  int* status;
};

// (two saturated sums make 2^31: added as unsigned numbers)
__device__ __forceinline__ int sat_add(int a, int b) {
  return static_cast<int>(min(static_cast<unsigned>(a) + static_cast<unsigned>(b), static_cast<unsigned>(kPlanCap)));
}

// what a launch does: map the tokens and blocks, write the lengths, or both
enum { kPlanMap = 1, kPlanFinish = 2 };

// the r in [0, n) with sum[r] <= x < sum[r + 1]
__device__ __forceinline__ int find_request(const int* sum, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sum[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

template <int PART>
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanArgs a) {
  __shared__ int tok[K2_PAGED_MAX_REQUESTS + 1], take[K2_PAGED_MAX_REQUESTS + 1], give[K2_PAGED_MAX_REQUESTS + 1];
  __shared__ int cached[K2_PAGED_MAX_REQUESTS];
  __shared__ int part[3][32];
  __shared__ int reasons;
  if (PART == kPlanMap) pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, R = a.requests;
  const int mask = (1 << a.block_log2) - 1;
  auto blocks = [&](int n) { return (n >> a.block_log2) + ((n & mask) != 0); };
  const int F = *a.free_count;
  const long long room = static_cast<long long>(a.table_stride) << a.block_log2;
  int bad = F < 0 || F > a.free_capacity ? K2_PLAN_NO_BLOCKS : 0;
  if (tid == 0) reasons = 0;
  __syncthreads();

  // this thread's kPlanPer requests, then the sums over the block
  int own[3] = {0, 0, 0}, v[kPlanPer][3];
#pragma unroll
  for (int i = 0; i < kPlanPer; ++i) {
    const int r = tid * kPlanPer + i;
    v[i][0] = v[i][1] = v[i][2] = 0;
    if (r < R) {
      const int c = a.cached[r], f = a.fresh[r];
      cached[r] = c;
      if (c < 0 || f < -1) {
        bad |= K2_PLAN_BAD_LENGTH;
      } else if (static_cast<long long>(c) + max(f, 0) > min(room, 0x7fffffffll)) {
        bad |= K2_PLAN_TABLE_FULL;
      } else if (f >= 0) {
        v[i][0] = min(f, kPlanCap);
        v[i][1] = blocks(c + f) - blocks(c);
      } else {
        v[i][2] = blocks(c);
      }
    }
#pragma unroll
    for (int q = 0; q < 3; ++q) own[q] = sat_add(own[q], v[i][q]);
  }
  int inc[3];
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    inc[q] = own[q];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, inc[q], o);
      if (lane >= o) inc[q] = sat_add(inc[q], u);
    }
    if (lane == 31) part[q][warp] = inc[q];
  }
  __syncthreads();
  if (warp < 3) {
    int t = part[warp][lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, t, o);
      if (lane >= o) t = sat_add(t, u);
    }
    part[warp][lane] = t;
  }
  if (bad) atomicOr(&reasons, bad);
  __syncthreads();
  bad = reasons;
  {
    int* sums[3] = {tok, take, give};
#pragma unroll
    for (int q = 0; q < 3; ++q) {
      const int before = __shfl_up_sync(0xffffffffu, inc[q], 1);
      int run = sat_add(warp ? part[q][warp - 1] : 0, lane ? before : 0);
#pragma unroll
      for (int i = 0; i < kPlanPer; ++i) {
        const int r = tid * kPlanPer + i;
        if (r < R) sums[q][r] = run;
        run = sat_add(run, v[i][q]);
      }
    }
  }
  const int T = part[0][31], taken = part[1][31], given = part[2][31];
  if (tid == 0) {
    tok[R] = T;
    take[R] = taken;
    give[R] = given;
  }
  const long long top = static_cast<long long>(F) + given;  // the stack with the returned blocks on it
  if (taken > top || top - taken > a.free_capacity) bad |= K2_PLAN_NO_BLOCKS;
  if (T > a.max_tokens) bad |= K2_PLAN_TOKENS_FULL;
  __syncthreads();

  const int step = gridDim.x * kPlanThreads, first = blockIdx.x * kPlanThreads + tid;
  if ((PART & kPlanMap) && !bad) {
    auto returned = [&](int k) -> int {
      const int r = find_request(give, R, k);
      return a.table[static_cast<size_t>(r) * a.table_stride + (k - give[r])];
    };
    auto popped = [&](int k) -> int {
      const long long x = top - 1 - k;
      return x < F ? a.free_ids[x] : returned(static_cast<int>(x - F));
    };
    for (int t = first; t < a.max_tokens; t += step) {
      int pos = 0, slot = -1;
      if (t < T) {
        const int r = find_request(tok, R, t);
        pos = cached[r] + (t - tok[r]);
        const int b = pos >> a.block_log2, old = blocks(cached[r]);
        const int id = b < old ? a.table[static_cast<size_t>(r) * a.table_stride + b] : popped(take[r] + b - old);
        // an id that is no block (a caller's stray entry) gives no slot
        if (id >= 0 && id <= (0x7fffffff >> a.block_log2)) slot = (id << a.block_log2) | (pos & mask);
      }
      a.slots[t] = slot;
      a.positions[t] = pos;
    }
    for (int k = first; k < taken; k += step) {
      const int r = find_request(take, R, k);
      a.table[static_cast<size_t>(r) * a.table_stride + blocks(cached[r]) + (k - take[r])] = popped(k);
    }
    for (int k = first; k < given - taken; k += step) a.free_ids[F + k] = returned(k);
  } else if (PART & kPlanMap) {
    for (int t = first; t < a.max_tokens; t += step) {
      a.slots[t] = -1;
      a.positions[t] = 0;
    }
  }
  if constexpr ((PART & kPlanFinish) != 0) {
    // kv_len may be cached and free_count_out free_count: written once everything has read them
    int keep[kPlanPer];
#pragma unroll
    for (int i = 0; i < kPlanPer; ++i) {
      const int r = tid * kPlanPer + i;
      keep[i] = r < R && !bad ? (a.fresh[r] < 0 ? 0 : cached[r] + a.fresh[r]) : r < R ? max(cached[r], 0) : 0;
    }
    if (PART == kPlanFinish) pdl_wait();
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPlanPer; ++i) {
      const int r = tid * kPlanPer + i;
      if (r < R) {
        a.kv_len[r] = keep[i];
        a.cu_new[r] = bad ? 0 : tok[r];
      }
    }
    if (tid == 0) {
      a.cu_new[R] = bad ? 0 : T;
      *a.free_count_out = bad ? F : static_cast<int>(top - taken);
      a.status[0] = bad ? 0 : T;
      a.status[1] = taken;
      a.status[2] = given;
      a.status[3] = bad;
    }
  }
}

// ---- quantizing append -------------------------------------------------------------------------
//
// A run is the maximal stretch of consecutive tokens with consecutive slots of
// one block.  A unit of work is a run's K or V rows of one head, so the scale of a
// block and head has one writer and no atomics decide anything.  A unit is taken
// by block_tokens / 16 warps, each with up to 16 rows in registers: the rows are
// read once, their maxima joined, then rounded and stored.  Such a group of warps
// looks through a window of tokens for runs that begin there; the window is wide
// where tokens are many (most of a prompt's tokens begin no run), one token where
// they are few (every token of a decode step begins one).
//
// Bound by the rows' bytes (4 in and 2 out per element pair) for prompts, of which 8192 fp16 rows of 8 heads of 128 to
// E4M3 move 3.4 TB/s in 14.7 us (20 with the division in line: its instructions, sixteen times over, no longer fit the
// instruction cache; 16 with four CTAs per SM, 17 with 8 rows per warp), and by latency for decode steps (64 rows: 3.0 us).  The
// quotient x / s decides a code only through its rounding, so it is taken as x * (1 / s), at most 2^-22 |x / s| off, and
// divided, in a second pass, only where that could change the code.
template <typename T, int E>
struct RowBits;  // E neighbouring elements of a row, as loaded
template <>
struct RowBits<float, 4> { using type = float4; };
template <>
struct RowBits<float, 2> { using type = float2; };
template <>
struct RowBits<__nv_bfloat16, 4> { using type = uint2; };
template <>
struct RowBits<__nv_bfloat16, 2> { using type = uint32_t; };
template <>
struct RowBits<__half, 4> { using type = uint2; };
template <>
struct RowBits<__half, 2> { using type = uint32_t; };

template <typename T, int E>
__device__ __forceinline__ void to_floats(const typename RowBits<T, E>::type& v, float* f) {
  if constexpr (sizeof(T) == 4) {
    const float* p = reinterpret_cast<const float*>(&v);
#pragma unroll
    for (int i = 0; i < E; ++i) f[i] = p[i];
  } else {
    const uint32_t* p = reinterpret_cast<const uint32_t*>(&v);
#pragma unroll
    for (int i = 0; i < E; i += 2) {
      if constexpr (std::is_same<T, __half>::value) {
        const float2 t = __half22float2(*reinterpret_cast<const __half2*>(p + i / 2));
        f[i] = t.x;
        f[i + 1] = t.y;
      } else {
        f[i] = bf16lo(p[i / 2]);
        f[i + 1] = bf16hi(p[i / 2]);
      }
    }
  }
}

template <int N>
struct Codes;  // N neighbouring codes
template <>
struct Codes<4> { using type = uint32_t; };
template <>
struct Codes<2> { using type = uint16_t; };

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
__device__ __forceinline__ float2 parts(f32x2 v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}
// two fp32 values to E4M3 codes, the first in the low byte
__device__ __forceinline__ uint32_t e4m3x2(f32x2 v) {
  const float2 f = parts(v);
  return __nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3);
}

template <typename C, int E>
__device__ __forceinline__ uint32_t exact_codes(const float* f, float s) {
  uint32_t u = 0;
#pragma unroll
  for (int e = 0; e < E; ++e) u |= quantize<C>(f[e], s) << (8 * e);
  return u;
}
// Codes of E finite elements under a scale of reciprocal inv; `unsure` if a quotient by the scale might have another code.
template <typename C, int E>
__device__ __forceinline__ uint32_t fast_codes(const float* f, float inv, bool& unsure) {
  uint32_t u = 0;
  if constexpr (std::is_same<C, CodeI8>::value) {
    // |y| <= 127 (1 + 2^-22).  Added to 1.5 2^23 it is rounded to an integer, whose low byte is the code; y is within
    // 2^-15 of the quotient, so only one that near a midpoint can round the other way.
    float far = 0.f;
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      const f32x2 y = mul2(pk2(f[e], f[e + 1]), pk2(inv, inv)), r = add2(y, pk2(12582912.f, 12582912.f));
      const float2 d = parts(fma2(add2(r, pk2(-12582912.f, -12582912.f)), pk2(-1.f, -1.f), y)), t = parts(r);
      far = fmaxf(far, fmaxf(fabsf(d.x), fabsf(d.y)));
      u |= (__byte_perm(__float_as_uint(t.x), __float_as_uint(t.y), 0x0040) & 0xFFFFu) << (8 * e);
    }
    unsure = far > 0.4999f;
  } else {
    // the quotient lies between the products with inv (1 - 2^-20) and inv (1 + 2^-20): the same code for both is its code
    const float a = inv * (1.f - 9.5367432e-7f), b = inv * (1.f + 9.5367432e-7f);
    uint32_t hi = 0;
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      const f32x2 x = pk2(f[e], f[e + 1]);
      u |= e4m3x2(mul2(x, pk2(a, a))) << (8 * e);
      hi |= e4m3x2(mul2(x, pk2(b, b))) << (8 * e);
    }
    unsure = u != hi;
  }
  return u;
}

constexpr int kAppendThreads = 256, kRunRows = 16;  // rows of a run that one warp takes

struct AppendArgs {
  const void* k;
  const void* v;
  long long k_stride, v_stride;
  const int* slots;
  int tokens;
  int window;  // tokens that a group looks through (1 .. 32)
};

template <typename T, typename C, int D>
__global__ void __launch_bounds__(kAppendThreads, sizeof(T) == 4 ? 2 : 3) append_kernel(const PagedPool p, const AppendArgs a) {
  constexpr int E = D / 32;
  using Bits = typename RowBits<T, E>::type;
  using Word = typename Codes<E>::type;
  __shared__ float s_top[kAppendThreads / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int B = 1 << p.block_log2, bmask = B - 1;
  const int W = B / kRunRows, group = warp / W, wi = warp & (W - 1);  // warps of a unit; this one's unit and place in it
  const int unit = blockIdx.y * (kAppendThreads / 32 / W) + group;
  if (unit >= 2 * p.n_kv) return;  // (whole groups)
  auto sync_group = [&] {
    if (W > 1) asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(32 * W) : "memory");
    else __syncwarp();
  };
  const int g = unit >> 1;
  const bool is_v = unit & 1;
  const long long limit = static_cast<long long>(p.n_blocks) << p.block_log2;
  const int t0 = blockIdx.x * a.window;
  // the runs that begin in the window
  const int tl = t0 + lane;
  const bool inside = lane < a.window && tl < a.tokens;
  const int mine = inside ? __ldg(a.slots + tl) : -1, prior = inside && tl > 0 ? __ldg(a.slots + tl - 1) : -1;
  const int ta = t0 + a.window + lane;  // 32 tokens behind the window, whose slots are on their way with the window's
  const int ahead = ta < a.tokens ? __ldg(a.slots + ta) : -1;
  const int last = __shfl_sync(0xffffffffu, mine, a.window - 1), up = __shfl_up_sync(0xffffffffu, ahead, 1);
  if (mine >= limit && unit == 0) raise_flag(p.flags, K2_PAGED_BAD_SLOT);
  // bit i: token t0 + i continues the run of the token before
  const bool goes_on = (mine & bmask) != 0 && prior == mine - 1;
  const unsigned long long on = __ballot_sync(0xffffffffu, inside && mine >= 0 && goes_on) |
                                static_cast<unsigned long long>(__ballot_sync(0xffffffffu, ahead > 0 && (ahead & bmask) != 0 && (lane ? up : last) == ahead - 1))
                                    << a.window;
  unsigned starts = __ballot_sync(0xffffffffu, mine >= 0 && mine < limit && !goes_on);
  const long long stride = is_v ? a.v_stride : a.k_stride;
  while (starts) {
    const int first = __ffs(starts) - 1;
    starts &= starts - 1;
    const int t = t0 + first, slot = __shfl_sync(0xffffffffu, mine, first), o = slot & bmask;
    int n = __ffsll(static_cast<long long>(~(on >> first >> 1)));  // a run of n tokens: n - 1 that go on
    for (bool more = first + n == a.window + 32; more;) {
      const int i = n + lane;
      const bool same = o + i < B && t + i < a.tokens && __ldg(a.slots + t + i) == slot + i;
      const unsigned m = __ballot_sync(0xffffffffu, same);
      const int run = m == 0xffffffffu ? 32 : __ffs(~m) - 1;
      n += run;
      more = run == 32;
    }
    const size_t at = static_cast<size_t>(slot >> p.block_log2) * p.n_kv + g;
    const int i0 = wi * kRunRows;
    const T* src = static_cast<const T*>(is_v ? a.v : a.k) + (t + i0) * stride + g * D + lane * E;
    uint8_t* codes = (is_v ? p.v : p.k) + (at << p.block_log2) * D + lane * E;
    float* scale = (is_v ? p.vs : p.ks) + at;
    const float was = o > 0 ? *scale : 0.f;
    Bits x[kRunRows];
#pragma unroll
    for (int i = 0; i < kRunRows; ++i)
      if (i0 + i < n) x[i] = __ldg(reinterpret_cast<const Bits*>(src + i * stride));
    // the largest magnitude: 16-bit elements two at a time.  An infinity or a NaN shows in it; the finite elements'
    // largest is then found the slow way, and every code of the unit is divided for.
    float top = 0.f;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < kRunRows; ++i) {
        if (i0 + i >= n) break;
        float f[E];
        to_floats<T, E>(x[i], f);
#pragma unroll
        for (int e = 0; e < E; ++e) asm("max.NaN.f32 %0, %0, %1;" : "+f"(top) : "f"(fabsf(f[e])));
      }
    } else {
      using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
      uint32_t z = 0;
      T2 top2 = *reinterpret_cast<const T2*>(&z);
#pragma unroll
      for (int i = 0; i < kRunRows; ++i) {
        if (i0 + i >= n) break;
        const T2* h = reinterpret_cast<const T2*>(&x[i]);
#pragma unroll
        for (int e = 0; e < E / 2; ++e) top2 = __hmax2_nan(top2, __habs2(h[e]));
      }
      const float ta = to_f32(top2.x), tb = to_f32(top2.y);
      asm("max.NaN.f32 %0, %1, %2;" : "=f"(top) : "f"(ta), "f"(tb));
    }
    bool odd = __any_sync(0xffffffffu, !(top <= 3.402823466e38f));
    if (odd) {
      top = 0.f;
#pragma unroll 1
      for (int i = 0; i < kRunRows && i0 + i < n; ++i) {
        float f[E];
        to_floats<T, E>(__ldg(reinterpret_cast<const Bits*>(src + i * stride)), f);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float m = fabsf(f[e]);
          if (m <= 3.402823466e38f) top = fmaxf(top, m);
        }
      }
    }
    top = warp_max_redux(top);
    if (W > 1) {
      if (lane == 0) s_top[warp] = top;
      sync_group();
      for (int w = 0; w < W; ++w) top = fmaxf(top, s_top[group * W + w]);
    }
    const float now = fmaxf(was, __fdiv_rn(top, C::kMax));
    if (o > 0 && now > was) {  // the rows before, rounded to the larger scale
      const float ratio = __fdiv_rn(was, now);
      for (int i = wi; i < o; i += 8 * W) {
        Word c[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (i + j * W < o) c[j] = *reinterpret_cast<const Word*>(codes + static_cast<size_t>(i + j * W) * D);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (i + j * W >= o) break;
          uint32_t u = 0;
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const float y = __fmul_rn(C::value((c[j] >> (8 * e)) & 0xFFu), ratio);
            u |= (y == y ? C::round(y) : 0u) << (8 * e);
          }
          *reinterpret_cast<Word*>(codes + static_cast<size_t>(i + j * W) * D) = static_cast<Word>(u);
        }
      }
    }
    odd |= !(now > 1e-30f);  // (1 / now may not be finite)
    const float inv = __frcp_rn(now);
    Word* to = reinterpret_cast<Word*>(codes + static_cast<size_t>(o + i0) * D);
    unsigned unsure = 0;  // this lane's rows, a bit each
#pragma unroll
    for (int i = 0; i < kRunRows; ++i) {
      if (i0 + i >= n) break;
      float f[E];
      to_floats<T, E>(x[i], f);
      bool u;
      to[i * (D / sizeof(Word))] = static_cast<Word>(fast_codes<C, E>(f, inv, u));
      unsure |= static_cast<unsigned>(u) << i;
    }
    unsure = odd ? (1u << max(0, min(n - i0, kRunRows))) - 1 : unsure;
#pragma unroll 1
    while (unsure) {
      const int i = __ffs(unsure) - 1;
      unsure &= unsure - 1;
      float f[E];
      to_floats<T, E>(__ldg(reinterpret_cast<const Bits*>(src + i * stride)), f);
      to[i * (D / sizeof(Word))] = static_cast<Word>(exact_codes<C, E>(f, now));
    }
    sync_group();  // every warp of the unit has read the old scale, and s_top
    if (wi == 0 && lane == 0) *scale = now;
  }
}

template <typename T, typename C>
cudaError_t launch_append(const PagedPool& p, int head_dim, AppendArgs a, cudaStream_t s) {
  const int warps = (1 << p.block_log2) / kRunRows, units = 2 * p.n_kv, per_cta = kAppendThreads / 32 / warps;
  // windows so wide that some 32 warps per SM look through them
  const long long all = static_cast<long long>(a.tokens) * units * warps / (152 * 32);
  a.window = 1;
  while (a.window < 32 && a.window * 2 <= all) a.window *= 2;
  const dim3 grid((a.tokens + a.window - 1) / a.window, (units + per_cta - 1) / per_cta);
  if (head_dim == 128) append_kernel<T, C, 128><<<grid, kAppendThreads, 0, s>>>(p, a);
  else append_kernel<T, C, 64><<<grid, kAppendThreads, 0, s>>>(p, a);
  return cudaGetLastError();
}
template <typename T>
cudaError_t launch_append(const PagedPool& p, const k2_paged_kv& kv, const AppendArgs& a, cudaStream_t s) {
  return kv.dtype == K2_I8 ? launch_append<T, CodeI8>(p, kv.head_dim, a, s)
                           : launch_append<T, CodeF8>(p, kv.head_dim, a, s);
}

}  // namespace

}  // namespace k2

using namespace k2;

extern "C" {

k2_status k2_paged_plan(const int32_t* d_cached, const int32_t* d_fresh, int32_t requests, int32_t block_tokens,
                        int32_t* d_table, int32_t table_stride, int32_t* d_free, int32_t free_capacity,
                        const int32_t* d_free_count, int32_t* d_free_count_out, int32_t* d_kv_len,
                        int32_t* d_cu_new, int32_t* d_slots, int32_t* d_positions, int32_t max_tokens,
                        int32_t* d_status, void* stream) {
  if (!d_cached || !d_fresh || !d_table || !d_free || !d_free_count || !d_free_count_out || !d_kv_len || !d_cu_new ||
      !d_slots || !d_positions || !d_status) {
    set_error("every pointer of a plan must be non-null");
    return K2_ERR_ARG;
  }
  if (block_tokens != 16 && block_tokens != 32 && block_tokens != 64 && block_tokens != 128) {
    set_error("block_tokens must be 16, 32, 64 or 128 (got %d)", block_tokens);
    return K2_ERR_UNSUPPORTED;
  }
  if (requests < 1 || requests > K2_PAGED_MAX_REQUESTS) {
    set_error("requests %d outside [1, %d]", requests, K2_PAGED_MAX_REQUESTS);
    return K2_ERR_SHAPE;
  }
  if (table_stride < 1 || free_capacity < 1 || max_tokens < 1 || max_tokens > kPlanCap - 1) {
    set_error("table_stride, free_capacity and max_tokens must be positive, max_tokens below 2^30 (got %d, %d, %d)",
              table_stride, free_capacity, max_tokens);
    return K2_ERR_SHAPE;
  }
  PlanArgs a = {d_cached, d_fresh, requests, 31 - __builtin_clz(block_tokens), d_table, table_stride, d_free,
                free_capacity, d_free_count, d_free_count_out, d_kv_len, d_cu_new, d_slots, d_positions, max_tokens,
                d_status};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (max_tokens <= kPlanThreads) {
    plan_kernel<kPlanMap | kPlanFinish><<<1, kPlanThreads, 0, st>>>(a);
    e = cudaGetLastError();
  } else {
    plan_kernel<kPlanMap><<<std::min((max_tokens - 1) / kPlanThreads + 1, kPlanCtas), kPlanThreads, 0, st>>>(a);
    e = cudaGetLastError();
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(kPlanThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, plan_kernel<kPlanFinish>, a);
  }
  if (e == cudaSuccess) return K2_OK;
  set_error("plan launch: %s", cudaGetErrorString(e));
  return K2_ERR_CUDA;
}

k2_status k2_paged_append(const k2_paged_kv* kv, const void* d_k, const void* d_v, int32_t dtype, int64_t k_stride,
                          int64_t v_stride, const int32_t* d_slots, int32_t tokens, void* stream) {
  const k2_status st = check_paged_kv(kv);
  if (st != K2_OK) return st;
  if (dtype != K2_BF16 && dtype != K2_F16 && dtype != K2_F32) {
    set_error("K and V rows must be K2_BF16, K2_F16 or K2_F32 (got dtype %d)", dtype);
    return K2_ERR_UNSUPPORTED;
  }
  if (tokens < 0 || tokens > 1 << 30) {
    set_error("tokens must be in [0, 2^30] (got %d)", tokens);
    return K2_ERR_ARG;
  }
  if (tokens == 0) return K2_OK;
  if (!d_k || !d_v || !d_slots) {
    set_error("d_k, d_v and d_slots must be non-null");
    return K2_ERR_ARG;
  }
  const int64_t row = static_cast<int64_t>(kv->n_kv_heads) * kv->head_dim;
  const int bytes = dtype == K2_F32 ? 4 : 2;
  if ((tokens > 1 && (k_stride < row || v_stride < row || k_stride * bytes % 16 || v_stride * bytes % 16)) || !aligned16(d_k) || !aligned16(d_v)) {
    set_error("K and V rows must be 16-byte aligned and at least n_kv_heads * head_dim elements apart");
    return K2_ERR_ARG;
  }
  const PagedPool p(*kv);
  const AppendArgs a = {d_k, d_v, k_stride, v_stride, d_slots, tokens, 1};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == K2_F32    ? launch_append<float>(p, *kv, a, s)
                        : dtype == K2_BF16 ? launch_append<__nv_bfloat16>(p, *kv, a, s)
                                           : launch_append<__half>(p, *kv, a, s);
  if (e == cudaSuccess) return K2_OK;
  set_error("append launch: %s", cudaGetErrorString(e));
  return K2_ERR_CUDA;
}

}  // extern "C"
