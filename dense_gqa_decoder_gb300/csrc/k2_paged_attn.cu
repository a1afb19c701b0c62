// Causal attention of many requests' newest tokens over a block-paged 8-bit
// cache (k2_paged_attention; the formula is stated in include/k2.h).
#include <math.h>

#include <algorithm>

#include "k2_paged.cuh"

namespace k2 {

namespace {

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
};

constexpr int kThreads = 128, kWarps = kThreads / 32, kMaxRep = 16;

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// One CTA per query token and KV head: its warps take every fourth key, a lane
// head_dim / 32 neighbouring dims; each warp keeps a running maximum, sum and
// output per query head, merged at the end.
template <typename T, typename C, int D>
__global__ void __launch_bounds__(kThreads) paged_attn_simple_kernel(const PagedPool p, const PagedAttnArgs a) {
  constexpr int E = D / 32;
  __shared__ float qs[kMaxRep][D];
  __shared__ float sm[kWarps][kMaxRep], sl[kWarps][kMaxRep], so[kWarps][kMaxRep][D];
  const int t = blockIdx.x, g = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rep = a.n_heads / p.n_kv;
  if (t == 0 && g == 0)
    for (int i = tid; i < a.requests; i += kThreads)
      if (a.cu_q[i] < 0 || a.cu_q[i + 1] < a.cu_q[i] || a.cu_q[i + 1] > a.tokens) raise_flag(p.flags, K2_PAGED_BAD_LENGTH);
  int r = 0;
  while (r < a.requests && !(a.cu_q[r] <= t && t < a.cu_q[r + 1])) ++r;
  if (r == a.requests) return;
  const int q0 = a.cu_q[r], nq = a.cu_q[r + 1] - q0, len = a.kv_len[r];
  const bool ok = q0 >= 0 && a.cu_q[r + 1] <= a.tokens && nq <= a.max_q && nq <= len &&
                  len <= (static_cast<long long>(a.table_stride) << p.block_log2);
  if (!ok && tid == 0) raise_flag(p.flags, K2_PAGED_BAD_LENGTH);
  const int keys = ok ? len - nq + (t - q0) + 1 : 0;
  const T* q = static_cast<const T*>(a.q) + t * a.q_stride + static_cast<size_t>(g) * rep * D;
  for (int i = tid; i < rep * D; i += kThreads) qs[i / D][i % D] = to_f32(q[i]) * a.scale;
  __syncthreads();
  float m[kMaxRep], l[kMaxRep], o[kMaxRep][E];
  for (int h = 0; h < kMaxRep; ++h) {
    m[h] = -INFINITY;
    l[h] = 0.f;
    for (int e = 0; e < E; ++e) o[h][e] = 0.f;
  }
  for (int j = warp; j < keys; j += kWarps) {
    const int b = a.table[static_cast<size_t>(r) * a.table_stride + (j >> p.block_log2)];
    if (b < 0 || b >= p.n_blocks) {
      if (lane == 0) raise_flag(p.flags, K2_PAGED_BAD_BLOCK);
      continue;
    }
    const size_t at = static_cast<size_t>(b) * p.n_kv + g;
    const size_t row = ((at << p.block_log2) + (j & ((1 << p.block_log2) - 1))) * D + lane * E;
    float kf[E], vf[E];
    for (int e = 0; e < E; ++e) {
      kf[e] = C::value(p.k[row + e]) * p.ks[at];
      vf[e] = C::value(p.v[row + e]) * p.vs[at];
    }
    for (int h = 0; h < rep; ++h) {
      float s = 0.f;
      for (int e = 0; e < E; ++e) s += qs[h][lane * E + e] * kf[e];
      s = warp_sum(s);
      const float mn = fmaxf(m[h], s), al = expf(m[h] - mn), w = expf(s - mn);
      l[h] = l[h] * al + w;
      for (int e = 0; e < E; ++e) o[h][e] = o[h][e] * al + w * vf[e];
      m[h] = mn;
    }
  }
  for (int h = 0; h < rep; ++h) {
    sm[warp][h] = m[h];
    sl[warp][h] = l[h];
    for (int e = 0; e < E; ++e) so[warp][h][lane * E + e] = o[h][e];
  }
  __syncthreads();
  T* out = static_cast<T*>(a.out) + t * a.out_stride + static_cast<size_t>(g) * rep * D;
  for (int i = tid; i < rep * D; i += kThreads) {
    const int h = i / D, d = i % D;
    float mm = -INFINITY, ll = 0.f, oo = 0.f;
    for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, sm[w][h]);
    for (int w = 0; w < kWarps; ++w) {
      const float f = mm > -INFINITY ? expf(sm[w][h] - mm) : 0.f;
      ll += sl[w][h] * f;
      oo += so[w][h][d] * f;
    }
    out[i] = from_f32<T>(ll > 0.f ? oo / ll : 0.f);
  }
}

template <typename T, typename C>
cudaError_t launch(const PagedPool& p, int head_dim, const PagedAttnArgs& a, cudaStream_t s) {
  const dim3 grid(a.tokens, p.n_kv);
  if (head_dim == 128) paged_attn_simple_kernel<T, C, 128><<<grid, kThreads, 0, s>>>(p, a);
  else paged_attn_simple_kernel<T, C, 64><<<grid, kThreads, 0, s>>>(p, a);
  return cudaGetLastError();
}

}  // namespace

}  // namespace k2

using namespace k2;

extern "C" {

size_t k2_paged_workspace_bytes(void) { return 256; }

k2_status k2_paged_attention(const k2_paged_kv* kv, const void* d_q, int32_t dtype, int64_t q_stride,
                             const int32_t* d_cu_q, const int32_t* d_kv_len, const int32_t* d_table,
                             int32_t table_stride, int32_t requests, int32_t tokens, int32_t n_heads, int32_t max_q,
                             float scale, void* d_out, int64_t out_stride, void* d_workspace, size_t ws_bytes,
                             void* stream) {
  const k2_status st = check_paged_kv(kv);
  if (st != K2_OK) return st;
  if (dtype != K2_BF16 && dtype != K2_F16) {
    set_error("queries must be K2_BF16 or K2_F16 (got dtype %d)", dtype);
    return K2_ERR_UNSUPPORTED;
  }
  if (n_heads < 1 || n_heads % kv->n_kv_heads || n_heads / kv->n_kv_heads > kMaxRep) {
    set_error("n_heads must be 1 to %d times n_kv_heads (got %d over %d)", kMaxRep, n_heads, kv->n_kv_heads);
    return K2_ERR_SHAPE;
  }
  if (requests < 0 || requests > K2_PAGED_MAX_REQUESTS || tokens < 0 || max_q < 0 || table_stride < 1) {
    set_error("requests in [0, %d], tokens and max_q >= 0, table_stride >= 1 (got %d, %d, %d, %d)",
              K2_PAGED_MAX_REQUESTS, requests, tokens, max_q, table_stride);
    return K2_ERR_SHAPE;
  }
  if (!isfinite(scale)) {
    set_error("scale must be finite");
    return K2_ERR_ARG;
  }
  if (requests == 0 || tokens == 0 || max_q == 0) return K2_OK;
  if (!d_q || !d_cu_q || !d_kv_len || !d_table || !d_out) {
    set_error("d_q, d_cu_q, d_kv_len, d_table and d_out must be non-null");
    return K2_ERR_ARG;
  }
  const int64_t row = static_cast<int64_t>(n_heads) * kv->head_dim;
  if ((tokens > 1 && (q_stride < row || out_stride < row)) || q_stride % 8 || out_stride % 8 || !aligned16(d_q) ||
      !aligned16(d_out)) {
    set_error("query and output rows must be 16-byte aligned and at least n_heads * head_dim elements apart");
    return K2_ERR_ARG;
  }
  if (!d_workspace || reinterpret_cast<uintptr_t>(d_workspace) % 256 || ws_bytes < k2_paged_workspace_bytes()) {
    set_error("workspace must be 256-byte aligned and hold k2_paged_workspace_bytes() = %zu bytes (got %zu)",
              k2_paged_workspace_bytes(), ws_bytes);
    return K2_ERR_WORKSPACE;
  }
  const PagedPool p(*kv);
  const PagedAttnArgs a = {d_q, q_stride, d_cu_q, d_kv_len, d_table, table_stride, requests,
                           tokens, n_heads, std::min(max_q, tokens), scale, d_out, out_stride};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (dtype == K2_F16)
    e = kv->dtype == K2_I8 ? launch<__half, CodeI8>(p, kv->head_dim, a, s) : launch<__half, CodeF8>(p, kv->head_dim, a, s);
  else
    e = kv->dtype == K2_I8 ? launch<__nv_bfloat16, CodeI8>(p, kv->head_dim, a, s)
                           : launch<__nv_bfloat16, CodeF8>(p, kv->head_dim, a, s);
  if (e == cudaSuccess) return K2_OK;
  set_error("attention launch: %s", cudaGetErrorString(e));
  return K2_ERR_CUDA;
}

}  // extern "C"
