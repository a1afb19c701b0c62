// Matrix product with an epilogue: out = act(w_scale x_scale (x . w^T) + bias) + residual, on the 5th-generation tensor
// cores.
//
//   z[t][n] = sum_k x[t][k] w[n][k]      (E4M3, bf16 or fp16 operands, exact products, fp32 sums in tensor memory)
//   out[t][n] = act(z * w_scale[n] * x_scale[t] + bias[n]) + residual[t][n]
//
// The weights' 128-row tiles are the first operand (M), the tokens the second (N): few tokens then cost few columns and not 128
// rows.  Both arrive as K-major rows of 128 bytes by TMA (zeros behind the last row and behind the last value of a row) through
// a ring of stages; two warps request, one issues the MMAs.  Two kernels: for few tokens the weights' bytes bound the call
// (linear_few_kernel), for many the tensor cores (linear_pair_kernel).
#include <cuda.h>
#include <limits.h>
#include <math.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "k2_common.cuh"
#include "k2_linear.h"
#include "k2_paged.cuh"
#include "k2_tc.cuh"

namespace k2 {

namespace {

constexpr int kRows = 128;      // weight rows of a tile (TMEM lanes)
constexpr int kStepBytes = 128; // bytes of K per stage: one swizzle row
constexpr int kMaxSplit = 8;    // CTAs of a cluster (the portable limit)

__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void load_2d(void* dst, const CUtensorMap* m, int c0, int c1, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          smem_u32(dst)),
      "l"(m), "r"(c0), "r"(c1), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void load_4d(void* dst, const CUtensorMap* m, int c0, int c1, int c2, int c3, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];" ::"r"(smem_u32(dst)),
      "l"(m), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar))
      : "memory");
}
// Waits for a phase; false once limit_ns have passed (a single try may sleep for longer, so that counts as run out too).
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, unsigned long long limit_ns) {
  uint32_t ready;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ready)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  if (ready) return true;
  const uint64_t t0 = globaltimer();
  while (!mbar_try_wait(bar, parity))
    if (globaltimer() - t0 > limit_ns) return false;
  return globaltimer() - t0 <= limit_ns;
}
// The requesting and the issuing warp run their loops as whole warps, and one lane does what has to be done once: so the compiler
// keeps what those instructions take in uniform registers, where they want it.  (With the whole loop in one thread four MMAs took
// 231 clocks to issue, 107 to look at a barrier that had completed and 85 to commit, and a K step of few tokens 0.30 us.)
__device__ __forceinline__ int warp_index() { return __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) >> 5, 0); }
__device__ __forceinline__ bool elected() {
  uint32_t yes;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(yes));
  return yes != 0;
}
// the same answer in all lanes
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, unsigned long long limit_ns) {
  return __all_sync(0xffffffffu, wait_for(bar, parity, limit_ns));
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// the address in CTA `rank` of the cluster
__device__ __forceinline__ uint32_t peer_address(uint32_t addr, int rank) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(addr), "r"(rank));
  return at;
}
__device__ __forceinline__ void peer_store(uint32_t at, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(v) : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* m) { asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory"); }

// the activations, in fp32
__device__ __forceinline__ float activate(float z, int act) {
  if (act == K2_ACT_RELU) return z < 0.f ? 0.f : z;
  if (act == K2_ACT_SILU) return z / (1.0f + expf(-z));
  if (act == K2_ACT_GELU) return 0.5f * z * erfcf(z * -0.70710678f);
  if (act == K2_ACT_GELU_TANH) return z / (1.0f + expf(-1.5957691216f * (z + 0.044715f * z * z * z)));
  return z;
}

// silu(g) u.  With an fp32 output to four steps of fp32: exponential and reciprocal one each, the sum and the two products half of
// one each.  With a 16-bit output the exponential's argument is rounded, so that it is off by some 1.5 |g| + 6 steps: at most 2^-15
// of the value, a sixteenth of fp16's own half step.  (Gate and up of 2048 tokens in bf16 66.8 us so, 69.2 with expf.)  Below -88.7
// e^-g is infinite in fp32, and the result 0.
template <typename OT>
__device__ __forceinline__ float swiglu(float g, float u) {
  float r;
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(1.0f + (std::is_same<OT, float>::value ? expf(-g) : __expf(-g))));
  return g * r * u;
}

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

enum { kPlain, kPairsOfRows, kOther };  // what follows the sums: nothing, SwiGLU, another activation

constexpr int kColumns = 16;  // columns of the accumulator that a warp has in registers

// Some columns of the accumulator (tokens t ..) of this lane's row n: z = (v * ws) * xs + bias (a product of the two scales
// might leave the normal numbers where the result does not), then the activation, the
// residual and the stores.  Nothing waits for the column before: the scales are in shared memory, the residual is loaded ahead.
template <typename OT, int ACT, bool FULL>
__device__ __forceinline__ void finish_columns(const LinearArgs& a, const uint32_t (&v)[kColumns], const float* xs, int t, int n,
                                               float ws, float bias) {
  const bool odd = n & 1, row = n < a.rows;
  const int most = a.tokens - t;  // columns of tokens (not FULL: fewer than there are columns)
  if (ACT == kPairsOfRows) {
    // a gate and its factor lie in neighbouring lanes: of two columns the even lane finishes the first, the odd lane the second
    const int mine = odd ? 1 : 0;
    const long long first = t + mine;
    float res[kColumns / 2];
    if (a.residual != nullptr) {
      const OT* from = static_cast<const OT*>(a.residual) + first * a.residual_stride + (n >> 1);
#pragma unroll
      for (int j = 0; j < kColumns; j += 2, from += 2 * a.residual_stride)
        res[j / 2] = row && (FULL || j + mine < most) ? to_f32(*from) : 0.f;
    }
    OT* out = static_cast<OT*>(a.out) + first * a.out_stride + (n >> 1);
#pragma unroll
    for (int j = 0; j < kColumns; j += 2, out += 2 * a.out_stride) {
      const float2 x = *reinterpret_cast<const float2*>(xs + j);
      const float z0 = fmaf(__uint_as_float(v[j]) * ws, x.x, bias), z1 = fmaf(__uint_as_float(v[j + 1]) * ws, x.y, bias);
      const float other = __shfl_xor_sync(0xffffffffu, odd ? z0 : z1, 1);
      const float g = odd ? other : z0, u = odd ? z1 : other;
      float y = swiglu<OT>(g, u);
      if (a.residual != nullptr) y += res[j / 2];
      if (row && (FULL || j + mine < most)) *out = from_f32<OT>(y);
    }
    return;
  }
  float res[kColumns];
  if (a.residual != nullptr) {
    const OT* from = static_cast<const OT*>(a.residual) + static_cast<long long>(t) * a.residual_stride + n;
#pragma unroll
    for (int j = 0; j < kColumns; ++j, from += a.residual_stride) res[j] = row && (FULL || j < most) ? to_f32(*from) : 0.f;
  }
  OT* out = static_cast<OT*>(a.out) + static_cast<long long>(t) * a.out_stride + n;
#pragma unroll
  for (int j = 0; j < kColumns; j += 4) {
    const float4 x = *reinterpret_cast<const float4*>(xs + j);
    const float x4[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i, out += a.out_stride) {
      float y = fmaf(__uint_as_float(v[j + i]) * ws, x4[i], bias);
      if (ACT == kOther) y = activate(y, a.act);
      if (a.residual != nullptr) y += res[j + i];
      if (row && (FULL || j + i < most)) *out = from_f32<OT>(y);
    }
  }
}
// The residual of what four neighbouring rows n .. n + 3 of the matrix give token t.
template <typename OT, int ACT>
__device__ __forceinline__ void residual_four(const LinearArgs& a, long long t, int n, float (&r)[4]) {
  constexpr int kPer = ACT == kPairsOfRows ? 2 : 1, kOut = 4 / kPer;  // rows of an output, outputs
  const OT* from = static_cast<const OT*>(a.residual) + t * a.residual_stride + n / kPer;
#pragma unroll
  for (int j = 0; j < kOut; ++j) r[j] = a.residual != nullptr && n + kPer * j < a.rows ? to_f32(from[j]) : 0.f;
}
// What follows the sums of these.
template <typename OT, int ACT>
__device__ __forceinline__ void finish_four(const LinearArgs& a, long long t, int n, float4 z4, float xs, const float (&ws)[4],
                                            const float (&bias)[4], const float (&r)[4]) {
  constexpr int kPer = ACT == kPairsOfRows ? 2 : 1, kOut = 4 / kPer;
  float z[4] = {z4.x, z4.y, z4.z, z4.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) z[j] = fmaf(z[j] * ws[j], xs, bias[j]);
  OT* out = static_cast<OT*>(a.out) + t * a.out_stride + n / kPer;
#pragma unroll
  for (int j = 0; j < kOut; ++j) {
    float y = ACT == kPairsOfRows ? swiglu<OT>(z[2 * j % 4], z[(2 * j + 1) % 4])
              : ACT == kOther     ? activate(z[j], a.act)
                                  : z[j];
    if (a.residual != nullptr) y += r[j];
    if (n + kPer * j < a.rows) out[j] = from_f32<OT>(y);
  }
}

// where a stage's weights lie: rows apart, or packed pairs of rows in chunks of 512 bytes
struct WeightPlace {
  int packed;
  int step;  // elements of K per stage
};
__device__ __forceinline__ void load_weights(void* dst, const CUtensorMap* m, const WeightPlace& p, int k, int row, uint64_t* bar) {
  const int e = k * p.step;
  if (p.packed) load_4d(dst, m, e & 511, 0, e >> 9, row >> 1, bar);
  else load_4d(dst, m, e, row, 0, 0, bar);
}

// ---- few tokens -----------------------------------------------------------------------------------------------------------
//
// A CTA per tile of 128 rows x 16, 32 or 64 tokens.  Where there are fewer tiles than SMs, a cluster of up to eight CTAs splits
// K: token j's sums go to CTA j % split, each CTA writing its share into that CTA's shared memory, and are added there in the
// order of K, so that the result does not depend on which CTA came first.  One CTA per SM is enough (q|k|v of one token took 8.6
// us with twice as many, whose clusters no longer fit at once, and 5.7 with these; 4.8 now).  The weights stream at 6.7 TB/s
// behind some 3.6 us of start, first loads and end (gate and up of 16 tokens, 52 MB: 11.2 us).
constexpr int kFewTokens = 64, kFewStages = 5, kFewRing = 92 * 1024;  // two CTAs fit an SM

struct FewShape {
  int tokens;  // of a tile: 16, 32 or 64
  int steps;   // of K
  int stages;  // of the ring
  int split;   // CTAs that share a tile's K
};
__host__ __device__ constexpr int few_stage(int tokens) { return (kRows + tokens) * kStepBytes; }
// the sums that a CTA joins
__host__ __device__ constexpr int few_part(int tokens, int split) { return split > 1 ? (tokens + split - 1) * kRows * 4 : 0; }

template <bool F8, typename OT, int ACT>
__global__ void __launch_bounds__(128) linear_few_kernel(const __grid_constant__ CUtensorMap map_w,
                                                         const __grid_constant__ CUtensorMap map_x, const LinearArgs a,
                                                         const WeightPlace place, const FewShape sh) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  __shared__ __align__(8) uint64_t full[kFewStages], empty[kFewStages], done;
  __shared__ __align__(16) float xs[kFewTokens];
  __shared__ uint32_t tmem_slot;
  const int tid = threadIdx.x, warp = warp_index(), lane = tid & 31, split = sh.split;
  const int tile = blockIdx.x / split, rank = blockIdx.x - tile * split;
  const int n0 = tile * kRows, t0 = blockIdx.y * sh.tokens, tokens = min(sh.tokens, a.tokens - t0);
  const int k0 = static_cast<int>(static_cast<long long>(sh.steps) * rank / split);
  const int nk = static_cast<int>(static_cast<long long>(sh.steps) * (rank + 1) / split) - k0;
  const int stage = few_stage(sh.tokens);
  if (split > 1) cluster_arrive();  // this CTA runs: its shared memory may be written to
  if (tid == 0) {
    prefetch_map(&map_w);
    prefetch_map(&map_x);
    for (int s = 0; s < sh.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(&done, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)), "n"(kFewTokens)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = tmem_slot;
  pdl_wait();  // what the call reads and writes may be the previous kernel's
  pdl_trigger();
  // on their way meanwhile: scales and biases of what this thread finishes, its own row or (split) four neighbouring ones
  const int n = n0 + (split > 1 ? 4 * lane : tid);
  float ws[4], bias[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const bool there = n + j < a.rows && (j == 0 || split > 1);
    ws[j] = a.w_scale != nullptr && there ? __ldg(a.w_scale + n + j) : 1.f;
    bias[j] = a.bias != nullptr && there ? __ldg(a.bias + n + j) : 0.f;
  }
  constexpr int kEarly = 4;  // residuals of a warp's first tokens, loaded ahead of the sums
  float early[kEarly][4];
  if (split > 1) {
#pragma unroll
    for (int q = 0; q < kEarly; ++q) {
      const int j = rank + (warp + 4 * q) * split;
      if (j < tokens) residual_four<OT, ACT>(a, t0 + j, n, early[q]);
    }
  }
  if (warp == 3)
    for (int j = lane; j < kFewTokens; j += 32) xs[j] = a.x_scale != nullptr && j < tokens ? __ldg(a.x_scale + t0 + j) : 1.f;
  bool ok = true;
  if (warp == 0 || warp == 2) {  // the weights, the tokens: a request takes some 125 clocks to issue
    int i = 0, s = 0;
    uint32_t ph = 0;  // how often the ring wrapped
    for (; i < nk; ++i) {
      if (ph > 0 && !warp_wait(&empty[s], (ph - 1) & 1u, a.limit_ns)) {
        ok = false;
        break;
      }
      if (elected()) {
        uint8_t* st = smem + s * stage;
        if (warp == 0) {
          mbar_arrive_expect_tx(&full[s], static_cast<uint32_t>(stage));
          load_weights(st, &map_w, place, k0 + i, n0, &full[s]);
        } else {
          load_2d(st + kRows * kStepBytes, &map_x, (k0 + i) * place.step, t0, &full[s]);
        }
      }
      __syncwarp();
      if (++s == sh.stages) s = 0, ++ph;
    }
    // no copy may be on its way when this CTA ends (after a wait that ran out this one runs out too, a second during which what
    // is on its way lands)
    for (int j = min(i, sh.stages); j > 0; --j) {
      s = s == 0 ? (--ph, sh.stages - 1) : s - 1;
      if (!mbar_wait(&full[s], ph & 1u)) break;
    }
    __syncwarp();
  } else if (warp == 1) {
    const uint32_t idesc = (1u << 4) | (static_cast<uint32_t>(sh.tokens >> 3) << 17) | (8u << 24) |  // fp32 sums, M = 128
                           (a.dtype == K2_BF16 ? (1u << 7) | (1u << 10) : 0u);
    const uint64_t ring = smem_desc(smem);
    int s = 0;
    uint32_t ph = 0;
    for (int i = 0; i < nk; ++i) {
      if (!warp_wait(&full[s], ph & 1u, a.limit_ns)) {
        ok = false;
        break;
      }
      tc_after();
      const uint64_t at = ring + static_cast<uint32_t>(s * (stage >> 4));
      if (elected()) {
#pragma unroll
        for (int j = 0; j < kStepBytes / 32; ++j) {  // descriptors count 16 bytes
          if (F8) mma_f8(tmem, at + 2 * j, at + (kRows * kStepBytes >> 4) + 2 * j, idesc, (i | j) != 0);
          else mma(tmem, at + 2 * j, at + (kRows * kStepBytes >> 4) + 2 * j, idesc, (i | j) != 0);
        }
        mma_commit(&empty[s]);
      }
      __syncwarp();
      if (++s == sh.stages) s = 0, ++ph;
    }
    if (elected()) mma_commit(&done);
    __syncwarp();
  }
  if (split > 1) {
    __syncwarp();
    cluster_wait();  // the others run
  }
  __syncthreads();  // both roles have ended: what is waited for now are the MMAs that were issued
  ok = mbar_wait(&done, 0) && ok;
  ok = __syncthreads_and(ok);
  tc_after();
  if (!ok && tid == 0 && a.flags != nullptr) atomicOr(a.flags, a.bit);
  const uint32_t acc = tmem + (static_cast<uint32_t>(warp * 32) << 16);
  if (split == 1) {
    if (!ok) ws[0] = __uint_as_float(0x7FC00000u);
#pragma unroll 1
    for (int c = 0; c < tokens; c += kColumns) {
      uint32_t v[kColumns];
      tmem_ld16(acc + c, v);
      if (c + kColumns <= tokens) finish_columns<OT, ACT, true>(a, v, xs + c, t0 + c, n, ws[0], bias[0]);
      else finish_columns<OT, ACT, false>(a, v, xs + c, t0 + c, n, ws[0], bias[0]);
    }
    tc_before();
    __syncthreads();  // every warp has read the accumulator
    if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kFewTokens) : "memory");
  } else {
    // this thread's row of the sums, token by token, to the CTA that joins them: [rank][token / split][row]
    float* part = reinterpret_cast<float*>(smem + sh.stages * stage);
    const int slots = (sh.tokens + split - 1) / split;
    int owner = 0;
    uint32_t at = smem_u32(part) + static_cast<uint32_t>(rank * slots * kRows + tid) * 4u;
#pragma unroll 1
    for (int c = 0; c < tokens; c += kColumns) {
      uint32_t v[kColumns];
      tmem_ld16(acc + c, v);
#pragma unroll
      for (int j = 0; j < kColumns; ++j) {
        if (c + j < tokens) peer_store(peer_address(at, owner), ok ? __uint_as_float(v[j]) : __uint_as_float(0x7FC00000u));
        if (++owner == split) owner = 0, at += kRows * 4;
      }
    }
    // Tensor memory is given back before the others are waited for: no CTA holds any while one of its cluster may still be
    // waiting for its own behind another kernel's, so that kernels on several streams cannot wait for one another in a ring.
    tc_before();
    __syncthreads();
    if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kFewTokens) : "memory");
    cluster_arrive();
    cluster_wait();
    auto join = [&](int slot, const float (&r)[4]) {
      const float4* from = reinterpret_cast<const float4*>(part + slot * kRows) + lane;
      float4 z = from[0];
#pragma unroll
      for (int i = 1; i < kMaxSplit; ++i) {
        if (i < split) {
          const float4 p = from[i * slots * (kRows / 4)];
          z.x += p.x, z.y += p.y, z.z += p.z, z.w += p.w;
        }
      }
      const int j = rank + slot * split;
      finish_four<OT, ACT>(a, t0 + j, n, z, xs[j], ws, bias, r);
    };
#pragma unroll
    for (int q = 0; q < kEarly; ++q)
      if (rank + (warp + 4 * q) * split < tokens) join(warp + 4 * q, early[q]);
#pragma unroll 1
    for (int slot = warp + 4 * kEarly; rank + slot * split < tokens; slot += 4) {
      float r[4];
      residual_four<OT, ACT>(a, t0 + rank + slot * split, n, r);
      join(slot, r);
    }
  }
}

// ---- many tokens: pairs of CTAs -------------------------------------------------------------------------------------------
//
// A pair of CTAs (the two SMs of a TPC) works on tiles of 256 weight rows x up to 256 tokens with one MMA over both SMs
// (cta_group::2): each CTA holds its own 128 rows and half of the tokens, so that an SM takes in 32 KB for 128 x 256 x 128
// products of E4M3 codes (a CTA by itself would take in 48 KB).  Gate and up of 2048 tokens take 66 us (3250 TFLOP/s) in bursts and
// 76 (2810) back to back under the power cap, 240 by single CTAs; 4096 x 10240 by 2560 in bf16 131 us (1640) and 151 (1420).
// Persistent, roles as warps:
//   warps 0, 2  request the weights and the tokens of their CTA's stages (completion is counted by the first CTA's barriers)
//   warp 1      of the first CTA issues the MMAs, into one of two accumulators of 256 tensor-memory columns
//   warps 3-18  read the other accumulator and finish its tile; a warp's lanes are 32 neighbouring outputs of a token
// (Both SMs' tensor memory is taken at once and whole; what else may hold some there gives it back by itself, and a second
// pair has no room in shared memory.)
constexpr int kPairTokens = 256, kPairStages = 8, kPairRing = 208 * 1024;  // four stages of two steps of 160 tokens
constexpr int kPairSmem = kPairRing + 1024;
constexpr int kPairOthers = 3, kPairFinishers = 16, kPairThreads = 32 * (kPairOthers + kPairFinishers);

__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// the address of a barrier in the pair's first CTA
__device__ __forceinline__ uint32_t first_cta(const uint64_t* bar) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(at) : "r"(smem_u32(bar)));
  return at;
}
__device__ __forceinline__ void arrive_at(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void pair_load_2d(void* dst, const CUtensorMap* m, int c0, int c1, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
      "[%4];" ::"r"(smem_u32(dst)),
      "l"(m), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void pair_load_4d(void* dst, const CUtensorMap* m, int c0, int c1, int c2, int c3, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, "
      "%5}], [%6];" ::"r"(smem_u32(dst)),
      "l"(m), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
      : "memory");
}
template <bool F8>
__device__ __forceinline__ void pair_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  if (F8)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// arrives at the same barrier of both CTAs once all MMAs issued so far are done
__device__ __forceinline__ void pair_commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_u32(bar)),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}

struct PairShape {
  int tokens;      // of a tile: 64 .. 256, a multiple of 32
  int steps;       // of K
  int group;       // steps of a stage: 1 or 2
  int stages;      // of the ring
  int row_tiles, token_tiles;
};

// Which of the pair's tiles come is for the issuing warp alone to say, so that all of a tile is right or all of it is NaN: `ends`
// is the first that does not.  It is told to both CTAs.
__device__ __forceinline__ void tell_both(int* ends, int tile) {
#pragma unroll
  for (int r = 0; r < 2; ++r)
    asm volatile("st.relaxed.cluster.shared::cluster.u32 [%0], %1;" ::"r"(peer_address(smem_u32(ends), r)), "r"(tile) : "memory");
}
__device__ __forceinline__ int told(const int* ends) {
  int tile;
  asm volatile("ld.relaxed.cluster.shared::cta.u32 %0, [%1];" : "=r"(tile) : "r"(smem_u32(ends)) : "memory");
  return tile;
}
// Waits for the sums of a tile; false where the issuing warp has said that they do not come.  (That warp's own waits all end, the
// longest time being limit_ns; it is never reached.)
__device__ __forceinline__ bool sums_come(uint64_t* bar, uint32_t parity, const int* ends, int tile, unsigned long long limit_ns) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer();
  while (!mbar_try_wait(bar, parity))
    if (told(ends) <= tile || globaltimer() - t0 > limit_ns) return false;
  return true;
}
// A warp's part of a tile: 32 rows (this lane's is n), `columns` of the accumulator from t on, whose scales are at xs.  `free`
// is the barrier that gives the accumulator back, as soon as the last columns are in registers.  Of a tile that does not come
// (`ok` false, ws NaN) neither is touched: its accumulator may be that of an earlier one, which other warps still read.
template <typename OT, int ACT>
__device__ __forceinline__ void finish_part(const LinearArgs& a, uint32_t acc, const float* xs, int columns, int t, int n, float ws,
                                            float bias, uint32_t free, bool ok) {
#pragma unroll 1
  for (int c = 0; c < columns; c += kColumns) {
    uint32_t v[kColumns] = {};
    if (ok) {
      tmem_ld16(acc + c, v);
      if (c + kColumns >= columns) {
        tc_before();
        __syncwarp();
        if ((threadIdx.x & 31) == 0) arrive_at(free);
      }
    }
    if (t + c + kColumns <= a.tokens) finish_columns<OT, ACT, true>(a, v, xs + c, t + c, n, ws, bias);
    else if (t + c < a.tokens) finish_columns<OT, ACT, false>(a, v, xs + c, t + c, n, ws, bias);
  }
}
template <bool F8, typename OT, int ACT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    linear_pair_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x, const LinearArgs a,
                       const WeightPlace place, const PairShape sh) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  __shared__ __align__(8) uint64_t full[kPairStages], empty[kPairStages], accf[2], acce[2], drain;
  __shared__ __align__(16) float x_scales[kPairFinishers][kPairTokens / 4];
  __shared__ uint32_t tmem_slot;
  __shared__ int ends;  // the first of the pair's tiles whose sums do not come
  const int tid = threadIdx.x, warp = warp_index(), lane = tid & 31;
  const int rank = static_cast<int>(cta_rank());
  const int step_bytes = (kRows + sh.tokens / 2) * kStepBytes, stage = sh.group * step_bytes;  // multiples of 1024
  const int fills = (sh.steps + sh.group - 1) / sh.group;  // of a tile
  const int tiles = sh.row_tiles * sh.token_tiles, pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int mine = pair < tiles ? (tiles - 1 - pair) / pairs + 1 : 0;
  if (tid == 0) {
    prefetch_map(&map_w);
    prefetch_map(&map_x);
    for (int s = 0; s < sh.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&accf[b], 1);
      mbar_init(&acce[b], 2 * kPairFinishers);
    }
    mbar_init(&drain, 1);
    fence_mbar_init();
    ends = INT_MAX;
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&tmem_slot)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers are ready
  tc_after();
  const uint32_t tmem = tmem_slot;
  pdl_wait();  // what the call reads and writes may be the previous kernel's
  pdl_trigger();
  if (warp == 0 || warp == 2) {
    const int half = sh.tokens / 2;
    int s = 0, filled = 0;
    uint32_t ph = 0;  // how often the ring wrapped
    bool ok = true;
    for (int i = 0; i < mine && ok; ++i) {
      const int tile = pair + i * pairs, rt = tile / sh.token_tiles;
      const int n0 = rt * 2 * kRows + rank * kRows, t0 = (tile - rt * sh.token_tiles) * sh.tokens + rank * half;
      for (int f = 0, e = 0; f < fills; ++f) {
        if (ph > 0 && !warp_wait(&empty[s], (ph - 1) & 1u, a.limit_ns)) {
          ok = false;
          break;
        }
        const int count = min(sh.group, sh.steps - f * sh.group);
        if (elected()) {
          if (warp == 0 && rank == 0) mbar_arrive_expect_tx(&full[s], static_cast<uint32_t>(2 * count * step_bytes));  // of both CTAs
          uint8_t* st = smem + s * stage;
          const uint32_t bar = first_cta(&full[s]);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            if (q >= count) break;
            const int at = e + q * place.step;
            if (warp == 2) pair_load_2d(st + q * step_bytes + kRows * kStepBytes, &map_x, at, t0, bar);
            else if (place.packed) pair_load_4d(st + q * step_bytes, &map_w, at & 511, 0, at >> 9, n0 >> 1, bar);
            else pair_load_4d(st + q * step_bytes, &map_w, at, n0, 0, 0, bar);
          }
        }
        __syncwarp();
        e += sh.group * place.step;
        filled = min(filled + 1, sh.stages);
        if (++s == sh.stages) s = 0, ++ph;
      }
    }
    // Every stage that was filled has been multiplied: its copies have landed, and its release has come, before this CTA ends.
    // (After a wait that ran out these run out too, a second during which what is on its way lands.)
    for (int j = 0; j < filled; ++j) {
      s = s == 0 ? (--ph, sh.stages - 1) : s - 1;
      if (!mbar_wait(&empty[s], ph & 1u)) break;
    }
    if (!ok && lane == 0 && a.flags != nullptr) atomicOr(a.flags, a.bit);
    __syncwarp();
  } else if (warp == 1 && rank == 0) {
    const uint32_t idesc = (1u << 4) | (static_cast<uint32_t>(sh.tokens >> 3) << 17) | (16u << 24) |
                           (a.dtype == K2_BF16 ? (1u << 7) | (1u << 10) : 0u);
    const uint64_t ring = smem_desc(smem);
    int s = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int i = 0; i < mine && ok; ++i) {
      const int b = i & 1;
      if (i >= 2) ok = warp_wait(&acce[b], static_cast<uint32_t>((i >> 1) - 1) & 1u, a.limit_ns);
      tc_after();
      const uint32_t acc = tmem + b * kPairTokens;
      for (int f = 0; f < fills && ok; ++f) {
        if (!warp_wait(&full[s], ph & 1u, a.limit_ns)) {
          ok = false;
          break;
        }
        tc_after();
        const uint64_t ad = ring + static_cast<uint32_t>(s * (stage >> 4));
        const int count = min(sh.group, sh.steps - f * sh.group);
        if (elected()) {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            if (q >= count) break;
            const uint64_t at = ad + (q ? step_bytes >> 4 : 0);
#pragma unroll
            for (int j = 0; j < kStepBytes / 32; ++j)  // descriptors count 16 bytes
              pair_mma<F8>(acc, at + 2 * j, at + (kRows * kStepBytes >> 4) + 2 * j, idesc, (f | q | j) != 0);
          }
          pair_commit(&empty[s]);
          if (f == fills - 1) pair_commit(&accf[b]);
        }
        __syncwarp();
        if (++s == sh.stages) s = 0, ++ph;
      }
      if (!ok && lane == 0) tell_both(&ends, i);
    }
    if (elected())
      asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(&drain)) : "memory");
    __syncwarp();
    const bool drained = __all_sync(0xffffffffu, mbar_wait(&drain, 0));
    if (!drained && lane == 0) tell_both(&ends, 0);  // of the tiles whose MMAs were issued, those that have not come
    if ((!drained || !ok) && lane == 0 && a.flags != nullptr) atomicOr(a.flags, a.bit);
    __syncwarp();
  } else if (warp >= kPairOthers) {
    // 32 of the rows, and a quarter of the columns, in whole passes
    const int group = warp & 3, quarter = (warp - kPairOthers) >> 2, passes = sh.tokens / kColumns;
    const int c0 = (quarter * passes >> 2) * kColumns, columns = ((quarter + 1) * passes >> 2) * kColumns - c0;
    float* xs = x_scales[warp - kPairOthers];
    const unsigned long long longest = (fills + 2) * a.limit_ns + 2 * kWaitLimitNs;
    bool ok = true;
    for (int i = 0; i < mine; ++i) {
      const int b = i & 1, tile = pair + i * pairs, rt = tile / sh.token_tiles;
      const int n = rt * 2 * kRows + rank * kRows + group * 32 + lane, t = (tile - rt * sh.token_tiles) * sh.tokens + c0;
      __syncwarp();  // the last tile's scales have been read
      for (int c = lane; c < columns; c += 32) xs[c] = a.x_scale != nullptr && t + c < a.tokens ? __ldg(a.x_scale + t + c) : 1.f;
      __syncwarp();
      const float ws = a.w_scale != nullptr && n < a.rows ? __ldg(a.w_scale + n) : 1.f;
      const float bias = a.bias != nullptr && n < a.rows ? __ldg(a.bias + n) : 0.f;
      // from the first tile that does not come on, the rest of the pair's is NaN
      if (ok) ok = __all_sync(0xffffffffu, sums_come(&accf[b], static_cast<uint32_t>(i >> 1) & 1u, &ends, i, longest));
      tc_after();
      const uint32_t acc = tmem + b * kPairTokens + c0 + (static_cast<uint32_t>(group * 32) << 16), free = first_cta(&acce[b]);
      finish_part<OT, ACT>(a, acc, xs, columns, t, n, ok ? ws : __uint_as_float(0x7FC00000u), bias, free, ok);
    }
    if (!ok && lane == 0 && a.flags != nullptr) atomicOr(a.flags, a.bit);
  }
  tc_before();
  __syncthreads();
  cluster_sync();  // both CTAs' roles have ended
  tc_after();
  if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiled encode_fn() {
  static std::atomic<EncodeTiled> fn{nullptr};
  EncodeTiled f = fn.load(std::memory_order_acquire);
  if (!f) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn.store(f = reinterpret_cast<EncodeTiled>(p), std::memory_order_release);
  }
  return f;
}
bool encode(CUtensorMap* m, int dtype, int rank, const void* base, const cuuint64_t* dims, const cuuint64_t* strides,
            const cuuint32_t* box) {
  const EncodeTiled f = encode_fn();
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return f && f(m, dtype == K2_F8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank,
                const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// K-major rows of the tokens (a bf16 map copies fp16 as well: it moves bytes)
bool encode_tokens(CUtensorMap* m, int dtype, const void* x, long long stride, int cols, int tokens, int box_tokens) {
  const int b = dtype == K2_F8 ? 1 : 2;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(tokens)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(stride) * b};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(kStepBytes / b), static_cast<cuuint32_t>(box_tokens)};
  return encode(m, dtype, 2, x, dims, strides, box);
}
bool encode_weights(CUtensorMap* m, int dtype, const LinearWeights& w, int rows, int cols) {
  const int b = dtype == K2_F8 ? 1 : 2;
  if (w.packed) {
    const cuuint64_t chunks = (static_cast<cuuint64_t>(cols) + 511) / 512;
    const cuuint64_t dims[4] = {512, 2, chunks, static_cast<cuuint64_t>(rows + 1) / 2};
    const cuuint64_t strides[3] = {512, 1024, 1024 * chunks};
    const cuuint32_t box[4] = {kStepBytes, 2, 1, kRows / 2};
    return encode(m, dtype, 4, w.base, dims, strides, box);
  }
  const cuuint64_t step = static_cast<cuuint64_t>(w.stride) * b;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), 1, 1};
  const cuuint64_t strides[3] = {step, step, step};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(kStepBytes / b), kRows, 1, 1};
  return encode(m, dtype, 4, w.base, dims, strides, box);
}

// launched as a dependent of the kernel before it: the start overlaps that kernel's end, then waits for all of it
cudaLaunchAttribute early_start() {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  return attr;
}

template <bool F8, typename OT, int ACT>
cudaError_t launch(const CUtensorMap& mw, const CUtensorMap& mx, const LinearArgs& a, const WeightPlace& place,
                   const FewShape& sh, int, int dev, cudaStream_t s) {
  auto kernel = linear_few_kernel<F8, OT, ACT>;
  static std::atomic<uint64_t> ready{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), kFewRing + few_part(kFewTokens, kMaxSplit) + 1024, dev, ready);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((a.rows + kRows - 1) / kRows * sh.split, (a.tokens + sh.tokens - 1) / sh.tokens);
  cfg.blockDim = dim3(128);
  cfg.dynamicSmemBytes = sh.stages * few_stage(sh.tokens) + few_part(sh.tokens, sh.split) + 1024;
  cfg.stream = s;
  cudaLaunchAttribute attr[2] = {early_start(), {}};
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = sh.split;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = sh.split > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, mw, mx, a, place, sh);
}
template <bool F8, typename OT, int ACT>
cudaError_t launch(const CUtensorMap& mw, const CUtensorMap& mx, const LinearArgs& a, const WeightPlace& place,
                   const PairShape& sh, int sms, int dev, cudaStream_t s) {
  auto kernel = linear_pair_kernel<F8, OT, ACT>;
  static std::atomic<uint64_t> ready{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), kPairSmem, dev, ready);
  if (e != cudaSuccess) return e;
  const int pairs = std::min(sms / 2, sh.row_tiles * sh.token_tiles);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * pairs);
  cfg.blockDim = dim3(kPairThreads);
  cfg.dynamicSmemBytes = kPairSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1] = {early_start()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, mw, mx, a, place, sh);
}
template <bool F8, typename OT, typename Shape>
cudaError_t launch(const CUtensorMap& mw, const CUtensorMap& mx, const LinearArgs& a, const WeightPlace& place, const Shape& sh,
                   int sms, int dev, cudaStream_t s) {
  return a.act == K2_ACT_SWIGLU ? launch<F8, OT, kPairsOfRows>(mw, mx, a, place, sh, sms, dev, s)
         : a.act == K2_ACT_NONE ? launch<F8, OT, kPlain>(mw, mx, a, place, sh, sms, dev, s)
                                : launch<F8, OT, kOther>(mw, mx, a, place, sh, sms, dev, s);
}
template <bool F8, typename Shape>
cudaError_t launch(const CUtensorMap& mw, const CUtensorMap& mx, const LinearArgs& a, const WeightPlace& place, const Shape& sh,
                   int sms, int dev, cudaStream_t s) {
  return a.out_dtype == K2_F32    ? launch<F8, float>(mw, mx, a, place, sh, sms, dev, s)
         : a.out_dtype == K2_BF16 ? launch<F8, __nv_bfloat16>(mw, mx, a, place, sh, sms, dev, s)
                                  : launch<F8, __half>(mw, mx, a, place, sh, sms, dev, s);
}
// tensor maps for tiles of box_tokens, and the kernel of the shape
template <typename Shape>
k2_status launch(const LinearWeights& w, const void* x, long long x_stride, const LinearArgs& a, const WeightPlace& place,
                 const Shape& sh, int box_tokens, int sms, int dev, cudaStream_t s) {
  CUtensorMap mw, mx;
  if (!encode_weights(&mw, a.dtype, w, a.rows, a.cols) || !encode_tokens(&mx, a.dtype, x, x_stride, a.cols, a.tokens, box_tokens)) {
    set_error("no tensor map for %d x %d weights and %d tokens", a.rows, a.cols, a.tokens);
    return K2_ERR_CUDA;
  }
  const cudaError_t e = a.dtype == K2_F8 ? launch<true>(mw, mx, a, place, sh, sms, dev, s)
                                         : launch<false>(mw, mx, a, place, sh, sms, dev, s);
  if (e == cudaSuccess) return K2_OK;
  set_error("linear launch: %s", cudaGetErrorString(e));
  return K2_ERR_CUDA;
}

}  // namespace

k2_status launch_linear(const LinearWeights& w, const void* x, long long x_stride, const LinearArgs& a, cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && (dev < 0 || dev >= 64)) e = cudaErrorInvalidDevice;
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) {
    set_error("linear: %s", cudaGetErrorString(e));
    return K2_ERR_CUDA;
  }
  const WeightPlace place = {w.packed ? 1 : 0, a.dtype == K2_F8 ? kStepBytes : kStepBytes / 2};
  const int steps = (a.cols + place.step - 1) / place.step;
  // Few tokens per tile and K split over CTAs, or wide tiles on pairs of SMs: the cheaper by what was measured, in nanoseconds.
  // Few: a K step takes 270, or 165 for each CTA of the SM where that is more; 2600 for the rest, again for every three
  // CTAs that an SM gets (300 tokens of 640 by 20480 in bf16: 17.4 us, pairs 12.9; 2000 by 1664 in E4M3, three each: 6.3 and 7.0),
  // 2200 more to join shares of K, and 2000 where those are more CTAs than SMs.  Pairs: a step takes kStepNs for 64, 96 .. 256 tokens a tile;
  // 3000 for the rest and 8 per column of the last tile.  (Down of 2048 tokens: two waves of 130 tiles of 160, 38 us; of 110 of
  // 192 tokens 43; of 80 of 256, 51.)  Neither is done before the weights have been read (6800 bytes a ns, 5400
  // as the few read them).  The costs serve to choose by: of more than 64 tokens they are up to a third below what the kernels
  // take, outputs and residuals not being counted, in both kernels alike (12.5 for the few and 14.7 measured, gate and up of 128
  // tokens; 23 for pairs and 28, q|k|v of 2048).  The choice was compared at (us, few and pairs): down of 128 tokens 14.3 and 16.6, of 256
  // 15.6 and 15.7, of 512 28.6 and 18.6; gate and up of 128 15.0 and 16.3, of 256 24.2 and 18.4; q|k|v of 128 9.8 and 7.0.
  // Activations take the few's four finishing warps longer.  Up to 64 tokens it is always the few (gate and up of 64 tokens 14.4
  // us against 16.5).
  FewShape few = {a.tokens <= 16 ? 16 : a.tokens <= 32 ? 32 : 64, steps, 0, 1};
  const long long few_tiles = static_cast<long long>((a.rows + kRows - 1) / kRows) * ((a.tokens + few.tokens - 1) / few.tokens);
  const long long bytes = static_cast<long long>(a.rows) * a.cols * (a.dtype == K2_F8 ? 1 : 2);
  long long few_cost = 0;
  for (int per_sm = 1; per_sm <= (a.tokens > 64 ? 2 : 1); ++per_sm) {
    int split = static_cast<int>(std::max<long long>(1, std::min<long long>({per_sm * sms / few_tiles, kMaxSplit, steps})));
    // SMs come in twos.  With clusters of six and of seven, 20 and 21 tiles (the numbers that seven would be taken for), us: 64 tokens
    // by 10240 9.1 .. 9.3 and 9.7 .. 9.9, by 4096 5.4 and 6.5, one by 4096 4.2 and 4.6 .. 4.8; by 640 (five steps) the same.
    if (split == 7) split = 6;
    const long long mine = (steps + split - 1) / split, ctas = few_tiles * split, load = (ctas + sms - 1) / sms;
    const long long cost = 2600 * ((load + 2) / 3) + std::max(mine * std::max(270ll, 165 * load), bytes / 5400) +
                           (split == 1 ? 0 : ctas <= sms ? 2200 : 4200);
    if (few_cost == 0 || cost < few_cost) few.split = split, few_cost = cost;
  }
  if (a.act != K2_ACT_NONE && a.act != K2_ACT_SWIGLU) few_cost += 60ll * few.tokens;
  if (a.tokens > 64) {
    constexpr int kStepNs[] = {140, 170, 175, 220, 250, 270, 305};
    PairShape sh = {0, steps, 1, 0, (a.rows + 2 * kRows - 1) / (2 * kRows), 0};
    long long best = 0;
    for (int n = kPairTokens; n >= 64; n -= 32) {
      const int tt = (a.tokens + n - 1) / n;
      const long long wave = static_cast<long long>(steps) * kStepNs[n / 32 - 2];
      const long long waves = (static_cast<long long>(sh.row_tiles) * tt + sms / 2 - 1) / (sms / 2);
      const long long cost = waves * wave + 3000 + 8 * n + std::max(0ll, bytes / 6800 - wave);
      if (sh.tokens == 0 || cost < best) sh.tokens = n, sh.token_tiles = tt, best = cost;
    }
    // a stage of one step costs 230 ns whatever the tile, so that narrow tiles' have two (down of 2048 tokens by tiles of 160: 38
    // and 43 us); of wider tiles only three such stages would fit (tiles of 160 with three: 46)
    sh.group = sh.tokens <= 160 ? 2 : 1;
    sh.stages = std::min(kPairStages, kPairRing / (sh.group * (kRows + sh.tokens / 2) * kStepBytes));
    if (best <= few_cost || a.tokens > 65535 * few.tokens) return launch(w, x, x_stride, a, place, sh, sh.tokens / 2, sms, dev, s);
  }
  few.stages = std::min({kFewStages, kFewRing / few_stage(few.tokens), (steps + few.split - 1) / few.split});
  return launch(w, x, x_stride, a, place, few, few.tokens, sms, dev, s);
}

}  // namespace k2

using namespace k2;

extern "C" {

k2_status k2_linear(const k2_linear_args* p, void* stream) {
  if (!p) {
    set_error("the arguments must be non-null");
    return K2_ERR_ARG;
  }
  const bool f8 = p->dtype == K2_F8;
  if (!f8 && p->dtype != K2_BF16 && p->dtype != K2_F16) {
    set_error("weights and tokens must be K2_F8, K2_BF16 or K2_F16 (got dtype %d)", p->dtype);
    return K2_ERR_UNSUPPORTED;
  }
  if (p->out_dtype != K2_F32 && p->out_dtype != K2_BF16 && p->out_dtype != K2_F16) {
    set_error("the output must be K2_F32, K2_BF16 or K2_F16 (got dtype %d)", p->out_dtype);
    return K2_ERR_UNSUPPORTED;
  }
  if (p->activation < K2_ACT_NONE || p->activation > K2_ACT_SWIGLU) {
    set_error("activation must be one of K2_ACT_* (got %d)", p->activation);
    return K2_ERR_ARG;
  }
  if (p->tokens < 0 || p->tokens > 1 << 22 || p->out_features < 1 || p->out_features > 1 << 24 || p->in_features < 1 ||
      p->in_features > 1 << 24) {
    set_error("tokens in [0, 2^22], features in [1, 2^24] (got %d, %d and %d)", p->tokens, p->out_features, p->in_features);
    return K2_ERR_SHAPE;
  }
  const bool pairs = p->activation == K2_ACT_SWIGLU;
  if (pairs && p->out_features % 2) {
    set_error("K2_ACT_SWIGLU needs an even number of out_features (got %d)", p->out_features);
    return K2_ERR_SHAPE;
  }
  if (p->wait_limit_us < 0 || p->wait_limit_us > 1000000) {
    set_error("wait_limit_us must be in [0, 1000000] (got %d)", p->wait_limit_us);
    return K2_ERR_ARG;
  }
  if (p->tokens == 0) return K2_OK;
  if (!p->w || !p->x || !p->out || f8 != (p->w_scale != nullptr) || f8 != (p->x_scale != nullptr)) {
    set_error("w, x and out must be non-null, and w_scale and x_scale for K2_F8 alone");
    return K2_ERR_ARG;
  }
  const int b = f8 ? 1 : 2, ob = p->out_dtype == K2_F32 ? 4 : 2;
  const int64_t width = pairs ? p->out_features / 2 : p->out_features, most = 1ll << 36;
  const int64_t ws = p->out_features > 1 ? p->w_stride : (p->in_features + 15) / 16 * 16;
  const int64_t xs = p->tokens > 1 ? p->x_stride : (p->in_features + 15) / 16 * 16;
  const int64_t os = p->tokens > 1 ? p->out_stride : width, rs = p->tokens > 1 ? p->residual_stride : width;
  if (ws < p->in_features || xs < p->in_features || os < width || (p->residual && rs < width) || ws > most || xs > most ||
      os > most || (p->residual && rs > most)) {
    set_error("rows must be at least as far apart as they are long, and at most 2^36 elements (got w %lld, x %lld, out %lld)",
              static_cast<long long>(ws), static_cast<long long>(xs), static_cast<long long>(os));
    return K2_ERR_ARG;
  }
  if (!aligned16(p->w) || !aligned16(p->x) || ws * b % 16 || xs * b % 16) {
    set_error("rows of w and x must be 16-byte aligned");
    return K2_ERR_ARG;
  }
  for (const void* q : {static_cast<const void*>(p->w_scale), static_cast<const void*>(p->x_scale), static_cast<const void*>(p->bias),
                        static_cast<const void*>(p->flags)})
    if (reinterpret_cast<uintptr_t>(q) % 4) {
      set_error("scales, bias and flags must be 4-byte aligned");
      return K2_ERR_ARG;
    }
  if (reinterpret_cast<uintptr_t>(p->out) % ob || reinterpret_cast<uintptr_t>(p->residual) % ob) {
    set_error("out and residual must be aligned to their type");
    return K2_ERR_ARG;
  }
  const RowSet out = {p->out, ob * os, ob * width, p->tokens}, res = {p->residual, ob * rs, ob * width, p->tokens},
               w = {p->w, b * ws, static_cast<int64_t>(b) * p->in_features, p->out_features},
               x = {p->x, b * xs, static_cast<int64_t>(b) * p->in_features, p->tokens},
               wsc = {p->w_scale, 4, 4, p->out_features}, xsc = {p->x_scale, 4, 4, p->tokens}, bias = {p->bias, 4, 4, p->out_features};
  const bool same = p->residual == p->out && os == rs;
  if (sets_meet(out, w) || sets_meet(out, x) || sets_meet(out, wsc) || sets_meet(out, xsc) || sets_meet(out, bias) ||
      (!same && sets_meet(out, res))) {
    set_error("the output may not lie over an input (but over the residual itself, with its stride)");
    return K2_ERR_ARG;
  }
  const LinearArgs a = {p->w_scale, p->x_scale, p->bias, p->residual, rs, p->out, os, p->tokens, p->out_features, p->in_features,
                        p->dtype, p->out_dtype, p->activation, p->flags, K2_LINEAR_TIMEOUT,
                        p->wait_limit_us ? 1000ull * p->wait_limit_us : kWaitLimitNs};
  return launch_linear({p->w, ws, false}, p->x, xs, a, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
