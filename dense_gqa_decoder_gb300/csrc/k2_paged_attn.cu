// Causal attention of many requests' newest tokens over a block-paged 8-bit
// cache (k2_paged_attention; the formula is stated in include/k2.h).
#include <math.h>

#include <algorithm>

#include "k2_paged.cuh"

namespace k2 {

namespace {

__device__ __forceinline__ uint32_t movmatrix(uint32_t a) {  // transpose of an 8 x 8 fp16 matrix held by the warp
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}

// ---- few query rows per request: decode and speculative steps -------------------------------
//
// Memory bound: every code is read once, for rep * queries rows (2 flop per code
// and row).  The tensor cores take the rows of a KV head together: with the rows
// as the narrow side of mma.m16n8k16, S^T = K Q^T and O^T = V^T P^T need one MMA
// each per 16 keys, 16 dims and 8 rows, and the codes, widened to fp16 in
// registers, are the wide operand.  Dims may be permuted inside a dot product, so
// a lane's codes of a K row are 32 (head_dim 64: 16) neighbouring bytes; a lane's
// dims of V are neighbours too, and pairs of keys are interleaved by byte
// permutes.  S^T's accumulators become P^T's operand by one 8 x 8 transpose each.
//
// Work is cut into tiles of 32 keys of one (request, KV head); the CTAs take
// equal shares of all tiles of the step, whatever the lengths, which they find
// from the lengths themselves (a prefix sum of the requests' tiles, each item
// counted with kDecStart more for what its start and end cost).  In a CTA
// the warps take the tiles of a share in turn, each through a ring of its own
// that cp.async fills ahead (no barrier inside a share).  A share that holds only
// a part of a (request, head) leaves (maximum, sum, output) in the workspace, and
// the CTA that arrives last joins the parts, in order.
//
// Query rows are scaled by a power of two to fp16's upper range (exact for bf16
// and fp16 inputs); probabilities p enter P.V as fp16(p * (vs / vref) * 2^14), vs
// the block's V scale and vref the power of two below the largest so far (2^-126 at
// least), so that no block's scale costs precision while the ratio stays above 2^-28.
// One fp16 number each, for one MMA each: its 2^-11 is the rounding of an fp16 output and an eighth of a bf16 one's (fp16
// outputs end up 1.1 to 1.4 times as far from the exact ones as with fp32 probabilities, bf16 outputs as far).
// vref, 1 / vref and 2^14 are exact normal factors, applied one after another: 2^14 / vref
// itself may not be finite.
//
// 16 requests of 8192 tokens, 32 heads of 128 over 8: 51 us, 5.3 TB/s (78 % of a copy's rate) from int8 codes; 48 requests
// of 1 .. 32768 in E4M3: 60 us, 5.7 TB/s.  What is left is each CTA's start (lengths, table, first tiles) and the join.
constexpr int kDecWarps = 4, kDecThreads = 32 * kDecWarps;
constexpr int kDecKeys = 32;   // of a tile: two halves of 16, which may lie in two blocks
constexpr int kDecStart = 10;  // an item's start and end in tiles (48 requests of 1 .. 32768 tokens: 62 us, 82 with 4)
constexpr int kDecShare = 4;   // smallest share (one request of 1000 tokens: 9.0 us, 10.6 with 8, 12.1 with 16)
constexpr int kDecMaxRows = 16;

template <int D, int NT>
struct Dec {
  static constexpr int kRows = 8 * NT;
  static constexpr int kHalf = 16 * D;                           // K (or V) codes of half a tile
  static constexpr int kStage = 4 * kHalf;                       // K half 0, K half 1, V half 0, V half 1
  static constexpr int kStages = D == 128 ? 2 : 4;
  static constexpr int kRing = kStage * kStages;                 // per warp
  static constexpr int kLd = D + 4;                              // floats of a row of the joined output
  static constexpr int kMerge = kDecWarps * kRows * (kLd + 2) * 4;
  static constexpr int kSmem = kRing * kDecWarps > kMerge ? kRing * kDecWarps : kMerge;
  static constexpr int kCtas = 3;                                // per SM
};
constexpr int kDecSlotFloats = kDecMaxRows * (128 + 2);  // one part: rows x (output, maximum, sum)

// byte offset of 16-byte chunk c of row r in a tile of D-byte rows, swizzled so
// that the fragment reads below are free of bank conflicts
template <int D>
__device__ __forceinline__ int tile_at(int r, int c) {
  if constexpr (D == 128) return r * 128 + ((c ^ (r & 7)) << 4);
  else return (r >> 1) * 128 + (((((r & 1) << 2) | c) ^ ((r & 6))) << 4);
}

template <typename T, typename C, int D, int NT>
__global__ void __launch_bounds__(kDecThreads, Dec<D, NT>::kCtas)
    paged_decode_kernel(const PagedPool p, const PagedAttnArgs a, int small_rows, unsigned* counters, float* parts) {
  using S = Dec<D, NT>;
  using W = Widen<C>;
  constexpr int KS = D / 16;        // k-steps of S^T
  constexpr int MT = D / 16;        // m-tiles of O^T
  constexpr int QW = D / 4;         // dims of a lane's query row
  constexpr int VB = D / 8;         // dims of a lane's V rows
  constexpr int NS = S::kStages;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ long long s_sum[kDecWarps];
  __shared__ long long s_base;
  __shared__ int s_req, s_last;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gq = lane >> 2, t = lane & 3;
  const int rep = a.n_heads / p.n_kv;
  pdl_trigger();  // a CTA of the kernel for prompt chunks may start on every SM that these CTAs have left

  // the tiles of every request, and this CTA's share of them
  auto tiles_of = [&](const Req& x) -> int {
    return x.ok && x.nq > 0 && static_cast<long long>(x.nq) * rep <= small_rows ? (x.len + kDecKeys - 1) / kDecKeys : 0;
  };
  auto units_of = [&](int tiles) -> long long { return tiles ? static_cast<long long>(tiles + kDecStart) * p.n_kv : 0; };
  const int per = (a.requests + kDecThreads - 1) / kDecThreads;
  long long own = 0;
  bool faulty = false;
  for (int i = 0; i < per; ++i) {
    const int r = tid * per + i;
    if (r < a.requests) {
      const Req x = request(a, p.block_log2, r);
      faulty |= !x.ok;
      own += units_of(tiles_of(x));
    }
  }
  long long inc = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  if (lane == 31) s_sum[warp] = inc;
  faulty = __syncthreads_or(faulty) != 0;
  long long total = 0, before = inc - own;
#pragma unroll
  for (int w = 0; w < kDecWarps; ++w) {
    if (w < warp) before += s_sum[w];
    total += s_sum[w];
  }
  if (faulty) {  // requests whose lengths contradict each other: zeros in their rows
    for (int r = blockIdx.x; r < a.requests; r += gridDim.x) {
      if (request(a, p.block_log2, r).ok) continue;
      if (tid == 0) raise_flag(p.flags, K2_PAGED_BAD_LENGTH);
      const int lo = max(a.cu_q[r], 0), hi = min(a.cu_q[r + 1], a.tokens), w = a.n_heads * D / 4;
      for (long long i = tid; i < static_cast<long long>(hi - lo) * w; i += kDecThreads)
        store4(static_cast<T*>(a.out) + (lo + i / w) * a.out_stride + 4 * (i % w), 0.f, 0.f, 0.f, 0.f);
    }
  }
  if (total == 0) return;
  const int ctas = static_cast<int>(min(static_cast<long long>(gridDim.x), (total + kDecShare - 1) / kDecShare));
  if (blockIdx.x >= ctas) return;
  const Share share(total, ctas);
  const long long x0 = share.first(blockIdx.x), x1 = share.first(blockIdx.x + 1);
  if (before <= x0 && x0 < before + own) {  // one thread: its requests hold the share's first unit
    long long at = before;
    for (int i = 0; i < per; ++i) {
      const int r = tid * per + i;
      if (r >= a.requests) break;
      const long long n = units_of(tiles_of(request(a, p.block_log2, r)));
      if (x0 < at + n) {
        s_req = r;
        s_base = at;
        break;
      }
      at += n;
    }
  }
  __syncthreads();
  int r = s_req;
  long long base = s_base;  // flat index of request r's first unit

  const uint32_t ring_u = smem_u32(smem + warp * S::kRing);
  float* mo = reinterpret_cast<float*>(smem);                 // joined: [warp][row][kLd] outputs
  float* mml = mo + kDecWarps * S::kRows * S::kLd;            // [warp][row] (maximum, sum)

  // where this lane's 16-byte chunks of half a tile go: chunk c0 + lane of 16 D / 16 (the rows lie one after another)
  constexpr int CP = D / 32;  // chunks per lane
  uint32_t put_at[CP];
  int row_of[CP];
#pragma unroll
  for (int c = 0; c < CP; ++c) {
    row_of[c] = (32 * c + lane) / (D / 16);
    put_at[c] = ring_u + tile_at<D>(row_of[c], (32 * c + lane) % (D / 16));
  }
  const uint8_t* src_k = p.k + 16 * lane;
  const uint8_t* src_v = p.v + 16 * lane;

  for (long long x = x0; x < x1;) {
    Req q = request(a, p.block_log2, r);
    int nt = tiles_of(q);
    while (x >= base + units_of(nt)) {
      base += units_of(nt);
      q = request(a, p.block_log2, ++r);
      nt = tiles_of(q);
    }
    const int g = static_cast<int>(quotient(x - base, nt + kDecStart));
    const long long item = base + static_cast<long long>(g) * (nt + kDecStart) + kDecStart;  // unit of (r, g)'s first tile
    const int ta = static_cast<int>(max(x0 - item, 0ll)), tb = static_cast<int>(min(static_cast<long long>(nt), x1 - item));
    x = item + nt;
    if (ta >= tb) continue;
    const int rows = q.nq * rep;
    const int* table = a.table + static_cast<size_t>(r) * a.table_stride;

    // this warp's tiles: ta + warp + kDecWarps i, i < n; lane l holds half l of 16 tiles: its place in the pool in
    // units of 16 rows (~0: no such block) and its scales
    const int n = tb - ta > warp ? (tb - ta - warp + kDecWarps - 1) / kDecWarps : 0;
    const int first = ta + warp;
    unsigned at = ~0u, at_next = ~0u;
    float ks = 0.f, vs = 0.f, ks_next = 0.f, vs_next = 0.f;
    auto fetch = [&](int c, unsigned& d, float& k_s, float& v_s) {
      const int i = 16 * c + (lane >> 1), key0 = (first + kDecWarps * i) * kDecKeys + 16 * (lane & 1);
      d = ~0u;
      k_s = v_s = 0.f;
      if (i < n && key0 < q.len) {
        const int id = __ldg(table + (key0 >> p.block_log2));
        if (id < 0 || id >= p.n_blocks) {
          raise_flag(p.flags, K2_PAGED_BAD_BLOCK);
        } else {
          const unsigned b = static_cast<unsigned>(id) * p.n_kv + g;
          d = (b << (p.block_log2 - 4)) + ((key0 & ((1 << p.block_log2) - 1)) >> 4);
          k_s = __ldg(p.ks + b);
          v_s = __ldg(p.vs + b);
        }
      }
    };
    fetch(0, at, ks, vs);
    if (n > 16) fetch(1, at_next, ks_next, vs_next);
    auto issue = [&](int i, int stage, int cur) {  // requests tile i into a stage; cur: the batch that `at` holds
      if (i < n) {
        const bool next = (i >> 4) != cur;
        const int key0 = (first + kDecWarps * i) * kDecKeys;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const unsigned d = __shfl_sync(0xffffffffu, next ? at_next : at, (2 * i + h) & 31);
          const int left = d == ~0u ? 0 : q.len - key0 - 16 * h;  // rows of this half (the others become zeros)
          const size_t off = d == ~0u ? 0 : static_cast<size_t>(d) * S::kHalf;
          const uint8_t* kp = src_k + off;
          const uint8_t* vp = src_v + off;
          const uint32_t st = stage * S::kStage + h * S::kHalf;
          if (left >= 16) {
#pragma unroll
            for (int c = 0; c < CP; ++c) {
              cp_async16_to(put_at[c] + st, kp + 512 * c);
              cp_async16_to(put_at[c] + st + 2 * S::kHalf, vp + 512 * c);
            }
          } else {
#pragma unroll
            for (int c = 0; c < CP; ++c) {
              const bool take = row_of[c] < left;
              cp_async16_zfill(put_at[c] + st, take ? kp + 512 * c : p.k, take);
              cp_async16_zfill(put_at[c] + st + 2 * S::kHalf, take ? vp + 512 * c : p.v, take);
            }
          }
        }
      }
      cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < NS - 1; ++i) issue(i, i, 0);

    // query rows as the narrow operand: n-tile j holds rows 8j + gq, this lane their dims QW t ..
    uint32_t qf[NT][KS][2];
    float f0[NT], f1[NT];  // what turns an accumulator of rows 8j + 2t, + 1 into base-2 scores (times the K scale)
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int row = 8 * j + gq;
      float v[QW], top = 0.f;
      if (row < rows) {
        const int i = row / rep, h = row - i * rep;
        const T* src = static_cast<const T*>(a.q) + (q.q0 + i) * a.q_stride + (g * rep + h) * D + QW * t;
#pragma unroll
        for (int e = 0; e < QW; e += 8) load8(src + e, v + e);
      } else {
#pragma unroll
        for (int e = 0; e < QW; ++e) v[e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < QW; ++e) top = fmaxf(top, fabsf(v[e]));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // 2^up brings the largest magnitude into [2^14, 2^15)
      const int ex = static_cast<int>(__float_as_uint(top) >> 23);
      const int up = top > 0.f && ex < 255 ? 14 + 127 - ex : 0;
      const int ua = up / 2, ub = up - ua;  // in two steps: 2^up itself may not be a normal number
      const float sa = __uint_as_float((127 + ua) << 23), sb = __uint_as_float((127 + ub) << 23);
#pragma unroll
      for (int kk = 0; kk < KS; ++kk) {
        qf[j][kk][0] = pack_half2(v[4 * kk] * sa * sb, v[4 * kk + 1] * sa * sb);
        qf[j][kk][1] = pack_half2(v[4 * kk + 2] * sa * sb, v[4 * kk + 3] * sa * sb);
      }
      const float ia = __uint_as_float((127 - ua) << 23), ib = __uint_as_float((127 - ub) << 23);
      const float back = a.scale * kLog2e * ia * ib;
      f0[j] = __shfl_sync(0xffffffffu, back, 8 * t);
      f1[j] = __shfl_sync(0xffffffffu, back, 8 * t + 4);
    }

    float o[NT][MT][4], m0[NT], m1[NT], l0[NT], l1[NT], vref = 0.f, vinv = 0.f;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      m0[j] = m1[j] = -INFINITY;
      l0[j] = l1[j] = 0.f;
#pragma unroll
      for (int e = 0; e < MT; ++e) o[j][e][0] = o[j][e][1] = o[j][e][2] = o[j][e][3] = 0.f;
    }

    int stage = 0, ahead = NS - 1;  // of tile i, of tile i + NS - 1
    for (int i = 0; i < n; ++i) {
      const int cur = i >> 4;
      if (i > 0 && (i & 15) == 0) {
        at = at_next;
        ks = ks_next;
        vs = vs_next;
        if (16 * (cur + 1) < n) fetch(cur + 1, at_next, ks_next, vs_next);
      }
      cp_async_wait<NS - 2>();
      __syncwarp();  // everyone's copies of tile i have landed, and everyone is done with tile i - 1
      issue(i + NS - 1, ahead, cur);
      const uint32_t kt = ring_u + stage * S::kStage, vt = kt + 2 * S::kHalf;
      ahead = ahead + 1 == NS ? 0 : ahead + 1;
      stage = stage + 1 == NS ? 0 : stage + 1;
      float k_s[2], v_s[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        k_s[h] = __shfl_sync(0xffffffffu, ks, (2 * i + h) & 31);
        v_s[h] = __shfl_sync(0xffffffffu, vs, (2 * i + h) & 31);
      }
      // S^T: keys gq and gq + 8 of each half, this lane's QW dims of each
      float sc[NT][8];
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) sc[j][e] = 0.f;
#pragma unroll
      for (int c = 0; c < QW / 16; ++c) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint4 ka = lds128(kt + h * S::kHalf + tile_at<D>(gq, (QW / 16) * t + c));
          const uint4 kb = lds128(kt + h * S::kHalf + tile_at<D>(gq + 8, (QW / 16) * t + c));
          const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const uint32_t xa = W::prep(wa[w]), xb = W::prep(wb[w]);
            const uint32_t af[4] = {W::template pair<false>(xa), W::template pair<false>(xb), W::template pair<true>(xa),
                                    W::template pair<true>(xb)};
#pragma unroll
            for (int j = 0; j < NT; ++j) mma16816(sc[j] + 4 * h, af, qf[j][4 * c + w][0], qf[j][4 * c + w][1]);
          }
        }
      }
      // V: the reference scale, and what each half's probabilities are multiplied with
      const float av = fmaxf(fabsf(v_s[0]), fabsf(v_s[1]));
      float shrink = 1.f;
      if (av >= 2.f * vref && av > 0.f) {
        const float now = __uint_as_float(max(__float_as_uint(av) & 0x7f800000u, 0x00800000u));
        vinv = __frcp_rn(now);
        shrink = vref * vinv;
        vref = now;
      }
      const int key = (first + kDecWarps * i) * kDecKeys;
      // some row does not see all of the tile, or a half is missing
      const bool edge = key + kDecKeys > q.len - q.nq + 1 || __shfl_sync(0xffffffffu, at, (2 * i) & 31) == ~0u ||
                        __shfl_sync(0xffffffffu, at, (2 * i + 1) & 31) == ~0u;
      uint32_t pf[NT][4];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        float s[8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float fa = f0[j] * k_s[h], fb = f1[j] * k_s[h];
#pragma unroll
          for (int e = 0; e < 4; ++e) s[4 * h + e] = sc[j][4 * h + e] * (e & 1 ? fb : fa);
        }
        if (edge) {
          const int ra = 8 * j + 2 * t, seen = q.len - q.nq;  // a row's last key: seen + row / rep
          const int la = seen + ra / rep - key, lb = seen + (ra + 1) / rep - key;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const bool off = __shfl_sync(0xffffffffu, at, (2 * i + h) & 31) == ~0u;
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (off || 16 * h + gq + (e & 2) * 4 > (e & 1 ? lb : la)) s[4 * h + e] = -INFINITY;
          }
        }
        float ma = fmaxf(fmaxf(s[0], s[2]), fmaxf(s[4], s[6])), mb = fmaxf(fmaxf(s[1], s[3]), fmaxf(s[5], s[7]));
#pragma unroll
        for (int sh = 4; sh < 32; sh <<= 1) {
          ma = fmaxf(ma, __shfl_xor_sync(0xffffffffu, ma, sh));
          mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, sh));
        }
        if (__any_sync(0xffffffffu, ma > m0[j] || mb > m1[j]) || shrink != 1.f) {
          const float na = fmaxf(m0[j], ma), nb = fmaxf(m1[j], mb);
          const float ca = na == -INFINITY ? 1.f : exp2_approx(m0[j] - na), cb = nb == -INFINITY ? 1.f : exp2_approx(m1[j] - nb);
          l0[j] *= ca;
          l1[j] *= cb;
#pragma unroll
          for (int e = 0; e < MT; ++e) {
            o[j][e][0] *= ca * shrink;
            o[j][e][1] *= cb * shrink;
            o[j][e][2] *= ca * shrink;
            o[j][e][3] *= cb * shrink;
          }
          m0[j] = na;
          m1[j] = nb;
        }
        const float za = m0[j] == -INFINITY ? 0.f : m0[j], zb = m1[j] == -INFINITY ? 0.f : m1[j];  // no key seen yet: every p is 0
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] = exp2_approx(s[e] - (e & 1 ? zb : za));
        l0[j] += (s[0] + s[2]) + (s[4] + s[6]);
        l1[j] += (s[1] + s[3]) + (s[5] + s[7]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float pv = v_s[h] * vinv * 16384.f;
          pf[j][2 * h] = movmatrix(pack_half2(s[4 * h] * pv, s[4 * h + 1] * pv));
          pf[j][2 * h + 1] = movmatrix(pack_half2(s[4 * h + 2] * pv, s[4 * h + 3] * pv));
        }
      }
      // O^T += V^T P^T: keys 2t, 2t + 1, 2t + 8, 2t + 9 of each half, this lane's VB dims of each
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t vw[4][VB / 4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int row = 2 * t + (e & 1) + (e & 2) * 4;
          if constexpr (D == 128) {
            const uint4 v = lds128(vt + h * S::kHalf + tile_at<D>(row, gq));
            vw[e][0] = W::prep(v.x);
            vw[e][1] = W::prep(v.y);
            vw[e][2] = W::prep(v.z);
            vw[e][3] = W::prep(v.w);
          } else {
            const uint2 v = lds64(vt + h * S::kHalf + tile_at<D>(row, gq >> 1) + (gq & 1) * 8);
            vw[e][0] = W::prep(v.x);
            vw[e][1] = W::prep(v.y);
          }
        }
#pragma unroll
        for (int w = 0; w < VB / 4; ++w) {
          const uint32_t xa = __byte_perm(vw[0][w], vw[1][w], 0x5140), xb = __byte_perm(vw[0][w], vw[1][w], 0x7362);
          const uint32_t ya = __byte_perm(vw[2][w], vw[3][w], 0x5140), yb = __byte_perm(vw[2][w], vw[3][w], 0x7362);
          const uint32_t a0[4] = {W::template pair<false>(xa), W::template pair<true>(xa), W::template pair<false>(ya),
                                  W::template pair<true>(ya)};
          const uint32_t a1[4] = {W::template pair<false>(xb), W::template pair<true>(xb), W::template pair<false>(yb),
                                  W::template pair<true>(yb)};
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            mma16816(o[j][2 * w], a0, pf[j][2 * h], pf[j][2 * h + 1]);
            mma16816(o[j][2 * w + 1], a1, pf[j][2 * h], pf[j][2 * h + 1]);
          }
        }
      }
    }

    // join the warps' parts in shared memory (the rings are drained)
    cp_async_wait<0>();
    __syncthreads();
    const float unit = vref * (1.f / 16384.f);
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
      for (int sh = 4; sh < 32; sh <<= 1) {
        l0[j] += __shfl_xor_sync(0xffffffffu, l0[j], sh);
        l1[j] += __shfl_xor_sync(0xffffffffu, l1[j], sh);
      }
      const int ra = 8 * j + 2 * t;
      float* oa = mo + (warp * S::kRows + ra) * S::kLd + VB * gq;
      float* ob = oa + S::kLd;
#pragma unroll
      for (int e = 0; e < MT; ++e) {
        *reinterpret_cast<float2*>(oa + 2 * e) = make_float2(o[j][e][0] * unit, o[j][e][2] * unit);
        *reinterpret_cast<float2*>(ob + 2 * e) = make_float2(o[j][e][1] * unit, o[j][e][3] * unit);
      }
      if (gq == 0) {
        *reinterpret_cast<float2*>(mml + 2 * (warp * S::kRows + ra)) = make_float2(m0[j], l0[j]);
        *reinterpret_cast<float2*>(mml + 2 * (warp * S::kRows + ra + 1)) = make_float2(m1[j], l1[j]);
      }
    }
    __syncthreads();
    const bool whole = ta == 0 && tb == nt;
    // a part's place: this CTA's slot 0 if the item began before the share, else slot 1
    float* slot = parts + (2 * static_cast<size_t>(blockIdx.x) + (ta == 0 ? 1 : 0)) * kDecSlotFloats;
    auto put = [&](int row, int c, float4 v, float l) {
      const float inv = l > 0.f ? 1.f / l : 0.f;
      const int i = row / rep, h = row - i * rep;
      store4(static_cast<T*>(a.out) + (q.q0 + i) * a.out_stride + (g * rep + h) * D + c, v.x * inv, v.y * inv, v.z * inv, v.w * inv);
    };
    for (int e = tid; e < rows * (D / 4); e += kDecThreads) {
      const int row = e / (D / 4), c = 4 * (e % (D / 4));
      float m = -INFINITY, l = 0.f;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kDecWarps; ++w) m = fmaxf(m, mml[2 * (w * S::kRows + row)]);
#pragma unroll
      for (int w = 0; w < kDecWarps; ++w) {
        const float2 ml = *reinterpret_cast<const float2*>(mml + 2 * (w * S::kRows + row));
        const float f = m > -INFINITY ? exp2_approx(ml.x - m) : 0.f;
        const float4 u = *reinterpret_cast<const float4*>(mo + (w * S::kRows + row) * S::kLd + c);
        l += ml.y * f;
        v.x += u.x * f;
        v.y += u.y * f;
        v.z += u.z * f;
        v.w += u.w * f;
      }
      if (whole) {
        put(row, c, v, l);
      } else {
        *reinterpret_cast<float4*>(slot + row * D + c) = v;
        if (c == 0) *reinterpret_cast<float2*>(slot + kDecMaxRows * D + 2 * row) = make_float2(m, l);
      }
    }
    if (!whole) {
      // the item's parts lie with CTAs c0 .. c1; the last to arrive joins them in that order
      const int c0 = share.cta_of(item), c1 = share.cta_of(item + nt - 1);
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        s_last = atomicAdd(counters + c0, 1u) == static_cast<unsigned>(c1 - c0);
        if (s_last) counters[c0] = 0u;  // as the next call wants it
      }
      __syncthreads();
      if (s_last) {
        __threadfence();
        const int np = c1 - c0 + 1;
        auto part = [&](int k) { return parts + (2 * static_cast<size_t>(c0 + k) + (k == 0 ? 1 : 0)) * kDecSlotFloats; };
        float* wt = reinterpret_cast<float*>(smem);  // [row][np] what each part's output is multiplied with
        __shared__ float s_inv[kDecMaxRows];
        for (int row = warp; row < rows; row += kDecWarps) {
          float m = -INFINITY, l = 0.f;
          for (int k = lane; k < np; k += 32) m = fmaxf(m, __ldcg(part(k) + kDecMaxRows * D + 2 * row));
          m = warp_max(m);
          for (int k = lane; k < np; k += 32) {
            const float2 ml = __ldcg(reinterpret_cast<const float2*>(part(k) + kDecMaxRows * D + 2 * row));
            const float f = m > -INFINITY ? exp2_approx(ml.x - m) : 0.f;
            wt[row * np + k] = f;
            l += ml.y * f;
          }
          l = warp_sum(l);
          if (lane == 0) s_inv[row] = l;
        }
        __syncthreads();
        for (int e = tid; e < rows * (D / 4); e += kDecThreads) {
          const int row = e / (D / 4), c = 4 * (e % (D / 4));
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
          for (int k = 0; k < np; ++k) {
            const float4 u = __ldcg(reinterpret_cast<const float4*>(part(k) + row * D + c));
            const float f = wt[row * np + k];
            v.x += u.x * f;
            v.y += u.y * f;
            v.z += u.z * f;
            v.w += u.w * f;
          }
          put(row, c, v, s_inv[row]);
        }
      }
    }
    __syncthreads();  // the rings take the next item's tiles
  }
}

// ---- launches ------------------------------------------------------------------------------------
struct AttnWorkspace {
  unsigned* counters;
  float* parts;
};

template <typename T, typename C, int D, int NT>
cudaError_t launch_decode(const PagedPool& p, const PagedAttnArgs& a, int small_rows, const AttnWorkspace& w, int sms, int dev, cudaStream_t s) {
  using S = Dec<D, NT>;
  auto kernel = paged_decode_kernel<T, C, D, NT>;
  static std::atomic<uint64_t> ready{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), S::kSmem, dev, ready);
  if (e != cudaSuccess) return e;
  kernel<<<std::min(sms * S::kCtas, kAttnMaxCtas), kDecThreads, S::kSmem, s>>>(p, a, small_rows, w.counters, w.parts);
  return cudaGetLastError();
}

// all requests with few rows: the narrower kernel that holds them; else only the single tokens (and what fits
// beside them) are taken apart from the prompt chunks
int small_rows_of(const PagedAttnArgs& a, int rep) {
  const long long most = static_cast<long long>(a.max_q) * rep;
  return most <= 8 ? 8 : most <= kDecMaxRows ? kDecMaxRows : rep <= 8 ? 8 : 16;
}
template <typename T, typename C, int D>
cudaError_t launch(const PagedPool& p, const PagedAttnArgs& a, int small_rows, const AttnWorkspace& w, int sms, int dev, cudaStream_t s) {
  return small_rows == 8 ? launch_decode<T, C, D, 1>(p, a, small_rows, w, sms, dev, s)
                         : launch_decode<T, C, D, 2>(p, a, small_rows, w, sms, dev, s);
}
template <typename T, typename C>
cudaError_t launch(const PagedPool& p, int head_dim, const PagedAttnArgs& a, int small_rows, const AttnWorkspace& w, int sms, int dev, cudaStream_t s) {
  return head_dim == 128 ? launch<T, C, 128>(p, a, small_rows, w, sms, dev, s) : launch<T, C, 64>(p, a, small_rows, w, sms, dev, s);
}

// the current device and its SMs (0: none)
int sm_count(int* dev) {
  int n = 0;
  *dev = 0;
  if (cudaGetDevice(dev) != cudaSuccess || *dev < 0 || *dev >= 64) return 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, *dev) != cudaSuccess) return 0;
  return n;
}

// the workspace: the decode kernel's counters (one per CTA) and two parts of each CTA's share, then the chunk kernel's parts
constexpr size_t kCounterBytes = sizeof(unsigned) * kAttnMaxCtas;
size_t few_bytes(size_t sms) {
  return kCounterBytes + sizeof(float) * 2 * kDecSlotFloats * std::min<size_t>(3 * sms, kAttnMaxCtas);
}

}  // namespace

}  // namespace k2

using namespace k2;

extern "C" {

size_t k2_paged_workspace_bytes(void) {
  int dev = 0;
  const size_t sms = static_cast<size_t>(sm_count(&dev));
  return few_bytes(sms) + paged_chunk_part_bytes() * std::min<size_t>(sms, kAttnMaxCtas);
}

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
  if (requests < 0 || requests > K2_PAGED_MAX_REQUESTS || tokens < 0 || tokens > 1 << 30 || max_q < 0 || table_stride < 1) {
    set_error("requests in [0, %d], tokens in [0, 2^30], max_q >= 0, table_stride >= 1 (got %d, %d, %d, %d)",
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
  if ((tokens > 1 && (q_stride < row || out_stride < row || q_stride % 8 || out_stride % 8)) || !aligned16(d_q) ||
      !aligned16(d_out)) {
    set_error("query and output rows must be 16-byte aligned and at least n_heads * head_dim elements apart");
    return K2_ERR_ARG;
  }
  if (!d_workspace || reinterpret_cast<uintptr_t>(d_workspace) % 256 || ws_bytes < k2_paged_workspace_bytes()) {
    set_error("workspace must be 256-byte aligned and hold k2_paged_workspace_bytes() = %zu bytes (got %zu)",
              k2_paged_workspace_bytes(), ws_bytes);
    return K2_ERR_WORKSPACE;
  }
  if (rows_meet(d_q, 2 * q_stride, d_out, 2 * out_stride, 2 * row, tokens)) {  // a request's queries are read by several CTAs, some after another has stored its rows
    set_error("the output may not lie over the queries");
    return K2_ERR_ARG;
  }
  int dev = 0;
  const int sms = sm_count(&dev);
  if (sms == 0) {
    set_error("no CUDA device");
    return K2_ERR_CUDA;
  }
  uint8_t* ws = static_cast<uint8_t*>(d_workspace);
  const AttnWorkspace w = {reinterpret_cast<unsigned*>(ws), reinterpret_cast<float*>(ws + kCounterBytes)};
  const PagedPool p(*kv);
  const PagedAttnArgs a = {d_q, q_stride, d_cu_q, d_kv_len, d_table, table_stride, requests,
                           tokens, n_heads, std::min(max_q, tokens), scale, d_out, out_stride,
                           kv->wait_limit_us ? 1000ull * kv->wait_limit_us : kWaitLimitNs};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int d = kv->head_dim;
  const int rep = n_heads / kv->n_kv_heads, small = small_rows_of(a, rep);
  cudaError_t e;
  if (dtype == K2_F16)
    e = kv->dtype == K2_I8 ? launch<__half, CodeI8>(p, d, a, small, w, sms, dev, s)
                           : launch<__half, CodeF8>(p, d, a, small, w, sms, dev, s);
  else
    e = kv->dtype == K2_I8 ? launch<__nv_bfloat16, CodeI8>(p, d, a, small, w, sms, dev, s)
                           : launch<__nv_bfloat16, CodeF8>(p, d, a, small, w, sms, dev, s);
  if (e == cudaSuccess && static_cast<int64_t>(a.max_q) * rep > small)
    e = launch_paged_chunk(p, a, d, kv->dtype, dtype, small, reinterpret_cast<float*>(ws + few_bytes(static_cast<size_t>(sms))), sms, dev, s);
  if (e == cudaSuccess) return K2_OK;
  set_error("attention launch: %s", cudaGetErrorString(e));
  return K2_ERR_CUDA;
}

}  // extern "C"
