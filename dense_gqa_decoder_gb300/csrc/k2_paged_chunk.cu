// Attention of prompt chunks over a block-paged 8-bit cache (k2_paged_attention
// for requests with many query rows), on the 5th-generation tensor cores.
//
// Compute bound: 4 flop per (query row, key, dim) and an exponential per score.
// A CTA takes up to 256 query rows of one KV head -- two tiles of 128 = 128 / rep
// tokens x rep heads -- over the keys in tiles of 64:
//   one warp fetches the tile's codes (bulk copies of 16 rows, kCodeTiles tiles ahead) and its scales;
//   four warps widen the codes to fp16 (exact) into shared memory, K and V
//     alike as swizzled rows (V enters P.V through an MN-major descriptor);
//   one warp per query tile issues S = Q K^T (S in tensor memory) and O += P V (P and O in
//     tensor memory);
//   four warps per query tile take a row per thread: no exchange between threads
//     anywhere in the softmax.
// The two query tiles alternate: while one's softmax runs, the other's MMAs do,
// and S of the next key tile is issued as soon as the scores are in registers.
//
// Scales: the queries carry a power of two that brings a row into fp16's upper
// range (exact); a block's K scale multiplies its 16 scores' common factor, and its V
// scale enters the exponent, p' = 2^(s - m + log2(vs / vref) + 11), so neither costs
// an operation per score.  vref is the largest V scale of the CTA's keys; the row's
// sum takes each block's p' times 2^-(log2(vs / vref) + 11).  m moves only when a
// tile's maximum exceeds it by kLazy (then O is rescaled in tensor memory), so
// p' <= 2^15; p' is rounded to fp16, in full precision down to 2^-14 (one number, for the same reason as for few rows).
//
// As for single tokens, every CTA takes an equal share of the step's keys (an item =
// request, KV head, block of query tokens; counted in keys, each with kChStart more
// for its start and end); a kernel of its own joins the parts of an item.
//
// 2048 tokens of 32 heads of 128 on 8192 cached ones take 310 us, 1000 TFLOP/s: the exponentials and conversions of the
// softmax warps and the widening share the issue slots, and the tensor pipe is busy for 45 % of the SMs' active cycles.
#include <math.h>

#include <algorithm>

#include "k2_paged.cuh"
#include "k2_tc.cuh"

namespace k2 {

namespace {

constexpr int kSoftWarps = 8, kConvWarps = 4;
constexpr int kFetchWarp = kSoftWarps + kConvWarps, kMmaWarp = kFetchWarp + 1;  // and one more: one per query tile
constexpr int kChThreads = 32 * (kMmaWarp + 2);
constexpr int kChRows = 128, kChKeys = 64, kChStages = 3;
constexpr int kCodeTiles = 4;  // key tiles of codes on their way
// tiles whose scales are kept: one is read by a softmax warp up to kCodeTiles + kChStages - 1 tiles after it was fetched
constexpr int kScaleTiles = 8;
static_assert(kScaleTiles >= kCodeTiles + kChStages, "scales outlive their tile");
// An item's start and end count as 768 keys (2048 new tokens on 1 cached one: 92 us, 130 with 256; 8 requests of 512 on 512:
// 142 and 147; 1536 is slower again), and a CTA's share is 512 keys at least (12 requests, three with chunks of 509, heads of
// 64: 35 us, 48 with 1024).
constexpr int kChStart = 768, kChShare = 512;
constexpr float kLazy = 4.0f, kUp = 11.0f;
constexpr int kPartFloats = 2 * kChRows * (128 + 2);  // one part: rows x (output, maximum, sum)

template <int D>
struct Ch {
  static constexpr int NA = D / 64;                  // 64-dim swizzle atoms of a row
  static constexpr int QA = kChRows * 128;           // one atom of a query tile
  static constexpr int QB = NA * QA;                 // a query tile
  static constexpr int KA = kChKeys * 128;           // one atom of K (or V) of a key tile
  static constexpr int KB = NA * KA;
  static constexpr int OFF_ST = 2 * QB;
  static constexpr int OFF_CODES = OFF_ST + kChStages * 2 * KB;
  static constexpr int CODES = 2 * kChKeys * D;      // K and V codes of a key tile
  static constexpr int BYTES = OFF_CODES + kCodeTiles * CODES;
  static constexpr int DYN = BYTES + 1024;           // + alignment to 1024 B
  // tensor memory: O of both query tiles, S, then P (two fp16 per column)
  static constexpr int TM_S = 2 * D, TM_P = 2 * D + 2 * kChKeys, TM_COLS = 512;
  // instruction descriptors (kind::f16): fp16 A and B, fp32 D, M = 128; for O, B (V) is MN-major (bit 16)
  static constexpr uint32_t IDESC_S = (1u << 4) | (static_cast<uint32_t>(kChKeys >> 3) << 17) | (8u << 24);
  static constexpr uint32_t IDESC_O = (1u << 4) | (1u << 16) | (static_cast<uint32_t>(D >> 3) << 17) | (8u << 24);
};

// One lane of a warp, chosen so that the compiler knows it is one: the operands of what it then issues go through
// uniform registers without a detour (8 MMAs take 45 cycles each to issue, against 78 from a branch on the lane's
// number, and the smaller ones execute in 48).
__device__ __forceinline__ bool elect() {
  uint32_t ok;
  asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}" : "=r"(ok));
  return ok != 0;
}
// D (+)= A B, A and B in shared memory / A in tensor memory
template <bool ACC>
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(idesc), "n"(ACC ? 1 : 0)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// 64 columns of this warp's lanes
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, uint32_t* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
      "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];\n\ttcgen05.wait::ld.sync.aligned;"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
        "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
        "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31]), "=r"(v[32]),
        "=r"(v[33]), "=r"(v[34]), "=r"(v[35]), "=r"(v[36]), "=r"(v[37]), "=r"(v[38]), "=r"(v[39]), "=r"(v[40]),
        "=r"(v[41]), "=r"(v[42]), "=r"(v[43]), "=r"(v[44]), "=r"(v[45]), "=r"(v[46]), "=r"(v[47]), "=r"(v[48]),
        "=r"(v[49]), "=r"(v[50]), "=r"(v[51]), "=r"(v[52]), "=r"(v[53]), "=r"(v[54]), "=r"(v[55]), "=r"(v[56]),
        "=r"(v[57]), "=r"(v[58]), "=r"(v[59]), "=r"(v[60]), "=r"(v[61]), "=r"(v[62]), "=r"(v[63])
      : "r"(taddr)
      : "memory");
}

// What a wait that runs out ends: its limit, and the CTA's word that says that one did
struct Patience {
  volatile int* stop;
  uint64_t limit_ns;
};
// A wait for completion `n` (0, 1, ...) of a barrier; false once it, or another wait of the CTA, gave up
__device__ __forceinline__ bool await(uint64_t* bar, int n, const Patience& w) {
  const uint32_t parity = static_cast<uint32_t>(n) & 1u;
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer();
  while (!mbar_try_wait(bar, parity)) {
    if (*w.stop) return false;
    if (globaltimer() - t0 > w.limit_ns) {
      *w.stop = 1;
      return false;
    }
  }
  return true;
}

// The step's work as one line of keys: requests one after another, in each the KV heads, in each the blocks of query
// tokens (items), an item's keys after kChStart units for its start and end.  The CTAs take equal shares of it.
struct ChunkWork {
  int rep, qt, tt, n_kv, small_rows;  // query heads per KV head; tokens of a query tile, of an item
  const PagedAttnArgs& a;
  int block_log2;

  struct Cost {
    long long head;  // one KV head's items
    int nb, basek;   // items, keys before the first query
  };
  __device__ __forceinline__ ChunkWork(const PagedPool& p, const PagedAttnArgs& args, int small)
      : rep(args.n_heads / p.n_kv), qt(kChRows / rep), tt(2 * qt), n_kv(p.n_kv), small_rows(small), a(args),
        block_log2(p.block_log2) {}
  __device__ __forceinline__ Req req(int r) const { return request(a, block_log2, r); }
  __device__ __forceinline__ Cost cost(const Req& x) const {
    Cost c = {0, 0, 0};
    if (x.ok && static_cast<long long>(x.nq) * rep > small_rows) {
      c.nb = (x.nq + tt - 1) / tt;
      c.basek = x.len - x.nq;
      c.head = c.nb * (static_cast<long long>(kChStart) + c.basek) + static_cast<long long>(tt) * c.nb * (c.nb - 1) / 2 + x.nq;
    }
    return c;
  }
  // place of item b in its head
  __device__ __forceinline__ long long start(const Cost& c, int b) const {
    return b * (static_cast<long long>(kChStart) + c.basek) + static_cast<long long>(tt) * b * (b + 1) / 2;
  }
  __device__ __forceinline__ static int ctas(long long total, int most) {
    return static_cast<int>(min(static_cast<long long>(most), (total + kChShare - 1) / kChShare));
  }

  struct Item {
    Req q;
    int r, g, t0;       // request, KV head, first query token
    int kend, nkt, basek;
    long long at;       // place of its first key
    long long end;      // and behind its last
  };
  // the item at place x, of request r or a later one; base: place of request r
  __device__ __forceinline__ Item item(long long x, int& r, long long& base) const {
    Item i;
    i.q = req(r);
    Cost c = cost(i.q);
    while (x >= base + c.head * n_kv) {
      base += c.head * n_kv;
      i.q = req(++r);
      c = cost(i.q);
    }
    i.r = r;
    i.g = static_cast<int>(quotient(x - base, c.head));
    const long long rem = x - base - i.g * c.head;
    int b = 0;
    for (int hi = c.nb; hi - b > 1;) {
      const int mid = (b + hi) >> 1;
      if (start(c, mid) <= rem) b = mid;
      else hi = mid;
    }
    i.t0 = b * tt;
    i.basek = c.basek;
    i.kend = c.basek + min(i.q.nq, i.t0 + tt);
    i.nkt = (i.kend + kChKeys - 1) / kChKeys;
    i.at = base + i.g * c.head + start(c, b) + kChStart;
    i.end = i.at + i.kend;
    return i;
  }
};

// The prefix sums over the requests, by a block of THREADS threads: the total, and (find) the request at a place
template <int THREADS>
struct ChunkScan {
  long long total, own, before;
  int per;
  __device__ __forceinline__ ChunkScan(const ChunkWork& w, long long* sums) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    per = (w.a.requests + THREADS - 1) / THREADS;
    own = 0;
    for (int i = 0; i < per; ++i) {
      const int r = tid * per + i;
      if (r < w.a.requests) own += w.cost(w.req(r)).head * w.n_kv;
    }
    long long inc = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += u;
    }
    if (lane == 31) sums[warp] = inc;
    __syncthreads();
    total = 0;
    before = inc - own;
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) {
      if (i < warp) before += sums[i];
      total += sums[i];
    }
  }
  // one thread writes the request that holds place x, and that request's place
  __device__ __forceinline__ void find(const ChunkWork& w, long long x, int* req, long long* base) const {
    if (x < before || x >= before + own) return;
    long long at = before;
    for (int i = 0; i < per; ++i) {
      const int r = threadIdx.x * per + i;
      if (r >= w.a.requests) break;
      const long long n = w.cost(w.req(r)).head * w.n_kv;
      if (x < at + n) {
        *req = r;
        *base = at;
        return;
      }
      at += n;
    }
  }
};

// two waits whose first tries overlap (a try takes over a hundred cycles)
__device__ __forceinline__ bool await2(uint64_t* a, int na, uint64_t* b, int nb, const Patience& w) {
  const bool x = mbar_try_wait(a, static_cast<uint32_t>(na) & 1u), y = mbar_try_wait(b, static_cast<uint32_t>(nb) & 1u);
  return (x || await(a, na, w)) && (y || await(b, nb, w));
}

template <typename T, typename C, int D>
__global__ void __launch_bounds__(kChThreads, 1)
    paged_chunk_kernel(const PagedPool p, const PagedAttnArgs a, int small_rows, float* parts) {
  using S = Ch<D>;
  using W = Widen<C>;
  constexpr int ST = kChStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  __shared__ __align__(8) uint64_t kv_full[ST], kv_empty[ST], code_full[kCodeTiles], code_empty[kCodeTiles], s_full[2], s_free[2], p_ready[2], o_done[2], drained[2];
  // of a tile's 16-key quarters: the K scale (-1: no keys), log2(vs / vref) + kUp and 2^- of that
  __shared__ __align__(16) float sc_k[kScaleTiles][4], sc_up[kScaleTiles][4], sc_down[kScaleTiles][4];
  __shared__ uint8_t s_up[2 * kChRows];  // each query row's power of two (+ 113)
  __shared__ uint32_t tmem_slot;
  __shared__ int stop, s_req;
  __shared__ unsigned s_vref;
  __shared__ long long s_sum[kChThreads / 32], s_base;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Patience patience = {&stop, a.wait_ns};
  const ChunkWork work(p, a, small_rows);
  const int rep = work.rep, QT = work.qt;
  const unsigned rep_inv = (65536u + rep - 1) / rep;  // x / rep = x * rep_inv >> 16 for x < 128 (rep <= 16)
  auto by_rep = [&](int ro) { return static_cast<int>(static_cast<unsigned>(ro) * rep_inv >> 16); };
  pdl_trigger();  // the kernel that joins the parts waits for this one's end
  if (tid == 0) {
    stop = 0;
    s_vref = 0u;
    for (int i = 0; i < ST; ++i) {
      mbar_init(&kv_full[i], kConvWarps);
      mbar_init(&kv_empty[i], 2);
    }
    for (int i = 0; i < kCodeTiles; ++i) {
      mbar_init(&code_full[i], 1);
      mbar_init(&code_empty[i], kConvWarps);
    }
    for (int q = 0; q < 2; ++q) {
      mbar_init(&s_full[q], 1);
      mbar_init(&s_free[q], 4);
      mbar_init(&p_ready[q], 4);
      mbar_init(&o_done[q], 1);
      mbar_init(&drained[q], 1);
    }
    fence_mbar_init();
  }
  const ChunkScan<kChThreads> scan(work, s_sum);
  const long long total = scan.total;
  const int ctas = ChunkWork::ctas(total, gridDim.x);
  if (blockIdx.x >= ctas) {
    pdl_wait();  // this kernel may have started before the one for few rows has ended: it ends after it
    return;
  }
  const Share share(total, ctas);
  const long long x0 = share.first(blockIdx.x), x1 = share.first(blockIdx.x + 1);
  scan.find(work, x0, &s_req, &s_base);
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)), "r"(S::TM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = tmem_slot;
  int r = s_req;
  long long base = s_base;
  int n_kv = 0, n_q[2] = {0, 0};  // key tiles so far: of the ring, of each query tile
  bool dead = false;

  for (long long x = x0; x < x1;) {
    // ---- the item at x -----------------------------------------------------------------------
    const ChunkWork::Item it = work.item(x, r, base);
    const Req q = it.q;
    const int g = it.g, t0 = it.t0, kend = it.kend, nkt = it.nkt;
    const long long item = it.at;
    const int ta = x0 <= item ? 0 : static_cast<int>(min((x0 - item + kChKeys - 1) / kChKeys, static_cast<long long>(nkt)));
    const int tb = x1 <= item ? 0 : static_cast<int>(min((x1 - item + kChKeys - 1) / kChKeys, static_cast<long long>(nkt)));
    x = it.end;
    if (ta >= tb) continue;
    const bool whole = ta == 0 && tb == nkt;
    const int nqt = t0 + QT < q.nq ? 2 : 1, tiles = tb - ta;
    const int* table = a.table + static_cast<size_t>(r) * a.table_stride;
    // softmax threads: row `row` of query tile qi
    const int qi = warp >> 2, row = (warp & 3) * 32 + lane;
    const int dt = by_rep(row), tok = t0 + qi * QT + dt, head = g * rep + row - dt * rep;
    const bool soft = warp < kSoftWarps && qi < nqt;
    const bool row_ok = soft && row < QT * rep && tok < q.nq;
    if (!dead) {
      const int j0 = (ta * kChKeys) >> p.block_log2, j1 = (min(tb * kChKeys, kend) - 1) >> p.block_log2;
      int vid[4];  // blocks of the CTA's keys, for their V scales: on their way while the queries are read
#pragma unroll
      for (int e = 0; e < 4; ++e) vid[e] = j0 + tid + e * kChThreads <= j1 ? __ldg(table + j0 + tid + e * kChThreads) : -1;
      // the query rows into shared memory as fp16, each scaled by a power of two; D / 8 lanes take a row
      constexpr int LR = D / 8, RW = 32 / LR;  // lanes per row, rows per warp and step
      const float sign = a.scale < 0.f ? -1.f : 1.f;
#pragma unroll 10
      for (int e = warp * RW + lane / LR; e < nqt * kChRows; e += RW * (kChThreads / 32)) {
        const int j = e / kChRows, ro = e % kChRows, dt = by_rep(ro), i = t0 + j * QT + dt, c = lane % LR;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (ro < QT * rep && i < q.nq)
          v = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(a.q) + (q.q0 + i) * a.q_stride + static_cast<size_t>(g * rep + ro - dt * rep) * D) + c);
        float f[8], top = 0.f;
        Unpack<T>::run(v, f);
#pragma unroll
        for (int d = 0; d < 8; ++d) top = fmaxf(top, fabsf(f[d]));
#pragma unroll
        for (int o = 1; o < LR; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const int ex = static_cast<int>(__float_as_uint(top) >> 23);
        const int up = top > 0.f && ex < 255 ? 14 + 127 - ex : 0;
        const int ua = up / 2, ub = up - ua;  // in two steps: 2^up itself may not be a normal number
        const float sa = __uint_as_float((127 + ua) << 23) * sign, sb = __uint_as_float((127 + ub) << 23);
        uint32_t h[4];
#pragma unroll
        for (int d = 0; d < 4; ++d) h[d] = pack_half2(f[2 * d] * sa * sb, f[2 * d + 1] * sa * sb);
        *reinterpret_cast<uint4*>(smem + j * S::QB + (c >> 3) * S::QA + sw128(ro, 8 * (c & 7))) = make_uint4(h[0], h[1], h[2], h[3]);
        if (c == 0) s_up[e] = static_cast<uint8_t>(up + 113);  // -113 .. 141
      }
      // the largest V scale of the CTA's keys
      float top = 0.f;
#pragma unroll 1
      for (int j = j0 + tid; j <= j1; j += 4 * kChThreads) {
        if (j != j0 + tid)
#pragma unroll
          for (int e = 0; e < 4; ++e) vid[e] = j + e * kChThreads <= j1 ? __ldg(table + j + e * kChThreads) : -1;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (static_cast<unsigned>(vid[e]) < static_cast<unsigned>(p.n_blocks))
            top = fmaxf(top, __ldg(p.vs + static_cast<size_t>(vid[e]) * p.n_kv + g));
      }
      top = warp_max(top);
      if (lane == 0) atomicMax(&s_vref, __float_as_uint(top));
      fence_proxy_async();  // Q (generic stores) before the MMAs read it
      __syncthreads();
    }
    const float vref = __uint_as_float(s_vref);
    float m_ref = -INFINITY, l = 0.f;
    int fetched = 0;  // key tiles of the item whose codes this warp has requested

    if (dead) {
    } else if (warp >= kSoftWarps && warp < kSoftWarps + kConvWarps) {
      // ---- codes to fp16 ---------------------------------------------------------------------
      const int ct = tid - 32 * kSoftWarps;
      constexpr int CH = D / 8, N = kChKeys * CH / (32 * kConvWarps);  // 8-code chunks per row, per thread
      constexpr int RS = 32 * kConvWarps / CH;                          // rows between a thread's chunks
      const int row0 = ct / CH, ch = ct % CH;
      uint32_t put[N];  // where this thread's codes go, within K (or V) of a stage
#pragma unroll
      for (int c = 0; c < N; ++c) put[c] = (ch >> 3) * S::KA + sw128(row0 + c * RS, 8 * (ch & 7));
#pragma unroll 1
      for (int i = 0; i < tiles; ++i) {
        const int n = n_kv + i, st = n % ST, slot = n % kCodeTiles;
        if (!__all_sync(0xffffffffu, await(&code_full[slot], n / kCodeTiles, patience))) break;
        const uint8_t* cst = smem + S::OFF_CODES + slot * S::CODES + 8 * ct;
        uint2 kc[N], vc[N];
#pragma unroll
        for (int c = 0; c < N; ++c) {
          kc[c] = *reinterpret_cast<const uint2*>(cst + 8 * 32 * kConvWarps * c);
          vc[c] = *reinterpret_cast<const uint2*>(cst + 8 * 32 * kConvWarps * c + S::CODES / 2);
        }
        // rows behind the request's last key, and quarters without a block, are zeros
        const float4 kq = *reinterpret_cast<const float4*>(sc_k[n % kScaleTiles]);
        if ((ta + i + 1) * kChKeys > q.len || fminf(fminf(kq.x, kq.y), fminf(kq.z, kq.w)) < 0.f) {
#pragma unroll
          for (int c = 0; c < N; ++c) {
            const int rr = row0 + c * RS;
            if ((ta + i) * kChKeys + rr >= q.len || sc_k[n % kScaleTiles][rr >> 4] < 0.f) kc[c] = vc[c] = make_uint2(0, 0);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&code_empty[slot]);
        if (n >= ST && !__all_sync(0xffffffffu, await(&kv_empty[st], n / ST - 1, patience))) break;
        uint8_t* kst = smem + S::OFF_ST + st * 2 * S::KB;
#pragma unroll
        for (int c = 0; c < N; ++c) {
          const uint32_t k0 = W::prep(kc[c].x), k1 = W::prep(kc[c].y), v0 = W::prep(vc[c].x), v1 = W::prep(vc[c].y);
          *reinterpret_cast<uint4*>(kst + put[c]) = make_uint4(W::template pair<false>(k0), W::template pair<true>(k0),
                                                               W::template pair<false>(k1), W::template pair<true>(k1));
          *reinterpret_cast<uint4*>(kst + S::KB + put[c]) = make_uint4(W::template pair<false>(v0), W::template pair<true>(v0),
                                                                       W::template pair<false>(v1), W::template pair<true>(v1));
        }
        fence_proxy_async();  // generic stores before the MMAs read them
        __syncwarp();
        if (lane == 0) mbar_arrive(&kv_full[st]);
      }
    } else if (warp == kFetchWarp) {
      // ---- codes and scales from memory -------------------------------------------------------------
      // lanes 0 .. 7: K (even) and V codes of quarter lane / 2; lanes 8 .. 11: the scales of quarter lane - 8
      const int quarter = lane < 8 ? lane >> 1 : lane & 3;
      const bool copies = lane < 8, scales = lane >= 8 && lane < 12;
      auto id_of = [&](int i) {
        const int key0 = (ta + i) * kChKeys + 16 * quarter;
        return i < tiles && key0 < kend ? __ldg(table + (key0 >> p.block_log2)) : -2;  // -2: behind the last key
      };
      auto scales_of = [&](int id, float& k_s, float& v_s) {
        k_s = -1.f;
        v_s = 0.f;
        if (scales && static_cast<unsigned>(id) < static_cast<unsigned>(p.n_blocks)) {
          const size_t at = static_cast<size_t>(id) * p.n_kv + g;
          k_s = __ldg(p.ks + at);
          v_s = __ldg(p.vs + at);
        }
      };
      int id = id_of(0), id_next = id_of(1);
      float k_s, v_s, k_next, v_next;
      scales_of(id, k_s, v_s);
#pragma unroll 1
      for (int i = 0; i < tiles; ++i) {
        const int n = n_kv + i, slot = n % kCodeTiles;
        const int id_after = id_of(i + 2);
        scales_of(id_next, k_next, v_next);
        if (n >= kCodeTiles && !__all_sync(0xffffffffu, await(&code_empty[slot], n / kCodeTiles - 1, patience))) break;
        const bool valid = static_cast<unsigned>(id) < static_cast<unsigned>(p.n_blocks);
        if (!valid && id != -2 && lane < 8) raise_flag(p.flags, K2_PAGED_BAD_BLOCK);
        if (scales) {
          // a scale of (as good as) zero counts as 2^-60; divided exactly, for vref may lie below (or near the end of) the
          // range of normal numbers
          const float up = __log2f(vref > 0.f ? fmaxf(__fdiv_rn(v_s, vref), 8.6736174e-19f) : 8.6736174e-19f) + kUp;
          sc_k[n % kScaleTiles][quarter] = k_s;
          sc_up[n % kScaleTiles][quarter] = k_s < 0.f ? 0.f : up;
          sc_down[n % kScaleTiles][quarter] = k_s < 0.f ? 0.f : exp2_approx(-up);
        }
        const unsigned some = __ballot_sync(0xffffffffu, copies && valid);
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(&code_full[slot], __popc(some) * 16 * D);  // after the warp's scale stores
        __syncwarp();
        if (copies && valid) {
          const int key0 = (ta + i) * kChKeys + 16 * quarter;
          const size_t off = (((static_cast<size_t>(id) * p.n_kv + g) << p.block_log2) + (key0 & ((1 << p.block_log2) - 1))) * D;
          bulk_g2s(smem + S::OFF_CODES + slot * S::CODES + (lane & 1) * (S::CODES / 2) + quarter * 16 * D,
                   (lane & 1 ? p.v : p.k) + off, 16 * D, &code_full[slot]);
        }
        id = id_next;
        id_next = id_after;
        k_s = k_next;
        v_s = v_next;
        fetched = i + 1;
      }
    } else if (warp >= kMmaWarp) {
      // ---- the MMAs of query tile j ----------------------------------------------------------------
      const int j = warp - kMmaWarp;
      if (elect()) {
        const uint64_t qd = smem_desc(smem) + static_cast<uint64_t>(j * (S::QB >> 4)), kd = smem_desc(smem + S::OFF_ST),
                       vd = smem_desc_mn(smem + S::OFF_ST + S::KB, S::KA, 8 * 128);
        const uint32_t ts = tmem + S::TM_S + kChKeys * j, tp = tmem + S::TM_P + 32 * j, to = tmem + j * D;
        auto issue_s = [&](int st) {  // S over stage st (offsets in units of 16 bytes)
          const uint64_t ks = kd + static_cast<uint64_t>(st * (2 * S::KB >> 4));
          mma_ss<false>(ts, qd, ks, S::IDESC_S);
#pragma unroll
          for (int e = 1; e < D / 16; ++e)
            mma_ss<true>(ts, qd + ((e >> 2) * S::QA + (e & 3) * 32 >> 4), ks + ((e >> 2) * S::KA + (e & 3) * 32 >> 4), S::IDESC_S);
          mma_commit(&s_full[j]);
        };
        bool ok = true;
        int st = n_kv % ST;
        if (j < nqt) {
          if ((ok = await(&kv_full[st], n_kv / ST, patience))) {
            tc_after();
            issue_s(st);
          }
          for (int i = 0; i < tiles && ok; ++i) {
            const int n = n_kv + i, m = n_q[j] + i, next = st + 1 == ST ? 0 : st + 1;
            if (i + 1 < tiles) {  // the scores of tile i are in registers: S of the next tile
              if (!(ok = await2(&kv_full[next], (n + 1) / ST, &s_free[j], m, patience))) break;
              tc_after();
              issue_s(next);
            }
            if (!(ok = await(&p_ready[j], m, patience))) break;
            tc_after();
            const uint64_t vs = vd + static_cast<uint64_t>(st * (2 * S::KB >> 4));
#pragma unroll
            for (int e = 0; e < kChKeys / 16; ++e)
              mma_ts(to, tp + 8 * e, vs + (e * 16 * 128 >> 4), S::IDESC_O, i == 0 && e == 0 ? 0u : 1u);
            mma_commit(&kv_empty[st]);
            mma_commit(&o_done[j]);  // last: what waits for it has waited for the stage's release too
            st = next;
          }
        } else {  // no such query tile: the stages are only given back
          for (int i = 0; i < tiles && ok; ++i, st = st + 1 == ST ? 0 : st + 1)
            if ((ok = await(&kv_full[st], (n_kv + i) / ST, patience))) mbar_arrive(&kv_empty[st]);
        }
      }
    } else if (soft) {
      // ---- softmax: one row per thread -------------------------------------------------------------
      const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
      const int qpos = it.basek + tok;  // the row sees keys 0 .. qpos
      const int up = s_up[qi * kChRows + row] - 113, ua = up / 2;
      // from accumulators to base-2 scores
      const float f_row = fabsf(a.scale) * kLog2e * __uint_as_float((127 - ua) << 23) * __uint_as_float((127 - up + ua) << 23);
      bool ok = true;
      for (int i = 0; i < tiles; ++i) {
        const int n = n_kv + i, m = n_q[qi] + i, st = n % ST;
        ok = await2(&kv_full[st], n / ST, &s_full[qi], m, patience);  // the tile's scales; its scores
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        const int sl = n % kScaleTiles;
        const float4 kq = *reinterpret_cast<const float4*>(sc_k[sl]), uq = *reinterpret_cast<const float4*>(sc_up[sl]),
                     dq = *reinterpret_cast<const float4*>(sc_down[sl]);
        const float kk[4] = {kq.x, kq.y, kq.z, kq.w}, uu[4] = {uq.x, uq.y, uq.z, uq.w}, dd[4] = {dq.x, dq.y, dq.z, dq.w};
        tc_after();
        uint32_t raw[kChKeys];
        tmem_ld64(tmem + lanes + S::TM_S + kChKeys * qi, raw);
        tc_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_free[qi]);
        float s[kChKeys], c1[4];
#pragma unroll
        for (int e = 0; e < kChKeys; ++e) s[e] = __uint_as_float(raw[e]);
#pragma unroll
        for (int h = 0; h < 4; ++h) c1[h] = f_row * kk[h];
        const int last = row_ok ? qpos - (ta + i) * kChKeys : kChKeys;  // last visible column (padding rows: of no account)
        const bool gap = fminf(fminf(kk[0], kk[1]), fminf(kk[2], kk[3])) < 0.f;
        const bool masked = __any_sync(0xffffffffu, last < kChKeys - 1) || gap;
        if (masked) {
#pragma unroll
          for (int e = 0; e < kChKeys; ++e) s[e] = e <= last && kk[e >> 4] >= 0.f ? s[e] * c1[e >> 4] : -INFINITY;
#pragma unroll
          for (int h = 0; h < 4; ++h) c1[h] = 1.f;
        }
        float mt = -INFINITY;
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          float v = max3(s[16 * h], s[16 * h + 1], s[16 * h + 2]);
#pragma unroll
          for (int e = 3; e < 15; e += 2) v = max3(v, s[16 * h + e], s[16 * h + e + 1]);
          mt = fmaxf(mt, fmaxf(v, s[16 * h + 15]) * c1[h]);  // factors are >= 0
        }
        const bool move = mt > -INFINITY && (m_ref == -INFINITY || mt > m_ref + kLazy);
        const float alpha = move ? (m_ref == -INFINITY ? 0.f : exp2_approx(m_ref - mt)) : 1.f;
        if (move) {
          l *= alpha;
          m_ref = mt;
        }
        const float zm = m_ref == -INFINITY ? 0.f : m_ref;  // no visible key yet: every p is 0
        uint32_t pk[kChKeys / 2];
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const float c2 = uu[h] - zm;
          const f32x2 c11 = pk2(c1[h], c1[h]), c22 = pk2(c2, c2);
          f32x2 sums = pk2(0.f, 0.f);
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            const f32x2 x2 = fma2(pk2(s[16 * h + e], s[16 * h + e + 1]), c11, c22);
            float p0, p1;
            asm("mov.b64 {%0, %1}, %2;" : "=f"(p0), "=f"(p1) : "l"(x2));
            p0 = exp2_approx(p0);
            p1 = exp2_approx(p1);
            sums = add2(sums, pk2(p0, p1));
            pk[8 * h + e / 2] = pack_half2(p0, p1);
          }
          const float sum = sum2(sums);
          l = fmaf(sum, dd[h], l);
        }
        if (i > 0) {  // the previous P.V has read P and written O
          ok = __all_sync(0xffffffffu, await(&o_done[qi], m - 1, patience));
          if (!ok) break;
          tc_after();
          if (__any_sync(0xffffffffu, move)) {
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              uint32_t ov[32];
              tmem_ld32(tmem + lanes + qi * D + c, ov);
#pragma unroll
              for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
              tmem_st32(tmem + lanes + qi * D + c, ov);
            }
          }
        }
        tmem_st32(tmem + lanes + S::TM_P + 32 * qi, pk);
        tc_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_ready[qi]);
      }
      if (ok) (void)await(&o_done[qi], n_q[qi] + tiles - 1, patience);
    }
    __syncthreads();
    tc_after();
    if (stop && !dead) {
      // given up, whoever did: the copies and MMAs that are still on their way end before their memory is left
      dead = true;
      if (tid == 0) raise_flag(p.flags, K2_PAGED_TIMEOUT);
      if (warp == kFetchWarp) {
        for (int n = n_kv + max(0, fetched - kCodeTiles); n < n_kv + fetched; ++n)
          (void)mbar_wait(&code_full[n % kCodeTiles], (n / kCodeTiles) & 1);
      } else if (warp >= kMmaWarp && elect()) {
        mma_commit(&drained[warp - kMmaWarp]);
        (void)mbar_wait(&drained[warp - kMmaWarp], 0);
      }
      __syncthreads();
      tc_after();
    }
    n_kv += tiles;
    n_q[0] += tiles;
    if (nqt == 2) n_q[1] += tiles;
    if (tid == 0) s_vref = 0u;  // read above by everyone

    // ---- the item's rows, or this CTA's part of them -----------------------------------------------
    float* part = parts + (2 * static_cast<size_t>(blockIdx.x) + (ta == 0 ? 1 : 0)) * kPartFloats;
    if (soft) {
      const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
      const float nan = __uint_as_float(0x7fffffffu);
      // outputs are multiplied with 2^-kUp (over the row's sum), then with vref: 2^-kUp vref may not be a normal number
      const float unit = dead ? nan : 1.f / 2048.f;
      const float inv = whole ? (l > 0.f ? unit / l : dead ? nan : 0.f) : unit;
      T* out = static_cast<T*>(a.out) + (q.q0 + tok) * a.out_stride + static_cast<size_t>(head) * D;
      const int lrow = qi * kChRows + row;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t ov[32];
        tmem_ld32(tmem + lanes + qi * D + c, ov);
#pragma unroll
        for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * inv * vref);
        if (whole) {
          if (row_ok) {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              store4(out + c + e, __uint_as_float(ov[e]), __uint_as_float(ov[e + 1]), __uint_as_float(ov[e + 2]),
                     __uint_as_float(ov[e + 3]));
          }
        } else {
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            *reinterpret_cast<float4*>(part + (static_cast<size_t>((c + e) / 4) * (2 * kChRows) + lrow) * 4) =
                make_float4(__uint_as_float(ov[e]), __uint_as_float(ov[e + 1]), __uint_as_float(ov[e + 2]), __uint_as_float(ov[e + 3]));
        }
      }
      if (!whole) *reinterpret_cast<float2*>(part + 2 * kChRows * D + 2 * lrow) = make_float2(dead ? 0.f : m_ref, dead ? 1.f : l);
    }
    tc_before();
    __syncthreads();  // Q, the stages and tensor memory take the next item
    tc_after();
  }
  pdl_wait();  // as above
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(S::TM_COLS) : "memory");
}

// Items that several CTAs had a part of: block (c, slice) joins the one that began in CTA c's share, a slice of its
// columns.  Joined by the last CTA to arrive, as the few rows of a decode step are, the parts (133 KB each) would
// pass through one SM: 23 us for nine of them.
constexpr int kJoinThreads = 2 * kChRows, kJoinSlices = 8;
template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads) paged_join_kernel(const PagedPool p, const PagedAttnArgs a, int small_rows, const float* parts) {
  __shared__ long long s_sum[kJoinThreads / 32], s_base;
  __shared__ int s_req;
  const ChunkWork work(p, a, small_rows);
  const ChunkScan<kJoinThreads> scan(work, s_sum);
  const int ctas = ChunkWork::ctas(scan.total, gridDim.x), c0 = blockIdx.x;
  bool job = c0 + 1 < ctas;  // the last share ends with its last item
  ChunkWork::Item it;
  int c1 = 0;
  if (job) {
    const Share share(scan.total, ctas);
    const long long last = share.first(c0 + 1) - 1;  // of this CTA's share
    scan.find(work, last, &s_req, &s_base);
    __syncthreads();
    int r = s_req;
    long long base = s_base;
    it = work.item(last, r, base);
    c1 = share.cta_of(it.at + static_cast<long long>(kChKeys) * (it.nkt - 1));
    job = share.cta_of(it.at) == c0 && c1 > c0;
  }
  pdl_wait();  // the parts
  if (!job) return;
  const int lr = threadIdx.x, ro = lr % kChRows, i = it.t0 + (lr / kChRows) * work.qt + ro / work.rep;
  if (ro >= work.qt * work.rep || i >= it.q.nq) return;
  auto part = [&](int k) { return parts + (2 * static_cast<size_t>(k) + (k == c0 ? 1 : 0)) * kPartFloats; };
  float m = -INFINITY, l = 0.f;
#pragma unroll 4
  for (int k = c0; k <= c1; ++k) m = fmaxf(m, __ldcg(part(k) + 2 * kChRows * D + 2 * lr));
  constexpr int N = D / 4 / kJoinSlices;
  float4 v[N];
#pragma unroll
  for (int c = 0; c < N; ++c) v[c] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int k = c0; k <= c1; ++k) {
    const float* from = part(k);
    const float2 ml = __ldcg(reinterpret_cast<const float2*>(from + 2 * kChRows * D + 2 * lr));
    const float f = m > -INFINITY ? exp2_approx(ml.x - m) : 0.f;
    l += ml.y * f;
#pragma unroll
    for (int c = 0; c < N; ++c) {
      const float4 u = __ldcg(reinterpret_cast<const float4*>(from + (static_cast<size_t>(blockIdx.y * N + c) * (2 * kChRows) + lr) * 4));
      v[c].x += u.x * f;
      v[c].y += u.y * f;
      v[c].z += u.z * f;
      v[c].w += u.w * f;
    }
  }
  const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;  // a NaN stays one
  T* out = static_cast<T*>(a.out) + (it.q.q0 + i) * a.out_stride + static_cast<size_t>(it.g * work.rep + ro % work.rep) * D + 4 * blockIdx.y * N;
#pragma unroll
  for (int c = 0; c < N; ++c) store4(out + 4 * c, v[c].x * inv, v[c].y * inv, v[c].z * inv, v[c].w * inv);
}

template <typename T, typename C, int D>
cudaError_t launch(const PagedPool& p, const PagedAttnArgs& a, int small_rows, float* w, int sms, int dev, cudaStream_t s) {
  auto kernel = paged_chunk_kernel<T, C, D>;
  static std::atomic<uint64_t> ready{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), Ch<D>::DYN, dev, ready);
  if (e != cudaSuccess) return e;
  // after the kernel for few rows, SM by SM: the shared memory of its three CTAs leaves no room for one of these, so one
  // starts where those have ended (at once where they had no work)
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(std::min(sms, kAttnMaxCtas));
  cfg.blockDim = dim3(kChThreads);
  cfg.dynamicSmemBytes = Ch<D>::DYN;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kernel, p, a, small_rows, w);
  if (e != cudaSuccess) return e;
  cfg.gridDim.y = kJoinSlices;
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, paged_join_kernel<T, D>, p, a, small_rows, static_cast<const float*>(w));
}
template <typename T, typename C>
cudaError_t launch(const PagedPool& p, const PagedAttnArgs& a, int d, int small_rows, float* w, int sms, int dev, cudaStream_t s) {
  return d == 128 ? launch<T, C, 128>(p, a, small_rows, w, sms, dev, s) : launch<T, C, 64>(p, a, small_rows, w, sms, dev, s);
}

}  // namespace

size_t paged_chunk_part_bytes() { return 2 * sizeof(float) * kPartFloats; }

cudaError_t launch_paged_chunk(const PagedPool& p, const PagedAttnArgs& a, int head_dim, int kv_dtype, int q_dtype,
                               int small_rows, float* w, int sms, int dev, cudaStream_t s) {
  if (q_dtype == K2_F16)
    return kv_dtype == K2_I8 ? launch<__half, CodeI8>(p, a, head_dim, small_rows, w, sms, dev, s)
                             : launch<__half, CodeF8>(p, a, head_dim, small_rows, w, sms, dev, s);
  return kv_dtype == K2_I8 ? launch<__nv_bfloat16, CodeI8>(p, a, head_dim, small_rows, w, sms, dev, s)
                           : launch<__nv_bfloat16, CodeF8>(p, a, head_dim, small_rows, w, sms, dev, s);
}

}  // namespace k2
