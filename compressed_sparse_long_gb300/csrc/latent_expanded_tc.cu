// Expanded latent attention on tcgen05 tensor cores, by pairs of CTAs (cta_group::2): bf16, keys
// of 128 projected + 64 rotary dims (the rotary part shared by the heads), values of 128 dims.
//
//   S = Q K^T      M = 256 queries (128 a CTA), N = 128 keys, K = 192    (12 MMAs)
//   P = 2^(scale log2(e) S - m), bf16, in tensor memory over S
//   O += P V       M = 256 queries, N = 128 dims, K = 128 keys           (8 MMAs)
// A work item is 512 consecutive queries of one head of one sequence, as two tiles of 256 that
// take turns: while one tile's softmax runs, the other tile's products do. Each CTA holds 128
// queries of a tile, its S/P and O (tensor memory is full with both tiles'), and runs their
// softmax, a thread a query. Of a step's keys and values each CTA copies and holds half (64 keys;
// 64 of the values' 128 dims), which the products read from both CTAs: per CTA half the copies
// and 6 KB of shared-memory operands a product instead of 8. That is what one CTA's rate hangs
// on: alone, S's 128 x 128 x 16 products take 96 cycles instead of the pipe's 64 (the same
// kernel for single CTAs, 256 queries an item, ran an 8192-token prompt of 64 heads in 1102 us).
// Three stages of 40 KB keep copies two steps ahead.
//
// Bound: the tensor pipe (40 products a step of 512 queries x 128 keys, 2560 cycles; a step takes
// 3050, a tile's chain of S, softmax and P V being a little longer) and, in long runs, the power
// it draws: that prompt takes 850-930 us in runs of milliseconds and 920-945 (1.45-1.5 PFLOP/s) in
// longer ones.
//
// All (item, key tile) steps form one line, a sequence's blocks from the last (the longest, when
// causal) to the first, heads within a block; each pair takes an equal part of it. An item whose
// tiles fall to several pairs is left as partial results that a second kernel merges: without
// that, a long sequence's few items would decide the time (ragged chunks 391 us, now 190).
//
// Roles in each CTA: warps 0-7 softmax and output (tile 0 / 1), warp 8 copies, warp 11 watches
// the copies land and reports to the CTA of rank 0, whose warp 9 issues the pair's products.
#include "kernels.h"
#include "latent.h"
#include "tc.cuh"

namespace v4a {
namespace {

constexpr int kThreads = 384, kStages = 3;
constexpr int kT = 128;                                          // a CTA's queries of a tile; keys of a step
constexpr int kItem = 512;                                       // queries of an item
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRoom = 16.0f, kRaise = -8.0f;                   // log2 units: a reference above its maximum;
                                                                 // a weight that raises it

__device__ __forceinline__ float fast_exp2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ void tma_3d(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(tc::smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(tc::smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void st32(uint32_t taddr, const float (&v)[32]) {
  uint32_t u[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) u[i] = __float_as_uint(v[i]);
  tc::tmem_st32(taddr, u);
}
// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Weights 2^(k2 s + nm) of a query's 128 logits, rounded to bf16 for the second product, in
// pairs; returns their sum, unrounded.
__device__ __forceinline__ float weights(const float (&s)[128], uint64_t k22, float nm, uint32_t (&pw)[64]) {
  const uint64_t nm2 = pack2(nm, nm);
  uint64_t acc[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 64; ++i) {
    float a, b;
    unpack2(fma2(pack2(s[2 * i], s[2 * i + 1]), k22, nm2), a, b);
    a = fast_exp2(a);
    b = fast_exp2(b);
    acc[i & 3] = add2(acc[i & 3], pack2(a, b));
    pw[i] = pack_bf16(a, b);
  }
  float a, b;
  unpack2(add2(add2(acc[0], acc[1]), add2(acc[2], acc[3])), a, b);
  return a + b;
}

constexpr int kBlk = kT * 128, kHalf = kBlk / 2;                 // 128 and 64 rows of 128 bytes
constexpr int kStage = 3 * kHalf + kBlk;                         // half the keys, half the values
constexpr int kOffQ = 0, kOffKV = 6 * kBlk;
constexpr int kOffBar = kOffKV + kStages * kStage;
constexpr int kNBar = 24;
constexpr int kOffMisc = kOffBar + kNBar * 8;
constexpr int kSmemBytes = kOffMisc + 128 + 1024;
static_assert(kStage % 1024 == 0, "swizzled operands need 1 KB alignment");
static_assert(kSmemBytes <= 227 * 1024, "shared memory of one CTA");
static_assert((V4A_MAX_SEQ + 1) * 4 <= kStage, "the plan's prefix sums use a stage before its first copy");
constexpr uint32_t kTmemCols = 512;

// Softmax of a query's key tiles t0 .. t1 - 1 (t1 <= t0: none). S of a tile appears in tensor
// memory at scol (sfull), P is written over it (arrive_p). A query sees the first `seen` keys (a
// thread without a query, row false, must not hold up its warp); g counts steps. Weights are taken
// against the reference m, and l is their sum. False when a wait gave up.
template <typename ArriveP>
__device__ __forceinline__ bool softmax_steps(const LatentExpandedParams& p, int t0, int t1, int seen, bool row,
                                              uint32_t scol, uint32_t ocol, uint64_t* sfull, int& g, float& m,
                                              float& l, volatile int* abort_flag, ArriveP arrive_p) {
  const float k2 = p.scale * kLog2e;
  const uint64_t k22 = pack2(k2, k2);
  m = -INFINITY;
  l = 0.f;
  for (int t = t0; t < t1; ++t, ++g) {
    if (!tc::mbar_wait(sfull, g & 1, abort_flag, p.err)) return false;
    tc::fence_after_sync();
    float s[128];
#pragma unroll
    for (int i = 0; i < 4; ++i) tc::tmem_ld32(scol + 32 * i, *reinterpret_cast<float(*)[32]>(&s[32 * i]));
    tc::tmem_wait_ld();
    const int here = row ? seen - t * kT : kT;   // keys of the tile that this query sees
    // Weights are floating-point numbers, so the reference m need not be the maximum (it is set
    // 2^16 above it): a tile that every query of the warp sees whole is taken against m as it is,
    // and only if a sum passes 1 is the tile done again with its maxima. So no weight counts for
    // more than 1, and sums overflow only where the plain softmax's would.
    uint32_t pw[64];
    float sum = 0.f;
    bool slow = __any_sync(0xffffffffu, row && (here < kT || m == -INFINITY));
    if (!slow) {
      sum = weights(s, k22, -m, pw);
      slow = __any_sync(0xffffffffu, row && !(sum <= 1.f));
      if (slow) {
#pragma unroll
        for (int i = 0; i < 4; ++i) tc::tmem_ld32(scol + 32 * i, *reinterpret_cast<float(*)[32]>(&s[32 * i]));
        tc::tmem_wait_ld();
      }
    }
    if (slow) {
      if (__any_sync(0xffffffffu, here < kT)) {
#pragma unroll
        for (int i = 0; i < 128; ++i)
          if (i >= here) s[i] = -INFINITY;
      }
      float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
      for (int i = 4; i < 128; ++i) mx[i & 3] = fmaxf(mx[i & 3], s[i]);
      const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * k2;
      float corr = 1.f;
      if (t == t0) {
        m = mt + kRoom;
      } else if (mt > m + kRaise) {
        corr = fast_exp2(m - (mt + kRoom));   // 0 from -inf
        m = mt + kRoom;
      }
      if (t > t0 && __any_sync(0xffffffffu, corr != 1.f)) {
        // S of this tile is done, and with it every product issued before it
        l *= corr;
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {
          float o[32];
          tc::tmem_ld32(ocol + 32 * i, o);
          tc::tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 32; ++c) o[c] *= corr;
          st32(ocol + 32 * i, o);
        }
      }
      sum = weights(s, k22, m == -INFINITY ? 0.f : -m, pw);
    }
    l += sum;
    tc::tmem_st32(scol, *reinterpret_cast<const uint32_t(*)[32]>(&pw[0]));
    tc::tmem_st32(scol + 32, *reinterpret_cast<const uint32_t(*)[32]>(&pw[32]));
    tc::tmem_wait_st();
    tc::fence_before_sync();
    __syncwarp();
    arrive_p();
  }
  return true;
}

// One piece of work of a pair: queries qa + q0 .. of a sequence (nq in all), head h, keys
// ka .. ka + nk - 1, key tiles t0 .. t1 - 1 of the item's.
struct Piece {
  int qa, nq, ka, nk, q0, h;
  int t0, t1;
  int end[2];                        // where the piece's steps end for each query tile (t0: none)
  int whole, slot;                   // every tile of the item; where a partial result goes
  int job_last;                      // the second piece of an item posts its merge: the last
                                     // pair that holds a piece of it, -1 otherwise
  __device__ __forceinline__ int seen(const LatentExpandedParams& p, int i) const {   // keys of query i
    return i >= nq ? 0 : p.causal ? max(0, min(nk, nk - nq + i + 1)) : nk;
  }
};

// A sequence's blocks of 512 queries and their key tiles (at least one each, so that queries
// without a key are answered too).
struct Seq {
  int qa, nq, ka, nk, blocks;
  __device__ __forceinline__ Seq(const LatentExpandedParams& p, int b) {
    qa = cu_at(p.cu_q, b, p.n_q);
    nq = max(cu_at(p.cu_q, b + 1, p.n_q) - qa, 0);
    ka = cu_at(p.cu_k, b, p.n_k);
    nk = max(cu_at(p.cu_k, b + 1, p.n_k) - ka, 0);
    blocks = (nq + kItem - 1) / kItem;
  }
  __device__ __forceinline__ int tiles(const LatentExpandedParams& p, int blk) const {
    const int last = min((blk + 1) * kItem, nq) - 1;
    const int seen = p.causal ? max(0, min(nk, nk - nq + last + 1)) : nk;
    return max(1, (seen + kT - 1) / kT);
  }
  // Steps of one head, p.setup a block included (what starting an item is worth): the last block,
  // and before it blocks whose tiles fall by kItem / kT each until they reach one.
  __device__ __forceinline__ int steps(const LatentExpandedParams& p) const {
    if (blocks == 0) return 0;
    const int last = tiles(p, blocks - 1), full = blocks - 1;
    if (full == 0 || !p.causal) return (last + p.setup) * blocks;
    const int top = tiles(p, full - 1), d = kItem / kT;
    const int falling = min(full, (top - 1) / d + 1);            // blocks of more than one tile, and the next
    return last + falling * top - d * (falling * (falling - 1) / 2) + (full - falling) + p.setup * blocks;
  }
};

// Walks a pair's part of the line.
struct Walk {
  int x, x1, pair, per;
  int b, base;                       // current sequence and the steps before it
  int blk, blk_base;                 // current block and the steps before it
  __device__ __forceinline__ void begin(const LatentExpandedParams& p, const int32_t* pre) {
    const int total = pre[p.n_seq];
    pair = blockIdx.x >> 1;
    per = latent_per_team(total, p.pairs);
    x = min(pair * per, total);
    x1 = min(x + per, total);
    b = x < x1 ? latent_seq_at(pre, p.n_seq, x) : 0;
    base = x < x1 ? pre[b] : 0;
    blk = -1;
    blk_base = base;
  }
  __device__ __forceinline__ bool next(const LatentExpandedParams& p, Piece& w) {
    if (x >= x1) return false;
    Seq s(p, b);
    while (b + 1 < p.n_seq && (s.blocks == 0 || x >= base + s.steps(p) * p.H)) {
      base += s.steps(p) * p.H;
      s = Seq(p, ++b);
      blk = -1;
    }
    if (blk < 0) {
      blk = s.blocks - 1;
      blk_base = base;
    }
    int len = s.tiles(p, blk) + p.setup;
    while (blk > 0 && x >= blk_base + len * p.H) {
      blk_base += len * p.H;
      len = s.tiles(p, --blk) + p.setup;
    }
    const int r = x - blk_base;
    w.qa = s.qa;
    w.nq = s.nq;
    w.ka = s.ka;
    w.nk = s.nk;
    w.q0 = blk * kItem;
    w.h = r / len;
    const int from = r - w.h * len, take = min(len - from, x1 - x);
    w.t0 = max(0, from - p.setup);
    w.t1 = max(0, from + take - p.setup);
    w.whole = take == len;
    w.slot = (pair << 1) + (from == 0 ? 1 : 0);
    const int x0 = x - from;
    w.job_last = from > 0 && (pair - 1) * per <= x0 ? (x0 + len - 1) / per : -1;
    for (int i = 0; i < 2; ++i) {
      const int first = w.q0 + i * (kItem / 2), last = min(first + kItem / 2, w.nq) - 1;
      w.end[i] = last < first ? w.t0 : max(w.t0, min(w.t1, (w.seen(p, last) + kT - 1) / kT));
    }
    x += take;
    return true;
  }
};

__global__ void __launch_bounds__(kThreads, 1)
    latent_expanded_tc(const __grid_constant__ LatentExpandedParams p, const __grid_constant__ CUtensorMap qmap,
                         const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap pmap,
                         const __grid_constant__ CUtensorMap vmap) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* qbuf = sm + kOffQ;                    // [2 tiles][3 blocks]
  uint8_t* kvbuf = sm + kOffKV;                  // [stages]: keys [3][64 rows], values [128 rows]
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + kOffBar);
  // this CTA's copies have landed
  uint64_t* qfull = bars;                        // [2] by tile
  uint64_t* full = bars + 2;                     // [3] by stage
  // both CTAs' have (used in rank 0)
  uint64_t* qready = bars + 5;                   // [2]
  uint64_t* ready = bars + 7;                    // [3]
  // products done (signalled in both CTAs)
  uint64_t* qempty = bars + 10;                  // [2]
  uint64_t* empty = bars + 12;                   // [3]
  uint64_t* sfull = bars + 15;                   // [2]
  uint64_t* ofull = bars + 17;                   // [2]
  // softmax warps of both CTAs (used in rank 0)
  uint64_t* pfull = bars + 19;                   // [2]
  uint64_t* oempty = bars + 21;                  // [2]
  uint64_t* done = bars + 23;
  int* misc = reinterpret_cast<int*>(sm + kOffMisc);
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(misc);
  volatile int* abort_flag = misc + 1;
  int32_t* warp_tot = misc + 4;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)tc::cluster_rank();
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(qfull + i, 1);
      tc::mbar_init(qready + i, 2);
      tc::mbar_init(qempty + i, 1);
      tc::mbar_init(sfull + i, 1);
      tc::mbar_init(ofull + i, 1);
      tc::mbar_init(pfull + i, 8);
      tc::mbar_init(oempty + i, 8);
    }
    for (int i = 0; i < kStages; ++i) {
      tc::mbar_init(full + i, 1);
      tc::mbar_init(ready + i, 2);
      tc::mbar_init(empty + i, 1);
    }
    tc::mbar_init(done, 1);
    *abort_flag = 0;
    tc::fence_mbar_init();
  }
  if (warp == 9) tc::tmem_alloc_pair(tmem_at, kTmemCols);
  pdl_wait();
  Walk walk;
  Piece w{};
  {
    int32_t* pre = reinterpret_cast<int32_t*>(kvbuf);
    seq_prefix(p.n_seq, pre, warp_tot, [&](int b) { return Seq(p, b).steps(p) * p.H; });
    walk.begin(p, pre);
  }
  tc::fence_proxy_async();     // the prefix sums' buffer is the copies' next
  tc::fence_before_sync();
  __syncthreads();
  tc::cluster_sync();          // the other CTA's barriers and tensor memory are set up
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_at;

  // 384 threads start with 168 registers; the copy and product warps' share goes to the
  // softmax warps (2 x 192 + 120 = 3 x 168)
  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
    // ------------------------------------------------------------- softmax and output
    const int tile = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t scol = tmem + lane_base + tile * 128, ocol = scol + 256;
    const uint32_t p_at = tc::map_rank(pfull + tile, 0), o_at = tc::map_rank(oempty + tile, 0);
    int g = 0, items = 0;
    bool posted = p.split == 0;
    auto post = [&](bool piece) {                 // each pair posts one merge job, empty or not
      if (tid == 0 && rank == 0 && !posted) {
        int32_t* job = p.part_job + 8 * (blockIdx.x >> 1);
        const bool have = piece && w.job_last >= 0;
        *reinterpret_cast<int4*>(job) = make_int4(have ? min(kItem, w.nq - w.q0) : 0, w.qa + w.q0, w.h, w.job_last);
      }
      posted = true;
    };
    while (walk.next(p, w)) {
      post(true);
      const int mine = tile * 256 + rank * kT + row, qi = w.q0 + mine;
      const bool any = w.end[tile] > w.t0, store = qi < w.nq;
      float m, l;
      if (!softmax_steps(p, w.t0, w.end[tile], w.seen(p, qi), store, scol, ocol, sfull + tile, g, m, l, abort_flag,
                         [&] { if (lane == 0) tc::mbar_arrive_cluster(p_at); }))
        break;
      if (any) {
        if (!tc::mbar_wait(ofull + tile, items & 1, abort_flag, p.err)) break;
        tc::fence_after_sync();
        ++items;
      }
      const float inv = !w.whole ? 1.f : l == 0.f ? 0.f : 1.f / l;
      const int64_t at = (int64_t)w.slot * kItem + mine;
      uint4* out = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(p.out) +
                                            ((int64_t)(w.qa + qi) * p.H + w.h) * kT);
      float4* part = reinterpret_cast<float4*>(p.part_o + at * kT);
      if (!w.whole && store) *reinterpret_cast<float2*>(p.part_ml + at * 2) = make_float2(m, l);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float o[32];
        if (any) {
          tc::tmem_ld32(ocol + 32 * i, o);
          tc::tmem_wait_ld();
        } else {
#pragma unroll
          for (int c = 0; c < 32; ++c) o[c] = 0.f;
        }
        if (!store) continue;
        if (w.whole) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
            out[4 * i + c] = make_uint4(pack_bf16(o[8 * c] * inv, o[8 * c + 1] * inv),
                                        pack_bf16(o[8 * c + 2] * inv, o[8 * c + 3] * inv),
                                        pack_bf16(o[8 * c + 4] * inv, o[8 * c + 5] * inv),
                                        pack_bf16(o[8 * c + 6] * inv, o[8 * c + 7] * inv));
        } else if (any) {
#pragma unroll
          for (int c = 0; c < 8; ++c)
            part[8 * i + c] = make_float4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
        }
      }
      if (any) {
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive_cluster(o_at);
      }
    }
    post(false);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 120;");
  }
  if (warp == 8) {
    // ------------------------------------------------------------------------ copies
    if (lane == 0) {
      int s = 0, use = 0;                         // stage, and how often the ring was passed
      int nq[2] = {0, 0}, nkv = 0;
      bool ok = true;
      auto wait = [&](uint64_t* bar, int parity) {
        if (ok) ok = tc::mbar_wait(bar, parity, abort_flag, p.err);
        return ok;
      };
      auto load_q = [&](int i) {
        if (w.end[i] <= w.t0 || (nq[i] > 0 && !wait(qempty + i, (nq[i] - 1) & 1))) return;
        tc::mbar_arrive_tx(qfull + i, 3 * kBlk);
        for (int b = 0; b < 3; ++b)
          tma_3d(qbuf + (3 * i + b) * kBlk, &qmap, b * 128, w.h, w.qa + w.q0 + i * 256 + rank * kT, qfull + i);
        ++nq[i];
      };
      while (ok && walk.next(p, w)) {
        const int end = max(w.end[0], w.end[1]);
        for (int t = w.t0; t < end && ok; ++t) {
          const int tok = w.ka + t * kT;
          uint8_t* st = kvbuf + s * kStage;
          if (use > 0) wait(empty + s, (use - 1) & 1);
          if (t == w.t0 && ok) load_q(0);
          if (!ok) break;
          tc::mbar_arrive_tx(full + s, kStage);
          tma_3d(st, &kmap, 0, w.h, tok + rank * 64, full + s);
          tma_3d(st + kHalf, &kmap, 128, w.h, tok + rank * 64, full + s);
          tma_3d(st + 2 * kHalf, &pmap, 0, 0, tok + rank * 64, full + s);
          tma_3d(st + 3 * kHalf, &vmap, rank * 128, w.h, tok, full + s);
          ++nkv;
          if (t == w.t0) load_q(1);
          if (++s == kStages) { s = 0; ++use; }
        }
      }
      if (*abort_flag) {                          // leave no copy in flight
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (nq[i] > 0) tc::mbar_wait_drain(qfull + i, (nq[i] - 1) & 1);
        for (int k = nkv > kStages ? nkv - kStages : 0; k < nkv; ++k)
          tc::mbar_wait_drain(full + k % kStages, (k / kStages) & 1);
      }
    }
    __syncwarp();
  } else if (warp == 11) {
    // --------------------------------------------------------------- copies that landed
    int s = 0, use = 0;
    int nq[2] = {0, 0};
    bool ok = true;
    auto relay = [&](uint64_t* landed, uint32_t parity, uint64_t* ready, bool wrote = false) {
      if (ok) ok = __all_sync(0xffffffffu, tc::mbar_wait(landed, parity, abort_flag, p.err));
      if (!ok || lane != 0) return;
      const uint32_t at = tc::map_rank(ready, 0);
      if (wrote) tc::mbar_arrive_cluster_release(at); else tc::mbar_arrive_cluster(at);
    };
    while (ok && walk.next(p, w)) {
      const int end = max(w.end[0], w.end[1]);
      for (int t = w.t0; t < end && ok; ++t) {
        if (t == w.t0 && w.end[0] > t) relay(qfull, nq[0]++ & 1, qready);
        const int valid = w.nk - t * kT;
        if (valid < kT) {                          // 0 times what lies behind the keys must be 0
          if (ok) ok = __all_sync(0xffffffffu, tc::mbar_wait(full + s, use & 1, abort_flag, p.err));
          uint8_t* v = kvbuf + s * kStage + 3 * kHalf;
          if (ok)
            for (int o = valid * 128 + lane * 16; o < kBlk; o += 512)
              *reinterpret_cast<uint4*>(v + o) = make_uint4(0, 0, 0, 0);
          tc::fence_proxy_async();
          __syncwarp();
        }
        relay(full + s, use & 1, ready + s, valid < kT);
        if (t == w.t0 && w.end[1] > t) relay(qfull + 1, nq[1]++ & 1, qready + 1);
        if (++s == kStages) { s = 0; ++use; }
      }
    }
    __syncwarp();
  } else if (warp == 9 && rank == 0) {
    // ---------------------------------------------------------------------- products
    constexpr uint32_t idesc_s = tc::idesc_bf16(2 * kT, kT);
    constexpr uint32_t idesc_o = tc::idesc_bf16(2 * kT, kT, false, true);
    const uint32_t ut = tc::uniform(tmem), kv = tc::uniform(tc::smem_u32(kvbuf));
    const uint32_t q_lo = tc::sdesc_lo(tc::uniform(tc::smem_u32(qbuf)), 16);
    int s = 0, use = 0;                           // stage of step t
    int nq[2] = {0, 0}, gp[2] = {0, 0};           // items and products P V of each tile
    bool ok = true;
    auto wait_all = [&](uint64_t* bar, uint32_t parity) {
      if (ok) ok = __all_sync(0xffffffffu, tc::mbar_wait(bar, parity, abort_flag, p.err));
      return ok;
    };
    auto commit = [&](uint64_t* bar) {
      if (ok && tc::elect_one()) tc::mma_commit_pair(bar);
      __syncwarp();
    };
    // S of tile i with the keys of stage ks (ready)
    auto issue_s = [&](int i, int ks) {
      const uint32_t k_lo = tc::uniform(tc::sdesc_lo(kv + ks * kStage, 16));
      const uint32_t a_lo = q_lo + ((i * 3 * kBlk) >> 4), d = ut + i * 128;
      if (ok && tc::elect_one()) {
#pragma unroll
        for (int b = 0; b < 3; ++b) {
#pragma unroll
          for (int k = 0; k < 4; ++k)              // 16 dims, 32 bytes
            tc::mma_bf16_pair_lo<idesc_s>(d, a_lo + ((b * kBlk) >> 4) + 2 * k, k_lo + ((b * kHalf) >> 4) + 2 * k,
                                          (b | k) ? 1u : 0u);
        }
        tc::mma_commit_pair(sfull + i);
      }
      __syncwarp();
    };
    // One warp issues everything in this order, P V of a tile, its next S, then the other tile's:
    // the tiles stay out of step, one's softmax running during the other's products. (Issued by a
    // warp each they fall into step, and the pipe idles during both softmaxes.)
    while (ok && walk.next(p, w)) {
      const int end = max(w.end[0], w.end[1]);
      if (end == w.t0) continue;
      wait_all(ready + s, use & 1);
#pragma unroll
      for (int i = 0; i < 2; ++i) {                // the first step's logits
        if (w.end[i] == w.t0 || !wait_all(qready + i, nq[i] & 1)) continue;
        tc::fence_after_sync();
        issue_s(i, s);
        if (w.end[i] == w.t0 + 1) commit(qempty + i);
      }
      for (int t = w.t0; t < end && ok; ++t) {
        const int s1 = s + 1 == kStages ? 0 : s + 1, use1 = s1 == 0 ? use + 1 : use;
        const uint32_t v_lo = tc::uniform(tc::sdesc_lo(kv + s * kStage + 3 * kHalf, 16));
        const uint32_t acc = tc::uniform(t > w.t0);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (t < w.end[i]) {
            if (!wait_all(pfull + i, gp[i] & 1)) break;
            if (t == w.t0 && nq[i] > 0 && !wait_all(oempty + i, (nq[i] - 1) & 1)) break;
            tc::fence_after_sync();
            if (tc::elect_one()) {
#pragma unroll
              for (int k = 0; k < 8; ++k)          // 16 keys: 8 columns of P, 2 KB of V
                tc::mma_bf16_ta_pair_lo<idesc_o>(ut + 256 + i * 128, ut + i * 128 + 8 * k, v_lo + ((k * 2048) >> 4),
                                                 k > 0 ? 1u : acc);
              if (t + 1 == w.end[i]) tc::mma_commit_pair(ofull + i);
            }
            __syncwarp();
            ++gp[i];
          }
          if (i == 0 && t + 1 < end) {
            wait_all(ready + s1, use1 & 1);
            tc::fence_after_sync();
          }
          if (i == 1) commit(empty + s);
          if (t + 1 < w.end[i]) {
            issue_s(i, s1);
            if (t + 2 == w.end[i]) commit(qempty + i);
          }
        }
        s = s1;
        use = use1;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (w.end[i] > w.t0) ++nq[i];
    }
    if (tc::elect_one()) {
      tc::mma_commit_pair(done);
      tc::mbar_wait_drain(done, 0);
    }
    __syncwarp();
  }

  tc::fence_before_sync();
  __syncthreads();
  if (tid == 0 && rank != 0) tc::mbar_wait_drain(done, 0);       // the last signal of the products
  __syncwarp();
  tc::cluster_sync();          // the other CTA has no more use for this one's memory
  if (warp == 9) {
    tc::fence_after_sync();
    tc::tmem_dealloc_pair(tmem, kTmemCols);
  }
}

// The results of items whose tiles fell to several pairs, as in the absorbed form's merge. Block
// (pair, rows) does the job that the pair posted; a warp a query.
constexpr int kMergeWarps = 8;

__global__ void __launch_bounds__(32 * kMergeWarps)
    latent_expanded_merge(const __grid_constant__ LatentExpandedParams p) {
  pdl_wait();
  const int lane = threadIdx.x & 31, r = blockIdx.y * kMergeWarps + (threadIdx.x >> 5), g = blockIdx.x;
  const int4 job = *reinterpret_cast<const int4*>(p.part_job + 8 * g);   // rows, first row, head, last pair
  if (r >= job.x) return;
  const int last = job.w;
  // pair g - 1's piece begins the item (slot 1), the others begin inside it (slot 0)
  auto at = [&](int i) { return (int64_t)((i << 1) + (i == g - 1 ? 1 : 0)) * kItem + r; };
  float m = -INFINITY;
  for (int i = g - 1 + lane; i <= last; i += 32) m = fmaxf(m, p.part_ml[at(i) * 2]);
  m = warp_max(m);
  const float ref = m == -INFINITY ? 0.f : m;
  float l = 0.f;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = g - 1; i0 <= last; i0 += 32) {
    // a lane a piece: its weight, 0 for a range without a key (whose o was not written)
    const int i = i0 + lane;
    float w = 0.f;
    if (i <= last) {
      const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + at(i) * 2);
      if (ml.x != -INFINITY || ml.y != 0.f) w = exp2f(ml.x - ref);
      l = fmaf(w, ml.y, l);
    }
    const int cnt = min(32, last - i0 + 1);
#pragma unroll 4
    for (int k = 0; k < cnt; ++k) {
      const float wk = __shfl_sync(0xffffffffu, w, k);
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (wk != 0.f) v = *reinterpret_cast<const float4*>(p.part_o + at(i0 + k) * kT + lane * 4);
      a.x = fmaf(wk, v.x, a.x);
      a.y = fmaf(wk, v.y, a.y);
      a.z = fmaf(wk, v.z, a.z);
      a.w = fmaf(wk, v.w, a.w);
    }
  }
  l = warp_sum(l);
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint2* out = reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(p.out) +
                                        ((int64_t)(job.y + r) * p.H + job.z) * kT);
  out[lane] = make_uint2(pack_bf16(a.x * inv, a.y * inv), pack_bf16(a.z * inv, a.w * inv));
}

}  // namespace

cudaError_t launch_latent_expanded_tc(const LatentExpandedParams& p, cudaStream_t st) {
  // boxes of 128 queries, 64 keys, 128 values; without keys nothing is read through their maps
  CUtensorMap qmap, kmap, pmap, vmap;
  const uint64_t H = (uint64_t)p.H, nk = p.n_k > 0 ? (uint64_t)p.n_k : 1;
  const bool none = p.n_k == 0;
  const void *k = none ? p.q : p.k, *pe = none ? p.q : p.k_pe, *v = none ? p.q : p.v;
  const uint64_t kts = none ? 256 : p.k_ts * 2, khs = none ? 256 : p.k_hs * 2, vts = none ? 256 : p.v_ts * 2,
                 vhs = none ? 256 : p.v_hs * 2, pts = none ? 128 : p.pe_ts * 2;
  if (!encode_byte_rows_map3(&qmap, p.q, 384, H, 384, (uint64_t)p.n_q, H * 384, 128, kT) ||
      !encode_byte_rows_map3(&kmap, k, 256, H, khs, nk, kts, 128, kT / 2) ||
      !encode_byte_rows_map3(&vmap, v, 256, H, vhs, nk, vts, 128, kT) ||
      !encode_byte_rows_map3(&pmap, pe, 128, 1, pts, nk, pts, 128, kT / 2))
    return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * p.pairs));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaError_t e =
      cudaFuncSetAttribute(latent_expanded_tc, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return e;
  e = cudaLaunchKernelEx(&cfg, latent_expanded_tc, p, qmap, kmap, pmap, vmap);
  if (e != cudaSuccess || !p.split) return e;
  return launch_pdl(latent_expanded_merge, dim3((unsigned)p.pairs, kItem / kMergeWarps), dim3(32 * kMergeWarps), 0, st,
                    p);
}

}  // namespace v4a
