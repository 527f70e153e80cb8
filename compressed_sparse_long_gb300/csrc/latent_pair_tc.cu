// Absorbed latent attention by pairs of CTAs (cta_group::2), for sequences with more than 64
// (token, head) rows: 128 heads at decode, chunks of new tokens.
//
//   S = Q K^T     M = 128 rows (64 a CTA), N = 128 keys, K = 576           (36 products)
//   P = 2^(scale log2(e) S - m), bf16
//   O += P V      M = 128 rows, N = 2 x 256 dims, K = 128 keys             (16 products)
// A unit is 128 consecutive rows of a sequence, a key tile 128 consecutive cache rows (half a
// page). As S's B operand each CTA copies 64 of the tile's keys in full (72 KB); as P V's B operand
// half of the dims of all 128 keys (64 KB): what the other CTA holds, the products read there. With
// 64 rows a CTA, S (64 keys beside 64 keys on the lanes) takes 64 tensor-memory columns, twice, and
// O 256. Keys and values have buffers of their own, so the next tile's S runs during this tile's
// softmax, and its keys are copied block by block as S releases them.
//
// Bound: the products' shared-memory reads (S 4 KB, P V 6 KB a product and CTA), then HBM. The
// kernel for single CTAs (latent_tc.cu) spends 3890 cycles on products for 64 rows x 128 keys and
// cannot overlap the softmax with them.
//
// Roles in each CTA: warps 0-3 softmax and output (thread: a row and one half of the tile's keys;
// its partner, 64 threads on, has the other half), warp 4 copies of Q and K, which report to the
// barriers of rank 0, warp 5 copies of V, warp 6 of rank 0 the pair's products.
#include "kernels.h"
#include "latent.h"
#include "tc.cuh"

namespace v4a {
namespace {

constexpr int kRows = 64, kTK = 128, kC = 512, kW = 576;         // rows of a CTA
constexpr int kThreads = 256;
constexpr int kBlk = 64 * 128, kVBlk = kTK * 128;                // 64 and 128 rows of 128 bytes
constexpr int kOffQ = 0, kOffK = 9 * kBlk, kOffV = kOffK + 9 * kBlk, kOffP = kOffV + 4 * kVBlk;
constexpr int kOffF = kOffP + 2 * kBlk;                          // red[2][128] floats
constexpr int kOffBar = kOffF + 256 * 4;
constexpr int kNBar = 24;
constexpr int kOffMisc = kOffBar + kNBar * 8;
constexpr int kSmemBytes = kOffMisc + 128 + 1024;
static_assert(kOffV % 1024 == 0 && kOffP % 1024 == 0, "swizzled operands need 1 KB alignment");
static_assert(kSmemBytes <= 227 * 1024, "shared memory of one CTA");
static_assert((V4A_MAX_SEQ + 1) * 4 <= kBlk, "the plan's prefix sums use a key block before its first copy");
constexpr uint32_t kSCol = 0, kOCol = 128, kTmemCols = 512;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRaise = 8.0f;                                   // log2 units
constexpr float kLimit = 65536.0f;                               // of a tile's sum

__device__ __forceinline__ float fast_exp2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ void st32(uint32_t taddr, const float (&v)[32]) {
  uint32_t u[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) u[i] = __float_as_uint(v[i]);
  tc::tmem_st32(taddr, u);
}
// A copy into this CTA that reports to a barrier of this CTA.
__device__ __forceinline__ void tma_2d(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          tc::smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(tc::smem_u32(bar))
      : "memory");
}
// A copy into this CTA that reports to a barrier of either CTA of the pair (cluster address).
__device__ __forceinline__ void tma_2d_pair(void* dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3}], "
      "[%4];" ::"r"(tc::smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
// 2^(k2 s + nm) of a thread's 64 logits in place; returns their sum.
__device__ __forceinline__ float weights(float (&s)[64], float k2, float nm) {
  float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 64; ++i) {
    s[i] = fast_exp2(fmaf(s[i], k2, nm));
    sum[i & 3] += s[i];
  }
  return (sum[0] + sum[1]) + (sum[2] + sum[3]);
}

__device__ __forceinline__ int64_t tile_slot(const LatentAttnParams& p, int seq, int tile) {
  return slot_of(p.cache, seq, (int64_t)tile * kTK);
}

__global__ void __launch_bounds__(kThreads, 1)
    latent_attn_pair(const __grid_constant__ LatentAttnParams p, const __grid_constant__ CUtensorMap qmap,
                     const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* qbuf = sm + kOffQ;                                    // [9][64 rows]
  uint8_t* kbuf = sm + kOffK;                                    // [9][64 keys]
  uint8_t* vbuf = sm + kOffV;                                    // [2 halves of the dims][2][128 keys]
  uint8_t* pbuf = sm + kOffP;                                    // [2 halves of the keys][64 rows]
  float* red = reinterpret_cast<float*>(sm + kOffF);             // [2][128]
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + kOffBar);
  // both CTAs' copies have landed (used in rank 0)
  uint64_t* qfull = bars;
  uint64_t* kfull = bars + 1;                                    // [5] blocks 0-1, 2-3, 4-5, 6-7, 8
  // products done (signalled in both CTAs)
  uint64_t* qempty = bars + 6;
  uint64_t* kempty = bars + 7;                                   // [5]
  uint64_t* sfull = bars + 12;                                   // [2] by S buffer
  uint64_t* pvdone = bars + 14;
  uint64_t* done = bars + 15;
  // softmax warps of both CTAs (used in rank 0)
  uint64_t* pfull = bars + 16;
  uint64_t* oempty = bars + 17;
  // this CTA's own
  uint64_t* vfull = bars + 18;
  uint64_t* redb = bars + 19;
  int* misc = reinterpret_cast<int*>(sm + kOffMisc);
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(misc);
  volatile int* abort_flag = misc + 1;
  volatile int* raised = misc + 2;                               // [2] by tile parity: tile + 1
  int32_t* warp_tot = misc + 4;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)tc::cluster_rank();
  if (tid == 0) {
    tc::mbar_init(qfull, 1);
    tc::mbar_init(qempty, 1);
    for (int i = 0; i < 5; ++i) {
      tc::mbar_init(kfull + i, 1);
      tc::mbar_init(kempty + i, 1);
    }
    tc::mbar_init(sfull, 1);
    tc::mbar_init(sfull + 1, 1);
    tc::mbar_init(pvdone, 1);
    tc::mbar_init(done, 1);
    tc::mbar_init(pfull, 8);
    tc::mbar_init(oempty, 8);
    tc::mbar_init(vfull, 1);
    tc::mbar_init(redb, 4);
    *abort_flag = 0;
    raised[0] = raised[1] = 0;
    tc::fence_mbar_init();
  }
  if (warp == 6) tc::tmem_alloc_pair(tmem_at, kTmemCols);
  pdl_wait();
  LatentWalk walk;
  LatentPiece w;
  {
    int32_t* pre = reinterpret_cast<int32_t*>(kbuf);
    walk.begin(p, pre, latent_prefix(p, pre, warp_tot), blockIdx.x >> 1);
  }
  tc::fence_proxy_async();     // the prefix sums' buffer is the copies' next
  tc::fence_before_sync();
  __syncthreads();
  tc::cluster_sync();          // the other CTA's barriers and tensor memory are set up
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_at;

  if (warp < 4) {
    // ------------------------------------------------------------- softmax and output
    const int r = tid & 63, half = tid >> 6;      // row of this CTA, half of the keys (and dims)
    const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
    const uint32_t p_at = tc::map_rank(pfull, 0), o_at = tc::map_rank(oempty, 0);
    const float k2 = p.scale * kLog2e;
    int g = 0, ru = 0;
    bool ok = true, posted = false;
    auto group_sync = [&]() -> bool {             // the four warps
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(redb);
      const bool got = tc::mbar_wait(redb, ru & 1, abort_flag, p.err);
      ++ru;
      return got;
    };
    while (ok && walk.next(p, w)) {
      if (tid == 0 && rank == 0 && !posted) walk.post(p, &w);
      posted = true;
      if (w.rows == 0) continue;
      const int mine = rank * kRows + r;
      const bool row = mine < w.rows;
      int64_t vis = 0;
      if (row) {
        const int64_t pos = w.start + (w.row0 + mine - w.seq_row0) / p.H;
        vis = max((int64_t)0, min(pos, p.max_pos) + 1);
        if (half == 0 && (pos > p.max_pos || pos < 0)) raise_err(p.err, V4A_DEV_BAD_POS);
      }
      float m = -INFINITY, l = 0.f;               // the row's reference (log2 units), this half's sum
      for (int t = w.tile0; t < w.tile1; ++t, ++g) {
        const int64_t x0 = (int64_t)t * kTK;
        const int valid = tile_slot(p, w.seq, t) < 0 ? 0 : (int)min((int64_t)kTK, w.keys - x0);
        // keys of this half that the row sees
        const int here = row ? (int)min((int64_t)64, max((int64_t)0, min(vis - x0, (int64_t)valid) - 64 * half)) : 64;
        // (alike in all four warps but for the reference, which the partners share)
        bool slow = valid < kTK || w.keys0 < x0 + kTK || t == w.tile0;
        if (!tc::mbar_wait(sfull + (g & 1), (g >> 1) & 1, abort_flag, p.err)) { ok = false; break; }
        tc::fence_after_sync();
        const uint32_t scol = tmem + lane_base + kSCol + (g & 1) * 64;
        float s[64];
        tc::tmem_ld32(scol, *reinterpret_cast<float(*)[32]>(&s[0]));
        tc::tmem_ld32(scol + 32, *reinterpret_cast<float(*)[32]>(&s[32]));
        tc::tmem_wait_ld();
        float sum = 0.f;
        if (!slow) {
          // against the reference as it is, unless a sum passes kLimit (see latent_tc.cu) or a row
          // has none yet; the warps agree on that
          sum = weights(s, k2, -m);
          const bool over = __any_sync(0xffffffffu, row && (!(sum <= kLimit) || m == -INFINITY));
          if (over && lane == 0) raised[g & 1] = g + 1;
          if (!group_sync()) { ok = false; break; }
          slow = raised[g & 1] == g + 1;
          if (slow) {
            tc::tmem_ld32(scol, *reinterpret_cast<float(*)[32]>(&s[0]));
            tc::tmem_ld32(scol + 32, *reinterpret_cast<float(*)[32]>(&s[32]));
            tc::tmem_wait_ld();
          }
        }
        float corr = 1.f;
        if (slow) {
          if (__any_sync(0xffffffffu, here < 64)) {
#pragma unroll
            for (int i = 0; i < 64; ++i)
              if (i >= here) s[i] = -INFINITY;
          }
          float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
          for (int i = 4; i < 64; ++i) mx[i & 3] = fmaxf(mx[i & 3], s[i]);
          float* rb = red + (ru & 1) * 128;
          rb[tid] = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
          if (!group_sync()) { ok = false; break; }
          const float mt = fmaxf(rb[r], rb[r + 64]) * k2;
          if (t == w.tile0) {
            m = mt;
          } else if (mt > m + kRaise) {
            corr = fast_exp2(m - mt);             // 0 from -inf
            m = mt;
          }
          sum = weights(s, k2, m == -INFINITY ? 0.f : -m);
        }
        // the previous tile's P V is done: P may be overwritten, O rescaled
        if (g > 0 && !tc::mbar_wait(pvdone, (g - 1) & 1, abort_flag, p.err)) { ok = false; break; }
        if (t > w.tile0 && __any_sync(0xffffffffu, corr != 1.f)) {
          tc::fence_after_sync();
          l *= corr;
#pragma unroll 1
          for (int i = 0; i < 8; ++i) {
            float o[32];
            tc::tmem_ld32(tmem + lane_base + kOCol + 32 * i, o);
            tc::tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < 32; ++c) o[c] *= corr;
            st32(tmem + lane_base + kOCol + 32 * i, o);
          }
          tc::tmem_wait_st();
        }
        l += sum;
        // P, K-major: this row's 64 keys, rounded to bf16 for the second product
#pragma unroll
        for (int i = 0; i < 8; ++i)
          *reinterpret_cast<uint4*>(pbuf + half * kBlk + tc::sw128_off(r, i)) =
              make_uint4(pack_bf16(s[8 * i], s[8 * i + 1]), pack_bf16(s[8 * i + 2], s[8 * i + 3]),
                         pack_bf16(s[8 * i + 4], s[8 * i + 5]), pack_bf16(s[8 * i + 6], s[8 * i + 7]));
        if (!tc::mbar_wait(vfull, g & 1, abort_flag, p.err)) { ok = false; break; }
        if (tid >= valid) {                       // 0 times whatever lies behind the keys must be 0
#pragma unroll 1
          for (int b = 0; b < 4; ++b)
#pragma unroll
            for (int c = 0; c < 8; ++c)
              *reinterpret_cast<uint4*>(vbuf + b * kVBlk + tc::sw128_off(tid, c)) = make_uint4(0, 0, 0, 0);
        }
        tc::fence_proxy_async();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive_cluster(p_at);
      }
      if (!ok) break;
      const bool any = w.tile1 > w.tile0;
      if (any) {
        float* rb = red + (ru & 1) * 128;
        rb[tid] = l;
        if (!group_sync()) { ok = false; break; }
        l = rb[r] + rb[r + 64];
        if (!tc::mbar_wait(pvdone, (g - 1) & 1, abort_flag, p.err)) { ok = false; break; }
        tc::fence_after_sync();
      }
      const float inv = !w.whole ? 1.f : l == 0.f ? 0.f : 1.f / l;
      const int64_t at = (int64_t)w.slot * (2 * kRows) + mine;
      if (!w.whole && half == 0) *reinterpret_cast<float2*>(p.part_ml + at * 2) = make_float2(m, l);
#pragma unroll 1
      for (int i = 0; i < 8; ++i) {               // 32 dims of each of the two products' four parts
        const int d = (i >> 2) * 256 + half * 128 + (i & 3) * 32;
        float o[32];
        if (any) {
          tc::tmem_ld32(tmem + lane_base + kOCol + 32 * i, o);
          tc::tmem_wait_ld();
        } else {
#pragma unroll
          for (int c = 0; c < 32; ++c) o[c] = 0.f;
        }
        if (!row) continue;
        if (w.whole) {
          uint4* out = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(p.out) +
                                                (int64_t)(w.row0 + mine) * kC + d);
#pragma unroll
          for (int c = 0; c < 4; ++c)
            out[c] = make_uint4(pack_bf16(o[8 * c] * inv, o[8 * c + 1] * inv),
                                pack_bf16(o[8 * c + 2] * inv, o[8 * c + 3] * inv),
                                pack_bf16(o[8 * c + 4] * inv, o[8 * c + 5] * inv),
                                pack_bf16(o[8 * c + 6] * inv, o[8 * c + 7] * inv));
        } else if (any) {
          float4* part = reinterpret_cast<float4*>(p.part_o + at * kC + d);
#pragma unroll
          for (int c = 0; c < 8; ++c) part[c] = make_float4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
        }
      }
      if (any) {
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive_cluster(o_at);
      }
    }
    if (tid == 0 && rank == 0 && !posted) walk.post(p, nullptr);
  } else if (warp == 4) {
    // ----------------------------------------------------------------- copies of Q and K
    if (lane == 0) {
      const uint32_t q_at = tc::map_rank(qfull, 0);
      int g = 0, u = 0, nk = 0;
      bool ok = true;
      while (ok && walk.next(p, w)) {
        if (w.tile0 >= w.tile1) continue;
        if (u > 0 && !tc::mbar_wait(qempty, (u - 1) & 1, abort_flag, p.err)) break;
        if (rank == 0) tc::mbar_arrive_tx(qfull, 2 * 9 * kBlk);
        for (int b = 0; b < 9; ++b) tma_2d_pair(qbuf + b * kBlk, &qmap, b * 128, w.row0 + rank * kRows, q_at);
        ++u;
        for (int t = w.tile0; t < w.tile1 && ok; ++t, ++g) {
          const int64_t slot = tile_slot(p, w.seq, t);
          const bool have = slot >= 0;
          if (!have && rank == 0) slot_ok(slot, p.err);
          const int y = (int)slot + rank * 64;
#pragma unroll
          for (int j = 0; j < 5; ++j) {
            if (g > 0 && ok) ok = tc::mbar_wait(kempty + j, (g - 1) & 1, abort_flag, p.err);
            if (!ok) continue;
            const int nb = j < 4 ? 2 : 1;
            ++nk;
            if (rank == 0) {
              if (have) tc::mbar_arrive_tx(kfull + j, 2 * nb * kBlk);
              else tc::mbar_arrive(kfull + j);
            }
            if (have)
              for (int b = 2 * j; b < 2 * j + nb; ++b)
                tma_2d_pair(kbuf + b * kBlk, &kmap, b * 128, y, tc::map_rank(kfull + j, 0));
          }
          if (ok && t + 1 < w.tile1) {            // this CTA's keys of the next tile into L2
            const int64_t ahead = tile_slot(p, w.seq, t + 1);
            if (ahead >= 0) {
              const uint8_t* rows = reinterpret_cast<const uint8_t*>(p.cache.data) + (ahead + rank * 64) * (kW * 2);
#pragma unroll 1
              for (int i = 0; i < 4; ++i)
                asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(rows + i * (16 * kW * 2)),
                             "r"(16 * kW * 2)
                             : "memory");
            }
          }
        }
      }
      if (*abort_flag && rank == 0) {             // leave no copy in flight (the other CTA waits for this one)
        if (u > 0) tc::mbar_wait_drain(qfull, (u - 1) & 1);
        for (int k = nk > 5 ? nk - 5 : 0; k < nk; ++k) tc::mbar_wait_drain(kfull + k % 5, (k / 5) & 1);
      }
    }
    __syncwarp();
  } else if (warp == 5) {
    // ----------------------------------------------------------------------- copies of V
    if (lane == 0) {
      int g = 0;
      bool ok = true;
      while (ok && walk.next(p, w)) {
        for (int t = w.tile0; t < w.tile1; ++t, ++g) {
          const int64_t slot = tile_slot(p, w.seq, t);
          if (g > 0 && !tc::mbar_wait(pvdone, (g - 1) & 1, abort_flag, p.err)) { ok = false; break; }
          if (slot >= 0) {
            tc::mbar_arrive_tx(vfull, 4 * kVBlk);
            for (int b = 0; b < 4; ++b)           // dims 256 (b / 2) + 128 rank + 64 (b % 2) ..
              tma_2d(vbuf + b * kVBlk, &vmap, (b >> 1) * 512 + rank * 256 + (b & 1) * 128, (int)slot, vfull);
          } else {
            tc::mbar_arrive(vfull);
          }
        }
      }
      if (*abort_flag && g > 0) {                 // leave no copy in flight
        tc::mbar_wait_drain(vfull, (g - 1) & 1);
        tc::mbar_wait_drain(vfull, g & 1);
      }
    }
    __syncwarp();
  } else if (warp == 6 && rank == 0) {
    // ---------------------------------------------------------------------- products
    constexpr uint32_t idesc_s = tc::idesc_bf16(2 * kRows, kTK);
    constexpr uint32_t idesc_o = tc::idesc_bf16(2 * kRows, 256, false, true);
    const uint32_t ut = tc::uniform(tmem);
    const uint32_t q_lo = tc::sdesc_lo(tc::uniform(tc::smem_u32(qbuf)), 16);
    const uint32_t k_lo = tc::sdesc_lo(tc::uniform(tc::smem_u32(kbuf)), 16);
    const uint32_t p_lo = tc::sdesc_lo(tc::uniform(tc::smem_u32(pbuf)), 16);
    const uint32_t v_lo = tc::sdesc_lo(tc::uniform(tc::smem_u32(vbuf)), kVBlk);
    int g = 0, u = 0;                             // tiles of which S was issued; pieces
    bool ok = true;
    auto wait_all = [&](uint64_t* bar, uint32_t parity) {
      if (ok) ok = __all_sync(0xffffffffu, tc::mbar_wait(bar, parity, abort_flag, p.err));
      return ok;
    };
    // S of the next tile into buffer g % 2, releasing its key blocks as it goes
    auto issue_s = [&](bool last) {
      const uint32_t d = tc::uniform(ut + kSCol + (g & 1) * 64);
#pragma unroll
      for (int j = 0; j < 5; ++j) {
        if (!wait_all(kfull + j, g & 1)) continue;
        tc::fence_after_sync();
        if (tc::elect_one()) {
#pragma unroll
          for (int b = 2 * j; b < 2 * j + (j < 4 ? 2 : 1); ++b) {
#pragma unroll
            for (int k = 0; k < 4; ++k)            // 16 dims, 32 bytes
              tc::mma_bf16_pair_lo<idesc_s>(d, q_lo + ((b * kBlk) >> 4) + 2 * k, k_lo + ((b * kBlk) >> 4) + 2 * k,
                                            (b | k) ? 1u : 0u);
          }
          tc::mma_commit_pair(kempty + j);
          if (j == 4) {
            tc::mma_commit_pair(sfull + (g & 1));
            if (last) tc::mma_commit_pair(qempty);
          }
        }
        __syncwarp();
      }
      ++g;
    };
    while (ok && walk.next(p, w)) {
      if (w.tile0 >= w.tile1) continue;
      if (!wait_all(qfull, u & 1)) break;
      issue_s(w.tile0 + 1 == w.tile1);
      for (int t = w.tile0; t < w.tile1 && ok; ++t) {
        const int done_s = g - 1;                  // number of this tile
        if (t + 1 < w.tile1) issue_s(t + 2 == w.tile1);
        if (!wait_all(pfull, done_s & 1)) break;
        if (t == w.tile0 && u > 0 && !wait_all(oempty, (u - 1) & 1)) break;
        tc::fence_after_sync();
        const uint32_t acc = tc::uniform(t > w.tile0);
        if (tc::elect_one()) {
#pragma unroll
          for (int n = 0; n < 2; ++n) {
#pragma unroll
            for (int k = 0; k < 8; ++k)            // 16 keys: 32 bytes of P, 2 KB of V
              tc::mma_bf16_pair_lo<idesc_o>(ut + kOCol + n * 128, p_lo + (((k >> 2) * kBlk) >> 4) + 2 * (k & 3),
                                            v_lo + ((n * 2 * kVBlk + k * 2048) >> 4), k > 0 ? 1u : acc);
          }
          tc::mma_commit_pair(pvdone);
        }
        __syncwarp();
      }
      ++u;
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
  if (warp == 6) {
    tc::fence_after_sync();
    tc::tmem_dealloc_pair(tmem, kTmemCols);
  }
}

}  // namespace

cudaError_t launch_latent_attn_pair(const LatentAttnParams& p, cudaStream_t st) {
  CUtensorMap qmap, kmap, vmap;
  const int64_t rows = (int64_t)p.n_tokens * p.H;
  const int64_t pool_rows = (p.cache.n_pages > 0 ? p.cache.n_pages : 1) * kBlock;
  if (!encode_byte_rows_map(&qmap, p.q, (uint64_t)rows, kW * 2, 128, kRows) ||
      !encode_byte_rows_map(&kmap, p.cache.data, (uint64_t)pool_rows, kW * 2, 128, 64) ||
      !encode_byte_rows_map(&vmap, p.cache.data, (uint64_t)pool_rows, kW * 2, 128, kTK))
    return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * p.plan.ctas));
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
  const cudaError_t e =
      cudaFuncSetAttribute(latent_attn_pair, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return e;
  return cudaLaunchKernelEx(&cfg, latent_attn_pair, p, qmap, kmap, vmap);
}

}  // namespace v4a
