// Absorbed latent attention on tcgen05 tensor cores: bf16 rows of 512 latent + 64 rotary dims.
//
//   S^T = K Q^T           M = 128 keys, N = 64 rows, K = 576   (36 MMAs)
//   P^T = 2^(scale log2(e) S^T - m), bf16
//   O^T += V^T P^T        M = 4 x 128 dims, N = 64, K = 128 keys (32 MMAs), V = the key tile's
//                         first 512 dims
// A unit is 64 consecutive (token, head) rows of a sequence; the key tile is 128 consecutive
// cache rows, half a page, copied by TMA into eight 16 KB column blocks (64 dims each, 128-byte
// swizzle) and a ninth for the rotary dims. One copy serves both products: K-major as the keys,
// MN-major as the values. Keys lie on M (not the rows) because the accumulator of 64 rows x 512
// dims then takes 256 of the 512 tensor-memory columns, and P^T, the second product's B operand,
// goes through 16 KB of shared memory: the rotary block's, dead once S^T is done. Q (72 KB),
// the tile (144 KB) and this reuse fill the SM's shared memory.
//
// Bound: HBM for decode with up to 64 heads (1152 bytes a key for 2 * 64 * 1088 flop); for 128
// heads and chunks the operands' shared-memory reads: an M = 128, N = 64 product reads 6 KB and
// takes 54 (O^T) to 60 (S^T) cycles where the pipe would need 32. A tile then takes 5400 cycles:
// S^T 2160, softmax 930 with 560 of signalling, O^T 1730 (clock marks in a copy of the kernel).
// (One CTA cannot take 128 rows: O^T would fill the tensor memory.) 32 sequences x 32768 tokens, 64
// heads: 197 us with the merge, 6.1 TB/s; 16 sequences of 4616-108051 tokens, 128 heads: 195 us,
// 830 TFLOP/s.
//
// Warps 0-7: softmax and output. A thread holds one key's 32 logits (warps 0-3 rows 0-31, warps
// 4-7 rows 32-63 of the unit). A row's weights are taken against a reference, 2^16 times its
// largest over the first tile; maxima over the keys (redux, and through shared memory) are needed
// again only where a tile is masked or a weight would pass 1, and then the reference is raised
// where a weight passes 2^-8 and the accumulator and sums rescaled. So no weight counts for more
// than 1, and sums overflow only where the plain softmax's would. Warp 8: copies, with the
// next tile requested into L2 a tile ahead. Warp 9: products.
#include "kernels.h"
#include "latent.h"
#include "tc.cuh"

namespace v4a {
namespace {

constexpr int kNR = 64, kTK = 128, kC = 512, kW = 576;
constexpr int kThreads = 320;
constexpr int kQBlock = kNR * 128, kKBlock = kTK * 128;          // 8 KB, 16 KB
constexpr int kOffK = 0, kOffX = 8 * kKBlock, kOffQ = kOffX + kKBlock;
constexpr int kOffF = kOffQ + 9 * kQBlock;
// floats: red_max[2][64][4] red_sum[64][4] mrow[8 warps][32]
constexpr int kNFloats = 512 + 256 + 256;
constexpr int kOffBar = kOffF + kNFloats * 4;
constexpr int kNBar = 20;
constexpr int kOffMisc = kOffBar + kNBar * 8;
constexpr int kSmemBytes = kOffMisc + 192 + 1024;
static_assert(kSmemBytes <= 227 * 1024, "shared memory of one CTA");
static_assert((V4A_MAX_SEQ + 1) * 4 <= kKBlock, "the plan's prefix sums use a key block before its first copy");
constexpr uint32_t kSCol = 0, kOCol = 64, kTmemCols = 512;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRoom = 16.0f, kRaise = -8.0f;                   // log2 units: a reference above its maximum;
                                                                 // a weight that raises it

__device__ __forceinline__ float fast_exp2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float redux_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ void tma_2d(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          tc::smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(tc::smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void st32(uint32_t taddr, const float (&v)[32]) {
  uint32_t u[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) u[i] = __float_as_uint(v[i]);
  tc::tmem_st32(taddr, u);
}

// Sum of v[c] over the 32 lanes; lane c ends with column c's.
__device__ __forceinline__ float reduce_scatter_sum(const float (&v)[32]) {
  const int lane = threadIdx.x & 31;
  float a[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) a[i] = v[i];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int j = 0; j < o; ++j) {
      const float send = up ? a[j] : a[j + o], keep = up ? a[j + o] : a[j];
      a[j] = keep + __shfl_xor_sync(0xffffffffu, send, o);
    }
  }
  return a[0];
}

// Pool row of the first key of a tile, or a negative number when its page is missing or bad.
__device__ __forceinline__ int64_t tile_slot(const LatentAttnParams& p, int seq, int tile) {
  return slot_of(p.cache, seq, (int64_t)tile * kTK);
}

__global__ void __launch_bounds__(kThreads, 1)
    latent_attn_tc(const __grid_constant__ LatentAttnParams p, const __grid_constant__ CUtensorMap qmap,
                   const __grid_constant__ CUtensorMap kmap) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* kbuf = sm + kOffK;
  uint8_t* xbuf = sm + kOffX;                                    // rotary key block, then P^T
  uint8_t* qbuf = sm + kOffQ;
  float* red_max = reinterpret_cast<float*>(sm + kOffF);
  float* red_sum = red_max + 512;
  float* mrow = red_sum + 256;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + kOffBar);
  uint64_t* vfull = bars;                                        // [4] pairs of column blocks
  uint64_t* vempty = bars + 4;                                   // [4]
  uint64_t* xfull = bars + 8;
  uint64_t* pvdone = bars + 9;
  uint64_t* qfull = bars + 10;
  uint64_t* qempty = bars + 11;
  uint64_t* sfull = bars + 12;
  uint64_t* pfull = bars + 13;
  uint64_t* oempty = bars + 14;
  uint64_t* redb = bars + 15;                                    // [2] one per group of 4 warps
  uint64_t* done = bars + 17;
  int* misc = reinterpret_cast<int*>(sm + kOffMisc);
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(misc);
  volatile int* abort_flag = misc + 1;
  volatile int* tile_ok = misc + 2;                              // [2] by tile parity
  volatile int* raised = misc + 4;                               // [2 halves][2 parities] tile + 1
  int32_t* warp_tot = misc + 8;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < 4; ++i) {
      tc::mbar_init(vfull + i, 1);
      tc::mbar_init(vempty + i, 1);
    }
    tc::mbar_init(xfull, 1);
    tc::mbar_init(pvdone, 1);
    tc::mbar_init(qfull, 1);
    tc::mbar_init(qempty, 1);
    tc::mbar_init(sfull, 1);
    tc::mbar_init(pfull, 8);
    tc::mbar_init(oempty, 8);
    tc::mbar_init(redb, 4);
    tc::mbar_init(redb + 1, 4);
    tc::mbar_init(done, 1);
    *abort_flag = 0;
    for (int i = 0; i < 4; ++i) raised[i] = 0;
    tc::fence_mbar_init();
  }
  if (warp == 9) {
    tc::tmem_alloc(tmem_at, kTmemCols);
    tc::tmem_relinquish();
  }
  pdl_wait();
  LatentWalk walk;
  LatentPiece w;
  {
    walk.begin(p, reinterpret_cast<int32_t*>(kbuf), warp_tot);
  }
  tc::fence_proxy_async();     // the prefix sums' buffer is the copies' next
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_at;

  if (warp < 8) {
    // ------------------------------------------------------------- softmax and output
    const int quad = warp & 3, half = warp >> 2;
    const int row = quad * 32 + lane;             // TMEM lane: key of S^T, dim of O^T
    const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
    const uint32_t scol = tmem + lane_base + kSCol + half * 32, ocol = tmem + lane_base + kOCol + half * 32;
    float* mb = mrow + warp * 32;
    const float k2 = p.scale * kLog2e;
    int g = 0, ru = 0;
    bool ok = true;
    auto group_sync = [&]() -> bool {             // the four warps of this half
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(redb + half);
      const bool r = tc::mbar_wait(redb + half, ru & 1, abort_flag, p.err);
      ++ru;
      return r;
    };
    bool posted = false;
    while (ok && walk.next(p, w)) {
      if (tid == 0 && !posted) walk.post(p, &w);
      posted = true;
      if (w.rows == 0) continue;
      // lane c: row c of this half, the keys it sees
      const int my_row = half * 32 + lane;
      int64_t vis = 0;
      if (my_row < w.rows) {
        const int64_t pos = w.start + (w.row0 + my_row - w.seq_row0) / p.H;
        vis = latent_visible(p, pos);
        if (quad == 0) latent_report_pos(p, pos);
      }
      // row c's reference, log2 units; for the exponentials a row without one yet subtracts 0, a
      // row that sees nothing (or is none) infinity
      float m = -INFINITY;
      const float none = vis > 0 ? 0.f : INFINITY;
      __syncwarp();
      mb[lane] = none;
      __syncwarp();
      float l[32];                                // this key lane's sums, by row
#pragma unroll
      for (int c = 0; c < 32; ++c) l[c] = 0.f;
      for (int t = w.tile0; t < w.tile1; ++t, ++g) {
        // (the tile's last copy is complete before its products are)
        if (!tc::mbar_wait(xfull, g & 1, abort_flag, p.err)) { ok = false; break; }
        const int64_t x0 = (int64_t)t * kTK;
        const int valid = tile_ok[g & 1] ? (int)min((int64_t)kTK, w.keys - x0) : 0;
        // A tile that every row sees whole, with every row's reference set: the weights are
        // taken against the references as they are, unless one of them would pass 1 (weights
        // and sums are floating-point numbers, so a reference need not be the maximum). The
        // group agrees on that while it computes the exponentials.
        bool slow = valid < kTK || w.keys0 < x0 + kTK || __any_sync(0xffffffffu, m == -INFINITY && vis > 0);
        float4 ref[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) ref[c] = *reinterpret_cast<const float4*>(mb + 4 * c);
        if (!tc::mbar_wait(sfull, g & 1, abort_flag, p.err)) { ok = false; break; }
        tc::fence_after_sync();
        float s[32];
        tc::tmem_ld32(scol, s);
        tc::tmem_wait_ld();
        if (!slow) {
          float top = -INFINITY;
#pragma unroll
          for (int c = 0; c < 32; c += 4) {
            const float4 mv = ref[c / 4];
            s[c] = fmaf(s[c], k2, -mv.x);
            s[c + 1] = fmaf(s[c + 1], k2, -mv.y);
            s[c + 2] = fmaf(s[c + 2], k2, -mv.z);
            s[c + 3] = fmaf(s[c + 3], k2, -mv.w);
            top = fmaxf(top, fmaxf(fmaxf(s[c], s[c + 1]), fmaxf(s[c + 2], s[c + 3])));
          }
          const bool over = __any_sync(0xffffffffu, top > 0.f);
          if (lane == 0) {
            if (over) raised[half * 2 + (g & 1)] = g + 1;
            tc::mbar_arrive(redb + half);
          }
#pragma unroll
          for (int c = 0; c < 32; ++c) s[c] = fast_exp2(s[c]);
          if (!tc::mbar_wait(redb + half, ru & 1, abort_flag, p.err)) { ok = false; break; }
          ++ru;
          slow = raised[half * 2 + (g & 1)] == g + 1;
          if (slow) {
            tc::tmem_ld32(scol, s);
            tc::tmem_wait_ld();
          }
        }
        if (slow) {
          const int seen = min((int)max((int64_t)0, min(vis - x0, (int64_t)kTK)), valid);
#pragma unroll
          for (int c = 0; c < 32; ++c)
            if (row >= __shfl_sync(0xffffffffu, seen, c)) s[c] = -INFINITY;
          float* rb = red_max + (ru & 1) * 256 + half * 128;
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const float mc = redux_max(s[c]);
            if (lane == c) rb[c * 4 + quad] = mc;
          }
          if (!group_sync()) { ok = false; break; }
          const float4 v = *reinterpret_cast<const float4*>(rb + lane * 4);
          const float mt = fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w)) * k2;
          float corr = 1.f;
          if (t == w.tile0) {
            m = mt + kRoom;
          } else if (mt > m + kRaise) {
            corr = fast_exp2(m - (mt + kRoom));   // 0 from -inf
            m = mt + kRoom;
          }
          __syncwarp();
          mb[lane] = m == -INFINITY ? none : m;
          const bool raise = t > w.tile0 && __any_sync(0xffffffffu, corr != 1.f);
          __syncwarp();
          if (raise) {
            // S^T of this tile is done, and with it every product issued before it
#pragma unroll
            for (int c = 0; c < 32; ++c) l[c] *= __shfl_sync(0xffffffffu, corr, c);
#pragma unroll 1
            for (int b = 0; b < 4; ++b) {
              float o[32];
              tc::tmem_ld32(ocol + b * kNR, o);
              tc::tmem_wait_ld();
#pragma unroll
              for (int c = 0; c < 32; ++c) o[c] *= __shfl_sync(0xffffffffu, corr, c);
              st32(ocol + b * kNR, o);
            }
            tc::tmem_wait_st();
          }
#pragma unroll
          for (int c = 0; c < 32; c += 4) {
            const float4 mv = *reinterpret_cast<const float4*>(mb + c);
            s[c] = fast_exp2(fmaf(s[c], k2, -mv.x));
            s[c + 1] = fast_exp2(fmaf(s[c + 1], k2, -mv.y));
            s[c + 2] = fast_exp2(fmaf(s[c + 2], k2, -mv.z));
            s[c + 3] = fast_exp2(fmaf(s[c + 3], k2, -mv.w));
          }
        }
        // P^T, MN-major [128 keys][64 rows]: this key's half row. The weights are rounded to
        // bf16, the second product's type; the sums above take them unrounded.
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<uint4*>(xbuf + tc::sw128_off(row, half * 4 + i)) =
              make_uint4(pack_bf16(s[8 * i], s[8 * i + 1]), pack_bf16(s[8 * i + 2], s[8 * i + 3]),
                         pack_bf16(s[8 * i + 4], s[8 * i + 5]), pack_bf16(s[8 * i + 6], s[8 * i + 7]));
        if (row >= valid) {                       // 0 times whatever lies behind the keys must be 0
#pragma unroll 1
          for (int b = half * 4; b < half * 4 + 4; ++b)
#pragma unroll
            for (int c = 0; c < 8; ++c)
              *reinterpret_cast<uint4*>(kbuf + b * kKBlock + tc::sw128_off(row, c)) = make_uint4(0, 0, 0, 0);
        }
        tc::fence_proxy_async();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(pfull);
#pragma unroll
        for (int c = 0; c < 32; ++c) l[c] += s[c];
      }
      if (!ok) break;
      // ---- sums over the keys: lane c gets row c's
      const bool any = w.tile1 > w.tile0;
      float ls = 0.f;
      if (any) {
        red_sum[(half * 32 + lane) * 4 + quad] = reduce_scatter_sum(l);
        if (!group_sync()) { ok = false; break; }
        const float4 v = *reinterpret_cast<const float4*>(red_sum + (half * 32 + lane) * 4);
        ls = (v.x + v.y) + (v.z + v.w);
        if (!tc::mbar_wait(pvdone, (g - 1) & 1, abort_flag, p.err)) { ok = false; break; }
        tc::fence_after_sync();
      }
      const int n_out = min(32, w.rows - half * 32);   // rows of this half (may be <= 0)
      if (w.whole) {
        const float inv = ls == 0.f ? 0.f : 1.f / ls;
        const bool even = (lane & 1) == 0;
        uint32_t* out = reinterpret_cast<uint32_t*>(p.out) + (int64_t)(w.row0 + half * 32) * (kC / 2);
#pragma unroll 1
        for (int b = 0; b < 4; ++b) {
          float o[32];
          if (any) {
            tc::tmem_ld32(ocol + b * kNR, o);
            tc::tmem_wait_ld();
          } else {
#pragma unroll
            for (int c = 0; c < 32; ++c) o[c] = 0.f;
          }
          // lanes 2i, 2i + 1 hold dims d, d + 1: the even lane stores row c's pair, the odd
          // lane row c + 1's
          const int d0 = b * 128 + (row & ~1);
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            const float a0 = o[c] * __shfl_sync(0xffffffffu, inv, c);
            const float a1 = o[c + 1] * __shfl_sync(0xffffffffu, inv, c + 1);
            const float got = __shfl_xor_sync(0xffffffffu, even ? a1 : a0, 1);
            const int r = even ? c : c + 1;
            if (r < n_out) out[((int64_t)r * kC + d0) >> 1] = even ? pack_bf16(a0, got) : pack_bf16(got, a1);
          }
        }
      } else {
        const int64_t at = (int64_t)w.slot * kNR + half * 32;
        if (quad == 0) {
          p.part_ml[(at + lane) * 2] = m;
          p.part_ml[(at + lane) * 2 + 1] = ls;
        }
        if (any) {
#pragma unroll 1
          for (int b = 0; b < 4; ++b) {
            float o[32];
            tc::tmem_ld32(ocol + b * kNR, o);
            tc::tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (c < n_out) p.part_o[(at + c) * kC + b * 128 + row] = o[c];
          }
        }
      }
      if (any) {
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(oempty);
      }
    }
    if (tid == 0 && !posted) walk.post(p, nullptr);
  } else if (warp == 8) {
    // ------------------------------------------------------------------------ copies
    if (lane == 0) {
      int g = 0, u = 0;
      int nq = 0, nx = 0, nv[4] = {0, 0, 0, 0};   // phases of each barrier given copies
      bool ok = true;
      while (ok && walk.next(p, w)) {
        if (w.tile0 >= w.tile1) continue;
        if (u > 0 && !tc::mbar_wait(qempty, (u - 1) & 1, abort_flag, p.err)) break;
        tc::mbar_arrive_tx(qfull, 9 * kQBlock);
        ++nq;
        for (int b = 0; b < 9; ++b) tma_2d(qbuf + b * kQBlock, &qmap, b * 128, w.row0, qfull);
        for (int t = w.tile0; t < w.tile1; ++t, ++g) {
          const int64_t slot = tile_slot(p, w.seq, t);
          const bool have = slot >= 0;
          if (!have) slot_ok(slot, p.err);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (g > 0 && ok) ok = tc::mbar_wait(vempty + j, (g - 1) & 1, abort_flag, p.err);
            if (!ok) continue;
            ++nv[j];
            if (have) {
              tc::mbar_arrive_tx(vfull + j, 2 * kKBlock);
              tma_2d(kbuf + 2 * j * kKBlock, &kmap, 2 * j * 128, (int)slot, vfull + j);
              tma_2d(kbuf + (2 * j + 1) * kKBlock, &kmap, (2 * j + 1) * 128, (int)slot, vfull + j);
            } else {
              tc::mbar_arrive(vfull + j);
            }
          }
          if (!ok) break;
          // the rotary block's buffer holds P^T until the previous tile's products are done
          if (g > 0 && !tc::mbar_wait(pvdone, (g - 1) & 1, abort_flag, p.err)) { ok = false; break; }
          tile_ok[g & 1] = have;
          ++nx;
          if (have) {
            tc::mbar_arrive_tx(xfull, kKBlock);
            tma_2d(xbuf, &kmap, 8 * 128, (int)slot, xfull);
          } else {
            tc::mbar_arrive(xfull);
          }
          if (t + 1 < w.tile1) {             // the next tile's rows into L2
            const int64_t ahead = tile_slot(p, w.seq, t + 1);
            if (ahead >= 0) {
              const uint8_t* rows = reinterpret_cast<const uint8_t*>(p.cache.data) + ahead * (kW * 2);
#pragma unroll 1
              for (int i = 0; i < 9; ++i)
                asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(rows + i * kKBlock), "r"(kKBlock)
                             : "memory");
            }
          }
        }
        ++u;
      }
      if (*abort_flag) {                          // leave no copy in flight
        if (nq > 0) tc::mbar_wait_drain(qfull, (nq - 1) & 1);
        if (nx > 0) tc::mbar_wait_drain(xfull, (nx - 1) & 1);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (nv[j] > 0) tc::mbar_wait_drain(vfull + j, (nv[j] - 1) & 1);
      }
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------------- products
    constexpr uint32_t idesc_s = tc::idesc_bf16(kTK, kNR);
    constexpr uint32_t idesc_o = tc::idesc_bf16(128, kNR, true, true);
    const uint32_t k0 = tc::uniform(tc::smem_u32(kbuf)), x0 = tc::uniform(tc::smem_u32(xbuf));
    const uint32_t k_lo = tc::sdesc_lo(k0, 16), x_lo = tc::sdesc_lo(x0, 16);   // keys, rotary keys / P^T
    const uint32_t q_lo = tc::sdesc_lo(tc::uniform(tc::smem_u32(qbuf)), 16);   // rows
    const uint32_t v_lo = tc::sdesc_lo(k0, kKBlock);                           // V^T, MN-major
    const uint32_t dS = tc::uniform(tmem) + kSCol, dO = tc::uniform(tmem) + kOCol;
    int g = 0, u = 0;
    bool ok = true;
    auto wait_all = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, tc::mbar_wait(bar, parity, abort_flag, p.err));
    };
    while (ok && walk.next(p, w)) {
      if (w.tile0 >= w.tile1) continue;
      if (!wait_all(qfull, u & 1)) break;
      for (int t = w.tile0; t < w.tile1; ++t, ++g) {
#pragma unroll
        for (int j = 0; j < 5; ++j) {
          if (ok) ok = wait_all(j < 4 ? vfull + j : xfull, g & 1);
          if (!ok) continue;
          tc::fence_after_sync();
          if (tc::elect_one()) {
#pragma unroll
            for (int b = 0; b < (j < 4 ? 2 : 1); ++b) {
              const int kb = 2 * j + b;
#pragma unroll
              for (int s = 0; s < 4; ++s)          // 16 dims, 32 bytes
                tc::mma_bf16_lo<idesc_s>(dS, (j < 4 ? k_lo + ((kb * kKBlock) >> 4) : x_lo) + 2 * s,
                                         q_lo + ((kb * kQBlock) >> 4) + 2 * s, (kb | s) ? 1u : 0u);
            }
            if (j == 4) {
              tc::mma_commit(sfull);
              if (t + 1 == w.tile1) tc::mma_commit(qempty);
            }
          }
          __syncwarp();
        }
        if (!ok) break;
        if (!wait_all(pfull, g & 1)) { ok = false; break; }
        if (t == w.tile0 && u > 0 && !wait_all(oempty, (u - 1) & 1)) { ok = false; break; }
        tc::fence_after_sync();
        const uint32_t acc = tc::uniform(t > w.tile0);
        if (tc::elect_one()) {
#pragma unroll
          for (int b = 0; b < 4; ++b) {
#pragma unroll
            for (int s = 0; s < 8; ++s)            // 16 keys, 2 KB
              tc::mma_bf16_lo<idesc_o>(dO + b * kNR, v_lo + ((2 * b * kKBlock + s * 2048) >> 4),
                                       x_lo + ((s * 2048) >> 4), s > 0 ? 1u : acc);
            tc::mma_commit(vempty + b);
          }
          tc::mma_commit(pvdone);
        }
        __syncwarp();
      }
      ++u;
    }
    if (tc::elect_one()) {
      tc::mma_commit(done);
      tc::mbar_wait_drain(done, 0);
    }
    __syncwarp();
  }

  tc::fence_before_sync();
  __syncthreads();
  if (warp == 9) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace

cudaError_t launch_latent_attn_tc(const LatentAttnParams& p, cudaStream_t st) {
  CUtensorMap qmap, kmap;
  const int64_t rows = (int64_t)p.n_tokens * p.H;
  const int64_t pool_rows = (p.cache.n_pages > 0 ? p.cache.n_pages : 1) * kBlock;
  if (!encode_byte_rows_map(&qmap, p.q, (uint64_t)rows, kW * 2, 128, kNR) ||
      !encode_byte_rows_map(&kmap, p.cache.data, (uint64_t)pool_rows, kW * 2, 128, kTK))
    return cudaErrorInvalidValue;
  const cudaError_t e =
      cudaFuncSetAttribute(latent_attn_tc, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return e;
  return launch_pdl(latent_attn_tc, dim3((unsigned)p.plan.ctas), dim3(kThreads), kSmemBytes, st, p, qmap, kmap);
}

}  // namespace v4a
