// Expanded latent attention on tcgen05 tensor cores: bf16, keys of 128 projected + 64 rotary
// dims (the rotary part shared by the heads), values of 128 dims.
//
//   S = Q K^T      M = 128 queries, N = 128 keys, K = 192   (12 MMAs)
//   P = 2^(scale log2(e) S - m), bf16, in tensor memory over S
//   O += P V       M = 128 queries, N = 128 dims, K = 128 keys (8 MMAs)
// A work item is 256 consecutive queries of one head of one sequence, as two tiles of 128 that
// take turns: while one tile's softmax runs, the other tile's products do. Tensor memory holds
// S/P and O of both (512 columns). Shared memory: the queries (96 KB), three 32 KB slots through
// which projected keys and values pass in turn (K0 V0 K1 V1 ..: with three, a value tile is
// requested a whole step before its use and a key tile half a step), and two 16 KB slots for the
// rotary keys.
//
// Bound: the tensor pipe (40 MMAs of M = N = 128, K = 16 a step of 256 queries x 128 keys).
//
// Warps 0-3 / 4-7: softmax and output of tile 0 / 1, a thread a query (so maxima and sums need
// no exchange). The running maximum is raised only when it grows by more than 2^8. Warp 8:
// copies. Warps 9 and 10: products of tile 0 / 1. (Warp 11 only completes its warpgroup.)
#include "kernels.h"
#include "latent.h"
#include "tc.cuh"

namespace v4a {
namespace {

constexpr int kT = 128, kThreads = 384;
constexpr int kBlk = kT * 128;                                   // 16 KB: 128 rows x 64 dims
constexpr int kOffQ = 0, kOffKV = 6 * kBlk, kOffPe = kOffKV + 6 * kBlk;
constexpr int kOffBar = kOffPe + 2 * kBlk;
constexpr int kNBar = 28;
constexpr int kOffMisc = kOffBar + kNBar * 8;
constexpr int kSmemBytes = kOffMisc + 128 + 1024;
static_assert(kSmemBytes <= 227 * 1024, "shared memory of one CTA");
static_assert((V4A_MAX_SEQ + 1) * 4 <= kBlk, "the plan's prefix sums use a key block before its first copy");
constexpr uint32_t kTmemCols = 512;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRaise = 8.0f;                                   // log2 units

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

// A work item: queries q0 .. of a sequence (rows qa + q0 ..), head h, keys ka .. ka + nk - 1.
struct Item {
  int qa, nq, ka, nk, q0, h;
  int tiles[2];                      // key tiles that each query tile needs (0: no such tile or no key)
  __device__ __forceinline__ int seen(const LatentExpandedParams& p, int i) const {   // keys of query i
    return i >= nq ? 0 : p.causal ? max(0, min(nk, nk - nq + i + 1)) : nk;
  }
};

// Items of a sequence: its 256-query blocks from the last (the longest, when causal) to the
// first, all heads of a block in a row. The CTAs take the items in turn.
struct Walk {
  int x, step, total, b, base;
  static __device__ __forceinline__ int items(const LatentExpandedParams& p, int b) {
    const int n = max(cu_at(p.cu_q, b + 1, p.n_q) - cu_at(p.cu_q, b, p.n_q), 0);
    return (n + 255) / 256 * p.H;
  }
  __device__ __forceinline__ void begin(const LatentExpandedParams& p, const int32_t* pre) {
    x = blockIdx.x;
    step = gridDim.x;
    total = pre[p.n_seq];
    b = x < total ? latent_seq_at(pre, p.n_seq, x) : 0;
    base = x < total ? pre[b] : 0;
  }
  __device__ __forceinline__ bool next(const LatentExpandedParams& p, Item& w) {
    if (x >= total) return false;
    int n = items(p, b);
    while (x >= base + n) {
      base += n;
      n = items(p, ++b);
    }
    const int r = x - base;
    w.qa = cu_at(p.cu_q, b, p.n_q);
    w.nq = max(cu_at(p.cu_q, b + 1, p.n_q) - w.qa, 0);
    w.ka = cu_at(p.cu_k, b, p.n_k);
    w.nk = max(cu_at(p.cu_k, b + 1, p.n_k) - w.ka, 0);
    w.h = r % p.H;
    w.q0 = (n / p.H - 1 - r / p.H) * 256;
    for (int i = 0; i < 2; ++i) {
      const int last = min(w.q0 + i * kT + kT, w.nq) - 1;       // last query of the tile
      w.tiles[i] = last < w.q0 + i * kT ? 0 : (w.seen(p, last) + kT - 1) / kT;
    }
    x += step;
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
  uint8_t* kvbuf = sm + kOffKV;                  // [3 slots][2 blocks]
  uint8_t* pebuf = sm + kOffPe;                  // [2 slots]
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + kOffBar);
  uint64_t* qfull = bars;                        // [2] by query tile
  uint64_t* qempty = bars + 2;                   // [2]
  uint64_t* full = bars + 4;                     // [3] by slot
  uint64_t* empty = bars + 7;                    // [3]
  uint64_t* pefull = bars + 10;                  // [2]
  uint64_t* peempty = bars + 12;                 // [2]
  uint64_t* sfull = bars + 14;                   // [2] by query tile
  uint64_t* pfull = bars + 16;                   // [2]
  uint64_t* ofull = bars + 18;                   // [2]
  uint64_t* oempty = bars + 20;                  // [2]
  uint64_t* done = bars + 22;                    // [2]
  int* misc = reinterpret_cast<int*>(sm + kOffMisc);
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(misc);
  volatile int* abort_flag = misc + 1;
  int32_t* warp_tot = misc + 4;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(qfull + i, 1);
      tc::mbar_init(qempty + i, 1);
      tc::mbar_init(pefull + i, 1);
      tc::mbar_init(peempty + i, 2);
      tc::mbar_init(done + i, 1);
      tc::mbar_init(sfull + i, 1);
      tc::mbar_init(pfull + i, 4);
      tc::mbar_init(ofull + i, 1);
      tc::mbar_init(oempty + i, 4);
    }
    for (int i = 0; i < 3; ++i) {
      tc::mbar_init(full + i, 1);
      tc::mbar_init(empty + i, 2);                // both tiles' products
    }
    *abort_flag = 0;
    tc::fence_mbar_init();
  }
  if (warp == 9) {
    tc::tmem_alloc(tmem_at, kTmemCols);
    tc::tmem_relinquish();
  }
  pdl_wait();
  Walk walk;
  Item w;
  {
    int32_t* pre = reinterpret_cast<int32_t*>(kvbuf);
    seq_prefix(p.n_seq, pre, warp_tot, [&](int b) { return Walk::items(p, b); });
    walk.begin(p, pre);
  }
  tc::fence_proxy_async();     // the prefix sums' buffer is the copies' next
  tc::fence_before_sync();
  __syncthreads();
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
    const float k2 = p.scale * kLog2e;
    const uint64_t k22 = pack2(k2, k2);
    int g = 0, n_items = 0;
    bool ok = true;
    while (ok && walk.next(p, w)) {
      const int qi = w.q0 + tile * kT + row;
      const int seen = w.seen(p, qi);
      const int n = w.tiles[tile];
      float m = -INFINITY, l = 0.f;
      for (int t = 0; t < n; ++t, ++g) {
        if (!tc::mbar_wait(sfull + tile, g & 1, abort_flag, p.err)) { ok = false; break; }
        tc::fence_after_sync();
        float s[128];
#pragma unroll
        for (int i = 0; i < 4; ++i) tc::tmem_ld32(scol + 32 * i, *reinterpret_cast<float(*)[32]>(&s[32 * i]));
        tc::tmem_wait_ld();
        const int here = seen - t * kT;           // keys of the tile that this query sees
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
        if (t == 0) {
          m = mt;
        } else if (mt > m + kRaise) {
          corr = fast_exp2(m - mt);               // 0 from -inf
          m = mt;
        }
        if (t > 0 && __any_sync(0xffffffffu, corr != 1.f)) {
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
        const float ref = m == -INFINITY ? 0.f : m;
        const uint64_t nm = pack2(-ref, -ref);
        uint64_t acc[4] = {0, 0, 0, 0};
        // weights, rounded to bf16 for the second product; the sum takes them unrounded
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          uint32_t pw[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            float a, b;
            unpack2(fma2(pack2(s[64 * hf + 2 * i], s[64 * hf + 2 * i + 1]), k22, nm), a, b);
            a = fast_exp2(a);
            b = fast_exp2(b);
            acc[i & 3] = add2(acc[i & 3], pack2(a, b));
            pw[i] = pack_bf16(a, b);
          }
          tc::tmem_st32(scol + 32 * hf, pw);
        }
        tc::tmem_wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(pfull + tile);
        float a, b;
        unpack2(add2(add2(acc[0], acc[1]), add2(acc[2], acc[3])), a, b);
        l += a + b;
      }
      if (!ok) break;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      if (n > 0) {
        if (!tc::mbar_wait(ofull + tile, n_items & 1, abort_flag, p.err)) { ok = false; break; }
        tc::fence_after_sync();
        ++n_items;
      }
      uint4* out = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(p.out) +
                                            ((int64_t)(w.qa + qi) * p.H + w.h) * kT);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float o[32];
        if (n > 0) {
          tc::tmem_ld32(ocol + 32 * i, o);
          tc::tmem_wait_ld();
        } else {
#pragma unroll
          for (int c = 0; c < 32; ++c) o[c] = 0.f;
        }
        if (qi < w.nq) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
            out[4 * i + c] = make_uint4(pack_bf16(o[8 * c] * inv, o[8 * c + 1] * inv),
                                        pack_bf16(o[8 * c + 2] * inv, o[8 * c + 3] * inv),
                                        pack_bf16(o[8 * c + 4] * inv, o[8 * c + 5] * inv),
                                        pack_bf16(o[8 * c + 6] * inv, o[8 * c + 7] * inv));
        }
      }
      if (n > 0) {
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(oempty + tile);
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 120;");
  }
  if (warp == 8) {
    // ------------------------------------------------------------------------ copies
    if (lane == 0) {
      int c = 0, e = 0;                           // slot and rotary-slot uses
      int nq[2] = {0, 0};                         // query tiles loaded
      bool ok = true;
      auto wait = [&](uint64_t* bar, int parity) {
        if (ok) ok = tc::mbar_wait(bar, parity, abort_flag, p.err);
        return ok;
      };
      auto load = [&](const CUtensorMap* map, int h, int tok) {   // 128 rows x 128 dims
        const int sl = c % 3;
        if (c >= 3 && !wait(empty + sl, (c / 3 - 1) & 1)) return;
        tc::mbar_arrive_tx(full + sl, 2 * kBlk);
        tma_3d(kvbuf + 2 * sl * kBlk, map, 0, h, tok, full + sl);
        tma_3d(kvbuf + (2 * sl + 1) * kBlk, map, 128, h, tok, full + sl);
        ++c;
      };
      auto load_pe = [&](int tok) {
        const int sl = e & 1;
        if (e >= 2 && !wait(peempty + sl, (e / 2 - 1) & 1)) return;
        tc::mbar_arrive_tx(pefull + sl, kBlk);
        tma_3d(pebuf + sl * kBlk, &pmap, 0, 0, tok, pefull + sl);
        ++e;
      };
      auto load_q = [&](int i) {
        if (w.tiles[i] == 0) return;
        if (nq[i] > 0 && !wait(qempty + i, (nq[i] - 1) & 1)) return;
        tc::mbar_arrive_tx(qfull + i, 3 * kBlk);
        for (int b = 0; b < 3; ++b)
          tma_3d(qbuf + (3 * i + b) * kBlk, &qmap, b * 128, w.h, w.qa + w.q0 + i * kT, qfull + i);
        ++nq[i];
      };
      while (ok && walk.next(p, w)) {
        const int n = max(w.tiles[0], w.tiles[1]);
        for (int t = 0; t < n && ok; ++t) {
          const int tok = w.ka + t * kT;
          if (t == 0) load_q(0);
          if (ok) load_pe(tok);
          if (ok) load(&kmap, w.h, tok);
          if (t == 0 && ok) load_q(1);
          if (ok) load(&vmap, w.h, tok);
        }
      }
      if (*abort_flag) {                          // leave no copy in flight
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (nq[i] > 0) tc::mbar_wait_drain(qfull + i, (nq[i] - 1) & 1);
        for (int k = c > 3 ? c - 3 : 0; k < c; ++k) tc::mbar_wait_drain(full + k % 3, (k / 3) & 1);
        for (int k = e > 2 ? e - 2 : 0; k < e; ++k) tc::mbar_wait_drain(pefull + (k & 1), (k / 2) & 1);
      }
    }
    __syncwarp();
  } else if (warp == 9 || warp == 10) {
    // ---------------------------------------------------------------------- products
    const int tile = warp - 9;
    constexpr uint32_t idesc_s = tc::idesc_bf16(kT, kT);
    constexpr uint32_t idesc_o = tc::idesc_bf16(kT, kT, false, true);
    const uint32_t ut = tc::uniform(tile), dS = tc::uniform(tmem) + ut * 128, dO = dS + 256;
    const uint32_t kv = tc::uniform(tc::smem_u32(kvbuf)), pe = tc::uniform(tc::smem_u32(pebuf));
    const uint32_t q_lo = tc::sdesc_lo(tc::uniform(tc::smem_u32(qbuf)) + ut * 3 * kBlk, 16);
    int c = 0, e = 0;                             // slot uses: K of step t at c, V at c + 1
    int nq = 0, gp = 0;                           // items and products P V of this tile
    bool ok = true;
    auto wait_all = [&](uint64_t* bar, uint32_t parity) {
      if (ok) ok = __all_sync(0xffffffffu, tc::mbar_wait(bar, parity, abort_flag, p.err));
      return ok;
    };
    auto commit = [&](uint64_t* bar) {
      if (ok && tc::elect_one()) tc::mma_commit(bar);
      __syncwarp();
    };
    // S with the keys of slot use kc and rotary-slot use ec
    auto issue_s = [&](int kc, int ec) {
      if (!wait_all(full + kc % 3, (kc / 3) & 1) || !wait_all(pefull + (ec & 1), (ec / 2) & 1)) return;
      tc::fence_after_sync();
      const uint32_t k_lo = tc::uniform(tc::sdesc_lo(kv + (kc % 3) * 2 * kBlk, 16));
      const uint32_t e_lo = tc::uniform(tc::sdesc_lo(pe + (ec & 1) * kBlk, 16));
      if (tc::elect_one()) {
#pragma unroll
        for (int b = 0; b < 3; ++b) {
#pragma unroll
          for (int s = 0; s < 4; ++s)              // 16 dims, 32 bytes
            tc::mma_bf16_lo<idesc_s>(dS, q_lo + ((b * kBlk) >> 4) + 2 * s,
                                     (b < 2 ? k_lo + ((b * kBlk) >> 4) : e_lo) + 2 * s, (b | s) ? 1u : 0u);
        }
        tc::mma_commit(sfull + tile);
      }
      __syncwarp();
    };
    // Both warps release every slot use, a tile that skips it too, and only once it was full:
    // an arrival for a later use must not count for this one.
    auto release_k = [&](int kc, int ec) {
      if (!wait_all(full + kc % 3, (kc / 3) & 1) || !wait_all(pefull + (ec & 1), (ec / 2) & 1)) return;
      commit(empty + kc % 3);
      commit(peempty + (ec & 1));
    };
    while (ok && walk.next(p, w)) {
      const int n = max(w.tiles[0], w.tiles[1]), mine = w.tiles[tile];
      if (n == 0) continue;
      if (mine > 0) {
        if (!wait_all(qfull + tile, nq & 1)) break;
        issue_s(c, e);                             // step 0's logits
        if (mine == 1) commit(qempty + tile);
      }
      release_k(c, e);
      for (int t = 0; t < n && ok; ++t, c += 2, ++e) {
        const int vs = (c + 1) % 3;
        if (!wait_all(full + vs, ((c + 1) / 3) & 1)) break;
        if (t < mine) {
          if (!wait_all(pfull + tile, gp & 1)) break;
          if (t == 0 && nq > 0 && !wait_all(oempty + tile, (nq - 1) & 1)) break;
          const int valid = w.nk - t * kT;
          if (valid < kT) {                        // 0 times what lies behind the keys must be 0
            // (the other tile's warp may be doing the same, or its product reading these zeros)
            for (int b = 0; b < 2; ++b)
              for (int o = valid * 128 + lane * 16; o < kBlk; o += 512)
                *reinterpret_cast<uint4*>(kvbuf + (2 * vs + b) * kBlk + o) = make_uint4(0, 0, 0, 0);
            tc::fence_proxy_async();
            __syncwarp();
          }
          tc::fence_after_sync();
          const uint32_t v_lo = tc::uniform(tc::sdesc_lo(kv + vs * 2 * kBlk, kBlk));
          const uint32_t acc = tc::uniform(t > 0);
          if (tc::elect_one()) {
#pragma unroll
            for (int s = 0; s < 8; ++s)            // 16 keys: 8 columns of P, 2 KB of V
              tc::mma_bf16_ta_lo<idesc_o>(dO, dS + 8 * s, v_lo + ((s * 2048) >> 4), s > 0 ? 1u : acc);
            if (t + 1 == mine) tc::mma_commit(ofull + tile);
          }
          __syncwarp();
          ++gp;
        }
        commit(empty + vs);
        if (t + 1 < mine) {
          issue_s(c + 2, e + 1);
          if (t + 2 == mine) commit(qempty + tile);
        }
        if (t + 1 < n) release_k(c + 2, e + 1);
      }
      if (mine > 0) ++nq;
    }
    if (tc::elect_one()) {
      tc::mma_commit(done + tile);
      tc::mbar_wait_drain(done + tile, 0);
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

cudaError_t launch_latent_expanded_tc(const LatentExpandedParams& p, cudaStream_t st) {
  CUtensorMap qmap, kmap, pmap, vmap;
  const uint64_t H = (uint64_t)p.H, nk = p.n_k > 0 ? (uint64_t)p.n_k : 1;
  const bool none = p.n_k == 0;                    // then nothing is read through these maps
  const void *k = none ? p.q : p.k, *pe = none ? p.q : p.k_pe, *v = none ? p.q : p.v;
  const uint64_t kts = none ? 256 : p.k_ts * 2, khs = none ? 256 : p.k_hs * 2, vts = none ? 256 : p.v_ts * 2,
                 vhs = none ? 256 : p.v_hs * 2, pts = none ? 128 : p.pe_ts * 2;
  if (!encode_byte_rows_map3(&qmap, p.q, 384, H, 384, (uint64_t)p.n_q, H * 384, 128, kT) ||
      !encode_byte_rows_map3(&kmap, k, 256, H, khs, nk, kts, 128, kT) ||
      !encode_byte_rows_map3(&vmap, v, 256, H, vhs, nk, vts, 128, kT) ||
      !encode_byte_rows_map3(&pmap, pe, 128, 1, pts, nk, pts, 128, kT))
    return cudaErrorInvalidValue;
  int dev = 0, sms = 152;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const int64_t items = ((int64_t)p.n_q / 256 + p.n_seq) * p.H;   // at most
  const int grid = (int)(items < sms ? items : sms);
  const cudaError_t e =
      cudaFuncSetAttribute(latent_expanded_tc, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return e;
  return launch_pdl(latent_expanded_tc, dim3(grid), dim3(kThreads), kSmemBytes, st, p, qmap, kmap, pmap, vmap);
}

}  // namespace v4a
