// Absorbed latent attention over FP4 rows (512 latent + 64 rotary dims) on tcgen05 tensor cores, f16.
//
//   row = s (B code | h): s an fp32 number a key, B an e4m3 number a block of 16; B code and h are f16
//   S^T = [B code | h] (2^a Q)^T          M = 128 keys, N = 64 rows, K = 576   (36 MMAs)
//   x = scale log2(e) 2^-a s S^T + log2 s, P^T = 2^(x - m): the weight times its row's scale, f16
//   O^T += (B code)^T P^T                 M = 4 x 128 dims, N = 64, K = 128 keys (32 MMAs)
//   l += P / s,  out = O / l
// Units, teams and the split along the keys are the plain kernel's (LatentWalk). 2^a is a power of two
// a unit that brings its largest |q| to [2^14, 2^15): bf16 queries are f16 numbers then, but for
// elements 2^-32 of that and smaller. m is kept where the first tile's largest weight is 2^6 and raised
// where one would pass 2^15, so f16 has all its bits down to 2^-20 of the largest weight so far.
//
// If keys and values went through shared memory, as the plain kernel's do, a tile would move 570 KB
// there, 4400 cycles at 128 bytes a cycle, and the products would wait for each softmax. So both A
// operands go through tensor memory (a product of M = 128, N = 64 then takes 33 cycles, not 49):
//   keys:   a thread a key (tensor-memory lane) expands 64 dims of its row at a time, 32 columns
//   values: a thread four dims (lane l: dims 4l .. 4l + 3, one for each block of 128 of O^T) expands
//           32 keys of two of them at a time, 2 x 16 columns. Two keys' codes are brought side by side
//           in a byte first, so one conversion gives a pair of keys.
// Keys have a ring of two slots of 32 columns, values one of four (O^T 256, S^T 64, rings 192: all 512),
// and S^T of the next tile runs beside this tile's softmax and O^T. (Three and three: 217 us in the case
// below where this took 209. The values of a tile can wait for its weights in four slots.)
//
// Warps 0-7: softmax and output, as in the plain kernel. Warps 8-15: queries and keys, two warpgroups
// with a slot each. Warps 16-23: values, a warpgroup for each half of the keys. Warps 24 and 26: products,
// one for each of the two (a wait is long against four products). Warp 25: copies (raw rows, two tiles;
// scales; Q).
//
// Bound: instructions, and the waits between roles. A tile takes 16,900 warp instructions (each code is
// expanded twice) and 3.06 us, about 6,000 cycles: the four schedulers issue 2.8 a cycle. Over a whole
// launch, with its start and end, they issue 2.3, and the tensor pipe is active for 29 % of the time.
// A slot's way from one hand to the next (wait, store, arrive, wait, products, commit) is 1,200 cycles of
// those. 28 warps in six roles do not fit the small instruction caches: loops over slots are rolled
// (S^T's unrolled by three: 216 us), waits are short, and one thread walks for all. ptxas spills 196 bytes
// (248 under a window): more than half of them are the copies' thread's, which holds the walk in 40
// registers and has time, the rest the softmax's (a dozen words of a piece, 104 registers) and a few of
// the keys'; the values have none.
// 32 sequences x 32768 tokens, 64 heads: 192 us with the merge (760 TFLOP/s); 16 of 4616-108051, 128 heads:
// 216 us; 4 chunks, 3020 tokens, 16 heads, window 1024: 233 us. (The bf16 cache takes 196, 191 and 217: a
// smaller cache, not a faster one. The trials below are to be held against 200, the time of their day.)
// On the way: one warpgroup a role 276 us, the same with unrolled loops 431; masked tiles' maxima by
// redux.sync, 170 cycles each, 207 (300 under the window). Codes expanded once, from registers, keys to
// tensor memory and values to shared memory: 319 us (the values' stores wait while O^T's products read
// shared memory). P^T and its products by halves, to overlap the tiles' O^T: 255 us.
#include "kernels.h"
#include "latent.h"
#include "latent_tc.cuh"

namespace v4a {
namespace {

constexpr int kNR = 64, kTK = 128, kC = 512, kR = 64;
constexpr int kRowBytes = V4A_LATENT_FP4_ROW_BYTES(kC, kR), kRopeAt = kC / 2, kBlockAt = kC / 2 + 2 * kR;
static_assert(kRowBytes == 416 && kRowBytes % 16 == 0, "row chunks");
constexpr int kThreads = 896;
constexpr int kQBlock = kNR * 128;
constexpr int kRaw = kTK * kRowBytes;
constexpr int kScPitch = kTK + 4;                                // f16: 8 blocks' words in different banks
constexpr int kOffQ = 0, kOffP = 9 * kQBlock, kOffRaw = kOffP + kTK * 128;
constexpr int kOffSc = kOffRaw + 2 * kRaw;                       // [3][32 blocks][kScPitch] f16
constexpr int kOffInfo = kOffSc + 3 * 32 * kScPitch * 2;         // [3][128] float2: s, log2 s
constexpr int kOffS = kOffInfo + 3 * kTK * 8;                    // [2][128] row scales
constexpr int kOffF = kOffS + 2 * kTK * 4;
// floats: red_max[2][64][4] (red_sum[64][4] in the half that is not in use) mrow[8 warps][32]
constexpr int kNFloats = 512 + 256;
constexpr int kOffBar = kOffF + kNFloats * 4;
constexpr int kNBar = 40;
constexpr int kPieces = 4, kWalkers = 26;                        // pieces of work known ahead; warps that take them
constexpr int kOffMisc = kOffBar + kNBar * 8;
// words there: tensor memory's address, the abort flag, and what the roles tell one another
constexpr int kAbort = 1, kRaised = 2, kTileOk = 6, kTileValid = 8, kQMax = 11, kQScale = 19, kWarpTot = 32;
constexpr int kMiscWords = 64;
static_assert(kRaised + 4 <= kTileOk && kTileOk + 2 <= kTileValid && kTileValid + 3 <= kQMax && kQMax + 8 <= kQScale &&
                  kQScale + 2 <= kWarpTot && kWarpTot + kThreads / 32 <= kMiscWords,
              "words of their own: the plan's sums have one a warp");
constexpr int kOffPiece = kOffMisc + kMiscWords * 4;
constexpr int kSmemBytes = kOffPiece + kPieces * (int)sizeof(LatentPiece) + (int)sizeof(LatentWalk) + 1024;
static_assert(kOffPiece % 8 == 0 && sizeof(LatentPiece) % 8 == 0, "alignment");
static_assert(kSmemBytes <= 227 * 1024, "shared memory of one CTA");
static_assert(kOffP % 1024 == 0 && kOffRaw % 1024 == 0, "swizzled operands");
static_assert((V4A_MAX_SEQ + 1) * 4 <= kRaw, "the plan's prefix sums use a raw tile before its first copy");
constexpr uint32_t kSCol = 0, kOCol = 64, kKCol = 320, kVCol = 384, kTmemCols = 512;
constexpr int kKeySlots = 2, kValueSlots = 4;   // of 32 columns: one and two a warpgroup
constexpr float kRoom = -6.0f, kRaise = 12.0f, kOver = 15.0f;    // log2 units: a reference above its maximum,
                                                                 // what raises it in masked tiles and in others
// registers of softmax, key and value (two each) and other warpgroups: 896 threads x 72 in all
constexpr int kRegSoftmax = 104, kRegKeys = 56, kRegValues = 72, kRegOther = 40;
static_assert(kRegValues == 72, "the values' warpgroups keep what the launch gives");
static_assert(2 * (kRegSoftmax + kRegKeys + kRegValues) + kRegOther <= 7 * 72, "registers of the launch");

__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t mul_f16(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}
// Two products and sums in one instruction.
__device__ __forceinline__ void fma2(float& d0, float& d1, float a0, float a1, float b, float c0, float c1) {
  asm("{ .reg .b64 x, y, z; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %4}; mov.b64 z, {%5, %6};\n\t"
      "fma.rn.f32x2 x, x, y, z; mov.b64 {%0, %1}, x; }"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b), "f"(c0), "f"(c1));
}
// Two e4m3 numbers as f16.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t w) {
  uint32_t r;
  asm("{ .reg .b16 lo, hi; mov.b32 {lo, hi}, %1; cvt.rn.f16x2.e4m3x2 %0, lo; }" : "=r"(r) : "r"(w));
  return r;
}

template <bool kWindow>
__global__ void __launch_bounds__(kThreads, 1)
    latent_attn_fp4_tc(const __grid_constant__ LatentAttnParams p, const __grid_constant__ CUtensorMap qmap) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* qbuf = sm + kOffQ;
  uint8_t* pbuf = sm + kOffP;
  uint8_t* raw = sm + kOffRaw;
  __half* sc = reinterpret_cast<__half*>(sm + kOffSc);
  float2* info = reinterpret_cast<float2*>(sm + kOffInfo);
  float* srow = reinterpret_cast<float*>(sm + kOffS);
  float* red_max = reinterpret_cast<float*>(sm + kOffF);
  float* mrow = red_max + 512;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + kOffBar);
  uint64_t* rawfull = bars;                                      // [2]
  uint64_t* rawempty = bars + 2;                                 // [2] by keys' and values' warps
  uint64_t* kfull = bars + 4;                                    // [2]
  uint64_t* kempty = bars + 6;                                   // [2]
  uint64_t* vfull = bars + 8;                                    // [4]
  uint64_t* vempty = bars + 12;                                  // [4]
  uint64_t* infofull = bars + 16;                                // [3] block scales and info of a tile
  uint64_t* qfull = bars + 19;
  uint64_t* qready = bars + 20;
  uint64_t* qempty = bars + 21;
  uint64_t* sfull = bars + 22;
  uint64_t* sfree = bars + 23;
  uint64_t* pfull = bars + 24;
  uint64_t* pvdone = bars + 25;
  uint64_t* oempty = bars + 26;
  uint64_t* redb = bars + 27;                                    // [2] one per group of 4 warps
  uint64_t* qmaxb = bars + 29;
  uint64_t* done = bars + 30;                                    // [2] of the products' two warps
  uint64_t* piecefull = bars + 32;                               // [4]
  uint64_t* pieceempty = bars + 36;                              // [4]
  int* misc = reinterpret_cast<int*>(sm + kOffMisc);
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(misc);
  volatile int* abort_flag = misc + kAbort;
  volatile int* raised = misc + kRaised;                         // [2 halves][2 parities] tile + 1
  volatile int* tile_ok = misc + kTileOk;                        // [2] by raw buffer
  volatile int* tile_valid = misc + kTileValid;                  // [3] keys of a tile that exist
  int* qmax = misc + kQMax;                                      // [8] largest |q| of a warp's chunks, as bits
  volatile float* qscale = reinterpret_cast<float*>(misc + kQScale);   // [2] 2^-a of a piece
  int32_t* warp_tot = misc + kWarpTot;                           // [28] by warp

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(rawfull + i, 1);
      tc::mbar_init(rawempty + i, 16);
      tc::mbar_init(redb + i, 4);
    }
    for (int i = 0; i < kKeySlots; ++i) {
      tc::mbar_init(kfull + i, 4);
      tc::mbar_init(kempty + i, 1);
    }
    for (int i = 0; i < kValueSlots; ++i) {
      tc::mbar_init(vfull + i, 4);
      tc::mbar_init(vempty + i, 1);
    }
    for (int i = 0; i < 3; ++i) tc::mbar_init(infofull + i, 8);
    for (int i = 0; i < kPieces; ++i) {
      tc::mbar_init(piecefull + i, 1);
      tc::mbar_init(pieceempty + i, kWalkers);
    }
    tc::mbar_init(qfull, 1);
    tc::mbar_init(qready, 8);
    tc::mbar_init(qempty, 1);
    tc::mbar_init(sfull, 1);
    tc::mbar_init(sfree, 8);
    tc::mbar_init(pfull, 8);
    tc::mbar_init(pvdone, 1);
    tc::mbar_init(oempty, 8);
    tc::mbar_init(qmaxb, 8);
    tc::mbar_init(done, 1);
    tc::mbar_init(done + 1, 1);
    *abort_flag = 0;
    for (int i = 0; i < 4; ++i) raised[i] = 0;
    tc::fence_mbar_init();
  }
  if (warp == 24) {
    tc::tmem_alloc(tmem_at, kTmemCols);
    tc::tmem_relinquish();
  }
  pdl_wait();
  // The copies' thread walks; the others get the pieces from it, a piece ahead. (Walking is some
  // hundred instructions that would push six roles' loops out of the instruction cache each time.)
  LatentPiece* const pieces = reinterpret_cast<LatentPiece*>(sm + kOffPiece);
  LatentWalk* const plan = reinterpret_cast<LatentWalk*>(pieces + kPieces);
  LatentWalk walk;
  LatentPiece w;
  walk.begin(p, reinterpret_cast<int32_t*>(raw), warp_tot);
  tc::fence_proxy_async();     // the prefix sums' buffer is the copies' next
  if (tid == 0) *plan = walk;
  int np = 0;                                     // pieces taken
  auto next = [&]() -> bool {                     // by whole warps
    const int at = np % kPieces;
    if (!__all_sync(0xffffffffu, tc::mbar_wait_few(piecefull + at, (np / kPieces) & 1, abort_flag, p.err))) return false;
    w = pieces[at];
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(pieceempty + at);
    ++np;
    return w.seq >= 0;
  };
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_at;
  const int quad = warp & 3;
  const int row = quad * 32 + lane;               // TMEM lane: key of S^T; lane l of O^T: dims 4l ..
  const uint32_t lane_base = (uint32_t)(quad * 32) << 16;

  if (warp < 8) {
    // ------------------------------------------------------------- softmax and output
    tc::set_regs<true, kRegSoftmax>();
    const int half = warp >> 2;
    const uint32_t scol = tmem + lane_base + kSCol + half * 32, ocol = tmem + lane_base + kOCol + half * 32;
    float* mb = mrow + warp * 32;
    int g = 0, ru = 0, u = 0;
    bool ok = true;
    auto group_sync = [&]() -> bool {             // the four warps of this half
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(redb + half);
      const bool r = tc::mbar_wait_few(redb + half, ru & 1, abort_flag, p.err);
      ++ru;
      return r;
    };
    bool posted = false;
    while (ok && next()) {
      if (tid == 0 && !posted) plan->post(p, &w);
      posted = true;
      if (w.rows == 0) continue;
      // lane c: row c of this half, the keys it sees
      const int my_row = half * 32 + lane;
      int64_t vis = 0, from = 0;
      if (my_row < w.rows) {
        const int64_t pos = w.start + (w.row0 + my_row - w.seq_row0) / p.H;
        vis = latent_visible(p, pos);
        if (kWindow) from = latent_from(p, pos);
        if (quad == 0) latent_report_pos(p, pos);
      }
      const int64_t all_from = kWindow ? latent_from(p, w.start + (w.row0 + w.rows - 1 - w.seq_row0) / p.H) : 0;
      const bool any = w.tile1 > w.tile0;
      float k2 = 0.f;
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
        const int64_t x0 = w.tile_at<kWindow>(t) * kTK;
        if (!tc::mbar_wait_few(infofull + g % 3, (g / 3) & 1, abort_flag, p.err)) { ok = false; break; }
        if (t == w.tile0) k2 = p.scale * kLog2e * qscale[u++ & 1];
        const float2 in = info[(g % 3) * kTK + row];
        const int valid = tile_valid[g % 3];
        // (1 / s to 2 ulp, log2 s to 2^-20 or so, the exponentials to 2^-22: beside the weights' 2^-11)
        const float kf = in.x * k2, ls = in.y, is = in.x != 0.f ? __fdividef(1.f, in.x) : 0.f;
        bool slow = valid < kTK || w.keys0 < x0 + kTK || (kWindow && x0 < all_from && x0 + kTK > p.sinks) ||
                    __any_sync(0xffffffffu, m == -INFINITY && vis > 0);
        if (!tc::mbar_wait_few(sfull, g & 1, abort_flag, p.err)) { ok = false; break; }
        tc::fence_after_sync();
        float s[32];
        tc::tmem_ld32(scol, s);
        tc::tmem_wait_ld();
        // S^T is in registers: the next tile's may be written
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(sfree);
        if (!slow) {
          float top = -INFINITY;
#pragma unroll
          for (int c = 0; c < 32; c += 4) {
            const float4 mv = *reinterpret_cast<const float4*>(mb + c);
            float d[4];                            // ls - mv
            fma2(d[0], d[1], mv.x, mv.y, -1.f, ls, ls);
            fma2(d[2], d[3], mv.z, mv.w, -1.f, ls, ls);
            fma2(s[c], s[c + 1], s[c], s[c + 1], kf, d[0], d[1]);
            fma2(s[c + 2], s[c + 3], s[c + 2], s[c + 3], kf, d[2], d[3]);
            top = fmaxf(top, fmaxf(fmaxf(s[c], s[c + 1]), fmaxf(s[c + 2], s[c + 3])));
          }
          // the group agrees whether a weight would pass 2^15
          const bool over = __any_sync(0xffffffffu, top > kOver);
          if (lane == 0) {
            if (over) raised[half * 2 + (g & 1)] = g + 1;
            tc::mbar_arrive(redb + half);
          }
          if (!tc::mbar_wait_few(redb + half, ru & 1, abort_flag, p.err)) { ok = false; break; }
          ++ru;
          slow = raised[half * 2 + (g & 1)] == g + 1;
          if (!slow) {
#pragma unroll
            for (int c = 0; c < 32; ++c) s[c] = fast_exp2(s[c]);
          } else {
#pragma unroll
            for (int c = 0; c < 32; ++c) s[c] += mb[c];
          }
        } else {
#pragma unroll
          for (int c = 0; c < 32; ++c) s[c] = fmaf(s[c], kf, ls);
        }
        bool raise = false;
        float corr = 1.f;
        if (slow) {
          const int seen = min((int)max((int64_t)0, min(vis - x0, (int64_t)kTK)), valid);
          const int begin = kWindow ? (int)max((int64_t)0, min(from - x0, (int64_t)kTK)) : 0;
          const bool sink = kWindow && x0 + row < p.sinks;
          if (__any_sync(0xffffffffu, seen < kTK)) {
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (row >= __shfl_sync(0xffffffffu, seen, c)) s[c] = -INFINITY;
          }
          if (kWindow && __any_sync(0xffffffffu, begin > 0)) {
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (row < __shfl_sync(0xffffffffu, begin, c) && !sink) s[c] = -INFINITY;
          }
          float* rb = red_max + (ru & 1) * 256 + half * 128;
          rb[lane * 4 + quad] = reduce_scatter<true>(s);
          if (!group_sync()) { ok = false; break; }
          const float4 v = *reinterpret_cast<const float4*>(rb + lane * 4);
          const float mt = fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w));
          if (t == w.tile0) {
            m = mt + kRoom;
          } else if (mt > m + kRaise) {
            corr = fast_exp2(m - (mt + kRoom));   // 0 from -inf
            m = mt + kRoom;
          }
          __syncwarp();
          mb[lane] = m == -INFINITY ? none : m;
          raise = t > w.tile0 && __any_sync(0xffffffffu, corr != 1.f);
          __syncwarp();
#pragma unroll
          for (int c = 0; c < 32; c += 4) {
            const float4 mv = *reinterpret_cast<const float4*>(mb + c);
            s[c] = fast_exp2(s[c] - mv.x);
            s[c + 1] = fast_exp2(s[c + 1] - mv.y);
            s[c + 2] = fast_exp2(s[c + 2] - mv.z);
            s[c + 3] = fast_exp2(s[c + 3] - mv.w);
          }
        }
        // P^T's buffer and the accumulator are the previous tile's products' until they are done
        if (g > 0 && !tc::mbar_wait_few(pvdone, (g - 1) & 1, abort_flag, p.err)) { ok = false; break; }
        if (raise) {
          tc::fence_after_sync();
#pragma unroll
          for (int c = 0; c < 32; ++c) l[c] *= __shfl_sync(0xffffffffu, corr, c);
#pragma unroll 1
          for (int b = 0; b < 16; ++b) {          // 8 columns of a block at a time
            float o[8];
            const uint32_t at = ocol + (b >> 2) * kNR + (b & 3) * 8;
            tc::tmem_ld8(at, o);
            tc::tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < 8; ++c) o[c] *= __shfl_sync(0xffffffffu, corr, (b & 3) * 8 + c);
            tc::tmem_st8(at, o);
          }
          tc::tmem_wait_st();
        }
        // P^T, MN-major [128 keys][64 rows]: this key's half row. A weight times its row's scale is
        // rounded to f16, the second product's type; the sums take it unrounded.
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<uint4*>(pbuf + tc::sw128_off(row, half * 4 + i)) =
              make_uint4(pack_f16(s[8 * i], s[8 * i + 1]), pack_f16(s[8 * i + 2], s[8 * i + 3]),
                         pack_f16(s[8 * i + 4], s[8 * i + 5]), pack_f16(s[8 * i + 6], s[8 * i + 7]));
        tc::fence_proxy_async();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(pfull);
#pragma unroll
        for (int c = 0; c < 32; c += 2) fma2(l[c], l[c + 1], s[c], s[c + 1], is, l[c], l[c + 1]);
      }
      if (!ok) break;
      // ---- sums over the keys: lane c gets row c's
      float lsum = 0.f;
      if (any) {
        float* rb = red_max + (ru & 1) * 256 + half * 128;
        rb[lane * 4 + quad] = reduce_scatter<false>(l);
        if (!group_sync()) { ok = false; break; }
        const float4 v = *reinterpret_cast<const float4*>(rb + lane * 4);
        lsum = (v.x + v.y) + (v.z + v.w);
        if (!tc::mbar_wait_few(pvdone, (g - 1) & 1, abort_flag, p.err)) { ok = false; break; }
        tc::fence_after_sync();
      }
      const int n_out = min(32, w.rows - half * 32);   // rows of this half (may be <= 0)
      const float inv = lsum == 0.f ? 0.f : 1.f / lsum;
      const int64_t at = (int64_t)w.slot * kNR + half * 32;
      if (!w.whole && quad == 0) {
        p.part_ml[(at + lane) * 2] = m;
        p.part_ml[(at + lane) * 2 + 1] = lsum;
      }
      // eight rows, four dims each, at a time
      auto rows_out = [&](auto put) {
#pragma unroll 1
        for (int c0 = 0; c0 < n_out; c0 += 8) {
          float o[4][8];
#pragma unroll
          for (int b = 0; b < 4; ++b) tc::tmem_ld8(ocol + b * kNR + c0, o[b]);
          tc::tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 8; ++c) put(c0 + c, o[0][c], o[1][c], o[2][c], o[3][c]);
        }
      };
      if (!w.whole) {
        float4* to = reinterpret_cast<float4*>(p.part_o + at * kC) + row;
        if (any)
          rows_out([&](int c, float a, float b, float x, float y) {
            if (c < n_out) to[c * (kC / 4)] = make_float4(a, b, x, y);
          });
      } else {
        uint2* to = reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(p.out) +
                                             (int64_t)(w.row0 + half * 32) * kC) + row;
        if (any) {
          rows_out([&](int c, float a, float b, float x, float y) {
            const float f = __shfl_sync(0xffffffffu, inv, c & 31);
            __nv_bfloat162 u = __floats2bfloat162_rn(a * f, b * f), v = __floats2bfloat162_rn(x * f, y * f);
            if (c < n_out)
              to[c * (kC / 4)] = make_uint2(*reinterpret_cast<uint32_t*>(&u), *reinterpret_cast<uint32_t*>(&v));
          });
        } else {
#pragma unroll 1
          for (int c = 0; c < n_out; ++c) to[c * (kC / 4)] = make_uint2(0u, 0u);
        }
      }
      if (any) {
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(oempty);
      }
    }
    if (tid == 0 && !posted) plan->post(p, nullptr);
  } else if (warp < 16) {
    // --------------------------------------------------------------------------- keys
    tc::set_regs<false, kRegKeys>();
    const int mine = (warp >> 2) & 1;              // of the two warpgroups: every other slot
    const uint32_t dst = tmem + lane_base + kKCol + 32 * mine;
    int g = 0, n = 0, u = 0;                       // tiles, this warpgroup's slots, pieces
    bool ok = true;
    const int kt = tid - 256;
    while (ok && next()) {
      if (w.tile0 >= w.tile1) continue;
      // Q in place from bf16 to f16 times 2^a. (Rows behind the unit's are another's: they take part
      // in the products, but not in the choice of a; what they give is not looked at.)
      if (!tc::mbar_wait_few(qfull, u & 1, abort_flag, p.err)) break;
      // (a thread's chunks are 16 bytes of one row in each of 18 places: row kt / 8 or 32 + kt / 8)
      __nv_bfloat162 top2 = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll 3
      for (int i = 0; i < 9 * kNR * 8 / 256; ++i) {
        if ((i & 1) * 32 + (kt >> 3) >= w.rows) continue;
        const uint4 v = *reinterpret_cast<const uint4*>(qbuf + 16 * (kt + 256 * i));
        const __nv_bfloat162* e = reinterpret_cast<const __nv_bfloat162*>(&v);
#pragma unroll
        for (int k = 0; k < 4; ++k) top2 = __hmax2(top2, __habs2(e[k]));
      }
      const uint32_t two = *reinterpret_cast<const uint32_t*>(&top2);
      uint32_t most = max(two << 16, two & 0xFFFF0000u);
      if (most >= 0x7F800000u) {                 // infinities among them: the largest of the others
        most = 0;
#pragma unroll 1
        for (int i = 0; i < 9 * kNR * 8 / 256 * 8; ++i) {
          const uint32_t at = 16 * (kt + 256 * (i >> 3)) + 2 * (i & 7);
          const uint32_t a = (uint32_t)(*reinterpret_cast<const uint16_t*>(qbuf + at) & 0x7FFF) << 16;
          if (((i >> 3) & 1) * 32 + (kt >> 3) < w.rows && a < 0x7F800000u) most = max(most, a);
        }
      }
      most = __reduce_max_sync(0xffffffffu, most);
      if (lane == 0) {
        qmax[warp - 8] = (int)most;
        tc::mbar_arrive(qmaxb);
      }
      if (!tc::mbar_wait_few(qmaxb, u & 1, abort_flag, p.err)) break;
#pragma unroll
      for (int i = 0; i < 8; ++i) most = max(most, (uint32_t)qmax[i]);
      // (at most 2^126: queries that small give f16 numbers with all their bits all the same)
      const int a = most == 0 ? 0 : min(126, 14 + 127 - (int)(most >> 23));
      const float f = __uint_as_float((uint32_t)(127 + a) << 23);
      if (kt == 0) qscale[u & 1] = __uint_as_float((uint32_t)(127 - a) << 23);
#pragma unroll 2
      for (int i = 0; i < 9 * kNR * 8 / 256; ++i) {
        uint4* at = reinterpret_cast<uint4*>(qbuf + 16 * (kt + 256 * i));
        uint4 v = *at;
        uint32_t e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
          e[k] = pack_f16(__uint_as_float(e[k] << 16) * f, __uint_as_float(e[k] & 0xFFFF0000u) * f);
        *at = make_uint4(e[0], e[1], e[2], e[3]);
      }
      tc::fence_proxy_async();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(qready);
      ++u;
      const int64_t first_from = kWindow ? latent_from(p, w.start + (w.row0 - w.seq_row0) / p.H) : 0;
      for (int t = w.tile0; t < w.tile1; ++t, ++g) {
        const int buf = g & 1, ring = g % 3;
        if (!tc::mbar_wait_few(rawfull + buf, (g >> 1) & 1, abort_flag, p.err)) { ok = false; break; }
        const uint32_t src = tc::smem_u32(raw + buf * kRaw + row * kRowBytes);
        const int64_t x0 = w.tile_at<kWindow>(t) * kTK;
        const int valid = tile_ok[buf] ? (int)min((int64_t)kTK, w.keys - x0) : 0;
        // a key that no row sees counts for nothing, whatever its row holds
        const bool dead = row >= valid || (kWindow && x0 + row < first_from && x0 + row >= p.sinks);
        if (mine != (g & 1)) {                     // the warpgroup with four slots
          float s = dead ? 0.f : srow[buf * kTK + row];
          if (!dead && s == 0.f) s = 0x1p-100f;    // (a row of zeros, as the insert writes it)
          info[ring * kTK + row] = make_float2(s, dead ? 0.f : __log2f(s));
          if (row == 0) tile_valid[ring] = valid;
        }
        __half* const scales = sc + ring * 32 * kScPitch + row;
#pragma unroll 1
        for (int j = (g ^ mine) & 1; j < 9; j += 2, ++n) {   // (one body for all: the instruction cache is small)
          uint32_t o[32];
          if (j < 8) {                             // 64 latent dims
            const uint4 c0 = lds128(src + 32 * j), c1 = lds128(src + 32 * j + 16);
            const uint32_t code[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
            const uint32_t block = dead ? 0u : lds32(src + kBlockAt + 4 * j);
            const uint32_t two[2] = {e4m3x2_to_f16x2(block), e4m3x2_to_f16x2(block >> 16)};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t f = __byte_perm(two[k >> 1], 0, k & 1 ? 0x3232 : 0x1010);
              scales[(4 * j + k) * kScPitch] = __ushort_as_half((unsigned short)f);   // (for the values)
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                uint32_t v[4];
                e2m1x8_to_f16(code[2 * k + q], v);
#pragma unroll
                for (int i = 0; i < 4; ++i) o[8 * k + 4 * q + i] = mul_f16(v[i], f);
              }
            }
          } else {                                 // the rotary part
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const uint4 c = lds128(src + kRopeAt + 16 * k);
              o[4 * k] = c.x;
              o[4 * k + 1] = c.y;
              o[4 * k + 2] = c.z;
              o[4 * k + 3] = c.w;
            }
          }
          if (j >= 7) {                            // this warpgroup's last look at the tile
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(rawempty + buf);
          }
          if ((j | 1) == 7) {                      // its last scales
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(infofull + ring);
          }
          if (n > 0) ok = tc::mbar_wait_few(kempty + mine, (n - 1) & 1, abort_flag, p.err);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc::fence_after_sync();
          tc::tmem_st32(dst, o);
          tc::tmem_wait_st();
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(kfull + mine);
        }
        if (!ok) break;
      }
    }
  } else if (warp < 24) {
    // ------------------------------------------------------------------------- values
    const int mine = (warp >> 2) & 1;              // of the two warpgroups: keys 64 mine ..
    const uint32_t dst = tmem + lane_base + kVCol;
    constexpr uint32_t kLow = 0x0F0F0F0Fu;
    int g = 0;
    bool ok = true;
    while (ok && next()) {
      for (int t = w.tile0; t < w.tile1; ++t, ++g) {
        const int buf = g & 1, ring = g % 3;
        if (!tc::mbar_wait_few(rawfull + buf, (g >> 1) & 1, abort_flag, p.err)) { ok = false; break; }
        const uint32_t src = tc::smem_u32(raw + buf * kRaw + 64 * mine * kRowBytes + 2 * row);
        uint32_t c0[8], c1[8];                     // this thread's codes of keys 4i, 4i + 2 and 4i + 1, 4i + 3
        auto load = [&](int part) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t at = src + (32 * part + 4 * i) * kRowBytes;
            c0[i] = lds16(at) | lds16(at + 2 * kRowBytes) << 16;
            c1[i] = lds16(at + kRowBytes) | lds16(at + 3 * kRowBytes) << 16;
          }
        };
        load(0);
        if (!tc::mbar_wait_few(infofull + ring, (g / 3) & 1, abort_flag, p.err)) { ok = false; break; }
        const uint32_t scales = tc::smem_u32(sc + (ring * 32 + row / 4) * kScPitch + 64 * mine);
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {              // 32 keys (q / 2), dims 4 row + q % 2 and + 2 more
          const int n = 2 * g + (q >> 1), slot = 2 * (q & 1) + mine;   // times around the ring
          const int low = (q & 1) * 4, high = 4 - low;
          uint32_t o[32];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t pair = ((c0[i] >> low) & kLow) | ((c1[i] << high) & ~kLow);
            uint32_t v[4];                         // (dim, keys 0 1), (dim + 2, keys 0 1), the same of 2 3
            e2m1x8_to_f16(pair, v);
            const uint2 f = lds64(scales + 64 * (q >> 1) + 8 * i);
            o[2 * i] = mul_f16(v[0], f.x);
            o[2 * i + 1] = mul_f16(v[2], f.y);
            o[16 + 2 * i] = mul_f16(v[1], f.x);
            o[16 + 2 * i + 1] = mul_f16(v[3], f.y);
          }
          if (q == 1) {                            // the last codes, before the wait: the buffer is wanted
            load(1);
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(rawempty + buf);
          }
          if (n > 0) ok = tc::mbar_wait_few(vempty + slot, (n - 1) & 1, abort_flag, p.err);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc::fence_after_sync();
          tc::tmem_st32(dst + slot * 32, o);
          tc::tmem_wait_st();
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(vfull + slot);
        }
        if (!ok) break;
      }
    }
  } else {
    tc::set_regs<false, kRegOther>();
    if (warp == 25 && lane == 0) {
      // ---------------------------------------------------------------------- copies
      int g = 0, u = 0, nq = 0, nr[2] = {0, 0};    // phases of each barrier given copies
      bool ok = true;
      const uint8_t* data = reinterpret_cast<const uint8_t*>(p.cache.data);
      // the next piece, or the end, for everybody
      auto publish = [&](LatentPiece& x) -> bool {
        const bool more = walk.next(p, x);
        if (!more) x.seq = -1;
        const int at = np % kPieces;
        if (np >= kPieces) ok = tc::mbar_wait_few(pieceempty + at, (np / kPieces - 1) & 1, abort_flag, p.err);
        if (!ok) return false;
        pieces[at] = x;
        tc::mbar_arrive(piecefull + at);
        ++np;
        return more;
      };
      LatentPiece after;
      bool more = false;
      for (bool have = publish(w); have && ok; w = after, have = more) {
        more = publish(after);
        if (w.tile0 >= w.tile1) continue;
        // the first raw tile does not wait for Q's buffer
        bool asked = false;
        auto ask_q = [&]() {
          asked = true;
          if (u > 0 && !tc::mbar_wait_few(qempty, (u - 1) & 1, abort_flag, p.err)) return false;
          tc::mbar_arrive_tx(qfull, 9 * kQBlock);
          ++nq;
          for (int b = 0; b < 9; ++b) tma_2d(qbuf + b * kQBlock, &qmap, b * 128, w.row0, qfull);
          return true;
        };
        for (int t = w.tile0; t < w.tile1; ++t, ++g) {
          const int buf = g & 1;
          const int64_t slot = tile_slot(p, w.seq, w.tile_at<kWindow>(t), kTK);
          const bool have = slot >= 0;
          if (!have) slot_ok(slot, p.err);
          if (!asked && u == 0 && !ask_q()) { ok = false; break; }
          if (g >= 2 && !tc::mbar_wait_few(rawempty + buf, ((g >> 1) - 1) & 1, abort_flag, p.err)) { ok = false; break; }
          tile_ok[buf] = have;
          ++nr[buf];
          if (have) {
            tc::mbar_arrive_tx(rawfull + buf, kRaw + kTK * 4);
#pragma unroll 1
            for (int i = 0; i < 4; ++i)
              tc::bulk_g2s(raw + buf * kRaw + i * (kRaw / 4), data + slot * kRowBytes + i * (kRaw / 4), kRaw / 4,
                           rawfull + buf);
            tc::bulk_g2s(srow + buf * kTK, p.cache.scale + slot, kTK * 4, rawfull + buf);
          } else {
            tc::mbar_arrive(rawfull + buf);
          }
          if (!asked && !ask_q()) { ok = false; break; }
        }
        ++u;
      }
      if (*abort_flag) {                          // leave no copy in flight
        if (nq > 0) tc::mbar_wait_drain(qfull, (nq - 1) & 1);
        for (int i = 0; i < 2; ++i)
          if (nr[i] > 0) tc::mbar_wait_drain(rawfull + i, (nr[i] - 1) & 1);
      }
    } else if (warp == 24) {
      // ------------------------------------------------------------ products for S^T
      constexpr uint32_t idesc_s = tc::idesc_f16(kTK, kNR);
      const uint32_t q_lo = tc::uniform(tc::sdesc_lo(tc::smem_u32(qbuf), 16));
      const uint32_t d = tc::uniform(tmem + kSCol);
      int g = 0, u = 0, n = 0;
      bool ok = true;
      auto wait_all = [&](uint64_t* bar, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, tc::mbar_wait_few(bar, parity, abort_flag, p.err));
      };
      while (ok && next()) {
        if (w.tile0 >= w.tile1) continue;
        if (!wait_all(qready, u & 1)) break;
        for (int t = w.tile0; t < w.tile1; ++t, ++g) {
          if (g > 0 && !wait_all(sfree, (g - 1) & 1)) { ok = false; break; }
          bool ready = false;
#pragma unroll 1
          for (int j = 0; j < 9; ++j, ++n) {
            const int slot = n % kKeySlots;
            const uint32_t a = tc::uniform(tmem + kKCol + slot * 32), b = tc::uniform(q_lo + ((j * kQBlock) >> 4));
            const uint32_t add = tc::uniform(j > 0);
            if (!__all_sync(0xffffffffu, ready) && !wait_all(kfull + slot, (n / kKeySlots) & 1)) { ok = false; break; }
            tc::fence_after_sync();
            if (tc::elect_one()) {
#pragma unroll
              for (int s = 0; s < 4; ++s)          // 16 dims, 8 columns of A, 32 bytes of B
                tc::mma_ta_lo<idesc_s>(d, a + 8 * s, b + 2 * s, s ? 1u : add);
              tc::mma_commit(kempty + slot);
              if (j == 8) {
                tc::mma_commit(sfull);
                if (t + 1 == w.tile1) tc::mma_commit(qempty);
              }
            }
            // (the next slot's barrier is asked as this one's products go out)
            ready = j < 8 && tc::mbar_test(kfull + (n + 1) % kKeySlots, ((n + 1) / kKeySlots) & 1);
            __syncwarp();
          }
          if (!ok) break;
        }
        ++u;
      }
      if (tc::elect_one()) {
        tc::mma_commit(done);
        tc::mbar_wait_drain(done, 0);
      }
    } else if (warp == 26) {
      // ------------------------------------------------------------ products for O^T
      constexpr uint32_t idesc_o = tc::idesc_f16(128, kNR, false, true);
      const uint32_t p_lo = tc::uniform(tc::sdesc_lo(tc::smem_u32(pbuf), 16));
      const uint32_t d = tc::uniform(tmem + kOCol);
      int g = 0, u = 0, n = 0;
      bool ok = true;
      auto wait_all = [&](uint64_t* bar, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, tc::mbar_wait_few(bar, parity, abort_flag, p.err));
      };
      while (ok && next()) {
        if (w.tile0 >= w.tile1) continue;
        for (int t = w.tile0; t < w.tile1; ++t, ++g) {
          const uint32_t acc = tc::uniform(t > w.tile0);
          if (!wait_all(pfull, g & 1)) { ok = false; break; }
          if (t == w.tile0 && u > 0 && !wait_all(oempty, (u - 1) & 1)) { ok = false; break; }
          bool ready = false;
#pragma unroll 1
          for (int j = 0; j < 8; ++j, ++n) {
            const int slot = n % kValueSlots;
            // slot j: keys 64 (j % 2) + 32 (j / 4) .., dims 4l + j / 2 % 2 and + 2 more
            const uint32_t a = tc::uniform(tmem + kVCol + slot * 32), at = tc::uniform(d + ((j >> 1) & 1) * kNR);
            const uint32_t b = tc::uniform(p_lo + ((((j & 1) * 4 + (j >> 2) * 2) * 2048) >> 4));
            const uint32_t add = tc::uniform(j == 0 || j == 2 ? acc : 1u);
            if (!__all_sync(0xffffffffu, ready) && !wait_all(vfull + slot, (n / kValueSlots) & 1)) { ok = false; break; }
            tc::fence_after_sync();
            ready = j < 7 && tc::mbar_test(vfull + (n + 1) % kValueSlots, ((n + 1) / kValueSlots) & 1);
            if (tc::elect_one()) {
#pragma unroll
              for (int s = 0; s < 2; ++s) {        // 16 keys, 8 columns of A, 2 KB of B
                tc::mma_ta_lo<idesc_o>(at, a + 8 * s, b + ((s * 2048) >> 4), s ? 1u : add);
                tc::mma_ta_lo<idesc_o>(at + 2 * kNR, a + 16 + 8 * s, b + ((s * 2048) >> 4), s ? 1u : add);
              }
              tc::mma_commit(vempty + slot);
              if (j == 7) tc::mma_commit(pvdone);
            }
            __syncwarp();
          }
          if (!ok) break;
        }
        ++u;
      }
      if (tc::elect_one()) {
        tc::mma_commit(done + 1);
        tc::mbar_wait_drain(done + 1, 0);
      }
    }
    __syncwarp();
  }

  tc::fence_before_sync();
  __syncthreads();
  if (warp == 24) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace

cudaError_t launch_latent_attn_fp4_tc(const LatentAttnParams& p, cudaStream_t st) {
  CUtensorMap qmap;
  const int64_t rows = (int64_t)p.n_tokens * p.H;
  if (!encode_byte_rows_map(&qmap, p.q, (uint64_t)rows, (kC + kR) * 2, 128, kNR)) return cudaErrorInvalidValue;
  auto go = [&](auto kernel) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (e != cudaSuccess) return e;
    return launch_pdl(kernel, dim3((unsigned)p.plan.ctas), dim3(kThreads), kSmemBytes, st, p, qmap);
  };
  return p.window > 0 ? go(latent_attn_fp4_tc<true>) : go(latent_attn_fp4_tc<false>);
}

}  // namespace v4a
