// Latent attention on CUDA cores: rotary positions, the cache's insert and gather, attention in
// both forms for any supported shape and type, and the merge of split results.
//
//   rope    y = amp (x0 c - x1 s, x0 s + x1 c)
//   insert  row = [ gamma c / sqrt(mean c^2 + eps) | rope(k_pe) ]
//   attention, absorbed  out[t, h] = sum_x softmax_x(scale q . row_x) row_x[0:C]
//   attention, expanded  out[i, h] = sum_x softmax_x(scale (q_n . k + q_r . k_pe)) v
//
// None of these kernels lets its successor start early (no pdl_trigger): other kernels of the
// library read their queries before they wait for the kernel before them, which is right only
// if that kernel's writes are complete when they start.
#include "kernels.h"
#include "latent.h"

namespace v4a {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

// A kernel parameter array read with an index of each thread's own: through its address, as
// ordinary memory. (From the constant bank the lanes' different words come one at a time.)
__device__ __forceinline__ const float* by_address(const float* v) {
  const float* q;
  asm volatile("mov.b64 %0, %1;" : "=l"(q) : "l"(v));
  return q;
}

// ------------------------------------------------------------------------------- rope
// Bound: HBM for many tokens (8192 x 64 heads x 64 dims fp32: 44 us, 6.1 TB/s), latency for few
// (4.3 us). A thread takes `VEC` consecutive elements of
// each half (half layout) or 2 VEC consecutive ones (interleaved): VEC pairs. The block's
// tokens' cosines and sines are computed once, into shared memory, for all heads.
template <typename T, int N> struct Pack { T v[N]; };
template <typename T, int N>
__device__ __forceinline__ void load_pack(const T* p, float (&f)[N]) {
  if constexpr (N * sizeof(T) == 16) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const T* e = reinterpret_cast<const T*>(&u);
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = Elem<T>::to_f(e[i]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = Elem<T>::to_f(p[i]);
  }
}
template <typename T, int N>
__device__ __forceinline__ void store_pack(T* p, const float (&f)[N]) {
  if constexpr (N * sizeof(T) == 16) {
    uint4 u;
    T* e = reinterpret_cast<T*>(&u);
#pragma unroll
    for (int i = 0; i < N; ++i) e[i] = Elem<T>::from_f(f[i]);
    *reinterpret_cast<uint4*>(p) = u;
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = Elem<T>::from_f(f[i]);
  }
}

constexpr int kRopeThreads = 256;
constexpr int kRopeTable = 2048;   // cosine/sine pairs of a block's tokens

// kHalf: W elements from each half a step; else W consecutive elements (W/2 pairs).
template <typename T, bool kHalf, int W>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p, int tokens,
                                                            int heads) {
  __shared__ float2 cs[kRopeTable];
  __shared__ uint8_t bad[kRopeTable];
  const int np = p.rot.dim / 2;
  const int t0 = blockIdx.x * tokens, h0 = blockIdx.y * heads;
  const int nt = min(tokens, p.n_tokens - t0), nh = min(heads, p.n_heads - h0);
  pdl_wait();
  for (int k = threadIdx.x; k < nt * np; k += kRopeThreads) {
    const int t = k / np, i = k - t * np;
    const int64_t pos = __ldg(p.pos + t0 + t);
    const bool b = pos < 0 || pos >= V4A_MAX_POS;
    float c = 1.f, s = 0.f;
    if (!b)
      rot_cs(pos, by_address(p.rot.phi_hi)[i], by_address(p.rot.phi_lo)[i], by_address(p.rot.psi_hi)[i],
             by_address(p.rot.psi_lo)[i], c, s);
    if (i == 0) {
      bad[t] = b;
      if (b && h0 == 0) raise_err(p.err, V4A_DEV_BAD_POS);
    }
    cs[k] = make_float2(c * p.rot.amp, (p.inverse ? -s : s) * p.rot.amp);
  }
  __syncthreads();
  const int steps = (kHalf ? np : p.rot.dim) / W;    // of a (token, head) row
  const int per_t = nh * steps;
  for (int k = threadIdx.x; k < nt * per_t; k += kRopeThreads) {
    const int t = k / per_t, r = k - t * per_t, h = r / steps, e = (r - h * steps) * W;
    if (bad[t]) continue;
    const T* x = reinterpret_cast<const T*>(p.x) + (int64_t)(t0 + t) * p.x_ts + (int64_t)(h0 + h) * p.x_hs + e;
    T* y = reinterpret_cast<T*>(p.y) + (int64_t)(t0 + t) * p.y_ts + (int64_t)(h0 + h) * p.y_hs + e;
    if constexpr (kHalf) {
      float a[W], b[W];
      load_pack<T, W>(x, a);
      load_pack<T, W>(x + np, b);
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const float2 c = cs[t * np + e + i];
        const float u = a[i] * c.x - b[i] * c.y;
        b[i] = a[i] * c.y + b[i] * c.x;
        a[i] = u;
      }
      store_pack<T, W>(y, a);
      store_pack<T, W>(y + np, b);
    } else {
      float a[W];
      load_pack<T, W>(x, a);
#pragma unroll
      for (int i = 0; i < W; i += 2) {
        const float2 c = cs[t * np + ((e + i) >> 1)];
        const float u = a[i] * c.x - a[i + 1] * c.y;
        a[i + 1] = a[i] * c.y + a[i + 1] * c.x;
        a[i] = u;
      }
      store_pack<T, W>(y, a);
    }
  }
}

template <typename T>
int run_rope(const RopeParams& p, cudaStream_t st) {
  constexpr int kV = 16 / (int)sizeof(T);
  const int np = p.rot.dim / 2;
  const bool half = p.rot.layout == V4A_ROPE_HALF;
  // 16-byte accesses when every row (and its second half) starts on a 16-byte boundary
  const bool wide = reinterpret_cast<uintptr_t>(p.x) % 16 == 0 && reinterpret_cast<uintptr_t>(p.y) % 16 == 0 &&
                    p.x_ts % kV == 0 && p.x_hs % kV == 0 && p.y_ts % kV == 0 && p.y_hs % kV == 0 &&
                    (half ? np : p.rot.dim) % kV == 0;
  const int w = wide ? kV : (half ? 1 : 2);
  const int steps = (half ? np : p.rot.dim) / w;
  // a block takes about 1024 steps: all heads of a few tokens, or some heads of one
  int heads = p.n_heads, tokens = 1;
  if ((int64_t)heads * steps > 1024) heads = 1024 / steps > 0 ? 1024 / steps : 1;
  else tokens = 1024 / (heads * steps);
  if (tokens > kRopeTable / np) tokens = kRopeTable / np;
  const int64_t gx = ((int64_t)p.n_tokens + tokens - 1) / tokens, gy = ((int64_t)p.n_heads + heads - 1) / heads;
  if (gy > 65535) return V4A_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)gx, (unsigned)gy);
  cudaError_t e;
  if (half)
    e = wide ? launch_pdl(rope_kernel<T, true, kV>, grid, dim3(kRopeThreads), 0, st, p, tokens, heads)
             : launch_pdl(rope_kernel<T, true, 1>, grid, dim3(kRopeThreads), 0, st, p, tokens, heads);
  else
    e = wide ? launch_pdl(rope_kernel<T, false, kV>, grid, dim3(kRopeThreads), 0, st, p, tokens, heads)
             : launch_pdl(rope_kernel<T, false, 2>, grid, dim3(kRopeThreads), 0, st, p, tokens, heads);
  return e == cudaSuccess ? V4A_OK : V4A_ERR_CUDA;
}

// ----------------------------------------------------------------------------- insert
// A block takes up to 32 tokens, whose positions and pool rows are looked up first, a thread a
// token; a warp then takes one token after the other: the latent row in registers (16-byte
// vectors, lane l taking vectors l, l + 32, ..; the next token's row is requested before this
// one is worked on), its mean square by shuffles, and the rotary part, lane i turning pairs i,
// i + 32 with rates it keeps. Bound: latency at decode (4.1 us), HBM for prompts (each row is read and
// written once: 14,618 tokens 11.8 us, 2.9 TB/s, of which about 4 are launch and lookups).
constexpr int kInsertWarps = 8, kInsertTokens = 32;

template <typename T, int kMaxC>
struct InsertRow {
  static constexpr int kV = 16 / (int)sizeof(T), kMaxVec = kMaxC / kV / 32;
  uint4 v[kMaxVec];
  T x0[2], x1[2];
  __device__ __forceinline__ void load(const LatentInsertParams& p, int64_t t, int lane) {
    const T* c = reinterpret_cast<const T*>(p.c) + t * p.c_stride;
    const T* k = reinterpret_cast<const T*>(p.k_pe) + t * p.k_stride;
    const int nv = p.C / kV, np = p.rot.dim / 2;
    const bool half = p.rot.layout == V4A_ROPE_HALF;
#pragma unroll
    for (int i = 0; i < kMaxVec; ++i)
      if (lane + 32 * i < nv) v[i] = *reinterpret_cast<const uint4*>(c + (lane + 32 * i) * kV);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int i = lane + 32 * j;
      if (i < np) {
        x0[j] = k[half ? i : 2 * i];
        x1[j] = k[half ? i + np : 2 * i + 1];
      }
    }
  }
};

template <typename T, int kMaxC>
__global__ void __launch_bounds__(32 * kInsertWarps, kMaxC <= 512 ? 3 : 2)
    latent_insert_kernel(const __grid_constant__ LatentInsertParams p, int tokens) {
  using Row = InsertRow<T, kMaxC>;
  constexpr int kV = Row::kV, kMaxVec = Row::kMaxVec;
  __shared__ int64_t slots[kInsertTokens], at[kInsertTokens];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int np = p.rot.dim / 2, nv = p.C / kV;
  const int t0 = blockIdx.x * tokens, nt = min(tokens, p.n_tokens - t0);
  float rate[2][4];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int i = min(lane + 32 * j, np - 1);
    rate[j][0] = by_address(p.rot.phi_hi)[i];
    rate[j][1] = by_address(p.rot.phi_lo)[i];
    rate[j][2] = by_address(p.rot.psi_hi)[i];
    rate[j][3] = by_address(p.rot.psi_lo)[i];
  }
  pdl_wait();
  Row next;
  if (warp < nt) next.load(p, t0 + warp, lane);
  if (threadIdx.x < nt) {
    const int t = t0 + threadIdx.x, b = find_seq(p.cu, p.n_seq, t);
    int64_t slot = -1, pos = 0;
    if (b >= 0) {
      pos = __ldg(p.start + b) + (t - __ldg(p.cu + b));
      if (pos < 0 || pos >= V4A_MAX_POS) {
        raise_err(p.err, V4A_DEV_BAD_POS);
      } else {
        slot = slot_of(p.cache, b, pos);
        slot_ok(slot, p.err);
      }
    }
    slots[threadIdx.x] = slot;
    at[threadIdx.x] = pos;
  }
  __syncthreads();
  const bool half = p.rot.layout == V4A_ROPE_HALF;
  for (int k = warp; k < nt; k += kInsertWarps) {
    const Row in = next;
    if (k + kInsertWarps < nt) next.load(p, t0 + k + kInsertWarps, lane);
    const int64_t slot = slots[k], pos = at[k];
    if (slot < 0) continue;
    T* row = reinterpret_cast<T*>(p.cache.data) + slot * (int64_t)p.cache.width;
    float r = 1.f;
    if (p.gamma) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < kMaxVec; ++i)
        if (lane + 32 * i < nv) {
          const T* e = reinterpret_cast<const T*>(&in.v[i]);
#pragma unroll
          for (int q = 0; q < kV; ++q) {
            const float f = Elem<T>::to_f(e[q]);
            ss = fmaf(f, f, ss);
          }
        }
      r = 1.0f / sqrtf(warp_sum(ss) / (float)p.C + p.eps);
    }
#pragma unroll
    for (int i = 0; i < kMaxVec; ++i) {
      const int v = lane + 32 * i;
      if (v >= nv) continue;
      const T* e = reinterpret_cast<const T*>(&in.v[i]);
      float f[kV];
#pragma unroll
      for (int q = 0; q < kV; ++q) f[q] = Elem<T>::to_f(e[q]);
      if (p.gamma) {
#pragma unroll
        for (int q = 0; q < kV; q += 4) {
          const float4 g = __ldg(reinterpret_cast<const float4*>(p.gamma + v * kV + q));
          f[q] *= r * g.x;
          f[q + 1] *= r * g.y;
          f[q + 2] *= r * g.z;
          f[q + 3] *= r * g.w;
        }
      }
      store_pack<T, kV>(row + v * kV, f);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int i = lane + 32 * j;
      if (i >= np) continue;
      float cc, sn;
      rot_cs(pos, rate[j][0], rate[j][1], rate[j][2], rate[j][3], cc, sn);
      cc *= p.rot.amp;
      sn *= p.rot.amp;
      const float a = Elem<T>::to_f(in.x0[j]), b = Elem<T>::to_f(in.x1[j]);
      row[p.C + (half ? i : 2 * i)] = Elem<T>::from_f(a * cc - b * sn);
      row[p.C + (half ? i + np : 2 * i + 1)] = Elem<T>::from_f(a * sn + b * cc);
    }
  }
}

// ----------------------------------------------------------------------------- gather
// A block copies `rows` rows: their pool rows are looked up first, a thread a row, then all
// threads copy 16-byte vectors, eight in flight each. Bound: HBM (176,793 rows: 64 us, 6.4 TB/s);
// for few rows, latency (3.7 us).
constexpr int kGatherRows = 64, kGatherThreads = 256;

__global__ void __launch_bounds__(kGatherThreads) latent_gather_kernel(const __grid_constant__ LatentGatherParams p,
                                                                       int rows) {
  __shared__ int64_t slots[kGatherRows];   // pool row, -1: zeros, -2: no row of the batch
  const int r0 = blockIdx.x * rows, nr = min(rows, p.n_rows - r0);
  pdl_wait();
  if (threadIdx.x < nr) {
    const int t = r0 + threadIdx.x;
    const int b = find_seq(p.cu, p.n_seq, t);
    int64_t s = -2;
    if (b >= 0) {
      s = slot_of(p.cache, b, __ldg(p.start + b) + (t - __ldg(p.cu + b)));
      if (!slot_ok(s, p.err)) s = -1;
    }
    slots[threadIdx.x] = s;
  }
  __syncthreads();
  const int nv = p.row_bytes / 16, total = nr * nv;
  const uint4* pool = reinterpret_cast<const uint4*>(p.cache.data);
  uint4* out = reinterpret_cast<uint4*>(p.out) + (int64_t)r0 * nv;
  const int dr = kGatherThreads / nv, dc = kGatherThreads % nv;   // a step of all threads
  int r = threadIdx.x / nv, c = threadIdx.x % nv;
  for (int k = threadIdx.x; k < total; k += 8 * kGatherThreads) {
    uint4 v[8];
    bool put[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      put[i] = false;
      if (k + i * kGatherThreads < total) {
        const int64_t s = slots[r];
        put[i] = s != -2;
        v[i] = s < 0 ? make_uint4(0, 0, 0, 0) : __ldg(pool + s * nv + c);
        r += dr;
        c += dc;
        if (c >= nv) { c -= nv; ++r; }
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (put[i]) out[k + i * kGatherThreads] = v[i];
  }
}

// -------------------------------------------------------------------------- attention
// A unit of 16 query rows against tiles of 32 keys, in fp32. Warp w holds rows 2w, 2w + 1;
// lane x computes their products with key x of the tile (the key tile's rows are padded by one
// word, so the lanes' reads fall in different banks), the softmax statistics go by shuffles,
// and lane l accumulates output dims l, l + 32, .. . Bound: shared-memory reads (a word a product)
// and fp32 FMA: absorbed 14-17 TFLOP/s with 512 or 256 latent dims (8 sequences x 8,192 tokens, 64
// heads, 512 + 64, fp32: 538 us), 6 with 128; expanded 5-9 (2,048-token prompt, 16 heads, fp32,
// 128 + 64 / 128: 2.5 ms). The tensor-core kernels take 33 and 44 us at these sizes.
constexpr int kGenRows = 16, kGenKeys = 32, kGenThreads = 256;

struct RowState {
  float m, l;
};

// One tile: s (log2 units, -inf where masked) of this lane's key for one row; returns p and
// the factor on what is accumulated.
__device__ __forceinline__ float softmax_step(float s, RowState& st, float& corr) {
  const float m = fmaxf(st.m, warp_max(s));
  const float ref = m == -INFINITY ? 0.f : m;
  const float pr = exp2f(s - ref);
  corr = exp2f(st.m - ref);                 // 0 from -inf
  st.l = st.l * corr + warp_sum(pr);
  st.m = m;
  return pr;
}

template <typename T>
__device__ __forceinline__ void load_row_f(float* dst, const T* src, int n, int lane) {
  constexpr int kV = 16 / (int)sizeof(T);
  for (int v = lane; v < n / kV; v += 32) {
    float f[kV];
    load_pack<T, kV>(src + v * kV, f);
#pragma unroll
    for (int k = 0; k < kV; ++k) dst[v * kV + k] = f[k];
  }
}

// kNV: 32-dim groups of the output. kPaged: absorbed form (V = the row's first dims).
template <typename T, int kNV, bool kPaged, typename P>
__global__ void __launch_bounds__(kGenThreads) latent_attn_gen(const __grid_constant__ P p) {
  extern __shared__ __align__(16) float sm[];   // read as float4
  __shared__ int32_t pre[kPaged ? V4A_MAX_SEQ + 1 : 1];
  __shared__ int32_t warp_tot[kGenThreads / 32];
  __shared__ uint8_t kvalid[kGenKeys];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int DK, DV;
  if constexpr (kPaged) { DK = p.C + p.R; DV = p.C; } else { DK = p.DN + p.DR; DV = p.DV; }
  const int KS = DK + 1;
  float* qs = sm;                              // [16][DK]
  float* ks = qs + kGenRows * DK;              // [32][KS]
  float* vs = kPaged ? ks : ks + kGenKeys * KS;   // [32][VS]
  const int VS = kPaged ? KS : DV;
  pdl_wait();

  LatentWalk walk;
  LatentPiece w;
  int seq = 0, head = 0, item = blockIdx.x;
  bool posted = false;
  if constexpr (kPaged) {
    walk.begin(p, pre, warp_tot);
  }
  for (;;) {
    // ---- the next unit: its query rows and its keys
    int rows, t0, t1, qa = 0, ka = 0, nq = 0, nk = 0;
    int64_t keys;
    if constexpr (kPaged) {
      const bool more = walk.next(p, w);
      if (threadIdx.x == 0 && !posted) walk.post(p, more ? &w : nullptr);
      posted = true;
      if (!more) break;
      rows = w.rows;
      keys = w.keys;
      t0 = w.tile0;
      t1 = w.tile1;
      if (rows == 0) continue;
    } else {
      // item = (16-row block of a sequence, head); blocks counted sequence by sequence
      int blk = item / p.H, b = 0;
      head = item - blk * p.H;
      item += gridDim.x;
      for (; b < p.n_seq; ++b) {
        qa = cu_at(p.cu_q, b, p.n_q);
        nq = max(cu_at(p.cu_q, b + 1, p.n_q) - qa, 0);
        const int n = (nq + kGenRows - 1) / kGenRows;
        if (blk < n) break;
        blk -= n;
      }
      if (b == p.n_seq) break;
      seq = blk * kGenRows;                    // first query of the block
      ka = cu_at(p.cu_k, b, p.n_k);
      nk = max(cu_at(p.cu_k, b + 1, p.n_k) - ka, 0);
      rows = min(kGenRows, nq - seq);
      keys = p.causal ? max(0, nk - nq + seq + rows) : nk;
      t0 = 0;
      t1 = (int)((keys + kGenKeys - 1) / kGenKeys);
    }
    __syncthreads();                           // the previous unit's reads of qs
    for (int r = warp; r < kGenRows; r += kGenThreads / 32) {
      int64_t row = 0;
      if constexpr (kPaged) row = (int64_t)w.row0 + r; else row = (int64_t)(qa + seq + r) * p.H + head;
      if (r < rows) load_row_f<T>(qs + r * DK, reinterpret_cast<const T*>(p.q) + row * DK, DK, lane);
      else for (int d = lane; d < DK; d += 32) qs[r * DK + d] = 0.f;
    }
    int64_t vis[2];
    RowState st[2];
    float o[2][kNV];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = 2 * warp + i;
      if constexpr (kPaged) {
        const int tok = (w.row0 + r - w.seq_row0) / p.H;
        vis[i] = r < rows ? latent_visible(p, w.start + tok) : 0;
        if (r < rows && lane == 0) latent_report_pos(p, w.start + tok);
      } else {
        vis[i] = r >= rows ? 0 : p.causal ? max(0, nk - nq + seq + r + 1) : nk;
      }
      st[i].m = -INFINITY;
      st[i].l = 0.f;
#pragma unroll
      for (int d = 0; d < kNV; ++d) o[i][d] = 0.f;
    }
    for (int t = t0; t < t1; ++t) {
      const int64_t x0 = (int64_t)t * kGenKeys;
      __syncthreads();
      // lane k resolves key k's row; a warp then copies four rows
      int64_t at = -1;
      if (x0 + lane < keys) {
        if constexpr (kPaged) {
          at = slot_of(p.cache, w.seq, x0 + lane);
          if (at < 0 && warp == 0) slot_ok(at, p.err);
        } else {
          at = ka + x0 + lane;
        }
      }
      if (warp == 0) kvalid[lane] = at >= 0;
#pragma unroll
      for (int i = 0; i < kGenKeys / 8; ++i) {
        const int k = warp * (kGenKeys / 8) + i;
        const int64_t g = __shfl_sync(0xffffffffu, at, k);
        if (g >= 0) {
          if constexpr (kPaged) {
            load_row_f<T>(ks + k * KS, reinterpret_cast<const T*>(p.cache.data) + g * (int64_t)DK, DK, lane);
          } else {
            const T* key = reinterpret_cast<const T*>(p.k) + g * p.k_ts + (int64_t)head * p.k_hs;
            const T* value = reinterpret_cast<const T*>(p.v) + g * p.v_ts + (int64_t)head * p.v_hs;
            load_row_f<T>(ks + k * KS, key, p.DN, lane);
            load_row_f<T>(ks + k * KS + p.DN, reinterpret_cast<const T*>(p.k_pe) + g * p.pe_ts, p.DR, lane);
            load_row_f<T>(vs + k * VS, value, DV, lane);
          }
        } else {
          for (int d = lane; d < DK; d += 32) ks[k * KS + d] = 0.f;
          if (!kPaged) for (int d = lane; d < DV; d += 32) vs[k * VS + d] = 0.f;
        }
      }
      __syncthreads();
      float s0 = 0.f, s1 = 0.f;
      const float* q0 = qs + 2 * warp * DK;
      const float* q1 = q0 + DK;
      const float* kr = ks + lane * KS;
#pragma unroll 4
      for (int d = 0; d < DK; d += 4) {
        const float4 a = *reinterpret_cast<const float4*>(q0 + d), b = *reinterpret_cast<const float4*>(q1 + d);
        const float k0 = kr[d], k1 = kr[d + 1], k2 = kr[d + 2], k3 = kr[d + 3];
        s0 = fmaf(a.x, k0, fmaf(a.y, k1, fmaf(a.z, k2, fmaf(a.w, k3, s0))));
        s1 = fmaf(b.x, k0, fmaf(b.y, k1, fmaf(b.z, k2, fmaf(b.w, k3, s1))));
      }
      const float k2e = p.scale * kLog2e;
      const bool ok = kvalid[lane];
      s0 = ok && x0 + lane < vis[0] ? s0 * k2e : -INFINITY;
      s1 = ok && x0 + lane < vis[1] ? s1 * k2e : -INFINITY;
      float c0, c1;
      const float p0 = softmax_step(s0, st[0], c0), p1 = softmax_step(s1, st[1], c1);
#pragma unroll
      for (int d = 0; d < kNV; ++d) {
        o[0][d] *= c0;
        o[1][d] *= c1;
      }
      for (int k = 0; k < kGenKeys; ++k) {
        const float a = __shfl_sync(0xffffffffu, p0, k), b = __shfl_sync(0xffffffffu, p1, k);
        if (x0 + k >= vis[0] && x0 + k >= vis[1]) continue;   // alike in every lane
        const float* v = vs + k * VS + lane;
#pragma unroll
        for (int d = 0; d < kNV; ++d) {
          const float x = lane + 32 * d < DV ? v[32 * d] : 0.f;
          if (x0 + k < vis[0]) o[0][d] = fmaf(a, x, o[0][d]);
          if (x0 + k < vis[1]) o[1][d] = fmaf(b, x, o[1][d]);
        }
      }
    }
    // ---- the unit's result, or this range's share of it
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = 2 * warp + i;
      if (r >= rows) continue;
      if constexpr (kPaged) {
        if (!w.whole) {
          const int64_t at = (int64_t)w.slot * kGenRows + r;
          if (lane == 0) {
            p.part_ml[at * 2] = st[i].m;
            p.part_ml[at * 2 + 1] = st[i].l;
          }
#pragma unroll
          for (int d = 0; d < kNV; ++d)
            if (lane + 32 * d < DV) p.part_o[at * DV + lane + 32 * d] = o[i][d];
          continue;
        }
      }
      int64_t row = 0;
      if constexpr (kPaged) row = (int64_t)w.row0 + r; else row = (int64_t)(qa + seq + r) * p.H + head;
      const float inv = st[i].l == 0.f ? 0.f : 1.f / st[i].l;
      T* out = reinterpret_cast<T*>(p.out) + row * DV;
#pragma unroll
      for (int d = 0; d < kNV; ++d)
        if (lane + 32 * d < DV) out[lane + 32 * d] = Elem<T>::from_f(o[i][d] * inv);
    }
  }
}

// ------------------------------------------------------------------------------ merge
// The results of a unit whose tiles fell to several teams: out = sum_i w_i o_i / sum_i w_i l_i
// with w_i = 2^(m_i - max). Block (cta, rows, dims) does the job that the CTA posted; a warp
// 256 dims of a row.
// Bound: latency (job, statistics, partial results: three loads in a row).
constexpr int kMergeWarps = 8;

template <typename T>
__global__ void __launch_bounds__(32 * kMergeWarps) latent_merge_kernel(const __grid_constant__ LatentAttnParams p) {
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int4 job = *reinterpret_cast<const int4*>(p.part_job + 4 * blockIdx.x);
  const int r = blockIdx.y * kMergeWarps + warp, NR = p.plan.NR;
  if (r >= job.x) return;
  const int U = job.w, g = blockIdx.x / U, member = blockIdx.x % U, first = g - 1, last = job.z;
  const int d0 = blockIdx.z * 256 + lane * 4;
  // team g - 1's piece begins the unit (slot 1), the others begin inside it (slot 0)
  auto slot = [&](int i) { return (int64_t)(((i * U + member) << 1) + (i == first ? 1 : 0)) * NR + r; };
  auto load = [&](int i, float4 (&v)[2]) {
    const float* o = p.part_o + slot(i) * p.C + d0;
#pragma unroll
    for (int j = 0; j < 2; ++j)
      v[j] = d0 + 128 * j < p.C ? *reinterpret_cast<const float4*>(o + 128 * j) : make_float4(0.f, 0.f, 0.f, 0.f);
  };
  // the statistics, a lane a piece, and the first pieces' results are requested together (an
  // empty range's result was not written: it is left out below)
  float4 v[4][2];
  float2 ml = make_float2(-INFINITY, 0.f);
  if (first + lane <= last) ml = *reinterpret_cast<const float2*>(p.part_ml + slot(first + lane) * 2);
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (first + k <= last) load(first + k, v[k]);
  float m = ml.x;
  for (int i = first + 32 + lane; i <= last; i += 32) m = fmaxf(m, p.part_ml[slot(i) * 2]);
  m = warp_max(m);
  const float ref = m == -INFINITY ? 0.f : m;
  float l = 0.f;
  float4 a[2] = {};
  for (int i0 = first; i0 <= last; i0 += 32) {
    if (i0 > first) ml = i0 + lane <= last ? *reinterpret_cast<const float2*>(p.part_ml + slot(i0 + lane) * 2)
                                           : make_float2(-INFINITY, 0.f);
    const float w = ml.x != -INFINITY || ml.y != 0.f ? exp2f(ml.x - ref) : 0.f;
    l = fmaf(w, ml.y, l);
    const int cnt = min(32, last - i0 + 1);
    for (int k0 = 0; k0 < cnt; k0 += 4) {
      if (k0 > 0 || i0 > first) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (k0 + k < cnt) load(i0 + k0 + k, v[k]);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float wk = __shfl_sync(0xffffffffu, w, (k0 + k) & 31);
        if (k0 + k >= cnt || wk == 0.f) continue;   // alike in every lane
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          a[j].x = fmaf(wk, v[k][j].x, a[j].x);
          a[j].y = fmaf(wk, v[k][j].y, a[j].y);
          a[j].z = fmaf(wk, v[k][j].z, a[j].z);
          a[j].w = fmaf(wk, v[k][j].w, a[j].w);
        }
      }
    }
  }
  l = warp_sum(l);
  const float inv = l == 0.f ? 0.f : 1.f / l;
  T* out = reinterpret_cast<T*>(p.out) + (int64_t)(job.y + r) * p.C + d0;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    if (d0 + 128 * j >= p.C) continue;
    float f[4] = {a[j].x * inv, a[j].y * inv, a[j].z * inv, a[j].w * inv};
    if constexpr (sizeof(T) == 4) {
      store_pack<T, 4>(out + 128 * j, f);
    } else {
      uint2 u;
      T* e = reinterpret_cast<T*>(&u);
#pragma unroll
      for (int k = 0; k < 4; ++k) e[k] = Elem<T>::from_f(f[k]);
      *reinterpret_cast<uint2*>(out + 128 * j) = u;
    }
  }
}

template <typename T, bool kPaged, typename P>
cudaError_t run_gen(const P& p, int DK, int DV, int64_t grid, cudaStream_t st) {
  const size_t smem = sizeof(float) * ((size_t)kGenRows * DK + (size_t)kGenKeys * (DK + 1) +
                                       (kPaged ? 0 : (size_t)kGenKeys * DV));
  auto go = [&](auto kernel) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(kernel, dim3((unsigned)grid), dim3(kGenThreads), smem, st, p);
  };
  if constexpr (kPaged) {
    if (DV > 512) return go(latent_attn_gen<T, 32, kPaged, P>);
    if (DV > 256) return go(latent_attn_gen<T, 16, kPaged, P>);
  }
  return go(latent_attn_gen<T, 8, kPaged, P>);   // an expanded value has at most 256 dims
}

}  // namespace

int launch_rope(const RopeParams& p, int dtype, cudaStream_t st) {
  return dtype == V4A_BF16 ? run_rope<__nv_bfloat16>(p, st) : run_rope<float>(p, st);
}

int launch_latent_insert(const LatentInsertParams& p, int dtype, cudaStream_t st) {
  const int sms = sm_count();
  int tokens = kInsertTokens;                    // fewer a block while that leaves SMs without one
  while (tokens > kInsertWarps && (int64_t)p.n_tokens < (int64_t)tokens * 2 * sms) tokens /= 2;
  const dim3 grid((unsigned)((p.n_tokens + (int64_t)tokens - 1) / tokens)), block(32 * kInsertWarps);
  auto go = [&](auto kernel) {
    return launch_pdl(kernel, grid, block, 0, st, p, tokens) == cudaSuccess ? V4A_OK : V4A_ERR_CUDA;
  };
  if (dtype == V4A_BF16)
    return p.C <= 512 ? go(latent_insert_kernel<__nv_bfloat16, 512>) : go(latent_insert_kernel<__nv_bfloat16, 1024>);
  return p.C <= 512 ? go(latent_insert_kernel<float, 512>) : go(latent_insert_kernel<float, 1024>);
}

int launch_latent_gather(const LatentGatherParams& p, cudaStream_t st) {
  // fewer rows a block while that leaves SMs without one
  const int sms = sm_count();
  int rows = kGatherRows;
  while (rows > 8 && (int64_t)p.n_rows < (int64_t)rows * 2 * sms) rows /= 2;
  const dim3 grid((unsigned)(((int64_t)p.n_rows + rows - 1) / rows));
  return launch_pdl(latent_gather_kernel, grid, dim3(kGatherThreads), 0, st, p, rows) == cudaSuccess ? V4A_OK
                                                                                                   : V4A_ERR_CUDA;
}

cudaError_t launch_latent_merge(const LatentAttnParams& p, int dtype, cudaStream_t st) {
  if (p.plan.split == kSplitNone) return cudaSuccess;
  const dim3 grid((unsigned)p.plan.split_ctas, (unsigned)((p.plan.NR + kMergeWarps - 1) / kMergeWarps),
                  (unsigned)((p.C + 255) / 256));
  return dtype == V4A_BF16 ? launch_pdl(latent_merge_kernel<__nv_bfloat16>, grid, dim3(32 * kMergeWarps), 0, st, p)
                           : launch_pdl(latent_merge_kernel<float>, grid, dim3(32 * kMergeWarps), 0, st, p);
}

int launch_latent_attn(const LatentAttnParams& p, int dtype, cudaStream_t st) {
  cudaError_t e;
  if (p.plan.tc) {
    e = launch_latent_attn_tc(p, st);
  } else {
    e = dtype == V4A_BF16 ? run_gen<__nv_bfloat16, true>(p, p.C + p.R, p.C, p.plan.ctas, st)
                          : run_gen<float, true>(p, p.C + p.R, p.C, p.plan.ctas, st);
  }
  if (e == cudaSuccess) e = launch_latent_merge(p, dtype, st);
  return e == cudaSuccess ? V4A_OK : V4A_ERR_CUDA;
}

int launch_latent_expanded(const LatentExpandedParams& p, int dtype, cudaStream_t st) {
  if (p.tc) return launch_latent_expanded_tc(p, st) == cudaSuccess ? V4A_OK : V4A_ERR_CUDA;
  int64_t grid = ((int64_t)p.n_q / kGenRows + p.n_seq) * p.H;
  if (grid > 65536) grid = 65536;
  const cudaError_t e = dtype == V4A_BF16 ? run_gen<__nv_bfloat16, false>(p, p.DN + p.DR, p.DV, grid, st)
                                          : run_gen<float, false>(p, p.DN + p.DR, p.DV, grid, st);
  return e == cudaSuccess ? V4A_OK : V4A_ERR_CUDA;
}

}  // namespace v4a
