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

// ------------------------------------------------------------------------------- rope
// Bound: HBM for many tokens, latency for few. A thread takes `VEC` consecutive elements of
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
    if (!b) rot_cs(pos, p.rot.phi_hi[i], p.rot.phi_lo[i], p.rot.psi_hi[i], p.rot.psi_lo[i], c, s);
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
// One warp per token: the latent row in registers (16-byte vectors, lane l taking vectors
// l, l + 32, ..), its mean square by shuffles, then the rotary part. Bound: latency at decode,
// HBM for prompts (each row is read and written once).
constexpr int kInsertWarps = 4;

template <typename T>
__global__ void __launch_bounds__(32 * kInsertWarps) latent_insert_kernel(const __grid_constant__ LatentInsertParams p) {
  constexpr int kV = 16 / (int)sizeof(T), kMaxVec = 1024 / kV / 32;
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kInsertWarps + (threadIdx.x >> 5);
  pdl_wait();
  if (t >= p.n_tokens) return;
  const int b = warp_find_seq(p.cu, p.n_seq, t);
  if (b < 0) return;
  const int64_t pos = __ldg(p.start + b) + (t - __ldg(p.cu + b));
  if (pos < 0 || pos >= V4A_MAX_POS) {
    if (lane == 0) raise_err(p.err, V4A_DEV_BAD_POS);
    return;
  }
  const int64_t slot = slot_of(p.cache, b, pos);
  if (slot < 0) {
    if (lane == 0) slot_ok(slot, p.err);
    return;
  }
  T* row = reinterpret_cast<T*>(p.cache.data) + slot * (int64_t)p.cache.width;
  const T* c = reinterpret_cast<const T*>(p.c) + (int64_t)t * p.c_stride;
  const int nv = p.C / kV;
  float f[kMaxVec][kV];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < kMaxVec; ++i) {
    const int v = lane + 32 * i;
    if (v < nv) {
      load_pack<T, kV>(c + v * kV, f[i]);
#pragma unroll
      for (int k = 0; k < kV; ++k) ss = fmaf(f[i][k], f[i][k], ss);
    }
  }
  float r = 1.f;
  if (p.gamma) r = 1.0f / sqrtf(warp_sum(ss) / (float)p.C + p.eps);
#pragma unroll
  for (int i = 0; i < kMaxVec; ++i) {
    const int v = lane + 32 * i;
    if (v < nv) {
      if (p.gamma) {
#pragma unroll
        for (int k = 0; k < kV; k += 4) {
          const float4 g = __ldg(reinterpret_cast<const float4*>(p.gamma + v * kV + k));
          f[i][k] *= r * g.x;
          f[i][k + 1] *= r * g.y;
          f[i][k + 2] *= r * g.z;
          f[i][k + 3] *= r * g.w;
        }
      }
      store_pack<T, kV>(row + v * kV, f[i]);
    }
  }
  const T* k = reinterpret_cast<const T*>(p.k_pe) + (int64_t)t * p.k_stride;
  const int np = p.rot.dim / 2;
  for (int i = lane; i < np; i += 32) {
    const int a = p.rot.layout == V4A_ROPE_HALF ? i : 2 * i, d = p.rot.layout == V4A_ROPE_HALF ? np : 1;
    float cc, sn;
    rot_cs(pos, p.rot.phi_hi[i], p.rot.phi_lo[i], p.rot.psi_hi[i], p.rot.psi_lo[i], cc, sn);
    cc *= p.rot.amp;
    sn *= p.rot.amp;
    const float x0 = Elem<T>::to_f(k[a]), x1 = Elem<T>::to_f(k[a + d]);
    row[p.C + a] = Elem<T>::from_f(x0 * cc - x1 * sn);
    row[p.C + a + d] = Elem<T>::from_f(x0 * sn + x1 * cc);
  }
}

// ----------------------------------------------------------------------------- gather
// A block copies 64 rows: their pool rows are looked up first (a warp per row, in turn), then
// all threads copy 16-byte vectors, several in flight. Bound: HBM.
constexpr int kGatherRows = 64, kGatherThreads = 256;

__global__ void __launch_bounds__(kGatherThreads) latent_gather_kernel(const __grid_constant__ LatentGatherParams p) {
  __shared__ int64_t slots[kGatherRows];   // pool row, -1: zeros, -2: no row of the batch
  const int r0 = blockIdx.x * kGatherRows, nr = min(kGatherRows, p.n_rows - r0);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  for (int r = warp; r < nr; r += kGatherThreads / 32) {
    const int b = warp_find_seq(p.cu, p.n_seq, r0 + r);
    if (lane == 0) {
      int64_t s = -2;
      if (b >= 0) {
        s = slot_of(p.cache, b, __ldg(p.start + b) + (r0 + r - __ldg(p.cu + b)));
        if (!slot_ok(s, p.err)) s = -1;
      }
      slots[r] = s;
    }
  }
  __syncthreads();
  const int nv = p.row_bytes / 16;
  const uint4* pool = reinterpret_cast<const uint4*>(p.cache.data);
  uint4* out = reinterpret_cast<uint4*>(p.out) + (int64_t)r0 * nv;
#pragma unroll 6
  for (int k = threadIdx.x; k < nr * nv; k += kGatherThreads) {
    const int r = k / nv;
    const int64_t s = slots[r];
    if (s == -2) continue;
    out[k] = s < 0 ? make_uint4(0, 0, 0, 0) : __ldg(pool + s * nv + (k - r * nv));
  }
}

// -------------------------------------------------------------------------- attention
// A unit of 16 query rows against tiles of 32 keys, in fp32. Warp w holds rows 2w, 2w + 1;
// lane x computes their products with key x of the tile (the key tile's rows are padded by one
// word, so the lanes' reads fall in different banks), the softmax statistics go by shuffles,
// and lane l accumulates output dims l, l + 32, .. . Bound: shared-memory reads and fp32 FMA.
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
  extern __shared__ float sm[];
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
  if constexpr (kPaged) {
    latent_prefix(p, pre, warp_tot);
    walk.begin(p, pre, blockIdx.x, gridDim.x);
  }
  for (;;) {
    // ---- the next unit: its query rows and its keys
    int rows, t0, t1, qa = 0, ka = 0, nq = 0, nk = 0;
    int64_t keys;
    if constexpr (kPaged) {
      if (!walk.next(p, w)) break;
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
        vis[i] = r < rows ? max((int64_t)0, min(w.start + tok, p.max_pos) + 1) : 0;
        if (r < rows && lane == 0 && (w.start + tok > p.max_pos || w.start + tok < 0))
          raise_err(p.err, V4A_DEV_BAD_POS);
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
      for (int k = warp; k < kGenKeys; k += kGenThreads / 32) {
        const int64_t x = x0 + k;
        bool ok = x < keys;
        if constexpr (kPaged) {
          int64_t s = -1;
          if (ok) {
            s = slot_of(p.cache, w.seq, x);
            ok = s >= 0;
            if (!ok && lane == 0) slot_ok(s, p.err);
          }
          if (ok) load_row_f<T>(ks + k * KS, reinterpret_cast<const T*>(p.cache.data) + s * (int64_t)DK, DK, lane);
        } else if (ok) {
          const int64_t g = ka + x;
          load_row_f<T>(ks + k * KS, reinterpret_cast<const T*>(p.k) + g * p.k_ts + (int64_t)head * p.k_hs, p.DN, lane);
          load_row_f<T>(ks + k * KS + p.DN, reinterpret_cast<const T*>(p.k_pe) + g * p.pe_ts, p.DR, lane);
          load_row_f<T>(vs + k * VS, reinterpret_cast<const T*>(p.v) + g * p.v_ts + (int64_t)head * p.v_hs, DV, lane);
        }
        if (!ok) {
          for (int d = lane; d < DK; d += 32) ks[k * KS + d] = 0.f;
          if (!kPaged) for (int d = lane; d < DV; d += 32) vs[k * VS + d] = 0.f;
        }
        if (lane == 0) kvalid[k] = ok;
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
// with w_i = 2^(m_i - max). Block (g, member, rows): the share in which team g begins, if it
// is the first team to begin inside it. A warp per row.
constexpr int kMergeWarps = 8;

template <typename T>
__global__ void __launch_bounds__(32 * kMergeWarps) latent_merge_kernel(const __grid_constant__ LatentAttnParams p) {
  __shared__ int32_t pre[V4A_MAX_SEQ + 1];
  __shared__ int32_t warp_tot[kMergeWarps];
  pdl_wait();
  latent_prefix(p, pre, warp_tot);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int U = p.plan.U, NR = p.plan.NR;
  const int g = blockIdx.x / U + 1, member = blockIdx.x % U;
  const int total = pre[p.n_seq], n = latent_teams(p.plan, total);
  if (g >= n) return;
  const int x = latent_team_begin(g, total, n);
  const int b = latent_seq_at(pre, p.n_seq, x);
  const LatentSeq s = latent_seq(p, b);
  const int share = (x - pre[b]) / s.tiles, x0 = pre[b] + share * s.tiles;
  if (x == x0 || latent_team_begin(g - 1, total, n) > x0) return;
  const int last = latent_team_of(x0 + s.tiles - 1, total, n);
  const int unit_row = (share * U + member) * NR;
  const int r = blockIdx.y * kMergeWarps + warp;
  if (r >= NR || unit_row + r >= s.rows) return;
  // team g - 1's piece begins the share (slot 1), the others begin inside it (slot 0)
  auto slot = [&](int i) { return (int64_t)(((i * U + member) << 1) + (i == g - 1 ? 1 : 0)) * NR + r; };
  float m = -INFINITY;
  for (int i = g - 1 + lane; i <= last; i += 32) m = fmaxf(m, p.part_ml[slot(i) * 2]);
  m = warp_max(m);
  const float ref = m == -INFINITY ? 0.f : m;
  float l = 0.f;
  for (int i = g - 1 + lane; i <= last; i += 32)
    l += exp2f(p.part_ml[slot(i) * 2] - ref) * p.part_ml[slot(i) * 2 + 1];
  l = warp_sum(l);
  const float inv = l == 0.f ? 0.f : 1.f / l;
  T* out = reinterpret_cast<T*>(p.out) + (int64_t)(s.row0 + unit_row + r) * p.C;
  for (int d = lane * 4; d < p.C; d += 128) {
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int i = g - 1; i <= last; ++i) {
      const int64_t at = slot(i);
      const float mi = p.part_ml[at * 2];
      if (mi == -INFINITY && p.part_ml[at * 2 + 1] == 0.f) continue;    // a range without a key
      const float wi = exp2f(mi - ref);
      const float4 v = *reinterpret_cast<const float4*>(p.part_o + at * p.C + d);
      a.x = fmaf(wi, v.x, a.x);
      a.y = fmaf(wi, v.y, a.y);
      a.z = fmaf(wi, v.z, a.z);
      a.w = fmaf(wi, v.w, a.w);
    }
    float f[4] = {a.x * inv, a.y * inv, a.z * inv, a.w * inv};
    if constexpr (sizeof(T) == 4) {
      store_pack<T, 4>(out + d, f);
    } else {
      uint2 u;
      T* e = reinterpret_cast<T*>(&u);
#pragma unroll
      for (int k = 0; k < 4; ++k) e[k] = Elem<T>::from_f(f[k]);
      *reinterpret_cast<uint2*>(out + d) = u;
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
  const dim3 grid((unsigned)((p.n_tokens + (int64_t)kInsertWarps - 1) / kInsertWarps)), block(32 * kInsertWarps);
  const cudaError_t e = dtype == V4A_BF16 ? launch_pdl(latent_insert_kernel<__nv_bfloat16>, grid, block, 0, st, p)
                                          : launch_pdl(latent_insert_kernel<float>, grid, block, 0, st, p);
  return e == cudaSuccess ? V4A_OK : V4A_ERR_CUDA;
}

int launch_latent_gather(const LatentGatherParams& p, cudaStream_t st) {
  const dim3 grid((unsigned)((p.n_rows + (int64_t)kGatherRows - 1) / kGatherRows));
  return launch_pdl(latent_gather_kernel, grid, dim3(kGatherThreads), 0, st, p) == cudaSuccess ? V4A_OK : V4A_ERR_CUDA;
}

cudaError_t launch_latent_merge(const LatentAttnParams& p, int dtype, cudaStream_t st) {
  if (p.plan.teams < 2) return cudaSuccess;
  const dim3 grid((unsigned)((p.plan.teams - 1) * p.plan.U), (unsigned)((p.plan.NR + kMergeWarps - 1) / kMergeWarps));
  return dtype == V4A_BF16 ? launch_pdl(latent_merge_kernel<__nv_bfloat16>, grid, dim3(32 * kMergeWarps), 0, st, p)
                           : launch_pdl(latent_merge_kernel<float>, grid, dim3(32 * kMergeWarps), 0, st, p);
}

int launch_latent_attn(const LatentAttnParams& p, int dtype, cudaStream_t st) {
  cudaError_t e;
  if (p.plan.tc) {
    e = launch_latent_attn_tc(p, st);
  } else {
    int64_t grid = (int64_t)p.plan.teams * p.plan.U;
    if (grid == 0) {
      grid = ((int64_t)p.n_tokens * p.H + p.plan.NR - 1) / p.plan.NR + p.n_seq;
      if (grid > 65536) grid = 65536;
    }
    e = dtype == V4A_BF16 ? run_gen<__nv_bfloat16, true>(p, p.C + p.R, p.C, grid, st)
                          : run_gen<float, true>(p, p.C + p.R, p.C, grid, st);
  }
  if (e == cudaSuccess) e = launch_latent_merge(p, dtype, st);
  return e == cudaSuccess ? V4A_OK : V4A_ERR_CUDA;
}

int launch_latent_expanded(const LatentExpandedParams& p, int dtype, cudaStream_t st) {
  if (dtype == V4A_BF16 && p.DN == 128 && p.DR == 64 && p.DV == 128)
    return launch_latent_expanded_tc(p, st) == cudaSuccess ? V4A_OK : V4A_ERR_CUDA;
  int64_t grid = ((int64_t)p.n_q / kGenRows + p.n_seq) * p.H;
  if (grid > 65536) grid = 65536;
  const cudaError_t e = dtype == V4A_BF16 ? run_gen<__nv_bfloat16, false>(p, p.DN + p.DR, p.DV, grid, st)
                                          : run_gen<float, false>(p, p.DN + p.DR, p.DV, grid, st);
  return e == cudaSuccess ? V4A_OK : V4A_ERR_CUDA;
}

}  // namespace v4a
