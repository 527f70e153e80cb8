// The latent cache in 4 bits: insert and gather of FP4 rows (the format is stated in include/v4a.h at
// V4A_LATENT_FP4).
//
//   z = gamma c, r = 1 / sqrt(mean c^2 + eps), k = rope(k_pe)
//   row scale s = r max|z| / 2688 (more where the rotary part or 2^-100 asks for it), u = s / r
//   block of 16: B = e4m3(max|z / u| / 6), code = e2m1(z / (u B));  h = f16(k / s)
//
// Codes and block scales come from products of z with one number each, in the order that the header
// gives (no fused multiply-add), so they are the same whatever sums the mean square. Each rounding to
// fewer bits is the format's own.
#include "kernels.h"
#include "latent.h"

namespace v4a {
namespace {

// The larger one, or NaN where either is (fmaxf would drop it).
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float warp_max_nan(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// A sum of fp32 numbers and the sum of its roundings' errors, and 1 / sqrt(sum / n + eps) of it to half
// a step and little more. (fp32 layers: r reaches the row scale, and with it the rotary part's f16
// numbers; a scale a step off gives one in 7,000 of those its neighbour, 2^-10 away.)
struct Sum2 {
  float hi = 0.f, lo = 0.f;
  __device__ __forceinline__ void add(float v) {
    const float t = __fadd_rn(hi, v), b = __fsub_rn(t, hi);
    lo += __fadd_rn(__fsub_rn(hi, __fsub_rn(t, b)), __fsub_rn(v, b));
    hi = t;
  }
  __device__ __forceinline__ void add_square(float z) {
    const float p = __fmul_rn(z, z);
    lo += __fmaf_rn(z, z, -p);
    add(p);
  }
  __device__ __forceinline__ void over_warp() {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float h = __shfl_xor_sync(0xffffffffu, hi, o);
      lo += __shfl_xor_sync(0xffffffffu, lo, o);
      add(h);
    }
  }
  __device__ __forceinline__ float inv_root(float n, float eps) const {
    Sum2 m;
    m.hi = __fdiv_rn(hi, n);
    m.lo = (__fmaf_rn(-m.hi, n, hi) + lo) / n;
    m.add(eps);
    const float r = 1.0f / sqrtf(m.hi), rr = __fmul_rn(r, r);
    const float e = __fmaf_rn(-m.hi, rr, 1.f) - m.hi * __fmaf_rn(r, r, -rr) - m.lo * rr;   // 1 - m r^2
    return e > -1.f && e < 1.f ? __fmaf_rn(0.5f * r, e, r) : r;      // (r as it is at 0, infinity, NaN)
  }
};

// ----------------------------------------------------------------------------- insert
// As the kernel for plain rows: a block looks the pool rows of up to 32 tokens up, a thread a token,
// then a warp takes one token after the other, the next one's row requested ahead. A lane holds whole
// blocks of 16 values (blocks lane, lane + 32), so that a block's maximum needs no other lane, and
// pairs lane, lane + 32 of the rotary part. Bound: latency (32 tokens 3.9 us); for prompts instructions,
// about 500 a token (14,618 tokens: 14.8 us).
constexpr int kInsertWarps = 8, kInsertTokens = 32;

template <typename T, int kBlocks>
struct Fp4Row {
  static constexpr int kV = 16 / (int)sizeof(T), kVec = 16 / kV;   // vectors of a block
  uint4 v[kBlocks][kVec];
  T x0[2], x1[2];
  __device__ __forceinline__ void load(const LatentInsertParams& p, int64_t t, int lane) {
    const T* c = reinterpret_cast<const T*>(p.c) + t * p.c_stride;
    const T* k = reinterpret_cast<const T*>(p.k_pe) + t * p.k_stride;
    const int np = p.rot.dim / 2;
    const bool half = p.rot.layout == V4A_ROPE_HALF;
#pragma unroll
    for (int i = 0; i < kBlocks; ++i)
      if (lane + 32 * i < p.C / 16)
#pragma unroll
        for (int j = 0; j < kVec; ++j) v[i][j] = *reinterpret_cast<const uint4*>(c + (lane + 32 * i) * 16 + j * kV);
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

template <typename T, int kBlocks>
__global__ void __launch_bounds__(32 * kInsertWarps, kBlocks == 1 ? 3 : 2)
    latent_insert_fp4_kernel(const __grid_constant__ LatentInsertParams p, int tokens) {
  using Row = Fp4Row<T, kBlocks>;
  __shared__ int64_t slots[kInsertTokens], at[kInsertTokens];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int np = p.rot.dim / 2, nb = p.C / 16;
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
    constexpr bool kExact = sizeof(T) == 4;
    float z[kBlocks][16], ss = 0.f, zmax = 0.f, kmax = 0.f;
    Sum2 sq;
#pragma unroll
    for (int i = 0; i < kBlocks; ++i) {
      const int b = lane + 32 * i;
      if (b >= nb) continue;
      const T* e = reinterpret_cast<const T*>(&in.v[i][0]);
#pragma unroll
      for (int q = 0; q < 16; ++q) {
        z[i][q] = Elem<T>::to_f(e[q]);
        if constexpr (kExact) sq.add_square(z[i][q]);
        else ss = fmaf(z[i][q], z[i][q], ss);
      }
      if (p.gamma) {
#pragma unroll
        for (int q = 0; q < 16; q += 4) {
          const float4 g = __ldg(reinterpret_cast<const float4*>(p.gamma + 16 * b + q));
          z[i][q] *= g.x;
          z[i][q + 1] *= g.y;
          z[i][q + 2] *= g.z;
          z[i][q + 3] *= g.w;
        }
      }
#pragma unroll
      for (int q = 0; q < 16; ++q) zmax = max_nan(zmax, fabsf(z[i][q]));
    }
    float y0[2] = {0.f, 0.f}, y1[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (lane + 32 * j >= np) continue;
      float cc, sn;
      rot_cs(pos, rate[j][0], rate[j][1], rate[j][2], rate[j][3], cc, sn);
      cc *= p.rot.amp;
      sn *= p.rot.amp;
      const float a = Elem<T>::to_f(in.x0[j]), b = Elem<T>::to_f(in.x1[j]);
      // (rounded one by one: h then is the formula's f16 number wherever cosine and sine are its own)
      y0[j] = __fsub_rn(__fmul_rn(a, cc), __fmul_rn(b, sn));
      y1[j] = __fadd_rn(__fmul_rn(a, sn), __fmul_rn(b, cc));
      kmax = max_nan(kmax, max_nan(fabsf(y0[j]), fabsf(y1[j])));
    }
    float r = 1.f;
    if (p.gamma) {
      if constexpr (kExact) {
        sq.over_warp();
        r = sq.inv_root((float)p.C, p.eps);
      } else {
        r = 1.0f / sqrtf(warp_sum(ss) / (float)p.C + p.eps);
      }
    }
    zmax = warp_max_nan(zmax);
    kmax = warp_max_nan(kmax);
    float u = __fmul_rn(zmax, 1.0f / 2688.0f), s = __fmul_rn(r, u);
    const float least = max_nan(__fmul_rn(kmax, 1.0f / 32768.0f), 0x1p-100f);
    if (!(s >= least)) {
      u = least / r;
      s = s != s ? s : least;          // (NaN stays)
    }
    const float iu = 1.0f / u, is = 1.0f / s;
    uint8_t* row = reinterpret_cast<uint8_t*>(p.cache.data) + slot * (int64_t)p.cache.width;
#pragma unroll
    for (int i = 0; i < kBlocks; ++i) {
      const int b = lane + 32 * i;
      if (b >= nb) continue;
      float m = 0.f;
#pragma unroll
      for (int q = 0; q < 16; ++q) {
        z[i][q] = __fmul_rn(z[i][q], iu);
        m = fmaxf(m, fabsf(z[i][q]));
      }
      const __nv_fp8_storage_t code = __nv_cvt_float_to_fp8(__fmul_rn(m, 1.0f / 6.0f), __NV_SATFINITE, __NV_E4M3);
      const float block = e4m3_to_f32(code), ib = block > 0.f ? 1.0f / block : 0.f;
      float a[8], c[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        a[q] = __fmul_rn(z[i][q], ib);
        c[q] = __fmul_rn(z[i][q + 8], ib);
      }
      reinterpret_cast<uint2*>(row)[b] = make_uint2(f32x8_to_e2m1(a), f32x8_to_e2m1(c));
      row[p.C / 2 + 2 * p.rot.dim + b] = code;
    }
    __half* h = reinterpret_cast<__half*>(row + p.C / 2);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int i = lane + 32 * j;
      if (i >= np) continue;
      h[half ? i : 2 * i] = __float2half_rn(__fmul_rn(y0[j], is));
      h[half ? i + np : 2 * i + 1] = __float2half_rn(__fmul_rn(y1[j], is));
    }
    if (lane == 0) p.cache.scale[slot] = s;
  }
}

// ----------------------------------------------------------------------------- gather
// A block takes `rows` rows: their pool rows are looked up first, a thread a row; then a warp takes two
// rows at a time, a lane 16 bytes of each in up to three places at once, made from 2 or 4 bytes of codes
// and a block scale (or of rotary numbers). Bound: HBM, and the instructions of the expansion (254,681
// rows: 75 us, 5.4 TB/s, three quarters of it written); for few rows, latency (3.5 us).
constexpr int kGatherRows = 64, kGatherThreads = 256, kGatherFly = 3;

// 16 bytes of a row: kV values, from codes (x) and a block scale (y) or from f16 numbers.
template <typename T>
struct Fp4Vec {
  static constexpr int kV = 16 / (int)sizeof(T);
  uint4 raw;
  __device__ __forceinline__ void load(const uint8_t* row, int C, int R, int v) {
    const int lat = C / kV;
    if (v < lat) {
      if constexpr (kV == 8) raw.x = __ldg(reinterpret_cast<const uint32_t*>(row) + v);
      else raw.x = __ldg(reinterpret_cast<const uint16_t*>(row) + v);
      raw.y = __ldg(row + C / 2 + 2 * R + v * kV / 16);
    } else if constexpr (kV == 8) {
      raw = __ldg(reinterpret_cast<const uint4*>(row + C / 2) + (v - lat));
    } else {
      const uint2 h = __ldg(reinterpret_cast<const uint2*>(row + C / 2) + (v - lat));
      raw.x = h.x;
      raw.y = h.y;
    }
  }
  // scale (B code), the inner product exact in f16, or scale h
  __device__ __forceinline__ void store(T* out, int C, int v, float scale) const {
    uint32_t h[4] = {raw.x, raw.y, raw.z, raw.w};
    if (v < C / kV) {
      const __half b = __half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)raw.y, __NV_E4M3));
      e2m1x8_to_f16(raw.x, h);
#pragma unroll
      for (int q = 0; q < kV / 2; ++q) {
        const __half2 x = __hmul2(*reinterpret_cast<const __half2*>(&h[q]), __half2(b, b));
        h[q] = *reinterpret_cast<const uint32_t*>(&x);
      }
    }
    float f[kV];
#pragma unroll
    for (int q = 0; q < kV / 2; ++q) {
      const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&h[q]));
      f[2 * q] = scale * x.x;
      f[2 * q + 1] = scale * x.y;
    }
    store_pack<T, kV>(out, f);
  }
};

template <typename T>
__global__ void __launch_bounds__(kGatherThreads)
    latent_gather_fp4_kernel(const __grid_constant__ LatentGatherParams p, int rows) {
  constexpr int kV = Fp4Vec<T>::kV, kWarps = kGatherThreads / 32;
  __shared__ int64_t slots[kGatherRows];   // pool row, -1: zeros, -2: no row of the batch
  __shared__ float scales[kGatherRows];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
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
    scales[threadIdx.x] = s >= 0 ? __ldg(p.cache.scale + s) : 0.f;
  }
  __syncthreads();
  const int nv = (p.C + p.R) / kV;
  const uint8_t* pool = reinterpret_cast<const uint8_t*>(p.cache.data);
  T* const out = reinterpret_cast<T*>(p.out) + (int64_t)r0 * (p.C + p.R);
  for (int r = warp; r < nr; r += 2 * kWarps) {
    const int64_t s[2] = {slots[r], r + kWarps < nr ? slots[r + kWarps] : -2};
    const float sc[2] = {scales[r], r + kWarps < nr ? scales[r + kWarps] : 0.f};
    for (int v0 = lane; v0 < nv; v0 += 32 * kGatherFly) {
      Fp4Vec<T> x[2][kGatherFly];
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < kGatherFly; ++i) {
          x[k][i].raw = make_uint4(0, 0, 0, 0);
          if (s[k] >= 0 && v0 + 32 * i < nv) x[k][i].load(pool + s[k] * p.cache.width, p.C, p.R, v0 + 32 * i);
        }
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < kGatherFly; ++i)
          if (s[k] != -2 && v0 + 32 * i < nv)
            x[k][i].store(out + (int64_t)(r + k * kWarps) * (p.C + p.R) + (v0 + 32 * i) * kV, p.C, v0 + 32 * i, sc[k]);
    }
  }
}

}  // namespace

int launch_latent_insert_fp4(const LatentInsertParams& p, int dtype, cudaStream_t st) {
  const int sms = sm_count();
  int tokens = kInsertTokens;                    // fewer a block while that leaves SMs without one
  while (tokens > kInsertWarps && (int64_t)p.n_tokens < (int64_t)tokens * 2 * sms) tokens /= 2;
  const dim3 grid((unsigned)((p.n_tokens + (int64_t)tokens - 1) / tokens)), block(32 * kInsertWarps);
  auto go = [&](auto kernel) {
    return launch_pdl(kernel, grid, block, 0, st, p, tokens) == cudaSuccess ? V4A_OK : V4A_ERR_CUDA;
  };
  if (dtype == V4A_BF16)
    return p.C <= 512 ? go(latent_insert_fp4_kernel<__nv_bfloat16, 1>) : go(latent_insert_fp4_kernel<__nv_bfloat16, 2>);
  return p.C <= 512 ? go(latent_insert_fp4_kernel<float, 1>) : go(latent_insert_fp4_kernel<float, 2>);
}

int launch_latent_gather_fp4(const LatentGatherParams& p, int dtype, cudaStream_t st) {
  const int sms = sm_count();
  int rows = kGatherRows;
  while (rows > 8 && (int64_t)p.n_rows < (int64_t)rows * 2 * sms) rows /= 2;
  const dim3 grid((unsigned)(((int64_t)p.n_rows + rows - 1) / rows));
  auto go = [&](auto kernel) {
    return launch_pdl(kernel, grid, dim3(kGatherThreads), 0, st, p, rows) == cudaSuccess ? V4A_OK : V4A_ERR_CUDA;
  };
  return dtype == V4A_BF16 ? go(latent_gather_fp4_kernel<__nv_bfloat16>) : go(latent_gather_fp4_kernel<float>);
}

}  // namespace v4a
