// Device helpers of the absorbed latent-attention kernels on tensor cores.
#pragma once

#include "latent.h"
#include "tc.cuh"

namespace v4a {

__device__ __forceinline__ float fast_exp2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
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

// Sum or largest of v[c] over the 32 lanes; lane c ends with column c's.
template <bool kMax>
__device__ __forceinline__ float reduce_scatter(const float (&v)[32]) {
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
      const float got = __shfl_xor_sync(0xffffffffu, send, o);
      a[j] = kMax ? fmaxf(keep, got) : keep + got;
    }
  }
  return a[0];
}

// Pool row of the first key of a tile, or a negative number when its page is missing or bad.
__device__ __forceinline__ int64_t tile_slot(const LatentAttnParams& p, int seq, int64_t tile, int keys) {
  return slot_of(p.cache, seq, tile * keys);
}

}  // namespace v4a
