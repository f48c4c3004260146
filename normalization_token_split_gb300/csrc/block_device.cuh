// block_device.cuh -- device parts that the block-128 casts share: the scale and
// the codes of a block of 128 values.
#pragma once

#include "nts_device.cuh"

namespace nts {

// fp32(max(a, 2^-100) / 448) by one multiply and two fmas (Brisebarre, Muller
// and Raina, as div6_rn; the quotient is normal, and equal to the IEEE one for
// every such a).  An infinite a stays infinite.
__device__ __forceinline__ float block_scale(float a) {
  a = fmaxf(a, 0x1p-100f);
  const float z = 0x1.24924ap-9f;   // fl(1 / 448)
  const float q = __fmul_rn(a, z);
  const float s = __fmaf_rn(__fmaf_rn(-q, 448.0f, a), z, q);
  return a <= 3.402823466e38f ? s : a;
}

// 16 bf16 (two 16-byte loads; p is 16-byte aligned).
__device__ __forceinline__ void load16(uint4 (&v)[2], const __nv_bfloat16* p) {
  v[0] = __ldcs(reinterpret_cast<const uint4*>(p));
  v[1] = __ldcs(reinterpret_cast<const uint4*>(p) + 1);
}

__device__ __forceinline__ void unpack16(const uint4 (&v)[2], float (&f)[16]) {
  float a[8], b[8];
  bf16x8_to_f32(v[0], a);
  bf16x8_to_f32(v[1], b);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    f[j] = a[j];
    f[8 + j] = b[j];
  }
}

__device__ __forceinline__ float absmax16(const float (&f)[16]) {
  float m = 0.f;
#pragma unroll
  for (int j = 0; j < 16; j += 2) m = fmax3(m, fabsf(f[j]), fabsf(f[j + 1]));
  return m;
}

__device__ __forceinline__ uint4 codes16(const float (&f)[16], float inv) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    w[j] = cvt_e4m3x4(f[4 * j] * inv, f[4 * j + 1] * inv, f[4 * j + 2] * inv, f[4 * j + 3] * inv);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void named_barrier(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

}  // namespace nts
