// Device helpers of the tensor-core attention kernels (128-wide heads): paired fp32 arithmetic, the
// exponentials of a row's scores, and the q/k normalisation with RoPE.
#pragma once
#include <cuda_bf16.h>
#include <stdint.h>

#include "krea2_device.cuh"

namespace krea2 {

constexpr int AD = 128;          // head dim

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 1 / (1 + e^-x) with the approximate division (2 ulp, against 2^-9 of the bf16 output it scales): the exact one
// took 2.7 us of an output epilogue's 32 columns.
__device__ __forceinline__ float sigmoid_fast(float x) { return __fdividef(1.0f, 1.0f + __expf(-x)); }

// Paired fp32 ops of sm_100: two lanes of work per instruction.
__device__ __forceinline__ unsigned long long f2u(float lo, float hi) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void u2f(unsigned long long v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ unsigned long long ffma2(unsigned long long a, unsigned long long b, unsigned long long c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ unsigned long long fadd2(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("add.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// exp2 of (v * sl2 - m) for NE scores, packed to bf16 pairs; returns the sum of the fp32 values.
template <int NE>
__device__ __forceinline__ float exp_tile(const float* v, float sl2, float m, uint32_t* pk) {
  const unsigned long long s2 = f2u(sl2, sl2), nm2 = f2u(-m, -m);
  unsigned long long acc[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
  for (int e = 0; e < NE / 2; ++e) {
    float x0, x1;
    u2f(ffma2(f2u(v[2 * e], v[2 * e + 1]), s2, nm2), x0, x1);
    const float a = ex2(x0), c = ex2(x1);
    pk[e] = pack_bf16x2(a, c);
    acc[e & 3] = fadd2(acc[e & 3], f2u(a, c));
  }
  float t[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) u2f(acc[k], t[2 * k], t[2 * k + 1]);
  return ((t[0] + t[1]) + (t[2] + t[3])) + ((t[4] + t[5]) + (t[6] + t[7]));
}

// One warp normalises one 128-wide head (RMSNorm over head_dim with weight (1 + w), page §四.3)
// and rotates it by the position's RoPE angles (adjacent pairs); each lane holds 4 columns.
__device__ __forceinline__ uint2 norm_rope_head(const __nv_bfloat16* x, const float* w, const float* cs,
                                               const float* sn, int pos, float eps, int lane) {
  const uint2 raw = *reinterpret_cast<const uint2*>(x + lane * 4);
  float v[4] = {bf16_lo(raw.x), bf16_hi(raw.x), bf16_lo(raw.y), bf16_hi(raw.y)};
  const float ss = warp_sum(v[0] * v[0] + v[1] * v[1] + v[2] * v[2] + v[3] * v[3]);
  const float r = rsqrtf(ss / (float)AD + eps);
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] *= r * (1.f + w[lane * 4 + e]);
  const float c0 = cs[(long)pos * (AD / 2) + lane * 2], s0 = sn[(long)pos * (AD / 2) + lane * 2];
  const float c1 = cs[(long)pos * (AD / 2) + lane * 2 + 1], s1 = sn[(long)pos * (AD / 2) + lane * 2 + 1];
  uint2 o;
  o.x = pack_bf16x2(v[0] * c0 - v[1] * s0, v[1] * c0 + v[0] * s0);
  o.y = pack_bf16x2(v[2] * c1 - v[3] * s1, v[3] * c1 + v[2] * s1);
  return o;
}

}  // namespace krea2
