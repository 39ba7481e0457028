// lynx_f32x2.cuh -- two fp32 values in a 64-bit register pair: one instruction for
// both where a kernel would otherwise spend its issue slots on elementwise sums.
// Each half is rounded as the scalar instruction would round it.
#pragma once

#include <cstdint>

#include "lynx_ckpt8.cuh"

namespace lynx {

using f32x2 = uint64_t;

__device__ __forceinline__ f32x2 pair_f32(float lo, float hi) {
  f32x2 p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(lo), "f"(hi));
  return p;
}

__device__ __forceinline__ f32x2 both(float v) { return pair_f32(v, v); }

// a pair of bf16, widened (exact)
__device__ __forceinline__ f32x2 widen(uint32_t w) { return pair_f32(bf16_lo(w), bf16_hi(w)); }

__device__ __forceinline__ float2 halves(f32x2 p) {
  float2 v;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(p));
  return v;
}

__device__ __forceinline__ float sum_of(f32x2 p) {
  const float2 v = halves(p);
  return v.x + v.y;
}

// a pair of bf16, each rounded once
__device__ __forceinline__ uint32_t narrow(f32x2 p) {
  const float2 v = halves(p);
  return pack_bf16(v.x, v.y);
}

__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

}  // namespace lynx
