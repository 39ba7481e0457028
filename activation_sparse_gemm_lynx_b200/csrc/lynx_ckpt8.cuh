// lynx_ckpt8.cuh -- the 8-bit activation checkpoint's arithmetic, shared by the
// kernels that write one and those that read one.
//
// 32 consecutive values of a row share a power of two 2^n, so value = q * 2^n
// with q an int8 (7 significant bits) or an e4m3 number (4): exact in bf16, and
// a tensor-core product with it rounds nothing.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "lynx_internal.h"

namespace lynx {

// 2^n as fp32, -149 <= n <= 127 (subnormal below -126)
__device__ __forceinline__ float exp2_int(int n) {
  return __uint_as_float(n >= -126 ? static_cast<uint32_t>(n + 127) << 23 : 1u << (n + 149));
}

// The multiplier a block's exponent byte stands for; NaN for 255, so that every
// value of a block that held an infinity or a NaN comes back as NaN.
template <int FMT>
__device__ __forceinline__ float ckpt8_factor(uint32_t e) {
  if (e == 255u) return __uint_as_float(0x7FC00000u);
  return exp2_int(static_cast<int>(e) - (FMT == kCkpt8Int8 ? 133 : 127));
}

// 4 stored bytes -> 4 values (before the block's factor)
template <int FMT>
__device__ __forceinline__ void ckpt8_decode4(uint32_t w, float (&v)[4]) {
  if constexpr (FMT == kCkpt8Int8) {
    // the byte plus 128 in the low mantissa bits of 2^23, then minus 2^23 + 128
    const uint32_t u = w ^ 0x80808080u;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7540 | i)) - 8388736.0f;
  } else {
    uint32_t lo, hi;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
    const float2 a = __half22float2(*reinterpret_cast<__half2*>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<__half2*>(&hi));
    v[0] = a.x;
    v[1] = a.y;
    v[2] = b.x;
    v[3] = b.y;
  }
}

// The same multiplier for Ckpt8Widen: int8 takes it as a bf16 pair.
template <int FMT>
__device__ __forceinline__ uint32_t ckpt8_factor_bits(uint32_t e) {
  if constexpr (FMT == kCkpt8Int8) {
    // 2^(e - 133): exponent field e - 6, or a subnormal
    uint32_t f = e >= 7u ? (e - 6u) << 7 : 1u << e;
    if (e == 255u) f = 0x7FC0u;
    return f | (f << 16);
  } else {
    return __float_as_uint(ckpt8_factor<FMT>(e));
  }
}

// A constant that stays in a register: and_or() is then one instruction.  With both
// constants as immediates the compiler makes it two, and the integer pipe (half the
// rate of the others) is what bounds the kernels that unpack.
__device__ __forceinline__ uint32_t in_register(uint32_t v) {
  uint32_t r;
  asm volatile("mov.b32 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}

// 4 stored bytes -> 4 bf16 values times the block's factor (two packed pairs), exact.
// int8 in packed bf16 arithmetic, 5 instructions a pair: with the low 7 bits in
// the mantissa of 128 it reads 128 + low, and the sign bit turns the 128 that is
// taken off into 256.
template <int FMT>
struct Ckpt8Widen {
  uint32_t low, base, sign, minus;
  __device__ __forceinline__ Ckpt8Widen()
      : low(in_register(0x007F007Fu)), base(in_register(0x43004300u)), sign(in_register(0x00800080u)),
        minus(in_register(0xC300C300u)) {}
  __device__ __forceinline__ uint2 operator()(uint32_t w, uint32_t factor) const {
    if constexpr (FMT == kCkpt8Int8) {
      uint32_t out[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t b = __byte_perm(w, 0u, i == 0 ? 0x4140 : 0x4342);
        const uint32_t v = and_or(b, low, base), off = and_or(b, sign, minus);
        __nv_bfloat162 x = __hadd2(*reinterpret_cast<const __nv_bfloat162*>(&v),
                                   *reinterpret_cast<const __nv_bfloat162*>(&off));
        x = __hmul2(x, *reinterpret_cast<const __nv_bfloat162*>(&factor));
        out[i] = *reinterpret_cast<uint32_t*>(&x);
      }
      return make_uint2(out[0], out[1]);
    } else {
      const float f = __uint_as_float(factor);
      float v[4];
      ckpt8_decode4<FMT>(w, v);
      const __nv_bfloat162 a = __floats2bfloat162_rn(v[0] * f, v[1] * f), b = __floats2bfloat162_rn(v[2] * f, v[3] * f);
      return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    }
  }
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}

__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                   *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&d);
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// What v's first part `h` (rounded or cut off) leaves of it, exact; nothing where h is not
// finite, so that an infinity stays one in the sum of the parts
__device__ __forceinline__ float bf16_rest(float v, float h) {
  return fabsf(h) < __uint_as_float(0x7F800000u) ? v - h : 0.f;
}

}  // namespace lynx
