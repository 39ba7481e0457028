// ckpt8_kernel.cu -- an activation to 8 bits and back (lynx_ckpt8_store,
// lynx_ckpt8_restore).
//
// Per 32 values one exponent: store finds the block's largest magnitude on the
// bf16 bit patterns (which order like the magnitudes), scales by a power of two
// (exact) and rounds once; restore multiplies back (exact).  Both are bound by
// memory: 3.03 bytes move per value in each direction.  At 4608 x 12288 (172 MB):
// store 29 us (int8) and 30 us (e4m3), 5.8 TB/s; restore 26 us behind it, 6.7 TB/s,
// part of it from L2.
#include "lynx_ckpt8.cuh"
#include "lynx_ptx.cuh"

namespace lynx {

namespace {

constexpr int kThreads = 256;

// Two lanes share a block of 32: each takes 16 values (two 16-byte loads, one
// 16-byte store).  (4 lanes with 8 values each, whose loads are whole lines, double the
// instructions for the exponent: 38 us for 33.)
template <int FMT>
__global__ void __launch_bounds__(kThreads) ckpt8_store_kernel(const uint4* __restrict__ x, uint4* __restrict__ q,
                                                               uint8_t* __restrict__ e, int64_t n16) {
  pdl_wait();
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kThreads;
  // n16 is even (K % 64 == 0), so both lanes of a block are in or out together
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < n16; i += stride) {
    uint32_t w[8];
    *reinterpret_cast<uint4*>(w) = __ldcs(x + 2 * i);
    *reinterpret_cast<uint4*>(w + 4) = __ldcs(x + 2 * i + 1);
    uint32_t top2 = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) top2 = __vmaxu2(top2, w[j] & 0x7FFF7FFFu);
    uint32_t top = max(top2 & 0xFFFFu, top2 >> 16);
    const uint32_t pair = 3u << (threadIdx.x & 30u);
    top = max(top, __shfl_xor_sync(pair, top, 1));
    const bool bad = top >= 0x7F80u;
    const int lead = static_cast<int>(top >> 7) - 127;  // floor(log2 max|x|), -127 below the normal range
    int ex;
    if constexpr (FMT == kCkpt8Int8) {
      ex = lead;
    } else {
      ex = max(lead - ((top & 0x7Fu) > 96u ? 7 : 8), -127);  // 448 = 1.75 * 2^8
    }
    const int n = (FMT == kCkpt8Int8 ? 6 : 0) - ex;  // x * 2^n is what is rounded
    const float f = bad ? 0.f : exp2_int(min(n, 126));
    uint32_t out[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float v[4] = {bf16_lo(w[2 * j]), bf16_hi(w[2 * j]), bf16_lo(w[2 * j + 1]), bf16_hi(w[2 * j + 1])};
      if (n > 126) {  // 2^n is no fp32: the rest of it, exact on values this small
#pragma unroll
        for (int t = 0; t < 4; ++t) v[t] *= exp2_int(n - 126);
      }
      uint32_t o;
      if constexpr (FMT == kCkpt8Int8) {
        // Adding 1.5 * 2^23 rounds; the low byte is the integer
        uint32_t b[4];
#pragma unroll
        for (int t = 0; t < 4; ++t)
          b[t] = __float_as_uint(fminf(fmaxf(fmaf(v[t], f, 12582912.f), 12582912.f - 127.f), 12582912.f + 127.f));
        o = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
      } else {
        // The conversion saturates at 448, which a block below 2^127 needs no more than
#pragma unroll
        for (int t = 0; t < 4; ++t) v[t] *= f;
        if (ex == 120) {
#pragma unroll
          for (int t = 0; t < 4; ++t) v[t] = fminf(fmaxf(v[t], -240.f), 240.f);
        }
        asm("{\n\t.reg .b16 a, b;\n\t"
            "cvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n\t"
            "mov.b32 %0, {a, b};\n\t}"
            : "=r"(o)
            : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]));
      }
      out[j] = bad ? 0u : o;
    }
    q[i] = make_uint4(out[0], out[1], out[2], out[3]);
    if ((i & 1) == 0) e[i >> 1] = static_cast<uint8_t>(bad ? 255 : ex + 127);
  }
}

// A warp takes 512 values a turn, a lane 8 of the first 256 and 8 of the rest, so that
// its loads and stores are whole lines.  `units` is n / 8.
template <int FMT>
__global__ void __launch_bounds__(kThreads) ckpt8_restore_kernel(const uint2* __restrict__ q,
                                                                 const uint8_t* __restrict__ e,
                                                                 uint4* __restrict__ x, int64_t units) {
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kThreads * 2;
  for (int64_t i0 = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x - lane) * 2 + lane; i0 < units;
       i0 += stride) {
    uint2 in[2];
    uint32_t ex[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bool there = i0 + 32 * h < units;
      in[h] = there ? __ldcs(q + i0 + 32 * h) : make_uint2(0, 0);
      ex[h] = there ? e[(i0 + 32 * h) >> 2] : 0u;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float f = ckpt8_factor<FMT>(ex[h]);
      float a[4], b[4];
      ckpt8_decode4<FMT>(in[h].x, a);
      ckpt8_decode4<FMT>(in[h].y, b);
      if (i0 + 32 * h < units)
        x[i0 + 32 * h] = make_uint4(pack_bf16(a[0] * f, a[1] * f), pack_bf16(a[2] * f, a[3] * f),
                                    pack_bf16(b[0] * f, b[1] * f), pack_bf16(b[2] * f, b[3] * f));
    }
  }
}

// 16 values a thread; at most 8 blocks' worth of threads per SM loop over the rest
unsigned grid_of(int64_t n16, int sms) {
  const int64_t blocks = (n16 + kThreads - 1) / kThreads;
  const int64_t most = static_cast<int64_t>(sms) * 8 * 16;
  return static_cast<unsigned>(blocks < most ? blocks : most);
}

}  // namespace

cudaError_t launch_ckpt8_store(const void* x, void* q, void* e, int64_t n, int format, int sms, cudaStream_t s) {
  const int64_t n16 = n / 16;
  auto* xp = static_cast<const uint4*>(x);
  auto* qp = static_cast<uint4*>(q);
  auto* ep = static_cast<uint8_t*>(e);
  return launch_after_previous(format == kCkpt8Int8 ? ckpt8_store_kernel<kCkpt8Int8> : ckpt8_store_kernel<kCkpt8E4M3>,
                               dim3(grid_of(n16, sms)), dim3(kThreads), 0, s, xp, qp, ep, n16);
}

cudaError_t launch_ckpt8_restore(const void* q, const void* e, void* x, int64_t n, int format, int sms,
                                 cudaStream_t s) {
  auto* qp = static_cast<const uint2*>(q);
  auto* ep = static_cast<const uint8_t*>(e);
  auto* xp = static_cast<uint4*>(x);
  return launch_after_previous(
      format == kCkpt8Int8 ? ckpt8_restore_kernel<kCkpt8Int8> : ckpt8_restore_kernel<kCkpt8E4M3>,
      dim3(grid_of(n / 16, sms)), dim3(kThreads), 0, s, qp, ep, xp, n / 8);
}

}  // namespace lynx
