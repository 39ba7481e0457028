// sparsify_backward_kernel.cu -- the gradient through S(X) at an 8-bit
// checkpoint (lynx_sparsify_backward).
//
// S(X) = s m x with s = L / Lk, L = sum|x|, Lk = sum m|x| of the row.  With the
// selection m fixed, dL/dx_k = s m_k g_k + D ds/dx_k, D = sum_j m_j g_j x_j, and
// ds/dx_k = sign(x_k) / Lk - m_k sign(x_k) L / Lk^2 = sign(x_k) (1 - s m_k) / Lk.
#include "lynx_ckpt8.cuh"

namespace lynx {

namespace {

constexpr int kThreads = 256;

// Bit i set: value i of the 4 is kept (two largest magnitudes, ties to the lower
// position).
__device__ __forceinline__ uint32_t keep4(const float (&v)[4]) {
  const float a0 = fabsf(v[0]), a1 = fabsf(v[1]), a2 = fabsf(v[2]), a3 = fabsf(v[3]);
  // how many of the others go before each
  const int c01 = a1 > a0, c02 = a2 > a0, c03 = a3 > a0, c12 = a2 > a1, c13 = a3 > a1, c23 = a3 > a2;
  const int n0 = c01 + c02 + c03, n1 = (1 - c01) + c12 + c13, n2 = (1 - c02) + (1 - c12) + c23;
  const int n3 = (1 - c03) + (1 - c13) + (1 - c23);
  return (n0 < 2 ? 1u : 0u) | (n1 < 2 ? 2u : 0u) | (n2 < 2 ? 4u : 0u) | (n3 < 2 ? 8u : 0u);
}

template <int FMT>
__global__ void __launch_bounds__(kThreads) row_coef_kernel(SparsifyBackwardLaunch p) {
  const int64_t m = blockIdx.x;
  const auto* q = static_cast<const uint32_t*>(p.q) + m * p.K / 4;
  const auto* e = static_cast<const uint8_t*>(p.e) + m * p.K / 32;
  const auto* g = static_cast<const uint2*>(p.g) + m * p.K / 4;
  float l = 0.f, lk = 0.f, d = 0.f;
  for (int64_t i = threadIdx.x; i < p.K / 4; i += kThreads) {
    float v[4];
    ckpt8_decode4<FMT>(q[i], v);
    const float f = ckpt8_factor<FMT>(e[i / 8]);
    const uint2 gw = g[i];
    const float gv[4] = {bf16_lo(gw.x), bf16_hi(gw.x), bf16_lo(gw.y), bf16_hi(gw.y)};
    const uint32_t keep = keep4(v);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float x = v[j] * f;
      l += fabsf(x);
      if (keep >> j & 1u) {
        lk += fabsf(x);
        d = fmaf(gv[j], x, d);
      }
    }
  }
  __shared__ float sm[3][kThreads / 32];
  for (int o = 16; o > 0; o >>= 1) {
    l += __shfl_xor_sync(0xffffffffu, l, o);
    lk += __shfl_xor_sync(0xffffffffu, lk, o);
    d += __shfl_xor_sync(0xffffffffu, d, o);
  }
  if ((threadIdx.x & 31) == 0) {
    sm[0][threadIdx.x >> 5] = l;
    sm[1][threadIdx.x >> 5] = lk;
    sm[2][threadIdx.x >> 5] = d;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    l = lk = d = 0.f;
    for (int w = 0; w < kThreads / 32; ++w) {
      l += sm[0][w];
      lk += sm[1][w];
      d += sm[2][w];
    }
    p.coef[m] = lk == 0.f ? make_float2(1.f, 0.f) : make_float2(l / lk, d / lk);
  }
}

template <int FMT>
__global__ void __launch_bounds__(kThreads) apply_kernel(SparsifyBackwardLaunch p) {
  const int64_t m = blockIdx.x;
  const auto* q = static_cast<const uint32_t*>(p.q) + m * p.K / 4;
  const auto* e = static_cast<const uint8_t*>(p.e) + m * p.K / 32;
  const auto* g = static_cast<const uint2*>(p.g) + m * p.K / 4;
  auto* dx = static_cast<uint2*>(p.dx) + m * p.K / 4;
  const auto* dt = static_cast<const __nv_bfloat16*>(p.dt) + m * p.r;
  const auto* a = static_cast<const uint2*>(p.a);
  const float2 c = p.coef[m];
  for (int64_t i = threadIdx.x; i < p.K / 4; i += kThreads) {
    float v[4];
    ckpt8_decode4<FMT>(q[i], v);
    const float f = ckpt8_factor<FMT>(e[i / 8]);
    const uint2 gw = g[i];
    const float gv[4] = {bf16_lo(gw.x), bf16_hi(gw.x), bf16_lo(gw.y), bf16_hi(gw.y)};
    const uint32_t keep = keep4(v);
    float out[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float x = v[j] * f;
      const bool k = keep >> j & 1u;
      const float sign = x > 0.f ? 1.f : x < 0.f ? -1.f : x;
      out[j] = (k ? c.x * gv[j] : 0.f) + sign * c.y * (k ? 1.f - c.x : 1.f);
    }
    if (p.dt != nullptr) {
      for (int t = 0; t < p.r; ++t) {
        const float w = __bfloat162float(dt[t]);
        const uint2 aw = a[t * (p.K / 4) + i];
        out[0] = fmaf(w, bf16_lo(aw.x), out[0]);
        out[1] = fmaf(w, bf16_hi(aw.x), out[1]);
        out[2] = fmaf(w, bf16_lo(aw.y), out[2]);
        out[3] = fmaf(w, bf16_hi(aw.y), out[3]);
      }
    }
    dx[i] = make_uint2(pack_bf16(out[0], out[1]), pack_bf16(out[2], out[3]));
  }
}

}  // namespace

cudaError_t launch_sparsify_backward(const SparsifyBackwardLaunch& p, cudaStream_t s) {
  const unsigned rows = static_cast<unsigned>(p.M);
  if (p.format == kCkpt8Int8) {
    row_coef_kernel<kCkpt8Int8><<<rows, kThreads, 0, s>>>(p);
    apply_kernel<kCkpt8Int8><<<rows, kThreads, 0, s>>>(p);
  } else {
    row_coef_kernel<kCkpt8E4M3><<<rows, kThreads, 0, s>>>(p);
    apply_kernel<kCkpt8E4M3><<<rows, kThreads, 0, s>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace lynx
