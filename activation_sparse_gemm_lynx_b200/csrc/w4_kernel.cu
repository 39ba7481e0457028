// w4_kernel.cu -- the frozen weight to 4 bits and back (lynx_w4_quantize,
// lynx_w4_dequantize).
#include <cuda_bf16.h>

#include "lynx_ckpt8.cuh"
#include "lynx_internal.h"
#include "lynx_ptx.cuh"

namespace lynx {

namespace {

// ---------------------------------------------------------------------------
// to 4 bits and back: tiles of 32 rows x 256 k, 8 warps, 4 rows a warp, 8 k (one
// packed word) a lane.  2.5 bytes a weight each way.  The side arrays are
// [K/group, N], so a tile's scales go through shared memory to leave (or come) as
// rows of 32 instead of single values N apart.
//
// At 12288 x 4096, group 128 with zero points (127 MB a direction): quantise 33 us,
// 3.9 TB/s, bound by its instructions (about 18 a weight; three quarters of the issue
// slots are taken); dequantise 17 us behind it, 7.4 TB/s, the words still in L2.

constexpr int kTileN = 32;
constexpr int kTileK = 256;
constexpr int kThreads = 256;

using bf162 = __nv_bfloat162;

__device__ __forceinline__ bf162 as_pair(uint32_t w) { return *reinterpret_cast<const bf162*>(&w); }
__device__ __forceinline__ uint32_t as_word(const bf162& p) { return *reinterpret_cast<const uint32_t*>(&p); }

// Extremes that a NaN stays in: the group's scale is then NaN
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Saturated to 0..15, two at a time, in the word's order
__device__ __forceinline__ uint32_t pack_nibbles(const int (&q)[8]) {
  uint32_t w;
  asm("{\n\t.reg .b32 a;\n\t"
      "cvt.pack.sat.u4.s32.b32 a, %8, %6, 0;\n\tcvt.pack.sat.u4.s32.b32 a, %4, %2, a;\n\t"
      "cvt.pack.sat.u4.s32.b32 a, %7, %5, a;\n\tcvt.pack.sat.u4.s32.b32 %0, %3, %1, a;\n\t}"
      : "=r"(w)
      : "r"(q[0]), "r"(q[1]), "r"(q[2]), "r"(q[3]), "r"(q[4]), "r"(q[5]), "r"(q[6]), "r"(q[7]));
  return w;
}

template <int GROUP, bool ZEROS>
__global__ void __launch_bounds__(kThreads) w4_quantize_kernel(const __nv_bfloat16* __restrict__ w, int64_t N,
                                                               int64_t K, uint32_t* __restrict__ wq,
                                                               __nv_bfloat16* __restrict__ scales,
                                                               uint8_t* __restrict__ zeros) {
  constexpr int kLanes = GROUP / 8;            // lanes that share a group
  constexpr int kGroups = kTileK / GROUP;      // groups of a tile row
  __shared__ __nv_bfloat16 s_sm[kGroups][kTileN];
  __shared__ uint8_t z_sm[kGroups][kTileN];
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned k_tiles = static_cast<unsigned>((K + kTileK - 1) / kTileK);
  const int64_t kt = blockIdx.x % k_tiles;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x / k_tiles) * kTileN;
  const int64_t k0 = kt * kTileK + 8 * lane;
  const bool k_in = k0 < K;
  const int left = k_in ? static_cast<int>(min(N - n0 - 4 * warp, int64_t(4))) : 0;  // rows of this lane
  const int64_t at = (n0 + 4 * warp) * K + k0;
  uint4 rows[4];
  const __nv_bfloat16* src = w + at;
#pragma unroll
  for (int i = 0; i < 4; ++i, src += K)
    rows[i] = i < left ? __ldcs(reinterpret_cast<const uint4*>(src)) : make_uint4(0, 0, 0, 0);
  // Largest and smallest of a lane's 8 values, row by row; without zero points the
  // largest magnitude alone.
  float hi[4], lo[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bf162 v[4] = {as_pair(rows[i].x), as_pair(rows[i].y), as_pair(rows[i].z), as_pair(rows[i].w)};
    if constexpr (ZEROS) {
      const uint32_t most = as_word(__hmax2_nan(__hmax2_nan(v[0], v[1]), __hmax2_nan(v[2], v[3])));
      const uint32_t least = as_word(__hmin2_nan(__hmin2_nan(v[0], v[1]), __hmin2_nan(v[2], v[3])));
      hi[i] = max_nan(max_nan(bf16_lo(most), bf16_hi(most)), 0.f);
      lo[i] = min_nan(min_nan(bf16_lo(least), bf16_hi(least)), 0.f);
    } else {
      const uint32_t most = as_word(__hmax2_nan(__hmax2_nan(__habs2(v[0]), __habs2(v[1])),
                                                __hmax2_nan(__habs2(v[2]), __habs2(v[3]))));
      hi[i] = max_nan(bf16_lo(most), bf16_hi(most));
      lo[i] = 0.f;
    }
  }
  // Over the lanes of a group, each of 4 neighbours keeping one of the 4 rows, so
  // that a lane divides once for its row, lane % 4, and not for all four.
  const bool odd = lane & 1, upper = lane & 2;
  auto exchange = [&](const float (&v)[4], auto pick) {
    const float a = pick(odd ? v[1] : v[0], __shfl_xor_sync(0xffffffffu, odd ? v[0] : v[1], 1));
    const float c = pick(odd ? v[3] : v[2], __shfl_xor_sync(0xffffffffu, odd ? v[2] : v[3], 1));
    float r = pick(upper ? c : a, __shfl_xor_sync(0xffffffffu, upper ? a : c, 2));
#pragma unroll
    for (int d = 4; d < kLanes; d *= 2) r = pick(r, __shfl_xor_sync(0xffffffffu, r, d));
    return r;
  };
  const float top = exchange(hi, [](float a, float c) { return max_nan(a, c); });
  float ratio;
  if constexpr (ZEROS) {
    const float low = exchange(lo, [](float a, float c) { return min_nan(a, c); });
    const float range = top - low;
    lo[0] = low;
    // two bf16 more than 16 binades apart: their difference is no fp32 (and where one is
    // not finite, the scale is not either)
    if (range - top == -low && top - range == low)
      ratio = range / 15.f;
    else
      ratio = __double2float_rn((static_cast<double>(top) - static_cast<double>(low)) / 15.0);
  } else {
    ratio = top / 7.f;
  }
  const __nv_bfloat16 sb = __float2bfloat16_rn(ratio);
  const float my_s = __bfloat162float(sb);
  int my_z = 8;
  if constexpr (ZEROS) my_z = my_s == 0.f ? 0 : max(0, min(15, __float2int_rn(-lo[0] / my_s)));
  // 1 / s may not be finite below; 0 too where s is not: the conversion of NaN to 0 then
  // makes every q the zero point, and the group stands for NaN throughout
  const float my_inv = my_s >= 0x1p-100f ? 1.f / my_s : 0.f;
  if (lane % kLanes < 4) {
    s_sm[lane / kLanes][4 * warp + (lane & 3)] = sb;
    if constexpr (ZEROS) z_sm[lane / kLanes][4 * warp + (lane & 3)] = static_cast<uint8_t>(my_z);
  }
  uint32_t* dst = wq + (at >> 3);
#pragma unroll
  for (int i = 0; i < 4; ++i, dst += K / 8) {
    const uint32_t v[4] = {rows[i].x, rows[i].y, rows[i].z, rows[i].w};
    const int from = (lane & ~3) | i;
    const float s = __shfl_sync(0xffffffffu, my_s, from), inv = __shfl_sync(0xffffffffu, my_inv, from);
    const int z = ZEROS ? __shfl_sync(0xffffffffu, my_z, from) : 8;
    int q[8];
    if (inv != 0.f) {
      // The quotient with one Newton correction (Markstein's division): exact
      // wherever x / s is an fp32, so at every tie of rint; any other quotient of
      // two bf16 below 16 is over 2^-12 away from one.  Adding 1.5 * 2^23 rounds.
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float x = k % 2 ? bf16_hi(v[k / 2]) : bf16_lo(v[k / 2]);
        const float first = x * inv;
        const float quotient = fmaf(fmaf(-first, s, x), inv, first);
        q[k] = __float_as_int(quotient + 12582912.f) + (z - 0x4B400000);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float x = k % 2 ? bf16_hi(v[k / 2]) : bf16_lo(v[k / 2]);
        q[k] = s == 0.f ? z : __float2int_rn(x / s) + z;
      }
    }
    if (i < left) *dst = pack_nibbles(q);
  }
  __syncthreads();
  const int64_t kg0 = kt * kGroups;
  for (int i = threadIdx.x; i < kGroups * kTileN; i += kThreads) {
    const int g = i / kTileN, row = i % kTileN;
    if (n0 + row < N && (kg0 + g) * GROUP < K) {
      scales[(kg0 + g) * N + n0 + row] = s_sm[g][row];
      if constexpr (ZEROS) zeros[(kg0 + g) * N + n0 + row] = z_sm[g][row];
    }
  }
}

template <int GROUP, bool ZEROS>
__global__ void __launch_bounds__(kThreads) w4_dequantize_kernel(const uint32_t* __restrict__ wq,
                                                                 const __nv_bfloat16* __restrict__ scales,
                                                                 const uint8_t* __restrict__ zeros, int64_t N,
                                                                 int64_t K, __nv_bfloat16* __restrict__ w) {
  constexpr int kLanes = GROUP / 8;
  constexpr int kGroups = kTileK / GROUP;
  __shared__ uint32_t s_sm[kGroups][kTileN], z_sm[kGroups][kTileN];  // s, and 128 + z, as pairs of bf16
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned k_tiles = static_cast<unsigned>((K + kTileK - 1) / kTileK);
  const int64_t kt = blockIdx.x % k_tiles;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x / k_tiles) * kTileN;
  const int64_t k0 = kt * kTileK + 8 * lane;
  const bool k_in = k0 < K;
  const int left = k_in ? static_cast<int>(min(N - n0 - 4 * warp, int64_t(4))) : 0;  // rows of this lane
  const int64_t at = (n0 + 4 * warp) * K + k0;
  uint32_t word[4];
  const uint32_t* src = wq + (at >> 3);
#pragma unroll
  for (int i = 0; i < 4; ++i, src += K / 8) word[i] = i < left ? __ldcs(src) : 0u;
  const int64_t kg0 = kt * kGroups;
  for (int i = threadIdx.x; i < kGroups * kTileN; i += kThreads) {
    const int g = i / kTileN, row = i % kTileN;
    const bool in = n0 + row < N && (kg0 + g) * GROUP < K;
    const int64_t from = (kg0 + g) * N + n0 + row;
    s_sm[g][row] = in ? 0x10001u * __bfloat16_as_ushort(scales[from]) : 0u;
    z_sm[g][row] = 0x43004300u + 0x10001u * (ZEROS ? (in ? zeros[from] & 15u : 0u) : 8u);
  }
  __syncthreads();
  // 128 + q as bf16 (7 bits of mantissa), less 128 + z, exact, times s, rounded once:
  // in pairs, 2 instructions a value (14 through fp32, 25 us at 12288 x 4096)
  const uint32_t mask = in_register(0x000F000Fu), magic = in_register(0x43004300u);
  __nv_bfloat16* dst = w + at;
#pragma unroll
  for (int i = 0; i < 4; ++i, dst += K) {
    if (i >= left) continue;
    const int row = 4 * warp + i;
    const bf162 s = as_pair(s_sm[lane / kLanes][row]);
    const uint32_t z = z_sm[lane / kLanes][row];
    uint32_t out[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      out[j] = as_word(__hmul2(as_pair(sub_bf16x2(and_or(word[i] >> (4 * j), mask, magic), z)), s));
    *reinterpret_cast<uint4*>(dst) = make_uint4(out[0], out[1], out[2], out[3]);
  }
}

unsigned weight_tiles(int64_t N, int64_t K) {
  return static_cast<unsigned>(((K + kTileK - 1) / kTileK) * ((N + kTileN - 1) / kTileN));
}

}  // namespace

cudaError_t launch_w4_quantize(const void* w, int64_t N, int64_t K, int group, void* wq, void* scales, void* zeros,
                               cudaStream_t s) {
  const unsigned grid = weight_tiles(N, K);
  auto run = [&](auto kernel) {
    return launch_after_previous(kernel, dim3(grid), dim3(kThreads), 0, s, static_cast<const __nv_bfloat16*>(w), N, K,
                                 static_cast<uint32_t*>(wq), static_cast<__nv_bfloat16*>(scales),
                                 static_cast<uint8_t*>(zeros));
  };
  if (zeros != nullptr)
    return group == 32 ? run(w4_quantize_kernel<32, true>)
                       : group == 64 ? run(w4_quantize_kernel<64, true>) : run(w4_quantize_kernel<128, true>);
  return group == 32 ? run(w4_quantize_kernel<32, false>)
                     : group == 64 ? run(w4_quantize_kernel<64, false>) : run(w4_quantize_kernel<128, false>);
}

cudaError_t launch_w4_dequantize(const void* wq, const void* scales, const void* zeros, int64_t N, int64_t K,
                                 int group, void* w, cudaStream_t s) {
  const unsigned grid = weight_tiles(N, K);
  auto run = [&](auto kernel) {
    return launch_after_previous(kernel, dim3(grid), dim3(kThreads), 0, s, static_cast<const uint32_t*>(wq),
                                 static_cast<const __nv_bfloat16*>(scales), static_cast<const uint8_t*>(zeros), N, K,
                                 static_cast<__nv_bfloat16*>(w));
  };
  if (zeros != nullptr)
    return group == 32 ? run(w4_dequantize_kernel<32, true>)
                       : group == 64 ? run(w4_dequantize_kernel<64, true>) : run(w4_dequantize_kernel<128, true>);
  return group == 32 ? run(w4_dequantize_kernel<32, false>)
                     : group == 64 ? run(w4_dequantize_kernel<64, false>) : run(w4_dequantize_kernel<128, false>);
}

cudaError_t launch_linear_w4(const LinearW4Launch& p, int sms, cudaStream_t s) {
  return p.group == 32 ? launch_linear_w4_g32(p, sms, s)
                       : p.group == 64 ? launch_linear_w4_g64(p, sms, s) : launch_linear_w4_g128(p, sms, s);
}

}  // namespace lynx
