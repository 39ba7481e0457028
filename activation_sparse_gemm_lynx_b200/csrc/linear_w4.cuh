// linear_w4.cuh -- the layer for a few tokens on the weight in 4 bits
// (lynx_linear_w4); one source file per group size instantiates it.
//
// y[m,n] = sum_g s[g,n] sum_{k in g} x[m,k] (q[n,k] - z[g,n]).  q - z is an exact
// bf16 (at most 5 bits), so the inner sums run on the tensor cores
// (mma.m16n8k16: 16 weight rows x 8 tokens) with fp32 accumulators that start at
// zero in each group and enter the row's sum times s.
//
// The time is the reading of the nibbles.  A block has up to 6 tiles of 16
// weight rows, all of K.  It takes K in turns of 128 on 8 cp.async rings; two
// warps share a ring, fill it together and have half of the tiles each (with one
// or two tiles a warp has a ring of its own).  No
// barrier between rings until the end, where their sums meet in shared memory (a
// fixed order, no workspace).  (TMA, with its rows of 64 bytes, was issued at
// about 200 cycles a box and fed the rings at half of this rate.)
//
// One token, 12288 x 4096, group 128 with zero points: 10.2 us (26 MB, 2.6 TB/s), with
// an adapter of r = 64 11.0 us; 32 tokens, 9216 x 4096: 13.7 and 15.7 us.  The bytes take
// 4.4 us.  The time goes into the unpacking, 13,000 instructions a scheduler whose chain 4
// warps do not cover (half of the issue slots stay empty); then the start and the sums
// at the end, 1.6 us.
//
// mma wants k pairs (2t, 2t+1) and (2t+8, 2t+9) of thread t; any assignment of k
// to those places will do if both operands share it.  Thread t takes k = 8t..8t+7
// of each 32: one 32-bit word of nibbles, 16 bytes of x, two MMAs.

#pragma once

#include <cuda_bf16.h>

#include "lynx_act.cuh"
#include "lynx_ckpt8.cuh"
#include "lynx_internal.h"
#include "lynx_ptx.cuh"

namespace lynx {

namespace {

constexpr int kChunk = 128;        // k a stage
constexpr int kThreads = 512;      // of the adapter's kernel
constexpr int kWarps = kThreads / 32;
constexpr uint32_t kMaxSlots = 4;
constexpr uint32_t kFewSmem = 224 * 1024;
constexpr int kMaxCluster = 8;

// Most row tiles of a block (a warp holds half of them, 8 NT registers of sums
// each).  The count is a template parameter: with a bound known only at run time
// every tile sits behind a branch of its own and its loads and MMAs wait for one
// another.
template <int NT>
constexpr int kFewTiles = NT == 4 ? 4 : 6;

// Warps of a ring: two, or one where there are few tiles to share; and rings: 8, or
// 16 of one warp where the tokens' bytes leave room for them
template <int T, int NT>
constexpr int kHalves = T == 1 || (T == 2 && NT <= 2) ? 1 : 2;
template <int T, int NT>
constexpr int kRings = T <= 2 && NT <= 2 ? 16 : 8;
template <int T, int NT>
constexpr int kFewThreads = 32 * kHalves<T, NT> * kRings<T, NT>;

__device__ __forceinline__ void mma_m16n8k16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Both values' first 8 bits, as a pair of bf16
__device__ __forceinline__ uint32_t upper_halves(float2 v) {
  return __byte_perm(__float_as_uint(v.x), __float_as_uint(v.y), 0x7632);
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// T[m][j] = sum_k x[m,k] a[j,k]: 16 adapter rows a cluster, K over its blocks and
// their 16 warps, 8 NT tokens.  4 us for one token (r = 64, K = 4096), 8 us for 32, most of it
// latency: the main kernel starts beside it and needs T only at its end.
template <int NT>
__global__ void __launch_bounds__(kThreads) w4_lora_down_kernel(LinearW4Launch p) {
  __shared__ float part[kWarps][NT * 8][16];
  __shared__ float sum[NT * 8][16];
  pdl_wait();
  pdl_launch_dependents();  // the sums may start beside this, once all earlier work is done
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const uint32_t rank = cluster_ctarank(), ranks = cluster_nctarank();
  const int j0 = static_cast<int>(blockIdx.x / ranks) * 16;
  const int64_t steps = p.K / 32;
  const int64_t ways = static_cast<int64_t>(ranks) * kWarps;
  const auto* x = static_cast<const __nv_bfloat16*>(p.x);
  const auto* a = static_cast<const __nv_bfloat16*>(p.a) + j0 * p.K;
  float c[NT][4] = {};
  constexpr int kBatch = NT == 4 ? 2 : 4;  // steps whose loads are in flight together
  for (int64_t first = static_cast<int64_t>(rank) * kWarps + warp; first < steps; first += kBatch * ways) {
    uint4 a0[kBatch], a1[kBatch], b[kBatch][NT];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int64_t i = first + u * ways;
      const int64_t k = 32 * i + 8 * t;
      const uint4 none = make_uint4(0, 0, 0, 0);
      a0[u] = i < steps ? __ldg(reinterpret_cast<const uint4*>(a + g * p.K + k)) : none;
      a1[u] = i < steps ? __ldg(reinterpret_cast<const uint4*>(a + (g + 8) * p.K + k)) : none;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int m = 8 * n + g;
        b[u][n] = i < steps && m < p.M ? __ldg(reinterpret_cast<const uint4*>(x + m * p.K + k)) : none;
      }
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        mma_m16n8k16(c[n], a0[u].x, a1[u].x, a0[u].y, a1[u].y, b[u][n].x, b[u][n].y);
        mma_m16n8k16(c[n], a0[u].z, a1[u].z, a0[u].w, a1[u].w, b[u][n].z, b[u][n].w);
      }
    }
  }
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    part[warp][8 * n + 2 * t][g] = c[n][0];
    part[warp][8 * n + 2 * t + 1][g] = c[n][1];
    part[warp][8 * n + 2 * t][g + 8] = c[n][2];
    part[warp][8 * n + 2 * t + 1][g + 8] = c[n][3];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < NT * 8 * 16; i += kThreads) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += part[w][i / 16][i % 16];
    sum[i / 16][i % 16] = v;
  }
  __syncwarp();
  cluster_sync_all();
  for (int i = static_cast<int>(rank) * kThreads + threadIdx.x; i < p.M * 16; i += ranks * kThreads) {
    float v = 0.f;
#pragma unroll
    for (uint32_t q = 0; q < kMaxCluster; ++q)
      if (q < ranks) v += ld_cluster_f32(mapa_shared(smem_u32(&sum[i / 16][i % 16]), q));
    p.t[(i / 16) * p.r + j0 + i % 16] = v;
  }
  __syncwarp();
  cluster_sync_all();
}

// The ring of a block: a slot is weight rows | scales | zero points | x (M rows;
// the tokens past M that an MMA reads are whatever follows, and only their own
// columns of the result see them)
template <int T, int NT, int GROUP, bool ZEROS>
struct FewCfg {
  static constexpr int kGroups = kChunk / GROUP;
  static constexpr uint32_t kRows = 16 * T;
  static constexpr uint32_t kS = kRows * 64u;
  static constexpr uint32_t kZ = kS + kGroups * kRows * 2u;
  static constexpr uint32_t kX = kZ + (ZEROS ? kGroups * kRows : 0u);
  static constexpr uint32_t kPad = NT * 8u * 256u;  // behind the last slot
  static constexpr uint32_t kRed = kRings<T, NT> * NT * 8u * kRows * 4u;
  static constexpr uint32_t slot(int M) { return (kX + static_cast<uint32_t>(M) * 256u + 127u) & ~127u; }
};

template <int T, int NT, int GROUP, bool ZEROS>
__global__ void __launch_bounds__(kFewThreads<T, NT>, 1) linear_w4_kernel(LinearW4Launch p, int slots,
                                                                         uint32_t slot_bytes) {
  using C = FewCfg<T, NT, GROUP, ZEROS>;
  constexpr int kGroups = C::kGroups;
  constexpr uint32_t rows = C::kRows;
  constexpr int kRing = kRings<T, NT>;
  constexpr int TW = T / kHalves<T, NT>;             // tiles of a warp
  constexpr uint32_t kLanes = 32 * kHalves<T, NT>;   // threads of a ring
  extern __shared__ __align__(128) uint8_t sm[];
  const uint32_t warp = warp_id_sync(), lane = lane_id(), g = lane >> 2, t = lane & 3;
  const uint32_t ring = warp % kRing, half = warp / kRing, id = 32 * half + lane;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * rows;
  const int chunks = static_cast<int>((p.K + kChunk - 1) / kChunk);
  const int count = (chunks - static_cast<int>(ring) + kRing - 1) / kRing;  // of this ring
  uint8_t* const base = sm + ring * static_cast<uint32_t>(slots) * slot_bytes;

  // what this thread copies of a chunk: every kLanes-th 16 bytes
  constexpr int kWSteps = static_cast<int>((rows * 4 + kLanes - 1) / kLanes);
  constexpr int kWRows = kLanes / 4;             // rows between steps
  const auto* wq = static_cast<const uint8_t*>(p.wq);
  const auto* x = static_cast<const uint8_t*>(p.x);
  const auto* scales = static_cast<const uint8_t*>(p.scales);
  const auto* zeros = static_cast<const uint8_t*>(p.zeros);
  const uint32_t w_row = id >> 2, w_piece = id & 3;
  const uint8_t* w_src = wq + (n0 + w_row) * (p.K / 2) + 16 * w_piece + 64 * static_cast<int64_t>(ring);
  const uint32_t w_dst = w_row * 64 + ((w_piece ^ ((w_row >> 1) & 3)) << 4);
  const int64_t w_step = kWRows * (p.K / 2);
  const bool whole = n0 + rows <= p.N;
  const int w_left = static_cast<int>(p.N - n0 - w_row < 4096 ? p.N - n0 - w_row : 4096);  // rows from this one on

  auto fill = [&](int j, int slot) {
    if (j < count) {
      const uint32_t st = smem_u32(base) + static_cast<uint32_t>(slot) * slot_bytes;
      const int64_t k0 = (static_cast<int64_t>(ring) + static_cast<int64_t>(j) * kRing) * kChunk;
      const bool k_in = k0 + 32 * w_piece < p.K;
      const uint8_t* src = w_src + static_cast<int64_t>(j) * (kRing * 64);
      if (whole && k0 + kChunk <= p.K) {
        const uint8_t* at = src;
#pragma unroll
        for (int i = 0; i < kWSteps; ++i, at += w_step) cp_async_16(st + w_dst + i * kWRows * 64, at, 16u);
      } else {
#pragma unroll
        for (int i = 0; i < kWSteps; ++i) {
          const bool in = k_in && kWRows * i < w_left;
          cp_async_16(st + w_dst + i * kWRows * 64, in ? src + i * w_step : wq, in ? 16u : 0u);
        }
      }
      for (uint32_t i = id; i < static_cast<uint32_t>(p.M) * 16; i += kLanes) {
        const uint32_t m = i >> 4, piece = i & 15;
        const bool in = k0 + 8 * piece < p.K;
        cp_async_16(st + C::kX + m * 256 + ((piece ^ ((m & 1) << 2)) << 4),
                    in ? x + (m * p.K + k0) * 2 + 16 * piece : x, in ? 16u : 0u);
      }
      for (uint32_t i = id; i < kGroups * rows / 8; i += kLanes) {
        const uint32_t grp = i / (rows / 8), piece = i % (rows / 8);
        const int64_t kg = k0 / GROUP + grp, n = n0 + 8 * piece;
        const bool in = kg * GROUP < p.K && n < p.N;
        cp_async_16(st + C::kS + i * 16, in ? scales + (kg * p.N + n) * 2 : scales, in ? 16u : 0u);
        if constexpr (ZEROS) cp_async_8(st + C::kZ + i * 8, in ? zeros + kg * p.N + n : zeros, in ? 8u : 0u);
      }
    }
    cp_async_commit();
  };

  if (p.b == nullptr) pdl_wait();  // else the kernel before this one is T's, which has waited
  for (int j = 0; j < slots - 1; ++j) fill(j, j);
  if (p.b != nullptr) {  // needed at the end: bring B's rows near
    const uint32_t lines = (2 * p.r + 127) / 128;
    for (uint32_t i = threadIdx.x; i < rows * lines; i += kFewThreads<T, NT>) {
      const int64_t n = n0 + i / lines;
      if (n < p.N) prefetch_l2(static_cast<const uint8_t*>(p.b) + n * p.r * 2 + (i % lines) * 128);
    }
  }

  const uint32_t mask = in_register(0x000F000Fu), magic = in_register(0x43004300u), eight = in_register(0x43084308u);
  float acc[TW][NT][4] = {};
  const uint32_t w_at = half * TW * 1024 + g * 64 + 4 * t, w_swz = (g >> 1) & 3;
  const uint32_t r_at = 16 * TW * half + g;  // first row of this thread in the slot
  const uint32_t x_at = C::kX + g * 256, x_swz = (g & 1) << 2;
  int slot = 0, next = slots - 1;
  for (int j = 0; j < count; ++j) {
    if (slots == 4)
      cp_async_wait<2>();
    else if (slots == 3)
      cp_async_wait<1>();
    else
      cp_async_wait<0>();
    // all of the ring's threads have this chunk's bytes and are done with the one before
    if constexpr (kHalves<T, NT> == 2)
      named_bar_sync(1 + ring, kLanes);
    else
      __syncwarp();
    fill(j + slots - 1, next);
    const uint8_t* st = base + static_cast<uint32_t>(slot) * slot_bytes;
#pragma unroll
    for (int grp = 0; grp < kGroups; ++grp) {
      float c[TW][NT][4] = {};
      uint32_t z[TW][2];
      if constexpr (ZEROS) {
#pragma unroll
        for (int u = 0; u < TW; ++u) {
          const uint8_t* at = st + C::kZ + grp * rows + 16 * u + r_at;
          z[u][0] = 0x43004300u + (at[0] & 15u) * 0x10001u;
          z[u][1] = 0x43004300u + (at[8] & 15u) * 0x10001u;
        }
      }
#pragma unroll
      for (int i = grp * (GROUP / 32); i < (grp + 1) * (GROUP / 32); ++i) {
        uint4 b[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n)
          b[n] = *reinterpret_cast<const uint4*>(st + x_at + n * 2048 + (((4 * i + t) ^ x_swz) << 4));
#pragma unroll
        for (int u = 0; u < TW; ++u) {
          const uint8_t* q_at = st + w_at + u * 1024 + ((i ^ w_swz) << 4);
          const uint32_t q0 = *reinterpret_cast<const uint32_t*>(q_at);
          const uint32_t q1 = *reinterpret_cast<const uint32_t*>(q_at + 512);
          uint32_t a[2][4];  // 128 + q as bf16 (7 bits of mantissa), less 128 + z
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            a[0][h] = sub_bf16x2(and_or(q0 >> (4 * h), mask, magic), ZEROS ? z[u][0] : eight);
            a[1][h] = sub_bf16x2(and_or(q1 >> (4 * h), mask, magic), ZEROS ? z[u][1] : eight);
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma_m16n8k16(c[u][n], a[0][0], a[1][0], a[0][1], a[1][1], b[n].x, b[n].y);
            mma_m16n8k16(c[u][n], a[0][2], a[1][2], a[0][3], a[1][3], b[n].z, b[n].w);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < TW; ++u) {
        const auto* side = reinterpret_cast<const __nv_bfloat16*>(st + C::kS) + grp * rows + 16 * u + r_at;
        const float s0 = __bfloat162float(side[0]), s1 = __bfloat162float(side[8]);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          acc[u][n][0] = fmaf(s0, c[u][n][0], acc[u][n][0]);
          acc[u][n][1] = fmaf(s0, c[u][n][1], acc[u][n][1]);
          acc[u][n][2] = fmaf(s1, c[u][n][2], acc[u][n][2]);
          acc[u][n][3] = fmaf(s1, c[u][n][3], acc[u][n][3]);
        }
      }
    }
    if (++slot == slots) slot = 0;
    if (++next == slots) next = 0;
  }
  cp_async_wait<0>();
  if (p.b != nullptr) {
    // The adapter's T B^T, 16 of r a step, the steps dealt out to the rings.  T
    // stays fp32: it enters as the sum of three bf16 (8 bits each), cut off and not
    // rounded, since the upper one of a T next to fp32's largest would round to infinity.
    // T comes from the kernel before this one, which everything above ran beside.
    pdl_wait();
    const auto* b = static_cast<const uint32_t*>(p.b);
    for (int i = static_cast<int>(ring); i < p.r / 16; i += kRing) {
      float2 tv[NT][2];
#pragma unroll
      for (int c = 0; c < NT; ++c) {
        tv[c][0] = tv[c][1] = make_float2(0.f, 0.f);
        if (8 * c + static_cast<int>(g) < p.M) {
          const float2* tm = reinterpret_cast<const float2*>(p.t + (8 * c + g) * p.r + 16 * i + 2 * t);
          tv[c][0] = tm[0];
          tv[c][1] = tm[4];
        }
      }
      uint32_t a[TW][4];
#pragma unroll
      for (int u = 0; u < TW; ++u) {
        const int64_t n = n0 + 16 * u + r_at;
        const int64_t at = (n * p.r + 16 * i) / 2 + t;
        const bool in0 = n < p.N, in1 = n + 8 < p.N;
        a[u][0] = in0 ? __ldg(b + at) : 0u;
        a[u][1] = in1 ? __ldg(b + at + 4 * p.r) : 0u;
        a[u][2] = in0 ? __ldg(b + at + 4) : 0u;
        a[u][3] = in1 ? __ldg(b + at + 4 * p.r + 4) : 0u;
      }
#pragma unroll
      for (int h = 0; h < 3; ++h) {
#pragma unroll
        for (int c = 0; c < NT; ++c) {
          const uint32_t b0 = upper_halves(tv[c][0]), b1 = upper_halves(tv[c][1]);
          tv[c][0] = make_float2(bf16_rest(tv[c][0].x, bf16_lo(b0)), bf16_rest(tv[c][0].y, bf16_hi(b0)));
          tv[c][1] = make_float2(bf16_rest(tv[c][1].x, bf16_lo(b1)), bf16_rest(tv[c][1].y, bf16_hi(b1)));
#pragma unroll
          for (int u = 0; u < TW; ++u) mma_m16n8k16(acc[u][c], a[u][0], a[u][1], a[u][2], a[u][3], b0, b1);
        }
      }
    }
  }
  __syncthreads();  // the rings become [ring][token][rows] of sums
  float* red = reinterpret_cast<float*>(sm);
#pragma unroll
  for (int u = 0; u < TW; ++u) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float* at = red + (ring * NT * 8 + 8 * n + 2 * t) * rows + 16 * (TW * half + u) + g;
      at[0] = acc[u][n][0];
      at[rows] = acc[u][n][1];
      at[8] = acc[u][n][2];
      at[rows + 8] = acc[u][n][3];
    }
  }
  __syncthreads();
  const auto* bias = static_cast<const __nv_bfloat16*>(p.bias);
  auto* y = static_cast<__nv_bfloat16*>(p.y);
  for (uint32_t i = threadIdx.x; i < static_cast<uint32_t>(p.M) * rows; i += kFewThreads<T, NT>) {
    const int64_t n = n0 + i % rows;
    if (n >= p.N) continue;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kRing; ++w) v += red[w * NT * 8 * rows + i];
    if (bias != nullptr) v += __bfloat162float(bias[n]);
    if (p.act == kActGeluTanh) v = gelu_tanh(v);
    y[(i / rows) * p.N + n] = __float2bfloat16_rn(v);
  }
}

// Programmatic launch, in clusters where `cluster` is not 0
template <typename... P, typename... A>
cudaError_t launch_with(void (*kernel)(P...), unsigned blocks, int threads, unsigned cluster, size_t smem,
                        cudaStream_t s, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 0 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int T, int NT, int GROUP, bool ZEROS>
cudaError_t launch_few(const LinearW4Launch& p, int sms, cudaStream_t s) {
  using C = FewCfg<T, NT, GROUP, ZEROS>;
  constexpr uint32_t kMostSlot = C::slot(8 * NT);
  static_assert(kRings<T, NT> * 2 * kMostSlot + C::kPad <= kFewSmem && C::kRed <= kFewSmem, "a ring holds two chunks at least");
  static std::once_flag once[64];
  static cudaError_t configured[64];
  cudaError_t e = once_per_device(once, configured, []() {
    return cudaFuncSetAttribute(linear_w4_kernel<T, NT, GROUP, ZEROS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(kFewSmem));
  });
  if (e != cudaSuccess) return e;
  const uint32_t slot_bytes = C::slot(p.M);
  const uint32_t fit = (kFewSmem - C::kPad) / (kRings<T, NT> * slot_bytes);
  const int slots = static_cast<int>(fit < kMaxSlots ? fit : kMaxSlots);
  const uint32_t ring = kRings<T, NT> * slots * slot_bytes + C::kPad;
  const uint32_t smem = ring > C::kRed ? ring : C::kRed;
  const unsigned blocks = static_cast<unsigned>((p.N + C::kRows - 1) / C::kRows);
  if (p.b != nullptr) {
    const int64_t steps = (p.K / 32 + kWarps - 1) / kWarps, most = steps < kMaxCluster ? steps : kMaxCluster;
    // Where the main kernel leaves SMs over, T runs on those: a block of the main kernel
    // does not fit beside one of T's and would start late (a cluster of 8 in every case:
    // 14.3 us for 12.6 with one token, 12288 x 4096; 19.2 for 15.9 with 32, 9216 x 4096).
    const int64_t spare = (sms - static_cast<int64_t>(blocks)) / (p.r / 16);
    const unsigned ranks = static_cast<unsigned>(spare >= 1 && spare < most ? spare : most);
    e = launch_with(w4_lora_down_kernel<NT>, static_cast<unsigned>(p.r / 16) * ranks, kThreads, ranks, 0, s, p);
    if (e != cudaSuccess) return e;
  }
  return launch_with(linear_w4_kernel<T, NT, GROUP, ZEROS>, blocks, kFewThreads<T, NT>, 0, smem, s, p, slots,
                     slot_bytes);
}

template <int NT, int GROUP, bool ZEROS>
cudaError_t launch_few_tiles(const LinearW4Launch& p, int sms, cudaStream_t s) {
  // Row tiles of a block: as few as one block on every SM allows, the same in
  // every wave where N needs more than one
  const int64_t tiles = (p.N + 15) / 16, most = static_cast<int64_t>(sms) * kFewTiles<NT>;
  const int64_t blocks = (tiles + most - 1) / most * sms;
  const int64_t each = (tiles + blocks - 1) / blocks;
  if (each <= 1) return launch_few<1, NT, GROUP, ZEROS>(p, sms, s);
  if (each == 2) return launch_few<2, NT, GROUP, ZEROS>(p, sms, s);
  if constexpr (kFewTiles<NT> == 6)
    if (each > 4) return launch_few<6, NT, GROUP, ZEROS>(p, sms, s);
  return launch_few<4, NT, GROUP, ZEROS>(p, sms, s);
}

// 8 tokens are one MMA wide
template <int GROUP, bool ZEROS>
cudaError_t launch_few_tokens(const LinearW4Launch& p, int sms, cudaStream_t s) {
  return p.M <= 8 ? launch_few_tiles<1, GROUP, ZEROS>(p, sms, s)
                  : p.M <= 16 ? launch_few_tiles<2, GROUP, ZEROS>(p, sms, s)
                              : launch_few_tiles<4, GROUP, ZEROS>(p, sms, s);
}

template <int GROUP>
cudaError_t launch_linear_w4_group(const LinearW4Launch& p, int sms, cudaStream_t s) {
  return p.zeros != nullptr ? launch_few_tokens<GROUP, true>(p, sms, s) : launch_few_tokens<GROUP, false>(p, sms, s);
}

}  // namespace

}  // namespace lynx
