// column_pass_kernel.cu -- sums over the rows of a gradient: the activation's
// backward pass with the bias's gradient (lynx_act_backward), and the weight's and
// bias's gradients of layer norm where its rows are too wide for its own kernel.
//
//   kColSum    db = sum_m dy
//   kColGelu   dz = dy gelu'(z), db = sum_m dz
//   kColNorm   dw = sum_m dy (x - mu) rstd, db = sum_m dy
//
// One pass, bound by memory.  A block has a strip of columns and a range of rows;
// a thread has 8 columns (16 bytes) and every ry-th row, a few rows' loads in
// flight.  The block's sums meet in shared memory and leave as fp32, one row of
// `part` for each range; column_sums_kernel adds those in their order.  No atomics.
//
// gelu'(z) = sig + z sig (1 - sig) a' with sig = 1 / (1 + e^-a), a = 2 sqrt(2/pi)
// (z + 0.044715 z^3), the derivative of z sig(a).
#include <cuda_bf16.h>

#include "lynx_ckpt8.cuh"
#include "lynx_internal.h"
#include "lynx_ptx.cuh"

namespace lynx {

namespace {

enum ColumnMode : int { kColSum, kColGelu, kColNorm };

constexpr int kThreads = 256;
constexpr int kUnroll = 4;  // rows of a thread in flight
constexpr int kSumThreads = 256;

constexpr int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct ColumnPlan {
  int tx;          // threads across a strip (8 columns each), a power of two
  int strips, chunks;
  int64_t rows;    // of a chunk
};

// Strips of 256 columns, or as narrow as the matrix; rows in ranges of equal length, as many as
// fill the card with a few blocks an SM, a range no shorter than 4 turns of its threads.
ColumnPlan column_plan(int64_t M, int64_t N) {
  ColumnPlan c;
  c.tx = 32;
  while (c.tx > 8 && 8 * (c.tx / 2) >= N) c.tx /= 2;
  c.strips = static_cast<int>(ceil_div(N, 8 * c.tx));
  const int64_t turn = kThreads / c.tx * kUnroll;
  int64_t chunks = ceil_div(148 * 8, c.strips);
  const int64_t most = ceil_div(M, turn);
  if (chunks > most) chunks = most;
  c.rows = ceil_div(ceil_div(M, chunks), kThreads / c.tx) * (kThreads / c.tx);
  c.chunks = static_cast<int>(ceil_div(M, c.rows));
  return c;
}

// d gelu / dz.  Beyond |z| = 16 it is 0 or 1 in fp32: cut off there, z^2 stays finite.
__device__ __forceinline__ float gelu_tanh_slope(float z) {
  const float q = z * z;
  const float x = z * __fmaf_rn(q, 0.044715f, 1.0f) * -2.3022081981f;  // -a log2 e
  float e, sig;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(sig) : "f"(1.0f + e));
  const float slope = __fmaf_rn(q, 0.2140644488f, 1.5957691216f);  // a'
  return __fmaf_rn(z * slope, __fmaf_rn(-sig, sig, sig), sig);
}

__device__ __forceinline__ uint32_t clamp16(uint32_t pair) {
  __nv_bfloat162 v = *reinterpret_cast<__nv_bfloat162*>(&pair);
  v = __hmin2_nan(__hmax2_nan(v, __floats2bfloat162_rn(-16.f, -16.f)), __floats2bfloat162_rn(16.f, 16.f));
  return *reinterpret_cast<uint32_t*>(&v);
}

template <int MODE>
__global__ void __launch_bounds__(kThreads) column_pass_kernel(ColumnPassLaunch p, int tx, int64_t rows) {
  constexpr int kSums = MODE == kColNorm ? 2 : 1;
  __shared__ float red[kSums][kThreads][9];  // 9: rows of 8 would share banks
  const int t = static_cast<int>(threadIdx.x) % tx, ry = static_cast<int>(threadIdx.x) / tx, ways = kThreads / tx;
  const int64_t piece = static_cast<int64_t>(blockIdx.x) * tx + t;  // of 8 columns
  const int64_t pieces = p.N / 8;
  const int64_t row0 = static_cast<int64_t>(blockIdx.y) * rows;
  const int64_t end = row0 + rows < p.M ? row0 + rows : p.M;
  const bool on = piece < pieces;
  const auto* dy = static_cast<const uint4*>(p.dy) + piece;
  const auto* z = static_cast<const uint4*>(p.z) + piece;
  auto* dz = static_cast<uint4*>(p.dz) + piece;
  float s0[8] = {}, s1[8] = {};
  pdl_wait();
  if (on) {
    for (int64_t row = row0 + ry; row < end; row += kUnroll * ways) {
      uint4 a[kUnroll], b[kUnroll];
      float mean[kUnroll], rstd[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int64_t r = row + u * ways;
        if (r < end) {
          a[u] = __ldcs(dy + r * pieces);
          if constexpr (MODE != kColSum) b[u] = __ldcs(z + r * pieces);
          if constexpr (MODE == kColNorm) mean[u] = p.mean[r], rstd[u] = p.rstd[r];
        }
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int64_t r = row + u * ways;
        if (r < end) {
          const uint32_t aw[4] = {a[u].x, a[u].y, a[u].z, a[u].w};
          float f[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) f[2 * i] = bf16_lo(aw[i]), f[2 * i + 1] = bf16_hi(aw[i]);
          if constexpr (MODE == kColGelu) {
            const uint32_t bw[4] = {clamp16(b[u].x), clamp16(b[u].y), clamp16(b[u].z), clamp16(b[u].w)};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              f[2 * i] *= gelu_tanh_slope(bf16_lo(bw[i]));
              f[2 * i + 1] *= gelu_tanh_slope(bf16_hi(bw[i]));
            }
            dz[r * pieces] = make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                                        pack_bf16(f[6], f[7]));
          }
          if constexpr (MODE == kColNorm) {
            const uint32_t bw[4] = {b[u].x, b[u].y, b[u].z, b[u].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              s1[2 * i] += f[2 * i];
              s1[2 * i + 1] += f[2 * i + 1];
              f[2 * i] *= (bf16_lo(bw[i]) - mean[u]) * rstd[u];
              f[2 * i + 1] *= (bf16_hi(bw[i]) - mean[u]) * rstd[u];
            }
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) s0[i] += f[i];
        }
      }
    }
  }
  if (p.part == nullptr) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    red[0][threadIdx.x][i] = s0[i];
    if constexpr (kSums == 2) red[1][threadIdx.x][i] = s1[i];
  }
  __syncthreads();
  float* out = p.part + static_cast<int64_t>(blockIdx.y) * kSums * p.N;
  for (int i = static_cast<int>(threadIdx.x); i < kSums * 8 * tx; i += kThreads) {
    const int which = i / (8 * tx), c = i % (8 * tx);
    const int64_t n = static_cast<int64_t>(blockIdx.x) * 8 * tx + c;
    if (n >= p.N) continue;
    float s = 0.f;
    for (int w = 0; w < ways; ++w) s += red[which][w * tx + c / 8][c % 8];
    out[which * p.N + n] = s;
  }
}

// part [count][C] -> bf16, the first `split` columns to out0, the rest to out1 (either may be null).
// A block has 32 columns (a line of each row) and adds kSumThreads / 8 rows at a time, so
// that all of `part` is on its way at once: 4608 x 4096's 296 rows of 8192, 9.7 MB from L2.
__global__ void __launch_bounds__(kSumThreads) column_sums_kernel(const float* part, int count, int64_t C, int64_t split,
                                                                  __nv_bfloat16* out0, __nv_bfloat16* out1) {
  constexpr int kWays = kSumThreads / 8;
  __shared__ float4 red[kWays][8];
  const int t = static_cast<int>(threadIdx.x) & 7, way = static_cast<int>(threadIdx.x) >> 3;
  const int64_t c = (static_cast<int64_t>(blockIdx.x) * 8 + t) * 4;  // C is a multiple of 8
  pdl_wait();
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (c < C) {
#pragma unroll 8
    for (int i = way; i < count; i += kWays) {
      const float4 v = *reinterpret_cast<const float4*>(part + static_cast<int64_t>(i) * C + c);
      s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
    }
  }
  red[way][t] = s;
  __syncthreads();
  if (threadIdx.x < 32) {  // column threadIdx.x: its sums in the order of the ways, 4 chains
    const int64_t n = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x;
    const float* at = reinterpret_cast<const float*>(red) + threadIdx.x;
    float a[4] = {};
#pragma unroll
    for (int w = 0; w < kWays; w += 4) {
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] += at[32 * (w + i)];
    }
    __nv_bfloat16* out = n < split ? out0 : out1;
    if (n < C && out != nullptr) out[n < split ? n : n - split] = __float2bfloat16_rn((a[0] + a[1]) + (a[2] + a[3]));
  }
}

template <int MODE>
cudaError_t launch_pass(const ColumnPassLaunch& p, cudaStream_t s) {
  const ColumnPlan c = column_plan(p.M, p.N);
  return launch_after_previous(column_pass_kernel<MODE>,
                               dim3(static_cast<unsigned>(c.strips), static_cast<unsigned>(c.chunks)), dim3(kThreads), 0, s, p,
                               c.tx, c.rows);
}

cudaError_t launch_sums(const float* part, int count, int64_t C, int64_t split, void* out0, void* out1, cudaStream_t s) {
  return launch_after_previous(column_sums_kernel, dim3(static_cast<unsigned>(ceil_div(C, 32))), dim3(kSumThreads), 0, s, part,
                               count, C, split, static_cast<__nv_bfloat16*>(out0), static_cast<__nv_bfloat16*>(out1));
}

}  // namespace

size_t column_pass_workspace(int64_t M, int64_t N, int sums) {
  return static_cast<size_t>(column_plan(M, N).chunks) * static_cast<size_t>(sums) * static_cast<size_t>(N) * 4;
}

cudaError_t launch_column_sums(const float* part, int count, int64_t K, void* out0, void* out1, cudaStream_t s) {
  return launch_sums(part, count, 2 * K, K, out0, out1, s);
}

cudaError_t launch_act_backward(const ColumnPassLaunch& p, int act, cudaStream_t s) {
  cudaError_t e = act == kActGeluTanh ? launch_pass<kColGelu>(p, s) : launch_pass<kColSum>(p, s);
  if (e != cudaSuccess || p.part == nullptr) return e;
  return launch_sums(p.part, column_plan(p.M, p.N).chunks, p.N, p.N, p.out0, nullptr, s);
}

cudaError_t launch_layer_norm_columns(const ColumnPassLaunch& p, cudaStream_t s) {
  cudaError_t e = launch_pass<kColNorm>(p, s);
  if (e != cudaSuccess) return e;
  return launch_sums(p.part, column_plan(p.M, p.N).chunks, 2 * p.N, p.N, p.out0, p.out1, s);
}

}  // namespace lynx
