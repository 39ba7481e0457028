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
// flight.  The block's sums meet in shared memory.  Up to kClusterRows rows the ranges of a
// strip are a cluster, whose blocks add each other's sums from there: one launch, 2.5 us of
// the host's time less and no more of the device's up to 100 rows (300 x 1000: 4.8 us for 4.2, so
// that up to 320 rows it pays for eager calls and loses 0.6 us in a captured step).
// Above, the sums leave as fp32, one row of `part` for each range, and
// column_sums_kernel adds those.  Either in the order of the ranges; no atomics.
//
// gelu'(z) = sig + z sig (1 - sig) a' with sig = 1 / (1 + e^-a), a = 2 sqrt(2/pi)
// (z + 0.044715 z^3), the derivative of z sig(a).
#include <cuda_bf16.h>

#include "lynx_f32x2.cuh"
#include "lynx_internal.h"
#include "lynx_ptx.cuh"

namespace lynx {

namespace {

enum ColumnMode : int { kColSum, kColGelu, kColNorm };

constexpr int kThreads = 256;
constexpr int kUnroll = 4;  // rows of a thread in flight
constexpr int kSumThreads = 256;
constexpr int kMaxCluster = 8;
constexpr int64_t kClusterRows = 320;
constexpr int kSlots = 148 * 3;  // blocks a B200 holds; with fewer SMs the ranges are only less even

constexpr int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct ColumnPlan {
  int tx;          // threads across a strip (8 columns each), a power of two
  int strips, chunks;
  int64_t rows;    // of a chunk
  bool cluster;    // the chunks of a strip are one cluster
};

// Strips of 256 columns, or as narrow as the matrix; rows in ranges of equal length, so many
// that strips x ranges come out just below a whole number of times what the card holds (up to
// four; 4608 x 12288 in one round of 432 of 444 blocks), a range no shorter than one turn of
// its threads.
ColumnPlan column_plan(int64_t M, int64_t N, bool sums) {
  ColumnPlan c;
  c.tx = 32;
  while (c.tx > 8 && 8 * (c.tx / 2) >= N) c.tx /= 2;
  c.strips = static_cast<int>(ceil_div(N, 8 * c.tx));
  const int64_t turn = kThreads / c.tx * kUnroll, most = ceil_div(M, turn);
  int64_t chunks = 1;
  double best = 0;
  c.cluster = sums && M <= kClusterRows;
  if (c.cluster) chunks = kMaxCluster;
  for (int rounds = 1; rounds <= 4 && !c.cluster; ++rounds) {
    const int64_t slots = static_cast<int64_t>(rounds) * kSlots, n = slots / c.strips;
    const double full = static_cast<double>(n * c.strips) / static_cast<double>(slots) - 0.02 * rounds;
    if (n > 0 && full > best) best = full, chunks = n;
  }
  if (chunks > most) chunks = most;
  c.rows = ceil_div(ceil_div(M, chunks), kThreads / c.tx) * (kThreads / c.tx);
  c.chunks = static_cast<int>(ceil_div(M, c.rows));
  return c;
}

// d gelu / dz of a pair.  Beyond |z| = 16 it is 0 or 1 in fp32: cut off there, z^2 stays finite (clamp16).
__device__ __forceinline__ f32x2 gelu_tanh_slope(f32x2 z) {
  const f32x2 one = both(1.f), q = mul2(z, z);
  const float2 x = halves(mul2(z, fma2(q, both(-2.3022081981f * 0.044715f), both(-2.3022081981f))));  // -a log2 e
  float2 e, sig;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(x.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(x.y));
  const float2 d = halves(add2(pair_f32(e.x, e.y), one));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(sig.x) : "f"(d.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(sig.y) : "f"(d.y));
  const f32x2 s = pair_f32(sig.x, sig.y);
  const f32x2 u = mul2(z, fma2(q, both(0.2140644488f), both(1.5957691216f)));  // z a'
  return fma2(u, mul2(s, fma2(s, both(-1.f), one)), s);
}

// An infinity has no slope (GELU of -inf is NaN): 0 v is NaN there and adds nothing to a finite v's.
__device__ __forceinline__ uint32_t clamp16(uint32_t pair) {
  const __nv_bfloat162 v = *reinterpret_cast<__nv_bfloat162*>(&pair);
  __nv_bfloat162 c = __hmin2_nan(__hmax2_nan(v, __floats2bfloat162_rn(-16.f, -16.f)), __floats2bfloat162_rn(16.f, 16.f));
  c = __hfma2(v, __floats2bfloat162_rn(0.f, 0.f), c);
  return *reinterpret_cast<uint32_t*>(&c);
}

template <int MODE>
__global__ void __launch_bounds__(kThreads, 3) column_pass_kernel(ColumnPassLaunch p, int tx, int64_t rows) {
  constexpr int kSums = MODE == kColNorm ? 2 : 1;
  __shared__ float red[kSums][kThreads][9];  // 9: rows of 8 would share banks
  __shared__ float own[kSums * 256];
  const int t = static_cast<int>(threadIdx.x) % tx, ry = static_cast<int>(threadIdx.x) / tx, ways = kThreads / tx;
  const int64_t piece = static_cast<int64_t>(blockIdx.x) * tx + t;  // of 8 columns
  const int64_t pieces = p.N / 8;
  const int64_t row0 = static_cast<int64_t>(blockIdx.y) * rows;
  const int64_t end = row0 + rows < p.M ? row0 + rows : p.M;
  const bool on = piece < pieces;
  const auto* dy = static_cast<const uint4*>(p.dy) + piece;
  const auto* z = static_cast<const uint4*>(p.z) + piece;
  auto* dz = static_cast<uint4*>(p.dz) + piece;
  f32x2 s0[4] = {}, s1[4] = {};  // +0
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
          const uint32_t bw[4] = {b[u].x, b[u].y, b[u].z, b[u].w};
          uint32_t out[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            f32x2 f = widen(aw[i]);
            if constexpr (MODE == kColGelu) {
              f = mul2(f, gelu_tanh_slope(widen(clamp16(bw[i]))));
              out[i] = narrow(f);
            }
            if constexpr (MODE == kColNorm) {
              s1[i] = add2(s1[i], f);
              f = mul2(f, mul2(add2(widen(bw[i]), both(-mean[u])), both(rstd[u])));
            }
            s0[i] = add2(s0[i], f);
          }
          if constexpr (MODE == kColGelu) dz[r * pieces] = make_uint4(out[0], out[1], out[2], out[3]);
        }
      }
    }
  }
  if (p.out0 == nullptr && p.out1 == nullptr) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = halves(s0[i]), w = halves(s1[i]);
    red[0][threadIdx.x][2 * i] = v.x;
    red[0][threadIdx.x][2 * i + 1] = v.y;
    if constexpr (kSums == 2) {
      red[1][threadIdx.x][2 * i] = w.x;
      red[1][threadIdx.x][2 * i + 1] = w.y;
    }
  }
  __syncthreads();
  const int cols = 8 * tx;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * cols;
  float* out = p.part + static_cast<int64_t>(blockIdx.y) * kSums * p.N;
  for (int i = static_cast<int>(threadIdx.x); i < kSums * cols; i += kThreads) {
    const int which = i / cols, c = i % cols;
    float s = 0.f;
    for (int w = 0; w < ways; ++w) s += red[which][w * tx + c / 8][c % 8];
    if (p.part == nullptr)
      own[i] = s;
    else if (n0 + c < p.N)
      out[which * p.N + n0 + c] = s;
  }
  if (p.part != nullptr) return;
  __syncwarp();
  cluster_sync_all();
  const int ranks = static_cast<int>(cluster_nctarank());
  for (int i = static_cast<int>(cluster_ctarank()) * kThreads + static_cast<int>(threadIdx.x); i < kSums * cols;
       i += ranks * kThreads) {
    float v[kMaxCluster], s = 0.f;  // all ranks' on their way at once
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r)
      v[r] = r < ranks ? ld_cluster_f32(mapa_shared(smem_u32(own + i), static_cast<uint32_t>(r))) : 0.f;
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) s += v[r];
    auto* to = static_cast<__nv_bfloat16*>(i < cols ? p.out0 : p.out1);
    if (to != nullptr && n0 + i % cols < p.N) to[n0 + i % cols] = __float2bfloat16_rn(s);
  }
  __syncwarp();
  cluster_sync_all();  // the others have read this block's sums
}

// part [count][C] -> bf16, the first `split` columns to out0, the rest to out1 (either may be null).
// A block has 32 columns (a line of each row) and adds kSumThreads / 8 rows at a time, so
// that all of `part` is on its way at once: 4608 x 4096's 148 rows of 8192, 4.9 MB from L2.
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
cudaError_t launch_pass(const ColumnPassLaunch& p, const ColumnPlan& c, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(c.strips), static_cast<unsigned>(c.chunks));
  if (!c.cluster) return launch_after_previous(column_pass_kernel<MODE>, grid, dim3(kThreads), 0, s, p, c.tx, c.rows);
  return launch_clusters_after_previous(column_pass_kernel<MODE>, grid, dim3(kThreads), dim3(1, grid.y), 0, s, p, c.tx, c.rows);
}

cudaError_t launch_sums(const float* part, int count, int64_t C, int64_t split, void* out0, void* out1, cudaStream_t s) {
  return launch_after_previous(column_sums_kernel, dim3(static_cast<unsigned>(ceil_div(C, 32))), dim3(kSumThreads), 0, s, part,
                               count, C, split, static_cast<__nv_bfloat16*>(out0), static_cast<__nv_bfloat16*>(out1));
}

}  // namespace

size_t column_pass_workspace(int64_t M, int64_t N, int sums) {
  const ColumnPlan c = column_plan(M, N, true);
  return c.cluster ? 0 : static_cast<size_t>(c.chunks) * static_cast<size_t>(sums) * static_cast<size_t>(N) * 4;
}

cudaError_t launch_column_sums(const float* part, int count, int64_t K, void* out0, void* out1, cudaStream_t s) {
  return launch_sums(part, count, 2 * K, K, out0, out1, s);
}

cudaError_t launch_act_backward(const ColumnPassLaunch& p, int act, cudaStream_t s) {
  const ColumnPlan c = column_plan(p.M, p.N, p.out0 != nullptr);
  const cudaError_t e = act == kActGeluTanh ? launch_pass<kColGelu>(p, c, s) : launch_pass<kColSum>(p, c, s);
  if (e != cudaSuccess || p.out0 == nullptr || c.cluster) return e;
  return launch_sums(p.part, c.chunks, p.N, p.N, p.out0, nullptr, s);
}

cudaError_t launch_layer_norm_columns(const ColumnPassLaunch& p, cudaStream_t s) {
  const ColumnPlan c = column_plan(p.M, p.N, true);
  const cudaError_t e = launch_pass<kColNorm>(p, c, s);
  if (e != cudaSuccess || c.cluster) return e;
  return launch_sums(p.part, c.chunks, 2 * p.N, p.N, p.out0, p.out1, s);
}

}  // namespace lynx
