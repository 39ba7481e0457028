// layer_norm_kernel.cu -- layer norm of the layer's input rows, forward and
// backward (lynx_layer_norm, lynx_layer_norm_backward).
//
//   mu = mean(x), v = mean((x - mu)^2), rstd = (v + eps)^(-1/2),
//   y  = (x - mu) rstd w + b
//   with xh = (x - mu) rstd and g = dy w:
//   dx = rstd (g - mean(g) - xh mean(g xh)) + dr,  dw = sum_m dy xh,  db = sum_m dy
//
// Both are bound by memory: each tensor moves once.  A row belongs to a group of
// tx threads, which own its 16-byte pieces t, t + tx, ... and keep them in
// registers from the first sum to the result (the mean is taken off before
// anything is squared).  Rows come through a ring of cp.async copies a few rows
// deep; a thread copies what it will read itself, so the ring needs no barrier,
// and what is left between the threads of a row is the two sums.
//
// dw and db: each thread adds up its columns over the block's rows, the blocks'
// sums go to the workspace and launch_column_sums adds them in the order of the
// blocks.  2 x 8 fp32 sums a piece fit in registers up to kFusedCols columns; wider
// rows read dY and X once more, by columns (column_pass_kernel.cu).
#include <cuda_bf16.h>

#include "lynx_ckpt8.cuh"
#include "lynx_internal.h"
#include "lynx_ptx.cuh"

namespace lynx {

namespace {

constexpr int kMaxThreads = 512;
constexpr int kMaxStages = 4;
constexpr uint32_t kRingMost = 200 * 1024;
constexpr int64_t kFusedCols = 8192;
constexpr int kBackwardBlocks = 296;  // two on every SM of a B200

constexpr int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The sums of `a` and `b` over the tx threads of a row, in a fixed order.  `red` is
// this call's own [2][kMaxThreads / 32] floats: two calls in a row take different ones,
// and the barrier of the second says that all have read the first's.
__device__ __forceinline__ float2 row_sums(float a, float b, float (*red)[kMaxThreads / 32], int group, int tx) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, d);
    b += __shfl_xor_sync(0xffffffffu, b, d);
  }
  if (tx == 32) return make_float2(a, b);
  const int warp = threadIdx.x >> 5, warps = tx >> 5, first = group * warps;
  if ((threadIdx.x & 31u) == 0) {
    red[0][warp] = a;
    red[1][warp] = b;
  }
  named_bar_sync(1 + group, tx);
  float2 s = make_float2(0.f, 0.f);
  for (int w = first; w < first + warps; ++w) {
    s.x += red[0][w];
    s.y += red[1][w];
  }
  return s;
}

__device__ __forceinline__ void unpack8(const uint4& p, float (&v)[8]) {
  v[0] = bf16_lo(p.x), v[1] = bf16_hi(p.x), v[2] = bf16_lo(p.y), v[3] = bf16_hi(p.y);
  v[4] = bf16_lo(p.z), v[5] = bf16_hi(p.z), v[6] = bf16_lo(p.w), v[7] = bf16_hi(p.w);
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}

__device__ __forceinline__ uint4 ones() { return make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u); }

__device__ __forceinline__ void wait_ring(int stages) {
  if (stages == 4)
    cp_async_wait<3>();
  else if (stages == 3)
    cp_async_wait<2>();
  else if (stages == 2)
    cp_async_wait<1>();
  else
    cp_async_wait<0>();
}

template <int V>
__global__ void __launch_bounds__(kMaxThreads) layer_norm_kernel(LayerNormLaunch p, int tx, int stages) {
  extern __shared__ __align__(16) uint4 ring[];  // [stage][V][threads]
  __shared__ float red[2][2][kMaxThreads / 32];
  const int threads = static_cast<int>(blockDim.x), tid = static_cast<int>(threadIdx.x);
  const int group = tid / tx, t = tid % tx, ty = threads / tx;
  const int pieces = static_cast<int>(p.K / 8);
  const int64_t step = static_cast<int64_t>(gridDim.x) * ty;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * ty + group;
  const auto* x = static_cast<const uint4*>(p.x) + t;
  auto* y = static_cast<uint4*>(p.y) + t;
  pdl_wait();
  auto fill = [&](int64_t row, int stage) {
    if (row < p.M) {
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (t + v * tx < pieces)
          cp_async_16(smem_u32(ring + (stage * V + v) * threads + tid), x + row * pieces + v * tx, 16u);
    }
    cp_async_commit();
  };
  for (int s = 0; s < stages; ++s) fill(row0 + s * step, s);
  // weight and bias stay in registers where they fit, else they come from L1 for each row
  constexpr bool kKeep = V <= 2;
  auto weight = [&](int v) { return p.w ? __ldg(static_cast<const uint4*>(p.w) + t + v * tx) : ones(); };
  auto bias = [&](int v) { return p.b ? __ldg(static_cast<const uint4*>(p.b) + t + v * tx) : make_uint4(0, 0, 0, 0); };
  uint4 w[kKeep ? V : 1], b[kKeep ? V : 1];
  if (kKeep) {
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (t + v * tx < pieces) w[v] = weight(v), b[v] = bias(v);
  }
  const float inv_k = 1.f / static_cast<float>(p.K);
  int stage = 0;
  for (int64_t row = row0; row < p.M; row += step) {
    wait_ring(stages);
    uint4 in[V];
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      in[v] = make_uint4(0, 0, 0, 0);
      if (t + v * tx < pieces) in[v] = ring[(stage * V + v) * threads + tid];
      float f[8];
      unpack8(in[v], f);
      s += ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]));
    }
    const float mean = row_sums(s, 0.f, red[0], group, tx).x * inv_k;
    fill(row + stages * step, stage);  // its values are in registers
    if (++stage == stages) stage = 0;
    float q = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (t + v * tx < pieces) {
        float f[8];
        unpack8(in[v], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) q = fmaf(f[i] - mean, f[i] - mean, q);
      }
    }
    const float rstd = rsqrtf(fmaf(row_sums(q, 0.f, red[1], group, tx).x, inv_k, p.eps));
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (t + v * tx < pieces) {
        float f[8], ww[8], bb[8];
        unpack8(in[v], f);
        unpack8(kKeep ? w[kKeep ? v : 0] : weight(v), ww);
        unpack8(kKeep ? b[kKeep ? v : 0] : bias(v), bb);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = fmaf((f[i] - mean) * rstd, ww[i], bb[i]);
        y[row * pieces + v * tx] = pack8(f);
      }
    }
    if (t == 0 && p.mean != nullptr) {
      p.mean[row] = mean;
      p.rstd[row] = rstd;
    }
  }
}

// SUMS: the columns' sums of the block's rows go to part[block][2][K] (dw, then db).
template <int V, bool SUMS>
__global__ void __launch_bounds__(kMaxThreads) layer_norm_backward_kernel(LayerNormBackwardLaunch p, int tx, int stages) {
  constexpr bool kKeep = V <= 2;  // a row's values in registers between the sums and the results
  extern __shared__ __align__(16) uint4 ring[];  // [stage][dy, x, dr][V][threads]
  __shared__ float red[2][2][kMaxThreads / 32];
  const int threads = static_cast<int>(blockDim.x), tid = static_cast<int>(threadIdx.x);
  const int group = tid / tx, t = tid % tx, ty = threads / tx;
  const int pieces = static_cast<int>(p.K / 8);
  const int64_t step = static_cast<int64_t>(gridDim.x) * ty;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * ty + group;
  const bool add = p.dr != nullptr;
  const int streams = add ? 3 : 2;
  const auto* dy = static_cast<const uint4*>(p.dy) + t;
  const auto* x = static_cast<const uint4*>(p.x) + t;
  const auto* dr = static_cast<const uint4*>(p.dr) + t;
  auto* dx = static_cast<uint4*>(p.dx) + t;
  pdl_wait();
  auto fill = [&](int64_t row, int stage) {
    if (row < p.M) {
      uint4* at = ring + stage * streams * V * threads + tid;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (t + v * tx < pieces) {
          const int64_t from = row * pieces + v * tx;
          cp_async_16(smem_u32(at + v * threads), dy + from, 16u);
          cp_async_16(smem_u32(at + (V + v) * threads), x + from, 16u);
          if (add) cp_async_16(smem_u32(at + (2 * V + v) * threads), dr + from, 16u);
        }
      }
    }
    cp_async_commit();
  };
  for (int s = 0; s < stages; ++s) fill(row0 + s * step, s);
  uint4 w[V];
#pragma unroll
  for (int v = 0; v < V; ++v)
    w[v] = p.w && t + v * tx < pieces ? __ldg(static_cast<const uint4*>(p.w) + t + v * tx) : ones();
  float sw[SUMS ? V : 1][8] = {}, sb[SUMS ? V : 1][8] = {};
  const float inv_k = 1.f / static_cast<float>(p.K);
  float mean = 0.f, rstd = 0.f;
  if (row0 < p.M) mean = p.mean[row0], rstd = p.rstd[row0];
  int stage = 0, turn = 0;
  for (int64_t row = row0; row < p.M; row += step) {
    const int64_t next = row + step;
    float mean_next = 0.f, rstd_next = 0.f;
    if (next < p.M) mean_next = p.mean[next], rstd_next = p.rstd[next];
    wait_ring(stages);
    const uint4* at = ring + stage * streams * V * threads + tid;
    uint4 keep[kKeep ? V : 1][3];
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (t + v * tx < pieces) {
        uint4(&k)[3] = keep[kKeep ? v : 0];
        k[0] = at[v * threads];
        k[1] = at[(V + v) * threads];
        if (kKeep) k[2] = add ? at[(2 * V + v) * threads] : make_uint4(0, 0, 0, 0);
        float f[8], h[8], ww[8];
        unpack8(k[0], f);
        unpack8(k[1], h);
        unpack8(w[v], ww);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float xh = (h[i] - mean) * rstd, g = f[i] * ww[i];
          s1 += g;
          s2 = fmaf(g, xh, s2);
          if constexpr (SUMS) {
            sw[v][i] = fmaf(f[i], xh, sw[v][i]);
            sb[v][i] += f[i];
          }
        }
      }
    }
    const float2 s = row_sums(s1, s2, red[turn], group, tx);
    turn ^= 1;
    if (kKeep) fill(row + stages * step, stage);  // its values are in registers
    const float c1 = s.x * inv_k, c2 = s.y * inv_k;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (t + v * tx < pieces) {
        uint4(&k)[3] = keep[kKeep ? v : 0];
        if (!kKeep) {
          k[0] = at[v * threads];
          k[1] = at[(V + v) * threads];
          k[2] = add ? at[(2 * V + v) * threads] : make_uint4(0, 0, 0, 0);
        }
        float f[8], h[8], ww[8], r[8];
        unpack8(k[0], f);
        unpack8(k[1], h);
        unpack8(w[v], ww);
        unpack8(k[2], r);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float xh = (h[i] - mean) * rstd;
          f[i] = fmaf(rstd, fmaf(-xh, c2, fmaf(f[i], ww[i], -c1)), r[i]);
        }
        dx[row * pieces + v * tx] = pack8(f);
      }
    }
    if (!kKeep) fill(row + stages * step, stage);  // the results above have used its values
    if (++stage == stages) stage = 0;
    mean = mean_next;
    rstd = rstd_next;
  }
  if constexpr (SUMS) {
    float* out = p.part + static_cast<int64_t>(blockIdx.x) * 2 * p.K;
    const int K = static_cast<int>(p.K);
    if (ty > 1) {  // the groups' sums meet in the ring: [group][2][K]
      cp_async_wait<0>();
      __syncthreads();
      out = reinterpret_cast<float*>(ring) + group * 2 * K;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (t + v * tx < pieces) {
        float* at = out + 8 * (t + v * tx);
        *reinterpret_cast<float4*>(at) = make_float4(sw[v][0], sw[v][1], sw[v][2], sw[v][3]);
        *reinterpret_cast<float4*>(at + 4) = make_float4(sw[v][4], sw[v][5], sw[v][6], sw[v][7]);
        *reinterpret_cast<float4*>(at + K) = make_float4(sb[v][0], sb[v][1], sb[v][2], sb[v][3]);
        *reinterpret_cast<float4*>(at + K + 4) = make_float4(sb[v][4], sb[v][5], sb[v][6], sb[v][7]);
      }
    }
    if (ty > 1) {
      __syncthreads();
      const auto* sums = reinterpret_cast<const float4*>(ring);
      auto* to = reinterpret_cast<float4*>(p.part + static_cast<int64_t>(blockIdx.x) * 2 * p.K);
      for (int i = tid; i < K / 2; i += threads) {
        float4 a = sums[i];
        for (int g = 1; g < ty; ++g) {
          const float4 c = sums[g * (K / 2) + i];
          a.x += c.x, a.y += c.y, a.z += c.z, a.w += c.w;
        }
        to[i] = a;
      }
    }
  }
}

// Threads of a row, rows of a block.  Two pieces a thread (16 values) make the
// shuffles of the sums cheap beside the values; narrow rows share a block of 256.
struct RowShape {
  int v, tx, ty;
};

RowShape row_shape(int64_t K) {
  const int64_t pieces = K / 8;
  RowShape s;
  s.v = pieces <= 128 ? 1 : 2;
  while (ceil_div(pieces, s.v) > kMaxThreads) s.v *= 2;
  s.tx = static_cast<int>(ceil_div(ceil_div(pieces, s.v), 32) * 32);
  s.ty = s.tx >= 256 ? 1 : 256 / s.tx;
  return s;
}

// Stages and shared memory of a ring of `streams` rows
int ring_stages(const RowShape& s, int streams) {
  const int64_t row = static_cast<int64_t>(streams) * s.v * s.tx * s.ty * 16;
  const int64_t fit = kRingMost / row;
  return static_cast<int>(fit < kMaxStages ? fit : kMaxStages);
}

template <typename Kernel>
cudaError_t allow_ring(Kernel* kernel, std::once_flag (&once)[64], cudaError_t (&configured)[64]) {
  return once_per_device(once, configured, [kernel]() {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kRingMost));
  });
}

template <int V>
cudaError_t launch_forward(const LayerNormLaunch& p, const RowShape& s, int sms, cudaStream_t stream) {
  static std::once_flag once[64];
  static cudaError_t configured[64];
  cudaError_t e = allow_ring(layer_norm_kernel<V>, once, configured);
  if (e != cudaSuccess) return e;
  const int threads = s.tx * s.ty, stages = ring_stages(s, 1);
  const size_t smem = static_cast<size_t>(stages) * V * threads * 16;
  const int64_t want = ceil_div(p.M, s.ty), most = static_cast<int64_t>(sms) * (1024 / threads);
  return launch_after_previous(layer_norm_kernel<V>, dim3(static_cast<unsigned>(want < most ? want : most)), dim3(threads),
                               smem, stream, p, s.tx, stages);
}

template <int V, bool SUMS>
cudaError_t launch_backward(const LayerNormBackwardLaunch& p, const RowShape& s, int blocks, cudaStream_t stream) {
  static std::once_flag once[64];
  static cudaError_t configured[64];
  cudaError_t e = allow_ring(layer_norm_backward_kernel<V, SUMS>, once, configured);
  if (e != cudaSuccess) return e;
  const int threads = s.tx * s.ty, streams = p.dr != nullptr ? 3 : 2, stages = ring_stages(s, streams);
  size_t smem = static_cast<size_t>(stages) * streams * V * threads * 16;
  if (SUMS && s.ty > 1) {
    const size_t sums = static_cast<size_t>(s.ty) * 2 * static_cast<size_t>(p.K) * 4;
    if (sums > smem) smem = sums;
  }
  return launch_after_previous(layer_norm_backward_kernel<V, SUMS>, dim3(static_cast<unsigned>(blocks)), dim3(threads), smem,
                               stream, p, s.tx, stages);
}

int backward_blocks(int64_t M, const RowShape& s) {
  const int64_t want = ceil_div(M, s.ty);
  return static_cast<int>(want < kBackwardBlocks ? want : kBackwardBlocks);
}

}  // namespace

cudaError_t launch_layer_norm(const LayerNormLaunch& p, int sms, cudaStream_t stream) {
  const RowShape s = row_shape(p.K);
  switch (s.v) {
    case 1: return launch_forward<1>(p, s, sms, stream);
    case 2: return launch_forward<2>(p, s, sms, stream);
    case 4: return launch_forward<4>(p, s, sms, stream);
    default: return launch_forward<8>(p, s, sms, stream);
  }
}

size_t layer_norm_backward_workspace(int64_t M, int64_t K) {
  if (K > kFusedCols) return column_pass_workspace(M, K, 2);
  return static_cast<size_t>(backward_blocks(M, row_shape(K))) * 2 * static_cast<size_t>(K) * 4;
}

cudaError_t launch_layer_norm_backward(const LayerNormBackwardLaunch& p, cudaStream_t stream) {
  const RowShape s = row_shape(p.K);
  const int blocks = backward_blocks(p.M, s);
  if ((p.dw != nullptr || p.db != nullptr) && p.K <= kFusedCols) {
    cudaError_t e = s.v == 1 ? launch_backward<1, true>(p, s, blocks, stream) : launch_backward<2, true>(p, s, blocks, stream);
    if (e != cudaSuccess) return e;
    return launch_column_sums(p.part, blocks, p.K, p.dw, p.db, stream);
  }
  cudaError_t e;
  switch (s.v) {
    case 1: e = launch_backward<1, false>(p, s, blocks, stream); break;
    case 2: e = launch_backward<2, false>(p, s, blocks, stream); break;
    case 4: e = launch_backward<4, false>(p, s, blocks, stream); break;
    default: e = launch_backward<8, false>(p, s, blocks, stream); break;
  }
  if (e != cudaSuccess || (p.dw == nullptr && p.db == nullptr)) return e;
  ColumnPassLaunch c = {};
  c.dy = p.dy;
  c.z = p.x;
  c.mean = p.mean;
  c.rstd = p.rstd;
  c.out0 = p.dw;
  c.out1 = p.db;
  c.part = p.part;
  c.M = p.M;
  c.N = p.K;
  return launch_layer_norm_columns(c, stream);
}

}  // namespace lynx
