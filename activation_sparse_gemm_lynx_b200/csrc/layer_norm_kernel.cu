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
// anything is squared).  Rows come through shared memory by cp.async, forward one
// ahead of the row at work, backward in a ring of up to kMaxStages; a thread copies
// what it will read itself, so that no barrier is needed, and what is left between
// the threads of a row is the two sums.
//
// dw and db: each thread adds up its columns over the block's rows, the blocks'
// sums go to the workspace and launch_column_sums adds them in the order of the
// blocks.  Few rows are one block, whose sums are the result.  2 x 8 fp32 sums a
// piece fit in registers up to kFusedCols columns; wider rows read dY and X once
// more, by columns (column_pass_kernel.cu).
//
// 4608 x 4096: forward 13.6 us for 75.5 MB, backward with dr, dw and db 30.1 for 151.
#include <cuda_bf16.h>

#include "lynx_f32x2.cuh"
#include "lynx_internal.h"
#include "lynx_ptx.cuh"

namespace lynx {

namespace {

constexpr int kMaxThreads = 1024;  // forward
constexpr int kMaxThreadsBackward = 512;
constexpr int kMaxWarps = kMaxThreads / 32;
constexpr int kMaxWarpsBackward = kMaxThreadsBackward / 32;
constexpr int kMaxGroups = 8;  // rows of a block
constexpr int kMaxStages = 4;
constexpr uint32_t kRingMost = 200 * 1024;
constexpr int64_t kFusedCols = 8192;
constexpr int kRowsAlone = 2;
constexpr int kBackwardBlocks = 148;  // one on every SM of a B200; any number is right

constexpr int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The sums over the threads of a row, in an order that only their number fixes.
// `mine` is this warp's entry of the row's own in shared memory, `all` the first of
// them (those past its warps stay zero).  Two calls in a row take different ones, and the
// barrier of the second says that all have read the first's.
__device__ __forceinline__ float row_sum(float a, float* mine, const float* all, int warps, int barrier) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) a += __shfl_xor_sync(0xffffffffu, a, d);
  if (warps == 1) return a;
  *mine = a;  // every lane the same
  named_bar_sync(barrier, 32 * warps);
  a = 0.f;
#pragma unroll 1  // unrolled behind conditions, every step would be issued
  for (int w = 0; w < warps; w += 4) {
    const float4 v = *reinterpret_cast<const float4*>(all + w);
    a += (v.x + v.y) + (v.z + v.w);
  }
  return a;
}

// Two sums at once: the first step leaves a lane with one of them
__device__ __forceinline__ float2 row_sums(float a, float b, float2* mine, const float2* all, int warps, int barrier) {
  const bool low = (threadIdx.x & 16u) == 0;
  float v = (low ? a : b) + __shfl_xor_sync(0xffffffffu, low ? b : a, 16);
#pragma unroll
  for (int d = 8; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  if (warps == 1) return make_float2(__shfl_sync(0xffffffffu, v, 0), __shfl_sync(0xffffffffu, v, 16));
  reinterpret_cast<float*>(mine)[low ? 0 : 1] = v;
  named_bar_sync(barrier, 32 * warps);
  f32x2 s = both(0.f);
#pragma unroll 1
  for (int w = 0; w < warps; w += 4) {
    const float4 q = *reinterpret_cast<const float4*>(all + w), r = *reinterpret_cast<const float4*>(all + w + 2);
    s = add2(s, add2(add2(pair_f32(q.x, q.y), pair_f32(q.z, q.w)), add2(pair_f32(r.x, r.y), pair_f32(r.z, r.w))));
  }
  return halves(s);
}

// sum / k, given inv = 1 / k rounded: sum inv, off by two roundings at most, and one step of iterative
// refinement, q + (sum - q k) inv, whose residual fma leaves unrounded.  A row of equal values c has
// the sum k c exactly, and c comes out: sum inv alone, one rounding off for some k, would set a row
// of 30080 0.9 standard deviations (of sqrt(eps)) apart.  (__fdiv_rn spills: 14.0 us for 13.6.)
__device__ __forceinline__ float quotient(float sum, float k, float inv) {
  const float q = sum * inv, rest = fmaf(-q, k, sum);
  return rest == rest ? fmaf(rest, inv, q) : q;  // an infinite sum leaves no residual
}

__device__ __forceinline__ void widen8(const uint4& p, f32x2 (&v)[4]) {
  v[0] = widen(p.x), v[1] = widen(p.y), v[2] = widen(p.z), v[3] = widen(p.w);
}

__device__ __forceinline__ uint4 narrow8(const f32x2 (&v)[4]) {
  return make_uint4(narrow(v[0]), narrow(v[1]), narrow(v[2]), narrow(v[3]));
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

// A warp owns 32 V neighbouring pieces of a row, a lane every 32nd of them, so that
// its addresses are one register and constants.  FULL: there is no piece past the row's
// end (K == 8 V tx); else each is behind a branch, about 60 of them a row and warp.
template <int V, bool FULL>
__global__ void __launch_bounds__(kMaxThreads) layer_norm_kernel(LayerNormLaunch p, int tx) {
  extern __shared__ __align__(16) uint4 ring[];  // [V threads]
  __shared__ __align__(16) float red[2][kMaxGroups][kMaxWarps];
  const int threads = static_cast<int>(blockDim.x), tid = static_cast<int>(threadIdx.x);
  const int group = tid / tx, t = tid - group * tx, ty = threads / tx, warps = tx / 32;
  const int pieces = static_cast<int>(p.K / 8), first = (t >> 5) * (32 * V) + (t & 31);
  auto on = [&](int v) { return FULL || first + 32 * v < pieces; };
  const int M = static_cast<int>(p.M), step = static_cast<int>(gridDim.x) * ty;
  int row = static_cast<int>(blockIdx.x) * ty + group;
  for (int i = tid; i < 2 * kMaxGroups * kMaxWarps; i += threads) (&red[0][0][0])[i] = 0.f;
  __syncthreads();
  const uint4* const slot = ring + (tid >> 5) * (32 * V) + (tid & 31);
  const uint4* w = static_cast<const uint4*>(p.w) + first;
  const uint4* b = static_cast<const uint4*>(p.b) + first;
  const float cols = static_cast<float>(p.K), inv_k = 1.f / cols;
  pdl_wait();
  auto fetch = [&](int next) {
    if (next < M) {
      const uint4* x = static_cast<const uint4*>(p.x) + static_cast<int64_t>(next) * pieces + first;
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (on(v)) cp_async_16(smem_u32(slot) + 512 * v, x + 32 * v, 16u);
    }
    cp_async_commit();
  };
  fetch(row);
  for (; row < M; row += step) {
    cp_async_wait<0>();
    f32x2 d[V][4];
    f32x2 s2 = both(0.f);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (on(v)) {
        widen8(slot[32 * v], d[v]);
        s2 = add2(s2, add2(add2(d[v][0], d[v][1]), add2(d[v][2], d[v][3])));
      }
    }
    const float mean = quotient(row_sum(sum_of(s2), &red[0][group][t >> 5], red[0][group], warps, 1 + group), cols, inv_k);
    fetch(row + step);  // this row's values are in registers
    const f32x2 less = both(-mean);
    f32x2 q2 = both(0.f);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (on(v)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          d[v][i] = add2(d[v][i], less);
          q2 = fma2(d[v][i], d[v][i], q2);
        }
      }
    }
    const float rstd = rsqrtf(fmaf(row_sum(sum_of(q2), &red[1][group][t >> 5], red[1][group], warps, 1 + group), inv_k, p.eps));
    const f32x2 scale = both(rstd);
    uint4* y = static_cast<uint4*>(p.y) + static_cast<int64_t>(row) * pieces + first;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (on(v)) {
        // weight and bias from L1 for each row: in registers they would halve the rows an SM holds
        f32x2 ww[4], bb[4];
        widen8(p.w ? __ldg(w + 32 * v) : ones(), ww);
        widen8(p.b ? __ldg(b + 32 * v) : make_uint4(0, 0, 0, 0), bb);
#pragma unroll
        for (int i = 0; i < 4; ++i) d[v][i] = fma2(mul2(d[v][i], scale), ww[i], bb[i]);
        y[32 * v] = narrow8(d[v]);
      }
    }
    if (t == 0 && p.mean != nullptr) {
      p.mean[row] = mean;
      p.rstd[row] = rstd;
    }
  }
}

// SUMS: the columns' sums of the block's rows go to part[block][2][K] (dw, then db).
template <int V, bool SUMS, bool FULL>
__global__ void __launch_bounds__(kMaxThreadsBackward, 1)
layer_norm_backward_kernel(LayerNormBackwardLaunch p, int tx, int stages) {
  constexpr bool kKeep = V <= 2;  // the row's values in registers between the sums and the results
  // and dr's too, where the columns' sums leave room: with them it stays in the ring until it is
  // used (4608 x 4096: 30.1 us for 32.6, 4608 x 8192 55 for 61)
  constexpr bool kKeepAll = kKeep && !SUMS;
  extern __shared__ __align__(16) uint4 ring[];  // [stage][dy, x, dr][V threads]
  __shared__ __align__(16) float2 red[2][kMaxGroups][kMaxWarpsBackward];
  const int threads = static_cast<int>(blockDim.x), tid = static_cast<int>(threadIdx.x);
  const int group = tid / tx, t = tid - group * tx, ty = threads / tx, warps = tx / 32;
  const int pieces = static_cast<int>(p.K / 8), first = (t >> 5) * (32 * V) + (t & 31);
  auto on = [&](int v) { return FULL || first + 32 * v < pieces; };
  const int M = static_cast<int>(p.M), step = static_cast<int>(gridDim.x) * ty;
  int row = static_cast<int>(blockIdx.x) * ty + group;
  for (int i = tid; i < 2 * kMaxGroups * kMaxWarpsBackward; i += threads) (&red[0][0][0])[i] = make_float2(0.f, 0.f);
  __syncthreads();
  const bool add = p.dr != nullptr;
  const int stream = V * threads, stage_size = (add ? 3 : 2) * stream;  // in pieces
  int ahead = row;  // what is copied next
  const uint4* const slot = ring + (tid >> 5) * (32 * V) + (tid & 31);
  pdl_wait();
  auto fill = [&](int stage) {
    if (ahead < M) {
      const uint32_t at = smem_u32(slot + stage * stage_size);
      const int64_t next = static_cast<int64_t>(ahead) * pieces + first;
      const uint4* dy = static_cast<const uint4*>(p.dy) + next;
      const uint4* x = static_cast<const uint4*>(p.x) + next;
      const uint4* dr = static_cast<const uint4*>(p.dr) + next;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (on(v)) {
          cp_async_16(at + 512 * v, dy + 32 * v, 16u);
          cp_async_16(at + stream * 16 + 512 * v, x + 32 * v, 16u);
          if (add) cp_async_16(at + stream * 32 + 512 * v, dr + 32 * v, 16u);
        }
      }
    }
    ahead += step;
    cp_async_commit();
  };
  for (int s = 0; s < stages; ++s) fill(s);
  f32x2 w[V][4];
#pragma unroll
  for (int v = 0; v < V; ++v) widen8(p.w && on(v) ? __ldg(static_cast<const uint4*>(p.w) + first + 32 * v) : ones(), w[v]);
  f32x2 sw[SUMS ? V : 1][4] = {}, sb[SUMS ? V : 1][4] = {};  // +0
  const float inv_k = 1.f / static_cast<float>(p.K);
  float mean = 0.f, rstd = 0.f;
  if (row < M) mean = p.mean[row], rstd = p.rstd[row];
  int stage = 0, turn = 0;
  for (; row < M; row += step) {
    wait_ring(stages);
    const uint4* at = slot + stage * stage_size;
    const f32x2 less = both(-mean), scale = both(rstd);
    f32x2 g[kKeep ? V : 1][4], xh[kKeep ? V : 1][4];
    uint4 r[kKeepAll ? V : 1];
    f32x2 s1 = both(0.f), s2 = both(0.f);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (on(v)) {
        f32x2 f[4];
        auto& gv = g[kKeep ? v : 0];
        auto& xv = xh[kKeep ? v : 0];
        widen8(at[32 * v], f);
        widen8(at[stream + 32 * v], xv);
        if (kKeepAll) r[kKeepAll ? v : 0] = add ? at[2 * stream + 32 * v] : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          xv[i] = mul2(add2(xv[i], less), scale);
          gv[i] = mul2(f[i], w[v][i]);
          s1 = add2(s1, gv[i]);
          s2 = fma2(gv[i], xv[i], s2);
          if constexpr (SUMS) {
            sw[v][i] = fma2(f[i], xv[i], sw[v][i]);
            sb[v][i] = add2(f[i], sb[v][i]);
          }
        }
      }
    }
    if (row + step < M) mean = p.mean[row + step], rstd = p.rstd[row + step];
    const float2 s = row_sums(sum_of(s1), sum_of(s2), &red[turn][group][t >> 5], red[turn][group], warps, 1 + group);
    turn ^= 1;
    if (kKeepAll) fill(stage);  // its values are in registers
    const f32x2 c1 = both(-s.x * inv_k), c2 = both(-s.y * inv_k);
    uint4* to = static_cast<uint4*>(p.dx) + static_cast<int64_t>(row) * pieces + first;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (on(v)) {
        auto& gv = g[kKeep ? v : 0];
        auto& xv = xh[kKeep ? v : 0];
        auto& rv = r[kKeepAll ? v : 0];
        if (!kKeepAll) rv = add ? at[2 * stream + 32 * v] : make_uint4(0, 0, 0, 0);
        if (!kKeep) {
          widen8(at[32 * v], gv);
          widen8(at[stream + 32 * v], xv);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            xv[i] = mul2(add2(xv[i], less), scale);
            gv[i] = mul2(gv[i], w[v][i]);
          }
        }
        f32x2 out[4];
        widen8(rv, out);
#pragma unroll
        for (int i = 0; i < 4; ++i) out[i] = fma2(scale, fma2(xv[i], c2, add2(gv[i], c1)), out[i]);
        to[32 * v] = narrow8(out);
      }
    }
    if (!kKeepAll) fill(stage);  // the results above have used its values
    if (++stage == stages) stage = 0;
  }
  if constexpr (SUMS) {
    // The sums of the rows side by side in a block meet in the ring: [group][2][K]
    const int K = static_cast<int>(p.K);
    const bool alone = p.part == nullptr;  // one block: its sums are dw and db
    auto* const sums = reinterpret_cast<float4*>(ring);
    auto* const block_sums = reinterpret_cast<float4*>(p.part + static_cast<int64_t>(blockIdx.x) * 2 * p.K);
    const bool meet = ty > 1 || alone;
    if (meet) {
      cp_async_wait<0>();
      __syncthreads();
    }
    float* out = reinterpret_cast<float*>(meet ? sums + group * (K / 2) : block_sums);
    auto put = [](float* to, const f32x2(&s)[4]) {
      const float2 a = halves(s[0]), b = halves(s[1]), c = halves(s[2]), d = halves(s[3]);
      *reinterpret_cast<float4*>(to) = make_float4(a.x, a.y, b.x, b.y);
      *reinterpret_cast<float4*>(to + 4) = make_float4(c.x, c.y, d.x, d.y);
    };
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (on(v)) {
        put(out + 8 * (first + 32 * v), sw[v]);
        put(out + K + 8 * (first + 32 * v), sb[v]);
      }
    }
    if (!meet) return;
    __syncthreads();
    for (int i = tid; i < K / 2; i += threads) {
      float4 a = sums[i];
      for (int q = 1; q < ty; ++q) {
        const float4 c = sums[q * (K / 2) + i];
        a.x += c.x, a.y += c.y, a.z += c.z, a.w += c.w;
      }
      if (!alone) {
        block_sums[i] = a;
        continue;
      }
      auto* to = static_cast<__nv_bfloat16*>(4 * i < K ? p.dw : p.db);
      if (to != nullptr)
        *reinterpret_cast<uint2*>(to + (4 * i < K ? 4 * i : 4 * i - K)) = make_uint2(pack_bf16(a.x, a.y), pack_bf16(a.z, a.w));
    }
  }
}

// Pieces of a thread, threads of a row, rows of a block
struct RowShape {
  int v, tx, ty;
};

RowShape row_shape(int64_t K, int v, int block) {
  RowShape s;
  s.v = v;
  s.tx = static_cast<int>(ceil_div(K / 8, 32 * v) * 32);
  s.ty = s.tx >= block ? 1 : block / s.tx;
  if (s.ty > kMaxGroups) s.ty = kMaxGroups;
  return s;
}

// Four pieces a thread (32 values) make the two sums, about 30 instructions a warp each,
// cheap beside the values: 4608 x 4096 takes 13.8 us with four, 16.2 with two, 26.1 with one.
RowShape forward_shape(int64_t K) {
  const int64_t pieces = K / 8;
  return row_shape(K, pieces <= 32 ? 1 : pieces <= 64 ? 2 : 4, 256);
}

// Two pieces a thread leave room for the sums of their columns; 512 threads of 128
// registers are what an SM holds, so each gets one block, whose rows' sums meet in it
// (4608 x 4096: 30.1 us; 31.3 with two blocks of 256, 35 with one piece and two rows at a time).
RowShape backward_shape(int64_t K) {
  int v = 2;
  while (K / 8 > v * kMaxThreadsBackward) v *= 2;
  return row_shape(K, v, 512);
}

template <typename Kernel>
cudaError_t allow_ring(Kernel* kernel, std::once_flag (&once)[64], cudaError_t (&configured)[64]) {
  return once_per_device(once, configured, [kernel]() {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kRingMost));
  });
}

template <int V, bool FULL>
cudaError_t launch_forward(const LayerNormLaunch& p, const RowShape& s, int sms, cudaStream_t stream) {
  static std::once_flag once[64];
  static cudaError_t configured[64];
  cudaError_t e = allow_ring(layer_norm_kernel<V, FULL>, once, configured);
  if (e != cudaSuccess) return e;
  const int threads = s.tx * s.ty;
  const int64_t want = ceil_div(p.M, s.ty), most = static_cast<int64_t>(sms) * (kMaxThreads / threads);
  return launch_after_previous(layer_norm_kernel<V, FULL>, dim3(static_cast<unsigned>(want < most ? want : most)),
                               dim3(threads), static_cast<size_t>(V) * threads * 16, stream, p, s.tx);
}

template <int V, bool SUMS, bool FULL>
cudaError_t launch_backward(const LayerNormBackwardLaunch& p, const RowShape& s, int blocks, cudaStream_t stream) {
  static std::once_flag once[64];
  static cudaError_t configured[64];
  cudaError_t e = allow_ring(layer_norm_backward_kernel<V, SUMS, FULL>, once, configured);
  if (e != cudaSuccess) return e;
  const int threads = s.tx * s.ty, stage = (p.dr != nullptr ? 3 : 2) * V * threads * 16;
  const int fit = static_cast<int>(kRingMost) / stage, stages = fit < kMaxStages ? fit : kMaxStages;
  size_t smem = static_cast<size_t>(stages) * stage;
  if (SUMS) {
    const size_t sums = static_cast<size_t>(s.ty) * 2 * static_cast<size_t>(p.K) * 4;
    if (sums > smem) smem = sums;
  }
  return launch_after_previous(layer_norm_backward_kernel<V, SUMS, FULL>, dim3(static_cast<unsigned>(blocks)), dim3(threads),
                               smem, stream, p, s.tx, stages);
}

template <int V>
cudaError_t launch_forward_as(const LayerNormLaunch& p, const RowShape& s, int sms, cudaStream_t stream) {
  return p.K == 8 * V * s.tx ? launch_forward<V, true>(p, s, sms, stream) : launch_forward<V, false>(p, s, sms, stream);
}

template <int V, bool SUMS>
cudaError_t launch_backward_as(const LayerNormBackwardLaunch& p, const RowShape& s, int blocks, cudaStream_t stream) {
  return p.K == 8 * V * s.tx ? launch_backward<V, SUMS, true>(p, s, blocks, stream)
                             : launch_backward<V, SUMS, false>(p, s, blocks, stream);
}

// A second kernel for the blocks' sums takes as long as two rows after one another (2 us;
// and another launch on the host): so many stay in one block.  (A cluster of 8 blocks for eight
// times as many was slower: 7.0 us for 5.6 with 16 x 4096.)
bool one_block(int64_t M, const RowShape& s) { return M <= static_cast<int64_t>(s.ty) * kRowsAlone; }

int backward_blocks(int64_t M, const RowShape& s) {
  const int64_t want = ceil_div(M, s.ty);
  return static_cast<int>(want < kBackwardBlocks ? want : kBackwardBlocks);
}

}  // namespace

cudaError_t launch_layer_norm(const LayerNormLaunch& p, int sms, cudaStream_t stream) {
  const RowShape s = forward_shape(p.K);
  switch (s.v) {
    case 1: return launch_forward_as<1>(p, s, sms, stream);
    case 2: return launch_forward_as<2>(p, s, sms, stream);
    default: return launch_forward_as<4>(p, s, sms, stream);
  }
}

size_t layer_norm_backward_workspace(int64_t M, int64_t K) {
  if (K > kFusedCols) return column_pass_workspace(M, K, 2);
  const RowShape s = backward_shape(K);
  return one_block(M, s) ? 0 : static_cast<size_t>(backward_blocks(M, s)) * 2 * static_cast<size_t>(K) * 4;
}

cudaError_t launch_layer_norm_backward(const LayerNormBackwardLaunch& p, cudaStream_t stream) {
  const RowShape s = backward_shape(p.K);
  const int blocks = backward_blocks(p.M, s);
  const bool sums = p.dw != nullptr || p.db != nullptr;
  if (sums && p.K <= kFusedCols) {
    const bool alone = one_block(p.M, s);
    const cudaError_t e = launch_backward_as<2, true>(p, s, alone ? 1 : blocks, stream);
    return e != cudaSuccess || alone ? e : launch_column_sums(p.part, blocks, p.K, p.dw, p.db, stream);
  }
  const cudaError_t e = s.v == 2   ? launch_backward_as<2, false>(p, s, blocks, stream)
                        : s.v == 4 ? launch_backward_as<4, false>(p, s, blocks, stream)
                                   : launch_backward_as<8, false>(p, s, blocks, stream);
  if (e != cudaSuccess || !sums) return e;
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
