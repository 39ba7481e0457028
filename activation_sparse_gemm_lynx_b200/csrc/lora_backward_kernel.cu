// lora_backward_kernel.cu -- the adapter's gradients from an 8-bit checkpoint
// (lynx_lora_backward):  T = x A^T, dT = dY B, dB = dY^T T, dA = dT^T x.
#include "lynx_ckpt8.cuh"

namespace lynx {

namespace {

constexpr int kThreads = 256;
constexpr int kTile = 32;

// Readers of an operand by (i, p): i an output index, p along the sum.
struct Bf16At {
  const __nv_bfloat16* base;
  int64_t si, sp;
  __device__ float operator()(int64_t i, int64_t p) const { return __bfloat162float(base[i * si + p * sp]); }
};

template <int FMT>
struct CkptAt {
  const uint8_t* q;
  const uint8_t* e;
  int64_t K;
  bool k_is_sum;  // (i, p) = (m, k), else (k, m)
  __device__ float operator()(int64_t i, int64_t p) const {
    const int64_t m = k_is_sum ? i : p, k = k_is_sum ? p : i;
    float v[4];
    ckpt8_decode4<FMT>(q[m * K + k], v);
    return v[0] * ckpt8_factor<FMT>(e[(m * K + k) / 32]);
  }
};

// out[i * si + j * sj] = bf16(sum_p left(i, p) right(j, p)), 32 x 32 a block
template <typename L, typename R>
__global__ void __launch_bounds__(kThreads) product_kernel(L left, R right, int64_t I, int64_t J, int64_t P,
                                                           __nv_bfloat16* out, int64_t si, int64_t sj) {
  __shared__ float ls[kTile][kTile + 1], rs[kTile][kTile + 1];
  const int tx = threadIdx.x % kTile, ty = threadIdx.x / kTile;
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * kTile, j0 = static_cast<int64_t>(blockIdx.y) * kTile;
  float acc[4] = {};
  for (int64_t p0 = 0; p0 < P; p0 += kTile) {
    for (int y = ty; y < kTile; y += 8) {
      ls[y][tx] = i0 + y < I && p0 + tx < P ? left(i0 + y, p0 + tx) : 0.f;
      rs[y][tx] = j0 + y < J && p0 + tx < P ? right(j0 + y, p0 + tx) : 0.f;
    }
    __syncthreads();
    for (int p = 0; p < kTile; ++p)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[c] = fmaf(ls[ty + 8 * c][p], rs[tx][p], acc[c]);
    __syncthreads();
  }
#pragma unroll
  for (int c = 0; c < 4; ++c)
    if (i0 + ty + 8 * c < I && j0 + tx < J) out[(i0 + ty + 8 * c) * si + (j0 + tx) * sj] = __float2bfloat16_rn(acc[c]);
}

template <typename L, typename R>
void product(L left, R right, int64_t I, int64_t J, int64_t P, void* out, int64_t si, int64_t sj, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>((I + kTile - 1) / kTile), static_cast<unsigned>((J + kTile - 1) / kTile));
  product_kernel<<<grid, kThreads, 0, s>>>(left, right, I, J, P, static_cast<__nv_bfloat16*>(out), si, sj);
}

template <int FMT>
void run(const LoraBackwardLaunch& p, cudaStream_t s) {
  const auto* q = static_cast<const uint8_t*>(p.q);
  const auto* e = static_cast<const uint8_t*>(p.e);
  const auto* dy = static_cast<const __nv_bfloat16*>(p.dy);
  const auto* a = static_cast<const __nv_bfloat16*>(p.a);
  const auto* b = static_cast<const __nv_bfloat16*>(p.b);
  auto* t = reinterpret_cast<__nv_bfloat16*>(p.ws);
  auto* dt = p.dt != nullptr ? static_cast<__nv_bfloat16*>(p.dt) : t + p.M * p.r;
  const int64_t r = p.r;
  product(CkptAt<FMT>{q, e, p.K, true}, Bf16At{a, p.K, 1}, p.M, r, p.K, t, r, 1, s);
  product(Bf16At{dy, p.N, 1}, Bf16At{b, 1, r}, p.M, r, p.N, dt, r, 1, s);
  product(Bf16At{dy, 1, p.N}, Bf16At{t, 1, r}, p.N, r, p.M, p.db, r, 1, s);
  product(CkptAt<FMT>{q, e, p.K, false}, Bf16At{dt, 1, r}, p.K, r, p.M, p.da, 1, p.K, s);
}

}  // namespace

size_t lora_backward_workspace(int64_t M, int64_t N, int64_t K, int64_t r) {
  (void)N;
  (void)K;
  return static_cast<size_t>(M) * static_cast<size_t>(r) * 4;
}

cudaError_t launch_lora_backward(const LoraBackwardLaunch& p, int sms, cudaStream_t s) {
  (void)sms;
  if (p.format == kCkpt8Int8)
    run<kCkpt8Int8>(p, s);
  else
    run<kCkpt8E4M3>(p, s);
  return cudaGetLastError();
}

}  // namespace lynx
