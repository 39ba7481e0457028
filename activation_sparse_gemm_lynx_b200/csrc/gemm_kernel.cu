// gemm_kernel.cu -- persistent tcgen05 GEMM for the Lynx layer:
//   Y[M,N] = bf16( S(X) W^T  (+ T B^T)  (+ bias) )
// with S(X) either the 2:4-compressed activations (tcgen05.mma.sp, sparse
// operand on the A side, metadata in TMEM) or the dense X (tcgen05.mma, the
// path of layers left dense by selective layer skipping).  T = X A^T is the
// LoRA down-projection produced by the sparsify pass; the LoRA up-projection
// runs as two extra dense K=32 steps into the same TMEM accumulator tile, and
// the bias is added in fp32 before the single bf16 rounding of Y (after an
// optional activation, GELU tanh form, also in fp32).
// (RT-Lynx pages: qingkeai.online article section 02, Y = S(X) W^T; section
// 03.2, LoRA residual; section 03.3, skipped layers; section 04, sparse GEMM
// and LoRA residual fused into the CUDA kernel.)
//
// Tile: 128 rows x BN columns per CTA (32 to 256: as narrow as give every SM a tile),
// one CTA per SM (persistent, static round-robin over tiles, M-grouped raster for L2
// reuse).
//   warp 0      TMA producer, per K-step of 64 (two a stage, one at BN = 256): A tile
//               (vals 128x32 compressed, 64B swizzle, or X 128x64, 128B swizzle), W
//               tile (BNx64, 128B swizzle) and, for every two steps of the sparse
//               path, one 2 KB metadata block (plain bulk copy).  LoRA stages: T
//               (128x32) and B (BNx32), 64B swizzle.
//   warp 1      TMEM owner + MMA issuer: tcgen05.cp of metadata into a 4-slot TMEM
//               ring, tcgen05.mma(.sp) into the accumulator, tcgen05.commit to release
//               stages / publish the accumulator.
//   warps 2-9   epilogue: tcgen05.ld 32x32b -> s * acc + bias -> bf16 -> global
//               (two warps per TMEM lane quarter, half of the columns each).
// Accumulators: 1 TMEM buffer for BN = 256, 2 (double buffered) below.
//
// 20 rows of 4096 -> 4096, dense: 15.0 us, 33.5 MB of W (5.1 us); 64 rows of 2048 -> 1000
// 8.3 us.  Bound by the MMA warp: a stage's wait, election and commit take it about 300
// cycles beside 8 MMAs of 40.
#include <cuda_bf16.h>

#include "lynx_act.cuh"
#include "lynx_internal.h"
#include "lynx_ptx.cuh"
#include "lynx_rows.cuh"

namespace lynx {

namespace {

constexpr int kGemmThreads = 320;  // producer, MMA, 8 epilogue warps
constexpr uint32_t kTmemCols = 512;
constexpr int kGroupM = 16;
constexpr int kEslots = 4;

template <int BN, bool SPARSE>
struct Cfg {
  // K-steps of 64 a stage.  A wait and a commit take the MMA warp about as long as the
  // MMAs of four steps; at 256 columns two steps would leave two stages.
  static constexpr int kSub = BN == 256 ? 1 : 2;
  static constexpr uint32_t kARowBytes = SPARSE ? 64u : 128u;             // a row of one k-step of A
  static constexpr uint32_t kABytes = 128u * kARowBytes;
  static constexpr uint32_t kBBytes = static_cast<uint32_t>(BN) * 128u;   // BN rows x 64 dense K
  static constexpr uint32_t kEBytes = SPARSE ? 2048u : 0u;
  static constexpr uint32_t kBOff = kSub * kABytes;                       // the steps' A, then their B, then metadata
  static constexpr uint32_t kEOff = kSub * (kABytes + kBBytes);
  static constexpr uint32_t kStageBytes = ((kEOff + kEBytes + 1023u) / 1024u) * 1024u;
  static constexpr int kStages = static_cast<int>((212u * 1024u) / kStageBytes);
  static constexpr int kAcc = BN > 128 ? 1 : 2;
  static constexpr uint32_t kEcol0 = static_cast<uint32_t>(kAcc * BN);
  static constexpr uint32_t kLoraBBytes = static_cast<uint32_t>(BN) * 64u;  // B: BN rows x 32
  static_assert(kStages >= 3, "pipeline too shallow");
  static_assert(kEcol0 + 4 * kEslots <= kTmemCols, "TMEM budget");
};

template <int BN, bool SPARSE>
struct __align__(1024) GemmSmem {
  using C = Cfg<BN, SPARSE>;
  uint8_t stage[C::kStages][C::kStageBytes];
  uint64_t full[C::kStages];
  uint64_t empty[C::kStages];
  uint64_t acc_full[2];
  uint64_t acc_empty[2];
  uint64_t drain;
  float bias_s[BN];  // the current tile's bias, fp32
  uint32_t tmem_base;
  volatile uint32_t abort_flag;
};

__device__ __forceinline__ void tmem_ld_chunk(uint32_t taddr, uint32_t (&r)[32]) { tmem_ld_32x32b_x32(taddr, r); }
__device__ __forceinline__ void tmem_ld_chunk(uint32_t taddr, uint32_t (&r)[16]) { tmem_ld_32x32b_x16(taddr, r); }

constexpr uint32_t kBarEpilogue = 2;  // named barrier of the 8 epilogue warps
constexpr uint32_t kEpiThreads = 256;

__device__ __forceinline__ void tile_coords(int tile, int ntm, int ntn, int& mb, int& nb) {
  const int per_group = kGroupM * ntn;
  const int group = tile / per_group;
  const int first_m = group * kGroupM;
  const int gm = min(kGroupM, ntm - first_m);
  const int in_group = tile - group * per_group;
  mb = first_m + in_group % gm;
  nb = in_group / gm;
}

// EXT: a residual is added to the activation's value, or the value before the
// activation is stored too.  A kernel of its own, so that the plain layer's
// epilogue keeps its registers.
template <int BN, bool SPARSE, bool EXT>
__global__ void __launch_bounds__(kGemmThreads, 1)
lynx_gemm_kernel(const __grid_constant__ GemmLaunch p) {
  using C = Cfg<BN, SPARSE>;
  extern __shared__ uint8_t smem_raw[];
  GemmSmem<BN, SPARSE>& sm = *reinterpret_cast<GemmSmem<BN, SPARSE>*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));

  const uint32_t warp = warp_id_sync();
  const uint32_t lane = lane_id();
  const int ntm = static_cast<int>((p.M + 127) / 128);
  const int ntn = static_cast<int>((p.N + BN - 1) / BN);
  const int ntiles = ntm * ntn;
  const int nk = static_cast<int>(p.K / 64);  // steps of 64 dense K
  const int nks = (nk + C::kSub - 1) / C::kSub;  // and their stages
  const int kblocks = static_cast<int>((p.K + 127) / 128);
  const bool lora = p.lora != 0;
  const int lsteps = lora ? (p.r + 31) / 32 : 0;  // LoRA-up stages of K = 32 (zero-filled past r)
  const uint32_t a_rows = static_cast<uint32_t>(p.a_rows);  // rows of a box of A or T: the rest of its 128 is not written

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&sm.acc_full[a], 1);
      mbar_init(&sm.acc_empty[a], 8);
    }
    mbar_init(&sm.drain, 1);
    sm.abort_flag = 0u;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&sm.tmem_base, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // the prologue above may overlap the previous kernel (programmatic launch);
  // its outputs are read only from here on
  pdl_wait();

  // a bounded wait of a whole warp: every lane waits, and all take the same decision
  auto wait = [&](uint64_t* bar, uint32_t parity, uint32_t code) {
    const bool late = sm.abort_flag || !mbar_wait(bar, parity);
    if (!__any_sync(0xffffffffu, late)) return true;
    if (lane == 0 && !sm.abort_flag) {
      record_error(p.status, code);
      sm.abort_flag = 1u;
    }
    return false;
  };

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    // (the whole warp, one elected lane issuing: see the MMA issuer)
    if (elect_one()) {
      tma_prefetch_desc(&p.tm_a);
      tma_prefetch_desc(&p.tm_b);
      if (lora) {
        tma_prefetch_desc(&p.tm_t);
        tma_prefetch_desc(&p.tm_lb);
      }
    }
    __syncwarp();
    uint32_t g = 0;
    bool ok = !p.stall_test;
    for (int tile = blockIdx.x; ok && tile < ntiles; tile += gridDim.x) {
      int mb, nb;
      tile_coords(tile, ntm, ntn, mb, nb);
      const int32_t row0 = mb * 128;
      const int32_t col0 = nb * BN;
      const int steps = nks + lsteps;
      for (int kit = 0; kit < steps; ++kit, ++g) {
        const uint32_t slot = g % C::kStages;
        const uint32_t ph = (g / C::kStages) & 1u;
        ok = wait(&sm.empty[slot], ph ^ 1u, kDevTimeoutEmpty);
        if (!ok) break;
        uint8_t* st = sm.stage[slot];
        if (kit < nks) {
          const int k0 = kit * C::kSub;
          const uint32_t subs = k0 + C::kSub <= nk ? C::kSub : 1u;
          const bool load_e = SPARSE && k0 % 2 == 0;
          if (elect_one()) {
            mbar_arrive_expect_tx(&sm.full[slot], subs * (a_rows * C::kARowBytes + C::kBBytes) + (load_e ? 2048u : 0u));
#pragma unroll
            for (uint32_t u = 0; u < C::kSub; ++u) {
              if (u < subs) {
                tma_load_2d(st + u * C::kABytes, &p.tm_a, &sm.full[slot], (k0 + u) * (SPARSE ? 32 : 64), row0);
                tma_load_2d(st + C::kBOff + u * C::kBBytes, &p.tm_b, &sm.full[slot], (k0 + u) * 64, col0);
              }
            }
            if (load_e) {
              const uint8_t* src =
                  p.meta + (static_cast<size_t>(mb) * kblocks + k0 / 2) * kMetaBlockBytes;
              bulk_load(st + C::kEOff, src, 2048u, &sm.full[slot]);
            }
          }
        } else {
          const int l = kit - nks;
          if (elect_one()) {
            mbar_arrive_expect_tx(&sm.full[slot], a_rows * 64u + C::kLoraBBytes);
            tma_load_2d(st, &p.tm_t, &sm.full[slot], l * 32, row0);
            tma_load_2d(st + C::kBOff, &p.tm_lb, &sm.full[slot], l * 32, col0);
          }
        }
        __syncwarp();
      }
    }
    // drain: the last fill of every stage must have landed before exit
    const uint32_t issued = g;
    for (uint32_t b = issued; b > 0 && b + C::kStages > issued; --b) {
      const uint32_t x = b - 1;
      if (!mbar_wait(&sm.full[x % C::kStages], (x / C::kStages) & 1u, kWaitLimitNs / 4) && lane == 0)
        record_error(p.status, kDevTimeoutDrain);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    // The whole warp runs the loop, so that the operands stay warp-uniform, and one
    // elected lane issues each tcgen05 instruction.  Issued from a branch that only one
    // lane takes, an MMA costs more than its bytes: 20 tokens of 4096 -> 4096 took 34 us.
    const uint32_t idesc_main = make_idesc_bf16(128, BN, SPARSE);
    const uint32_t idesc_dense = make_idesc_bf16(128, BN, false);
    uint32_t g = 0, eslot = 0;
    int acc_count = 0;
    bool ok = true;
    for (int tile = blockIdx.x; ok && tile < ntiles; tile += gridDim.x, ++acc_count) {
      const int acc = acc_count % C::kAcc;
      const uint32_t acc_ph = static_cast<uint32_t>(acc_count / C::kAcc) & 1u;
      if (!wait(&sm.acc_empty[acc], acc_ph ^ 1u, kDevTimeoutAccum)) break;
      tc_fence_after();
      const uint32_t d_tmem = sm.tmem_base + static_cast<uint32_t>(acc * BN);
      const int steps = nks + lsteps;
      for (int kit = 0; kit < steps; ++kit, ++g) {
        const uint32_t slot = g % C::kStages;
        const uint32_t ph = (g / C::kStages) & 1u;
        ok = wait(&sm.full[slot], ph, kDevTimeoutFull);
        if (!ok) break;
        tc_fence_after();
        const uint32_t sa = smem_u32(sm.stage[slot]);
        const uint32_t sb = sa + C::kBOff;
        const int k0 = kit * C::kSub;
        if (SPARSE && kit < nks && k0 % 2 == 0) eslot = (eslot + 1) % kEslots;
        // one election a stage: each costs as much as an MMA of this size
        if (elect_one()) {
          if (kit < nks) {
            if (SPARSE && k0 % 2 == 0) {
              const uint64_t edesc = make_sdesc(sa + C::kEOff, 2048, 128, kSwNone);
              tc_cp_128x128b(sm.tmem_base + C::kEcol0 + 4 * eslot, edesc);
            }
#pragma unroll
            for (int u = 0; u < C::kSub; ++u) {
              if (k0 + u >= nk) break;
              const uint32_t ua = sa + u * C::kABytes, ub = sb + u * C::kBBytes;
              if (SPARSE) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                  const uint32_t ecol = C::kEcol0 + 4 * eslot + 2 * ((k0 + u) % 2) + j;
                  const uint64_t da = make_sdesc(ua + 32 * j, 16, 512, kSw64);
                  const uint64_t db = make_sdesc(ub + 64 * j, 16, 1024, kSw128);
                  const uint32_t idesc = idesc_main | (ecol & 1u);
                  mma_sp_bf16(d_tmem, da, db, sm.tmem_base + (ecol & ~1u), idesc, kit > 0 || u > 0 || j > 0);
                }
              } else {
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                  const uint64_t da = make_sdesc(ua + 32 * kk, 16, 1024, kSw128);
                  const uint64_t db = make_sdesc(ub + 32 * kk, 16, 1024, kSw128);
                  mma_bf16(d_tmem, da, db, idesc_main, kit > 0 || u > 0 || kk > 0);
                }
              }
            }
          } else {
            const int l = kit - nks;
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
              if (32 * l + 16 * kk >= p.r) break;  // past r: the zero-filled half of the box
              const uint64_t da = make_sdesc(sa + 32 * kk, 16, 512, kSw64);
              const uint64_t db = make_sdesc(sb + 32 * kk, 16, 512, kSw64);
              mma_bf16(d_tmem, da, db, idesc_dense, 1);
            }
          }
          tc_commit(&sm.empty[slot]);
        }
        __syncwarp();
      }
      if (!ok) break;
      if (elect_one()) tc_commit(&sm.acc_full[acc]);
      __syncwarp();
    }
    if (elect_one()) tc_commit(&sm.drain);
    __syncwarp();
    if (!mbar_wait(&sm.drain, 0) && lane == 0) record_error(p.status, kDevTimeoutDrain);
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    // Y = bf16(act(s_row * acc + bias)).  Two warps per TMEM lane quarter, each
    // draining half of the columns into registers; the TMEM buffer is released
    // before the global stores, so the next tile's MMAs overlap them.
    constexpr int kHalf = BN / 2;
    constexpr int kChunk = kHalf < 32 ? kHalf : 32;  // columns read from TMEM at a time
    const uint32_t q = warp & 3u;              // TMEM lane quarter this warp may access
    const uint32_t ch = (warp - 2u) >> 2;      // which half of the columns
    const uint32_t row = 32u * q + lane;
    const uint32_t et = threadIdx.x - 64u;     // 0..255
    const __nv_bfloat16* bias = static_cast<const __nv_bfloat16*>(p.bias);
    __nv_bfloat16* y = static_cast<__nv_bfloat16*>(p.y);
    int acc_count = 0;
    for (int tile = blockIdx.x; tile < ntiles; tile += gridDim.x, ++acc_count) {
      int mb, nb;
      tile_coords(tile, ntm, ntn, mb, nb);
      const int acc = acc_count % C::kAcc;
      const uint32_t acc_ph = static_cast<uint32_t>(acc_count / C::kAcc) & 1u;
      const int64_t grow = static_cast<int64_t>(mb) * 128 + row;
      const bool row_ok = grow < p.M;
      const int64_t n_base = static_cast<int64_t>(nb) * BN;
      named_bar_sync(kBarEpilogue, kEpiThreads);  // the previous tile's bias is no longer read
      for (uint32_t j = et; j < static_cast<uint32_t>(BN); j += kEpiThreads) {
        const int64_t n = n_base + j;
        sm.bias_s[j] = (bias != nullptr && n < p.N) ? __bfloat162float(bias[n]) : 0.f;
      }
      const float s = (p.row_scale != nullptr && row_ok) ? p.row_scale[grow] : 1.f;
      bool ok = !sm.abort_flag;
      if (ok && !mbar_wait(&sm.acc_full[acc], acc_ph)) {
        record_error(p.status, kDevTimeoutAccum);
        sm.abort_flag = 1u;
        ok = false;
      }
      // publishes the bias tile and makes the stop decision identical in all warps
      if (named_bar_red_or(kBarEpilogue, kEpiThreads, !ok)) break;
      tc_fence_after();
      uint32_t out[kHalf / 2];
#pragma unroll
      for (int c = 0; c < kHalf / kChunk; ++c) {
        const int col = static_cast<int>(ch) * kHalf + kChunk * c;
        uint32_t r[kChunk];
        tmem_ld_chunk(sm.tmem_base + ((32u * q) << 16) + static_cast<uint32_t>(acc * BN + col), r);
        tmem_ld_wait();
        uint32_t add[kChunk / 16][8] = {}, pre[kChunk / 16][8];
        const int left = row_ok ? static_cast<int>(p.N - n_base) - col : 0;
        const int64_t at = grow * p.N + n_base + col;
        if constexpr (EXT) {
          if (p.residual != nullptr) {
#pragma unroll
            for (int v = 0; v < kChunk / 16; ++v)
              load_row16(add[v], static_cast<const __nv_bfloat16*>(p.residual) + at + 16 * v, left - 16 * v, p.wide);
          }
        }
#pragma unroll
        for (int i = 0; i < kChunk / 2; ++i) {
          float a = __fmaf_rn(s, __uint_as_float(r[2 * i]), sm.bias_s[col + 2 * i]);
          float b = __fmaf_rn(s, __uint_as_float(r[2 * i + 1]), sm.bias_s[col + 2 * i + 1]);
          if constexpr (EXT) {
            __nv_bfloat162 z = __floats2bfloat162_rn(a, b);
            pre[i / 8][i % 8] = *reinterpret_cast<uint32_t*>(&z);
          }
          if (p.act == kActGeluTanh) {
            a = gelu_tanh(a);
            b = gelu_tanh(b);
          }
          if constexpr (EXT) {
            if (p.residual != nullptr) {  // +0 added would turn -0 into +0
              a = __fadd_rn(a, __uint_as_float(add[i / 8][i % 8] << 16));
              b = __fadd_rn(b, __uint_as_float(add[i / 8][i % 8] & 0xFFFF0000u));
            }
          }
          __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
          out[kChunk / 2 * c + i] = *reinterpret_cast<uint32_t*>(&h);
        }
        if constexpr (EXT) {
          if (p.z != nullptr) {
#pragma unroll
            for (int v = 0; v < kChunk / 16; ++v)
              store_row16<false>(static_cast<__nv_bfloat16*>(p.z) + at + 16 * v, pre[v], left - 16 * v, p.wide);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.acc_empty[acc]);
      // whole sectors: in two halves of 16 bytes, rows of whole lines cost up to a fifth of the kernel's
      // time (1000 x 512 -> 2304, dense, 8.5 us for 6.9; -> 2296, whose rows are on 16 bytes, 7.3)
      const int64_t n0 = n_base + static_cast<int64_t>(ch) * kHalf;
      const int left = row_ok && n0 < p.N ? static_cast<int>(p.N - n0) : 0;
#pragma unroll
      for (int v = 0; v < kHalf / 16; ++v) {
        uint32_t pk[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) pk[i] = out[8 * v + i];
        store_row16<true>(y + grow * p.N + n0 + 16 * v, pk, left - 16 * v, p.wide_y);
      }
    }
  }

  __syncthreads();
  if (warp == 1) tmem_dealloc(sm.tmem_base, kTmemCols);
}

template <int BN, bool SPARSE, bool EXT>
cudaError_t launch_variant(const GemmLaunch& p, cudaStream_t stream) {
  const size_t smem = sizeof(GemmSmem<BN, SPARSE>) + 1024;
  static std::once_flag once[64];
  static cudaError_t configured[64];
  cudaError_t e = once_per_device(once, configured, [smem]() {
    return cudaFuncSetAttribute(lynx_gemm_kernel<BN, SPARSE, EXT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(smem));
  });
  if (e != cudaSuccess) return e;
  return launch_after_previous(lynx_gemm_kernel<BN, SPARSE, EXT>, dim3(static_cast<unsigned>(p.grid)),
                               dim3(kGemmThreads), smem, stream, p);
}

template <int BN>
cudaError_t launch_bn(const GemmLaunch& p, cudaStream_t stream) {
  if (p.ext) return p.sparse ? launch_variant<BN, true, true>(p, stream) : launch_variant<BN, false, true>(p, stream);
  return p.sparse ? launch_variant<BN, true, false>(p, stream) : launch_variant<BN, false, false>(p, stream);
}

}  // namespace

cudaError_t launch_gemm(const GemmLaunch& p, cudaStream_t stream) {
  switch (p.bn) {
    case 32: return launch_bn<32>(p, stream);
    case 64: return launch_bn<64>(p, stream);
    case 128: return launch_bn<128>(p, stream);
    default: return launch_bn<256>(p, stream);
  }
}

}  // namespace lynx
