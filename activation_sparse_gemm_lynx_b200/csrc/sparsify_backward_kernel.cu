// sparsify_backward_kernel.cu -- the gradient through S(X) at an 8-bit
// checkpoint (lynx_sparsify_backward).
//
// S(X) = s m x with s = L / Lk, L = sum|x|, Lk = sum m|x| of the row.  With the
// selection m fixed, dL/dx_k = s m_k g_k + D ds/dx_k, D = sum_j m_j g_j x_j, and
// ds/dx_k = sign(x_k) / Lk - m_k sign(x_k) L / Lk^2 = sign(x_k) (1 - s m_k) / Lk.
// The LoRA branch adds dT A, a product of rank r.
//
// Two phases over the same tiles, since every output needs its row's three sums:
// a cluster has 128 rows, each block a range of their columns, in tiles of 64.
//   phase 1  L, Lk and D of the block's columns; the blocks exchange them
//   phase 2  the tiles again, last first (the most recent are still in L2), with
//            dT A from tcgen05.mma in TMEM, dX out by TMA
// In both a thread has one row (a TMEM lane) and 32 columns of a tile, so a group
// of 4 never leaves a thread and the row sums need no shuffles.
//   warp 0   TMA: G, the stored bytes and, in phase 2, A's rows of the columns
//   warp 1   the MMAs of phase 2
//   warp 2   the tiles' exponents (2 bytes a row: too narrow for TMA)
//   warp 3   TMA stores of dX
//   warps 4-11  sums and outputs
// Two blocks an SM where the rank leaves room, so that one's loads run beside the
// other's exchange and tails.
#include "lynx_ckpt8.cuh"
#include "lynx_internal.h"
#include "lynx_ptx.cuh"

namespace lynx {

namespace {

constexpr int kRoleWarps = 4;
constexpr int kSumWarps = 8;
constexpr int kThreads = 32 * (kRoleWarps + kSumWarps);
constexpr int kCols = 64;
constexpr int kMaxStages = 6;
constexpr int kMaxCluster = 8;
constexpr uint32_t kGBytes = 128 * 128;  // 128 rows x 64 bf16, 128B swizzle
constexpr uint32_t kQBytes = 128 * 64;   // 128 rows x 64 bytes, 64B swizzle
constexpr uint32_t kTBox = 128 * 128;    // dT: 128 rows x 64 of r
// dynamic shared memory of a block, alone on its SM or one of two (16 KB are static)
constexpr uint32_t kSmemAlone = 208 * 1024;
constexpr uint32_t kSmemShared = 97 * 1024;

struct BackLaunch {
  CUtensorMap tm_g;   // G [M,K], box 64 x 128
  CUtensorMap tm_q;   // q [M,K] bytes, box 64 x 128, 64B swizzle
  CUtensorMap tm_dt;  // dT [M,r], box 64 x 128
  CUtensorMap tm_a;   // A [r,K], box 64 x r
  CUtensorMap tm_dx;  // dX [M,K], box 64 x 128
  const uint8_t* e;
  int64_t M, K;
  int r;
  int ranks;          // blocks of a cluster
  int per;            // tiles of a block
  int stages;
  uint32_t stage_bytes;
  int stall_test;
  uint32_t* status;
};

struct BackBars {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t a_full[kMaxStages];
  uint64_t dt_full, d_full[2], d_empty[2], sums, done, out_empty;
  uint32_t tmem_base;
  volatile uint32_t abort_flag;
};

__device__ __forceinline__ bool back_wait(BackBars& b, uint64_t* bar, uint32_t parity, uint32_t* status,
                                          uint32_t code) {
  bool ok = !b.abort_flag && mbar_wait(bar, parity);
  if (!ok && !b.abort_flag) {
    record_error(status, code);
    b.abort_flag = 1u;
  }
  return ok;
}

__device__ __forceinline__ bool two_of_three(bool a, bool b, bool c) { return (a && b) || (a && c) || (b && c); }

// keep[i]: value i is one of the two largest magnitudes of 4, ties to the lower
// position: it is kept if it goes before at least two of the others.
__device__ __forceinline__ void keep4(const float (&v)[4], bool (&keep)[4]) {
  const bool b01 = fabsf(v[0]) >= fabsf(v[1]), b02 = fabsf(v[0]) >= fabsf(v[2]), b03 = fabsf(v[0]) >= fabsf(v[3]);
  const bool b12 = fabsf(v[1]) >= fabsf(v[2]), b13 = fabsf(v[1]) >= fabsf(v[3]), b23 = fabsf(v[2]) >= fabsf(v[3]);
  keep[0] = two_of_three(b01, b02, b03);
  keep[1] = two_of_three(!b01, b12, b13);
  keep[2] = two_of_three(!b02, !b12, b23);
  keep[3] = two_of_three(!b03, !b13, !b23);
}

// Sign of a stored value before the block's factor (an integer, or an e4m3 whose
// smallest magnitude is 2^-9): 1, -1 or 0 (NaN: 0, its row is NaN through s)
template <int FMT>
__device__ __forceinline__ float stored_sign(float v) {
  constexpr float k = FMT == kCkpt8Int8 ? 1.f : 512.f;
  return __saturatef(v * k) - __saturatef(v * -k);
}

template <int FMT, bool LORA>
__global__ void __launch_bounds__(kThreads, 2) sparsify_backward_kernel(const __grid_constant__ BackLaunch p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ BackBars bars;
  __shared__ float inbox[kMaxCluster][3][128];  // every block's row sums
  __shared__ float half_sums[3][128];           // this block's, of the second half of its tiles' columns
  __shared__ uint16_t exps[kMaxStages][128];    // a stage's exponents, two a row
  uint8_t* const sm = smem_raw + ((0u - smem_u32(smem_raw)) & 1023u);
  const uint32_t warp = warp_id_sync(), lane = lane_id();
  const uint32_t rank = cluster_ctarank();
  const int stages = p.stages;
  const int32_t row0 = static_cast<int32_t>(blockIdx.x / static_cast<unsigned>(p.ranks)) * 128;
  const int tile0 = static_cast<int>(rank) * p.per;
  const int tiles = max(0, min(p.per, static_cast<int>(p.K / kCols) - tile0));
  const uint32_t t_boxes = LORA ? static_cast<uint32_t>((p.r + 63) / 64) : 0u;
  uint8_t* const out_sm = sm + t_boxes * kTBox;  // a tile of dX
  uint8_t* const ring = out_sm + kGBytes;
  // tile of step i: phase 1 goes up, phase 2 comes back down
  auto column = [&](int i) { return static_cast<int32_t>(tile0 + (i < tiles ? i : 2 * tiles - 1 - i)) * kCols; };

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&bars.full[s], 2);  // the TMA's and the exponents'
      mbar_init(&bars.a_full[s], 1);
      mbar_init(&bars.empty[s], kSumWarps);
    }
    mbar_init(&bars.done, kSumWarps);
    mbar_init(&bars.out_empty, 1);
    mbar_init(&bars.dt_full, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.d_full[i], 1);
      mbar_init(&bars.d_empty[i], kSumWarps);
    }
    mbar_init(&bars.sums, static_cast<uint32_t>(p.ranks) * 128u);
    bars.abort_flag = 0u;
    fence_mbar_init();
  }
  if (LORA && warp == 1) {
    tmem_alloc(&bars.tmem_base, 128);
    tmem_relinquish();
  }
  tc_fence_before();
  cluster_sync_all();  // the other blocks' barriers exist from here on
  tc_fence_after();
  pdl_wait();

  if (warp == 0) {
    // ------------------------------------------------------------ loads
    if (lane == 0 && !p.stall_test) {
      if (LORA) {
        mbar_arrive_expect_tx(&bars.dt_full, t_boxes * kTBox);
        for (uint32_t b = 0; b < t_boxes; ++b)
          tma_load_2d(sm + b * kTBox, &p.tm_dt, &bars.dt_full, static_cast<int32_t>(64 * b), row0);
      }
      int slot = 0;
      uint32_t phase = 1;
      int issued = 0;
      for (int i = 0; i < 2 * tiles; ++i) {
        if (!back_wait(bars, &bars.empty[slot], phase, p.status, kDevTimeoutEmpty)) break;
        uint8_t* st = ring + static_cast<uint32_t>(slot) * p.stage_bytes;
        mbar_arrive_expect_tx(&bars.full[slot], kGBytes + kQBytes);
        tma_load_2d(st, &p.tm_g, &bars.full[slot], column(i), row0);
        tma_load_2d(st + kGBytes, &p.tm_q, &bars.full[slot], column(i), row0);
        if (LORA && i >= tiles) {
          mbar_arrive_expect_tx(&bars.a_full[slot], 128u * static_cast<uint32_t>(p.r));
          tma_load_2d(st + kGBytes + kQBytes, &p.tm_a, &bars.a_full[slot], column(i), 0);
        }
        ++issued;
        if (++slot == stages) slot = 0, phase ^= 1u;
      }
      if (bars.abort_flag) {
        // copies in flight must land before the block exits
        if (LORA) mbar_wait(&bars.dt_full, 0, kWaitLimitNs / 8);
        for (int i = issued - 1; i >= 0 && i >= issued - stages; --i)
          mbar_wait(&bars.full[i % stages], (i / stages) & 1, kWaitLimitNs / 8);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ dT A
    if constexpr (LORA) {
      constexpr uint32_t idesc = make_idesc_bf16(128, kCols, false) | kIdescBMnMajor;
      auto arrived = [&](uint64_t* bar, uint32_t parity, uint32_t code) {
        return __all_sync(0xffffffffu, back_wait(bars, bar, parity, p.status, code)) != 0;
      };
      bool ok = arrived(&bars.dt_full, 0, kDevTimeoutFull);
      // A's barriers count phase 2 alone, which begins at this slot
      const int slot0 = tiles % stages;
      int slot = slot0;
      uint32_t phase = 0;
      for (int i = 0; ok && i < tiles; ++i) {
        const int buf = i & 1;
        ok = arrived(&bars.a_full[slot], phase, kDevTimeoutFull) &&
             arrived(&bars.d_empty[buf], ((i >> 1) & 1) ^ 1, kDevTimeoutAccum);
        if (!ok) break;
        tc_fence_after();
        const uint32_t sa = smem_u32(sm);
        const uint32_t sb = smem_u32(ring) + static_cast<uint32_t>(slot) * p.stage_bytes + kGBytes + kQBytes;
        for (int k = 0; k < p.r / 16; ++k) {
          const uint64_t da = make_sdesc(sa + (k / 4) * kTBox + (k % 4) * 32, 16, 1024, kSw128);
          const uint64_t db = make_sdesc(sb + k * 2048, 16, 1024, kSw128);
          if (elect_one()) mma_bf16(bars.tmem_base + buf * kCols, da, db, idesc, k != 0);
          __syncwarp();
        }
        if (elect_one()) tc_commit(&bars.d_full[buf]);
        __syncwarp();
        if (++slot == stages) slot = 0;
        if (slot == slot0) phase ^= 1u;
      }
    }
  } else if (warp == 2) {
    // ------------------------------------------------------------ exponents
    // Rows lane + 32 j; a tile's two bytes a row, read one tile ahead.
    if (!p.stall_test) {
      const int64_t pitch = p.K / 32;
      uint32_t ahead[4];
      auto load = [&](int i) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int64_t row = static_cast<int64_t>(row0) + lane + 32 * j;
          ahead[j] = i < 2 * tiles && row < p.M
                         ? __ldg(reinterpret_cast<const uint16_t*>(p.e + row * pitch + column(i) / 32))
                         : 0u;
        }
      };
      load(0);
      int slot = 0;
      uint32_t phase = 1;
      for (int i = 0; i < 2 * tiles; ++i) {
        const uint32_t now[4] = {ahead[0], ahead[1], ahead[2], ahead[3]};
        load(i + 1);
        const bool ok = __all_sync(
            0xffffffffu, back_wait(bars, &bars.empty[slot], phase, p.status, kDevTimeoutEmpty));
        if (!ok) break;
#pragma unroll
        for (int j = 0; j < 4; ++j) exps[slot][lane + 32 * j] = static_cast<uint16_t>(now[j]);
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.full[slot]);
        if (++slot == stages) slot = 0, phase ^= 1u;
      }
    }
  } else if (warp == 3) {
    // ------------------------------------------------------------ stores of dX
    if (lane == 0) {
      for (int i = 0; i < tiles; ++i) {
        if (!back_wait(bars, &bars.done, i & 1, p.status, kDevTimeoutAccum)) break;
        tma_store_2d(&p.tm_dx, out_sm, column(tiles + i), row0);
        bulk_commit();
        bulk_wait_read_all();
        mbar_arrive(&bars.out_empty);
      }
      bulk_wait_all();
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ sums and outputs
    const uint32_t quarter = warp & 3u, half = (warp - kRoleWarps) >> 2;
    const uint32_t row = 32u * quarter + lane;
    // 16 bytes of the stored values are 32 of G; units are swizzled by the row
    auto q_unit = [&](int h) { return kGBytes + row * 64 + (((2 * half + h) ^ ((row >> 1) & 3u)) << 4); };
    auto g_unit = [&](int h, int u) { return row * 128 + (((4 * half + 2 * h + u) ^ (row & 7u)) << 4); };
    int slot = 0;
    uint32_t phase = 0;
    bool ok = true;
    float l = 0.f, lk = 0.f, d = 0.f;
    for (int i = 0; i < tiles; ++i) {
      ok = __all_sync(0xffffffffu, back_wait(bars, &bars.full[slot], phase, p.status, kDevTimeoutFull));
      if (!ok) break;
      const uint8_t* st = ring + static_cast<uint32_t>(slot) * p.stage_bytes;
      const float f = ckpt8_factor<FMT>(reinterpret_cast<const uint8_t*>(&exps[slot][row])[half]);
      float bl = 0.f, bk = 0.f, bd = 0.f;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint4 qv = *reinterpret_cast<const uint4*>(st + q_unit(h));
        const uint4 ga = *reinterpret_cast<const uint4*>(st + g_unit(h, 0));
        const uint4 gb = *reinterpret_cast<const uint4*>(st + g_unit(h, 1));
        const uint32_t qw[4] = {qv.x, qv.y, qv.z, qv.w};
        const uint32_t gw[8] = {ga.x, ga.y, ga.z, ga.w, gb.x, gb.y, gb.z, gb.w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          float v[4];
          bool keep[4];
          ckpt8_decode4<FMT>(qw[w], v);
          keep4(v, keep);
          const float g[4] = {bf16_lo(gw[2 * w]), bf16_hi(gw[2 * w]), bf16_lo(gw[2 * w + 1]), bf16_hi(gw[2 * w + 1])};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            bl += fabsf(v[j]);
            if (keep[j]) {
              bk += fabsf(v[j]);
              bd = fmaf(g[j], v[j], bd);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.empty[slot]);
      l = fmaf(bl, f, l);
      lk = fmaf(bk, f, lk);
      d = fmaf(bd, f, d);
      if (++slot == stages) slot = 0, phase ^= 1u;
    }
    // the block's sums of a row, then every block's, in the order of the ranks
    if (half == 1) {
      half_sums[0][row] = l;
      half_sums[1][row] = lk;
      half_sums[2][row] = d;
    }
    named_bar_sync(1, 32 * kSumWarps);
    if (half == 0) {
      const float mine[3] = {l + half_sums[0][row], lk + half_sums[1][row], d + half_sums[2][row]};
#pragma unroll
      for (int k = 0; k < 3; ++k)
        for (int q = 0; q < p.ranks; ++q) st_cluster_f32(mapa_shared(smem_u32(&inbox[rank][k][row]), q), mine[k]);
      for (int q = 0; q < p.ranks; ++q) mbar_arrive_cluster_release(mapa_shared(smem_u32(&bars.sums), q));
    }
    if (ok && !mbar_wait_cluster(&bars.sums, 0)) {
      record_error(p.status, kDevTimeoutFinalize);
      bars.abort_flag = 1u;
      ok = false;
    }
    ok = __all_sync(0xffffffffu, ok);
    l = lk = d = 0.f;
    for (int q = 0; q < p.ranks; ++q) {
      l += inbox[q][0][row];
      lk += inbox[q][1][row];
      d += inbox[q][2][row];
    }
    // dX = kept: s g + sign(x) c (1 - s); dropped: sign(x) c, c = D / Lk
    const float s = lk == 0.f ? 1.f : l / lk;
    const float dropped = lk == 0.f ? 0.f : d / lk;
    const float kept = dropped * (1.f - s);

    for (int i = 0; ok && i < tiles; ++i) {
      ok = __all_sync(0xffffffffu, back_wait(bars, &bars.full[slot], phase, p.status, kDevTimeoutFull));
      if (!ok) break;
      const uint8_t* st = ring + static_cast<uint32_t>(slot) * p.stage_bytes;
      if constexpr (LORA) {
        ok = __all_sync(0xffffffffu,
                        back_wait(bars, &bars.d_full[i & 1], (i >> 1) & 1, p.status, kDevTimeoutAccum));
        if (!ok) break;
        tc_fence_after();
      }
      ok = __all_sync(0xffffffffu, back_wait(bars, &bars.out_empty, (i & 1) ^ 1, p.status, kDevTimeoutEmpty));
      if (!ok) break;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t branch[16] = {};
        if constexpr (LORA) {
          tmem_ld_32x32b_x16(bars.tmem_base + (i & 1) * kCols + 32 * half + 16 * h + ((32u * quarter) << 16), branch);
          tmem_ld_wait();
        }
        const uint4 qv = *reinterpret_cast<const uint4*>(st + q_unit(h));
        const uint4 ga = *reinterpret_cast<const uint4*>(st + g_unit(h, 0));
        const uint4 gb = *reinterpret_cast<const uint4*>(st + g_unit(h, 1));
        const uint32_t qw[4] = {qv.x, qv.y, qv.z, qv.w};
        const uint32_t gw[8] = {ga.x, ga.y, ga.z, ga.w, gb.x, gb.y, gb.z, gb.w};
        uint32_t out[8];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          float v[4], o[4];
          bool keep[4];
          ckpt8_decode4<FMT>(qw[w], v);
          keep4(v, keep);
          const float g[4] = {bf16_lo(gw[2 * w]), bf16_hi(gw[2 * w]), bf16_lo(gw[2 * w + 1]), bf16_hi(gw[2 * w + 1])};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            o[j] = fmaf(stored_sign<FMT>(v[j]), keep[j] ? kept : dropped, __uint_as_float(branch[4 * w + j]));
            if (keep[j]) o[j] = fmaf(s, g[j], o[j]);
          }
          out[2 * w] = pack_bf16(o[0], o[1]);
          out[2 * w + 1] = pack_bf16(o[2], o[3]);
        }
        *reinterpret_cast<uint4*>(out_sm + g_unit(h, 0)) = make_uint4(out[0], out[1], out[2], out[3]);
        *reinterpret_cast<uint4*>(out_sm + g_unit(h, 1)) = make_uint4(out[4], out[5], out[6], out[7]);
      }
      if constexpr (LORA) tc_fence_before();
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&bars.empty[slot]);
        if (LORA) mbar_arrive(&bars.d_empty[i & 1]);
        mbar_arrive(&bars.done);
      }
      if (++slot == stages) slot = 0, phase ^= 1u;
    }
  }

  __syncwarp();
  tc_fence_before();
  cluster_sync_all();  // a block that gave up stays until the others no longer write to it
  if (LORA && warp == 1) {
    tc_fence_after();
    tmem_dealloc(bars.tmem_base, 128);
  }
}

// The launch of `blocks` blocks in clusters of `ranks`; with `most` the clusters
// that the device can hold at once are counted instead.
template <int FMT, bool LORA>
cudaError_t launch(const BackLaunch& b, unsigned blocks, uint32_t smem, cudaStream_t s, int* most = nullptr) {
  static std::once_flag once[64];
  static cudaError_t configured[64];
  const cudaError_t e = once_per_device(once, configured, []() {
    return cudaFuncSetAttribute(sparsify_backward_kernel<FMT, LORA>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(kSmemAlone));
  });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(b.ranks);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (most != nullptr) return cudaOccupancyMaxActiveClusters(most, sparsify_backward_kernel<FMT, LORA>, &cfg);
  return cudaLaunchKernelEx(&cfg, sparsify_backward_kernel<FMT, LORA>, b);
}

// Clusters of each size that the device holds at once, two blocks an SM or one
// (the same for every variant: shared memory decides)
struct ClusterRoom {
  int shared[kMaxCluster + 1], alone[kMaxCluster + 1];
};
const ClusterRoom* cluster_room() {
  static std::once_flag once[64];
  static cudaError_t results[64];
  static ClusterRoom rooms[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return nullptr;
  ClusterRoom& room = rooms[dev];
  const cudaError_t e = once_per_device(once, results, [&room]() {
    for (int c = 1; c <= kMaxCluster; ++c) {
      BackLaunch b = {};
      b.ranks = c;
      cudaError_t err = launch<kCkpt8Int8, true>(b, static_cast<unsigned>(c), kSmemShared, nullptr, &room.shared[c]);
      if (err == cudaSuccess)
        err = launch<kCkpt8Int8, true>(b, static_cast<unsigned>(c), kSmemAlone, nullptr, &room.alone[c]);
      if (err != cudaSuccess) return err;
    }
    return cudaSuccess;
  });
  return e == cudaSuccess ? &room : nullptr;
}

}  // namespace

cudaError_t launch_sparsify_backward(const SparsifyBackwardLaunch& p, cudaStream_t s) {
  const ClusterRoom* room = cluster_room();
  if (room == nullptr) return cudaErrorUnknown;
  BackLaunch b = {};
  b.e = static_cast<const uint8_t*>(p.e);
  b.M = p.M;
  b.K = p.K;
  b.r = p.r;
  b.stall_test = p.stall_test;
  b.status = p.status;
  const bool lora = p.dt != nullptr;
  const uint32_t fixed = 1024 + kGBytes + (lora ? static_cast<uint32_t>((p.r + 63) / 64) * kTBox : 0u);
  b.stage_bytes = kGBytes + kQBytes + 128u * static_cast<uint32_t>(p.r);
  // two blocks an SM if each then has two stages (r <= 64)
  const bool shared = fixed + 2 * b.stage_bytes <= kSmemShared;
  const uint32_t fit = ((shared ? kSmemShared : kSmemAlone) - fixed) / b.stage_bytes;
  b.stages = static_cast<int>(fit < kMaxStages ? fit : kMaxStages);
  // blocks of a row block: the cluster size with the fewest tiles one after another
  // (waves of clusters times tiles of a block)
  const int64_t row_blocks = (p.M + 127) / 128, tiles = p.K / kCols;
  int64_t best = 0;
  for (int c = 1; c <= kMaxCluster && c <= tiles; ++c) {
    const int at_once = shared ? room->shared[c] : room->alone[c];
    if (at_once < 1) continue;
    const int64_t steps = (row_blocks + at_once - 1) / at_once * ((tiles + c - 1) / c);
    if (best == 0 || steps < best) {
      best = steps;
      b.ranks = c;
    }
  }
  if (best == 0) return cudaErrorUnknown;
  b.per = static_cast<int>((tiles + b.ranks - 1) / b.ranks);
  const uint32_t smem = fixed + b.stages * b.stage_bytes;
  const uint64_t M = p.M, K = p.K, r = p.r;
  constexpr auto kSw = CU_TENSOR_MAP_SWIZZLE_128B;
  if (!encode_bf16_2d(&b.tm_g, p.g, K, M, K * 2, kCols, 128, kSw) ||
      !encode_bf16_2d(&b.tm_dx, p.dx, K, M, K * 2, kCols, 128, kSw) ||
      !encode_u8_2d(&b.tm_q, p.q, K, M, K, kCols, 128, CU_TENSOR_MAP_SWIZZLE_64B))
    return cudaErrorInvalidValue;
  if (lora && (!encode_bf16_2d(&b.tm_dt, p.dt, r, M, r * 2, 64, 128, kSw) ||
               !encode_bf16_2d(&b.tm_a, p.a, K, r, K * 2, kCols, static_cast<uint32_t>(r), kSw)))
    return cudaErrorInvalidValue;
  const unsigned blocks = static_cast<unsigned>(row_blocks * b.ranks);
  if (p.format == kCkpt8Int8)
    return lora ? launch<kCkpt8Int8, true>(b, blocks, smem, s) : launch<kCkpt8Int8, false>(b, blocks, smem, s);
  return lora ? launch<kCkpt8E4M3, true>(b, blocks, smem, s) : launch<kCkpt8E4M3, false>(b, blocks, smem, s);
}

}  // namespace lynx
