// lora_backward_kernel.cu -- the adapter's gradients from an 8-bit checkpoint
// (lynx_lora_backward):
//
//   T = x A^T,   dT = dY B,   dB = dY^T T,   dA = dT^T x.
//
// Every product has one large matrix S (x from its 8-bit form, or dY) and an
// adapter-sized one, and r is small: the time is the reading of S.  So one kernel
// streams S once, in 128 x 128 tiles, and takes from each tile in shared memory
//
//   the row product  U[rows, r] += S P      (P [cols, r])
//   the col product  V[cols, r] += S^T Q    (Q [rows, r])
//
// T is a row product of x with P = A^T, dT and dB are the row and the column
// product of one pass over dY (P = B, Q = T), dA^T a column product of x with
// Q = dT.  The same tile serves as a K-major and as an MN-major operand of
// tcgen05.mma; the accumulators (one U, one V per 128 columns) stay in TMEM.
//
// A CTA has a range of 128-row blocks and a range of 128-column blocks.  P of its
// columns stays in shared memory, U leaves after each row block and V at the end,
// as fp32 partial sums per range, which reduce_kernel adds in the order of the
// ranges and rounds: no atomics, the order is the shape's.  Partial sums lie as
// [block][column of r][128]: a TMEM lane is a row, so a warp stores 128 bytes at a
// time (with rows of r floats the 4608 x 12288 pass spent 14 of 41 us storing).
#include "lynx_ckpt8.cuh"
#include "lynx_internal.h"
#include "lynx_ptx.cuh"

namespace lynx {

namespace {

constexpr int kSrcBf16 = 2;  // beside kCkpt8Int8 and kCkpt8E4M3

constexpr uint32_t kBox = 16384;        // 128 rows x 64 bf16, 128B swizzle
constexpr uint32_t kTileBytes = 2 * kBox;  // an S tile: two boxes of 64 columns
constexpr int kMaxStages = 6;
constexpr int kConvWarps = 16;
constexpr int kAhead = 3;                // 8-bit tiles in flight
constexpr uint32_t kRawBytes = 16384;    // one of them
constexpr uint32_t kSmemMost = 227 * 1024 - 1024;  // leaves the static part 1 KB
constexpr int kPlanSms = 148;           // B200; the plan (and the workspace) go by the shape alone

struct PassPlan {
  int nb;        // column blocks of a CTA
  int rpr;       // row blocks of a CTA
  int n_cr, n_rr;  // ranges
  int stages, q_bufs, u_bufs;
  uint32_t tmem_cols;
  uint32_t smem;
};

struct PassLaunch {
  CUtensorMap tm_s;  // dY [R,C] bf16, box 64 x 128 (bf16 source)
  CUtensorMap tm_p;  // B [C,r], box 64 x 128; or A [r,C], box 64 x r (8-bit source)
  CUtensorMap tm_q;  // Q [R,r], box 64 x 128
  const uint8_t* q8;
  const uint8_t* e8;
  float* u_part;  // [n_cr][row blocks][r][128]
  float* v_part;  // [n_rr][column blocks][r][128]
  int64_t R, C;
  int r;
  PassPlan plan;
  int stall_test;
  uint32_t* status;
};

struct PassBars {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t p_full, q_full[2], q_empty[2], u_full[2], u_empty[2], done;
  uint32_t tmem_base;
  volatile uint32_t abort_flag;
};

__device__ __forceinline__ bool pass_wait(PassBars& b, uint64_t* bar, uint32_t parity, uint32_t* status,
                                          uint32_t code) {
  if (b.abort_flag) return false;
  if (mbar_wait(bar, parity)) return true;
  record_error(status, code);
  b.abort_flag = 1u;
  return false;
}

template <int SRC>
constexpr int pass_threads() {
  // TMA producer, MMA issuer, 4 epilogue warps, and the warps that widen 8-bit tiles
  return 32 * (6 + (SRC == kSrcBf16 ? 0 : kConvWarps));
}

template <int SRC, bool ROW, bool COL>
__global__ void __launch_bounds__(pass_threads<SRC>(), 1) adapter_pass_kernel(const __grid_constant__ PassLaunch p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ PassBars bars;
  uint8_t* const sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                 ~static_cast<uintptr_t>(1023));
  const uint32_t warp = warp_id_sync();
  const uint32_t lane = lane_id();
  const int r = p.r;
  const uint32_t r_boxes = static_cast<uint32_t>((r + 63) / 64);   // 64-column boxes of an [*, r] operand
  const uint32_t r_cols = static_cast<uint32_t>((r + 31) / 32) * 32;  // TMEM columns of an accumulator
  const int nb = p.plan.nb, stages = p.plan.stages;
  const int cr = static_cast<int>(blockIdx.x % p.plan.n_cr), rr = static_cast<int>(blockIdx.x / p.plan.n_cr);
  const int cb0 = cr * nb;
  const int ncb = min(nb, static_cast<int>((p.C + 127) / 128) - cb0);
  const int rb0 = rr * p.plan.rpr;
  const int nrb = min(p.plan.rpr, static_cast<int>((p.R + 127) / 128) - rb0);

  // shared memory: P | Q buffers | S stages | 8-bit tiles
  constexpr bool kPKmajor = SRC != kSrcBf16;
  const uint32_t p_block = kPKmajor ? 256u * static_cast<uint32_t>(r) : r_boxes * kBox;
  const uint32_t q_bytes = r_boxes * kBox;
  uint8_t* const sm_p = sm;
  uint8_t* const sm_q = sm_p + (ROW ? static_cast<uint32_t>(nb) * p_block : 0u);
  uint8_t* const sm_s = sm_q + (COL ? static_cast<uint32_t>(p.plan.q_bufs) * q_bytes : 0u);

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&bars.full[s], SRC == kSrcBf16 ? 1 : kConvWarps);
      mbar_init(&bars.empty[s], 1);
    }
    mbar_init(&bars.p_full, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.q_full[i], 1);
      mbar_init(&bars.q_empty[i], 1);
      mbar_init(&bars.u_full[i], 1);
      mbar_init(&bars.u_empty[i], 4);
    }
    mbar_init(&bars.done, 1);
    bars.abort_flag = 0u;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&bars.tmem_base, p.plan.tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait();

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0 && !p.stall_test) {
      bool ok = true;
      if (ROW) {
        tma_prefetch_desc(&p.tm_p);
        mbar_arrive_expect_tx(&bars.p_full, static_cast<uint32_t>(ncb) * p_block);
        for (int cb = 0; cb < ncb; ++cb) {
          uint8_t* dst = sm_p + static_cast<uint32_t>(cb) * p_block;
          const int32_t c0 = (cb0 + cb) * 128;
          if constexpr (kPKmajor) {
            for (int j = 0; j < 2; ++j)
              tma_load_2d(dst + static_cast<uint32_t>(j) * (p_block / 2), &p.tm_p, &bars.p_full, c0 + 64 * j, 0);
          } else {
            for (uint32_t b = 0; b < r_boxes; ++b)
              tma_load_2d(dst + b * kBox, &p.tm_p, &bars.p_full, static_cast<int32_t>(64 * b), c0);
          }
        }
      }
      uint32_t g = 0;
      int q_issued = 0;
      for (int rb = 0; ok && rb < nrb; ++rb) {
        const int32_t row0 = (rb0 + rb) * 128;
        if (COL) {
          const int qb = rb % p.plan.q_bufs;
          ok = pass_wait(bars, &bars.q_empty[qb], ((rb / p.plan.q_bufs) & 1) ^ 1, p.status, kDevTimeoutEmpty);
          if (!ok) break;
          mbar_arrive_expect_tx(&bars.q_full[qb], q_bytes);
          for (uint32_t b = 0; b < r_boxes; ++b)
            tma_load_2d(sm_q + static_cast<uint32_t>(qb) * q_bytes + b * kBox, &p.tm_q, &bars.q_full[qb],
                        static_cast<int32_t>(64 * b), row0);
          q_issued = rb + 1;
        }
        if constexpr (SRC == kSrcBf16) {
          for (int cb = 0; cb < ncb; ++cb, ++g) {
            const uint32_t slot = g % stages;
            ok = pass_wait(bars, &bars.empty[slot], ((g / stages) & 1u) ^ 1u, p.status, kDevTimeoutEmpty);
            if (!ok) break;
            uint8_t* dst = sm_s + slot * kTileBytes;
            mbar_arrive_expect_tx(&bars.full[slot], kTileBytes);
            tma_load_2d(dst, &p.tm_s, &bars.full[slot], (cb0 + cb) * 128, row0);
            tma_load_2d(dst + kBox, &p.tm_s, &bars.full[slot], (cb0 + cb) * 128 + 64, row0);
          }
        }
      }
      // the last fill of every buffer must have landed before the block exits
      bool drained = true;
      if (ROW) drained = mbar_wait(&bars.p_full, 0, kWaitLimitNs / 4);
      for (int x = q_issued - 1; x >= 0 && x >= q_issued - p.plan.q_bufs; --x)
        drained &= mbar_wait(&bars.q_full[x % p.plan.q_bufs], (x / p.plan.q_bufs) & 1, kWaitLimitNs / 4);
      for (uint32_t b = g; b > 0 && b + stages > g; --b)
        drained &= mbar_wait(&bars.full[(b - 1) % stages], ((b - 1) / stages) & 1u, kWaitLimitNs / 4);
      if (!drained) record_error(p.status, kDevTimeoutDrain);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    // The whole warp walks the loop and one elected lane issues, so that the
    // descriptors stay in warp-uniform registers (issued by a lone lane, a tile's
    // 16 MMAs took 1400 cycles, more than the tile's bytes).
    const uint32_t idesc_row = make_idesc_bf16(128, r, false) | (kPKmajor ? 0u : kIdescBMnMajor);
    const uint32_t idesc_col = make_idesc_bf16(128, r, false) | kIdescAMnMajor | kIdescBMnMajor;
    const uint32_t t_u = bars.tmem_base;
    const uint32_t t_v = t_u + (ROW ? static_cast<uint32_t>(p.plan.u_bufs) * r_cols : 0u);
    auto arrived = [&](uint64_t* bar, uint32_t parity, uint32_t code) {
      return __all_sync(0xffffffffu, pass_wait(bars, bar, parity, p.status, code)) != 0;
    };
    bool ok = !ROW || arrived(&bars.p_full, 0, kDevTimeoutFull);
    uint32_t slot = 0, phase = 0;
    for (int rb = 0; ok && rb < nrb; ++rb) {
      const int qb = COL ? rb % p.plan.q_bufs : 0, ub = ROW ? rb % p.plan.u_bufs : 0;
      if (COL) ok = arrived(&bars.q_full[qb], (rb / p.plan.q_bufs) & 1, kDevTimeoutFull);
      if (ok && ROW) ok = arrived(&bars.u_empty[ub], ((rb / p.plan.u_bufs) & 1) ^ 1, kDevTimeoutAccum);
      if (!ok) break;
      const uint32_t sq = smem_u32(sm_q) + static_cast<uint32_t>(qb) * q_bytes;
      const uint32_t d_u = t_u + static_cast<uint32_t>(ub) * r_cols;
      for (int cb = 0; cb < ncb; ++cb) {
        ok = arrived(&bars.full[slot], phase, kDevTimeoutFull);
        if (!ok) break;
        tc_fence_after();
        const uint32_t ss = smem_u32(sm_s) + slot * kTileBytes;
        if constexpr (ROW) {  // 16 columns of S a step
          const uint32_t sp = smem_u32(sm_p) + static_cast<uint32_t>(cb) * p_block;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const uint64_t da = make_sdesc(ss + (k / 4) * kBox + (k % 4) * 32, 16, 1024, kSw128);
            const uint64_t db = kPKmajor ? make_sdesc(sp + (k / 4) * (p_block / 2) + (k % 4) * 32, 16, 1024, kSw128)
                                         : make_sdesc(sp + k * 2048, kBox, 1024, kSw128);
            if (elect_one()) mma_bf16(d_u, da, db, idesc_row, (cb | k) != 0);
            __syncwarp();
          }
        }
        if constexpr (COL) {  // 16 rows of S a step
          const uint32_t d_v = t_v + static_cast<uint32_t>(cb) * r_cols;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const uint64_t da = make_sdesc(ss + k * 2048, kBox, 1024, kSw128);
            const uint64_t db = make_sdesc(sq + k * 2048, kBox, 1024, kSw128);
            if (elect_one()) mma_bf16(d_v, da, db, idesc_col, (rb | k) != 0);
            __syncwarp();
          }
        }
        if (elect_one()) tc_commit(&bars.empty[slot]);
        __syncwarp();
        if (++slot == static_cast<uint32_t>(stages)) slot = 0, phase ^= 1u;
      }
      if (!ok) break;
      if (elect_one()) {
        if (COL) tc_commit(&bars.q_empty[qb]);
        if (ROW) tc_commit(&bars.u_full[ub]);
      }
      __syncwarp();
    }
    if (elect_one()) tc_commit(&bars.done);
    __syncwarp();
    if (!mbar_wait(&bars.done, 0) && lane == 0) record_error(p.status, kDevTimeoutDrain);
    __syncwarp();
  } else if (warp < 6) {
    // ------------------------------------------------------------ epilogue: partial sums out
    const uint32_t quarter = warp & 3u;  // the TMEM lanes this warp may read
    const uint32_t t_lane = (32u * quarter) << 16;
    bool ok = true;
    auto store = [&](uint32_t taddr, float* part, int64_t block) {
      float* dst = part + block * r * 128 + 32 * quarter + lane;
      for (int c = 0; c < r; c += 16) {
        uint32_t v[16];
        tmem_ld_32x32b_x16(taddr + t_lane + static_cast<uint32_t>(c), v);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i) dst[(c + i) * 128] = __uint_as_float(v[i]);
      }
    };
    if constexpr (ROW) {
      for (int rb = 0; rb < nrb; ++rb) {
        const int ub = rb % p.plan.u_bufs;
        ok = pass_wait(bars, &bars.u_full[ub], (rb / p.plan.u_bufs) & 1, p.status, kDevTimeoutAccum);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        store(bars.tmem_base + static_cast<uint32_t>(ub) * r_cols, p.u_part, cr * ((p.R + 127) / 128) + rb0 + rb);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.u_empty[ub]);
      }
    }
    if constexpr (COL) {
      ok = ok && pass_wait(bars, &bars.done, 0, p.status, kDevTimeoutAccum);
      ok = __all_sync(0xffffffffu, ok && !bars.abort_flag);
      if (ok) {
        tc_fence_after();
        const uint32_t t_v = bars.tmem_base + (ROW ? static_cast<uint32_t>(p.plan.u_bufs) * r_cols : 0u);
        for (int cb = 0; cb < ncb; ++cb)
          store(t_v + static_cast<uint32_t>(cb) * r_cols, p.v_part, rr * ((p.C + 127) / 128) + cb0 + cb);
        tc_fence_before();
      }
    }
  } else if constexpr (SRC != kSrcBf16) {
    // ------------------------------------------------------------ 8 bits -> bf16 tiles
    // 16 bytes (half a block) a step: 8 lanes cover a row of the tile, a thread
    // takes rows t / 8 + kRowStep i.  The bytes arrive by cp.async in slots that
    // only this thread reads, kAhead tiles before they are needed; the exponents
    // (one byte per 32) come through registers, two tiles ahead.
    constexpr int kSteps = 4 * 8 / kConvWarps;
    constexpr int kRowStep = 4 * kConvWarps;
    const uint32_t t = threadIdx.x - 192u;
    const uint32_t chunk = t & 7u;
    const uint32_t row_t = t >> 3;
    const int tiles = p.stall_test ? 0 : nrb * ncb;
    const int64_t row0 = static_cast<int64_t>(rb0) * 128 + row_t;
    const int rows0 = static_cast<int>(p.R - row0);                                      // rows left at the first tile
    const int cols0 = static_cast<int>(p.C - static_cast<int64_t>(cb0) * 128) - 16 * static_cast<int>(chunk);
    const int64_t e_pitch = p.C / 32;
    // This thread's place in the tile that is asked for next, bytes and exponents:
    // tiles are taken along the columns, then down
    const uint8_t* q_at = p.q8 + row0 * p.C + static_cast<int64_t>(cb0) * 128 + 16 * chunk;
    const uint8_t* e_at = p.e8 + row0 * e_pitch + static_cast<int64_t>(cb0) * 4 + chunk / 2;
    const int64_t q_down = 128 * p.C - 128 * (ncb - 1), e_down = 128 * e_pitch - 4 * (ncb - 1);
    int q_cb = 0, q_rows = rows0, q_left = tiles, e_cb = 0, e_rows = rows0, e_left = tiles;
    const uint32_t raw = smem_u32(sm_s) + static_cast<uint32_t>(stages) * kTileBytes + 16u * t;
    uint32_t fetch_at = 0, take_at = 0;  // byte offsets of the slots
    auto fetch = [&]() {
      if (q_left > 0) {
        const bool col_in = 128 * q_cb < cols0;
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          const bool in = col_in && kRowStep * i < q_rows;
          cp_async_16(raw + fetch_at + (kRawBytes / kSteps) * i, in ? q_at + i * kRowStep * p.C : p.q8, in ? 16u : 0u);
        }
        --q_left;
        if (++q_cb < ncb) {
          q_at += 128;
        } else {
          q_cb = 0;
          q_at += q_down;
          q_rows -= 128;
        }
        fetch_at = fetch_at == kAhead * kRawBytes ? 0u : fetch_at + kRawBytes;
      }
      cp_async_commit();
    };
    auto exponents = [&](uint32_t (&ex)[kSteps]) {
      if (e_left > 0) {
        const bool col_in = 128 * e_cb < cols0;
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
          ex[i] = col_in && kRowStep * i < e_rows ? __ldg(e_at + i * kRowStep * e_pitch) : 0u;
        --e_left;
        if (++e_cb < ncb) {
          e_at += 4;
        } else {
          e_cb = 0;
          e_at += e_down;
          e_rows -= 128;
        }
      }
    };
    const uint32_t x = row_t & 7u, u = (chunk & 3u) * 2u;  // kRowStep is a multiple of 8
    const uint32_t line = smem_u32(sm_s) + (chunk >> 2) * kBox + row_t * 128u;
    const uint32_t line0 = line + ((u ^ x) << 4), line1 = line + (((u + 1u) ^ x) << 4);
    uint32_t slot = 0, phase = 1;
    bool ok = true;
    auto widen = [&](const uint32_t (&ex)[kSteps]) {
      cp_async_wait<kAhead - 1>();  // this tile's bytes are here
      uint2 out[kSteps][4];
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const uint32_t f = ckpt8_factor_bits<SRC>(ex[i]);
        const uint4 w = ld_shared_v4(raw + take_at + (kRawBytes / kSteps) * i);
        out[i][0] = ckpt8_widen4<SRC>(w.x, f);
        out[i][1] = ckpt8_widen4<SRC>(w.y, f);
        out[i][2] = ckpt8_widen4<SRC>(w.z, f);
        out[i][3] = ckpt8_widen4<SRC>(w.w, f);
      }
      take_at = take_at == kAhead * kRawBytes ? 0u : take_at + kRawBytes;
      fetch();
      ok = __all_sync(0xffffffffu, pass_wait(bars, &bars.empty[slot], phase, p.status, kDevTimeoutEmpty));
      if (!ok) return;
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const uint32_t at = slot * kTileBytes + static_cast<uint32_t>(i) * kRowStep * 128u;
        st_shared_v4(line0 + at, make_uint4(out[i][0].x, out[i][0].y, out[i][1].x, out[i][1].y));
        st_shared_v4(line1 + at, make_uint4(out[i][2].x, out[i][2].y, out[i][3].x, out[i][3].y));
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.full[slot]);
      if (++slot == static_cast<uint32_t>(stages)) slot = 0, phase ^= 1u;
    };
    for (int i = 0; i < kAhead; ++i) fetch();
    uint32_t ex0[kSteps] = {}, ex1[kSteps] = {}, now[kSteps];
    exponents(ex0);
    exponents(ex1);
    for (int tile = 0; ok && tile < tiles; tile += 2) {
#pragma unroll
      for (int i = 0; i < kSteps; ++i) now[i] = ex0[i];
      exponents(ex0);
      widen(now);
      if (!ok || tile + 1 >= tiles) break;
#pragma unroll
      for (int i = 0; i < kSteps; ++i) now[i] = ex1[i];
      exponents(ex1);
      widen(now);
    }
    cp_async_wait<0>();
  }

  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(bars.tmem_base, p.plan.tmem_cols);
  }
}

// ---------------------------------------------------------------------------
// the ranges' partial sums, added in order and rounded

struct ReduceJob {
  const float* part;   // [n][blocks][r][128]
  __nv_bfloat16* out;  // [rows][r], or [r][rows] (transposed)
  int64_t rows;
  int n, r;
};

constexpr int kRedThreads = 256;

// A block of threads takes one 128-row block x 16 columns; a warp a column at a
// time, 4 rows a lane.  The first a_blocks take job a, the rest job b.
template <bool TRANSPOSED>
__global__ void __launch_bounds__(kRedThreads) reduce_kernel(ReduceJob a, ReduceJob b, unsigned a_blocks) {
  __shared__ float tile[16][128 + 4];
  pdl_wait();
  const bool first = blockIdx.x < a_blocks;
  const ReduceJob& j = first ? a : b;
  const unsigned id = blockIdx.x - (first ? 0u : a_blocks);
  const unsigned groups = static_cast<unsigned>(j.r) / 16;
  const int64_t block = id / groups;
  const int c0 = static_cast<int>(id % groups) * 16;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t stride = (j.rows + 127) / 128 * j.r * 128;
  const float* src = j.part + (block * j.r + c0 + warp) * 128 + 4 * lane;
  float4 s0 = make_float4(0.f, 0.f, 0.f, 0.f), s1 = s0;
#pragma unroll 4
  for (int i = 0; i < j.n; ++i) {
    const float4 v = __ldcg(reinterpret_cast<const float4*>(src + i * stride));
    const float4 w = __ldcg(reinterpret_cast<const float4*>(src + i * stride + 8 * 128));
    s0.x += v.x, s0.y += v.y, s0.z += v.z, s0.w += v.w;
    s1.x += w.x, s1.y += w.y, s1.z += w.z, s1.w += w.w;
  }
  if constexpr (TRANSPOSED) {
    const int64_t row = block * 128 + 4 * lane;  // rows is a multiple of 64
    if (row < j.rows) {
      __nv_bfloat16* dst = j.out + (c0 + warp) * j.rows + row;
      *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16(s0.x, s0.y), pack_bf16(s0.z, s0.w));
      *reinterpret_cast<uint2*>(dst + 8 * j.rows) = make_uint2(pack_bf16(s1.x, s1.y), pack_bf16(s1.z, s1.w));
    }
  } else {
    *reinterpret_cast<float4*>(&tile[warp][4 * lane]) = s0;
    *reinterpret_cast<float4*>(&tile[warp + 8][4 * lane]) = s1;
    __syncthreads();
    const int row = threadIdx.x >> 1, c = (threadIdx.x & 1) * 8;
    if (block * 128 + row < j.rows) {
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = pack_bf16(tile[c + 2 * i][row], tile[c + 2 * i + 1][row]);
      *reinterpret_cast<uint4*>(j.out + (block * 128 + row) * j.r + c0 + c) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

// ---------------------------------------------------------------------------
// host side

// The ranges of one pass.  A CTA's columns are bounded by shared memory (their P
// stays there) and TMEM (their V); of the column counts that fit, the one with
// the least of (tiles of the busiest CTA + partial sums written and read back)
// is taken, both as bytes over the rate they move at.
PassPlan plan_pass(int64_t R, int64_t C, int r, bool row, bool col, bool eight) {
  const int64_t rb = (R + 127) / 128, cb = (C + 127) / 128;
  const uint32_t rp = static_cast<uint32_t>((r + 63) / 64) * 64, rc = static_cast<uint32_t>((r + 31) / 32) * 32;
  // 1 KB of the dynamic part goes into its alignment
  const uint32_t raw = eight ? (kAhead + 1) * kRawBytes : 0u;
  const uint32_t p_block = row ? 256u * (eight ? static_cast<uint32_t>(r) : rp) : 0u;
  const uint32_t q_one = col ? 256u * rp : 0u;
  const int min_stages = eight ? 2 : 3;
  PassPlan best = {};
  double best_cost = 0;
  for (int nb = 1; nb <= 16 && nb <= cb; ++nb) {
    const uint32_t v_cols = col ? nb * rc : 0u;
    int u_bufs = row ? 2 : 0;
    if (v_cols + u_bufs * rc > 512) u_bufs = row ? 1 : 0;
    if (v_cols + u_bufs * rc > 512) break;
    int q_bufs = col ? 2 : 0;
    if (nb * p_block + q_bufs * q_one + min_stages * kTileBytes + raw + 1024 > kSmemMost) q_bufs = col ? 1 : 0;
    if (nb * p_block + q_bufs * q_one + min_stages * kTileBytes + raw + 1024 > kSmemMost) break;
    PassPlan c = {};
    c.nb = nb;
    c.n_cr = static_cast<int>((cb + nb - 1) / nb);
    int64_t n_rr = kPlanSms / c.n_cr;
    n_rr = n_rr < 1 ? 1 : (n_rr > rb ? rb : n_rr);
    c.rpr = static_cast<int>((rb + n_rr - 1) / n_rr);
    c.n_rr = static_cast<int>((rb + c.rpr - 1) / c.rpr);
    c.q_bufs = q_bufs;
    c.u_bufs = u_bufs;
    uint32_t cols = 32;
    while (cols < v_cols + u_bufs * rc) cols *= 2;
    c.tmem_cols = cols;
    const uint32_t fixed = nb * p_block + q_bufs * q_one + raw;
    const int stages = static_cast<int>((kSmemMost - 1024 - fixed) / kTileBytes);
    const int most = eight ? 3 : kMaxStages;
    c.stages = stages > most ? most : stages;
    c.smem = fixed + c.stages * kTileBytes + 1024;
    const double waves = static_cast<double>((static_cast<int64_t>(c.n_cr) * c.n_rr + kPlanSms - 1) / kPlanSms);
    const double cost = waves * c.rpr * nb * (eight ? 16384.0 : 32768.0) * kPlanSms / 6.0e12 +
                        2.0 * 4 * r * (row ? static_cast<double>(c.n_cr) * R : 0.0) / 6.0e12 +
                        2.0 * 4 * r * (col ? static_cast<double>(c.n_rr) * C : 0.0) / 6.0e12;
    if (best.nb == 0 || cost < best_cost) {
      best = c;
      best_cost = cost;
    }
  }
  return best;
}

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

struct LoraPlan {
  PassPlan down, dy, up;  // T; dT and dB; dA
  size_t t, dt, u, v, total;
};

LoraPlan plan_lora(int64_t M, int64_t N, int64_t K, int r) {
  LoraPlan l;
  l.down = plan_pass(M, K, r, true, false, true);
  l.dy = plan_pass(M, N, r, true, true, false);
  l.up = plan_pass(M, K, r, false, true, true);
  const size_t mr = static_cast<size_t>(M) * r;
  auto part = [r](int64_t rows, int n) { return static_cast<size_t>((rows + 127) / 128) * 512 * r * n; };
  const size_t u = part(M, l.down.n_cr > l.dy.n_cr ? l.down.n_cr : l.dy.n_cr);
  const size_t v_dy = part(N, l.dy.n_rr), v_up = part(K, l.up.n_rr);
  l.t = 0;
  l.dt = align256(l.t + mr * 2);
  l.u = align256(l.dt + mr * 2);
  l.v = align256(l.u + u);
  l.total = align256(l.v + (v_dy > v_up ? v_dy : v_up));
  return l;
}

template <int SRC, bool ROW, bool COL>
cudaError_t launch_pass(const PassLaunch& p, cudaStream_t s) {
  static std::once_flag once[64];
  static cudaError_t configured[64];
  const cudaError_t e = once_per_device(once, configured, []() {
    return cudaFuncSetAttribute(adapter_pass_kernel<SRC, ROW, COL>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(kSmemMost));
  });
  if (e != cudaSuccess) return e;
  return launch_after_previous(adapter_pass_kernel<SRC, ROW, COL>,
                               dim3(static_cast<unsigned>(p.plan.n_cr) * static_cast<unsigned>(p.plan.n_rr)),
                               dim3(pass_threads<SRC>()), p.plan.smem, s, p);
}

unsigned reduce_blocks(const ReduceJob& j) {
  return static_cast<unsigned>((j.rows + 127) / 128) * static_cast<unsigned>(j.r / 16);
}

template <bool TRANSPOSED>
cudaError_t launch_reduce(const ReduceJob& a, const ReduceJob& b, cudaStream_t s) {
  const unsigned na = reduce_blocks(a);
  return launch_after_previous(reduce_kernel<TRANSPOSED>, dim3(na + (b.rows > 0 ? reduce_blocks(b) : 0u)),
                               dim3(kRedThreads), 0, s, a, b, na);
}

template <int FMT>
cudaError_t run(const LoraBackwardLaunch& l, cudaStream_t s) {
  const LoraPlan plan = plan_lora(l.M, l.N, l.K, l.r);
  const uint64_t M = l.M, N = l.N, K = l.K, r = l.r;
  auto* t = reinterpret_cast<__nv_bfloat16*>(l.ws + plan.t);
  auto* dt = l.dt != nullptr ? static_cast<__nv_bfloat16*>(l.dt) : reinterpret_cast<__nv_bfloat16*>(l.ws + plan.dt);
  const ReduceJob none = {};
  PassLaunch p = {};
  p.q8 = static_cast<const uint8_t*>(l.q);
  p.e8 = static_cast<const uint8_t*>(l.e);
  p.u_part = reinterpret_cast<float*>(l.ws + plan.u);
  p.v_part = reinterpret_cast<float*>(l.ws + plan.v);
  p.R = l.M;
  p.r = l.r;
  p.stall_test = l.stall_test;
  p.status = l.status;
  constexpr auto kSw = CU_TENSOR_MAP_SWIZZLE_128B;

  // T = x A^T
  PassLaunch down = p;
  down.C = l.K;
  down.plan = plan.down;
  if (!encode_bf16_2d(&down.tm_p, l.a, K, r, K * 2, 64, static_cast<uint32_t>(r), kSw)) return cudaErrorInvalidValue;
  cudaError_t e = launch_pass<FMT, true, false>(down, s);
  if (e != cudaSuccess) return e;
  e = launch_reduce<false>(ReduceJob{p.u_part, t, l.M, plan.down.n_cr, l.r}, none, s);
  if (e != cudaSuccess) return e;

  // dT = dY B and dB = dY^T T
  PassLaunch dy = p;
  dy.C = l.N;
  dy.plan = plan.dy;
  if (!encode_bf16_2d(&dy.tm_s, l.dy, N, M, N * 2, 64, 128, kSw) ||
      !encode_bf16_2d(&dy.tm_p, l.b, r, N, r * 2, 64, 128, kSw) ||
      !encode_bf16_2d(&dy.tm_q, t, r, M, r * 2, 64, 128, kSw))
    return cudaErrorInvalidValue;
  e = launch_pass<kSrcBf16, true, true>(dy, s);
  if (e != cudaSuccess) return e;
  e = launch_reduce<false>(ReduceJob{p.u_part, dt, l.M, plan.dy.n_cr, l.r},
                    ReduceJob{p.v_part, static_cast<__nv_bfloat16*>(l.db), l.N, plan.dy.n_rr, l.r}, s);
  if (e != cudaSuccess) return e;

  // dA^T = x^T dT
  PassLaunch up = p;
  up.C = l.K;
  up.plan = plan.up;
  if (!encode_bf16_2d(&up.tm_q, dt, r, M, r * 2, 64, 128, kSw)) return cudaErrorInvalidValue;
  e = launch_pass<FMT, false, true>(up, s);
  if (e != cudaSuccess) return e;
  return launch_reduce<true>(ReduceJob{p.v_part, static_cast<__nv_bfloat16*>(l.da), l.K, plan.up.n_rr, l.r}, none, s);
}

}  // namespace

size_t lora_backward_workspace(int64_t M, int64_t N, int64_t K, int64_t r) {
  return plan_lora(M, N, K, static_cast<int>(r)).total;
}

cudaError_t launch_lora_backward(const LoraBackwardLaunch& p, cudaStream_t s) {
  return p.format == kCkpt8Int8 ? run<kCkpt8Int8>(p, s) : run<kCkpt8E4M3>(p, s);
}

}  // namespace lynx
