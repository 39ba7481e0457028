// sparsify_backward_kernel.cu -- the gradient through S(X) at an 8-bit
// checkpoint (lynx_sparsify_backward).
//
// S(X) = s m x with s = L / Lk, L = sum|x|, Lk = sum m|x| of the row.  With the
// selection m fixed, dL/dx_k = s m_k g_k + D ds/dx_k, D = sum_j m_j g_j x_j, and
// ds/dx_k = sign(x_k) / Lk - m_k sign(x_k) L / Lk^2 = sign(x_k) (1 - s m_k) / Lk.
// The LoRA branch adds dT A, a product of rank r.
//
// The selection m is the forward pass's where its metadata is given (META): the 8-bit
// values tie where x did not, and a selection made again from them differs in 3 to 12 %
// of the groups (heavy-tailed and GELU inputs).  The metadata adds 1/8 byte a value to
// each reading (4608 x 12288, rank 64: 90 us for 87).  Without it m is the 2:4 selection
// of the checkpoint's values.
//
// Every output needs its row's three sums, so there are two passes over G and
// the checkpoint: row_sums_kernel streams them once, sparsify_backward_kernel
// takes 128 x 64 tiles in the opposite order (the rows read last are still in
// L2), adds dT A from tcgen05.mma and writes dX.  (One kernel over clusters that
// kept a row block between the two passes measured 118 us at 4608 x 12288: the
// rows in flight are more than L2 holds, and the exchange stalls the loads.  The two
// passes over a quarter of the rows at a time, so that L2 holds them between, took
// 111 us: every launch starts and drains anew.)
//
// At 4608 x 12288, rank 64, 87 us: row sums 38 us and outputs 55 us, 6 us of them
// side by side (90 us with the metadata, the sums 42).  They read G and the bytes twice
// and write dX, 458 MB, a quarter of the second reading out of L2: 4.8 and 4.3 TB/s from
// memory with the integer pipe half busy.  What stalls them is not found: neither fewer
// instructions (sums), missing stores (outputs) nor more loads in flight (both) change
// the time much.
#include "lynx_ckpt8.cuh"
#include "lynx_internal.h"
#include "lynx_ptx.cuh"

namespace lynx {

namespace {

// The bits that at least two of a, b and not c have
__device__ __forceinline__ uint32_t two_of_three(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xD4;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}

template <uint32_t SEL>
__device__ __forceinline__ uint32_t prmt(uint32_t a) {
  uint32_t r;
  asm("prmt.b32 %0, %1, 0, %2;" : "=r"(r) : "r"(a), "n"(SEL));
  return r;
}

// Magnitudes of 4 stored values as bytes of 0..127 that order as they do
template <int FMT>
__device__ __forceinline__ uint32_t magnitudes(uint32_t q) {
  if constexpr (FMT == kCkpt8Int8) {
    const uint32_t sign = prmt<0xBA98>(q);  // the sign bit over each byte
    return (q ^ sign) + (sign & 0x01010101u);
  } else {
    return q & 0x7F7F7F7Fu;
  }
}

// Bit 7 of byte i: value i is one of the two largest magnitudes of 4, ties to the lower
// position: it is kept if it goes before at least two of the others.  Byte i of `next`
// says a_i goes before a_(i+1), of `over` before a_(i+2), indices modulo 4: a_i + 128 -
// a_j has bit 7 set where a_i >= a_j, and with 127 where a_i > a_j, which is what a
// higher position needs.  No byte borrows from its neighbour.  (Six fp32 differences a
// group of 4 took 61 us for 55 in the outputs' kernel at 4608 x 12288.)
__device__ __forceinline__ uint32_t keep_bits(uint32_t a) {
  const uint32_t next = a + 0x7F808080u - prmt<0x0321>(a);
  const uint32_t over = a + 0x7F7F8080u - prmt<0x1032>(a);
  return two_of_three(next, over, prmt<0x2103>(next));
}

// The same bits from the metadata, for word w of 16 values: a nibble lo | hi << 2 a word
__device__ __forceinline__ uint32_t kept_bits(uint32_t nibbles, int w) {
  const uint32_t n = nibbles >> (4 * w);
  return (0x80u << ((n & 3u) << 3)) | (0x80u << ((n & 12u) << 1));
}

// Where the 16 bits of a row's first 16 values lie in its row block's metadata; those of
// 16-value unit i are meta_unit(i) behind it (the operand layout of tcgen05.mma.sp)
__device__ __forceinline__ uint32_t meta_row(uint32_t row) {
  return ((row & 7u) + 16u * (row >> 4)) * 16u + ((row >> 3) & 1u) * 2u;
}
__device__ __forceinline__ int64_t meta_unit(int i) {
  return static_cast<int64_t>(i >> 3) * kMetaBlockBytes + (i & 1) * 128 + ((i >> 1) & 3) * 4;
}

// ---------------------------------------------------------------------------
// row sums

constexpr int kRowThreads = 256;
constexpr int kRowWarps = kRowThreads / 32;
constexpr int kAhead = 2;  // steps in flight (3, with a quarter fewer blocks an SM, took 49 us for 38)

// 16 values: sums of |x|, of the kept |x| and of the kept g x, before the factor
template <int FMT, bool META>
__device__ __forceinline__ void sums16(const uint4& qv, const uint4& ga, const uint4& gb, uint32_t nibbles, float& bl,
                                       float& bk, float& bd) {
  const uint32_t qw[4] = {qv.x, qv.y, qv.z, qv.w};
  const uint32_t gw[8] = {ga.x, ga.y, ga.z, ga.w, gb.x, gb.y, gb.z, gb.w};
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const uint32_t keep = META ? kept_bits(nibbles, w) : keep_bits(magnitudes<FMT>(qw[w]));
    float v[4];
    ckpt8_decode4<FMT>(qw[w], v);
    const float g[4] = {bf16_lo(gw[2 * w]), bf16_hi(gw[2 * w]), bf16_lo(gw[2 * w + 1]), bf16_hi(gw[2 * w + 1])};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      bl += fabsf(v[j]);
      if (keep & (0x80u << 8 * j)) {
        bk += fabsf(v[j]);
        bd = fmaf(g[j], v[j], bd);
      }
    }
  }
}

// 2^-n, 0 below the normal range
__device__ __forceinline__ float exp2_down(int n) {
  return __uint_as_float(n < 127 ? static_cast<uint32_t>(127 - n) << 23 : 0u);
}

// A row's three sums in units of 2^top, top the largest block exponent so far.  Only their
// ratios are wanted, and in absolute terms fp32 holds neither a row near 2^124 (L is
// infinite) nor one near 2^-130 (D is 0).
struct RowSums {
  float l, lk, d;
  int top;
  __device__ __forceinline__ void raise(int to) {  // to >= top
    const float f = exp2_down(to - top);
    l *= f;
    lk *= f;
    d *= f;
    top = to;
  }
};

// coef[m] = (s, D / Lk).  A block has `rows` rows, kRowWarps / rows warps each;
// 16 columns a lane and step.
template <int FMT, bool META>
__global__ void __launch_bounds__(kRowThreads, 4) row_sums_kernel(SparsifyBackwardLaunch p, int rows) {
  __shared__ RowSums part[kRowWarps];
  pdl_wait();
  pdl_launch_dependents();  // the outputs' loads may start beside this, once all earlier work is done
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ways = kRowWarps / rows, way = warp % ways;
  const int64_t m = static_cast<int64_t>(blockIdx.x) * rows + warp / ways;
  RowSums s = {0.f, 0.f, 0.f, 0};
  if (m < p.M) {
    const auto* q = static_cast<const uint4*>(p.q) + m * p.K / 16;
    const auto* e = static_cast<const uint8_t*>(p.e) + m * p.K / 32;
    const auto* g = static_cast<const uint4*>(p.g) + m * p.K / 8;
    const uint8_t* meta = nullptr;
    if (META)
      meta = static_cast<const uint8_t*>(p.meta) + (m / kRowBlock) * ((p.K + 127) / 128) * kMetaBlockBytes +
             meta_row(static_cast<uint32_t>(m % kRowBlock));
    const int n = static_cast<int>(p.K / 16), step = 32 * ways;
    uint4 qv[kAhead], ga[kAhead], gb[kAhead];
    uint32_t ev[kAhead], nv[kAhead] = {};
    auto load = [&](int k, int i) {
      if (i < n) {
        qv[k] = __ldg(q + i);
        ga[k] = __ldg(g + 2 * i);
        gb[k] = __ldg(g + 2 * i + 1);
        ev[k] = __ldg(e + i / 2);
        if (META) nv[k] = __ldg(reinterpret_cast<const uint16_t*>(meta + meta_unit(i)));
      }
    };
    int i = 32 * way + lane;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) load(k, i + k * step);
    while (i < n) {
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        if (i < n) {
          const uint4 q0 = qv[k], a0 = ga[k], b0 = gb[k];
          const uint32_t n0 = nv[k];
          const int ex = static_cast<int>(ev[k]);  // 255: NaN throughout
          if (ex > s.top && ex < 255) s.raise(ex);
          const float f = ex < 255 ? exp2_down(s.top - ex) : __uint_as_float(0x7FC00000u);
          load(k, i + kAhead * step);
          float bl = 0.f, bk = 0.f, bd = 0.f;
          sums16<FMT, META>(q0, a0, b0, n0, bl, bk, bd);
          s.l = fmaf(bl, f, s.l);
          s.lk = fmaf(bk, f, s.lk);
          s.d = fmaf(bd, f, s.d);
          i += step;
        }
      }
    }
  }
  s.raise(__reduce_max_sync(0xffffffffu, s.top));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s.l += __shfl_xor_sync(0xffffffffu, s.l, o);
    s.lk += __shfl_xor_sync(0xffffffffu, s.lk, o);
    s.d += __shfl_xor_sync(0xffffffffu, s.d, o);
  }
  if (lane == 0) part[warp] = s;
  __syncthreads();
  if (way == 0 && lane == 0 && m < p.M) {
    for (int w = warp + 1; w < warp + ways; ++w) {
      RowSums other = part[w];
      if (other.top > s.top) s.raise(other.top);
      other.raise(s.top);
      s.l += other.l;
      s.lk += other.lk;
      s.d += other.d;
    }
    p.coef[m] = s.lk == 0.f ? make_float2(1.f, 0.f) : make_float2(s.l / s.lk, s.d / s.lk);
  }
}

// ---------------------------------------------------------------------------
// outputs
//   warp 0   TMA: G, the stored bytes and A's rows of a tile
//   warp 1   the MMAs
//   warps 2, 3  TMA stores of dX
//   warps 4-19  two groups of 8 that take the tiles in turn; a thread has one row
//               (a TMEM lane) and 32 columns.  Selection and sign need no
//               exponents, which the row coefficients have seen.

constexpr int kGroups = 2;
constexpr int kGroupWarps = 8;
constexpr int kRoleWarps = 2 + kGroups;
constexpr int kOutWarps = kGroups * kGroupWarps;
constexpr int kThreads = 32 * (kRoleWarps + kOutWarps);
constexpr int kCols = 64;
constexpr uint32_t kTmemCols = kGroups <= 2 ? 128 : 256;
constexpr int kMaxStages = 6;
constexpr uint32_t kGBytes = 128 * 128;  // 128 rows x 64 bf16, 128B swizzle
constexpr uint32_t kQBytes = 128 * 64;   // 128 rows x 64 bytes, 64B swizzle
constexpr uint32_t kTBox = 128 * 128;    // dT: 128 rows x 64 of r
constexpr uint32_t kSmemMost = 222 * 1024;

struct BackLaunch {
  CUtensorMap tm_g;   // G [M,K], box 64 x 128
  CUtensorMap tm_q;   // q [M,K] bytes, box 64 x 128, 64B swizzle
  CUtensorMap tm_dt;  // dT [M,r], box 64 x 128
  CUtensorMap tm_a;   // A [r,K], box 64 x r
  CUtensorMap tm_dx;  // dX [M,K], box 64 x 128
  const float2* coef;
  const uint8_t* meta;  // the selection (META)
  int64_t M, K;
  int r;
  int ranges;         // blocks of a row block
  int per;            // tiles of a block
  int stages;
  uint32_t stage_bytes;
  int stall_test;
  uint32_t* status;
};

struct BackBars {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t dt_full, mma_done, d_full[kGroups], d_empty[kGroups], done[kGroups], out_empty[kGroups];
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

template <int FMT, bool LORA, bool META>
__global__ void __launch_bounds__(kThreads, 1) sparsify_backward_kernel(const __grid_constant__ BackLaunch p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ BackBars bars;
  uint8_t* const sm = smem_raw + ((0u - smem_u32(smem_raw)) & 1023u);
  const uint32_t warp = warp_id_sync(), lane = lane_id();
  const int stages = p.stages;
  // the last rows first: row_sums_kernel read them last
  const unsigned at = gridDim.x - 1 - blockIdx.x;
  const int32_t row0 = static_cast<int32_t>(at / static_cast<unsigned>(p.ranges)) * 128;
  const int tile0 = static_cast<int>(at % static_cast<unsigned>(p.ranges)) * p.per;
  const int tiles = max(0, min(p.per, static_cast<int>(p.K / kCols) - tile0));
  const uint32_t t_boxes = LORA ? static_cast<uint32_t>((p.r + 63) / 64) : 0u;
  uint8_t* const out_sm = sm + t_boxes * kTBox;  // a tile of dX for each group
  uint8_t* const ring = out_sm + kGroups * kGBytes;

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&bars.full[s], 1);
      mbar_init(&bars.empty[s], kGroupWarps);
    }
    mbar_init(&bars.dt_full, 1);
    mbar_init(&bars.mma_done, 1);
    for (int i = 0; i < kGroups; ++i) {
      mbar_init(&bars.d_full[i], 1);
      mbar_init(&bars.d_empty[i], kGroupWarps);
      mbar_init(&bars.done[i], kGroupWarps);
      mbar_init(&bars.out_empty[i], 1);
    }
    bars.abort_flag = 0u;
    fence_mbar_init();
  }
  if (LORA && warp == 1) {
    tmem_alloc(&bars.tmem_base, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  // Only the row coefficients come from the kernel before this one, which let this one
  // start after all earlier work on the stream: everything else may be read beside it.
  if (warp == 0) {
    // ------------------------------------------------------------ loads
    if (lane == 0 && !p.stall_test) {
      if constexpr (LORA) {
        mbar_arrive_expect_tx(&bars.dt_full, t_boxes * kTBox);
        for (uint32_t b = 0; b < t_boxes; ++b)
          tma_load_2d(sm + b * kTBox, &p.tm_dt, &bars.dt_full, static_cast<int32_t>(64 * b), row0);
      }
      int slot = 0;
      uint32_t phase = 1;
      int issued = 0;
      for (int i = 0; i < tiles; ++i) {
        if (!back_wait(bars, &bars.empty[slot], phase, p.status, kDevTimeoutEmpty)) break;
        uint8_t* st = ring + static_cast<uint32_t>(slot) * p.stage_bytes;
        const int32_t col = (tile0 + i) * kCols;
        mbar_arrive_expect_tx(&bars.full[slot], kGBytes + kQBytes + 128u * static_cast<uint32_t>(p.r));
        tma_load_2d(st, &p.tm_g, &bars.full[slot], col, row0);
        tma_load_2d(st + kGBytes, &p.tm_q, &bars.full[slot], col, row0);
        if (LORA) tma_load_2d(st + kGBytes + kQBytes, &p.tm_a, &bars.full[slot], col, 0);
        ++issued;
        if (++slot == stages) slot = 0, phase ^= 1u;
      }
      // Copies in flight must land before the block exits, whichever warp gives up and
      // whenever it does (behind the last tile they have landed already).
      bool drained = !LORA || mbar_wait(&bars.dt_full, 0, kWaitLimitNs / 8);
      for (int i = issued - 1; i >= 0 && i >= issued - stages; --i)
        drained &= mbar_wait(&bars.full[i % stages], (i / stages) & 1, kWaitLimitNs / 8);
      if (!drained) record_error(p.status, kDevTimeoutDrain);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ dT A
    if constexpr (LORA) {
      constexpr uint32_t idesc = make_idesc_bf16(128, kCols, false) | kIdescBMnMajor;
      auto arrived = [&](uint64_t* bar, uint32_t parity, uint32_t code) {
        return __all_sync(0xffffffffu, back_wait(bars, bar, parity, p.status, code)) != 0;
      };
      bool ok = arrived(&bars.dt_full, 0, kDevTimeoutFull);
      int slot = 0;
      uint32_t phase = 0;
      for (int i = 0; ok && i < tiles; ++i) {
        const int buf = i % kGroups;
        ok = arrived(&bars.full[slot], phase, kDevTimeoutFull) &&
             arrived(&bars.d_empty[buf], ((i / kGroups) & 1) ^ 1, kDevTimeoutAccum);
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
        if (++slot == stages) slot = 0, phase ^= 1u;
      }
      // and MMAs in flight must be done before their TMEM is freed
      if (elect_one()) tc_commit(&bars.mma_done);
      __syncwarp();
      if (!mbar_wait(&bars.mma_done, 0, kWaitLimitNs / 8) && lane == 0) record_error(p.status, kDevTimeoutDrain);
      __syncwarp();
    }
  } else if (warp < kRoleWarps) {
    // ------------------------------------------------------------ stores of dX
    // One warp a group, so that neither group waits for the other's tile.
    if (lane == 0) {
      const int group = static_cast<int>(warp) - 2;
      uint32_t parity = 0;
      for (int i = group; i < tiles; i += kGroups, parity ^= 1u) {
        if (!back_wait(bars, &bars.done[group], parity, p.status, kDevTimeoutAccum)) break;
        tma_store_2d(&p.tm_dx, out_sm + group * kGBytes, (tile0 + i) * kCols, row0);
        bulk_commit();
        bulk_wait_read_all();
        mbar_arrive(&bars.out_empty[group]);
      }
      bulk_wait_all();
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ outputs
    const uint32_t quarter = warp & 3u, half = ((warp - kRoleWarps) >> 2) & 1u;
    const int buf = static_cast<int>((warp - kRoleWarps) >> 3);  // this group: its tiles and TMEM buffer
    const uint32_t row = 32u * quarter + lane;
    // 16 columns: one 16-byte unit of the stored values, two of G (swizzled by the row)
    auto q_unit = [&](uint32_t h) { return kGBytes + row * 64 + (((2 * half + h) ^ ((row >> 1) & 3u)) << 4); };
    auto g_unit = [&](uint32_t h, uint32_t u) { return row * 128 + (((4 * half + 2 * h + u) ^ (row & 7u)) << 4); };
    const uint32_t t_at = bars.tmem_base + buf * kCols + 32 * half + ((32u * quarter) << 16);
    pdl_wait();
    const float2 c = row0 + static_cast<int64_t>(row) < p.M ? __ldcg(p.coef + row0 + row) : make_float2(0.f, 0.f);
    // dX = kept: s g + sign(x) c (1 - s); dropped: sign(x) c, c = D / Lk
    const float s = c.x;
    const float dropped = 2.f * c.y, kept = 2.f * (c.y * (1.f - s));
    // the selection of this thread's two units of a tile, a tile ahead (the metadata has
    // whole row blocks, so rows past M can be read)
    const uint8_t* meta = nullptr;
    uint32_t nibbles[2] = {}, following[2] = {};
    auto select = [&](int i) {
      if (META && i < tiles) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          following[h] = __ldg(reinterpret_cast<const uint16_t*>(
              meta + meta_unit((tile0 + i) * 4 + 2 * static_cast<int>(half) + h)));
      }
    };
    if (META) meta = p.meta + (row0 / kRowBlock) * ((p.K + 127) / 128) * kMetaBlockBytes + meta_row(row);
    select(buf);
    int slot = buf % stages;
    uint32_t phase = static_cast<uint32_t>(buf / stages) & 1u, parity = 0;
    for (int i = buf; i < tiles; i += kGroups) {
      nibbles[0] = following[0], nibbles[1] = following[1];
      select(i + kGroups);
      bool ok = back_wait(bars, &bars.full[slot], phase, p.status, kDevTimeoutFull) &&
                back_wait(bars, &bars.out_empty[buf], parity ^ 1u, p.status, kDevTimeoutEmpty);
      if (LORA) ok = ok && back_wait(bars, &bars.d_full[buf], parity, p.status, kDevTimeoutAccum);
      if (!__all_sync(0xffffffffu, ok)) break;
      const uint8_t* st = ring + static_cast<uint32_t>(slot) * p.stage_bytes;
      uint8_t* const dst = out_sm + buf * kGBytes;
      if constexpr (LORA) tc_fence_after();
#pragma unroll
      for (uint32_t h = 0; h < 2; ++h) {
        uint32_t branch[16] = {};
        if constexpr (LORA) tmem_ld_32x32b_x16(t_at + 16 * h, branch);
        const uint4 qv = *reinterpret_cast<const uint4*>(st + q_unit(h));
        const uint4 ga = *reinterpret_cast<const uint4*>(st + g_unit(h, 0));
        const uint4 gb = *reinterpret_cast<const uint4*>(st + g_unit(h, 1));
        if constexpr (LORA) tmem_ld_wait();
        if (h == 1) {
          if constexpr (LORA) tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&bars.empty[slot]);
            if (LORA) mbar_arrive(&bars.d_empty[buf]);
          }
        }
        const uint32_t qw[4] = {qv.x, qv.y, qv.z, qv.w};
        const uint32_t gw[8] = {ga.x, ga.y, ga.z, ga.w, gb.x, gb.y, gb.z, gb.w};
        uint32_t out[8];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const uint32_t a = magnitudes<FMT>(qw[w]), bits = META ? kept_bits(nibbles[h], w) : keep_bits(a);
          // the upper half of 0.5 with the sign, or of 0
          const uint32_t half_sign = ((qw[w] & 0x80808080u) | 0x3F3F3F3Fu) & prmt<0xBA98>(a + 0x7F7F7F7Fu);
          const float g[4] = {bf16_lo(gw[2 * w]), bf16_hi(gw[2 * w]), bf16_lo(gw[2 * w + 1]), bf16_hi(gw[2 * w + 1])};
          float o[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float sign = __uint_as_float(__byte_perm(half_sign, 0u, (j << 12) | 0x0444));
            const bool keep = bits & (0x80u << 8 * j);
            o[j] = fmaf(sign, keep ? kept : dropped, __uint_as_float(branch[4 * w + j]));
            if (keep) o[j] = fmaf(s, g[j], o[j]);
          }
          out[2 * w] = pack_bf16(o[0], o[1]);
          out[2 * w + 1] = pack_bf16(o[2], o[3]);
        }
        *reinterpret_cast<uint4*>(dst + g_unit(h, 0)) = make_uint4(out[0], out[1], out[2], out[3]);
        *reinterpret_cast<uint4*>(dst + g_unit(h, 1)) = make_uint4(out[4], out[5], out[6], out[7]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.done[buf]);
      parity ^= 1u;
      for (slot += kGroups; slot >= stages; slot -= stages) phase ^= 1u;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (LORA && warp == 1) {
    tc_fence_after();
    tmem_dealloc(bars.tmem_base, kTmemCols);
  }
}

template <int FMT, bool LORA, bool META>
cudaError_t launch(const BackLaunch& b, unsigned blocks, uint32_t smem, cudaStream_t s) {
  static std::once_flag once[64];
  static cudaError_t configured[64];
  const cudaError_t e = once_per_device(once, configured, []() {
    return cudaFuncSetAttribute(sparsify_backward_kernel<FMT, LORA, META>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(kSmemMost));
  });
  if (e != cudaSuccess) return e;
  return launch_after_previous(sparsify_backward_kernel<FMT, LORA, META>, dim3(blocks), dim3(kThreads), smem, s, b);
}

template <int FMT, bool META>
cudaError_t run(const SparsifyBackwardLaunch& p, const BackLaunch& b, unsigned blocks, uint32_t smem, int sms,
                cudaStream_t s) {
  // a warp a row, more where the rows alone would leave SMs idle
  int rows = kRowWarps;
  while (rows > 1 && (p.M + rows - 1) / rows < 2 * sms) rows /= 2;
  const cudaError_t e = launch_after_previous(
      row_sums_kernel<FMT, META>, dim3(static_cast<unsigned>((p.M + rows - 1) / rows)), dim3(kRowThreads), 0, s, p, rows);
  if (e != cudaSuccess) return e;
  return p.dt != nullptr ? launch<FMT, true, META>(b, blocks, smem, s) : launch<FMT, false, META>(b, blocks, smem, s);
}

}  // namespace

cudaError_t launch_sparsify_backward(const SparsifyBackwardLaunch& p, int sms, cudaStream_t s) {
  BackLaunch b = {};
  b.coef = p.coef;
  b.meta = static_cast<const uint8_t*>(p.meta);
  b.M = p.M;
  b.K = p.K;
  b.r = p.r;
  b.stall_test = p.stall_test;
  b.status = p.status;
  const bool lora = p.dt != nullptr;
  const uint32_t t_bytes = lora ? static_cast<uint32_t>((p.r + 63) / 64) * kTBox : 0u;
  b.stage_bytes = kGBytes + kQBytes + 128u * static_cast<uint32_t>(p.r);
  const uint32_t fit = (kSmemMost - 1024 - t_bytes - kGroups * kGBytes) / b.stage_bytes;
  b.stages = static_cast<int>(fit < kMaxStages ? fit : kMaxStages);
  // blocks of a row block: the number with the fewest tiles one after another
  // (waves of one block an SM times tiles of a block), the smallest such
  const int64_t row_blocks = (p.M + 127) / 128, tiles = p.K / kCols;
  int64_t best = 0;
  for (int64_t n = 1; n <= tiles && n <= sms; ++n) {
    const int64_t steps = (row_blocks * n + sms - 1) / sms * ((tiles + n - 1) / n);
    if (best == 0 || steps < best) {
      best = steps;
      b.ranges = static_cast<int>(n);
    }
  }
  b.per = static_cast<int>((tiles + b.ranges - 1) / b.ranges);
  b.ranges = static_cast<int>((tiles + b.per - 1) / b.per);
  const uint32_t smem = 1024 + t_bytes + kGroups * kGBytes + b.stages * b.stage_bytes;
  const uint64_t M = p.M, K = p.K, r = p.r;
  constexpr auto kSw = CU_TENSOR_MAP_SWIZZLE_128B;
  if (!encode_bf16_2d(&b.tm_g, p.g, K, M, K * 2, kCols, 128, kSw) ||
      !encode_bf16_2d(&b.tm_dx, p.dx, K, M, K * 2, kCols, 128, kSw) ||
      !encode_u8_2d(&b.tm_q, p.q, K, M, K, kCols, 128, CU_TENSOR_MAP_SWIZZLE_64B))
    return cudaErrorInvalidValue;
  if (lora && (!encode_bf16_2d(&b.tm_dt, p.dt, r, M, r * 2, 64, 128, kSw) ||
               !encode_bf16_2d(&b.tm_a, p.a, K, r, K * 2, kCols, static_cast<uint32_t>(r), kSw)))
    return cudaErrorInvalidValue;
  const unsigned blocks = static_cast<unsigned>(row_blocks * b.ranges);
  if (p.meta != nullptr)
    return p.format == kCkpt8Int8 ? run<kCkpt8Int8, true>(p, b, blocks, smem, sms, s)
                                  : run<kCkpt8E4M3, true>(p, b, blocks, smem, sms, s);
  return p.format == kCkpt8Int8 ? run<kCkpt8Int8, false>(p, b, blocks, smem, sms, s)
                                : run<kCkpt8E4M3, false>(p, b, blocks, smem, sms, s);
}

}  // namespace lynx
