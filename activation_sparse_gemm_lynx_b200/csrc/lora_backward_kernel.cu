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
// in three modes: T is the row product of x with P = A^T (kRow), dT and dB are both
// products of one pass over dY with P = B and Q = T (kBoth), dA^T the col product of
// x with Q = dT (kCol).  The same tile serves as a K-major and as an MN-major operand
// of tcgen05.mma.  At large ranks (from 128 at 4608 x 12288) kBoth's sums U weigh more
// than dY, and two passes over dY, kRow and kCol, take its place.
//
// A block has some inner blocks of 128 (rows for kRow, else columns), whose
// accumulators stay in TMEM, and walks a range of outer ones, whose operand (P of
// the columns, or Q of the rows) streams beside the tiles.  The outer ranges of the
// same inner blocks are a cluster's blocks: they add their accumulators through
// distributed shared memory, in the order of the ranks, and write the rounded
// result.  Only where one cluster is too few for the length (few inner blocks),
// groups of clusters leave fp32 sums that reduce_kernel adds.  kBoth's U leaves
// after each row block, as fp32 sums per column range for reduce_kernel.  No
// atomics: the order is the shape's.  T and dT enter their second product as the sum of
// two bf16 (Q's two halves, a col product each): 2^-17 off, below what the rounding of
// the results shows.  One bf16 (2^-8) put the gradients 0.0024 of their norm away from the
// formula, where that rounding alone takes 0.0017; three (all of fp32) would change
// nothing in bf16 results.  fp32 sums lie as [block][column of r][128]: a
// TMEM lane is a row, so a warp stores 128 bytes at a time (with rows of r floats
// the 4608 x 12288 pass spent 14 of 41 us storing).
//
// At 4608 x 4096 -> 12288, rank 64, int8 (137 MB in all) 72 us: T 18 us (19 MB, bound by
// the warps that widen it and the cluster's sums), the pass over dY 30 us behind it
// (113 MB in, 28 MB of sums out; its 24 MMAs a tile read 144 KB of shared memory),
// reduce_kernel 7 us (those 28 MB from L2), dA 17 us.  One bf16 for T and dT takes 65 us;
// at ranks 128 and 256 101 and 145 us for 126 and 202.
#include "lynx_ckpt8.cuh"
#include "lynx_internal.h"
#include "lynx_ptx.cuh"

namespace lynx {

namespace {

constexpr int kSrcBf16 = 2;  // beside kCkpt8Int8 and kCkpt8E4M3

enum PassMode : int { kRow, kBoth, kCol };

constexpr uint32_t kBox = 16384;        // 128 rows x 64 bf16, 128B swizzle
constexpr uint32_t kTileBytes = 2 * kBox;  // an S tile: two boxes of 64 columns
constexpr int kMaxStages = 6;
constexpr int kConvWarps = 16;
constexpr int kAhead = 3;                // 8-bit tiles in flight
constexpr uint32_t kRawBytes = 16384;    // one of them
constexpr int kMaxRanks = 6;
constexpr uint32_t kSmemMost = 227 * 1024 - 1024;  // leaves the static part 1 KB

struct PassPlan {
  int inner;             // inner blocks of a block
  int outer;             // outer blocks of a block
  int n_inner;           // ranges of inner blocks
  int ranks, groups;     // outer ranges: blocks of a cluster, clusters
  int stages, u_bufs;
  int op_bufs, subs;     // buffers of the streamed operand; pieces of an outer block that it comes in
  uint32_t tmem_cols;
  uint32_t smem;
  double cost;           // the estimated time, s
};

struct PassLaunch {
  CUtensorMap tm_s;   // dY [R,C], box 64 x 128 (bf16 source)
  CUtensorMap tm_p;   // kBoth: B [C,r], box 64 x 128
  CUtensorMap tm_op;  // the streamed operand: kRow A [r,C], box 64 x r (x), or B [C,r], box 64 x 128 (dY);
                      // else Q's two halves side by side [R,2r], box 64 x 128 / subs
  const uint8_t* q8;
  const uint8_t* e8;
  float* u_part;       // kBoth: [n_inner][row blocks][r][128]
  float* part;         // groups > 1: [groups][inner blocks][r][128]
  // groups == 1, either may be null:
  __nv_bfloat16* out;   // [inner rows][r], or [r][inner rows] (transposed)
  __nv_bfloat16* pair;  // [inner rows][2 r]: two bf16 whose sum is the value, first the upper ones
  int transposed;
  int early;           // a pass follows: it may launch beside this one's end
  int64_t R, C;
  int r;
  PassPlan plan;
  int stall_test;
  uint32_t* status;
};

struct PassBars {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t p_full, op_full[2], op_empty[2], u_full[2], u_empty[2], done;
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

// Two fp32 as the sums of two bf16 each (16 bits, 2^-17 off at most): the upper halves
// are the values rounded.
struct Halves {
  uint32_t hi, lo;
};

__device__ __forceinline__ Halves split_bf16(float a, float b) {
  Halves h;
  h.hi = pack_bf16(a, b);
  h.lo = pack_bf16(bf16_rest(a, bf16_lo(h.hi)), bf16_rest(b, bf16_hi(h.hi)));
  return h;
}

// 8 columns of a row, rounded in `out` and as two halves in `pair`
__device__ __forceinline__ void store_halves(__nv_bfloat16* out, __nv_bfloat16* pair, int64_t row, int r, int col,
                                             Halves a, Halves b, Halves c, Halves d) {
  const uint4 hi = make_uint4(a.hi, b.hi, c.hi, d.hi);
  if (out != nullptr) *reinterpret_cast<uint4*>(out + row * r + col) = hi;
  if (pair != nullptr) {
    *reinterpret_cast<uint4*>(pair + row * 2 * r + col) = hi;
    *reinterpret_cast<uint4*>(pair + row * 2 * r + r + col) = make_uint4(a.lo, b.lo, c.lo, d.lo);
  }
}

// TMA producer, MMA issuer, 4 epilogue warps, and the warps that widen 8-bit tiles
template <int SRC>
constexpr int kPassThreads = 32 * (6 + (SRC == kSrcBf16 ? 0 : kConvWarps));

template <int SRC, int MODE>
__global__ void __launch_bounds__(kPassThreads<SRC>, 1) adapter_pass_kernel(const __grid_constant__ PassLaunch p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ PassBars bars;
  uint8_t* const sm = smem_raw + ((0u - smem_u32(smem_raw)) & 1023u);
  const uint32_t warp = warp_id_sync();
  const uint32_t lane = lane_id();
  const int r = p.r;
  const uint32_t r_boxes = static_cast<uint32_t>((r + 63) / 64);   // 64-column boxes of an [*, r] operand
  const uint32_t r_cols = static_cast<uint32_t>((r + 31) / 32) * 32;  // TMEM columns of an accumulator
  const int stages = p.plan.stages;
  const int row_blocks = static_cast<int>((p.R + 127) / 128), col_blocks = static_cast<int>((p.C + 127) / 128);
  const int inner_blocks = MODE == kRow ? row_blocks : col_blocks, outer_blocks = MODE == kRow ? col_blocks : row_blocks;
  const uint32_t rank = cluster_ctarank();
  const int ranks = p.plan.ranks;
  const int cluster = static_cast<int>(blockIdx.x) / ranks;
  const int group = cluster % p.plan.groups, range = cluster / p.plan.groups;
  const int i0 = range * p.plan.inner;
  const int ni = min(p.plan.inner, inner_blocks - i0);
  const int o0 = (group * ranks + static_cast<int>(rank)) * p.plan.outer;
  const int no = max(0, min(p.plan.outer, outer_blocks - o0));

  // shared memory: P (kBoth) | streamed operand | S stages | 8-bit tiles
  const uint32_t p_block = r_boxes * kBox;
  constexpr bool kOpKmajor = MODE == kRow && SRC != kSrcBf16;  // A, whose rows lie along the sum
  // Q comes in pieces of 128 / subs rows, the upper halves of all columns and then the low
  // ones: with both, a whole block does not always leave room for two buffers.
  const int subs = MODE == kRow ? 1 : p.plan.subs;
  const uint32_t op_box = kBox / static_cast<uint32_t>(subs), op_half = r_boxes * op_box;
  const uint32_t op_bytes = kOpKmajor ? 256u * static_cast<uint32_t>(r) : MODE == kRow ? op_half : 2 * op_half;
  uint8_t* const sm_p = sm;
  uint8_t* const sm_op = sm_p + (MODE == kBoth ? static_cast<uint32_t>(p.plan.inner) * p_block : 0u);
  uint8_t* const sm_s = sm_op + static_cast<uint32_t>(p.plan.op_bufs) * op_bytes;

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&bars.full[s], SRC == kSrcBf16 ? 1 : kConvWarps);
      mbar_init(&bars.empty[s], 1);
    }
    mbar_init(&bars.p_full, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.op_full[i], 1);
      mbar_init(&bars.op_empty[i], 1);
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

  // one block a cluster and several groups: its sums are one of the partial sums
  const bool alone = ranks == 1 && p.plan.groups > 1;
  const uint32_t t_acc = bars.tmem_base;  // the inner blocks' accumulators, then U
  const uint32_t t_u = t_acc + static_cast<uint32_t>(p.plan.inner) * r_cols;
  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0 && !p.stall_test) {
      bool ok = true;
      if constexpr (MODE == kBoth) {
        mbar_arrive_expect_tx(&bars.p_full, static_cast<uint32_t>(ni) * p_block);
        for (int i = 0; i < ni; ++i)
          for (uint32_t b = 0; b < r_boxes; ++b)
            tma_load_2d(sm_p + static_cast<uint32_t>(i) * p_block + b * kBox, &p.tm_p, &bars.p_full,
                        static_cast<int32_t>(64 * b), (i0 + i) * 128);
      }
      const uint64_t once = l2_evict_first();  // dY is read once: leave L2 to the sums
      uint32_t g = 0;
      int issued = 0;
      auto operand = [&](int o, int sb) {  // a piece of outer block o's operand
        const int n = o * subs + sb, buf = n % p.plan.op_bufs;
        ok = pass_wait(bars, &bars.op_empty[buf], ((n / p.plan.op_bufs) & 1) ^ 1, p.status, kDevTimeoutEmpty);
        if (!ok) return;
        const int32_t at = (o0 + o) * 128 + sb * (128 / subs);
        uint8_t* dst = sm_op + static_cast<uint32_t>(buf) * op_bytes;
        mbar_arrive_expect_tx(&bars.op_full[buf], op_bytes);
        if constexpr (kOpKmajor) {
          for (int j = 0; j < 2; ++j)
            tma_load_2d(dst + static_cast<uint32_t>(j) * (op_bytes / 2), &p.tm_op, &bars.op_full[buf], at + 64 * j, 0);
        } else {
          for (uint32_t b = 0; b < r_boxes; ++b) {
            const int32_t col = static_cast<int32_t>(64 * b);
            tma_load_2d(dst + b * op_box, &p.tm_op, &bars.op_full[buf], col, at);
            if (MODE != kRow) tma_load_2d(dst + op_half + b * op_box, &p.tm_op, &bars.op_full[buf], r + col, at);
          }
        }
        issued = n + 1;
      };
      for (int o = 0; ok && o < no; ++o) {
        operand(o, 0);
        if constexpr (SRC == kSrcBf16) {
          const int32_t at = (o0 + o) * 128;
          for (int i = 0; ok && i < ni; ++i) {
            const uint32_t slot = g % stages;
            ok = pass_wait(bars, &bars.empty[slot], ((g / stages) & 1u) ^ 1u, p.status, kDevTimeoutEmpty);
            if (!ok) break;
            uint8_t* tile = sm_s + slot * kTileBytes;
            mbar_arrive_expect_tx(&bars.full[slot], kTileBytes);
            const int32_t in = (i0 + i) * 128, col = MODE == kRow ? at : in, row = MODE == kRow ? in : at;
            tma_load_2d_once(tile, &p.tm_s, &bars.full[slot], col, row, once);
            tma_load_2d_once(tile + kBox, &p.tm_s, &bars.full[slot], col + 64, row, once);
            ++g;
          }
        }
        for (int sb = 1; ok && sb < subs; ++sb) operand(o, sb);
      }
      // the last fill of every buffer must have landed before the block exits
      bool drained = true;
      if (MODE == kBoth) drained = mbar_wait(&bars.p_full, 0, kWaitLimitNs / 4);
      for (int x = issued - 1; x >= 0 && x >= issued - p.plan.op_bufs; --x)
        drained &= mbar_wait(&bars.op_full[x % p.plan.op_bufs], (x / p.plan.op_bufs) & 1, kWaitLimitNs / 4);
      for (uint32_t b = g; b > 0 && b + stages > g; --b)
        drained &= mbar_wait(&bars.full[(b - 1) % stages], ((b - 1) / stages) & 1u, kWaitLimitNs / 4);
      if (!drained) record_error(p.status, kDevTimeoutDrain);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    // The whole warp walks the loop and one elected lane issues, so that the
    // descriptors stay in warp-uniform registers (issued by a lone lane, a tile's
    // 16 MMAs took 1400 cycles, more than the tile's bytes).
    constexpr bool kHasRow = MODE != kCol, kHasCol = MODE != kRow;
    const uint32_t idesc_row = make_idesc_bf16(128, r, false) | (kOpKmajor ? 0u : kIdescBMnMajor);
    const uint32_t idesc_col = make_idesc_bf16(128, r, false) | kIdescAMnMajor | kIdescBMnMajor;
    auto arrived = [&](uint64_t* bar, uint32_t parity, uint32_t code) {
      return __all_sync(0xffffffffu, pass_wait(bars, bar, parity, p.status, code)) != 0;
    };
    bool ok = MODE != kBoth || arrived(&bars.p_full, 0, kDevTimeoutFull);
    uint32_t slot = 0, phase = 0;  // of an outer block's first tile
    for (int o = 0; ok && o < no; ++o) {
      const int ub = MODE == kBoth ? o % p.plan.u_bufs : 0;
      // The pieces of the operand one after another, each over all the tiles, which stay
      // until the last one has been multiplied.
      for (int sb = 0; ok && sb < subs; ++sb) {
        const int n = o * subs + sb, buf = n % p.plan.op_bufs;
        ok = arrived(&bars.op_full[buf], (n / p.plan.op_bufs) & 1, kDevTimeoutFull);
        if (ok && MODE == kBoth && sb == 0)
          ok = arrived(&bars.u_empty[ub], ((o / p.plan.u_bufs) & 1) ^ 1, kDevTimeoutAccum);
        if (!ok) break;
        const uint32_t sop = smem_u32(sm_op) + static_cast<uint32_t>(buf) * op_bytes;
        uint32_t at = slot, at_phase = phase;
        for (int i = 0; i < ni; ++i) {
          if (sb == 0) {
            ok = arrived(&bars.full[at], at_phase, kDevTimeoutFull);
            if (!ok) break;
            tc_fence_after();
          }
          const uint32_t ss = smem_u32(sm_s) + at * kTileBytes;
          const uint32_t d_inner = t_acc + static_cast<uint32_t>(i) * r_cols;
          if constexpr (kHasRow) {  // 16 columns of S a step
            const uint32_t d_row = MODE == kRow ? d_inner : t_u + static_cast<uint32_t>(ub) * r_cols;
            const uint32_t sp = smem_u32(sm_p) + static_cast<uint32_t>(i) * p_block;
            if (sb == 0) {
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const uint64_t da = make_sdesc(ss + (k / 4) * kBox + (k % 4) * 32, 16, 1024, kSw128);
                const uint64_t db = kOpKmajor
                                        ? make_sdesc(sop + (k / 4) * (op_bytes / 2) + (k % 4) * 32, 16, 1024, kSw128)
                                        : make_sdesc((MODE == kRow ? sop : sp) + k * 2048, kBox, 1024, kSw128);
                if (elect_one()) mma_bf16(d_row, da, db, idesc_row, ((MODE == kRow ? o : i) | k) != 0);
                __syncwarp();
              }
            }
          }
          if constexpr (kHasCol) {  // 16 rows of S a step, with the upper and the low halves
            const int steps = 8 / subs;
#pragma unroll 2
            for (int k = 0; k < steps; ++k) {
              const uint64_t da = make_sdesc(ss + (sb * steps + k) * 2048, kBox, 1024, kSw128);
              const uint64_t db = make_sdesc(sop + k * 2048, op_box, 1024, kSw128);
              const uint64_t db_low = make_sdesc(sop + op_half + k * 2048, op_box, 1024, kSw128);
              if (elect_one()) {
                mma_bf16(d_inner, da, db, idesc_col, (o | sb | k) != 0);
                mma_bf16(d_inner, da, db_low, idesc_col, true);
              }
              __syncwarp();
            }
          }
          if (sb == subs - 1) {
            if (elect_one()) tc_commit(&bars.empty[at]);
            __syncwarp();
          }
          if (++at == static_cast<uint32_t>(stages)) at = 0, at_phase ^= 1u;
        }
        if (!ok) break;
        if (elect_one()) {
          tc_commit(&bars.op_empty[buf]);
          if (MODE == kBoth && sb == 0) tc_commit(&bars.u_full[ub]);
        }
        __syncwarp();
        if (sb == subs - 1) slot = at, phase = at_phase;
      }
    }
    if (elect_one()) tc_commit(&bars.done);
    __syncwarp();
    if (!mbar_wait(&bars.done, 0) && lane == 0) record_error(p.status, kDevTimeoutDrain);
    __syncwarp();
  } else if (warp < 6) {
    // ------------------------------------------------------------ accumulators out
    const uint32_t quarter = warp & 3u;  // the TMEM lanes this warp may read
    const uint32_t t_lane = (32u * quarter) << 16;
    bool ok = true;
    // 16 columns at a time to dst[column][128]
    auto store = [&](uint32_t taddr, float* dst) {
      for (int c = 0; c < r; c += 16) {
        uint32_t v[16];
        tmem_ld_32x32b_x16(taddr + t_lane + static_cast<uint32_t>(c), v);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i) dst[(c + i) * 128 + 32 * quarter + lane] = __uint_as_float(v[i]);
      }
    };
    if constexpr (MODE == kBoth) {
      for (int o = 0; o < no; ++o) {
        const int ub = o % p.plan.u_bufs;
        ok = pass_wait(bars, &bars.u_full[ub], (o / p.plan.u_bufs) & 1, p.status, kDevTimeoutAccum);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        store(t_u + static_cast<uint32_t>(ub) * r_cols,
              p.u_part + (static_cast<int64_t>(range) * row_blocks + o0 + o) * r * 128);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.u_empty[ub]);
      }
    }
    // every MMA is done: the block's sums go out, or take the place of the operands
    ok = ok && pass_wait(bars, &bars.done, 0, p.status, kDevTimeoutAccum);
    ok = __all_sync(0xffffffffu, ok && !bars.abort_flag);
    if (ok) {
      tc_fence_after();
      float* dst = alone ? p.part + (static_cast<int64_t>(group) * inner_blocks + i0) * r * 128
                         : reinterpret_cast<float*>(sm);
      if (no > 0) {
        for (int i = 0; i < ni; ++i) store(t_acc + static_cast<uint32_t>(i) * r_cols, dst + i * r * 128);
      } else {  // no outer block for this rank
        for (int i = static_cast<int>(threadIdx.x) - 64; i < ni * r * 128; i += 128) dst[i] = 0.f;
      }
      tc_fence_before();
    }
  } else if constexpr (SRC != kSrcBf16) {
    // ------------------------------------------------------------ 8 bits -> bf16 tiles
    // 16 bytes (half a block) a step: 8 lanes cover a row of the tile, a thread
    // takes every kRowStep-th row.  4 lanes have one row's half and the next 4 the
    // row below's, whose swizzled units are the other banks.  The bytes arrive by cp.async in slots that
    // only this thread reads, kAhead tiles before they are needed; the exponents
    // (one byte per 32) come through registers, two tiles ahead.
    constexpr int kSteps = 4 * 8 / kConvWarps;
    constexpr int kRowStep = 4 * kConvWarps;
    const uint32_t t = threadIdx.x - 192u;
    const uint32_t chunk = (t & 3u) | ((t >> 1) & 4u);
    const uint32_t row_t = ((t >> 2) & 1u) | ((t >> 4) << 1);
    const int tiles = p.stall_test ? 0 : no * ni;
    // The walk over the tiles, inner blocks first: offsets of the next inner block
    // and, from the last one, of the next outer block's first
    const int64_t row0 = static_cast<int64_t>(MODE == kRow ? i0 : o0) * 128 + row_t;
    const int64_t col0 = static_cast<int64_t>(MODE == kRow ? o0 : i0) * 128;
    const int64_t e_pitch = p.C / 32;
    const int64_t q_row = 128 * p.C, e_row = 128 * e_pitch;
    const int64_t q_inner = MODE == kRow ? q_row : 128, e_inner = MODE == kRow ? e_row : 4;
    const int64_t q_outer = (MODE == kRow ? 128 : q_row) - q_inner * (ni - 1);
    const int64_t e_outer = (MODE == kRow ? 4 : e_row) - e_inner * (ni - 1);
    struct Walk {
      int rows, cols;  // rows from this thread's first one on, columns from its first one on
      int i, left;     // inner block, tiles left
    };
    Walk wq = {static_cast<int>(p.R - row0), static_cast<int>(p.C - col0) - 16 * static_cast<int>(chunk), 0, tiles};
    Walk we = wq;
    auto advance = [&](Walk& w) {
      --w.left;
      const bool next_outer = ++w.i == ni;
      if (next_outer) w.i = 0;
      if constexpr (MODE == kRow) {
        w.rows += next_outer ? 128 * (ni - 1) : -128;
        if (next_outer) w.cols -= 128;
      } else {
        w.cols += next_outer ? 128 * (ni - 1) : -128;
        if (next_outer) w.rows -= 128;
      }
      return next_outer;
    };
    const uint8_t* q_at = p.q8 + row0 * p.C + col0 + 16 * chunk;
    const uint8_t* e_at = p.e8 + row0 * e_pitch + col0 / 32 + chunk / 2;
    const uint32_t raw = smem_u32(sm_s) + static_cast<uint32_t>(stages) * kTileBytes + 16u * t;
    uint32_t fetch_at = 0, take_at = 0;  // byte offsets of the slots
    auto fetch = [&]() {
      if (wq.left > 0) {
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          const bool in = wq.cols > 0 && kRowStep * i < wq.rows;
          cp_async_16(raw + fetch_at + (kRawBytes / kSteps) * i, in ? q_at + i * kRowStep * p.C : p.q8, in ? 16u : 0u);
        }
        q_at += advance(wq) ? q_outer : q_inner;
        fetch_at = fetch_at == kAhead * kRawBytes ? 0u : fetch_at + kRawBytes;
      }
      cp_async_commit();
    };
    auto exponents = [&](uint32_t (&ex)[kSteps]) {
      if (we.left > 0) {
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
          ex[i] = we.cols > 0 && kRowStep * i < we.rows ? __ldg(e_at + i * kRowStep * e_pitch) : 0u;
        e_at += advance(we) ? e_outer : e_inner;
      }
    };
    const uint32_t x = row_t & 7u, u = (chunk & 3u) * 2u;  // kRowStep is a multiple of 8
    const uint32_t line = smem_u32(sm_s) + (chunk >> 2) * kBox + row_t * 128u;
    const uint32_t line0 = line + ((u ^ x) << 4), line1 = line + (((u + 1u) ^ x) << 4);
    const Ckpt8Widen<SRC> to_bf16;
    uint32_t slot = 0, phase = 1;
    bool ok = true;
    auto widen = [&](const uint32_t (&ex)[kSteps]) {
      cp_async_wait<kAhead - 1>();  // this tile's bytes are here
      uint2 out[kSteps][4];
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const uint32_t f = ckpt8_factor_bits<SRC>(ex[i]);
        const uint4 w = ld_shared_v4(raw + take_at + (kRawBytes / kSteps) * i);
        out[i][0] = to_bf16(w.x, f);
        out[i][1] = to_bf16(w.y, f);
        out[i][2] = to_bf16(w.z, f);
        out[i][3] = to_bf16(w.w, f);
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

  // ------------------------------------------------------------ the cluster's sums
  // Only for a pass, whose blocks take an SM each.  reduce_kernel's small blocks would
  // crowd onto the first SMs that are free (4608 x 12288: 72 us for 65).
  if (p.early) pdl_launch_dependents();
  __syncwarp();
  tc_fence_before();
  if (ranks == 1)
    __syncthreads();
  else
    cluster_sync_all();
  if (!alone && !bars.abort_flag) {
    const uint32_t red = smem_u32(sm);
    const int64_t inner_rows = MODE == kRow ? p.R : p.C;
    // 4 rows of one column a lane; the columns of the inner blocks dealt out to the
    // ranks' warps
    auto column_sum = [&](int column) {
      float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int q = 0; q < kMaxRanks; ++q) {
        if (q < ranks) {
          const float4 v = ld_cluster_f32x4(mapa_shared(red + (column * 128 + 4 * lane) * 4, q));
          s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
        }
      }
      return s;
    };
    const int ways = ranks * (kPassThreads<SRC> / 32), way = static_cast<int>(rank) * (kPassThreads<SRC> / 32) + warp;
    if (p.plan.groups > 1) {
      for (int c = way; c < ni * r; c += ways)
        *reinterpret_cast<float4*>(p.part + ((static_cast<int64_t>(group) * inner_blocks + i0) * r + c) * 128 + 4 * lane) =
            column_sum(c);
    } else if (p.transposed) {
      for (int c = way; c < ni * r; c += ways) {
        const float4 s = column_sum(c);
        const int64_t row = static_cast<int64_t>(i0 + c / r) * 128 + 4 * lane;  // inner_rows is a multiple of 64
        if (row < inner_rows)
          *reinterpret_cast<uint2*>(p.out + static_cast<int64_t>(c % r) * inner_rows + row) =
              make_uint2(pack_bf16(s.x, s.y), pack_bf16(s.z, s.w));
      }
    } else {
      // 8 columns at a time, so that 4 rows leave as 16 bytes each
      for (int c = 8 * way; c < ni * r; c += 8 * ways) {
        float4 s[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) s[j] = column_sum(c + j);
        const int64_t row = static_cast<int64_t>(i0 + c / r) * 128 + 4 * lane;
        auto put = [&](int k, float a0, float a1, float a2, float a3, float a4, float a5, float a6, float a7) {
          if (row + k < inner_rows)
            store_halves(p.out, p.pair, row + k, r, c % r, split_bf16(a0, a1), split_bf16(a2, a3), split_bf16(a4, a5),
                         split_bf16(a6, a7));
        };
        put(0, s[0].x, s[1].x, s[2].x, s[3].x, s[4].x, s[5].x, s[6].x, s[7].x);
        put(1, s[0].y, s[1].y, s[2].y, s[3].y, s[4].y, s[5].y, s[6].y, s[7].y);
        put(2, s[0].z, s[1].z, s[2].z, s[3].z, s[4].z, s[5].z, s[6].z, s[7].z);
        put(3, s[0].w, s[1].w, s[2].w, s[3].w, s[4].w, s[5].w, s[6].w, s[7].w);
      }
    }
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(bars.tmem_base, p.plan.tmem_cols);
  }
  __syncwarp();
  if (ranks > 1) cluster_sync_all();  // no block leaves while another reads its sums
}

// ---------------------------------------------------------------------------
// the ranges' partial sums, added in order and rounded

struct ReduceJob {
  const float* part;    // [n][blocks][r][128]
  __nv_bfloat16* out;   // [rows][r], or [r][rows] (transposed)
  __nv_bfloat16* pair;  // [rows][2 r], two bf16 a value (not transposed; either may be null)
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
#pragma unroll 8
  for (int i = 0; i < j.n; ++i) {
    const float4 v = __ldcg(reinterpret_cast<const float4*>(src + i * stride));
    const float4 w = __ldcg(reinterpret_cast<const float4*>(src + i * stride + 8 * 128));
    s0.x += v.x, s0.y += v.y, s0.z += v.z, s0.w += v.w;
    s1.x += w.x, s1.y += w.y, s1.z += w.z, s1.w += w.w;
  }
  pdl_launch_dependents();
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
      Halves o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = split_bf16(tile[c + 2 * i][row], tile[c + 2 * i + 1][row]);
      store_halves(j.out, j.pair, block * 128 + row, j.r, c0 + c, o[0], o[1], o[2], o[3]);
    }
  }
}

// ---------------------------------------------------------------------------
// host side

// The ranges of one pass: of the inner block counts that shared memory and TMEM
// hold and of the cluster sizes, the one with the least estimated time.  What it
// adds up, each measured on the passes themselves: a tile takes 0.7 us to widen, or
// the time of its bytes at 6.2 TB/s over the blocks at work (0.4 us at least) and
// 0.2 us, more where U has one buffer; the streamed operand comes at 80 GB/s a block,
// beside the tiles where it has two buffers (a piece more costs 0.1 us then, else 0.5);
// a cluster's sums cost 3 us and 40 GB/s a
// block (80 GB/s without a cluster); sums that go through memory are written and read
// at 8 TB/s (kBoth's are read at 3.5 where L2 no longer holds them), and a reduce_kernel
// of its own costs 5 us with its launch.
PassPlan plan_pass(int64_t R, int64_t C, int r, int mode, bool eight) {
  const int64_t rb = (R + 127) / 128, cb = (C + 127) / 128;
  const int64_t inner_blocks = mode == kRow ? rb : cb, outer_blocks = mode == kRow ? cb : rb;
  const uint32_t boxes = static_cast<uint32_t>((r + 63) / 64), rc = static_cast<uint32_t>((r + 31) / 32) * 32;
  // 1 KB of the dynamic part goes into its alignment
  const uint32_t raw = eight ? (kAhead + 1) * kRawBytes : 0u;
  const uint32_t p_block = mode == kBoth ? boxes * kBox : 0u;
  const uint32_t op_one = mode != kRow ? 2 * boxes * kBox : eight ? 256u * static_cast<uint32_t>(r) : boxes * kBox;
  const uint32_t min_stages = eight ? 2 : 3, most_stages = eight ? 3 : kMaxStages;
  // clusters of 1 to 6 such blocks that a B200 holds at once, less one for the sizes
  // that depend on which SMs a chip has
  constexpr int kRoom[kMaxRanks + 1] = {0, 148, 74, 44, 32, 25, 21};
  PassPlan best = {};
  for (int inner = 1; inner <= 8 && inner <= inner_blocks; ++inner) {
    PassPlan c = {};
    c.inner = inner;
    c.u_bufs = mode == kBoth ? 2 : 0;
    if (inner * rc + c.u_bufs * rc > 512 && c.u_bufs == 2) c.u_bufs = 1;
    if (inner * rc + c.u_bufs * rc > 512) break;
    const uint32_t red = static_cast<uint32_t>(inner * r) * 512u;
    if (red + 1024u > kSmemMost) break;
    c.tmem_cols = 32;
    while (c.tmem_cols < inner * rc + c.u_bufs * rc) c.tmem_cols *= 2;
    const int64_t n_inner = (inner_blocks + inner - 1) / inner;
    c.n_inner = static_cast<int>(n_inner);
    // written at 8 TB/s, read back at 3.5 where they no longer all lie in L2
    const double u_bytes = mode == kBoth ? 4.0 * r * 128 * static_cast<double>(n_inner * rb) : 0.0;
    const double u_cost = u_bytes / 8.0e12 + u_bytes / (u_bytes < 60e6 ? 8.0e12 : 3.5e12);
    // kBoth's sums are too many for a cluster's exchange to pay (17 us at 4608 x 12288)
    const int most_ranks = mode == kBoth ? 1 : kMaxRanks;
    for (int form = 0; form < 6; ++form) {  // one or two buffers; 1, 2 or 4 pieces
      c.op_bufs = 2 - form % 2;
      c.subs = 1 << form / 2;
      if (mode == kRow && c.subs > 1) break;
      const uint32_t fixed = inner * p_block + c.op_bufs * (op_one / c.subs) + raw + 1024u;
      if (fixed + min_stages * kTileBytes > kSmemMost) continue;
      const uint32_t fit = (kSmemMost - fixed) / kTileBytes;
      c.stages = static_cast<int>(fit < most_stages ? fit : most_stages);
      if (c.subs > 1 && c.stages <= inner) continue;  // the tiles of an outer block stay, and one comes
      c.smem = fixed + c.stages * kTileBytes;
      if (c.smem < red + 1024u) c.smem = red + 1024u;
      for (int ranks = 1; ranks <= most_ranks && ranks <= outer_blocks; ++ranks) {
        const int64_t fill = kRoom[ranks] / n_inner;  // groups that still fit at once
        for (int pass = 0; pass < (fill > 1 ? 2 : 1); ++pass) {
          int64_t groups = pass == 0 ? 1 : fill;
          const int64_t outer = (outer_blocks + ranks * groups - 1) / (ranks * groups);
          groups = (outer_blocks + ranks * outer - 1) / (ranks * outer);
          if (pass == 1 && groups == 1) continue;
          const int64_t clusters = n_inner * groups;
          const double waves = static_cast<double>((clusters + kRoom[ranks] - 1) / kRoom[ranks]);
          const double at_work = static_cast<double>(clusters < kRoom[ranks] ? clusters * ranks : kRoom[ranks] * ranks);
          const double bytes = (eight ? 16384.0 : 32768.0) * at_work / 6.2e12, least = eight ? 0.7e-6 : 0.4e-6;
          double tile = (bytes > least ? bytes : least) + (eight ? 0.0 : 0.2e-6);
          if (mode == kBoth && (c.u_bufs == 1 || c.op_bufs == 1)) tile *= 1.3;
          const double tiles = inner * tile, op = op_one / 80e9;
          const double step = c.op_bufs == 1 ? tiles + op + 0.5e-6 * c.subs
                                             : (tiles > op ? tiles : op) + 0.1e-6 * (c.subs - 1);
          double sums = 1e-6;
          if (ranks > 1) sums += 3e-6 + inner * r * 512 / 40e9;
          if (ranks == 1 && groups == 1) sums += inner * r * 512 / 80e9;
          double cost = waves * (outer * step + sums) + u_cost;
          if (groups > 1)
            cost += (mode == kBoth ? 0.0 : 5e-6) + 8.0 * r * 128 * static_cast<double>(groups * inner_blocks) / 8.0e12;
          if (best.inner == 0 || cost < best.cost) {
            best = c;
            best.cost = cost;
            best.ranks = ranks;
            best.groups = static_cast<int>(groups);
            best.outer = static_cast<int>(outer);
          }
        }
      }
      if (c.op_bufs == 2) break;  // more pieces are no better
    }
  }
  return best;
}

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

struct LoraPlan {
  PassPlan down, dy, dy_col, up;  // T; dT and dB, or dT alone; dB; dA
  bool both;
  size_t t, dt, u, part, total;
};

LoraPlan plan_lora(int64_t M, int64_t N, int64_t K, int r) {
  LoraPlan l;
  l.down = plan_pass(M, K, r, kRow, true);
  l.up = plan_pass(M, K, r, kCol, true);
  l.dy = plan_pass(M, N, r, kBoth, false);
  const PassPlan row = plan_pass(M, N, r, kRow, false);
  l.dy_col = plan_pass(M, N, r, kCol, false);
  // (measured at 4608 x 12288: rank 64 72 us with kBoth; rank 128 131 with, 126 without)
  l.both = l.dy.cost <= row.cost + l.dy_col.cost + 5e-6;
  if (!l.both) l.dy = row;
  const size_t mr = static_cast<size_t>(M) * r;  // T and dT are two bf16 a value
  auto sums = [r](int64_t rows, int n) { return static_cast<size_t>((rows + 127) / 128) * 512 * r * n; };
  size_t part = 0;
  auto more = [&part](size_t n) { part = n > part ? n : part; };
  if (l.down.groups > 1) more(sums(M, l.down.groups));
  if (l.dy.groups > 1) more(sums(l.both ? N : M, l.dy.groups));
  if (!l.both && l.dy_col.groups > 1) more(sums(N, l.dy_col.groups));
  if (l.up.groups > 1) more(sums(K, l.up.groups));
  l.t = 0;
  l.dt = align256(l.t + mr * 4);
  l.u = align256(l.dt + mr * 4);
  l.part = align256(l.u + (l.both ? sums(M, l.dy.n_inner) : 0));
  l.total = align256(l.part + part);
  return l;
}

template <int SRC, int MODE>
cudaError_t launch_pass(const PassLaunch& p, cudaStream_t s) {
  static std::once_flag once[64];
  static cudaError_t configured[64];
  const cudaError_t e = once_per_device(once, configured, []() {
    return cudaFuncSetAttribute(adapter_pass_kernel<SRC, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(kSmemMost));
  });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.plan.n_inner) * static_cast<unsigned>(p.plan.groups * p.plan.ranks));
  cfg.blockDim = dim3(kPassThreads<SRC>);
  cfg.dynamicSmemBytes = p.plan.smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(p.plan.ranks);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, adapter_pass_kernel<SRC, MODE>, p);
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
  auto* dt = reinterpret_cast<__nv_bfloat16*>(l.ws + plan.dt);
  auto* part = reinterpret_cast<float*>(l.ws + plan.part);
  const ReduceJob none = {};
  PassLaunch p = {};
  p.q8 = static_cast<const uint8_t*>(l.q);
  p.e8 = static_cast<const uint8_t*>(l.e);
  p.u_part = reinterpret_cast<float*>(l.ws + plan.u);
  p.part = part;
  p.R = l.M;
  p.r = l.r;
  p.stall_test = l.stall_test;
  p.status = l.status;
  constexpr auto kSw = CU_TENSOR_MAP_SWIZZLE_128B;

  // one pass and, where its clusters leave several sums, their reduction
  auto pass = [&](auto launch, const PassPlan& pass_plan, int64_t C, __nv_bfloat16* out, __nv_bfloat16* pair,
                  int64_t rows, bool transposed) {
    p.C = C;
    p.plan = pass_plan;
    p.out = out;
    p.pair = pair;
    p.transposed = transposed ? 1 : 0;
    p.early = pass_plan.groups == 1 && !transposed ? 1 : 0;  // dA's pass is the last
    const cudaError_t e = launch(p, s);
    if (e != cudaSuccess || pass_plan.groups == 1) return e;
    const ReduceJob job = {part, out, pair, rows, pass_plan.groups, l.r};
    return transposed ? launch_reduce<true>(job, none, s) : launch_reduce<false>(job, none, s);
  };
  auto* db = static_cast<__nv_bfloat16*>(l.db);
  auto* dt_out = static_cast<__nv_bfloat16*>(l.dt);

  // T = x A^T
  if (!encode_bf16_2d(&p.tm_op, l.a, K, r, K * 2, 64, static_cast<uint32_t>(r), kSw)) return cudaErrorInvalidValue;
  cudaError_t e = pass(launch_pass<FMT, kRow>, plan.down, l.K, nullptr, t, l.M, false);
  if (e != cudaSuccess) return e;

  // dT = dY B and dB = dY^T T
  CUtensorMap tm_b;
  auto halves_of = [&](const __nv_bfloat16* pair, const PassPlan& c) {
    return encode_bf16_2d(&p.tm_op, pair, 2 * r, M, 4 * r, 64, 128u / static_cast<uint32_t>(c.subs), kSw);
  };
  if (!encode_bf16_2d(&p.tm_s, l.dy, N, M, N * 2, 64, 128, kSw) ||
      !encode_bf16_2d(&tm_b, l.b, r, N, r * 2, 64, 128, kSw))
    return cudaErrorInvalidValue;
  if (plan.both) {
    p.tm_p = tm_b;
    if (!halves_of(t, plan.dy)) return cudaErrorInvalidValue;
    p.C = l.N;
    p.plan = plan.dy;
    p.out = db;
    p.pair = nullptr;
    p.transposed = 0;
    p.early = 0;
    e = launch_pass<kSrcBf16, kBoth>(p, s);
    if (e == cudaSuccess)
      e = launch_reduce<false>(ReduceJob{p.u_part, dt_out, dt, l.M, plan.dy.n_inner, l.r},
                               plan.dy.groups > 1 ? ReduceJob{part, db, nullptr, l.N, plan.dy.groups, l.r} : none, s);
  } else {
    p.tm_op = tm_b;
    e = pass(launch_pass<kSrcBf16, kRow>, plan.dy, l.N, dt_out, dt, l.M, false);
    if (e != cudaSuccess) return e;
    if (!halves_of(t, plan.dy_col)) return cudaErrorInvalidValue;
    e = pass(launch_pass<kSrcBf16, kCol>, plan.dy_col, l.N, db, nullptr, l.N, false);
  }
  if (e != cudaSuccess) return e;

  // dA^T = x^T dT
  if (!halves_of(dt, plan.up)) return cudaErrorInvalidValue;
  return pass(launch_pass<FMT, kCol>, plan.up, l.K, static_cast<__nv_bfloat16*>(l.da), nullptr, l.K, true);
}

}  // namespace

size_t lora_backward_workspace(int64_t M, int64_t N, int64_t K, int64_t r) {
  return plan_lora(M, N, K, static_cast<int>(r)).total;
}

cudaError_t launch_lora_backward(const LoraBackwardLaunch& p, cudaStream_t s) {
  return p.format == kCkpt8Int8 ? run<kCkpt8Int8>(p, s) : run<kCkpt8E4M3>(p, s);
}

}  // namespace lynx
