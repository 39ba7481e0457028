// lynx_rows.cuh -- 16 columns (32 bytes) of a lane's own row of Y, Z or the residual,
// between memory and the epilogue's registers.
//
// The GEMMs' stages leave next to no L1, so what is asked for twice comes from L2 twice,
// and the operands keep L2 at its rate: 32 bytes (a sector) go in one access where the rows
// lie on 32 bytes (`wide`), else in two of 16.  `left` is what remains of the row, a
// multiple of 8.  Plain loads, not the read-only path: the residual may be Y itself, whose
// tiles a CTA writes only after it has read them.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

namespace lynx {

__device__ __forceinline__ void load_row16(uint32_t (&v)[8], const __nv_bfloat16* at, int left, bool wide) {
  if (wide) {
    if (left > 0)
      asm volatile("ld.global.L1::no_allocate.L2::256B.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                   : "l"(at)
                   : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (left > 8 * i)
        asm volatile("ld.global.L1::no_allocate.L2::256B.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v[4 * i]), "=r"(v[4 * i + 1]), "=r"(v[4 * i + 2]), "=r"(v[4 * i + 3])
                     : "l"(at + 8 * i)
                     : "memory");
    }
  }
}

// SOON: the next kernel reads them; else they make way in L2 (Z, until the backward pass).  Past L1
// either way: allocating there, 500 x 512 -> 4096, dense, takes 7.2 us for 6.7.
template <bool SOON>
__device__ __forceinline__ void store_row16(__nv_bfloat16* at, const uint32_t (&v)[8], int left, bool wide) {
  if (wide) {
    if (left <= 0) return;
    if constexpr (SOON)
      asm volatile("st.global.L1::no_allocate.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at), "r"(v[0]),
                   "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                   : "memory");
    else
      asm volatile("st.global.L1::no_allocate.L2::evict_first.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at),
                   "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                   : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (left > 8 * i)
        *reinterpret_cast<uint4*>(at + 8 * i) = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
  }
}

}  // namespace lynx
