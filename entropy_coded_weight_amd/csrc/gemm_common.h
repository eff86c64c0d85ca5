// What the products of 4-bit and of 8-bit weights share: copies into LDS, the order of
// tiles, stores of results.
#pragma once
#include <type_traits>

#include "mx4_common.h"

namespace ecw {

template <int DT>
__device__ __forceinline__ void store_y(void* y, uint64_t at, float v) {
  if constexpr (DT == ECW_DT_F32)
    static_cast<float*>(y)[at] = v;
  else if constexpr (DT == ECW_DT_F16)
    static_cast<_Float16*>(y)[at] = (_Float16)v;
  else
    static_cast<__bf16*>(y)[at] = (__bf16)v;
}
// f<DT>() for the output's type
template <class F>
__device__ __forceinline__ void with_type(int dt, F&& f) {
  if (dt == ECW_DT_F32)
    f(std::integral_constant<int, ECW_DT_F32>{});
  else if (dt == ECW_DT_F16)
    f(std::integral_constant<int, ECW_DT_F16>{});
  else
    f(std::integral_constant<int, ECW_DT_BF16>{});
}

// Copies 16 bytes per lane from global memory to LDS, lane after lane from `to` on, without
// registers between.  The caller counts them: they are done when `s_waitcnt vmcnt` says so.
__device__ __forceinline__ void to_lds(const void* from, uint32_t to) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(from), "s"(to) : "m0", "memory");
}
template <int N>
__device__ __forceinline__ void wait_copies() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
}

// 16 bytes at piece p of row r's 128 lie at p ^ stirred(r), so that the 16 lanes that LDS
// serves together meet no bank twice.
__device__ __forceinline__ uint32_t stirred(uint32_t r) { return ((r >> 1) + 2) & 7; }

// A block's place among the tiles: blocks go to the 8 dies in turn, so each die takes a
// contiguous run of tiles, and within it 8 tiles of x rows stand next to each other, for
// the die's L2 to hold what its blocks share.
__device__ __forceinline__ void tile_of(uint32_t m_tiles, uint32_t n_tiles, uint32_t* m, uint32_t* n) {
  const uint32_t all = m_tiles * n_tiles, per = all / 8, more = all % 8;
  const uint32_t die = blockIdx.x % 8, i = blockIdx.x / 8;
  const uint32_t id = die * per + min(die, more) + i;
  const uint32_t band = id / (8 * n_tiles), first = band * 8, high = min(8u, m_tiles - first);
  const uint32_t in = id - band * 8 * n_tiles;
  *m = first + in % high;
  *n = in / high;
}

// With w's rows down the result's registers, row i of a wave's tile t stands for its row
// 4 TN (i / 4) + 4 t + i % 4: a lane then holds 4 TN neighbouring outputs of one row of x,
// four lanes a whole line.  (With one 2-byte store per output the stores took 78 of 205 us
// of the product of 4-bit operands at 4096 x 14336 x 4096.)
template <int TN>
__device__ __forceinline__ uint32_t spread(uint32_t t, uint32_t i) {
  return (i >> 2) * (4 * TN) + t * 4 + (i & 3);
}

// The N neighbouring outputs of a lane, the first `left` of them.  Runs go out as wide wherever
// they start (2444 rows of x by 10781 x 495 in 8 bits with short sums, fp16 outputs 38 us, with
// single elements where rows are not aligned 104).
template <int DT, int N>
__device__ __forceinline__ void store_run(void* y, uint64_t at, const float (&v)[N], uint32_t left) {
  if (left < N) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if ((uint32_t)i < left) store_y<DT>(y, at + i, v[i]);
    return;
  }
  if constexpr (DT == ECW_DT_F32) {
    float* o = static_cast<float*>(y) + at;
#pragma unroll
    for (int i = 0; i < N; i += 4) reinterpret_cast<Loose32*>(o + i)->v = f32x4{v[i], v[i + 1], v[i + 2], v[i + 3]};
  } else {
    uint32_t w[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      if constexpr (DT == ECW_DT_F16)
        w[i] = __builtin_bit_cast(uint32_t, f16x2{(_Float16)v[2 * i], (_Float16)v[2 * i + 1]});
      else
        w[i] = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)v[2 * i], (__bf16)v[2 * i + 1]});
    }
    uint16_t* o = static_cast<uint16_t*>(y) + at;
    if constexpr (N % 8 == 0) {
#pragma unroll
      for (int i = 0; i < N / 2; i += 4) reinterpret_cast<Loose16*>(o + 2 * i)->v = u32x4{w[i], w[i + 1], w[i + 2], w[i + 3]};
    } else {
      static_assert(N == 4, "");
      reinterpret_cast<Loose8*>(o)->v = u32x2{w[0], w[1]};
    }
  }
}

}  // namespace ecw
