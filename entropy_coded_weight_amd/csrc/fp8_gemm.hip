// y[b][n] = sum_k x[b][k] w[n][k], both in the block-scaled 8-bit format.
//
// Two instructions multiply.  The bf16 one (16x16x32) is what a call gets: E4M3 numbers times
// their scale are exact in bf16, products exact in fp32, and sums fp32.  The scaled 8-bit one
// (16x16x128) takes one block of 128 columns of 16 rows of each operand, 32 bytes a lane, and
// a scale byte of each lane's row, so that a block's product takes one instruction, scales
// included (4.3 PFLOP/s measured, 2.1 for bf16).  But it adds up to 16 neighbouring products
// with 12 fraction bits under the largest one's power of two before they go into the fp32
// sum: each may lose 2^-12 of the largest, so the sum up to 15 * 2^-12 < 2^-8 of the
// products' magnitudes (448^2 - 448^2 + 2^2 is 0).  Measured against 64 bits 1.5e-5 of the
// result in 2-norm for normal numbers, 7e-5 with columns a hundred times as large, where fp32
// sums are off by 1e-7.  So it multiplies only where the caller asks for short sums, of
// 16-bit outputs and more rows of x than go by k_fp8_gemm_few.
//
// Which of the columns of a block a lane holds is free as long as both operands agree and all
// of a row's lanes give the same scale: lane l has row l % 16 and the 16-byte pieces l / 16
// and l / 16 + 4.  w's rows go down the result's registers: a lane holds neighbouring outputs
// of one row of x.
#include "fp8_common.h"
#include "gemm_common.h"

#include <algorithm>
#include <atomic>

namespace ecw {

struct Fp8GemmArgs {
  const uint8_t *w, *ws, *x, *xs;  // codes and scale bytes
  void* y;
  uint32_t rows, batch;
  uint32_t row, scale_row, spans;  // bytes of a row of codes and of scales, blocks of 128 columns
  uint32_t y_row;                  // elements from one row of y to the next
  uint32_t splits, chunk;          // parts of the columns, spans of one
  float* part;                     // with more than one: [splits][part_size] sums
  uint64_t part_size;
};

typedef int i32x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ i32x8 join(u32x4 a, u32x4 b) {
  return i32x8{(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
}
__device__ __forceinline__ f32x4 block_product(f32x4 acc, i32x8 w, uint32_t sw, i32x8 x, uint32_t sx) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, acc, 0, 0, 0, (int)sw, 0, (int)sx);
}

// codes 8 J .. 8 J + 7 of a lane's 32, times their scale
template <int J>
__device__ __forceinline__ bf16x8 oct_fp8(const i32x8& v, float scale) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)v[2 * J], scale, false);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)v[2 * J], scale, true);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)v[2 * J + 1], scale, false);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)v[2 * J + 1], scale, true);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}
// acc[n][m] += w tile n times x tile m over columns 8 J.. of every lane
template <int J, int TN, int TM>
__device__ __forceinline__ void exact_product(f32x4 (&acc)[TN][TM], const i32x8 (&w)[TN], const float (&sw)[TN],
                                              const i32x8 (&x)[TM], const float (&sx)[TM]) {
  bf16x8 wj[TN], xj[TM];
#pragma unroll
  for (int n = 0; n < TN; ++n) wj[n] = oct_fp8<J>(w[n], sw[n]);
#pragma unroll
  for (int m = 0; m < TM; ++m) xj[m] = oct_fp8<J>(x[m], sx[m]);
#pragma unroll
  for (int m = 0; m < TM; ++m)
#pragma unroll
    for (int n = 0; n < TN; ++n)
      acc[n][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wj[n], xj[m], acc[n][m], 0, 0, 0);
}
template <int TN, int TM>
__device__ __forceinline__ void exact_products(f32x4 (&acc)[TN][TM], const i32x8 (&w)[TN], const float (&sw)[TN],
                                               const i32x8 (&x)[TM], const float (&sx)[TM]) {
  exact_product<0>(acc, w, sw, x, sx);
  exact_product<1>(acc, w, sw, x, sx);
  exact_product<2>(acc, w, sw, x, sx);
  exact_product<3>(acc, w, sw, x, sx);
}

// ------------------------------------------------------------------ a few rows
// Up to 16 rows of x, which fit LDS.  A block takes groups of 16 rows of w in turn; each of its
// waves has every kFewWaves-th span of them, a ring of copies of w that never runs dry from
// one group to the next, and the x of its spans, copied once.  After each group the waves'
// sums are joined through LDS in the order of the waves, by another wave each time, while the
// others go on.  8 rows of 128 bytes are copied at a time, so that neighbouring lanes read
// whole lines.  Bound by reading w: one row by 4096 x 14336 11.4 us (5.1 TB/s), by
// 14336 x 4096 13.2 (4.4; with a block for each group and no ring 16.4), by 28672 x 8192
// 41 (5.7; 60).  Rings of 3 and 4 slots gain nothing (11.8 and 12.3 us for the first), nor do
// blocks of 4 or 16 waves (11.6 to 12.6).
constexpr uint32_t kFewWaves = 8, kFewRing = 2;
constexpr uint32_t kFewSlot = 16 * 128 + 256;  // 16 rows of w, and a word of each lane's scales

struct FewShape {
  uint32_t each;     // spans of a wave, at most
  uint32_t shift;    // 2^shift rows of x in LDS
  uint32_t x_bytes;  // of a wave
  uint32_t lds;
};

// 4 bytes a lane into LDS, as to_lds.
__device__ __forceinline__ void word_to_lds(const void* from, uint32_t to) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, off" ::"v"(from), "s"(to) : "m0", "memory");
}

__global__ void __launch_bounds__(64 * kFewWaves) k_fp8_gemm_few(Fp8GemmArgs a, FewShape f, int y_dtype) {
  extern __shared__ __align__(16) uint8_t lds[];  // rings, x, scales of x (16 bytes a span), sums
  constexpr uint32_t W = kFewWaves, R = kFewRing;
  const uint32_t base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;
  const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t r16 = lane & 15, g = lane >> 4;
  const uint32_t groups = (a.rows + 15) / 16;
  const uint32_t ring = wave * R * kFewSlot;
  const uint32_t x_at = W * R * kFewSlot + wave * f.x_bytes;
  const uint32_t s_at = W * (R * kFewSlot + f.x_bytes) + wave * f.each * 16;
  f32x4* part = reinterpret_cast<f32x4*>(lds + W * (R * kFewSlot + f.x_bytes + f.each * 16));  // [2][W][64]
  const uint32_t mine = wave < a.spans ? (a.spans - wave + W - 1) / W : 0;

  // x: [span][2^shift rows][128 bytes], its pieces stirred by row; rows past the last are the last
  const uint32_t x_rows = (1u << f.shift) - 1;
  if (mine) {
    const uint32_t units = ((mine << f.shift) + 7) / 8;
    for (uint32_t u = 0; u < units; ++u) {
      const uint32_t i = u * 8 + (lane >> 3), row = i & x_rows, j = min(i >> f.shift, mine - 1);
      to_lds(a.x + (uint64_t)min(row, a.batch - 1) * a.row + (uint64_t)(wave + j * W) * 128 + ((lane & 7) ^ stirred(row)) * 16,
             base + x_at + u * 1024);
    }
    for (uint32_t j = g; j < mine; j += 4)
      lds[s_at + j * 16 + r16] = a.xs[(uint64_t)min(r16, a.batch - 1) * a.scale_row + wave + j * W];
  }
  // the next slot of the ring: group `of`, the wave's span `j`; behind the last group the last
  // again, which is not multiplied
  uint32_t of = blockIdx.x, j_next = 0, slot_next = 0;
  auto issue = [&]() {
    const uint32_t first = min(of, groups - 1) * 16, s = wave + j_next * W, to = base + ring + slot_next * kFewSlot;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t row = i * 8 + (lane >> 3);
      to_lds(a.w + (uint64_t)min(first + row, a.rows - 1) * a.row + (uint64_t)s * 128 + ((lane & 7) ^ stirred(row)) * 16,
             to + i * 1024);
    }
    word_to_lds(a.ws + (uint64_t)min(first + r16, a.rows - 1) * a.scale_row + (s & ~3u), to + 2048);
    if (++j_next == mine) j_next = 0, of += gridDim.x;
    slot_next = slot_next + 1 == R ? 0 : slot_next + 1;
  };
  constexpr int kCopies = 3;  // of a slot
  if (mine)
    for (uint32_t i = 0; i < R; ++i) issue();
  const uint32_t w0 = r16 * 8 + (g ^ stirred(r16)), w1 = r16 * 8 + ((g + 4) ^ stirred(r16));
  const uint32_t xr = r16 & x_rows, x0 = xr * 8 + (g ^ stirred(xr)), x1 = xr * 8 + ((g + 4) ^ stirred(xr));
  uint32_t slot = 0, turn = 0, joins = 0;  // the wave that joins
  for (uint32_t group = blockIdx.x; group < groups; group += gridDim.x) {
    f32x4 acc[1][1] = {{f32x4{0.f, 0.f, 0.f, 0.f}}};
    for (uint32_t j = 0; j < mine; ++j) {
      wait_copies<(R - 1) * kCopies>();
      const uint8_t* at = lds + ring + slot * kFewSlot;
      const u32x4* w = reinterpret_cast<const u32x4*>(at);
      const u32x4* x = reinterpret_cast<const u32x4*>(lds + x_at + ((j * 128) << f.shift));
      const i32x8 wv[1] = {join(w[w0], w[w1])}, xv[1] = {join(x[x0], x[x1])};
      const float sw[1] = {scale_of(at[2048 + r16 * 4 + ((wave + j * W) & 3)])}, sx[1] = {scale_of(lds[s_at + j * 16 + r16])};
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the slot is read
      issue();
      slot = slot + 1 == R ? 0 : slot + 1;
      exact_products(acc, wv, sw, xv, sx);
    }
    part[(turn * W + wave) * 64 + lane] = acc[0][0];
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");  // copies stay in flight
    if (wave == joins) {
      f32x4 sum = part[turn * W * 64 + lane];
#pragma unroll
      for (uint32_t v = 1; v < W; ++v) sum += part[(turn * W + v) * 64 + lane];
      // lane l: rows 4 (l / 16) .. + 3 of w, row l % 16 of x
      const uint32_t n = group * 16 + g * 4;
      if (r16 < a.batch && n < a.rows) {
        with_type(y_dtype, [&](auto dt) {
          const float v[4] = {sum[0], sum[1], sum[2], sum[3]};
          store_run<dt.value>(a.y, (uint64_t)r16 * a.rows + n, v, a.rows - n);
        });
      }
    }
    turn ^= 1;
    joins = joins + 1 == W ? 0 : joins + 1;
  }
  wait_copies<0>();
}

// ------------------------------------------------------------------ many rows
// A block of WM x WN waves multiplies 16 TM WM rows of x and 16 TN WN rows of w, a span of
// 128 columns at a time, from NS stages in LDS that copies fill ahead.  KG: it has KG times
// the waves, which take KG spans at once and add their sums up at the end, in order.  Where
// there are few tiles the columns are cut too: blockIdx.y has `chunk` spans (a multiple of
// KG), and k_fp8_gemm_join adds the parts up.
//
// The large tiles by the 8-bit instruction are bound by the copies next to the matrix
// instructions: 8192 x 8192 x 8192 takes 443 us (2.5 PFLOP/s), the matrix instructions alone
// 297, they and the copies without a read of LDS 408, they and the reads without the copies
// 326.  Copies alone run at 85 to 105 KB a us and CU, next to the instructions at 40 to 60.
// Reads of LDS that run ahead of the instructions, the sums in accumulation registers, gained
// 3%, waves that take turns at reading and multiplying lost 30%, words of later spans asked
// for ahead, to have them in L2, lost 5%, operands of a whole span read ahead gained nothing
// in any tile: not kept.  By the bf16 instruction the same takes 830 us (1.3 PFLOP/s; a bf16
// library product of this size runs at 1.38).
template <int WM, int WN, int TM, int TN, int NS, int KG>
struct Fp8Tiles {
  static constexpr int kWaves = WM * WN, BM = 16 * TM * WM, BN = 16 * TN * WN;
  static constexpr uint32_t kX = BM * 128, kSpan = (BM + BN) * 128, kStage = KG * kSpan;
  static constexpr uint32_t kScaleRows = (BM + BN + 63) / 64 * 64;   // those of x first
  static constexpr uint32_t kScalePlaces = (NS * KG + 15) / 16 + 1;  // of 16 spans each
  static constexpr uint32_t kBytes = kStage * NS + kScalePlaces * kScaleRows * 16;
  static constexpr int kXLoads = BM / 8 / kWaves, kWLoads = BN / 8 / kWaves;  // copies per wave and span
  static constexpr int kSLoads = (kScaleRows / 64 + kWaves - 1) / kWaves;    // per 16 spans
  static_assert(BM % (8 * kWaves) == 0 && BN % (8 * kWaves) == 0, "");
  static_assert(kBytes <= 160 * 1024 && 16 % KG == 0, "");
  static_assert((KG - 1) * kWaves * TM * TN * 1024 <= (int)kStage * NS, "");  // sums of the other groups
};

// EXACT: by the bf16 instruction, else by the 8-bit one.
template <int WM, int WN, int TM, int TN, int NS, int KG, bool EXACT>
__global__ void __launch_bounds__(64 * WM * WN * KG) k_fp8_gemm_tile(Fp8GemmArgs a, uint32_t m_tiles, uint32_t n_tiles,
                                                                     int y_dtype) {
  using T = Fp8Tiles<WM, WN, TM, TN, NS, KG>;
  __shared__ __align__(16) uint8_t lds[T::kBytes];
  const uint32_t base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;
  const uint32_t lane = threadIdx.x & 63, waves = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t kg = waves / T::kWaves, wave = waves % T::kWaves;
  const uint32_t r16 = lane & 15, g = lane >> 4;
  uint32_t mt, nt;
  tile_of(m_tiles, n_tiles, &mt, &nt);
  const uint32_t m0 = mt * T::BM, n0 = nt * T::BN;
  const uint32_t begin = blockIdx.y * a.chunk, end = min(begin + a.chunk, a.spans);
  const uint32_t steps = (end - begin + KG - 1) / KG;
  const uint32_t wm = wave / WN * TM, wn = wave % WN * TN;  // first 16-row tiles of the wave

  // what the lane copies: 16 bytes of one of eight rows; rows past the end are the last again
  const uint8_t *xp[T::kXLoads], *wp[T::kWLoads], *sp[T::kSLoads];
#pragma unroll
  for (int i = 0; i < T::kXLoads; ++i) {
    const uint32_t row = (wave * T::kXLoads + i) * 8 + (lane >> 3), piece = (lane & 7) ^ stirred(row & 15);
    xp[i] = a.x + (uint64_t)min(m0 + row, a.batch - 1) * a.row + piece * 16;
  }
#pragma unroll
  for (int i = 0; i < T::kWLoads; ++i) {
    const uint32_t at = (wave * T::kWLoads + i) * 8 + (lane >> 3), piece = (lane & 7) ^ stirred(at & 15);
    const uint32_t row = at / (16 * TN) * (16 * TN) + spread<TN>(at / 16 % TN, at & 15);
    wp[i] = a.w + (uint64_t)min(n0 + row, a.rows - 1) * a.row + piece * 16;
  }
#pragma unroll
  for (int i = 0; i < T::kSLoads; ++i) {
    const uint32_t at = (wave + i * T::kWaves) * 64 + lane;
    if (at < T::BM) {
      sp[i] = a.xs + (uint64_t)min(m0 + at, a.batch - 1) * a.scale_row;
    } else {
      const uint32_t in = at - T::BM, row = in / (16 * TN) * (16 * TN) + spread<TN>(in / 16 % TN, in & 15);
      sp[i] = a.ws + (uint64_t)min(n0 + row, a.rows - 1) * a.scale_row;
    }
  }

  // Copies of one step's spans into a stage; past the last span the last one again, into a
  // place that is not multiplied, so that every step waits for the same number.
  auto fill = [&](uint32_t step, uint32_t stage) {
    const uint32_t span = begin + step * KG + kg;
    const uint64_t s = min(span, end - 1);
    if (kg == 0 && (span % 16 == 0 || step == 0) && span < end) {
#pragma unroll
      for (int i = 0; i < T::kSLoads; ++i) {
        const uint32_t part = wave + i * T::kWaves;
        if (part < T::kScaleRows / 64)
          to_lds(sp[i] + (s & ~15ull), base + T::kStage * NS + (span / 16 % T::kScalePlaces) * T::kScaleRows * 16 + part * 1024);
      }
    }
    const uint32_t to = base + stage * T::kStage + kg * T::kSpan;
#pragma unroll
    for (int i = 0; i < T::kXLoads; ++i) to_lds(xp[i] + s * 128, to + (wave * T::kXLoads + i) * 1024);
#pragma unroll
    for (int i = 0; i < T::kWLoads; ++i) to_lds(wp[i] + s * 128, to + T::kX + (wave * T::kWLoads + i) * 1024);
  };

  f32x4 acc[TN][TM];
#pragma unroll
  for (int n = 0; n < TN; ++n)
#pragma unroll
    for (int m = 0; m < TM; ++m) acc[n][m] = f32x4{0.f, 0.f, 0.f, 0.f};
  const uint32_t in0 = r16 * 8 + (g ^ stirred(r16)), in1 = r16 * 8 + ((g + 4) ^ stirred(r16));

  constexpr int kCopies = T::kXLoads + T::kWLoads;  // of a step; scales may be among those waited for too
  uint32_t stage = 0, before = NS - 1;              // of the step that is multiplied, and of the one before
#pragma unroll
  for (int i = 0; i < NS - 1; ++i) fill(i, i);
  for (uint32_t step = 0; step < steps; ++step) {
    wait_copies<(NS - 2) * kCopies>();
    __builtin_amdgcn_s_barrier();  // this step is there, and the one before it is done with
    fill(step + NS - 1, before);
    const uint32_t s = begin + step * KG + kg;
    const uint8_t* at = lds + stage * T::kStage + kg * T::kSpan;
    const u32x4* x = reinterpret_cast<const u32x4*>(at) + wm * 128;
    const u32x4* w = reinterpret_cast<const u32x4*>(at + T::kX) + wn * 128;
    const uint8_t* xs = lds + T::kStage * NS + (s / 16 % T::kScalePlaces) * T::kScaleRows * 16 + s % 16 + (wm * 16 + r16) * 16;
    const uint8_t* ws = xs + (T::BM - wm * 16 + wn * 16) * 16;
    if (KG == 1 || s < end) {
      i32x8 wv[TN], xv[TM];
      uint32_t sw[TN], sx[TM];
#pragma unroll
      for (int n = 0; n < TN; ++n) wv[n] = join(w[n * 128 + in0], w[n * 128 + in1]), sw[n] = ws[n * 256];
#pragma unroll
      for (int m = 0; m < TM; ++m) xv[m] = join(x[m * 128 + in0], x[m * 128 + in1]), sx[m] = xs[m * 256];
      if constexpr (EXACT) {
        float fw[TN], fx[TM];
#pragma unroll
        for (int n = 0; n < TN; ++n) fw[n] = scale_of(sw[n]);
#pragma unroll
        for (int m = 0; m < TM; ++m) fx[m] = scale_of(sx[m]);
        exact_products(acc, wv, fw, xv, fx);
      } else {
#pragma unroll
        for (int m = 0; m < TM; ++m)
#pragma unroll
          for (int n = 0; n < TN; ++n) acc[n][m] = block_product(acc[n][m], wv[n], sw[n], xv[m], sx[m]);
      }
    }
    before = stage;
    stage = stage + 1 == NS ? 0 : stage + 1;
  }
  wait_copies<0>();
  if constexpr (KG > 1) {
    __builtin_amdgcn_s_barrier();  // every wave is done with the stages
    f32x4* sums = reinterpret_cast<f32x4*>(lds) + wave * TN * TM * 64 + lane;
#pragma unroll
    for (int n = 0; n < TN; ++n)
#pragma unroll
      for (int m = 0; m < TM; ++m)
        if (kg > 0) sums[((kg - 1) * T::kWaves * TN * TM + n * TM + m) * 64] = acc[n][m];
    __syncthreads();
    if (kg > 0) return;
#pragma unroll
    for (int k = 0; k < KG - 1; ++k)
#pragma unroll
      for (int n = 0; n < TN; ++n)
#pragma unroll
        for (int m = 0; m < TM; ++m) acc[n][m] += sums[(k * T::kWaves * TN * TM + n * TM + m) * 64];
  }
  const uint32_t at = n0 + wn * 16 + g * (4 * TN);
  if (at >= a.rows) return;
  const bool whole = a.splits == 1;
  void* y = whole ? a.y : a.part + blockIdx.y * a.part_size;
  const uint32_t y_row = whole ? a.y_row : a.rows;
  if (!whole) y_dtype = ECW_DT_F32;
  with_type(y_dtype, [&](auto dt) {
#pragma unroll
    for (int m = 0; m < TM; ++m) {
      const uint32_t b = m0 + (wm + m) * 16 + r16;
      float v[4 * TN];
#pragma unroll
      for (int n = 0; n < TN; ++n)
#pragma unroll
        for (int r = 0; r < 4; ++r) v[n * 4 + r] = acc[n][m][r];
      if (b < a.batch) store_run<dt.value>(y, (uint64_t)b * y_row + at, v, a.rows - at);
    }
  });
}

// The parts of the columns added up, in order, 4 outputs a lane, 4 parts asked for at once.
template <int DT>
__global__ void __launch_bounds__(256) k_fp8_gemm_join(const float* __restrict__ part, void* __restrict__ y, uint64_t all,
                                                       uint64_t part_size, uint32_t splits) {
  const uint64_t at = ((uint64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (at >= all) return;
  f32x4 sum = {0.f, 0.f, 0.f, 0.f};
  for (uint32_t s = 0; s < splits; s += 4) {
    f32x4 p[4];
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i) p[i] = *reinterpret_cast<const f32x4*>(part + min(s + i, splits - 1) * part_size + at);
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i)
      if (s + i < splits) sum += p[i];
  }
  const float v[4] = {sum[0], sum[1], sum[2], sum[3]};
  store_run<DT>(y, at, v, (uint32_t)min(all - at, (uint64_t)4));
}

}  // namespace ecw

using namespace ecw;

namespace {

constexpr uint32_t kCus = 256, kLds = 160 * 1024;

// The shape of the kernel for a few rows; false: they are too many, or too long for LDS.
bool few_shape(uint32_t batch, uint32_t spans, FewShape* f) {
  if (batch > 16) return false;
  f->each = (spans + kFewWaves - 1) / kFewWaves;
  f->shift = 0;
  while (1u << f->shift < batch) ++f->shift;
  const uint64_t x = ((((uint64_t)f->each * 128) << f->shift) + 1023) / 1024 * 1024;
  const uint64_t lds = kFewWaves * (kFewRing * kFewSlot + x + f->each * 16) + 2 * kFewWaves * 1024;
  f->x_bytes = (uint32_t)x;
  f->lds = (uint32_t)lds;
  return lds <= kLds;
}

ecw_status launch_few(hipStream_t stream, const Fp8GemmArgs& a, const FewShape& f, int y_dtype) {
  const uint32_t groups = (a.rows + 15) / 16;
  // as many blocks as the card holds at once, each with as many groups as the others
  const uint32_t most = kCus * std::min(kLds / f.lds, 2048 / (64 * kFewWaves)), rounds = (groups + most - 1) / most;
  const uint32_t grid = (groups + rounds - 1) / rounds;
  if (f.lds > 64 * 1024) {  // to be allowed once on each device
    static std::atomic<uint64_t> allowed{0};
    int device = 0;
    const bool known = hipGetDevice(&device) == hipSuccess && device >= 0 && device < 64;
    if (!known || !(allowed.load(std::memory_order_relaxed) >> device & 1)) {
      if (hipFuncSetAttribute(reinterpret_cast<const void*>(k_fp8_gemm_few), hipFuncAttributeMaxDynamicSharedMemorySize,
                              (int)kLds) != hipSuccess) {
        (void)hipGetLastError();
        return refuse(ECW_E_HIP, "hipFuncSetAttribute failed");
      }
      if (known) allowed.fetch_or(uint64_t(1) << device, std::memory_order_relaxed);
    }
  }
  hipLaunchKernelGGL(k_fp8_gemm_few, dim3(grid), dim3(64 * kFewWaves), f.lds, stream, a, f, y_dtype);
  return launched("fp8_gemm");
}

template <int WM, int WN, int TM, int TN, int NS, int KG, bool EXACT>
ecw_status launch_tile(hipStream_t stream, const Fp8GemmArgs& a, int y_dtype) {
  using T = Fp8Tiles<WM, WN, TM, TN, NS, KG>;
  const uint32_t m_tiles = (a.batch + T::BM - 1) / T::BM, n_tiles = (a.rows + T::BN - 1) / T::BN;
  if (!launchable((uint64_t)m_tiles * n_tiles * a.splits, 64 * T::kWaves * KG))
    return refuse(ECW_E_UNSUPPORTED, "product too large for one launch");
  hipLaunchKernelGGL((k_fp8_gemm_tile<WM, WN, TM, TN, NS, KG, EXACT>), dim3(m_tiles * n_tiles, a.splits),
                     dim3(64 * T::kWaves * KG), 0, stream, a, m_tiles, n_tiles, y_dtype);
  return launched("fp8_gemm");
}

// The tiles that there are: rows of x and of w, spans at once, and what a span takes, in us,
// with every CU at work (8192 x 8192 x 8192: 1675, 1151, 799, 747, 530 and 443 us; by the
// bf16 instruction 1473, 1053, 929 and 830).
struct TileKind {
  uint32_t bm, bn, kg;
  float span;
};
constexpr TileKind kFast[] = {{32, 64, 2, 0.205f}, {64, 64, 2, 0.281f}, {64, 128, 2, 0.39f},
                              {128, 128, 2, 0.73f}, {128, 256, 1, 1.035f}, {256, 256, 1, 1.73f}};
constexpr TileKind kExact[] = {{64, 64, 4, 0.36f}, {128, 128, 2, 1.03f}, {128, 256, 1, 1.81f}, {256, 256, 1, 3.24f}};

ecw_status launch_kind(hipStream_t st, const Fp8GemmArgs& a, uint32_t kind, bool exact, int dt) {
  if (exact) switch (kind) {
      case 0: return launch_tile<2, 2, 2, 2, 2, 4, true>(st, a, dt);
      case 1: return launch_tile<2, 4, 4, 2, 2, 2, true>(st, a, dt);
      case 2: return launch_tile<2, 4, 4, 4, 3, 1, true>(st, a, dt);
      default: return launch_tile<2, 4, 8, 4, 2, 1, true>(st, a, dt);
    }
  switch (kind) {
    case 0: return launch_tile<1, 4, 2, 1, 4, 2, false>(st, a, dt);
    case 1: return launch_tile<1, 4, 4, 1, 3, 2, false>(st, a, dt);
    case 2: return launch_tile<1, 4, 4, 2, 3, 2, false>(st, a, dt);
    case 3: return launch_tile<2, 4, 4, 2, 2, 2, false>(st, a, dt);
    case 4: return launch_tile<2, 4, 4, 4, 3, 1, false>(st, a, dt);
    default: return launch_tile<2, 4, 8, 4, 2, 1, false>(st, a, dt);
  }
}

// A product in tiles: of which kind, and into how many parts its columns are cut.  Chosen by
// an estimate of the time: rounds of tiles over the CUs, each a start and its spans, and with
// parts their sums through memory and a second launch.
struct Plan {
  uint32_t kind, splits, chunk;
  float us;
};
template <size_t N>
Plan plan_tiles(const TileKind (&kinds)[N], uint32_t batch, uint32_t rows, uint32_t spans, bool splittable) {
  Plan best{0, 1, spans, 1e30f};
  for (uint32_t k = 0; k < N; ++k) {
    const TileKind& t = kinds[k];
    const uint64_t tiles = (uint64_t)((batch + t.bm - 1) / t.bm) * ((rows + t.bn - 1) / t.bn);
    uint32_t parts = 1;
    if (splittable && tiles < kCus) parts = std::max<uint32_t>(1, std::min<uint32_t>(kCus / (uint32_t)tiles, spans / (2 * t.kg)));
    for (uint32_t p : {1u, parts}) {
      const uint32_t chunk = ((spans + p - 1) / p + t.kg - 1) / t.kg * t.kg, splits = (spans + chunk - 1) / chunk;
      const uint64_t rounds = (tiles * splits + kCus - 1) / kCus;
      float us = rounds * (1.f + std::min(chunk, spans) * t.span) + 1.5f;
      if (splits > 1) us += 2.f + (float)splits * batch * rows * 3.5e-6f;
      if (us < best.us) best = {k, splits, chunk, us};
    }
  }
  return best;
}
Plan plan_tiles(uint32_t batch, uint32_t rows, uint32_t spans, bool exact, bool splittable = true) {
  return exact ? plan_tiles(kExact, batch, rows, spans, splittable) : plan_tiles(kFast, batch, rows, spans, splittable);
}

// Rows of w whose tiles fill the CUs for whole rounds, if the rest is better off in tiles of
// another kind (4096 rows by 14336 x 4096 with short sums: 896 tiles are three and a half
// rounds, 222 us, cut 214); else 0.  A second launch starts when the first has ended, which costs about 10 us
// (1500 rows by 16384 x 2048 64.5 us cut, 60.5 not).
uint32_t plan_cut(const Plan& p, uint32_t batch, uint32_t rows, uint32_t spans, bool exact) {
  const TileKind& t = exact ? kExact[p.kind] : kFast[p.kind];
  const uint64_t m = (batch + t.bm - 1) / t.bm, n = (rows + t.bn - 1) / t.bn, full = m * n / kCus;
  if (p.splits > 1 || full == 0 || m * n % kCus == 0) return 0;
  const uint64_t first = full * kCus / m;
  if (first == 0 || first >= n) return 0;
  const uint32_t cut = (uint32_t)(first * t.bn);
  const Plan rest = plan_tiles(batch, rows - cut, spans, exact, false);
  return full * (1.f + spans * t.span) + 1.5f + rest.us + 10.f < p.us ? cut : 0;
}

uint64_t part_size(uint32_t batch, uint32_t rows) { return ((uint64_t)batch * rows + 3) / 4 * 4; }

ecw_status check_product(uint32_t rows, uint32_t cols, uint32_t batch, int y_dtype) {
  if (cols == 0 || cols > (1u << 30) || rows > (1u << 30)) return refuse(ECW_E_INVALID_ARG, "cols must be in [1, 2^30], rows at most 2^30");
  if (batch > (1u << 24)) return refuse(ECW_E_INVALID_ARG, "batch must be at most 2^24");
  const int dt = y_dtype & ~ECW_FP8_SHORT_SUMS;
  if (!is_float(dt)) return refuse(ECW_E_INVALID_ARG, "y dtype must be F16, BF16 or F32");
  if (dt != y_dtype && dt == ECW_DT_F32) return refuse(ECW_E_INVALID_ARG, "short sums are for F16 and BF16 outputs");
  return ECW_OK;
}

}  // namespace

extern "C" {

ecw_status fp8_gemm_workspace_size(uint32_t rows, uint32_t cols, uint32_t batch, int y_dtype, size_t* bytes) {
  if (!bytes) return refuse(ECW_E_INVALID_ARG, "bytes is NULL");
  *bytes = 0;
  if (ecw_status s = check_product(rows, cols, batch, y_dtype)) return s;
  if (rows == 0 || batch == 0) return ECW_OK;
  FewShape f;
  const uint32_t spans = fp8_row(cols) / 128;
  if (few_shape(batch, spans, &f)) return ECW_OK;
  const Plan p = plan_tiles(batch, rows, spans, !(y_dtype & ECW_FP8_SHORT_SUMS));
  if (p.splits > 1) *bytes = p.splits * part_size(batch, rows) * sizeof(float);
  return ECW_OK;
}

ecw_status fp8_gemm(ecw_stream stream, const void* w_codes, const void* w_scales, uint32_t rows, uint32_t cols,
                    const void* x_codes, const void* x_scales, uint32_t batch, void* y, int y_dtype, void* workspace,
                    size_t workspace_bytes) {
  if (ecw_status s = check_product(rows, cols, batch, y_dtype)) return s;
  if (ecw_status s = check_fp8(w_codes, w_scales, rows, cols)) return s;
  if (ecw_status s = check_fp8(x_codes, x_scales, batch, cols)) return s;
  if (rows == 0 || batch == 0) return ECW_OK;
  if (!y || !aligned(y, 16)) return refuse(ECW_E_INVALID_ARG, "y must be a 16-byte aligned device pointer");
  Fp8GemmArgs a{static_cast<const uint8_t*>(w_codes), static_cast<const uint8_t*>(w_scales),
                static_cast<const uint8_t*>(x_codes), static_cast<const uint8_t*>(x_scales), y, rows, batch,
                fp8_row(cols), fp8_scale_row(cols), fp8_row(cols) / 128, rows, 1, fp8_row(cols) / 128, nullptr, 0};
  const auto st = (hipStream_t)stream;
  const bool exact = !(y_dtype & ECW_FP8_SHORT_SUMS);
  y_dtype &= ~ECW_FP8_SHORT_SUMS;
  FewShape f;
  if (few_shape(batch, a.spans, &f)) return launch_few(st, a, f, y_dtype);
  const Plan p = plan_tiles(batch, rows, a.spans, exact);
  if (p.splits > 1) {
    a.splits = p.splits, a.chunk = p.chunk, a.part_size = part_size(batch, rows);
    if (!workspace || !aligned(workspace, 16)) return refuse(ECW_E_INVALID_ARG, "the workspace must be a 16-byte aligned device pointer");
    if (workspace_bytes < a.splits * a.part_size * sizeof(float)) return refuse(ECW_E_BUFFER_TOO_SMALL, "workspace too small");
    a.part = static_cast<float*>(workspace);
    if (ecw_status s = launch_kind(st, a, p.kind, exact, y_dtype)) return s;
    const uint64_t all = (uint64_t)batch * rows, grid = (all + 1023) / 1024;
    auto* fn = y_dtype == ECW_DT_F32   ? k_fp8_gemm_join<ECW_DT_F32>
               : y_dtype == ECW_DT_F16 ? k_fp8_gemm_join<ECW_DT_F16>
                                       : k_fp8_gemm_join<ECW_DT_BF16>;
    hipLaunchKernelGGL(fn, dim3((uint32_t)grid), dim3(256), 0, st, a.part, y, all, a.part_size, a.splits);
    return launched("fp8_gemm");
  }
  if (const uint32_t cut = plan_cut(p, batch, rows, a.spans, exact)) {
    Fp8GemmArgs rest = a;
    rest.rows = rows - cut;
    rest.w += (uint64_t)cut * a.row, rest.ws += (uint64_t)cut * a.scale_row;
    rest.y = static_cast<uint8_t*>(y) + (uint64_t)cut * size_of(y_dtype);
    a.rows = cut;
    if (ecw_status s = launch_kind(st, a, p.kind, exact, y_dtype)) return s;
    return launch_kind(st, rest, plan_tiles(batch, rest.rows, a.spans, exact, false).kind, exact, y_dtype);
  }
  return launch_kind(st, a, p.kind, exact, y_dtype);
}

}  // extern "C"
