// y[b][n] = sum_k x[b][k] w[n][k] with w in the microscaled 4-bit format, and x either
// 16-bit floats or in the same format.
//
// Matrix instructions take w as it lies in memory.  A wave reads 16 rows of w over a
// span of 128 columns as one 16-byte load per lane: lane l has row l % 16 and block
// l / 16 of the span, 32 codes, which is the operand of the scaled 4-bit instruction
// (16x16x128).  For 16-bit x the order of k inside an instruction is free as long as
// both operands agree, so word j of the 16 bytes is the operand of the j-th 16x16x32
// instruction: its lanes cover columns 32 (l / 16) + 8 j .. + 7.
//
// Sums are held in fp32.  4-bit values times a power of two are exact in bf16, so bf16
// x needs no rounding.  In fp16 they are exact relative to the span's largest scale
// when its scales span at most 2^23 (0.5 * 2^-23 is fp16's smallest number); the
// span's sum is multiplied by that scale in fp32.  A wider span takes further passes
// (2^40 apart in every span, 1003 rows by 14336 x 4096: 306 us, close ones 157).
#include <atomic>
#include <type_traits>

#include "mx4_common.h"

namespace ecw {

constexpr int kActMX4 = 0;  // x in the 4-bit format; else ECW_DT_F16 or ECW_DT_BF16

struct GemmArgs {
  const uint8_t* w;       // codes, 16 bytes a block
  const uint8_t* ws;      // scale bytes
  const void* x;          // 16-bit rows, or codes
  const uint8_t* xs;      // scale bytes of 4-bit x
  void* y;
  int64_t x_stride;       // elements (16-bit x)
  uint32_t rows, cols, batch;
  uint32_t blocks, scales;  // of a padded row: blocks of codes, bytes of scales
};

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

// the largest and smallest byte of a word
__device__ __forceinline__ void byte_range(uint32_t w, uint32_t* lo, uint32_t* hi) {
  const uint32_t a = w & 255, b = w >> 8 & 255, c = w >> 16 & 255, d = w >> 24;
  *hi = max(max(a, b), max(c, d));
  *lo = min(min(a, b), min(c, d));
}
// a word without its bytes of `from` or more
__device__ __forceinline__ uint32_t bytes_below(uint32_t w, uint32_t from) {
  uint32_t r = 0;
#pragma unroll
  for (int i = 0; i < 32; i += 8)
    if ((w >> i & 255) < from) r |= w & 255u << i;
  return r;
}

// acc[t] += x tile t times codes w of scale s, summed apart and then multiplied by the scale
// `top` of the lane's row of w, its column of the result.
template <int NT>
__device__ __forceinline__ void add_pass(f32x4 (&acc)[NT], u32x4 w, float s, float top, const u32x4 (&x)[NT][4]) {
  f32x4 sum[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) sum[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const f16x8 b = oct_f16(w[j], s);
#pragma unroll
    for (int t = 0; t < NT; ++t)
      sum[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, x[t][j]), b, sum[t], 0, 0, 0);
  }
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r) acc[t][r] = fmaf(sum[t][r], top, acc[t][r]);
}

// One span in which some of a wave's 16 rows of w have scales more than 2^23 apart, or a NaN
// block: a pass for each group of blocks within 2^23 of the largest left, the others as
// zeros.  An infinity in x makes NaN of such a zero, in every row: where NaN came out, the
// span is multiplied once more, in bf16, which holds w whole, with x as the sum of two bf16
// numbers.  Loops are not unrolled: this is seldom reached, and the code next to it has to
// stay in the instruction cache.
template <int NT>
__device__ __forceinline__ void span_product_far(f32x4 (&acc)[NT], u32x4 w, uint32_t sw, uint32_t g,
                                                 const u32x4 (&x)[NT][4]) {
  const uint32_t mine = sw >> 8 * g & 255;
  f32x4 sum[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) sum[t] = f32x4{0.f, 0.f, 0.f, 0.f};
  bool nan = mine == kScaleNaN;
  uint32_t left = bytes_below(sw, kScaleNaN);
#pragma unroll 1
  do {
    uint32_t lo, hi;
    byte_range(left, &lo, &hi);
    const uint32_t my = left >> 8 * g & 255;
    const bool in = my != 0 && my + 23 >= hi;
    add_pass(sum, nan || in ? w : u32x4{0, 0, 0, 0}, scale_of(nan ? kScaleNaN : in ? my + kScaleOne - hi : kScaleOne),
             scale_of(hi), x);
    nan = false;
    left = bytes_below(left, hi > 23 ? hi - 23 : 0);
  } while (__any(left != 0));
  bool again = false;
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r) again |= sum[t][r] != sum[t][r];
  if (__any(again)) {
#pragma unroll
    for (int t = 0; t < NT; ++t) sum[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
    for (int j = 0; j < 4; ++j) {
      auto pick = [j](auto a, auto b, auto c, auto d) { return j < 2 ? (j == 0 ? a : b) : j == 2 ? c : d; };
      const bf16x8 b = oct_bf16(pick(w[0], w[1], w[2], w[3]), scale_of(mine));
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        bf16x8 high, low;
        split_f16(pick(x[t][0], x[t][1], x[t][2], x[t][3]), &high, &low);
        sum[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(high, b, sum[t], 0, 0, 0);
        sum[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(low, b, sum[t], 0, 0, 0);
      }
    }
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) acc[t] += sum[t];
}

// acc[t] += x tile t (rows: 16 of x) times a wave's 16 rows of w over one span.
// w: the lane's block; sw: the span's four scale bytes; x[t][j]: the lane's columns.
template <int ACT, int NT>
__device__ __forceinline__ void span_product(f32x4 (&acc)[NT], u32x4 w, uint32_t sw, uint32_t g,
                                             const u32x4 (&x)[NT][4]) {
  if constexpr (ACT == ECW_DT_BF16) {
    const float s = scale_of(sw >> 8 * g & 255);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bf16x8 b = oct_bf16(w[j], s);
#pragma unroll
      for (int t = 0; t < NT; ++t)
        acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x[t][j]), b, acc[t], 0, 0, 0);
    }
  } else {
    const uint32_t mine = sw >> 8 * g & 255;
    uint32_t lo, hi;
    byte_range(sw, &lo, &hi);
    if (__builtin_expect(!__any(hi - lo > 23 || hi == kScaleNaN), 1))
      add_pass(acc, w, scale_of(mine + kScaleOne - hi), scale_of(hi), x);
    else
      span_product_far(acc, w, sw, g, x);
  }
}

__device__ __forceinline__ f32x4 span_product_mx4(f32x4 acc, u32x4 w, uint32_t sw, uint32_t g, u32x4 x, uint32_t sx) {
  typedef int i32x8 __attribute__((ext_vector_type(8)));
  const i32x8 a = {(int)x[0], (int)x[1], (int)x[2], (int)x[3], 0, 0, 0, 0};
  const i32x8 b = {(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, acc, 4, 4, 0, (int)(sx >> 8 * g), 0,
                                                          (int)(sw >> 8 * g));
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

__device__ const u32x4 zeros16 = {0, 0, 0, 0};

// Eight elements of a row of x from column c on come from column min(c, cols - 8), so that
// they lie in the row wherever it starts and ends; in a row's last span they are moved
// down by what is too much, with zeros behind them.
__device__ __forceinline__ uint32_t within(uint32_t c, uint32_t cols) { return min(c, cols - 8); }
__device__ __forceinline__ u32x4 moved_down(u32x4 v, uint32_t elements) {
  const unsigned __int128 t = __builtin_bit_cast(unsigned __int128, v);
  return __builtin_bit_cast(u32x4, elements < 8 ? t >> (16 * elements) : (unsigned __int128)0);
}

// ------------------------------------------------------------------ a few rows
// A block computes 16 rows of w times up to 16 rows of x; its waves take pairs of spans in
// turn and join their sums through LDS, in the order of the waves.  A wave copies w for up
// to four turns straight to LDS, 8 rows of 128 bytes at a time, so that neighbouring lanes
// read whole lines: as operands they would be 16-byte pieces of 16 rows.  16 bytes at
// piece p of row r's 8 lie at p ^ stirred(r), so that the 16 lanes that LDS serves together
// meet no bank twice.  The first turn's x is asked for before w, later turns' one turn
// ahead: behind w in a CU's queue, x took 1 us more for one row by 14336 x 4096 (9.2 us with
// the 31 MB of w in the last-level cache, 12.0 from memory).  Bound by reading w.
__device__ __forceinline__ uint32_t stirred(uint32_t r) { return ((r >> 1) + 2) & 7; }

constexpr uint32_t kTurns = 4;             // pairs of spans that a wave has in LDS
constexpr uint32_t kTurnBytes = 16 * 128;  // 16 rows of w
constexpr uint32_t kFewWaves = 16;         // at most

// NEAR: 16-bit x ends within 2^31 bytes.  Its rows may start at any element (one row by
// 14336 x 4095: 9.0 and 12.0 us too).
template <int ACT, bool NEAR>
__global__ void __launch_bounds__(64 * kFewWaves) k_mx4_gemm_few(GemmArgs a, int y_dtype) {
  extern __shared__ __align__(16) uint8_t lds[];  // each wave's turns, then (over them) the sums
  const uint32_t base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;
  const uint32_t lane = threadIdx.x & 63, waves = blockDim.x >> 6;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t r16 = lane & 15, g = lane >> 4;
  const uint32_t n0 = blockIdx.x * 16;
  const uint32_t spans = a.blocks / 4, pairs = (spans + 1) / 2;

  const uint8_t* from[2];  // the lane's 16 bytes of rows 0-7 and 8-15, in pair 0
  bool late[2];            // whether they are of the pair's second span
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t row = i * 8 + (lane >> 3), piece = (lane & 7) ^ stirred(row);
    from[i] = a.w + (uint64_t)min(n0 + row, a.rows - 1) * a.blocks * 16 + piece * 16;
    late[i] = piece >= 4;
  }
  const uint8_t* ws = a.ws + (uint64_t)min(n0 + r16, a.rows - 1) * a.scales;
  const uint64_t m = min(r16, a.batch - 1);
  const uint8_t* xrow = static_cast<const uint8_t*>(a.x) + (ACT == kActMX4 ? m * a.blocks * 16 : (int64_t)m * a.x_stride * 2);
  const uint8_t* xs = ACT == kActMX4 ? a.xs + m * a.scales : nullptr;
  constexpr int kWords = ACT == kActMX4 ? 1 : 4;
  // 16-bit x as a buffer of bytes: what is past its end, rows there are not, reads as zero
  // and fetches nothing
  const auto xbuf = __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(a.x), 0,
                                                      (uint32_t)(((a.batch - 1) * a.x_stride + a.cols) * 2), 0x00027000);
  const uint32_t xoff = r16 < a.batch ? (uint32_t)(r16 * a.x_stride * 2) : 1u << 31;
  struct Span {
    u32x4 x[1][kWords];
    uint32_t sx;
  };
  // the operands of x in span s; past the last span nothing is fetched, or the last again
  auto load_x = [&](Span& to, uint32_t s) {
    const uint32_t row = s < spans ? xoff : 1u << 31;
    s = min(s, spans - 1);
    if constexpr (ACT == kActMX4) {
      to.x[0][0] = *reinterpret_cast<const u32x4*>(xrow + (uint64_t)s * 64 + g * 16);
      to.sx = *reinterpret_cast<const uint32_t*>(xs + s * 4);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t c = within(s * 128 + g * 32 + j * 8, a.cols);
        if constexpr (NEAR)
          to.x[0][j] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(xbuf, row + c * 2, 0, 0));
        else
          to.x[0][j] = reinterpret_cast<const Loose16*>(xrow + (uint64_t)c * 2)->v;
      }
    }
  };

  f32x4 acc[1] = {f32x4{0.f, 0.f, 0.f, 0.f}};
  for (uint32_t first = wave; first < pairs; first += waves * kTurns) {
    u32x2 sw[kTurns];
#pragma unroll
    for (uint32_t k = 0; k < kTurns; ++k)
      sw[k] = *reinterpret_cast<const u32x2*>(ws + min(first + k * waves, pairs - 1) * 8);
    Span x[2];
#pragma unroll
    for (uint32_t h = 0; h < 2; ++h) load_x(x[h], first * 2 + h);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (uint32_t k = 0; k < kTurns; ++k) {
      const uint32_t p = first + k * waves;
      if (p < pairs) {
        // an odd last span has no second half to copy: those lanes copy the first again
        const uint32_t half = p * 2 + 1 < spans ? 0 : 64;
#pragma unroll
        for (int i = 0; i < 2; ++i)
          to_lds(from[i] + (uint64_t)p * 128 - (late[i] ? half : 0),
                     base + (wave * kTurns + k) * kTurnBytes + i * 1024);
      }
    }
    wait_copies<0>();
#pragma unroll
    for (uint32_t k = 0; k < kTurns; ++k) {
#pragma unroll
      for (uint32_t h = 0; h < 2; ++h) {
        const uint32_t s = (first + k * waves) * 2 + h;
        Span& now = x[h];
        const u32x4 wv = *reinterpret_cast<const u32x4*>(lds + (wave * kTurns + k) * kTurnBytes + r16 * 128 +
                                                         ((h * 4 + g) ^ stirred(r16)) * 16);
        if (s < spans) {
          if constexpr (ACT == kActMX4) {
            acc[0] = span_product_mx4(acc[0], wv, sw[k][h], g, now.x[0][0], now.sx);
          } else {
            if (s + 1 == spans) {
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const uint32_t c = s * 128 + g * 32 + j * 8;
                now.x[0][j] = moved_down(now.x[0][j], c - within(c, a.cols));
              }
            }
            span_product<ACT, 1>(acc, wv, sw[k][h], g, now.x);
          }
        }
        if (k + 1 < kTurns) load_x(now, (first + (k + 1) * waves) * 2 + h);
      }
    }
    wait_copies<0>();  // this wave's reads of LDS are done before it copies again
  }
  __syncthreads();
  f32x4* part = reinterpret_cast<f32x4*>(lds);  // [waves][64]
  part[wave * 64 + lane] = acc[0];
  __syncthreads();
  // lane l: rows 4 (l / 16) .. + 3 of x, row l % 16 of w
  if (wave == 0) {
    f32x4 sum = part[lane];
    for (uint32_t v = 1; v < waves; ++v) sum += part[v * 64 + lane];
    with_type(y_dtype, [&](auto dt) {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (n0 + r16 < a.rows && g * 4 + r < a.batch)
          store_y<dt.value>(a.y, (uint64_t)(g * 4 + r) * a.rows + n0 + r16, sum[r]);
    });
  }
}

// Rows of up to 8 columns: an output per lane.  Bound by instructions (4096 rows by 14336
// x 7 265 us).
template <int ACT>
__global__ void __launch_bounds__(256) k_mx4_gemm_narrow(GemmArgs a, int y_dtype) {
  const uint64_t at = (uint64_t)blockIdx.x * 256 + threadIdx.x, b = at / a.rows, n = at - b * a.rows;
  if (b >= a.batch) return;
  const bf16x8 w = oct_bf16(*reinterpret_cast<const uint32_t*>(a.w + n * a.blocks * 16), scale_of(a.ws[n * a.scales]));
  const int64_t row = (int64_t)b * a.x_stride;
  float sum = 0.f;
#pragma unroll
  for (uint32_t c = 0; c < 8; ++c) {
    if (c >= a.cols) break;
    float x;
    if constexpr (ACT == ECW_DT_F16)
      x = (float)static_cast<const _Float16*>(a.x)[row + c];
    else
      x = (float)static_cast<const __bf16*>(a.x)[row + c];
    sum = fmaf(x, (float)w[c], sum);
  }
  with_type(y_dtype, [&](auto dt) { store_y<dt.value>(a.y, at, sum); });
}

// ------------------------------------------------------------------ many rows
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

// Where a row's 16 column octets of a span lie in LDS: octet o of row r at place
// turned(o) ^ (r % 16), so that neither a row written nor a column read by 16 lanes meets
// a bank twice (LDS serves lanes 0-3, 12-15 and 20-27 of a wave together).
__device__ __forceinline__ uint32_t turned(uint32_t o) { return (o & 3) * 4 + (o >> 2); }

// 16 rows of 4 bits of a span are 1 KiB in LDS: row r's block b at place 4 r + (b ^
// shifted(r)), so that four neighbouring lanes copy 64 neighbouring bytes and the 16
// lanes that LDS serves together meet no bank twice.
__device__ __forceinline__ uint32_t shifted(uint32_t r) { return (0u - (r >> 2)) & 3; }

// A block of WM x WN waves multiplies 16 TM WM rows of x and 16 TN WN rows of w, a span
// at a time, from NS stages in LDS that copies fill ahead.  EARLY: a wave reads a span's
// operands from LDS while it multiplies the span before.  Scales come for four spans at
// once, into places of their own.
//
// LOOSE: rows of x start at any element, which copies cannot: they come through registers,
// asked for a step before they are written to LDS (more steps gained nothing; bound by
// loads that no 16 bytes are aligned for: 32 rows by 4096 x 14335 38 us).
//
// KG: a block has KG times the waves, which take KG spans at once and add their sums up at
// the end, in order.  With one wave a SIMD every instruction waits for the one before (64
// rows by 4096 x 14336 in 64x64 with KG 1 and 2 65 and 42 us, 32 rows in 32x64 with KG 1, 2
// and 4 42, 28 and 24).
//
// The large tiles are bound by LDS, which serves operands for about as long as the matrix
// instructions take and the copies' writes next to them (1003 rows by 4096 x 4096, in a
// graph: bf16 x 41 us, 820 TFLOP/s, fp16 50, whose spans' scales are vector instructions;
// 4-bit x, 4096 rows by 14336 x 4096 174 us, 2.76 PFLOP/s, of which the outputs' stores are
// a third).
template <int ACT, int WM, int WN, int TM, int TN, int NS, bool EARLY, bool LOOSE, int KG>
struct Tiles {
  static constexpr bool kX4 = ACT == kActMX4;
  static constexpr int kWaves = WM * WN, BM = 16 * TM * WM, BN = 16 * TN * WN;
  static constexpr uint32_t kX = kX4 ? BM * 64 : BM * 256, kW = BN * 64, kSpan = kX + kW, kStage = KG * kSpan;
  static constexpr uint32_t kScaleRows = (kX4 ? BM : 0) + BN;  // those of x first
  static constexpr uint32_t kScalePlaces = (NS * KG + 3) / 4 + 1;
  static constexpr uint32_t kBytes = kStage * NS + kScalePlaces * kScaleRows * 16;
  static constexpr int kXLoads = kX / 1024 / kWaves, kWLoads = kW / 1024 / kWaves;  // copies per wave and span
  static constexpr int kSLoads = (kScaleRows / 64 + kWaves - 1) / kWaves;           // per four spans
  static_assert(kX % (1024 * kWaves) == 0 && kW % (1024 * kWaves) == 0, "");
  static_assert(kBytes <= 160 * 1024, "");
  static_assert(4 % KG == 0, "");                                            // a step's scales come together
  static_assert((KG - 1) * kWaves * TM * TN * 1024 <= (int)kStage * NS, "");  // sums of the other groups
};

// Two 4-bit operands are multiplied the other way round, w's rows down the result's
// registers, and row i of a wave's tile t stands for its row 4 TN (i / 4) + 4 t + i % 4:
// a lane then holds 4 TN neighbouring outputs of one row of x, four lanes a whole line.
// (With one 2-byte store per output the stores took 78 of 205 us at 4096 x 14336 x 4096.)
template <int TN>
__device__ __forceinline__ uint32_t spread(uint32_t t, uint32_t i) {
  return (i >> 2) * (4 * TN) + t * 4 + (i & 3);
}

template <int DT, int N>
__device__ __forceinline__ void store_run(void* y, uint64_t at, const float (&v)[N], uint32_t left, bool vec) {
  if (vec && left >= N) {
    if constexpr (DT == ECW_DT_F32) {
#pragma unroll
      for (int i = 0; i < N; i += 4)
        *reinterpret_cast<f32x4*>(static_cast<float*>(y) + at + i) = f32x4{v[i], v[i + 1], v[i + 2], v[i + 3]};
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
        for (int i = 0; i < N / 2; i += 4)
          *reinterpret_cast<u32x4*>(o + 2 * i) = u32x4{w[i], w[i + 1], w[i + 2], w[i + 3]};
      } else {
        static_assert(N == 4, "");
        *reinterpret_cast<u32x2*>(o) = u32x2{w[0], w[1]};
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < N; ++i)
    if ((uint32_t)i < left) store_y<DT>(y, at + i, v[i]);
}

template <int ACT, int WM, int WN, int TM, int TN, int NS, bool EARLY, bool LOOSE, int KG>
__global__ void __launch_bounds__(64 * WM * WN * KG) k_mx4_gemm_tile(GemmArgs a, uint32_t m_tiles, uint32_t n_tiles,
                                                                int y_dtype) {
  using T = Tiles<ACT, WM, WN, TM, TN, NS, EARLY, LOOSE, KG>;
  __shared__ __align__(16) uint8_t lds[T::kBytes];
  const uint32_t base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;
  const uint32_t lane = threadIdx.x & 63, waves = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t kg = waves / T::kWaves, wave = waves % T::kWaves;
  const uint32_t r16 = lane & 15, g = lane >> 4;
  uint32_t mt, nt;
  tile_of(m_tiles, n_tiles, &mt, &nt);
  const uint32_t m0 = mt * T::BM, n0 = nt * T::BN, spans = a.blocks / 4;
  const uint32_t steps = (spans + KG - 1) / KG;

  const uint8_t *xp[T::kXLoads], *wp[T::kWLoads], *sp[T::kSLoads];
  const uint32_t r4 = lane >> 2, b4 = (lane & 3) ^ shifted(r4);  // row and block that the lane copies of 16 rows
#pragma unroll
  for (int i = 0; i < T::kXLoads; ++i) {
    const uint32_t part = wave * T::kXLoads + i;  // 1 KiB: 16 rows of 4 bits, or 4 rows of 16 bits
    if constexpr (T::kX4) {
      xp[i] = static_cast<const uint8_t*>(a.x) + (uint64_t)min(m0 + part * 16 + r4, a.batch - 1) * a.blocks * 16 + b4 * 16;
    } else {
      const uint32_t row = part * 4 + g;
      const uint32_t oct = LOOSE ? 0 : turned(r16 ^ (row & 15));
      xp[i] = static_cast<const uint8_t*>(a.x) + (int64_t)min(m0 + row, a.batch - 1) * a.x_stride * 2 + oct * 16;
    }
  }
#pragma unroll
  for (int i = 0; i < T::kWLoads; ++i) {
    const uint32_t part = wave * T::kWLoads + i;
    const uint32_t row = T::kX4 ? part / TN * (16 * TN) + spread<TN>(part % TN, r4) : part * 16 + r4;
    wp[i] = a.w + (uint64_t)min(n0 + row, a.rows - 1) * a.blocks * 16 + b4 * 16;
  }
#pragma unroll
  for (int i = 0; i < T::kSLoads; ++i) {
    const uint32_t row = (wave + i * T::kWaves) * 64 + lane;
    if (T::kX4 && row < T::BM)
      sp[i] = a.xs + (uint64_t)min(m0 + row, a.batch - 1) * a.scales;
    else
      sp[i] = a.ws + (uint64_t)min(n0 + row - (T::kX4 ? T::BM : 0), a.rows - 1) * a.scales;
  }

  // Rows at an odd element: eight elements from the second on, in whole words, and the
  // first (16 bytes that start between two words take three times as long).
  struct Held {
    u32x4 v;
    uint32_t first;
  };
  Held held[LOOSE ? T::kXLoads : 1];
  auto odd = [&](int i) { return (uint32_t)(reinterpret_cast<uintptr_t>(xp[i]) >> 1 & 1); };
  auto column = [&](uint32_t span, int i) {
    return span * 128 + turned(r16 ^ (((wave * T::kXLoads + i) * 4 + g) & 15)) * 8;
  };
  auto ask = [&](uint32_t span) {
#pragma unroll
    for (int i = 0; i < T::kXLoads; ++i) {
      const uint16_t* from = reinterpret_cast<const uint16_t*>(xp[i]) +
                             within(column(min(span, spans - 1), i), a.cols - odd(i));
      held[i].first = *from;
      held[i].v = reinterpret_cast<const Words*>(from + odd(i))->v;
    }
  };

  // copies of one step's span into a stage; past the last span the last one again, into a
  // place that is not multiplied, so that every turn waits for the same number
  auto fill = [&](uint32_t step, uint32_t stage) {
    const uint32_t span = step * KG + kg;
    const uint64_t s = min(span, spans - 1);
    if (kg == 0 && span % 4 == 0 && span < spans) {
#pragma unroll
      for (int i = 0; i < T::kSLoads; ++i) {
        const uint32_t part = wave + i * T::kWaves;
        if (part < T::kScaleRows / 64)
          to_lds(sp[i] + s * 4, base + T::kStage * NS + (span / 4 % T::kScalePlaces) * T::kScaleRows * 16 + part * 1024);
      }
    }
    const uint32_t to = base + stage * T::kStage + kg * T::kSpan;
    if constexpr (LOOSE) {
#pragma unroll
      for (int i = 0; i < T::kXLoads; ++i) {
        u32x4 v = held[i].v;
        if (odd(i))
          v = u32x4{held[i].first | v[0] << 16, v[0] >> 16 | v[1] << 16, v[1] >> 16 | v[2] << 16, v[2] >> 16 | v[3] << 16};
        if (span + 1 == spans) {
          const uint32_t more = column(span, i) - within(column(span, i), a.cols - odd(i));
          if (more) v = moved_down(held[i].v, more - odd(i));
        }
        reinterpret_cast<u32x4*>(lds + stage * T::kStage + kg * T::kSpan)[(wave * T::kXLoads + i) * 64 + lane] = v;
      }
      ask(span + KG);
    }
#pragma unroll
    for (int i = 0; i < (LOOSE ? 0 : T::kXLoads); ++i) {
      const uint32_t part = wave * T::kXLoads + i;
      const uint8_t* from = xp[i] + s * (T::kX4 ? 64 : 256);
      if constexpr (!T::kX4) {
        const uint32_t oct = turned(r16 ^ ((part * 4 + g) & 15));
        if ((uint32_t)s * 128 + oct * 8 >= a.cols) from = reinterpret_cast<const uint8_t*>(&zeros16);
      }
      to_lds(from, to + part * 1024);
    }
#pragma unroll
    for (int i = 0; i < T::kWLoads; ++i) to_lds(wp[i] + s * 64, to + T::kX + (wave * T::kWLoads + i) * 1024);
  };

  f32x4 acc[TN][TM];
#pragma unroll
  for (int n = 0; n < TN; ++n)
#pragma unroll
    for (int m = 0; m < TM; ++m) acc[n][m] = f32x4{0.f, 0.f, 0.f, 0.f};
  const uint32_t wm = wave / WN * TM, wn = wave % WN * TN;  // first 16-row tiles of the wave
  const uint32_t in = r16 * 4 + (g ^ shifted(r16));         // the lane's place in 16 rows of 4 bits

  struct Operands {
    u32x4 x[TM][T::kX4 ? 1 : 4], w[TN];
    uint32_t xs[TM], ws[TN];
  };
  auto read = [&](Operands& f, uint32_t step, uint32_t stage) {
    const uint32_t s = step * KG + kg;
    const uint8_t* at = lds + stage * T::kStage + kg * T::kSpan;
    const u32x4* x = reinterpret_cast<const u32x4*>(at);
    const u32x4* w = reinterpret_cast<const u32x4*>(at + T::kX);
    const uint32_t* xs = reinterpret_cast<const uint32_t*>(lds + T::kStage * NS + (s / 4 % T::kScalePlaces) * T::kScaleRows * 16) + s % 4;
    const uint32_t* ws = xs + (T::kX4 ? T::BM * 4 : 0);
#pragma unroll
    for (int n = 0; n < TN; ++n) {
      f.w[n] = w[(wn + n) * 64 + in];
      f.ws[n] = ws[(T::kX4 ? wn * 16 + spread<TN>(n, r16) : (wn + n) * 16 + r16) * 4];
    }
#pragma unroll
    for (int m = 0; m < TM; ++m) {
      if constexpr (T::kX4) {
        f.x[m][0] = x[(wm + m) * 64 + in];
        f.xs[m] = xs[((wm + m) * 16 + r16) * 4];
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) f.x[m][j] = x[((wm + m) * 16 + r16) * 16 + ((4 * j + g) ^ r16)];
      }
    }
  };
  auto multiply = [&](const Operands& f, uint32_t step) {
    if (KG > 1 && step * KG + kg >= spans) return;
#pragma unroll
    for (int n = 0; n < TN; ++n) {
      if constexpr (T::kX4) {
#pragma unroll
        for (int m = 0; m < TM; ++m)
          acc[n][m] = span_product_mx4(acc[n][m], f.x[m][0], f.xs[m], g, f.w[n], f.ws[n]);
      } else {
        span_product<ACT, TM>(acc[n], f.w[n], f.ws[n], g, f.x);
      }
    }
  };
  constexpr int kCopies = T::kXLoads + T::kWLoads;  // of a step; scales may be among those waited for too
  uint32_t stage = 0;                               // of the step that is multiplied
  if constexpr (LOOSE) ask(kg);
  if constexpr (EARLY) {
    auto turn = [&](uint32_t s, const Operands& now, Operands& next) {
      wait_copies<(NS - 2) * kCopies>();
      __builtin_amdgcn_s_barrier();  // the next step is there, and this one's stage is read
      fill(s + NS, stage);
      stage = stage + 1 == NS ? 0 : stage + 1;
      read(next, s + 1, stage);
      __builtin_amdgcn_sched_barrier(0);
      multiply(now, s);
    };
#pragma unroll
    for (int i = 0; i < NS; ++i) fill(i, i);
    wait_copies<(NS - 1) * kCopies>();
    __builtin_amdgcn_s_barrier();
    Operands even, odd;
    read(even, 0, 0);
    for (uint32_t s = 0; s < steps; s += 2) {
      turn(s, even, odd);
      if (s + 1 == steps) break;
      turn(s + 1, odd, even);
    }
  } else {
#pragma unroll
    for (int i = 0; i < NS - 1; ++i) fill(i, i);
    uint32_t before = NS - 1;  // the stage of the step before
    for (uint32_t s = 0; s < steps; ++s) {
      wait_copies<(NS - 2) * kCopies>();
      __builtin_amdgcn_s_barrier();  // this step is there, and the one before it is done with
      fill(s + NS - 1, before);
      Operands now;
      read(now, s, stage);
      multiply(now, s);
      before = stage;
      stage = stage + 1 == NS ? 0 : stage + 1;
    }
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
  with_type(y_dtype, [&](auto dt) {
    if constexpr (T::kX4) {
      const uint32_t at = n0 + wn * 16 + g * (4 * TN);
      if (at >= a.rows) return;
      const bool vec = a.rows % (dt.value == ECW_DT_F32 ? 4 : 8) == 0;
#pragma unroll
      for (int m = 0; m < TM; ++m) {
        const uint32_t b = m0 + (wm + m) * 16 + r16;
        float v[4 * TN];
#pragma unroll
        for (int n = 0; n < TN; ++n)
#pragma unroll
          for (int r = 0; r < 4; ++r) v[n * 4 + r] = acc[n][m][r];
        if (b < a.batch) store_run<dt.value>(a.y, (uint64_t)b * a.rows + at, v, a.rows - at, vec);
      }
    } else {
#pragma unroll
      for (int n = 0; n < TN; ++n)
#pragma unroll
        for (int m = 0; m < TM; ++m)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const uint32_t b = m0 + (wm + m) * 16 + g * 4 + r, at = n0 + (wn + n) * 16 + r16;
            if (b < a.batch && at < a.rows) store_y<dt.value>(a.y, (uint64_t)b * a.rows + at, acc[n][m][r]);
          }
    }
  });
}

}  // namespace ecw

using namespace ecw;

namespace {

ecw_status check_weight(const void* codes, const void* scales, uint32_t rows, uint32_t cols, const char* what) {
  if (cols == 0 || cols > (1u << 30) || rows > (1u << 30)) return refuse(ECW_E_INVALID_ARG, what);
  if ((uint64_t)rows * row_blocks(cols) >> 38) return refuse(ECW_E_INVALID_ARG, "matrix too large");
  if (rows && (!codes || !scales || !aligned(codes, 16) || !aligned(scales, 16)))
    return refuse(ECW_E_INVALID_ARG, "codes and scales must be 16-byte aligned device pointers");
  return ECW_OK;
}

template <int ACT, bool NEAR>
ecw_status launch_few(hipStream_t stream, const GemmArgs& a, int y_dtype) {
  const uint32_t nt = (a.rows + 15) / 16, pairs = (a.blocks / 4 + 1) / 2;
  // up to four pairs a wave, and waves enough to fill the card
  uint32_t waves = 4;
  while (waves < kFewWaves && (pairs > waves * kTurns || ((uint64_t)nt * waves < 2048 && waves < pairs))) waves *= 2;
  if (!launchable(nt, waves * 64)) return refuse(ECW_E_UNSUPPORTED, "product too large for one launch");
  const uint32_t lds = waves * kTurns * kTurnBytes;
  auto* fn = k_mx4_gemm_few<ACT, NEAR>;
  if (lds > 64 * 1024) {  // to be allowed once on each device
    static std::atomic<uint64_t> allowed{0};
    int device = 0;
    const bool known = hipGetDevice(&device) == hipSuccess && device >= 0 && device < 64;
    if (!known || !(allowed.load(std::memory_order_relaxed) >> device & 1)) {
      if (hipFuncSetAttribute(reinterpret_cast<const void*>(fn), hipFuncAttributeMaxDynamicSharedMemorySize,
                              160 * 1024) != hipSuccess) {
        (void)hipGetLastError();
        return refuse(ECW_E_HIP, "hipFuncSetAttribute failed");
      }
      if (known) allowed.fetch_or(uint64_t(1) << device, std::memory_order_relaxed);
    }
  }
  hipLaunchKernelGGL(fn, dim3(nt), dim3(waves * 64), lds, stream, a, y_dtype);
  return launched("mx4_gemm");
}

uint64_t tiles(const GemmArgs& a, uint32_t bm, uint32_t bn) {
  return (uint64_t)((a.batch + bm - 1) / bm) * ((a.rows + bn - 1) / bn);
}

template <int ACT, int WM, int WN, int TM, int TN, int NS, bool EARLY, bool LOOSE = false, int KG = 1>
ecw_status launch_tile(hipStream_t stream, const GemmArgs& a, int y_dtype) {
  using T = Tiles<ACT, WM, WN, TM, TN, NS, EARLY, LOOSE, KG>;
  const uint32_t m_tiles = (a.batch + T::BM - 1) / T::BM, n_tiles = (a.rows + T::BN - 1) / T::BN;
  if (!launchable((uint64_t)m_tiles * n_tiles, 64 * T::kWaves * KG))
    return refuse(ECW_E_UNSUPPORTED, "product too large for one launch");
  hipLaunchKernelGGL((k_mx4_gemm_tile<ACT, WM, WN, TM, TN, NS, EARLY, LOOSE, KG>), dim3(m_tiles * n_tiles), dim3(64 * T::kWaves * KG), 0,
                     stream, a, m_tiles, n_tiles, y_dtype);
  return launched("mx4_gemm");
}

// Tiles by size: the smallest that leaves no CU two of them, for most of a small one's time
// is waiting; when there are more, the largest, which reads least.  Measured with bf16 x,
// in us (32x64, 64x64, 64x128, 128x128, 128x256):
//   64 rows by 4096 x 14336    23.9  41.8  55.5   106   164
//   128 rows by 14336 x 4096   37.0  32.6  22.6  35.6  52.0
//   1024 rows by 4096 x 4096   67.4  62.2  47.3  39.2  54.9
//   512 rows by 14336 x 4096    122   111  83.3  75.8  60.9
// and with 4-bit x (64x64, 128x128, 128x256, 256x256):
//   64 rows by 4096 x 14336    21.0  37.9  65.4   103
//   256 rows by 14336 x 4096   31.8  18.3  25.0  36.9
//   1024 rows by 14336 x 4096   105  63.1  55.3  44.1
template <int ACT>
ecw_status launch(hipStream_t stream, const GemmArgs& a, int y_dtype) {
  constexpr uint64_t kCus = 256;
  // A few rows go a block per 16 rows of w, which reads x once for each; more than four do
  // so only where tiles would leave more than half of the CUs without one.  Blocks of 16 rows
  // and tiles, in us, w from memory where it is large:
  //                            bf16 x         4-bit x
  //   16 rows by 4096 x 14336   19.4  22.9     12.7  17.1
  //   16 rows by 4096 x 4096     8.6   9.4      7.5   7.9
  //   5 rows by 28672 x 8192    41.3  40.8     34.2  35.3
  //   16 rows by 28672 x 8192   71.9  39.0     42.3  34.4
  //   16 rows by 14336 x 4096   20.7  10.3     13.1   9.5
  //   4 rows by 14336 x 4096    12.7  10.0      9.6   9.2
  //   4 rows by 28672 x 8192    40.7  41.1     33.4  35.2
  // (fp16 x is as bf16, but for tiles that unpack in turn: 5 rows by 28672 x 8192 42 and 52, 16
  // rows 72 and 51, 5 rows by 16384 x 16384 52 and 38.)
  // Operands that start between two words are slow to load (16 rows by 4096 x 14335 54 us,
  // in tiles 35; 4 rows 20).
  const bool words = ACT == kActMX4 || (aligned(a.x, 4) && a.x_stride % 2 == 0);
  const bool few = a.batch <= 4 || (a.batch <= 16 && words && tiles(a, 32, 64) < kCus / 2);
  if constexpr (ACT == kActMX4) {
    if (few) return launch_few<ACT, true>(stream, a, y_dtype);
    if (tiles(a, 64, 64) <= kCus) return launch_tile<ACT, 1, 4, 4, 1, 3, true, false, 4>(stream, a, y_dtype);
    if (tiles(a, 128, 128) <= kCus) return launch_tile<ACT, 2, 4, 4, 2, 3, true, false, 2>(stream, a, y_dtype);
    if (tiles(a, 128, 256) <= kCus) return launch_tile<ACT, 2, 4, 4, 4, 4, true>(stream, a, y_dtype);
    return launch_tile<ACT, 2, 4, 8, 4, 3, false>(stream, a, y_dtype);
  } else {
    if (a.cols <= 8) {
      const uint64_t grid = ((uint64_t)a.batch * a.rows + 255) / 256;
      if (!launchable(grid, 256)) return refuse(ECW_E_UNSUPPORTED, "product too large for one launch");
      hipLaunchKernelGGL(k_mx4_gemm_narrow<ACT>, dim3((uint32_t)grid), dim3(256), 0, stream, a, y_dtype);
      return launched("mx4_gemm");
    }
    if (few) {
      const bool near = ((uint64_t)(a.batch - 1) * (uint64_t)a.x_stride + a.cols) >> 30 == 0;
      return near ? launch_few<ACT, true>(stream, a, y_dtype) : launch_few<ACT, false>(stream, a, y_dtype);
    }
    if (aligned(a.x, 16) && a.x_stride % 8 == 0 && a.cols % 8 == 0) {
      if (tiles(a, 32, 64) <= kCus) return launch_tile<ACT, 1, 4, 2, 1, 3, false, false, 4>(stream, a, y_dtype);
      if (tiles(a, 64, 64) <= kCus) return launch_tile<ACT, 1, 4, 4, 1, 3, true, false, 2>(stream, a, y_dtype);
      if (tiles(a, 64, 128) <= kCus) return launch_tile<ACT, 2, 4, 2, 2, 3, false, false, 2>(stream, a, y_dtype);
      if (tiles(a, 128, 128) <= kCus) return launch_tile<ACT, 2, 4, 4, 2, 3, false>(stream, a, y_dtype);
      return launch_tile<ACT, 2, 4, 4, 4, 3, false>(stream, a, y_dtype);
    }
    if (tiles(a, 32, 64) <= kCus) return launch_tile<ACT, 1, 4, 2, 1, 3, false, true, 4>(stream, a, y_dtype);
    if (tiles(a, 64, 64) <= kCus) return launch_tile<ACT, 1, 4, 4, 1, 3, false, true, 2>(stream, a, y_dtype);
    if (tiles(a, 64, 128) <= kCus) return launch_tile<ACT, 2, 4, 2, 2, 3, false, true, 2>(stream, a, y_dtype);
    if (tiles(a, 128, 128) <= kCus) return launch_tile<ACT, 2, 4, 4, 2, 3, false, true>(stream, a, y_dtype);
    return launch_tile<ACT, 2, 4, 4, 4, 3, false, true>(stream, a, y_dtype);
  }
}

ecw_status check_output(const void* y, int y_dtype, uint32_t batch) {
  if (y_dtype != ECW_DT_F16 && y_dtype != ECW_DT_BF16 && y_dtype != ECW_DT_F32)
    return refuse(ECW_E_INVALID_ARG, "y dtype must be F16, BF16 or F32");
  if (batch > (1u << 24)) return refuse(ECW_E_INVALID_ARG, "batch must be at most 2^24");
  if (!y || !aligned(y, 16)) return refuse(ECW_E_INVALID_ARG, "y must be a 16-byte aligned device pointer");
  return ECW_OK;
}

}  // namespace

extern "C" {

ecw_status mx4_gemm(ecw_stream stream, const void* w_codes, const void* w_scales, uint32_t rows, uint32_t cols,
                    const void* x, int x_dtype, int64_t x_stride, uint32_t batch, void* y, int y_dtype) {
  if (ecw_status s = check_weight(w_codes, w_scales, rows, cols, "cols must be in [1, 2^30], rows at most 2^30"))
    return s;
  if (x_dtype != ECW_DT_F16 && x_dtype != ECW_DT_BF16)
    return refuse(ECW_E_INVALID_ARG, "x dtype must be F16 or BF16");
  if (rows == 0 || batch == 0) return ECW_OK;
  if (ecw_status s = check_output(y, y_dtype, batch)) return s;
  if (!x || !aligned(x, 2) || x_stride < 0)
    return refuse(ECW_E_INVALID_ARG, "x must be an aligned device pointer with a row stride of 0 or more");
  const GemmArgs a{static_cast<const uint8_t*>(w_codes), static_cast<const uint8_t*>(w_scales), x, nullptr, y,
                   x_stride, rows, cols, batch, row_blocks(cols), scale_stride(cols)};
  return x_dtype == ECW_DT_F16 ? launch<ECW_DT_F16>((hipStream_t)stream, a, y_dtype)
                               : launch<ECW_DT_BF16>((hipStream_t)stream, a, y_dtype);
}

ecw_status mx4_gemm_mx4(ecw_stream stream, const void* w_codes, const void* w_scales, uint32_t rows, uint32_t cols,
                        const void* x_codes, const void* x_scales, uint32_t batch, void* y, int y_dtype) {
  if (ecw_status s = check_weight(w_codes, w_scales, rows, cols, "cols must be in [1, 2^30], rows at most 2^30"))
    return s;
  if (ecw_status s = check_weight(x_codes, x_scales, batch, cols, "batch must be at most 2^30")) return s;
  if (rows == 0 || batch == 0) return ECW_OK;
  if (ecw_status s = check_output(y, y_dtype, batch)) return s;
  const GemmArgs a{static_cast<const uint8_t*>(w_codes), static_cast<const uint8_t*>(w_scales), x_codes,
                   static_cast<const uint8_t*>(x_scales), y, 0, rows, cols, batch, row_blocks(cols), scale_stride(cols)};
  return launch<kActMX4>((hipStream_t)stream, a, y_dtype);
}

}  // extern "C"
