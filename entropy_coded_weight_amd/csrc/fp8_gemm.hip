// y[b][n] = sum_k x[b][k] w[n][k], both in the block-scaled 8-bit format.
//
// Two instructions multiply.  The scaled 8-bit one (16x16x128) takes one block of 128 columns
// of 16 rows of each operand, 32 bytes a lane, and a scale byte of each lane's row, so that a
// block's product takes one instruction, scales included (4.3 PFLOP/s measured, 2.1 for
// bf16).  But it adds up to 16 neighbouring products with 12 fraction bits under the largest
// one's power of two before they go into the fp32 sum: against 64 bits its sums are off by
// 1.5e-5 of the result (2-norm, normal numbers), 7e-5 with columns a hundred times as large,
// where fp32 sums are by 1e-7.  Next to an output rounded to 16 bits (1.7e-3 in bf16, 2e-4 in
// fp16) that is nothing; an fp32 output shows it.  So fp32 outputs, and a few rows of x, which
// are bound by reading w, go by the bf16 instruction (16x16x32): E4M3 numbers times their
// scale are exact in bf16, products exact in fp32, and sums fp32.
//
// Which of the columns of a block a lane holds is free as long as both operands agree and all
// of a row's lanes give the same scale: lane l has row l % 16 and the 16-byte pieces l / 16
// and l / 16 + 4.  w's rows go down the result's registers: a lane holds neighbouring outputs
// of one row of x.
#include "fp8_common.h"
#include "gemm_common.h"

#include <atomic>

namespace ecw {

struct Fp8GemmArgs {
  const uint8_t *w, *ws, *x, *xs;  // codes and scale bytes
  void* y;
  uint32_t rows, batch;
  uint32_t row, scale_row, spans;  // bytes of a row of codes and of scales, blocks of 128 columns
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
// A block computes 16 rows of w times up to 16 NT rows of x; its waves take spans of 128
// columns in turn and join their sums through LDS, in the order of the waves.  A wave copies
// w for kFewTurns turns straight to LDS, 8 rows of 128 bytes at a time, so that neighbouring
// lanes read whole lines; x, which blocks share, it reads into registers.  Bound by reading w.
constexpr uint32_t kFewTurns = 4;
constexpr uint32_t kFewTurnBytes = 16 * 128;  // 16 rows of w
constexpr uint32_t kFewMost = 16;             // waves

template <int NT>
__global__ void __launch_bounds__(64 * kFewMost) k_fp8_gemm_few(Fp8GemmArgs a, int y_dtype) {
  extern __shared__ __align__(16) uint8_t lds[];  // each wave's turns, then (over them) the sums
  const uint32_t base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;
  const uint32_t lane = threadIdx.x & 63, waves = blockDim.x >> 6;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t r16 = lane & 15, g = lane >> 4;
  const uint32_t n0 = blockIdx.x * 16;

  const uint8_t* from[2];  // the lane's 16 bytes of rows 0-7 and 8-15
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t row = i * 8 + (lane >> 3), piece = (lane & 7) ^ stirred(row);
    from[i] = a.w + (uint64_t)min(n0 + row, a.rows - 1) * a.row + piece * 16;
  }
  const uint8_t* ws = a.ws + (uint64_t)min(n0 + r16, a.rows - 1) * a.scale_row;
  const uint8_t *x[NT], *xs[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const uint64_t m = min(t * 16 + r16, a.batch - 1);
    x[t] = a.x + m * a.row + g * 16;
    xs[t] = a.xs + m * a.scale_row;
  }
  const uint32_t in0 = r16 * 8 + (g ^ stirred(r16)), in1 = r16 * 8 + ((g + 4) ^ stirred(r16));

  f32x4 acc[1][NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) acc[0][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (uint32_t first = wave; first < a.spans; first += waves * kFewTurns) {
#pragma unroll
    for (uint32_t k = 0; k < kFewTurns; ++k) {
      const uint32_t s = first + k * waves;
      if (s < a.spans) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
          to_lds(from[i] + (uint64_t)s * 128, base + (wave * kFewTurns + k) * kFewTurnBytes + i * 1024);
      }
    }
    wait_copies<0>();
#pragma unroll
    for (uint32_t k = 0; k < kFewTurns; ++k) {
      const uint32_t s = first + k * waves;
      if (s < a.spans) {
        const u32x4* w = reinterpret_cast<const u32x4*>(lds + (wave * kFewTurns + k) * kFewTurnBytes);
        const i32x8 wv[1] = {join(w[in0], w[in1])};
        const float sw[1] = {scale_of(ws[s])};
        i32x8 xv[NT];
        float sx[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const u32x4* p = reinterpret_cast<const u32x4*>(x[t] + (uint64_t)s * 128);
          xv[t] = join(p[0], p[4]);
          sx[t] = scale_of(xs[t][s]);
        }
        exact_products(acc, wv, sw, xv, sx);
      }
    }
    wait_copies<0>();  // this wave's reads of LDS are done before it copies again
  }
  __syncthreads();
  f32x4* part = reinterpret_cast<f32x4*>(lds);  // [waves][NT][64]
#pragma unroll
  for (int t = 0; t < NT; ++t) part[(wave * NT + t) * 64 + lane] = acc[0][t];
  __syncthreads();
  // lane l: rows 4 (l / 16) .. + 3 of w, row l % 16 of x
  for (uint32_t t = wave; t < NT; t += waves) {
    f32x4 sum = part[t * 64 + lane];
    for (uint32_t v = 1; v < waves; ++v) sum += part[(v * NT + t) * 64 + lane];
    const uint32_t b = t * 16 + r16, n = n0 + g * 4;
    if (b >= a.batch || n >= a.rows) continue;
    with_type(y_dtype, [&](auto dt) {
      const float v[4] = {sum[0], sum[1], sum[2], sum[3]};
      store_run<dt.value>(a.y, (uint64_t)b * a.rows + n, v, a.rows - n, a.rows % 4 == 0);
    });
  }
}

// ------------------------------------------------------------------ many rows
// A block of WM x WN waves multiplies 16 TM WM rows of x and 16 TN WN rows of w, a span of
// 128 columns at a time, from NS stages in LDS that copies fill ahead.  KG: it has KG times
// the waves, which take KG spans at once and add their sums up at the end, in order.
template <int WM, int WN, int TM, int TN, int NS, int KG>
struct Fp8Tiles {
  static constexpr int kWaves = WM * WN, BM = 16 * TM * WM, BN = 16 * TN * WN;
  static constexpr uint32_t kX = BM * 128, kSpan = (BM + BN) * 128, kStage = KG * kSpan;
  static constexpr uint32_t kScaleRows = BM + BN;                // those of x first
  static constexpr uint32_t kScalePlaces = (NS * KG + 15) / 16 + 1;  // of 16 spans each
  static constexpr uint32_t kBytes = kStage * NS + kScalePlaces * kScaleRows * 16;
  static constexpr int kXLoads = BM / 8 / kWaves, kWLoads = BN / 8 / kWaves;  // copies per wave and span
  static constexpr int kSLoads = (kScaleRows / 64 + kWaves - 1) / kWaves;    // per 16 spans
  static_assert(BM % (8 * kWaves) == 0 && BN % (8 * kWaves) == 0 && kScaleRows % 64 == 0, "");
  static_assert(kBytes <= 160 * 1024 && 16 % KG == 0, "");
  static_assert((KG - 1) * kWaves * TM * TN * 1024 <= (int)kStage * NS, "");  // sums of the other groups
};

// EXACT: by the bf16 instruction.
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
  const uint32_t steps = (a.spans + KG - 1) / KG;
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
    const uint32_t span = step * KG + kg;
    const uint64_t s = min(span, a.spans - 1);
    if (kg == 0 && span % 16 == 0 && span < a.spans) {
#pragma unroll
      for (int i = 0; i < T::kSLoads; ++i) {
        const uint32_t part = wave + i * T::kWaves;
        if (part < T::kScaleRows / 64)
          to_lds(sp[i] + s, base + T::kStage * NS + (span / 16 % T::kScalePlaces) * T::kScaleRows * 16 + part * 1024);
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
    const uint32_t s = step * KG + kg;
    const uint8_t* at = lds + stage * T::kStage + kg * T::kSpan;
    const u32x4* x = reinterpret_cast<const u32x4*>(at) + wm * 128;
    const u32x4* w = reinterpret_cast<const u32x4*>(at + T::kX) + wn * 128;
    const uint8_t* xs = lds + T::kStage * NS + (s / 16 % T::kScalePlaces) * T::kScaleRows * 16 + s % 16 + (wm * 16 + r16) * 16;
    const uint8_t* ws = xs + (T::BM - wm * 16 + wn * 16) * 16;
    if (KG == 1 || s < a.spans) {
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
  with_type(y_dtype, [&](auto dt) {
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
  });
}

}  // namespace ecw

using namespace ecw;

namespace {

template <int NT>
ecw_status launch_few(hipStream_t stream, const Fp8GemmArgs& a, int y_dtype) {
  const uint32_t blocks = (a.rows + 15) / 16;
  // up to four spans a wave, and waves enough to fill the card
  uint32_t waves = 4;
  while (waves < kFewMost && (a.spans > waves * kFewTurns || ((uint64_t)blocks * waves < 2048 && waves < a.spans))) waves *= 2;
  if (!launchable(blocks, waves * 64)) return refuse(ECW_E_UNSUPPORTED, "product too large for one launch");
  const uint32_t lds = waves * kFewTurns * kFewTurnBytes;
  auto* fn = k_fp8_gemm_few<NT>;
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
  hipLaunchKernelGGL(fn, dim3(blocks), dim3(waves * 64), lds, stream, a, y_dtype);
  return launched("fp8_gemm");
}

template <int WM, int WN, int TM, int TN, int NS, int KG, bool EXACT>
ecw_status launch_tile(hipStream_t stream, const Fp8GemmArgs& a, int y_dtype) {
  using T = Fp8Tiles<WM, WN, TM, TN, NS, KG>;
  const uint32_t m_tiles = (a.batch + T::BM - 1) / T::BM, n_tiles = (a.rows + T::BN - 1) / T::BN;
  if (!launchable((uint64_t)m_tiles * n_tiles, 64 * T::kWaves * KG))
    return refuse(ECW_E_UNSUPPORTED, "product too large for one launch");
  hipLaunchKernelGGL((k_fp8_gemm_tile<WM, WN, TM, TN, NS, KG, EXACT>), dim3(m_tiles * n_tiles), dim3(64 * T::kWaves * KG),
                     0, stream, a, m_tiles, n_tiles, y_dtype);
  return launched("fp8_gemm");
}

uint64_t tiles(const Fp8GemmArgs& a, uint32_t bm, uint32_t bn) {
  return (uint64_t)((a.batch + bm - 1) / bm) * ((a.rows + bn - 1) / bn);
}

template <bool EXACT>
ecw_status launch_tiles(hipStream_t stream, const Fp8GemmArgs& a, int y_dtype) {
  constexpr uint64_t kCus = 256;
  if (tiles(a, 64, 64) <= kCus) return launch_tile<1, 4, 4, 1, 2, 4, EXACT>(stream, a, y_dtype);
  if (tiles(a, 128, 128) <= kCus) return launch_tile<2, 4, 4, 2, 2, 2, EXACT>(stream, a, y_dtype);
  if (tiles(a, 128, 256) <= kCus) return launch_tile<2, 4, 4, 4, 3, 1, EXACT>(stream, a, y_dtype);
  return launch_tile<2, 4, 8, 4, 2, 1, EXACT>(stream, a, y_dtype);
}

}  // namespace

extern "C" ecw_status fp8_gemm(ecw_stream stream, const void* w_codes, const void* w_scales, uint32_t rows, uint32_t cols,
                               const void* x_codes, const void* x_scales, uint32_t batch, void* y, int y_dtype) {
  if (ecw_status s = check_fp8(w_codes, w_scales, rows, cols)) return s;
  if (ecw_status s = check_fp8(x_codes, x_scales, batch, cols)) return s;
  if (!is_float(y_dtype)) return refuse(ECW_E_INVALID_ARG, "y dtype must be F16, BF16 or F32");
  if (rows == 0 || batch == 0) return ECW_OK;
  if (batch > (1u << 24)) return refuse(ECW_E_INVALID_ARG, "batch must be at most 2^24");
  if (!y || !aligned(y, 16)) return refuse(ECW_E_INVALID_ARG, "y must be a 16-byte aligned device pointer");
  const Fp8GemmArgs a{static_cast<const uint8_t*>(w_codes), static_cast<const uint8_t*>(w_scales),
                      static_cast<const uint8_t*>(x_codes), static_cast<const uint8_t*>(x_scales), y, rows, batch,
                      fp8_row(cols), fp8_scale_row(cols), fp8_row(cols) / 128};
  const auto st = (hipStream_t)stream;
  if (batch <= 16) return launch_few<1>(st, a, y_dtype);
  if (batch <= 32) return launch_few<2>(st, a, y_dtype);
  if (batch <= 48) return launch_few<3>(st, a, y_dtype);
  if (batch <= 64) return launch_few<4>(st, a, y_dtype);
  return y_dtype == ECW_DT_F32 ? launch_tiles<true>(st, a, y_dtype) : launch_tiles<false>(st, a, y_dtype);
}
