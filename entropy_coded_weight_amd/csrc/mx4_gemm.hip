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
// span's sum is multiplied by that scale in fp32.  A wider span, or a NaN block, takes
// x as the sum of two bf16 numbers, which holds every fp16 number exactly.
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
  uint32_t rows, cols, batch, blocks;  // of w; blocks of a padded row
  bool vec;               // rows of x are 16-byte aligned
};

__device__ __forceinline__ void store_y(void* y, uint64_t at, float v, int dt) {
  if (dt == ECW_DT_F32)
    static_cast<float*>(y)[at] = v;
  else if (dt == ECW_DT_F16)
    static_cast<_Float16*>(y)[at] = (_Float16)v;
  else
    static_cast<__bf16*>(y)[at] = (__bf16)v;
}

// the largest and smallest byte of a word
__device__ __forceinline__ void byte_range(uint32_t w, uint32_t* lo, uint32_t* hi) {
  const uint32_t a = w & 255, b = w >> 8 & 255, c = w >> 16 & 255, d = w >> 24;
  *hi = max(max(a, b), max(c, d));
  *lo = min(min(a, b), min(c, d));
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
    uint32_t lo, hi;
    byte_range(sw, &lo, &hi);
    const uint32_t mine = sw >> 8 * g & 255;
    if (!__any(hi - lo > 23 || hi == kScaleNaN)) {
      f32x4 sum[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) sum[t] = f32x4{0.f, 0.f, 0.f, 0.f};
      const float s = scale_of(kScaleOne + mine - hi);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f16x8 b = oct_f16(w[j], s);
#pragma unroll
        for (int t = 0; t < NT; ++t)
          sum[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, x[t][j]), b, sum[t], 0, 0, 0);
      }
      const float top = scale_of(hi);  // of the lane's row of w: its column of the result
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[t][r] = fmaf(sum[t][r], top, acc[t][r]);
    } else {
      const float s = scale_of(mine);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bf16x8 b = oct_bf16(w[j], s);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          bf16x8 h, l;
          split_f16(x[t][j], &h, &l);
          acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(h, b, acc[t], 0, 0, 0);
          acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(l, b, acc[t], 0, 0, 0);
        }
      }
    }
  }
}

__device__ __forceinline__ f32x4 span_product_mx4(f32x4 acc, u32x4 w, uint32_t sw, uint32_t g, u32x4 x, uint32_t sx) {
  typedef int i32x8 __attribute__((ext_vector_type(8)));
  const i32x8 a = {(int)x[0], (int)x[1], (int)x[2], (int)x[3], 0, 0, 0, 0};
  const i32x8 b = {(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, acc, 4, 4, 0, (int)(sx >> 8 * g), 0,
                                                          (int)(sw >> 8 * g));
}

// A block computes 16 rows of w times 16 NT rows of x; its waves take the spans in
// turn and join their sums through LDS, in the order of the waves.
template <int ACT, int NT>
__global__ void __launch_bounds__(1024) k_mx4_gemm_few(GemmArgs a, int y_dtype) {
  extern __shared__ f32x4 part[];  // [waves][NT][64]
  const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const uint32_t r16 = lane & 15, g = lane >> 4;
  const uint32_t n0 = blockIdx.x * 16, m0 = blockIdx.y * (16 * NT);
  const uint32_t n = min(n0 + r16, a.rows - 1);
  const uint32_t spans = a.blocks / 4;
  const uint8_t* w = a.w + (uint64_t)n * a.blocks * 16 + g * 16;
  const uint8_t* ws = a.ws + (uint64_t)n * a.blocks;
  f32x4 acc[NT];
  uint64_t m[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    m[t] = min(m0 + t * 16 + r16, a.batch - 1);
  }
  for (uint32_t s = wave; s < spans; s += waves) {
    const u32x4 wv = *reinterpret_cast<const u32x4*>(w + (uint64_t)s * 64);
    const uint32_t sw = *reinterpret_cast<const uint32_t*>(ws + s * 4);
    if constexpr (ACT == kActMX4) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const uint8_t* x = static_cast<const uint8_t*>(a.x) + m[t] * a.blocks * 16 + (uint64_t)s * 64 + g * 16;
        const uint32_t sx = *reinterpret_cast<const uint32_t*>(a.xs + m[t] * a.blocks + s * 4);
        acc[t] = span_product_mx4(acc[t], wv, sw, g, *reinterpret_cast<const u32x4*>(x), sx);
      }
    } else {
      u32x4 x[NT][4];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          x[t][j] = load_oct16(static_cast<const uint16_t*>(a.x) + m[t] * a.x_stride, s * 128 + g * 32 + j * 8,
                               a.cols, a.vec).v;
      span_product<ACT, NT>(acc, wv, sw, g, x);
    }
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) part[(wave * NT + t) * 64 + lane] = acc[t];
  __syncthreads();
  // lane l of tile t: rows 4 (l / 16) .. + 3 of x, row l % 16 of w
  for (uint32_t i = threadIdx.x; i < NT * 64; i += blockDim.x) {
    f32x4 sum = part[i];
    for (uint32_t v = 1; v < waves; ++v) sum += part[v * NT * 64 + i];
    const uint32_t row = n0 + (i & 15), b = m0 + i / 64 * 16 + (i >> 4 & 3) * 4;
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (row < a.rows && b + r < a.batch) store_y(a.y, (uint64_t)(b + r) * a.rows + row, sum[r], y_dtype);
  }
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

template <int ACT, int NT>
ecw_status launch_few(hipStream_t stream, const GemmArgs& a, int y_dtype) {
  const uint32_t nt = (a.rows + 15) / 16, mt = (a.batch + 16 * NT - 1) / (16 * NT), spans = a.blocks / 4;
  if (mt > 65535) return refuse(ECW_E_UNSUPPORTED, "batch too large for one launch");
  uint32_t waves = 4;
  while (waves < 16 && (uint64_t)nt * mt * waves < 2048 && waves < spans) waves *= 2;
  hipLaunchKernelGGL((k_mx4_gemm_few<ACT, NT>), dim3(nt, mt), dim3(waves * 64), waves * NT * 64 * sizeof(f32x4),
                     stream, a, y_dtype);
  return launched("mx4_gemm");
}

template <int ACT>
ecw_status launch(hipStream_t stream, const GemmArgs& a, int y_dtype) {
  if (a.batch <= 16) return launch_few<ACT, 1>(stream, a, y_dtype);
  if (a.batch <= 32) return launch_few<ACT, 2>(stream, a, y_dtype);
  return launch_few<ACT, 4>(stream, a, y_dtype);
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
                   x_stride, rows, cols, batch, row_blocks(cols), aligned(x, 16) && x_stride % 8 == 0};
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
                   static_cast<const uint8_t*>(x_scales), y, 0, rows, cols, batch, row_blocks(cols), true};
  return launch<kActMX4>((hipStream_t)stream, a, y_dtype);
}

}  // extern "C"
