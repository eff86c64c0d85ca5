// Quantisation of matrices into the block-scaled 8-bit format, with a SiLU gate in the same
// pass where one is given, and back.
#include "fp8_common.h"

namespace ecw {

// silu(g) = g / (1 + e^-g).  Below -88.73 e^-g passes fp32's range and the gate is zero.  e^-g is
// 2^-t times e^(t ln 2 - g) with t the rounded product g log2(e): what t lost, times ln 2, is
// small, so the second factor is one plus that.  With the library's exponential the vector
// instructions took as long as the memory (2003 x 14336 bf16 4.0 us more).  The instruction gives
// zero for reciprocals under 2^-126, so it takes a quarter of 1 + e^-g, and g a quarter too.
__device__ __forceinline__ float silu(float g) {
  const float h = __builtin_amdgcn_fmed3f(g, -126.f, 126.f), t = h * 1.44269502f;
  const float lost = fmaf(h, 1.92596303e-8f, fmaf(h, 1.44269502f, -t));  // log2(e) = 1.44269502 + 1.926e-8
  const float e = __builtin_amdgcn_exp2f(-t) * fmaf(lost, -0.693147181f, 1.f);
  return 0.25f * g * __builtin_amdgcn_rcpf(fmaf(0.25f, e, 0.25f));
}

// One lane per 8 elements, 16 lanes per block, so that a block's maximum needs no more than
// its row of lanes.  Bound by memory (14336 x 4096 bf16 32.3 us, 5.5 TB/s; 2003 x 14336 bf16
// with a gate 30.5 us, 4.7 TB/s; one row of 14336 2.4 us).
template <int DT, bool GATED>
__global__ void __launch_bounds__(256) k_fp8_quantise(const void* __restrict__ x, int64_t x_stride,
                                                      const void* __restrict__ gate, int64_t gate_stride, uint32_t rows,
                                                      uint32_t cols, uint32_t octs, uint8_t* __restrict__ codes,
                                                      uint8_t* __restrict__ scales) {
  const uint32_t at = blockIdx.x * 256 + threadIdx.x;  // the host keeps the launch under 2^32 lanes
  const uint32_t row = at / octs, oct = at - row * octs;
  if (row >= rows) return;  // whole blocks: octs is a multiple of 16
  constexpr int kSize = DT == ECW_DT_F32 ? 4 : 2;
  float v[8];
  const auto in = load_oct<DT>(static_cast<const uint8_t*>(x) + row * x_stride * kSize, oct * 8, cols);
  if constexpr (GATED) {
    float g[8];
    widen<DT>(g, load_oct<DT>(static_cast<const uint8_t*>(gate) + row * gate_stride * kSize, oct * 8, cols));
    widen<DT>(v, in);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = silu(g[i]) * v[i];
  } else {
    widen<DT>(v, in);
  }
  uint32_t b;
  const u32x2 c = fp8_oct(v, &b);
  store_fp8(codes, scales, row, oct, octs, fp8_scale_row(cols), c, b);
}

// The same lanes the other way.  Bound by memory (14336 x 4096 to bf16 29.5 us, 6.0 TB/s,
// codes partly from the last-level cache).
template <int DT>
__global__ void __launch_bounds__(256) k_fp8_dequantise(const uint8_t* __restrict__ codes,
                                                        const uint8_t* __restrict__ scales, uint32_t rows,
                                                        uint32_t cols, uint32_t octs, void* __restrict__ out) {
  const uint32_t at = blockIdx.x * 256 + threadIdx.x;
  const uint32_t row = at / octs, oct = at - row * octs;
  if (row >= rows || oct * 8 >= cols) return;
  const u32x2 c = reinterpret_cast<const u32x2*>(codes)[at];
  const uint32_t b = scales[(uint64_t)row * fp8_scale_row(cols) + oct / 16];
  const float s = b == kScaleNaN ? __builtin_nanf("") : scale_of(b);
  float v[8];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[i], false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[i], true);
    v[4 * i] = a[0] * s, v[4 * i + 1] = a[1] * s, v[4 * i + 2] = b[0] * s, v[4 * i + 3] = b[1] * s;
  }
  store_values<DT>(out, (uint64_t)row * cols + oct * 8, v, cols - oct * 8);
}

}  // namespace ecw

using namespace ecw;

namespace {

// Blocks of 256 lanes, one lane per 8 columns.
bool oct_grid(uint32_t rows, uint32_t cols, uint32_t* octs, uint32_t* grid) {
  *octs = fp8_row(cols) / 8;
  const uint64_t n = ((uint64_t)rows * *octs + 255) / 256;
  *grid = (uint32_t)n;
  return launchable(n, 256);
}

}  // namespace

extern "C" {

ecw_status fp8_quantize(ecw_stream stream, const void* x, int dtype, int64_t x_stride, const void* gate,
                        int64_t gate_stride, uint32_t rows, uint32_t cols, void* codes, void* scales) {
  if (ecw_status s = check_fp8(codes, scales, rows, cols)) return s;
  if (!is_float(dtype)) return refuse(ECW_E_INVALID_ARG, "x dtype must be F16, BF16 or F32");
  if (rows == 0) return ECW_OK;
  if (!x || !aligned(x, size_of(dtype)) || !aligned(gate, size_of(dtype)))
    return refuse(ECW_E_INVALID_ARG, "x and gate must be aligned device pointers");
  if (x_stride < 0 || gate_stride < 0) return refuse(ECW_E_INVALID_ARG, "row strides must not be negative");
  uint32_t octs, grid;
  if (!oct_grid(rows, cols, &octs, &grid)) return refuse(ECW_E_UNSUPPORTED, "matrix too large for one launch");
  auto* fn = dtype == ECW_DT_F32   ? (gate ? k_fp8_quantise<ECW_DT_F32, true> : k_fp8_quantise<ECW_DT_F32, false>)
             : dtype == ECW_DT_F16 ? (gate ? k_fp8_quantise<ECW_DT_F16, true> : k_fp8_quantise<ECW_DT_F16, false>)
                                   : (gate ? k_fp8_quantise<ECW_DT_BF16, true> : k_fp8_quantise<ECW_DT_BF16, false>);
  hipLaunchKernelGGL(fn, dim3(grid), dim3(256), 0, (hipStream_t)stream, x, x_stride, gate, gate_stride, rows, cols, octs,
                     static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales));
  return launched("fp8_quantize");
}

ecw_status fp8_dequantize(ecw_stream stream, const void* codes, const void* scales, uint32_t rows, uint32_t cols,
                          void* out, int out_dtype) {
  if (ecw_status s = check_fp8(codes, scales, rows, cols)) return s;
  if (!is_float(out_dtype)) return refuse(ECW_E_INVALID_ARG, "output dtype must be F16, BF16 or F32");
  if (rows == 0) return ECW_OK;
  if (!out || !aligned(out, size_of(out_dtype)))
    return refuse(ECW_E_INVALID_ARG, "output must be an aligned device pointer");
  uint32_t octs, grid;
  if (!oct_grid(rows, cols, &octs, &grid)) return refuse(ECW_E_UNSUPPORTED, "matrix too large for one launch");
  auto* fn = out_dtype == ECW_DT_F32   ? k_fp8_dequantise<ECW_DT_F32>
             : out_dtype == ECW_DT_F16 ? k_fp8_dequantise<ECW_DT_F16>
                                       : k_fp8_dequantise<ECW_DT_BF16>;
  hipLaunchKernelGGL(fn, dim3(grid), dim3(256), 0, (hipStream_t)stream, static_cast<const uint8_t*>(codes),
                     static_cast<const uint8_t*>(scales), rows, cols, octs, out);
  return launched("fp8_dequantize");
}

}  // extern "C"
