// Quantisation of matrices into the microscaled 4-bit format and back.
#include "mx4_common.h"

namespace ecw {

ecw_status refuse(ecw_status s, const char* msg) noexcept {
  try {
    return fail(s, msg);
  } catch (...) {
    return s;
  }
}

ecw_status launched(const char* what) noexcept {
  const hipError_t e = hipGetLastError();
  if (e == hipSuccess) return ECW_OK;
  try {
    return fail(ECW_E_HIP, std::string(what) + ": launch failed: " + hipGetErrorString(e));
  } catch (...) {
    return ECW_E_HIP;
  }
}

// One lane per 8 elements, four lanes per block, so that a wave reads 1 KiB of 16-bit
// input in one load and writes 256 bytes of codes.  Bound by memory (14336 x 4096 bf16
// 27.5 us, 5.4 TB/s; 4096 x 14335, rows at any element, 31 us; one row of 4096 1.5 to 1.8 us,
// the latency of a load and a store).
template <int DT>
__global__ void __launch_bounds__(256) k_mx4_quantise(const void* __restrict__ x, int64_t stride, uint32_t rows,
                                                      uint32_t cols, uint32_t octs, uint32_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  const uint64_t at = (uint64_t)blockIdx.x * 256 + threadIdx.x;
  const uint32_t row = (uint32_t)(at / octs), oct = (uint32_t)(at - (uint64_t)row * octs);
  if (row >= rows) return;  // whole blocks: octs is a multiple of 16
  uint32_t c, b;
  if constexpr (DT == ECW_DT_F32)
    c = quantise_oct(load_oct32(static_cast<const float*>(x) + row * stride, oct * 8, cols), &b);
  else
    c = quantise_oct<DT == ECW_DT_F16>(
        load_oct16(static_cast<const uint16_t*>(x) + row * stride, oct * 8, cols), &b);
  codes[at] = c;
  if ((oct & 3) == 0) {
    const uint32_t stride = scale_stride(cols), block = oct >> 2, blocks = octs >> 2;
    uint8_t* to = scales + (uint64_t)row * stride + block;
    *to = (uint8_t)b;
    if (block == blocks - 1)  // the rest of the last 16 bytes
      for (uint32_t i = blocks; i < stride; ++i) *++to = kScaleOne;
  }
}

// The same lanes the other way.  Bound by memory (14336 x 4096 to bf16 22.4 us, 6.6 TB/s,
// codes partly from the last-level cache).
template <int DT>
__global__ void __launch_bounds__(256) k_mx4_dequantise(const uint32_t* __restrict__ codes,
                                                        const uint8_t* __restrict__ scales, uint32_t rows,
                                                        uint32_t cols, uint32_t octs, void* __restrict__ out) {
  const uint64_t at = (uint64_t)blockIdx.x * 256 + threadIdx.x;
  const uint32_t row = (uint32_t)(at / octs), oct = (uint32_t)(at - (uint64_t)row * octs);
  if (row >= rows || oct * 8 >= cols) return;
  store_oct<DT>(out, (uint64_t)row * cols + oct * 8, codes[at],
                scale_of(scales[(uint64_t)row * scale_stride(cols) + (oct >> 2)]), cols - oct * 8);
}

}  // namespace ecw

using namespace ecw;

namespace {

ecw_status check_matrix(const void* codes, const void* scales, uint32_t rows, uint32_t cols) {
  if (cols == 0 || cols > (1u << 30) || rows > (1u << 30))
    return refuse(ECW_E_INVALID_ARG, "cols must be in [1, 2^30], rows at most 2^30");
  if ((uint64_t)rows * row_blocks(cols) >> 38) return refuse(ECW_E_INVALID_ARG, "matrix too large");
  if (rows && (!codes || !scales || !aligned(codes, 16) || !aligned(scales, 16)))
    return refuse(ECW_E_INVALID_ARG, "codes and scales must be 16-byte aligned device pointers");
  return ECW_OK;
}

}  // namespace

extern "C" {

ecw_status mx4_quantize(ecw_stream stream, const void* x, int x_dtype, int64_t row_stride, uint32_t rows,
                        uint32_t cols, void* codes, void* scales) {
  if (ecw_status s = check_matrix(codes, scales, rows, cols)) return s;
  if (x_dtype != ECW_DT_F16 && x_dtype != ECW_DT_BF16 && x_dtype != ECW_DT_F32)
    return refuse(ECW_E_INVALID_ARG, "x dtype must be F16, BF16 or F32");
  if (rows == 0) return ECW_OK;
  const uint32_t size = x_dtype == ECW_DT_F32 ? 4 : 2;
  if (!x || !aligned(x, size)) return refuse(ECW_E_INVALID_ARG, "x must be an aligned device pointer");
  if (row_stride < 0) return refuse(ECW_E_INVALID_ARG, "row stride must not be negative");
  const uint32_t octs = row_blocks(cols) * 4;
  const uint64_t grid = ((uint64_t)rows * octs + 255) / 256;
  if (!launchable(grid, 256)) return refuse(ECW_E_UNSUPPORTED, "matrix too large for one launch");
  auto* fn = x_dtype == ECW_DT_F32   ? k_mx4_quantise<ECW_DT_F32>
             : x_dtype == ECW_DT_F16 ? k_mx4_quantise<ECW_DT_F16>
                                     : k_mx4_quantise<ECW_DT_BF16>;
  hipLaunchKernelGGL(fn, dim3((uint32_t)grid), dim3(256), 0, (hipStream_t)stream, x, row_stride, rows, cols, octs,
                     static_cast<uint32_t*>(codes), static_cast<uint8_t*>(scales));
  return launched("mx4_quantize");
}

ecw_status mx4_dequantize(ecw_stream stream, const void* codes, const void* scales, uint32_t rows, uint32_t cols,
                          void* out, int out_dtype) {
  if (ecw_status s = check_matrix(codes, scales, rows, cols)) return s;
  if (out_dtype != ECW_DT_F16 && out_dtype != ECW_DT_BF16 && out_dtype != ECW_DT_F32)
    return refuse(ECW_E_INVALID_ARG, "output dtype must be F16, BF16 or F32");
  if (rows == 0) return ECW_OK;
  const uint32_t size = out_dtype == ECW_DT_F32 ? 4 : 2;
  if (!out || !aligned(out, size)) return refuse(ECW_E_INVALID_ARG, "output must be an aligned device pointer");
  const uint32_t octs = row_blocks(cols) * 4;
  const uint64_t grid = ((uint64_t)rows * octs + 255) / 256;
  if (!launchable(grid, 256)) return refuse(ECW_E_UNSUPPORTED, "matrix too large for one launch");
  auto* fn = out_dtype == ECW_DT_F32   ? k_mx4_dequantise<ECW_DT_F32>
             : out_dtype == ECW_DT_F16 ? k_mx4_dequantise<ECW_DT_F16>
                                       : k_mx4_dequantise<ECW_DT_BF16>;
  hipLaunchKernelGGL(fn, dim3((uint32_t)grid), dim3(256), 0, (hipStream_t)stream,
                     static_cast<const uint32_t*>(codes), static_cast<const uint8_t*>(scales), rows, cols, octs, out);
  return launched("mx4_dequantize");
}

}  // extern "C"
