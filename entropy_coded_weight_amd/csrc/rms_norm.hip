// y = h / sqrt(mean(h^2) + eps) * weight over the rows of h = x + residual, y in a float
// type or in the block-scaled 8-bit format, h back into the residual stream.
//
// A row is held in registers between the sum of its squares and its output, so x and the
// residual are read once: LANES lanes hold it, 8 neighbouring columns at a time, OCTS times.
// h stays in fp32 and is rounded once, into the new residual; y is made of the unrounded h.
// The sum of squares is fp32: up to 32 products a lane in order, then a tree; numbers are
// multiplied by a power of two first, so that it stays in range as long as the mean does.  The factor and
// the products carry what their rounding lost along, so that y is rounded about once in fp32:
// next to the memory that costs nothing, and fewer numbers come to lie on the other side of
// an 8-bit border.  A group of lanes takes rows in turn and asks for the next one before it
// sums up the last.  Bound by memory (8191 rows of 4096 bf16 with a bf16 residual into 8 bits
// 39.5 us, 6.0 TB/s, with an fp32 one 69.5, 5.3); for a few rows by the latency of a load, the
// sum and a store (one row 3.5 us).  Rows of over 4096 columns, four octets a lane, need more
// scalar registers than there are, and from 1024 lanes on vector registers too, and read and
// write what is left over in between (1000 rows of 30000 52.7 us, 4.0 TB/s).
#include <type_traits>

#include "fp8_common.h"

namespace ecw {

struct NormArgs {
  const void *x, *residual, *weight;
  void *residual_out, *y;
  uint8_t* scales;  // of an 8-bit y
  int64_t x_stride, residual_stride, residual_out_stride;
  uint32_t rows, cols, octs, scale_row;
  int weight_dtype, y_dtype;  // weight_dtype 0: none; y_dtype 0: 8 bits
  float eps;
  float shrink, mean;         // a power of two, about 1 / sqrt(cols); 1 / cols without its square
};

// Eight columns of a row from column c on, as they lie (moved, see load_within) and as fp32.
// SMALL: rows may have less than eight.
template <int DT, bool SMALL>
__device__ __forceinline__ auto ask_oct(const void* row, uint32_t c, uint32_t cols) {
  if (SMALL && cols < 8) return load_oct<DT>(row, c, cols);
  return load_within<DT>(row, c, cols);
}
template <int DT, class T>
__device__ __forceinline__ void have_oct(float (&v)[8], T raw, uint32_t c, uint32_t cols) {
  if (c + 8 > cols && cols >= 8) raw = moved_down(raw, c - (cols - 8));
  widen<DT>(v, raw);
}
template <int DT, bool SMALL>
__device__ __forceinline__ void read_oct(float (&v)[8], const void* row, uint32_t c, uint32_t cols) {
  have_oct<DT>(v, ask_oct<DT, SMALL>(row, c, cols), c, cols);
}
template <bool SMALL>
__device__ __forceinline__ void weight_oct(float (&w)[8], const NormArgs& a, uint32_t c) {
  if (a.weight_dtype == ECW_DT_BF16) {
    read_oct<ECW_DT_BF16, SMALL>(w, a.weight, c, a.cols);
  } else if (a.weight_dtype == ECW_DT_F16) {
    read_oct<ECW_DT_F16, SMALL>(w, a.weight, c, a.cols);
  } else if (a.weight_dtype == ECW_DT_F32) {
    read_oct<ECW_DT_F32, SMALL>(w, a.weight, c, a.cols);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 1.f;
  }
}

// The sum over a row's LANES lanes, in every one of them.  `turn`: alternates between calls.
template <int LANES>
__device__ __forceinline__ float row_sum(float s, float (&sums)[2][16], uint32_t turn) {
  if constexpr (LANES == 8) {
    auto add = [&](auto step) { s += __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(s), decltype(step)::value, 0xf, 0xf, false)); };
    add(std::integral_constant<int, 0x141>{});  // lanes the other way round within 8
    add(std::integral_constant<int, 0xb1>{});   // neighbours
    add(std::integral_constant<int, 0x4e>{});   // pairs of a quad
    return s;
  }
  s = sum16(s);
  if constexpr (LANES >= 64) {
    s += __shfl_xor(s, 16);
    s += __shfl_xor(s, 32);
  }
  if constexpr (LANES > 64) {
    if ((threadIdx.x & 63) == 0) sums[turn][threadIdx.x / 64] = s;
    __syncthreads();
    s = 0.f;
#pragma unroll
    for (int i = 0; i < LANES / 64; ++i) s += sums[turn][i];
  }
  return s;
}

// DX: type of x; DR: of the residual, 0: none.  Blocks of max(LANES, 256) lanes take groups
// of rows in turn.
template <int DX, int DR, int LANES, int OCTS>
__global__ void __launch_bounds__(LANES < 256 ? 256 : LANES) k_rms_norm(NormArgs a) {
  constexpr uint32_t kBlock = LANES < 256 ? 256 : LANES, kRows = kBlock / LANES;
  constexpr int kX = DX == ECW_DT_F32 ? 4 : 2, kR = DR == ECW_DT_F32 ? 4 : 2;
  constexpr bool kSmall = LANES <= 16;
  constexpr bool kHold = OCTS <= 2;  // registers for the weight, and for the next row
  __shared__ float sums[2][16];
  const uint32_t lane = threadIdx.x % LANES;
  using X = std::conditional_t<DX == ECW_DT_F32, Oct32, Oct16>;
  using R = std::conditional_t<DR == ECW_DT_F32, Oct32, Oct16>;
  struct Row {
    X x[OCTS];
    R r[DR ? OCTS : 1];
  };
  auto row_of = [&](uint32_t first) { return kRows == 1 ? first : first + threadIdx.x / LANES; };
  // Only rows that there are are asked for: a residual that is written in place has another
  // lane's stores in it.  Lanes behind the last row take their turns over whatever they hold.
  // (Blocks of one row with registers for the next need no look here: each has a first row, and
  // the loop below looks before it asks.)
  auto ask = [&](Row& to, uint32_t first) {
    const uint32_t row = row_of(first);
    if ((kRows > 1 || !kHold) && row >= a.rows) return;
#pragma unroll
    for (int j = 0; j < OCTS; ++j) {
      const uint32_t c = (lane + j * LANES) * 8;
      to.x[j] = ask_oct<DX, kSmall>(static_cast<const uint8_t*>(a.x) + row * a.x_stride * kX, c, a.cols);
      if constexpr (DR != 0)
        to.r[j] = ask_oct<DR, kSmall>(static_cast<const uint8_t*>(a.residual) + row * a.residual_stride * kR, c, a.cols);
    }
  };
  Row raw;
  if constexpr (kRows > 1 || !kHold) raw = {};
  ask(raw, blockIdx.x * kRows);
  float w[kHold ? OCTS : 1][8];
  if constexpr (kHold) {
#pragma unroll
    for (int j = 0; j < OCTS; ++j) weight_oct<kSmall>(w[j], a, (lane + j * LANES) * 8);
  }
  // whether one of the lane's weights is infinite, which what was lost must not be multiplied by
  bool infinite = false;
  auto look = [&](const float (&of)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) infinite |= fabsf(of[i]) == INFINITY;
  };
  if constexpr (kHold) {
#pragma unroll
    for (int j = 0; j < OCTS; ++j) look(w[j]);
  }
  uint32_t turn = 0;
  for (uint32_t first = blockIdx.x * kRows; first < a.rows; first += gridDim.x * kRows, turn ^= 1) {
    const uint32_t row = row_of(first);
    const bool real = kRows == 1 || row < a.rows;
    float h[OCTS][8];
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < OCTS; ++j) {
      const uint32_t c = (lane + j * LANES) * 8;
      have_oct<DX>(h[j], raw.x[j], c, a.cols);
      if constexpr (DR != 0) {
        float r[8];
        have_oct<DR>(r, raw.r[j], c, a.cols);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[j][i] += r[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float u = h[j][i] * a.shrink;
        sum = fmaf(u, u, sum);
      }
    }
    if (kHold && first + gridDim.x * kRows < a.rows) ask(raw, first + gridDim.x * kRows);
    const float m = row_sum<LANES>(sum, sums, turn) * a.mean + a.eps;
    const bool tiny = m < 0x1p-96f;  // the instruction takes no subnormal numbers
    const float f = __builtin_amdgcn_rsqf(tiny ? m * 0x1p96f : m) * (tiny ? 0x1p48f : 1.f);
    // f + g is 1 / sqrt(m) to twice the precision: one step of Newton, its products exact (where
    // f is no ordinary number there is nothing to add)
    const float p = m * f, g0 = 0.5f * f * (fmaf(-p, f, 1.f) - fmaf(m, f, -p) * f), g = g0 - g0 == 0.f ? g0 : 0.f;
#pragma unroll
    for (int j = 0; j < OCTS; ++j) {
      const uint32_t oct = lane + j * LANES, c = oct * 8, n = a.cols > c ? a.cols - c : 0;
      if constexpr (DR != 0)
        if (real) store_values<DR>(static_cast<uint8_t*>(a.residual_out) + row * a.residual_out_stride * kR, c, h[j], n);
      float (&wj)[8] = w[kHold ? j : 0];
      if constexpr (!kHold) {
        weight_oct<kSmall>(wj, a, c);
        infinite = false;
        look(wj);
      }
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float hf = h[j][i] * f, lost = fmaf(h[j][i], g, fmaf(h[j][i], f, -hf));
        v[i] = fmaf(hf, wj[i], lost * wj[i]);
        if (infinite) v[i] = hf * wj[i];
      }
      const uint64_t at = (uint64_t)row * a.cols + c;
      if (a.y_dtype == 0) {
        uint32_t b;
        const u32x2 codes = fp8_oct(v, &b);
        if (real && oct < a.octs) store_fp8(static_cast<uint8_t*>(a.y), a.scales, row, oct, a.octs, a.scale_row, codes, b);
      } else if (real) {
        if (a.y_dtype == ECW_DT_BF16)
          store_values<ECW_DT_BF16>(a.y, at, v, n);
        else if (a.y_dtype == ECW_DT_F16)
          store_values<ECW_DT_F16>(a.y, at, v, n);
        else
          store_values<ECW_DT_F32>(a.y, at, v, n);
      }
    }
    if (!kHold) ask(raw, first + gridDim.x * kRows);
  }
}

}  // namespace ecw

using namespace ecw;

namespace {

constexpr uint32_t kNormMost = 32768;  // columns: 32 in each of 1024 lanes

template <int DX, int DR, int LANES, int OCTS>
ecw_status launch_norm(hipStream_t stream, const NormArgs& a) {
  constexpr uint32_t kBlock = LANES < 256 ? 256 : LANES, kRows = kBlock / LANES;
  const uint32_t groups = (a.rows + kRows - 1) / kRows, most = 256 * (2048 / kBlock);
  hipLaunchKernelGGL((k_rms_norm<DX, DR, LANES, OCTS>), dim3(groups < most ? groups : most), dim3(kBlock), 0, stream, a);
  return launched("rms_norm");
}

// Lanes of a row by its length.  Rows within a wave need no barrier (20000 rows of 1000 bf16
// columns with a residual into 8 bits 26.5 us in a wave of 2 octets a lane, 36.0 in blocks of
// 256 lanes), but 4 octets a lane are fewer rows in flight (8000 rows of 2048 18.4, in blocks
// 15.4).  300000 rows of 64 13.5 us by 8 lanes, 25.7 by 16.
template <int DX, int DR>
ecw_status launch_norm(hipStream_t stream, const NormArgs& a) {
  const uint32_t octs = (a.cols + 7) / 8;
  if (octs <= 8 && a.y_dtype != 0) return launch_norm<DX, DR, 8, 1>(stream, a);  // 8-bit blocks are 16 lanes
  if (octs <= 16) return launch_norm<DX, DR, 16, 1>(stream, a);
  if (octs <= 64) return launch_norm<DX, DR, 64, 1>(stream, a);
  if (octs <= 128) return launch_norm<DX, DR, 64, 2>(stream, a);
  if (octs <= 256) return launch_norm<DX, DR, 256, 1>(stream, a);
  if (octs <= 512) return launch_norm<DX, DR, 256, 2>(stream, a);
  if (octs <= 1024) return launch_norm<DX, DR, 256, 4>(stream, a);
  if (octs <= 2048) return launch_norm<DX, DR, 1024, 2>(stream, a);
  return launch_norm<DX, DR, 1024, 4>(stream, a);
}

}  // namespace

extern "C" ecw_status rms_norm(ecw_stream stream, const ecw_rms_norm* n) {
  if (!n) return refuse(ECW_E_INVALID_ARG, "norm is NULL");
  if (n->cols == 0 || n->rows > (1u << 30)) return refuse(ECW_E_INVALID_ARG, "cols must be positive, rows at most 2^30");
  if (n->cols > kNormMost) return refuse(ECW_E_UNSUPPORTED, "cols must be at most 32768");
  if (!is_float(n->x_dtype)) return refuse(ECW_E_INVALID_ARG, "x dtype must be F16, BF16 or F32");
  if (n->weight && !is_float(n->weight_dtype)) return refuse(ECW_E_INVALID_ARG, "weight dtype must be F16, BF16 or F32");
  const bool eight = n->y_dtype == ECW_DT_FP8_E4M3;
  if (!eight && !is_float(n->y_dtype)) return refuse(ECW_E_INVALID_ARG, "y dtype must be F16, BF16, F32 or FP8_E4M3");
  if (!(n->eps >= 0.f) || n->eps > 3.4e38f) return refuse(ECW_E_INVALID_ARG, "eps must be finite and not negative");
  if (n->residual && n->residual_dtype != n->x_dtype && n->residual_dtype != ECW_DT_F32)
    return refuse(ECW_E_UNSUPPORTED, "the residual must have x's dtype or F32");
  if (n->rows == 0) return ECW_OK;
  if (!n->x || !aligned(n->x, size_of(n->x_dtype))) return refuse(ECW_E_INVALID_ARG, "x must be an aligned device pointer");
  if (!n->y || !aligned(n->y, eight ? 16 : size_of(n->y_dtype)))
    return refuse(ECW_E_INVALID_ARG, "y must be an aligned device pointer");
  if (eight && (!n->y_scales || !aligned(n->y_scales, 16)))
    return refuse(ECW_E_INVALID_ARG, "scales must be a 16-byte aligned device pointer");
  if (n->weight && !aligned(n->weight, size_of(n->weight_dtype)))
    return refuse(ECW_E_INVALID_ARG, "weight must be an aligned device pointer");
  if (!n->residual != !n->residual_out)
    return refuse(ECW_E_INVALID_ARG, "residual and residual_out come together");
  if (n->residual && (!aligned(n->residual, size_of(n->residual_dtype)) || !aligned(n->residual_out, size_of(n->residual_dtype))))
    return refuse(ECW_E_INVALID_ARG, "residual and residual_out must be aligned device pointers");
  if (n->x_stride < 0 || (n->residual && (n->residual_stride < 0 || n->residual_out_stride < n->cols)))
    return refuse(ECW_E_INVALID_ARG, "row strides must not be negative, residual_out's at least cols");
  if (n->residual && n->residual == n->residual_out && n->rows > 1 && n->residual_stride != n->residual_out_stride)
    return refuse(ECW_E_INVALID_ARG, "in place the residual's strides must be the same");
  float shrink = 1.f;
  while (shrink * shrink * (float)n->cols > 1.f) shrink *= 0.5f;
  const NormArgs a{n->x, n->residual, n->weight, n->residual_out, n->y, static_cast<uint8_t*>(n->y_scales),
                   n->x_stride, n->residual_stride, n->residual_out_stride,
                   n->rows, n->cols, fp8_row(n->cols) / 8, fp8_scale_row(n->cols),
                   n->weight ? n->weight_dtype : 0, eight ? 0 : n->y_dtype, n->eps, shrink,
                   1.f / ((float)n->cols * shrink * shrink)};
  const auto s = (hipStream_t)stream;
  const int dr = n->residual ? n->residual_dtype : 0;
  if (n->x_dtype == ECW_DT_F32) return dr ? launch_norm<ECW_DT_F32, ECW_DT_F32>(s, a) : launch_norm<ECW_DT_F32, 0>(s, a);
  if (n->x_dtype == ECW_DT_F16)
    return dr == 0             ? launch_norm<ECW_DT_F16, 0>(s, a)
           : dr == ECW_DT_F32 ? launch_norm<ECW_DT_F16, ECW_DT_F32>(s, a)
                              : launch_norm<ECW_DT_F16, ECW_DT_F16>(s, a);
  return dr == 0             ? launch_norm<ECW_DT_BF16, 0>(s, a)
         : dr == ECW_DT_F32 ? launch_norm<ECW_DT_BF16, ECW_DT_F32>(s, a)
                            : launch_norm<ECW_DT_BF16, ECW_DT_BF16>(s, a);
}
