// The block-scaled 8-bit format (FP8) shared by its quantiser, the norm and the product.
//
// 128 neighbouring columns of a row form a block: one scale 2^s, held as the byte s + 127,
// and 128 E4M3 numbers (largest 448, smallest 2^-9).
//   s = the smallest with largest magnitude <= 448 * 2^s, held to -117..119 (an all-zero
//       block: 0);
//   numbers round to nearest, ties to even; magnitudes over 448 (at s = 119 only) become 448.
// The limits keep every value a normal fp32 and bf16 number.  A block that holds an infinity
// or a NaN has the byte 255, its numbers are NaN.  A power of two as the scale costs a normal
// number no precision, and the matrix instruction multiplies by it.
#pragma once
#include "mx4_common.h"

namespace ecw {

constexpr uint32_t kFp8Least = 10, kFp8Most = 246;  // bytes of s = -117 and 119
constexpr float kFp8Top = 448.f;

// bytes from one row's codes, and scales, to the next
inline __host__ __device__ uint32_t fp8_row(uint32_t cols) { return (cols + 127) / 128 * 128; }
inline __host__ __device__ uint32_t fp8_scale_row(uint32_t cols) { return (cols + 2047) / 2048 * 16; }

// x moved N lanes round within each 16
template <int N>
__device__ __forceinline__ uint32_t turn16(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x120 + N, 0xf, 0xf, false);
}
// the largest of 16 neighbouring lanes, and their sum
__device__ __forceinline__ uint32_t max16(uint32_t m) {
  m = max(m, turn16<8>(m));
  m = max(m, turn16<4>(m));
  m = max(m, turn16<2>(m));
  return max(m, turn16<1>(m));
}
__device__ __forceinline__ float sum16(float s) {
  s += __uint_as_float(turn16<8>(__float_as_uint(s)));
  s += __uint_as_float(turn16<4>(__float_as_uint(s)));
  s += __uint_as_float(turn16<2>(__float_as_uint(s)));
  return s + __uint_as_float(turn16<1>(__float_as_uint(s)));
}

// Byte of the scale, of the fp32 bits of the largest magnitude (448 = 1.75 * 2^8: one more
// where the fraction is over 0.75).
__device__ __forceinline__ uint32_t fp8_scale_byte(uint32_t max_bits) {
  if (max_bits >= 0x7f800000u) return kScaleNaN;
  const uint32_t e = (max_bits + 0x1fffffu) >> 23;
  return max_bits == 0 ? kScaleOne : min(max(e, kFp8Least + 8) - 8, kFp8Most);
}

// A sixteenth of a block: a lane holds 8 neighbouring values, 16 neighbouring lanes a block.
// Magnitudes are compared as integers, so that a NaN is never lost in a maximum.
__device__ __forceinline__ u32x2 fp8_oct(const float (&v)[8], uint32_t* byte) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
  const uint32_t b = fp8_scale_byte(max16(m));
  *byte = b;
  if (b == kScaleNaN) return u32x2{0x7f7f7f7fu, 0x7f7f7f7fu};
  const float s = scale_of(254 - b);  // 2^-s
  float u[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) u[i] = __builtin_amdgcn_fmed3f(v[i] * s, -kFp8Top, kFp8Top);
  int lo = 0, hi = 0;
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(u[0], u[1], lo, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(u[2], u[3], lo, true);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(u[4], u[5], hi, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(u[6], u[7], hi, true);
  return u32x2{(uint32_t)lo, (uint32_t)hi};
}

// Eight codes and their block's scale to memory.  The lane of a row's last block's first
// codes fills the row's scales up to 16 bytes.
__device__ __forceinline__ void store_fp8(uint8_t* codes, uint8_t* scales, uint32_t row, uint32_t oct, uint32_t octs,
                                          uint32_t scale_row, u32x2 c, uint32_t byte) {
  reinterpret_cast<u32x2*>(codes)[(uint64_t)row * octs + oct] = c;
  if (oct % 16 == 0) {
    uint8_t* to = scales + (uint64_t)row * scale_row + oct / 16;
    *to = (uint8_t)byte;
    if (oct + 16 == octs)
      for (uint32_t i = octs / 16; i < scale_row; ++i) *++to = kScaleOne;
  }
}

// Eight elements of a row of type DT from column c on, zeros from `cols` on.  What is left of
// a row's last eight goes in pieces of 4, 2 and 1: of each, and no element by itself, so that
// many of them in a kernel stay small.
struct __attribute__((packed, aligned(2))) Loose4 {
  uint32_t v;
};
struct __attribute__((packed, aligned(4))) Words2 {
  f32x2 v;
};
template <int DT>
__device__ __forceinline__ auto load_oct(const void* from, uint32_t c, uint32_t cols) {
  if constexpr (DT == ECW_DT_F32) {
    const float* row = static_cast<const float*>(from) + c;
    Oct32 r;
    if (c + 8 <= cols) {
      r.a = reinterpret_cast<const Loose32*>(row)->v;
      r.b = reinterpret_cast<const Loose32*>(row + 4)->v;
      return r;
    }
    const uint32_t n = c < cols ? cols - c : 0;
    r.a = r.b = f32x4{0.f, 0.f, 0.f, 0.f};
    f32x4 half = r.a;  // the last 0 to 3
    if (n & 2) {
      const f32x2 t = reinterpret_cast<const Words2*>(row + (n & 4))->v;
      half[0] = t[0], half[1] = t[1];
    }
    if (n & 1) {
      const float t = row[n - 1];
      half = n & 2 ? f32x4{half[0], half[1], t, 0.f} : f32x4{t, 0.f, 0.f, 0.f};
    }
    if (n & 4) {
      r.a = reinterpret_cast<const Loose32*>(row)->v;
      r.b = half;
    } else {
      r.a = half;
    }
    return r;
  } else {
    const uint16_t* row = static_cast<const uint16_t*>(from) + c;
    Oct16 r;
    if (c + 8 <= cols) {
      r.v = reinterpret_cast<const Loose16*>(row)->v;
      return r;
    }
    const uint32_t n = c < cols ? cols - c : 0;
    uint32_t pair = 0, one = 0;
    u32x2 four = {0, 0};
    if (n & 1) one = row[n - 1];
    if (n & 2) pair = reinterpret_cast<const Loose4*>(row + (n & 4))->v;
    if (n & 4) four = reinterpret_cast<const Loose8*>(row)->v;
    const uint32_t w0 = n & 2 ? pair : one, w1 = n & 2 ? one : 0;
    r.v = n & 4 ? u32x4{four[0], four[1], w0, w1} : u32x4{w0, w1, 0, 0};
    return r;
  }
}
// The same of a row of at least 8 columns, by one load that no branch is in the way of: from
// column min(c, cols - 8), and moved down by what is too much once it is there.
template <int DT>
__device__ __forceinline__ auto load_within(const void* row, uint32_t c, uint32_t cols) {
  const uint32_t at = min(c, cols - 8);
  if constexpr (DT == ECW_DT_F32) {
    const float* from = static_cast<const float*>(row) + at;
    return Oct32{reinterpret_cast<const Loose32*>(from)->v, reinterpret_cast<const Loose32*>(from + 4)->v};
  } else {
    return Oct16{reinterpret_cast<const Loose16*>(static_cast<const uint16_t*>(row) + at)->v};
  }
}
__device__ __forceinline__ Oct16 moved_down(const Oct16& x, uint32_t by) {
  const unsigned __int128 t = __builtin_bit_cast(unsigned __int128, x.v);
  return {__builtin_bit_cast(u32x4, by < 8 ? t >> (16 * by) : (unsigned __int128)0)};
}
__device__ __forceinline__ Oct32 moved_down(const Oct32& x, uint32_t by) {
  float v[16] = {x.a[0], x.a[1], x.a[2], x.a[3], x.b[0], x.b[1], x.b[2], x.b[3]};
#pragma unroll
  for (int k = 8; k > 0; k /= 2)
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = min(by, 8u) & k ? v[i + k] : v[i];
  return {{v[0], v[1], v[2], v[3]}, {v[4], v[5], v[6], v[7]}};
}
template <int DT>
__device__ __forceinline__ void widen(float (&v)[8], const Oct16& x) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (DT == ECW_DT_F16) {
      const f16x2 p = __builtin_bit_cast(f16x2, (uint32_t)x.v[i]);
      v[2 * i] = (float)p[0], v[2 * i + 1] = (float)p[1];
    } else {
      v[2 * i] = __uint_as_float(x.v[i] << 16), v[2 * i + 1] = __uint_as_float(x.v[i] & 0xffff0000u);
    }
  }
}
template <int DT>
__device__ __forceinline__ void widen(float (&v)[8], const Oct32& x) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = x.a[i], v[4 + i] = x.b[i];
}

// Eight fp32 values rounded to DT, the first `n` of them to memory.
template <int DT>
__device__ __forceinline__ void store_values(void* out, uint64_t at, const float (&v)[8], uint32_t n) {
  if constexpr (DT == ECW_DT_F32) {
    float* o = static_cast<float*>(out) + at;
    const f32x4 a = {v[0], v[1], v[2], v[3]}, b = {v[4], v[5], v[6], v[7]};
    if (n >= 4) reinterpret_cast<Loose32*>(o)->v = a;
    if (n >= 8) {
      reinterpret_cast<Loose32*>(o + 4)->v = b;
      return;
    }
    const f32x4 half = n & 4 ? b : a;
    if (n & 2) reinterpret_cast<Words2*>(o + (n & 4))->v = f32x2{half[0], half[1]};
    if (n & 1) o[n - 1] = n & 2 ? half[2] : half[0];
  } else {
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (DT == ECW_DT_F16)
        w[i] = __builtin_bit_cast(uint32_t, f16x2{(_Float16)v[2 * i], (_Float16)v[2 * i + 1]});
      else
        w[i] = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)v[2 * i], (__bf16)v[2 * i + 1]});
    }
    uint16_t* o = static_cast<uint16_t*>(out) + at;
    if (n >= 8) {
      reinterpret_cast<Loose16*>(o)->v = w;
      return;
    }
    const u32x2 half = n & 4 ? u32x2{w[2], w[3]} : u32x2{w[0], w[1]};
    if (n & 4) reinterpret_cast<Loose8*>(o)->v = u32x2{w[0], w[1]};
    if (n & 2) reinterpret_cast<Loose4*>(o + (n & 4))->v = half[0];
    if (n & 1) o[n - 1] = (uint16_t)(n & 2 ? half[1] : half[0]);
  }
}

inline ecw_status check_fp8(const void* codes, const void* scales, uint32_t rows, uint32_t cols) {
  if (cols == 0 || cols > (1u << 30) || rows > (1u << 30))
    return refuse(ECW_E_INVALID_ARG, "cols must be in [1, 2^30], rows at most 2^30");
  if ((uint64_t)rows * fp8_row(cols) >> 40) return refuse(ECW_E_INVALID_ARG, "matrix too large");
  if (rows && (!codes || !scales || !aligned(codes, 16) || !aligned(scales, 16)))
    return refuse(ECW_E_INVALID_ARG, "codes and scales must be 16-byte aligned device pointers");
  return ECW_OK;
}

inline bool is_float(int dt) { return dt == ECW_DT_F16 || dt == ECW_DT_BF16 || dt == ECW_DT_F32; }
inline uint32_t size_of(int dt) { return dt == ECW_DT_F32 ? 4 : 2; }

}  // namespace ecw
