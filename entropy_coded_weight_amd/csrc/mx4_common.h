// The microscaled 4-bit format (MX4) shared by its quantiser, product and key/value cache.
//
// 32 neighbouring elements form a block: one scale 2^s, held as the byte s + 127, and
// 32 codes of 4 bits (sign, two exponent bits, one mantissa bit: 0, 0.5, 1, 1.5, 2, 3,
// 4, 6 and their negatives), the lower element in the lower half of a byte.
//   s = floor(log2(largest magnitude)) - 2, held to -125..125 (an all-zero block: 0);
//   codes round to nearest, ties to the even code; magnitudes over 6 become 6.
// The lower limit keeps every value a normal fp32 and bf16 number.  A block that holds
// an infinity or a NaN has the byte 255 and stands for NaN throughout.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ecw_internal.h"

namespace ecw {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr uint32_t kScaleOne = 127;  // byte of the scale 1
constexpr uint32_t kScaleNaN = 255;

__device__ __forceinline__ float scale_of(uint32_t byte) { return __uint_as_float(byte << 23); }

// byte SEL of `codes` (two elements) as a pair of bf16 or fp16; the instruction takes the
// scale's exponent field, and 255 there gives NaN for every code.
template <int SEL>
__device__ __forceinline__ uint32_t pair_bf16(uint32_t codes, float scale) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, SEL));
}
template <int SEL>
__device__ __forceinline__ uint32_t pair_f16(uint32_t codes, float scale) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, scale, SEL));
}
// eight elements of one block
__device__ __forceinline__ bf16x8 oct_bf16(uint32_t codes, float scale) {
  const u32x4 v = {pair_bf16<0>(codes, scale), pair_bf16<1>(codes, scale), pair_bf16<2>(codes, scale),
                   pair_bf16<3>(codes, scale)};
  return __builtin_bit_cast(bf16x8, v);
}
__device__ __forceinline__ f16x8 oct_f16(uint32_t codes, float scale) {
  const u32x4 v = {pair_f16<0>(codes, scale), pair_f16<1>(codes, scale), pair_f16<2>(codes, scale),
                   pair_f16<3>(codes, scale)};
  return __builtin_bit_cast(f16x8, v);
}

// fp16 numbers as two bf16 numbers: the leading 8 bits and what is left.  An infinity or a
// NaN is whole in the first.
__device__ __forceinline__ void split_f16(u32x4 v, bf16x8* hi, bf16x8* lo) {
  u32x4 h, l;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const f16x2 p = __builtin_bit_cast(f16x2, (uint32_t)v[i]);
    const float a = (float)p[0], b = (float)p[1];
    const uint32_t ha = __float_as_uint(a) & 0xffff0000u, hb = __float_as_uint(b) & 0xffff0000u;
    const float la = (ha & 0x7f800000u) == 0x7f800000u ? 0.f : a - __uint_as_float(ha);
    const float lb = (hb & 0x7f800000u) == 0x7f800000u ? 0.f : b - __uint_as_float(hb);
    h[i] = ha >> 16 | hb;
    l[i] = __float_as_uint(la) >> 16 | (__float_as_uint(lb) & 0xffff0000u);
  }
  *hi = __builtin_bit_cast(bf16x8, h);
  *lo = __builtin_bit_cast(bf16x8, l);
}

// 16 bytes at any multiple of an element: memory instructions take them whole where rows
// are not 16-byte aligned too (a row of odd length in single elements costs 2 to 15 times
// the time).
struct __attribute__((packed, aligned(2))) Loose16 {
  u32x4 v;
};
struct __attribute__((packed, aligned(2))) Loose8 {
  u32x2 v;
};
struct __attribute__((packed, aligned(4))) Loose32 {
  f32x4 v;
};
struct __attribute__((packed, aligned(4))) Words {
  u32x4 v;
};

// Eight elements of an input row from column c on, zero from `cols` on.
struct Oct16 {
  u32x4 v;
};
__device__ __forceinline__ Oct16 load_oct16(const uint16_t* row, uint32_t c, uint32_t cols) {
  Oct16 r;
  if (c + 8 <= cols) {
    r.v = reinterpret_cast<const Loose16*>(row + c)->v;
    return r;
  }
  uint32_t e[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) e[i] = c + i < cols ? row[c + i] : 0u;
  r.v = u32x4{e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16};
  return r;
}
struct Oct32 {
  f32x4 a, b;
};
__device__ __forceinline__ Oct32 load_oct32(const float* row, uint32_t c, uint32_t cols) {
  Oct32 r;
  if (c + 8 <= cols) {
    r.a = reinterpret_cast<const Loose32*>(row + c)->v;
    r.b = reinterpret_cast<const Loose32*>(row + c + 4)->v;
    return r;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r.a[i] = c + i < cols ? row[c + i] : 0.f;
    r.b[i] = c + 4 + i < cols ? row[c + 4 + i] : 0.f;
  }
  return r;
}

// An eighth of a block's quantisation: a lane holds 8 neighbouring elements, four
// neighbouring lanes a block.  Gives the lane's 8 codes and the block's scale byte.
// Magnitudes are compared as integers (the order of finite floats, with infinities and
// NaN above them), so a NaN is never lost in a maximum.
__device__ __forceinline__ uint32_t block_max(uint32_t m) {
  m = max(m, (uint32_t)__shfl_xor((int)m, 1));
  return max(m, (uint32_t)__shfl_xor((int)m, 2));
}
__device__ __forceinline__ uint32_t scale_byte(uint32_t max_bits) {  // of the fp32 bits of the largest magnitude
  const uint32_t e = max_bits >> 23;
  const uint32_t b = e < 4 ? 2u : e - 2u;
  return e == 255 ? kScaleNaN : max_bits == 0 ? kScaleOne : b > 252 ? 252u : b;
}
template <bool F16>
__device__ __forceinline__ uint32_t quantise_oct(const Oct16& x, uint32_t* byte) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max(m, max(x.v[i] & 0x7fffu, (x.v[i] >> 16) & 0x7fffu));
  m = block_max(m);
  const uint32_t f = F16 ? __float_as_uint((float)__builtin_bit_cast(_Float16, (uint16_t)m)) : m << 16;
  const uint32_t b = scale_byte(f);
  const float s = scale_of(b);
  uint32_t c = 0;
  if constexpr (F16) {
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2, (uint32_t)x.v[0]), s, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2, (uint32_t)x.v[1]), s, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2, (uint32_t)x.v[2]), s, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2, (uint32_t)x.v[3]), s, 3);
  } else {
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, (uint32_t)x.v[0]), s, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, (uint32_t)x.v[1]), s, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, (uint32_t)x.v[2]), s, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, (uint32_t)x.v[3]), s, 3);
  }
  *byte = b;
  return c;
}
__device__ __forceinline__ uint32_t quantise_oct(const Oct32& x, uint32_t* byte) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    m = max(m, max(__float_as_uint(x.a[i]) & 0x7fffffffu, __float_as_uint(x.b[i]) & 0x7fffffffu));
  const uint32_t b = scale_byte(block_max(m));
  const float s = scale_of(b);
  uint32_t c = 0;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x.a[0], x.a[1], s, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x.a[2], x.a[3], s, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x.b[0], x.b[1], s, 2);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x.b[2], x.b[3], s, 3);
  *byte = b;
  return c;
}

// Eight elements of one block to memory as DT (ECW_DT_F16, _BF16 or _F32), the first
// `n` of them.
template <int DT>
__device__ __forceinline__ void store_oct(void* out, uint64_t at, uint32_t codes, float scale, uint32_t n) {
  if constexpr (DT == ECW_DT_F32) {
    float* o = static_cast<float*>(out) + at;
    const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, scale, 0);
    const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, scale, 1);
    const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, scale, 2);
    const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, scale, 3);
    if (n >= 8) {
      reinterpret_cast<Loose32*>(o)[0].v = f32x4{a[0], a[1], b[0], b[1]};
      reinterpret_cast<Loose32*>(o)[1].v = f32x4{c[0], c[1], d[0], d[1]};
      return;
    }
    const float v[8] = {a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if ((uint32_t)i < n) o[i] = v[i];
  } else {
    uint16_t* o = static_cast<uint16_t*>(out) + at;
    u32x4 v;
    if constexpr (DT == ECW_DT_F16)
      v = __builtin_bit_cast(u32x4, oct_f16(codes, scale));
    else
      v = __builtin_bit_cast(u32x4, oct_bf16(codes, scale));
    if (n >= 8) {
      reinterpret_cast<Loose16*>(o)->v = v;
      return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if ((uint32_t)i < n) o[i] = (uint16_t)(v[i / 2] >> (16 * (i & 1)));
  }
}

// blocks of a row, padded to whole 128-column spans: what a wave takes at a time
inline __host__ __device__ uint32_t row_blocks(uint32_t cols) { return (cols + 127) / 128 * 4; }
// bytes from one row's scales to the next: 16 bytes, the scales of four spans, are read at once
inline __host__ __device__ uint32_t scale_stride(uint32_t cols) { return (cols + 511) / 512 * 16; }

// fail() for entry points: no exception leaves them
ecw_status refuse(ecw_status s, const char* msg) noexcept;
ecw_status launched(const char* what) noexcept;  // the status after a launch

// A launch has fewer than 2^32 threads along its grid.
inline bool launchable(uint64_t blocks, uint32_t threads) { return blocks * threads >> 32 == 0; }

inline bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

}  // namespace ecw
