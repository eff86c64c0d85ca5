// Rotary positions: pairs of a head's dimensions turned by an angle that grows with the
// row's position, which may stand on several axes (time, height, width: each pair follows
// one of them).
//
// The angle of pair j of a row is position * inv_freq[j].  It is needed modulo a turn, and
// at position 2^20 fp32 holds it to a sixteenth of a radian.  Frequencies are kept as 64-bit
// fractions of a turn, so that a product with a whole position, of either sign, wraps round
// by itself and is exact to 2^-65 times the position.  Its upper 32 bits, an eighth of a
// turn to either side of a quarter, go through the Taylor series of sine and cosine (the
// first term left out is under 2^-29 and 2^-31).
//
// A lane holds 8 pairs of a row and turns them in some heads of q and k, one after the other
// with one set of sines, the next head asked for before one is stored.  Neighbouring lanes
// have neighbouring heads.  Bound by memory (8191 rows of 40 heads of 128 in bf16 on three axes
// 39.4 us, 4.3 TB/s, in place 34.3); for a few rows by latency (8 rows 3.8 us: positions,
// then sines, with the first head's load next to them).
#include <type_traits>

#include "fp8_common.h"

namespace ecw {

struct RotaryArgs {
  const void *q, *k;
  void *q_out, *k_out;
  const void* positions;
  const uint64_t* freqs;  // [pairs] fractions of a turn in 2^-64
  const uint8_t* axes;    // [pairs]
  int64_t q_row, q_head, k_row, k_head, qo_row, qo_head, ko_row, ko_head, axis_stride;
  uint32_t rows, q_heads, heads, dim, pairs, n_axes;  // heads: of q and k together
  uint32_t lanes;       // of a row and head: 8 pairs each, then 16 dimensions that are only copied
  uint32_t parts;       // lanes along a row's heads: part p has heads p, p + parts, ...
  uint32_t wide;        // positions of 64 bits
  uint32_t copy;        // dimensions past the pairs are copied
  float scale;
};

// cosine and sine of `turn` 2^-32 turns
__device__ __forceinline__ void cos_sin(uint32_t turn, float* c, float* s) {
  const uint32_t quarter = (turn + 0x20000000u) >> 30;
  const float a = (float)(int32_t)(turn - (quarter << 30)) * 1.46291807926715968e-9f;  // 2 pi / 2^32
  const float z = a * a;
  float sn = fmaf(z, 2.75573192e-6f, -1.98412698e-4f);  // 1/9!, -1/7!
  sn = fmaf(z, sn, 8.33333333e-3f);
  sn = fmaf(z, sn, -1.66666667e-1f);
  sn = fmaf(a * z, sn, a);
  float cs = fmaf(z, -2.75573192e-7f, 2.48015873e-5f);  // -1/10!, 1/8!
  cs = fmaf(z, cs, -1.38888889e-3f);
  cs = fmaf(z, cs, 4.16666667e-2f);
  cs = fmaf(z, cs, -0.5f);
  cs = fmaf(z, cs, 1.f);
  const float p = quarter & 1 ? sn : cs, r = quarter & 1 ? cs : sn;
  *c = (quarter + 1) & 2 ? -p : p;
  *s = quarter & 2 ? -r : r;
}

// NEAR: a pair is two neighbouring dimensions; else dimension j and j + pairs.  WHOLE: every
// lane has all of its 16 dimensions.
template <int DT, bool NEAR, bool WHOLE>
__global__ void __launch_bounds__(256) k_rotary(RotaryArgs a) {
  constexpr int kSize = DT == ECW_DT_F32 ? 4 : 2;
  const uint32_t at = blockIdx.x * 256 + threadIdx.x;  // the host keeps the launch under 2^32 lanes
  const uint32_t group = at / a.lanes, lane = at - group * a.lanes;
  const uint32_t row = group / a.parts, part = group - row * a.parts;
  if (row >= a.rows) return;
  const uint32_t turned = (a.pairs + 7) / 8;
  auto from = [&](uint32_t head) {
    return head < a.q_heads ? static_cast<const uint8_t*>(a.q) + (row * a.q_row + head * a.q_head) * kSize
                            : static_cast<const uint8_t*>(a.k) + (row * a.k_row + (head - a.q_heads) * a.k_head) * kSize;
  };
  auto to = [&](uint32_t head) {
    return head < a.q_heads ? static_cast<uint8_t*>(a.q_out) + (row * a.qo_row + head * a.qo_head) * kSize
                            : static_cast<uint8_t*>(a.k_out) + (row * a.ko_row + (head - a.q_heads) * a.ko_head) * kSize;
  };
  // two octets of dimensions of a head: where they start, and how much of each there is
  uint32_t d0, d1, n0, n1;
  const bool turns = lane < turned;
  const uint32_t j0 = lane * 8;
  if (!turns) {  // 16 dimensions that are only copied
    d0 = 2 * a.pairs + (lane - turned) * 16, d1 = d0 + 8;
    n0 = min(a.dim - d0, 8u), n1 = a.dim > d1 ? min(a.dim - d1, 8u) : 0;
  } else if (NEAR) {
    d0 = 2 * j0, d1 = d0 + 8;
    n0 = min(2 * a.pairs - d0, 8u), n1 = 2 * a.pairs > d1 ? min(2 * a.pairs - d1, 8u) : 0;
  } else {
    d0 = j0, d1 = a.pairs + j0;
    n0 = n1 = min(a.pairs - j0, 8u);
  }
  using Oct = std::conditional_t<DT == ECW_DT_F32, Oct32, Oct16>;
  Oct u, v;
  auto ask = [&](uint32_t head) {
    const uint8_t* x = from(head);
    u = load_oct<DT>(x, d0, WHOLE ? ~0u : d0 + n0);
    v = load_oct<DT>(x, d1, WHOLE ? ~0u : d1 + n1);
  };
  ask(part);
  float c[8], s[8];
  if (turns) {
    int64_t position = 0;
    auto position_of = [&](uint32_t axis) {
      const int64_t p = axis * a.axis_stride + row;
      return a.wide ? static_cast<const int64_t*>(a.positions)[p] : (int64_t)static_cast<const int32_t*>(a.positions)[p];
    };
    if (a.n_axes == 1) position = position_of(0);
#pragma unroll
    for (uint32_t i = 0; i < 8; ++i) {
      const uint32_t j = WHOLE ? j0 + i : min(j0 + i, a.pairs - 1);
      if (a.n_axes > 1) position = position_of(min((uint32_t)a.axes[j], a.n_axes - 1));
      cos_sin((uint32_t)(((uint64_t)position * a.freqs[j] + (1ull << 31)) >> 32), &c[i], &s[i]);
      c[i] *= a.scale;
      s[i] *= a.scale;
    }
  }
  for (uint32_t head = part; head < a.heads; head += a.parts) {
    float x[8], y[8];
    widen<DT>(x, u);
    widen<DT>(y, v);
    if (head + a.parts < a.heads) ask(head + a.parts);
    if (turns) {
      auto turn = [&](float& e, float& o, int k) {
        const float before = e;
        e = fmaf(e, c[k], -(o * s[k]));
        o = fmaf(o, c[k], before * s[k]);
      };
      if constexpr (NEAR) {
#pragma unroll
        for (int k = 0; k < 4; ++k) turn(x[2 * k], x[2 * k + 1], k), turn(y[2 * k], y[2 * k + 1], 4 + k);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) turn(x[k], y[k], k);
      }
    }
    store_values<DT>(to(head), d0, x, WHOLE ? 8 : n0);
    if (WHOLE || n1) store_values<DT>(to(head), d1, y, WHOLE ? 8 : n1);
  }
}

}  // namespace ecw

using namespace ecw;

namespace {

template <int DT, bool NEAR>
void launch_rotary(hipStream_t stream, uint32_t grid, const RotaryArgs& a) {
  const bool whole = a.pairs % 8 == 0 && (!a.copy || (a.dim - 2 * a.pairs) % 16 == 0);
  if (whole)
    hipLaunchKernelGGL((k_rotary<DT, NEAR, true>), dim3(grid), dim3(256), 0, stream, a);
  else
    hipLaunchKernelGGL((k_rotary<DT, NEAR, false>), dim3(grid), dim3(256), 0, stream, a);
}
template <int DT>
void launch_rotary(hipStream_t stream, uint32_t grid, bool near, const RotaryArgs& a) {
  if (near)
    launch_rotary<DT, true>(stream, grid, a);
  else
    launch_rotary<DT, false>(stream, grid, a);
}

}  // namespace

extern "C" ecw_status rotary_apply(ecw_stream stream, const ecw_rotary* r) {
  if (!r) return refuse(ECW_E_INVALID_ARG, "rotary is NULL");
  if (!is_float(r->dtype)) return refuse(ECW_E_INVALID_ARG, "dtype must be F16, BF16 or F32");
  if (r->head_dim == 0 || r->head_dim > 4096 || r->rotary_dim == 0 || r->rotary_dim % 2 || r->rotary_dim > r->head_dim)
    return refuse(ECW_E_INVALID_ARG, "head_dim must be in [1, 4096], rotary_dim even, positive and at most head_dim");
  if (r->axes == 0 || r->axes > 255) return refuse(ECW_E_INVALID_ARG, "axes must be in [1, 255]");
  if (r->rows >= 1u << 30 || r->q_heads > 65536 || r->k_heads > 65536)
    return refuse(ECW_E_INVALID_ARG, "rows must be below 2^30, heads at most 65536");
  if (!(r->scale - r->scale == 0.f)) return refuse(ECW_E_INVALID_ARG, "scale must be finite");
  const uint32_t heads = r->q_heads + r->k_heads, size = size_of(r->dtype);
  if (r->rows == 0 || heads == 0) return ECW_OK;
  if (!r->freqs || !aligned(r->freqs, 8) || !r->axis_of || !r->positions || !aligned(r->positions, r->wide_positions ? 8 : 4))
    return refuse(ECW_E_INVALID_ARG, "freqs, axis_of and positions must be aligned device pointers");
  if (r->q_heads && (!r->q || !r->q_out || !aligned(r->q, size) || !aligned(r->q_out, size)))
    return refuse(ECW_E_INVALID_ARG, "q and q_out must be aligned device pointers");
  if (r->k_heads && (!r->k || !r->k_out || !aligned(r->k, size) || !aligned(r->k_out, size)))
    return refuse(ECW_E_INVALID_ARG, "k and k_out must be aligned device pointers");
  const int64_t strides[] = {r->q_row, r->q_head, r->k_row, r->k_head, r->q_out_row, r->q_out_head, r->k_out_row,
                             r->k_out_head, r->axis_stride};
  for (int64_t s : strides)
    if (s < 0) return refuse(ECW_E_INVALID_ARG, "strides must not be negative");
  if ((r->q_heads && r->q == r->q_out && (r->q_row != r->q_out_row || r->q_head != r->q_out_head)) ||
      (r->k_heads && r->k == r->k_out && (r->k_row != r->k_out_row || r->k_head != r->k_out_head)))
    return refuse(ECW_E_INVALID_ARG, "in place the strides must be the same");
  RotaryArgs a{r->q, r->k, r->q_out, r->k_out, r->positions, static_cast<const uint64_t*>(r->freqs),
               static_cast<const uint8_t*>(r->axis_of), r->q_row, r->q_head, r->k_row, r->k_head, r->q_out_row,
               r->q_out_head, r->k_out_row, r->k_out_head, r->axis_stride, r->rows, r->q_heads, heads, r->head_dim,
               r->rotary_dim / 2, r->axes, 0, 0, r->wide_positions ? 1u : 0u, 0, r->scale};
  const bool in_place = (!r->q_heads || r->q == r->q_out) && (!r->k_heads || r->k == r->k_out);
  a.copy = !in_place && r->rotary_dim < r->head_dim;
  a.lanes = (a.pairs + 7) / 8 + (a.copy ? (r->head_dim - r->rotary_dim + 15) / 16 : 0);
  // up to eight heads a lane while there are lanes enough, for sines cost as much as a head or
  // two (8191 rows of 40 heads of 128: 8 heads 39 us, 4 45, 16 44; 4000 rows of 40 heads of 64
  // 12.2 us, with one head a lane 17.2)
  uint32_t each = 1;
  while (each < 8 && each < heads && (uint64_t)r->rows * a.lanes * ((heads + 2 * each - 1) / (2 * each)) >= 256 * 512) each *= 2;
  a.parts = (heads + each - 1) / each;
  const uint64_t grid = ((uint64_t)r->rows * a.parts * a.lanes + 255) / 256;
  if (!launchable(grid, 256)) return refuse(ECW_E_UNSUPPORTED, "too many rows and heads for one launch");
  const auto s = (hipStream_t)stream;
  if (r->dtype == ECW_DT_F32)
    launch_rotary<ECW_DT_F32>(s, (uint32_t)grid, r->neighbours, a);
  else if (r->dtype == ECW_DT_F16)
    launch_rotary<ECW_DT_F16>(s, (uint32_t)grid, r->neighbours, a);
  else
    launch_rotary<ECW_DT_BF16>(s, (uint32_t)grid, r->neighbours, a);
  return launched("rotary_apply");
}
