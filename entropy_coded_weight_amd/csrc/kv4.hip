// A paged key/value cache in the microscaled 4-bit format: append, read back, attention.
//
// Layout of one page of one head (P tokens of D = 32 NB dimensions), all regions
// whole multiples of 128 bytes:
//   keys    [P][D / 2]                    a token's codes in order: the matrix
//                                         instruction's operand for q k^T as it lies
//   values  [P / 4][16][4][NB]            four tokens x 16 groups of 2 NB dimensions: a
//                                         lane reads its dimensions of four tokens at once
//   key scales   [P][NB]
//   value scales [P / 4][NB][4]
// Writing a token touches only bytes of its own, so appends never read.
#include <algorithm>
#include <type_traits>

#include "mx4_common.h"

namespace ecw {

struct Cache {
  uint8_t* data;
  uint32_t pages, heads, dim, page_tokens;
};

// Which rows belong to which sequence and where they stand in it: sequence b's rows
// are its last tokens.
struct Batch {
  const int32_t* table;   // [batch][wide], entries outside 0..pages-1 hold no page
  const int32_t* lens;    // tokens of each sequence, its new rows among them
  const int32_t* starts;  // [batch + 1] first rows, or null: rows / batch each
  int64_t stride;         // of the table
  uint32_t batch, wide, rows;
};

inline __host__ __device__ uint64_t region_bytes(const Cache& c) { return (uint64_t)c.page_tokens * c.dim * 17 / 32 * 2; }
// parts of a region, in bytes
__device__ __forceinline__ uint32_t plane_bytes(const Cache& c) { return c.page_tokens * (c.dim / 2); }
__device__ __forceinline__ uint32_t scale_bytes(const Cache& c) { return c.page_tokens * (c.dim / 32); }

// The sequence of a row, its rows and the row's place among them; false: of none.
__device__ __forceinline__ bool find_row(const Batch& t, uint32_t row, uint32_t* b, int32_t* n, int32_t* i) {
  if (!t.starts) {
    const uint32_t each = t.rows / t.batch;
    *b = row / each;
    *n = (int32_t)each;
    *i = (int32_t)(row - *b * each);
    return true;
  }
  uint32_t lo = 0, hi = t.batch;
  while (hi - lo > 1) {
    const uint32_t mid = (lo + hi) / 2;
    if (t.starts[mid] <= (int32_t)row)
      lo = mid;
    else
      hi = mid;
  }
  const int32_t first = t.starts[lo], end = min(t.starts[lo + 1], (int32_t)t.rows);
  if (first < 0 || (int32_t)row < first || (int32_t)row >= end) return false;
  *b = lo;
  *n = end - first;
  *i = (int32_t)row - first;
  return true;
}

// The page region of a row's token and the token's place in it; null: it has none.
__device__ __forceinline__ uint8_t* place(const Cache& c, const Batch& t, uint32_t row, uint32_t head, uint32_t* at) {
  uint32_t b;
  int32_t n, i;
  if (!find_row(t, row, &b, &n, &i)) return nullptr;
  const int64_t pos = (int64_t)t.lens[b] - n + i;
  if (pos < 0 || pos >= (int64_t)t.wide * c.page_tokens) return nullptr;
  const uint32_t p = (uint32_t)((uint64_t)pos / c.page_tokens);
  const int32_t page = t.table[b * t.stride + p];
  if (page < 0 || (uint32_t)page >= c.pages) return nullptr;
  *at = (uint32_t)(pos - (int64_t)p * c.page_tokens);
  return c.data + ((uint64_t)page * c.heads + head) * region_bytes(c);
}

// Codes of dimensions 8 u .. 8 u + 7 of a token's value: one word, or for two
// dimensions a byte (NB = 2: four dimensions a group) two halves.
__device__ __forceinline__ uint32_t value_at(uint32_t nb, uint32_t token, uint32_t dim) {
  const uint32_t group = dim / (2 * nb), in = dim % (2 * nb);
  return ((token / 4 * 16 + group) * 4 + token % 4) * nb + in / 2;
}

template <int DT>
__device__ __forceinline__ uint32_t quantise_row(const void* x, int64_t at, uint32_t u, uint32_t dim,
                                                 uint32_t* byte) {
  if constexpr (DT == ECW_DT_F32)
    return quantise_oct(load_oct32(static_cast<const float*>(x) + at, u * 8, dim), byte);
  else
    return quantise_oct<DT == ECW_DT_F16>(load_oct16(static_cast<const uint16_t*>(x) + at, u * 8, dim), byte);
}

// A block has 256 / octs neighbouring rows of one head: four tokens' values share lines,
// which blocks on different dies would each write a part of.  Gives the lane's row and head.
__device__ __forceinline__ uint32_t row_of(const Cache& c, uint32_t octs, uint32_t* head) {
  const uint32_t group = blockIdx.x / c.heads;
  *head = blockIdx.x - group * c.heads;
  return group * (256 / octs) + threadIdx.x / octs;
}

// A lane per 8 dimensions of one head of one row, keys and values both.  Bound by memory
// (16384 rows of 8 heads of 128 dimensions 19.7 us, 4.3 TB/s; 24.0 with a block's rows of
// several heads); for a few rows by the latency of the page look-up and the loads next to
// it (64 rows 3.6 us).
template <int DT>
__global__ void __launch_bounds__(256) k_kv4_append(Cache c, Batch t, const void* __restrict__ k,
                                                    const void* __restrict__ v, int64_t k_row, int64_t k_head,
                                                    int64_t v_row, int64_t v_head) {
  const uint32_t octs = c.dim / 8, nb = c.dim / 32, u = threadIdx.x % octs;
  uint32_t head;
  const uint32_t row = row_of(c, octs, &head);
  if (row >= t.rows) return;  // whole blocks: a head's lanes stay together
  uint32_t kb, vb, at = 0;
  const uint32_t kc = quantise_row<DT>(k, row * k_row + head * k_head, u, c.dim, &kb);
  const uint32_t vc = quantise_row<DT>(v, row * v_row + head * v_head, u, c.dim, &vb);
  uint8_t* to = place(c, t, row, head, &at);
  if (!to) return;
  *reinterpret_cast<uint32_t*>(to + (uint64_t)at * (c.dim / 2) + u * 4) = kc;
  uint8_t* vals = to + plane_bytes(c);
  if (nb == 2) {
    *reinterpret_cast<uint16_t*>(vals + value_at(2, at, u * 8)) = (uint16_t)vc;
    *reinterpret_cast<uint16_t*>(vals + value_at(2, at, u * 8 + 4)) = (uint16_t)(vc >> 16);
  } else {
    *reinterpret_cast<uint32_t*>(vals + value_at(nb, at, u * 8)) = vc;
  }
  if ((u & 3) == 0) {
    uint8_t* s = to + 2 * plane_bytes(c);
    s[at * nb + u / 4] = (uint8_t)kb;
    s[scale_bytes(c) + (at / 4 * nb + u / 4) * 4 + at % 4] = (uint8_t)vb;
  }
}

// The values that append's rows stand for, [rows][heads][dim]; zeros where a row has no
// page.  Bound by memory (16384 rows of 8 heads of 128 dimensions 16.2 us, 5.2 TB/s).
template <int DT>
__global__ void __launch_bounds__(256) k_kv4_read(Cache c, Batch t, void* __restrict__ k, void* __restrict__ v) {
  const uint32_t octs = c.dim / 8, nb = c.dim / 32, u = threadIdx.x % octs;
  uint32_t head;
  const uint32_t row = row_of(c, octs, &head);
  if (row >= t.rows) return;
  uint32_t at = 0, kc = 0, vc = 0, kb = kScaleOne, vb = kScaleOne;
  const uint8_t* from = place(c, t, row, head, &at);
  if (from) {
    kc = *reinterpret_cast<const uint32_t*>(from + (uint64_t)at * (c.dim / 2) + u * 4);
    const uint8_t* vals = from + plane_bytes(c);
    if (nb == 2)
      vc = *reinterpret_cast<const uint16_t*>(vals + value_at(2, at, u * 8)) |
           (uint32_t) * reinterpret_cast<const uint16_t*>(vals + value_at(2, at, u * 8 + 4)) << 16;
    else
      vc = *reinterpret_cast<const uint32_t*>(vals + value_at(nb, at, u * 8));
    const uint8_t* s = from + 2 * plane_bytes(c);
    kb = s[at * nb + u / 4];
    vb = s[scale_bytes(c) + (at / 4 * nb + u / 4) * 4 + at % 4];
  }
  const uint64_t to = (((uint64_t)row * c.heads + head) * octs + u) * 8;
  store_oct<DT>(k, to, kc, scale_of(kb), 8);
  store_oct<DT>(v, to, vc, scale_of(vb), 8);
}

// ------------------------------------------------------------------ attention
// A wave takes 16 NQ query rows of one sequence and one key/value head (row r: token
// r / group, query head r % group) and tiles of 32 tokens.  Everything runs
// transposed, so that no value crosses lanes between the two products: of
// S^T = K q^T (16x16x32 instructions) lane l gets query l % 16 and tokens
// 4 (l / 16) .. + 3 of each half tile, which is the operand of O^T += V^T P^T if that
// instruction's order of tokens is taken the same way.  A third product, of ones, sums
// the weights as they were rounded.  Weights are 2^(scale s - c) with an offset c of the
// lane's own query column that only moves when a weight would pass 2^8 times the one it was
// set by, so that most tiles need neither a maximum across lanes nor a rescaling.
//
// With a bf16 query keys, values and weights are bf16; with an fp16 query fp16, which
// holds keys and values exactly between scales of 2^-23 and 2^13, all that fp16 keys and
// values can have.  Smaller ones round to multiples of 2^-24, larger ones count as NaN.
// Rounding the weights to q's type is what the matrix instruction takes; next to the
// output's own rounding to it, errors against 64 bits are 1.1 to 1.35 times those of weights
// in 32 bits.
//
// Four waves of a block take tiles of 32 tokens in turn, straight into registers, the next
// one asked for while one is multiplied.  For single tokens bound by memory (32 sequences
// up to 32768 tokens, 8 heads of 128 dimensions: 195 us, 4.4 TB/s of cache), for short ones
// by the latency of lengths, page table and pages in turn (1001 tokens 5.5 us, and 3.9 for
// the join), for many rows by vector instructions, which unpack 4-bit values and take
// exponentials (512 fp16 rows of 32 heads behind 16384 tokens 204 us, 660 TFLOP/s, bf16 220).
// Blocks whose waves share a tile's operands through LDS took 257 us there when these took
// 210: the copies, one tile ahead, were waited for.
struct AttendArgs {
  Cache c;
  Batch t;
  const uint16_t* q;
  void* o;
  float* part;            // per split and row: dim fp32 of O; then per split and row: offset and sum
  int64_t q_row, q_head;  // strides
  uint32_t group, q_heads, q_tiles, splits;
  uint32_t chunk;         // tiles of one split
  uint32_t rows_each;     // rows / batch
  uint32_t per_group;     // 2^32 / group, rounded up
  uint32_t per_page;      // 2^32 / tiles of a page, rounded up; 0 for one
  int32_t window, sinks;  // window 0: none
  float scale;            // times log2 e
};

// A row's softmax state: its offset and sum.  kNothing as the sum: no token was visible,
// so the output is zero; a sum of zero from tokens that were visible (all scores -inf)
// gives NaN, as the definition does.
constexpr float kNothing = -1.f;

template <int NB>
struct Tile {  // what a lane holds of 32 tokens
  uint32_t k[2][NB], v[2][NB];
  uint32_t ks[2], vs[2];  // scale bytes: of the lane's token and its NB octets; of its four tokens
};

template <int N>
__device__ __forceinline__ void load_words(uint32_t (&to)[N], const uint8_t* p) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const u32x4 v = *reinterpret_cast<const u32x4*>(p + i * 4);
      to[i] = v[0], to[i + 1] = v[1], to[i + 2] = v[2], to[i + 3] = v[3];
    }
  } else {
    const u32x2 v = *reinterpret_cast<const u32x2*>(p);
    to[0] = v[0], to[1] = v[1];
  }
}

template <int NB>
__device__ __forceinline__ void load_tile(Tile<NB>& t, const uint8_t* region, uint32_t page_tokens, uint32_t at,
                                          uint32_t r16, uint32_t g) {
  const uint8_t* v = region + page_tokens * (NB * 16);
  const uint8_t* ks = region + page_tokens * (NB * 32);
  const uint8_t* vs = ks + page_tokens * NB;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t token = at + 16 * h;
    load_words<NB>(t.k[h], region + (token + r16) * (NB * 16) + g * (NB * 4));
    load_words<NB>(t.v[h], v + ((token / 4 + g) * 16 + r16) * (NB * 4));
    // the lane's NB octets of dimensions, from g NB on, lie in the blocks from g NB / 4 on
    if constexpr (NB == 8)
      t.ks[h] = *reinterpret_cast<const uint16_t*>(ks + (token + r16) * NB + g * 2);
    else
      t.ks[h] = ks[(token + r16) * NB + g * NB / 4];
    t.vs[h] = *reinterpret_cast<const uint32_t*>(vs + ((token / 4 + g) * NB + r16 * NB / 16) * 4);
  }
}

// eight elements of 16-bit type, as the matrix instructions take them
template <bool F16>
__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
template <bool F16>
__device__ __forceinline__ u32x4 oct(uint32_t codes, float scale) {
  if constexpr (F16)
    return __builtin_bit_cast(u32x4, oct_f16(codes, scale));
  else
    return __builtin_bit_cast(u32x4, oct_bf16(codes, scale));
}
template <bool F16, int SEL>
__device__ __forceinline__ uint32_t pair(uint32_t codes, float scale) {
  if constexpr (F16)
    return pair_f16<SEL>(codes, scale);
  else
    return pair_bf16<SEL>(codes, scale);
}
template <bool F16>
__device__ __forceinline__ u32x4 round8(const float (&x)[8]) {
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (F16)
      r[i] = __builtin_bit_cast(uint32_t, f16x2{(_Float16)x[2 * i], (_Float16)x[2 * i + 1]});
    else
      r[i] = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)x[2 * i], (__bf16)x[2 * i + 1]});
  }
  return r;
}
template <bool F16>
__device__ __forceinline__ u32x4 ones() {
  const uint32_t w = F16 ? 0x3c003c00u : 0x3f803f80u;
  return u32x4{w, w, w, w};
}

// the operands of V^T for dimensions 2 B and 2 B + 1 of the lane's group: byte B of each
// of the eight tokens, turned from pairs of dimensions into pairs of tokens
template <bool F16, int NB, int B>
__device__ __forceinline__ void value_operands(const Tile<NB>& t, const float (&s)[8], u32x4* even, u32x4* odd) {
  uint32_t p[8];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if constexpr (NB == 2) {  // two tokens a word
      p[4 * h] = pair<F16, B>(t.v[h][0], s[4 * h]);
      p[4 * h + 1] = pair<F16, 2 + B>(t.v[h][0], s[4 * h + 1]);
      p[4 * h + 2] = pair<F16, B>(t.v[h][1], s[4 * h + 2]);
      p[4 * h + 3] = pair<F16, 2 + B>(t.v[h][1], s[4 * h + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) p[4 * h + i] = pair<F16, B % 4>(t.v[h][i * (NB / 4) + B / 4], s[4 * h + i]);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    (*even)[i] = __builtin_amdgcn_perm(p[2 * i + 1], p[2 * i], 0x05040100u);
    (*odd)[i] = __builtin_amdgcn_perm(p[2 * i + 1], p[2 * i], 0x07060302u);
  }
}

template <int I, int N, class F>
__device__ __forceinline__ void each(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    each<I + 1, N>(f);
  }
}

template <int NB, int NQ, bool F16>
struct Wave {
  // Exponent of the largest weight when an offset is set.  fp16 ends at 2^15, and what is lost
  // at its other end is then under 2^-31 of the largest weight.  bf16 values end at 2^128, as
  // the fp32 sums do: weights far under one keep sums of 2^24 tokens from passing the end, and
  // reach down to 2^-94 of the largest.
  static constexpr float kTop = F16 ? 7.f : -32.f, kSlack = 8.f;

  u32x4 q[NQ][NB];
  int32_t pos[NQ];  // of the lane's query row in each tile, -1: no row
  f32x4 o[NQ][2 * NB], l[NQ];
  float c[NQ], most[NQ];  // offset; largest exponent that it allows, -inf: none yet
  bool seen[NQ];

  __device__ __forceinline__ bool visible(const AttendArgs& a, int32_t t, int32_t p) const {
    return t <= p && (a.window == 0 || t > p - a.window || t < a.sinks);
  }

  // A token's value as zeros of scale 1; i: the token among the lane's four of half h.
  __device__ __forceinline__ void clear_value(Tile<NB>& t, int h, int i) const {
    if constexpr (NB == 2) {
      t.v[h][i / 2] &= i % 2 ? 0x0000ffffu : 0xffff0000u;
    } else {
#pragma unroll
      for (int w = 0; w < NB / 4; ++w) t.v[h][i * (NB / 4) + w] = 0;
    }
    t.vs[h] = (t.vs[h] & ~(255u << 8 * i)) | kScaleOne << 8 * i;
  }

  // Past fp16's range some of a block's keys would become infinities, and a token with a score
  // of -infinity would vanish without a sign: the whole block counts as NaN.
  static __device__ __forceinline__ float key_scale(uint32_t byte) {
    return scale_of(F16 && byte > kScaleOne + 13 ? kScaleNaN : byte);
  }

  __device__ __forceinline__ void scores(const Tile<NB>& t, f32x4 (&s)[2][NQ]) const {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int n = 0; n < NQ; ++n) s[h][n] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const u32x4 k = oct<F16>(t.k[h][j], key_scale(t.ks[h] >> 8 * (j / 4) & 255));
#pragma unroll
        for (int n = 0; n < NQ; ++n) s[h][n] = mfma16<F16>(k, q[n][j], s[h][n]);
      }
    }
  }

  // The weights of a tile's scores for query tile n, rounded to the product's type (half a
  // step of each), and which of the lane's eight tokens count.
  __device__ __forceinline__ u32x4 weights(const AttendArgs& a, const f32x4 (&s)[2][NQ], int n, int32_t t0, bool whole,
                                           uint32_t g, uint32_t& vis) {
    float p[8];
    vis = 0xff;
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = fmaf(s[i / 4][n][i % 4], a.scale, -c[n]);
    if (!whole) {
      vis = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (visible(a, t0 + 16 * (i / 4) + 4 * (int32_t)g + i % 4, pos[n]))
          vis |= 1u << i;
        else
          p[i] = -INFINITY;
      }
    }
    seen[n] |= vis != 0;
    float top = p[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) top = fmaxf(top, p[i]);
    if (__any(top > most[n])) {
      top = fmaxf(top, __shfl_xor(top, 16));
      top = fmaxf(top, __shfl_xor(top, 32));
      const bool fresh = most[n] == -INFINITY;
      const float up = fresh ? (top == -INFINITY ? 0.f : top - kTop) : fmaxf(top - kTop, 0.f);
      const float fade = fresh ? 1.f : __builtin_amdgcn_exp2f(-up);
      c[n] += up;
      if (top > -INFINITY) most[n] = kTop + kSlack;
      l[n] *= fade;
#pragma unroll
      for (int d = 0; d < 2 * NB; ++d) o[n][d] *= fade;
#pragma unroll
      for (int i = 0; i < 8; ++i) p[i] = vis >> i & 1 ? fmaf(s[i / 4][n][i % 4], a.scale, -c[n]) : -INFINITY;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = __builtin_amdgcn_exp2f(p[i]);
    return round8<F16>(p);
  }

  // Value blocks that are NaN, or past fp16's range: a weight of zero times such a value
  // must not reach rows that do not see the token, so these blocks count as zeros, and the
  // rows that see one become NaN in its dimensions.  A product of ones marks them.
  static constexpr float kMostScale = F16 ? 0x1p13f : 0x1p127f;
  __device__ __forceinline__ void mark_nan(Tile<NB>& t, float (&vs)[8], const uint32_t (&vis)[NQ]) {
    u32x4 is{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (vs[i] <= kMostScale) continue;
      is[i / 2] |= 0x3f80u << 16 * (i % 2);
      clear_value(t, i / 4, i % 4);
      vs[i] = 1.f;
    }
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      u32x4 see{0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (vis[n] >> i & 1) see[i / 2] |= 0x3f80u << 16 * (i % 2);
      const f32x4 hit = mfma16<false>(is, see, f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float bad = hit[r] > 0.f ? __builtin_nanf("") : 0.f;
#pragma unroll
        for (int d = 0; d < 2 * NB; ++d) o[n][d][r] += bad;
      }
    }
  }

  // One tile of tokens from t0 on; whole: every row sees every token.
  __device__ __forceinline__ void tile(const AttendArgs& a, Tile<NB>& t, int32_t t0, bool whole, int32_t stored,
                                       uint32_t r16, uint32_t g) {
    // tokens past the last one stored hold anything: as zeros they add nothing
    if (t0 + 32 > stored) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (t0 + 16 * h + (int32_t)r16 >= stored) t.ks[h] = kScaleOne * 0x101u;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (t0 + 16 * h + 4 * (int32_t)g + i >= stored) clear_value(t, h, i);
      }
    }
    f32x4 s[2][NQ];
    u32x4 w[NQ];
    uint32_t vis[NQ];
    scores(t, s);
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      w[n] = weights(a, s, n, t0, whole, g, vis[n]);
      l[n] = mfma16<F16>(ones<F16>(), w[n], l[n]);
    }
    float vs[8], most_scale = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      vs[i] = scale_of(t.vs[i / 4] >> 8 * (i % 4) & 255);
      most_scale = fmaxf(most_scale, vs[i]);
    }
    if (__any(most_scale > kMostScale)) mark_nan(t, vs, vis);
    each<0, NB>([&](auto b) {
      u32x4 even, odd;
      value_operands<F16, NB, b.value>(t, vs, &even, &odd);
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        o[n][2 * b.value] = mfma16<F16>(even, w[n], o[n][2 * b.value]);
        o[n][2 * b.value + 1] = mfma16<F16>(odd, w[n], o[n][2 * b.value + 1]);
      }
    });
  }
};

// Zeros for the rows before the first sequence's and behind the last one's.
template <int D>
__device__ void none(const AttendArgs& a) {
  if (blockIdx.y != 0) return;
  const uint32_t lo = (uint32_t)min(max(a.t.starts[0], 0), (int32_t)a.t.rows);
  const uint32_t hi = min((uint32_t)max(a.t.starts[a.t.batch], (int32_t)lo), a.t.rows);
  const uint64_t all = (uint64_t)a.t.rows * a.q_heads, before = (uint64_t)lo * a.q_heads;
  const uint64_t nobody = before + (uint64_t)(a.t.rows - hi) * a.q_heads;
  for (uint64_t e = threadIdx.x; e < nobody; e += 256) {
    const uint64_t at = e < before ? e : e - before + (uint64_t)hi * a.q_heads;
    if (a.splits > 1) {
      a.part[a.splits * all * D + (blockIdx.x * all + at) * 2 + 1] = kNothing;
    } else {
      for (int d = 0; d < D; ++d) static_cast<uint16_t*>(a.o)[at * D + d] = 0;
    }
  }
}

// How the parts of a row are joined: each part's factor is 2^(its offset - the largest),
// parts that saw nothing or only scores of -inf aside.
__device__ __forceinline__ bool has_weight(float sum) { return sum != kNothing && sum != 0.f; }

template <bool F16>
__device__ __forceinline__ void store_out(void* out, uint64_t at, f32x4 o, float l, bool seen) {
  f32x4 y;
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] = seen ? o[i] / l : 0.f;
  u32x2 w;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if constexpr (F16)
      w[i] = __builtin_bit_cast(uint32_t, f16x2{(_Float16)y[2 * i], (_Float16)y[2 * i + 1]});
    else
      w[i] = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)y[2 * i], (__bf16)y[2 * i + 1]});
  }
  *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(out) + at) = w;
}

// Blocks of four waves that a CU is given.  Its registers hold no more, but for heads of 64
// with two query tiles: three fit, and with three a prompt of 512 rows behind 16384 tokens
// takes 157 us and with two 158, 40 rows of 2 sequences over 30000 tokens 57 and 61, but 615
// rows of 16 sequences over 3211 tokens 40 and 32, for then two tiles are taken there.
constexpr int at_once(int dim, int nq) { return nq == 2 || dim == 256 ? 2 : dim == 128 ? 3 : 4; }

// A row's output: element 4 d + r of the lane (o[n][d][r]) is dimension 2 NB (4 g + r) + d.
template <int NB, int NQ, bool F16>
__global__ void __launch_bounds__(256, at_once(32 * NB, NQ)) k_kv4_attend(AttendArgs a) {
  constexpr int D = 32 * NB;
  const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t r16 = lane & 15, g = lane >> 4;
  const uint32_t b = blockIdx.z;
  uint32_t head = blockIdx.y, q_tile = 0;
  if (a.q_tiles > 1) q_tile = blockIdx.y / a.c.heads, head = blockIdx.y - q_tile * a.c.heads;
  if (b == a.t.batch) {  // rows of no sequence
    none<D>(a);
    return;
  }
  int32_t first, n_rows = (int32_t)a.rows_each;
  if (a.t.starts) {
    first = max(a.t.starts[b], 0);
    n_rows = max(min(a.t.starts[b + 1], (int32_t)a.t.rows), 0) - first;
  } else {
    first = (int32_t)b * n_rows;
  }
  const uint32_t all_rows = (uint32_t)max(n_rows, 0) * a.group;  // the host keeps this under 2^31
  const int32_t len = a.t.lens[b];
  const int32_t capacity = (int32_t)(a.t.wide * a.c.page_tokens);
  const int32_t stored = min(len, capacity);
  const int32_t* table = a.t.table + b * a.t.stride;
  __shared__ float sc[4][16 * NQ], sl[4][16 * NQ];
  __shared__ uint32_t rows_at[16 * NQ];  // of the output
  __shared__ __align__(16) float so[4][16][D + 4];

  for (uint32_t row0 = q_tile * (16 * NQ); row0 < all_rows; row0 += a.q_tiles * (16 * NQ)) {
    // positions of the tile's first and last rows
    const uint32_t last_row = min(row0 + 16 * NQ, all_rows) - 1;
    const int64_t p_lo = (int64_t)len - n_rows + (row0 ? row0 / a.group : 0);
    const int64_t p_hi = (int64_t)len - n_rows + (last_row + 1 == all_rows ? (uint32_t)n_rows - 1 : last_row / a.group);
    const int32_t hi = (int32_t)min(max(p_hi, (int64_t)-1), (int64_t)capacity - 1);
    // tiles: those of the sinks, then from the window's first on
    int32_t first_tile = 0, sink_tiles = 0, tiles = 0;
    if (hi >= 0) {
      if (a.window) first_tile = (int32_t)(max(p_lo - a.window + 1, (int64_t)0) / 32);
      sink_tiles = min(min((a.sinks + 31) / 32, first_tile), hi / 32 + 1);
      tiles = max(hi / 32 - first_tile + 1, 0) + sink_tiles;
    }
    // the block's tiles (the last split takes what is left), which its waves take in turn
    const int32_t cut = (int32_t)(blockIdx.x * a.chunk), step = 4;
    const int32_t to = blockIdx.x + 1 == a.splits ? tiles : min(cut + (int32_t)a.chunk, tiles);
    int32_t v = cut + (int32_t)wave;

    // The next tile's loads are in flight while a tile is worked on, and the page after it
    // is known by then.  A tile without a page, or none at all, loads page 0 and is passed
    // over: loads on a condition would have the wave wait for all of them each time.
    auto start_of = [&](int32_t i) { return (i < sink_tiles ? i : i - sink_tiles + first_tile) * 32; };
    auto page_index = [&](int32_t t0) { return a.per_page ? __umulhi((uint32_t)t0 / 32, a.per_page) : (uint32_t)t0 / 32; };
    auto page_of = [&](int32_t i) { return i < to ? table[page_index(start_of(i))] : -1; };
    auto fetch = [&](Tile<NB>& t, int32_t i, int32_t page) {
      const bool ok = (uint32_t)page < a.c.pages;
      const uint32_t t0 = (uint32_t)start_of(i), in = t0 - page_index(t0) * a.c.page_tokens;
      const uint64_t region = (ok ? (uint64_t)(uint32_t)page : 0) * a.c.heads + head;
      load_tile<NB>(t, a.c.data + region * region_bytes(a.c), a.c.page_tokens, ok ? in : 0, r16, g);
      return ok;
    };
    Tile<NB> t, next;
    const int32_t page0 = page_of(v);
    int32_t page1 = page_of(v + step);
    bool ok = fetch(t, v, page0);

    Wave<NB, NQ, F16> w;
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      const uint32_t r = min(row0 + n * 16 + r16, all_rows - 1);
      const uint32_t i = a.group == 1 ? r : all_rows <= 1u << 16 ? __umulhi(r, a.per_group) : r / a.group;
      const uint32_t hq = head * a.group + (r - i * a.group);
      const bool real = row0 + n * 16 + r16 < all_rows;
      w.pos[n] = real ? (int32_t)max((int64_t)len - n_rows + i, (int64_t)-1) : -1;
      const uint16_t* q = a.q + (first + (int64_t)i) * a.q_row + hq * a.q_head + g * (8 * NB);
#pragma unroll
      for (int j = 0; j < NB; ++j) w.q[n][j] = reinterpret_cast<const Loose16*>(q + j * 8)->v;
      if (wave == 0 && g == 0) rows_at[n * 16 + r16] = real ? (first + i) * a.q_heads + hq : ~0u;
      w.c[n] = 0.f;
      w.most[n] = -INFINITY;
      w.seen[n] = false;
      w.l[n] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int d = 0; d < 2 * NB; ++d) w.o[n][d] = f32x4{0.f, 0.f, 0.f, 0.f};
    }

    for (; v < to; v += step) {
      const int32_t page2 = page_of(v + 2 * step);
      const bool ok1 = fetch(next, v + step, page1);
      const int32_t t0 = start_of(v);
      const bool whole = t0 + 31 <= p_lo && row0 + 16 * NQ <= all_rows &&
                         (a.window == 0 || t0 > p_hi - a.window || t0 + 32 <= a.sinks);
      if (ok) w.tile(a, t, t0, whole, stored, r16, g);
      t = next;
      ok = ok1;
      page1 = page2;
    }

    // the four waves' states joined through LDS
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      uint32_t seen = w.seen[n];
      seen |= (uint32_t)__shfl_xor((int)seen, 16);
      seen |= (uint32_t)__shfl_xor((int)seen, 32);
      if (g == 0) {
        sc[wave][n * 16 + r16] = w.c[n];
        sl[wave][n * 16 + r16] = seen ? w.l[n][0] : kNothing;
      }
    }
    const uint64_t all = (uint64_t)a.t.rows * a.q_heads;
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      const uint32_t left = all_rows - row0;  // rows from the tile's first on
      if (n * 16u >= left) break;
      const uint32_t here = min(16u, left - n * 16);
      if (n) __syncthreads();
      if (r16 < here) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int d = 0; d < 2 * NB; d += 4)
            *reinterpret_cast<f32x4*>(&so[wave][r16][2 * NB * (4 * g + r) + d]) =
                f32x4{w.o[n][d][r], w.o[n][d + 1][r], w.o[n][d + 2][r], w.o[n][d + 3][r]};
      }
      __syncthreads();
      for (uint32_t e = threadIdx.x; e < here * (D / 4); e += 256) {
        const uint32_t row = e / (D / 4), d = e % (D / 4) * 4, in = n * 16 + row;
        const uint64_t at = rows_at[in];
        float c = -INFINITY, l = 0.f;
        f32x4 o = {0.f, 0.f, 0.f, 0.f};
        bool seen = false;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          seen |= sl[v][in] != kNothing;
          c = fmaxf(c, has_weight(sl[v][in]) ? sc[v][in] : -INFINITY);
        }
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const bool some = has_weight(sl[v][in]);
          const float f = some ? __builtin_amdgcn_exp2f(sc[v][in] - c) : 0.f;
          l += some ? f * sl[v][in] : 0.f;
          o += f * *reinterpret_cast<const f32x4*>(&so[v][row][d]);  // zero where there is no weight
        }
        if (a.splits == 1) {
          store_out<F16>(a.o, at * D + d, o, l, seen);
        } else {
          *reinterpret_cast<f32x4*>(a.part + (blockIdx.x * all + at) * D + d) = o;
          if (d == 0)
            *reinterpret_cast<f32x2*>(a.part + a.splits * all * D + (blockIdx.x * all + at) * 2) =
                f32x2{c, seen ? l : kNothing};
        }
      }
    }
    __syncthreads();
  }
}

// The splits of a row joined: `per` waves for a row, each the splits of its turn, and
// their sums in the order of the waves.  Lane s of every wave first holds the factors of
// splits s, s + 64, ..., EACH of them, then D / 64 dimensions.  One sequence of 131072
// tokens and 8 heads: 42 us, with at most 64 splits and a wave per row 62.  A split in which
// the row saw nothing may be unwritten and is passed over; one whose weight is zero counts,
// for it may hold a NaN.
constexpr uint32_t kMostSplits = 256, kJoinWaves = 16;
template <int D, bool F16, int EACH>
__global__ void __launch_bounds__(64 * kJoinWaves) k_kv4_join(const float* __restrict__ part, void* __restrict__ out,
                                                              uint64_t all, uint32_t splits, uint32_t per) {
  constexpr int N = D / 64;
  __shared__ float sums[kJoinWaves][D];
  const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6, first = wave % per;
  const uint64_t mine = (uint64_t)blockIdx.x * ((blockDim.x >> 6) / per) + wave / per;
  const uint64_t at = mine < all ? mine : all - 1;
  const float* cl = part + splits * all * D + at * 2;
  f32x2 state[EACH];
  float c = -INFINITY, l = 0.f, f[EACH];
  bool seen = false;
#pragma unroll
  for (int k = 0; k < EACH; ++k) {
    const uint32_t s = lane + 64 * k;
    state[k] = s < splits ? *reinterpret_cast<const f32x2*>(cl + s * all * 2) : f32x2{0.f, kNothing};
    if (has_weight(state[k][1])) c = fmaxf(c, state[k][0]);
  }
#pragma unroll
  for (int i = 1; i < 64; i *= 2) c = fmaxf(c, __shfl_xor(c, i));
#pragma unroll
  for (int k = 0; k < EACH; ++k) {
    const bool some = has_weight(state[k][1]);
    f[k] = some ? __builtin_amdgcn_exp2f(state[k][0] - c) : state[k][1] == kNothing ? kNothing : 0.f;
    l += some ? f[k] * state[k][1] : 0.f;
    seen = seen || __any(state[k][1] != kNothing);
  }
#pragma unroll
  for (int i = 1; i < 64; i *= 2) l += __shfl_xor(l, i);
  float o[N] = {};
#pragma unroll
  for (int k = 0; k < EACH; ++k) {
    for (uint32_t s = 64 * k + first; s < min(splits, 64u * k + 64); s += per) {
      const float fs = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(f[k]), s % 64));
      const float* p = part + (s * all + at) * D + lane * N;
      float x[N];
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = p[i];
#pragma unroll
      for (int i = 0; i < N; ++i) o[i] = fs != kNothing ? fmaf(fs, x[i], o[i]) : o[i];
    }
  }
  if (per > 1) {
#pragma unroll
    for (int i = 0; i < N; ++i) sums[wave][lane * N + i] = o[i];
    __syncthreads();
    if (first != 0) return;
    for (uint32_t k = 1; k < per; ++k)
#pragma unroll
      for (int i = 0; i < N; ++i) o[i] += sums[wave + k][lane * N + i];
  }
  if (mine >= all) return;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float y = seen ? o[i] / l : 0.f;
    if constexpr (F16)
      static_cast<_Float16*>(out)[at * D + lane * N + i] = (_Float16)y;
    else
      static_cast<__bf16*>(out)[at * D + lane * N + i] = (__bf16)y;
  }
}

}  // namespace ecw

using namespace ecw;

namespace {

ecw_status check_cache(const ecw_kv4* c) {
  if (!c) return refuse(ECW_E_INVALID_ARG, "cache is NULL");
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
    return refuse(ECW_E_UNSUPPORTED, "head_dim must be 64, 128 or 256");
  if (c->page_tokens == 0 || c->page_tokens % 32 || c->page_tokens > 4096)
    return refuse(ECW_E_INVALID_ARG, "page_tokens must be a multiple of 32 up to 4096");
  if (c->pages == 0 || c->pages >= 1u << 31 || c->kv_heads == 0 || c->kv_heads > 1024)
    return refuse(ECW_E_INVALID_ARG, "pages must be in [1, 2^31), kv_heads in [1, 1024]");
  return ECW_OK;
}

ecw_status check_rows(const ecw_kv4* c, const ecw_kv4_rows* r) {
  if (ecw_status s = check_cache(c)) return s;
  if (!c->data || !aligned(c->data, 256)) return refuse(ECW_E_INVALID_ARG, "cache data must be 256-byte aligned");
  if (!r) return refuse(ECW_E_INVALID_ARG, "rows are NULL");
  if (r->rows == 0) return ECW_OK;
  if (r->batch == 0 || r->batch > 65534 || r->rows >= 1u << 30)
    return refuse(ECW_E_INVALID_ARG, "batch must be in [1, 65534], rows below 2^30");
  if (!r->starts && r->rows % r->batch)
    return refuse(ECW_E_INVALID_ARG, "without starts every sequence has the same number of rows");
  if (!r->lens || (r->table_width && !r->page_table)) return refuse(ECW_E_INVALID_ARG, "lens or page table is NULL");
  if (!aligned(r->lens, 4) || !aligned(r->page_table, 4) || !aligned(r->starts, 4))
    return refuse(ECW_E_INVALID_ARG, "lens, page table and starts must be 4-byte aligned");
  if (r->table_stride < 0) return refuse(ECW_E_INVALID_ARG, "table stride must not be negative");
  if ((uint64_t)r->table_width * c->page_tokens >= 1u << 30)
    return refuse(ECW_E_INVALID_ARG, "the page table spans 2^30 tokens or more");
  return ECW_OK;
}

Cache cache_of(const ecw_kv4* c) {
  return {static_cast<uint8_t*>(c->data), c->pages, c->kv_heads, c->head_dim, c->page_tokens};
}
Batch batch_of(const ecw_kv4_rows* r) {
  return {r->page_table, r->lens, r->starts, r->table_stride, r->batch, r->table_width, r->rows};
}

bool row_grid(const ecw_kv4* c, const ecw_kv4_rows* r, uint32_t* grid) {
  const uint32_t rows = 256 / (c->head_dim / 8);
  const uint64_t n = ((uint64_t)r->rows + rows - 1) / rows * c->kv_heads;
  *grid = (uint32_t)n;
  return launchable(n, 256);
}

constexpr float kLog2E = 1.44269504088896f;
// tiles of 32 tokens of a split, for its four waves: no fewer, but where CUs are idle (plan_with)
constexpr uint64_t kChunk = 12;

// How an attention call is cut up: query tiles of 16 nq rows, and splits of each
// sequence's tokens.
struct Plan {
  uint32_t nq, q_tiles, splits, chunk;
  double time;  // estimate, in a tile of keys by one tile of rows with every wave of a CU at work
};

// The plan with nq tiles of 16 rows a wave, for sequences of `rows` rows and `tiles` tiles.
Plan plan_with(uint32_t nq, uint64_t rows, uint64_t tiles, const ecw_kv4* c, uint32_t batch, bool joinable) {
  Plan p;
  p.nq = nq;
  const uint64_t tiles_q = (rows + 16 * nq - 1) / (16 * nq), most = 65535 / c->kv_heads;
  p.q_tiles = (uint32_t)(tiles_q < most ? tiles_q : most);
  const uint64_t blocks = (uint64_t)p.q_tiles * c->kv_heads * batch, room = 256 * at_once((int)c->head_dim, (int)nq);
  // as many blocks as the card holds at once, and no second round of them: 32 sequences of
  // up to 32768 tokens take 209 us at 3 splits of each, 233 at 4
  uint64_t splits = room / blocks;
  uint64_t top = (tiles + kChunk - 1) / kChunk;
  // a tile a wave where CUs are idle and a join is needed anyway (1001 tokens of 8 heads
  // 10.6 -> 9.0 us; 300 tokens, one split, 7.5 us and 8.7 in three; a window of 4096 of 64
  // heads of sequences in splits of 12 tiles 14.8 us, of 8 15.4)
  if (top > 1) top = std::max(top, std::min<uint64_t>({(tiles + 3) / 4, 16, 512 / blocks}));
  if (splits > top) splits = top;
  if (splits > kMostSplits) splits = kMostSplits;
  if (!joinable) splits = 1;
  if (splits < 1) splits = 1;
  p.chunk = (uint32_t)((tiles + splits - 1) / splits);
  p.splits = (uint32_t)((tiles + p.chunk - 1) / p.chunk);
  // a wave's tiles of keys, one after the other: each takes its latency, or its turn among
  // those of the CU's other blocks
  const double per_cu = (double)((blocks * p.splits + 255) / 256);
  p.time = ((p.chunk + 3) / 4) * (nq == 2 ? std::max(3.2, 1.6 * per_cu) : std::max(2.5, per_cu));
  return p;
}

// One or two tiles of rows a wave: two take 1.6 times as long for a tile of keys, and half
// the blocks (512 rows of 32 heads behind 16384 tokens 220 us, one 278; 20 rows of 256 heads
// of sequences over 16000 tokens 155 and 185), but fewer blocks may leave CUs idle (615
// rows of dimension 64 over 3211 tokens, 16 sequences: 40 and 32 us; 48 rows over 8000
// tokens, 64 heads of sequences: 46 and 39; 20 rows over 2935 tokens, 6 of them: 13.4 and
// 10.8).  Four take all registers (512 rows behind 16384 tokens 275 us), and so do two of
// dimension 256 (300 rows of 6 heads behind 16000 tokens 92 us, one 81).
Plan plan_of(const ecw_kv4* c, const ecw_kv4_rows* r, const ecw_kv4_attention* at) {
  const uint64_t group = at->q_heads / c->kv_heads;
  const uint64_t each = at->max_rows ? (at->max_rows < r->rows ? at->max_rows : r->rows) : (r->rows + r->batch - 1) / r->batch;
  uint64_t len = (uint64_t)r->table_width * c->page_tokens;
  if (at->max_len && at->max_len < len) len = at->max_len;
  if (at->window) {
    const uint64_t seen = (uint64_t)at->window + at->sinks + each;
    if (seen < len) len = seen;
  }
  const uint64_t rows = each * group, tiles = (len + 31) / 32 + 1;
  const bool joinable = launchable((uint64_t)r->rows * at->q_heads + kJoinWaves, 64);  // a wave for each, at least
  const Plan one = plan_with(1, rows, tiles, c, r->batch, joinable);
  if (rows <= 16 || c->head_dim == 256) return one;
  const Plan two = plan_with(2, rows, tiles, c, r->batch, joinable);
  return one.time < two.time ? one : two;
}

ecw_status check_attention(const ecw_kv4* c, const ecw_kv4_rows* r, const ecw_kv4_attention* at) {
  if (ecw_status s = check_rows(c, r)) return s;
  if (!at) return refuse(ECW_E_INVALID_ARG, "attention is NULL");
  if (at->q_heads == 0 || at->q_heads % c->kv_heads || at->q_heads > 65536)
    return refuse(ECW_E_INVALID_ARG, "q_heads must be a positive multiple of kv_heads, at most 65536");
  if ((uint64_t)r->rows * at->q_heads >> 31)
    return refuse(ECW_E_UNSUPPORTED, "rows times q_heads must be below 2^31");
  if (at->window > 1u << 30 || at->sinks > 1u << 30)
    return refuse(ECW_E_INVALID_ARG, "window and sinks must be at most 2^30");
  const float scale = at->scale * kLog2E;
  if (!(scale - scale == 0.f)) return refuse(ECW_E_INVALID_ARG, "scale must be finite, times log2(e) too");
  return ECW_OK;
}

uint64_t part_bytes(const ecw_kv4* c, const ecw_kv4_rows* r, const ecw_kv4_attention* at, const Plan& p) {
  return p.splits == 1 ? 0 : (uint64_t)p.splits * r->rows * at->q_heads * (c->head_dim + 2) * 4;
}

template <int NB, int NQ, bool F16>
void launch_attend(hipStream_t stream, const AttendArgs& a) {
  const uint32_t z = a.t.batch + (a.t.starts ? 1 : 0);
  hipLaunchKernelGGL((k_kv4_attend<NB, NQ, F16>), dim3(a.splits, a.q_tiles * a.c.heads, z), dim3(256), 0, stream, a);
}

template <int NB, bool F16>
ecw_status launch_all(hipStream_t stream, const AttendArgs& a, const Plan& p) {
  if constexpr (NB == 8)
    launch_attend<NB, 1, F16>(stream, a);
  else if (p.nq == 1)
    launch_attend<NB, 1, F16>(stream, a);
  else
    launch_attend<NB, 2, F16>(stream, a);
  if (ecw_status s = launched("kv4_attend")) return s;
  if (a.splits == 1) return ECW_OK;
  const uint64_t all = (uint64_t)a.t.rows * a.q_heads;
  uint32_t per = 1;  // up to 4 splits a wave, while there are few rows (8: a window of 4096 15.7 us, 4: 14.8)
  while (per < kJoinWaves && a.splits > 4 * per && all * per < 4096) per *= 2;
  const uint32_t waves = per < 4 ? 4 : per;
  const uint64_t grid = (all * per + waves - 1) / waves;
  auto* fn = a.splits <= 64 ? k_kv4_join<32 * NB, F16, 1> : k_kv4_join<32 * NB, F16, kMostSplits / 64>;
  hipLaunchKernelGGL(fn, dim3((uint32_t)grid), dim3(64 * waves), 0, stream, a.part, a.o, all, a.splits, per);
  return launched("kv4_attend");
}

template <bool F16>
ecw_status launch_dim(hipStream_t stream, const AttendArgs& a, const Plan& p) {
  switch (a.c.dim) {
    case 64: return launch_all<2, F16>(stream, a, p);
    case 128: return launch_all<4, F16>(stream, a, p);
    default: return launch_all<8, F16>(stream, a, p);
  }
}

}  // namespace

extern "C" {

ecw_status kv4_bytes(const ecw_kv4* cache, size_t* bytes) {
  if (ecw_status s = check_cache(cache)) return s;
  if (!bytes) return refuse(ECW_E_INVALID_ARG, "bytes is NULL");
  *bytes = (size_t)cache->pages * cache->kv_heads * region_bytes(cache_of(cache));
  return ECW_OK;
}

ecw_status kv4_append(ecw_stream stream, const ecw_kv4* cache, const ecw_kv4_rows* rows, const void* k, const void* v,
                      int dtype, const int64_t* strides) {
  if (ecw_status s = check_rows(cache, rows)) return s;
  if (dtype != ECW_DT_F16 && dtype != ECW_DT_BF16 && dtype != ECW_DT_F32)
    return refuse(ECW_E_INVALID_ARG, "k and v must be F16, BF16 or F32");
  if (rows->rows == 0) return ECW_OK;
  const int64_t size = dtype == ECW_DT_F32 ? 4 : 2;
  if (!k || !v || !strides || !aligned(k, size) || !aligned(v, size))
    return refuse(ECW_E_INVALID_ARG, "k and v must be aligned device pointers with strides");
  for (int i = 0; i < 4; ++i)
    if (strides[i] < 0) return refuse(ECW_E_INVALID_ARG, "strides must not be negative");
  uint32_t grid;
  if (!row_grid(cache, rows, &grid)) return refuse(ECW_E_UNSUPPORTED, "too many rows for one launch");
  auto* fn = dtype == ECW_DT_F32   ? k_kv4_append<ECW_DT_F32>
             : dtype == ECW_DT_F16 ? k_kv4_append<ECW_DT_F16>
                                   : k_kv4_append<ECW_DT_BF16>;
  hipLaunchKernelGGL(fn, dim3(grid), dim3(256), 0, (hipStream_t)stream, cache_of(cache), batch_of(rows), k, v,
                     strides[0], strides[1], strides[2], strides[3]);
  return launched("kv4_append");
}

ecw_status kv4_read(ecw_stream stream, const ecw_kv4* cache, const ecw_kv4_rows* rows, void* k, void* v, int dtype) {
  if (ecw_status s = check_rows(cache, rows)) return s;
  if (dtype != ECW_DT_F16 && dtype != ECW_DT_BF16 && dtype != ECW_DT_F32)
    return refuse(ECW_E_INVALID_ARG, "k and v must be F16, BF16 or F32");
  if (rows->rows == 0) return ECW_OK;
  if (!k || !v || !aligned(k, 16) || !aligned(v, 16))
    return refuse(ECW_E_INVALID_ARG, "k and v must be 16-byte aligned device pointers");
  uint32_t grid;
  if (!row_grid(cache, rows, &grid)) return refuse(ECW_E_UNSUPPORTED, "too many rows for one launch");
  auto* fn = dtype == ECW_DT_F32   ? k_kv4_read<ECW_DT_F32>
             : dtype == ECW_DT_F16 ? k_kv4_read<ECW_DT_F16>
                                   : k_kv4_read<ECW_DT_BF16>;
  hipLaunchKernelGGL(fn, dim3(grid), dim3(256), 0, (hipStream_t)stream, cache_of(cache), batch_of(rows), k, v);
  return launched("kv4_read");
}

ecw_status kv4_attend_workspace_size(const ecw_kv4* cache, const ecw_kv4_rows* rows, const ecw_kv4_attention* at,
                                     size_t* bytes) {
  if (ecw_status s = check_attention(cache, rows, at)) return s;
  if (!bytes) return refuse(ECW_E_INVALID_ARG, "bytes is NULL");
  *bytes = rows->rows ? (size_t)part_bytes(cache, rows, at, plan_of(cache, rows, at)) : 0;
  return ECW_OK;
}

ecw_status kv4_attend(ecw_stream stream, const ecw_kv4* cache, const ecw_kv4_rows* rows, const ecw_kv4_attention* at,
                      const void* q, int dtype, int64_t q_row, int64_t q_head, void* o, void* workspace,
                      size_t workspace_bytes) {
  if (ecw_status s = check_attention(cache, rows, at)) return s;
  if (dtype != ECW_DT_F16 && dtype != ECW_DT_BF16) return refuse(ECW_E_INVALID_ARG, "q must be F16 or BF16");
  if (rows->rows == 0) return ECW_OK;
  if (!q || !aligned(q, 2) || q_row < 0 || q_head < 0)
    return refuse(ECW_E_INVALID_ARG, "q must be an aligned device pointer with strides of 0 or more");
  if (!o || !aligned(o, 16)) return refuse(ECW_E_INVALID_ARG, "o must be a 16-byte aligned device pointer");
  const Plan p = plan_of(cache, rows, at);
  if (part_bytes(cache, rows, at, p) > workspace_bytes || (p.splits > 1 && (!workspace || !aligned(workspace, 16))))
    return refuse(ECW_E_INVALID_ARG, "workspace missing, too small or not 16-byte aligned");
  AttendArgs a{};
  a.c = cache_of(cache);
  a.t = batch_of(rows);
  a.q = static_cast<const uint16_t*>(q);
  a.o = o;
  a.part = static_cast<float*>(workspace);
  a.q_row = q_row;
  a.q_head = q_head;
  a.group = at->q_heads / cache->kv_heads;
  a.q_heads = at->q_heads;
  a.q_tiles = p.q_tiles;
  a.splits = p.splits;
  a.chunk = p.chunk;
  a.rows_each = rows->rows / rows->batch;
  a.per_group = (uint32_t)(((uint64_t(1) << 32) + a.group - 1) / a.group);  // unused for one
  const uint32_t page_tiles = cache->page_tokens / 32;
  a.per_page = page_tiles == 1 ? 0 : (uint32_t)(((uint64_t(1) << 32) + page_tiles - 1) / page_tiles);
  a.window = (int32_t)at->window;
  a.sinks = (int32_t)at->sinks;
  a.scale = at->scale * kLog2E;
  return dtype == ECW_DT_F16 ? launch_dim<true>((hipStream_t)stream, a, p)
                             : launch_dim<false>((hipStream_t)stream, a, p);
}

}  // extern "C"
