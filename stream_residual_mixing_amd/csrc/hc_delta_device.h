// What the gated delta rule's kernels (hc_delta.hip, hc_delta_backward.hip) share: the layout of a
// chunk's record, operands in two bfloat16 parts, and the order of rows that lets one matrix
// product's result be the next one's operand without leaving its registers.
//
// v_mfma_f32_16x16x32_bf16: lane l = 16 g + n holds of A row n and of B column n the eight k
// values 8 g .. 8 g + 7, and of the result column n the four rows 4 g .. 4 g + 3. A product
// whose rows are to be the next one's k takes them in the order
//   row(t, m) = 32 (t / 2) + 8 (m / 4) + 4 (t % 2) + m % 4   (tile t of 16 rows, row m in it),
// so that a lane's four values of tile 2 b and four of tile 2 b + 1 are k = 32 b + 8 g + 0 .. 7.
#pragma once

#include "hc_sublayer.h"
#include "hc_sublayer_device.h"

namespace hc {

namespace {

constexpr int CH = 64;  // tokens of a chunk

typedef __bf16 bf8_t __attribute__((ext_vector_type(8)));
typedef float f4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u2_t __attribute__((ext_vector_type(2)));

__device__ __forceinline__ int row_of(int t, int m) { return 32 * (t >> 1) + 8 * (m >> 2) + 4 * (t & 1) + (m & 3); }

// the place of row x in that order
__device__ __forceinline__ int place_of(int x) { return (x & ~31) + 16 * ((x >> 2) & 1) + 4 * ((x >> 3) & 3) + (x & 3); }

// Eight float32 values as the sum of two bfloat16 parts, 16 bits of each value: the part left
// over is at most 2^-17 of it. Products of two such operands keep hi hi + hi lo + lo hi.
struct Split {
  bf8_t hi, lo;
};

__device__ __forceinline__ bf8_t as_bf8(u4_t q) { return __builtin_bit_cast(bf8_t, q); }

__device__ __forceinline__ u4_t pack8(const float v[8]) {
  u4_t q;
#pragma unroll
  for (int i = 0; i < 4; ++i) q[i] = pack_bf2_hw(v[2 * i], v[2 * i + 1]);
  return q;
}

__device__ __forceinline__ void split8(const float v[8], u4_t& hi, u4_t& lo) {
  hi = pack8(v);
  float rest[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    rest[2 * i] = v[2 * i] - __uint_as_float(hi[i] << 16);
    rest[2 * i + 1] = v[2 * i + 1] - __uint_as_float(hi[i] & 0xffff0000u);
  }
  lo = pack8(rest);
}

__device__ __forceinline__ Split split(const float v[8]) {
  u4_t h, l;
  split8(v, h, l);
  return {as_bf8(h), as_bf8(l)};
}

__device__ __forceinline__ Split split(f4_t a, f4_t b) {
  const float v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
  return split(v);
}

__device__ __forceinline__ f4_t mma(bf8_t a, bf8_t b, f4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ f4_t mma(const Split& a, const Split& b, f4_t c) {
  c = mma(a.lo, b.hi, c);
  c = mma(a.hi, b.lo, c);
  return mma(a.hi, b.hi, c);
}

// Stream operands: bfloat16 is exact in one part, float32 takes two.
template <typename T> struct Stream;
template <> struct Stream<bf16_t> {
  static constexpr int NP = 1;
};
template <> struct Stream<float> {
  static constexpr int NP = 2;
};

template <int NP>
struct Op {
  bf8_t p[NP];
};

template <int NP>
__device__ __forceinline__ f4_t mma(const Op<NP>& a, const Split& b, f4_t c) {
  if (NP == 2) c = mma(a.p[NP - 1], b.hi, c);
  c = mma(a.p[0], b.lo, c);
  return mma(a.p[0], b.hi, c);
}

template <int NP>
__device__ __forceinline__ f4_t mma(const Split& a, const Op<NP>& b, f4_t c) {
  if (NP == 2) c = mma(a.hi, b.p[NP - 1], c);
  c = mma(a.lo, b.p[0], c);
  return mma(a.hi, b.p[0], c);
}

template <int NP>
__device__ __forceinline__ f4_t mma(const Op<NP>& a, const Op<NP>& b, f4_t c) {
  if (NP == 2) {
    c = mma(a.p[NP - 1], b.p[0], c);
    c = mma(a.p[0], b.p[NP - 1], c);
  }
  return mma(a.p[0], b.p[0], c);
}

// Eight consecutive stream elements as stored; `cnt` of them exist (VEC: 8 or none).
template <typename T> struct Raw8;
template <> struct Raw8<bf16_t> {
  u4_t q;
  __device__ __forceinline__ Op<1> op() const { return {as_bf8(q)}; }
  __device__ __forceinline__ void open(float v[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(q[i] << 16);
      v[2 * i + 1] = __uint_as_float(q[i] & 0xffff0000u);
    }
  }
};
template <> struct Raw8<float> {
  f4_t a, b;
  __device__ __forceinline__ Op<2> op() const {
    const Split s = split(a, b);
    return {s.hi, s.lo};
  }
  __device__ __forceinline__ void open(float v[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = a[i], v[4 + i] = b[i];
  }
};

template <bool VEC>
__device__ __forceinline__ Raw8<bf16_t> load_raw8(const bf16_t* p, int cnt) {
  Raw8<bf16_t> r;
  r.q = u4_t{0, 0, 0, 0};
  if (VEC) {
    if (cnt > 0) r.q = *reinterpret_cast<const u4_t*>(p);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t x = e < cnt ? p[e] : 0;
      r.q[e >> 1] |= x << (16 * (e & 1));
    }
  }
  return r;
}

template <bool VEC>
__device__ __forceinline__ Raw8<float> load_raw8(const float* p, int cnt) {
  Raw8<float> r;
  r.a = r.b = f4_t{0.f, 0.f, 0.f, 0.f};
  if (VEC) {
    if (cnt > 0) {
      r.a = *reinterpret_cast<const f4_t*>(p);
      r.b = *reinterpret_cast<const f4_t*>(p + 4);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float x = e < cnt ? p[e] : 0.f;
      if (e < 4) r.a[e] = x;
      else r.b[e - 4] = x;
    }
  }
  return r;
}

// Tokens of sequence b.
__device__ __forceinline__ int64_t length_of(const int32_t* lengths, int64_t b, int64_t S) {
  if (lengths == nullptr) return S;
  const int64_t n = lengths[b];
  return n < 0 ? 0 : n > S ? S : n;
}

// A chunk's record: decays and betas, a float per token, and 16 x 32 operand tiles of 64 x 16 bytes in
// the lanes' order, first the six high parts and then the six low ones, of the two lower
// block-triangular matrices T (rows in row_of's order) and P (rows in their own), tile (t, kb) at
// tri(t, kb). The backward's holds T and, upper triangular at tri_t, the transposes of both with
// rows in row_of's order.
constexpr int TILE = 1024, TRI = 12 * TILE;
constexpr int REC_T = 0, REC_DEC = TRI, REC_P = TRI + 3 * CH * 4, REC = REC_P + TRI;
constexpr int REC_TT = REC, REC_BWD = REC + TRI;
constexpr int DEC_AHEAD = 0, DEC_TO_END = CH, DEC_BETA = 2 * CH;

__device__ __forceinline__ constexpr int tri(int t, int kb) { return t < 2 ? t : 2 * t - 2 + kb; }
__device__ __forceinline__ constexpr int tri_t(int t, int kb) { return t < 2 ? 2 * t + kb : t + 2; }

__device__ __forceinline__ Split load_tile(const char* m, int idx, int lane) {
  return {*reinterpret_cast<const bf8_t*>(m + idx * TILE + lane * 16),
          *reinterpret_cast<const bf8_t*>(m + (6 + idx) * TILE + lane * 16)};
}

__device__ __forceinline__ void store_tile(char* m, int idx, int lane, const float v[8]) {
  u4_t hi, lo;
  split8(v, hi, lo);
  *reinterpret_cast<u4_t*>(m + idx * TILE + lane * 16) = hi;
  *reinterpret_cast<u4_t*>(m + (6 + idx) * TILE + lane * 16) = lo;
}

// A chunk's keys or queries in LDS: rows of tokens [CH][KP], or transposed [KP][CH] with rows in
// row_of's order. Token rows hold an odd number of 16-byte pieces, so that 16 lanes reading a piece
// of 16 rows reach all 64 banks once. So do transposed rows, but of 256, where LDS has no room left
// for it (float32 streams): their pieces are exchanged within the row instead.
template <int KP>
struct Tokens {
  static constexpr int ROW = 2 * KP + 16;                      // bytes of a token's row
  static constexpr int COL = 2 * CH + (KP == 256 ? 0 : 16);    // bytes of a transposed row
  static constexpr int ROWS = CH * ROW;                        // bytes in all
  static constexpr int PART = KP * COL > ROWS ? KP * COL : ROWS;
  static __device__ __forceinline__ int row_at(int place, int byte) { return place * ROW + byte; }
  static __device__ __forceinline__ int col_at(int place, int byte) {
    return place * COL + (KP == 256 ? byte ^ ((place & 7) << 4) : byte);
  }
};

// Columns of a wave: NT tiles of 16, tile h's column n is NT n + h, so that a lane's are neighbours.
template <int NT> struct Cols { float v[NT]; };

template <int NT, bool VEC>
__device__ __forceinline__ Cols<NT> load_cols(const float* p, int cnt) {
  Cols<NT> r;
  if (VEC && NT == 2) {
    r.v[0] = r.v[NT - 1] = 0.f;
    if (cnt > 0) {
      const float2 q = *reinterpret_cast<const float2*>(p);
      r.v[0] = q.x;
      r.v[NT - 1] = q.y;
    }
  } else {
#pragma unroll
    for (int h = 0; h < NT; ++h) r.v[h] = h < cnt ? p[h] : 0.f;
  }
  return r;
}

template <int NT, bool VEC>
__device__ __forceinline__ Cols<NT> load_cols(const bf16_t* p, int cnt) {
  Cols<NT> r;
  if (VEC && NT == 2) {
    const uint32_t q = cnt > 0 ? *reinterpret_cast<const uint32_t*>(p) : 0;
    r.v[0] = __uint_as_float(q << 16);
    r.v[NT - 1] = __uint_as_float(q & 0xffff0000u);
  } else {
#pragma unroll
    for (int h = 0; h < NT; ++h) r.v[h] = h < cnt ? bf2f(p[h]) : 0.f;
  }
  return r;
}

template <int NT, bool VEC>
__device__ __forceinline__ void store_cols(float* p, int cnt, const Cols<NT>& c) {
  if (VEC && NT == 2) {
    if (cnt > 0) *reinterpret_cast<float2*>(p) = make_float2(c.v[0], c.v[NT - 1]);
  } else {
#pragma unroll
    for (int h = 0; h < NT; ++h)
      if (h < cnt) p[h] = c.v[h];
  }
}

template <int NT, bool VEC>
__device__ __forceinline__ void store_cols(bf16_t* p, int cnt, const Cols<NT>& c) {
  if (VEC && NT == 2) {
    if (cnt > 0) *reinterpret_cast<uint32_t*>(p) = pack_bf2_hw(c.v[0], c.v[NT - 1]);
  } else {
#pragma unroll
    for (int h = 0; h < NT; ++h)
      if (h < cnt) p[h] = (bf16_t)(pack_bf2_hw(c.v[h], 0.f) & 0xffffu);
  }
}

// The two bfloat16 parts of a lane's columns at p and p + lo.
template <int NT>
__device__ __forceinline__ void store_parts(bf16_t* p, int64_t lo, const Cols<NT>& c) {
  const uint32_t h = pack_bf2_hw(c.v[0], c.v[NT - 1]);
  const uint32_t l = pack_bf2_hw(c.v[0] - __uint_as_float(h << 16), c.v[NT - 1] - __uint_as_float(h & 0xffff0000u));
  if (NT == 2) {
    *reinterpret_cast<uint32_t*>(p) = h;
    *reinterpret_cast<uint32_t*>(p + lo) = l;
  } else {
    p[0] = (bf16_t)h;
    p[lo] = (bf16_t)l;
  }
}

// Two tokens' pieces into the transposed array: eight words of (token, token + 1).
template <int KP>
__device__ __forceinline__ void store_transposed(char* dst, int pair, int piece, bf8_t a, bf8_t b) {
  const u4_t e0 = __builtin_bit_cast(u4_t, a), e1 = __builtin_bit_cast(u4_t, b);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t lo = e & 1 ? e0[e >> 1] >> 16 : e0[e >> 1] & 0xffffu;
    const uint32_t hi = e & 1 ? e1[e >> 1] & 0xffff0000u : e1[e >> 1] << 16;
    *reinterpret_cast<uint32_t*>(dst + Tokens<KP>::col_at(place_of(8 * piece + e), 4 * pair)) = lo | hi;
  }
}

// The decay sums are float64 and their differences float32: a difference between two
// neighbours must not carry the rounding of a long sum. Below -200 a decay is 0 in float32
// whatever it is added to, so that -inf (a fresh start) stays a number here.
__device__ __forceinline__ double clamp_decay(float g) { return g < -200.f ? -200.0 : (double)g; }

// The running sum over a wave of 64 tokens.
__device__ __forceinline__ double running_sum(double s, int i) {
#pragma unroll
  for (int o = 1; o < CH; o <<= 1) {
    const double up = __shfl_up(s, o, 64);
    if (i >= o) s += up;
  }
  return s;
}

template <typename T, bool VEC>
__device__ __forceinline__ Op<Stream<T>::NP> token_op(const T* base, int64_t stride, int64_t tokens, int row, int k0,
                                                      int Dk) {
  const int cnt = row < tokens ? max(0, min(8, Dk - k0)) : 0;
  return load_raw8<VEC>(base + row * stride + k0, cnt).op();
}

}  // namespace

}  // namespace hc
