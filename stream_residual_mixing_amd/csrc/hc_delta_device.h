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

constexpr int CH = 64;        // tokens of a chunk
constexpr uint32_t DIES = 8;  // with an L2 each

typedef __bf16 bf8_t __attribute__((ext_vector_type(8)));
typedef float f4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u2_t __attribute__((ext_vector_type(2)));

__device__ __forceinline__ int row_of(int t, int m) { return 32 * (t >> 1) + 8 * (m >> 2) + 4 * (t & 1) + (m & 3); }

// the place of row x in that order
__device__ __forceinline__ int place_of(int x) { return (x & ~31) + 16 * ((x >> 2) & 1) + 4 * ((x >> 3) & 3) + (x & 3); }

// Eight values as the sum of NP bfloat16 parts. Three hold float32's own 24 bits; bfloat16 streams are
// their own single part.
template <int NP>
struct Op {
  bf8_t p[NP];
};
typedef Op<3> Fine;

__device__ __forceinline__ bf8_t as_bf8(u4_t q) { return __builtin_bit_cast(bf8_t, q); }

__device__ __forceinline__ u4_t pack8(const float v[8]) {
  u4_t q;
#pragma unroll
  for (int i = 0; i < 4; ++i) q[i] = pack_bf2_hw(v[2 * i], v[2 * i + 1]);
  return q;
}

template <int NP>
__device__ __forceinline__ Op<NP> split(f4_t a, f4_t b) {
  float v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
  Op<NP> o;
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const u4_t q = pack8(v);
    o.p[p] = as_bf8(q);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] -= __uint_as_float(q[i] << 16);
      v[2 * i + 1] -= __uint_as_float(q[i] & 0xffff0000u);
    }
  }
  return o;
}

template <int NP>
__device__ __forceinline__ Op<NP> split(const float v[8]) {
  return split<NP>(f4_t{v[0], v[1], v[2], v[3]}, f4_t{v[4], v[5], v[6], v[7]});
}

__device__ __forceinline__ f4_t mma(bf8_t a, bf8_t b, f4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// Parts i and j of two factors, the smallest products first: all but those with i + j > 2, each at most
// 2^-27 of the whole.
template <int NA, int NB>
__device__ __forceinline__ f4_t mma(const Op<NA>& a, const Op<NB>& b, f4_t c) {
#pragma unroll
  for (int s = 2; s >= 0; --s)
#pragma unroll
    for (int i = 0; i < NA; ++i)
      if (s - i >= 0 && s - i < NB) c = mma(a.p[i], b.p[s - i], c);
  return c;
}

// Stream operands: bfloat16 is exact in one part, float32 takes three.
template <typename T>
constexpr int PARTS = sizeof(T) == 4 ? 3 : 1;

// Memory from an address that the wave's lanes have in common, read and written at 32-bit offsets:
// what lies at or behind its end reads as 0 and is not written, so that neither the last chunk's
// missing tokens nor a head's missing keys and columns need a branch. NOWHERE is behind every end
// and stays so with a row's offset added (both below 2^31).
constexpr uint32_t NOWHERE = 0x80000000u;

struct F8 {
  f4_t a, b;
};

struct Range {
  __amdgpu_buffer_rsrc_t r;
  __device__ __forceinline__ Range(const void* p, int64_t bytes)
      : r(__builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)bytes, 0x00027000)) {}
  __device__ __forceinline__ u4_t quad(uint32_t o) const {
    return __builtin_bit_cast(u4_t, __builtin_amdgcn_raw_buffer_load_b128(r, o, 0, 0));
  }
  __device__ __forceinline__ float get(const float*, uint32_t o) const {
    return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, o, 0, 0));
  }
  __device__ __forceinline__ float get(const bf16_t*, uint32_t o) const {
    return bf2f(__builtin_amdgcn_raw_buffer_load_b16(r, o, 0, 0));
  }
  __device__ __forceinline__ void put(float* , uint32_t o, float v) const {
    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), r, o, 0, 0);
  }
  __device__ __forceinline__ void put(bf16_t*, uint32_t o, float v) const {
    __builtin_amdgcn_raw_buffer_store_b16((uint16_t)pack_bf2_hw(v, 0.f), r, o, 0, 0);
  }
  __device__ __forceinline__ void put_quad(uint32_t o, u4_t v) const {
    __builtin_amdgcn_raw_buffer_store_b128(v, r, o, 0, 0);
  }
  // eight floats of a kept array, at an offset `s` more that the lanes have in common; inside it
  __device__ __forceinline__ F8 floats(uint32_t o, uint32_t s) const {
    return {__builtin_bit_cast(f4_t, __builtin_amdgcn_raw_buffer_load_b128(r, o, s, 0)),
            __builtin_bit_cast(f4_t, __builtin_amdgcn_raw_buffer_load_b128(r, o, s + 16, 0))};
  }
  // an operand kept in three parts, `part` bytes apart, at an offset `s` more that the lanes have in common; inside it
  __device__ __forceinline__ Fine parts(uint32_t o, uint32_t s, uint32_t part) const {
    Fine f;
#pragma unroll
    for (int p = 0; p < 3; ++p)
      f.p[p] = __builtin_bit_cast(bf8_t, __builtin_amdgcn_raw_buffer_load_b128(r, o, s + p * part, 0));
    return f;
  }
};

// Rows of a head's keys, queries or values in a chunk: `left` of them, `stride` elements apart,
// `width` elements each.
template <typename T>
__device__ __forceinline__ Range head_rows(const T* p, int left, int64_t stride, int width) {
  return Range(p, left > 0 ? ((left - 1) * stride + width) * (int64_t)sizeof(T) : 0);
}

// Eight consecutive stream elements as stored, at byte offset o; the first `cnt` exist (VEC: all or
// none).
template <typename T> struct Raw8;
template <> struct Raw8<bf16_t> {
  u4_t q;
  template <bool VEC>
  __device__ __forceinline__ void load(const Range& m, uint32_t o, int cnt) {
    if (VEC) {
      q = m.quad(cnt > 0 ? o : NOWHERE);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        q[i] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(m.r, 2 * i < cnt ? o + 4 * i : NOWHERE, 0, 0) |
               (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(m.r, 2 * i + 1 < cnt ? o + 4 * i + 2 : NOWHERE, 0, 0) << 16;
    }
  }
  template <int NP>
  __device__ __forceinline__ Op<NP> op() const { return {as_bf8(q)}; }
};
template <> struct Raw8<float> {
  f4_t a, b;
  template <bool VEC>
  __device__ __forceinline__ void load(const Range& m, uint32_t o, int cnt) {
    if (VEC) {
      a = __builtin_bit_cast(f4_t, m.quad(cnt > 0 ? o : NOWHERE));
      b = __builtin_bit_cast(f4_t, m.quad(cnt > 0 ? o + 16 : NOWHERE));
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        a[e] = m.get((const float*)nullptr, e < cnt ? o + 4 * e : NOWHERE);
        b[e] = m.get((const float*)nullptr, 4 + e < cnt ? o + 16 + 4 * e : NOWHERE);
      }
    }
  }
  template <int NP>
  __device__ __forceinline__ Op<NP> op() const {
    return split<NP>(a, b);
  }
};

// Eight keys of a row from k0 on, as an operand.
template <typename T, bool VEC, int NP = PARTS<T>>
__device__ __forceinline__ Op<NP> token_op(const Range& m, uint32_t stride, int row, int k0, int width) {
  Raw8<T> x;
  x.template load<VEC>(m, (row * stride + k0) * (uint32_t)sizeof(T), width - k0);
  return x.template op<NP>();
}

// Tokens of sequence b.
__device__ __forceinline__ int64_t length_of(const int32_t* lengths, int64_t b, int64_t S) {
  if (lengths == nullptr) return S;
  const int64_t n = lengths[b];
  return n < 0 ? 0 : n > S ? S : n;
}

// A chunk's record, float32: decays and betas, a value per token, and 16 x 32 operand tiles of 64 lanes by
// eight values, first all lanes' four and then their other four, of the two lower block-triangular
// matrices T (rows in row_of's order) and P (rows in their own), tile (t, kb) at tri(t, kb). The backward's
// holds T and, upper triangular at tri_t, the transposes of both with rows in row_of's order.
constexpr int TILES = 6, TILE = 1024, TRI = TILES * 2 * TILE;
constexpr int REC_DEC = 0, REC_T = 3 * CH * 4, REC_P = REC_T + TRI, REC = REC_P + TRI;
constexpr int REC_TT = REC, REC_BWD = REC + TRI;
constexpr int DEC_AHEAD = 0, DEC_TO_END = CH, DEC_BETA = 2 * CH;

__device__ __forceinline__ constexpr int tri(int t, int kb) { return t < 2 ? t : 2 * t - 2 + kb; }
__device__ __forceinline__ constexpr int tri_t(int t, int kb) { return t < 2 ? 2 * t + kb : t + 2; }

__device__ __forceinline__ void store_tile(char* m, int idx, int lane, const float v[8]) {
  f4_t* p = reinterpret_cast<f4_t*>(m + idx * 2 * TILE) + lane;
  p[0] = f4_t{v[0], v[1], v[2], v[3]};
  p[64] = f4_t{v[4], v[5], v[6], v[7]};
}

// N of the record's matrices in LDS, as operands in three parts, with the decays and betas.
template <int N, int THREADS>
struct Record {
  static constexpr int PART = TILES * TILE, ALL = N * TILES * 64, ITEMS = (ALL + THREADS - 1) / THREADS;
  char m[N][3 * PART];
  float dec[3 * CH];
  struct Raw {  // on its way
    f4_t v[ITEMS][2], d;
    // `r` ends with the last of the matrices, the first lies at `from`
    __device__ __forceinline__ void load(const Range& r, int from, int tid) {
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        const int x = i * THREADS + tid, o = from + (x >> 6) * 2 * TILE + (x & 63) * 16;
        v[i][0] = __builtin_bit_cast(f4_t, r.quad(o));
        v[i][1] = __builtin_bit_cast(f4_t, r.quad(o + TILE));
      }
      d = __builtin_bit_cast(f4_t, r.quad(tid < 3 * CH / 4 ? REC_DEC + 16 * tid : NOWHERE));
    }
  };
  __device__ __forceinline__ void put(const Raw& raw, int tid) {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int x = i * THREADS + tid, of = x / (TILES * 64), at = x % (TILES * 64) * 16;
      if (ALL % THREADS == 0 || x < ALL) {
        const Fine f = split<3>(raw.v[i][0], raw.v[i][1]);
#pragma unroll
        for (int p = 0; p < 3; ++p) *reinterpret_cast<bf8_t*>(m[of] + p * PART + at) = f.p[p];
      }
    }
    if (tid < 3 * CH / 4) *reinterpret_cast<f4_t*>(dec + 4 * tid) = raw.d;
  }
  __device__ __forceinline__ Fine tile(int of, int idx, int lane) const {
    const char* at = m[of] + idx * TILE + lane * 16;
    Fine f;
#pragma unroll
    for (int p = 0; p < 3; ++p) f.p[p] = *reinterpret_cast<const bf8_t*>(at + p * PART);
    return f;
  }
};

// A chunk's keys or queries in LDS, [CH][KP] with the rows where the caller puts them. The 16-byte
// pieces of a row are exchanged so that both readings reach all banks: a piece of 16 rows (an
// operand whose rows are tokens), and four tokens by 16 keys (its transpose's).
template <int KP>
struct Tokens {
  static constexpr int ROW = 2 * KP, BYTES = CH * ROW;
  static __device__ __forceinline__ int key(int place) {
    return KP == 64 ? ((place << 1) & 4) | ((place >> 2) & 3) : ((place & 3) << 2) | ((place >> 2) & 3);
  }
  static __device__ __forceinline__ int at(int place, int piece) { return place * ROW + ((piece ^ key(place)) << 4); }
  // operand tile t by k block kb, rows 16 t + n: `lane_at` is the lane's own part
  static __device__ __forceinline__ int lane_at(int n, int g) { return at(n, g); }
  static __device__ __forceinline__ bf8_t rows(const char* m, int lane_at, int t, int kb) {
    return *reinterpret_cast<const bf8_t*>(m + 16 * t * ROW + (lane_at ^ (kb << 6)));
  }
  // the transpose's: rows are keys in row_of's order, k are tokens whose places are place_of theirs
  static __device__ __forceinline__ int lane_at_t(int n, int g) { return at(4 * g + (n >> 2), n & 3); }
  static __device__ __forceinline__ bf8_t cols(const char* m, int lane_at, int t, int kb) {
    typedef short s4_t __attribute__((ext_vector_type(4)));
    typedef short s8_t __attribute__((ext_vector_type(8)));
    typedef __attribute__((address_space(3))) s4_t lds_s4;
    const char* p = m + 32 * kb * ROW + (lane_at ^ ((t >> 1) << 6)) + 8 * (t & 1);
    const s4_t a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)p);
    const s4_t b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)(p + 16 * ROW));
    return __builtin_bit_cast(bf8_t, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
  }
};

// The wave's number in its workgroup, as a value that its lanes have in common.
__device__ __forceinline__ int wave_number() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// No instruction is moved across: the next step's operands are not all read ahead, for
// which there are no registers.
__device__ __forceinline__ void keep_order() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// The lane's numbers anew, so that what a loop forms of them is not kept in registers over it.
__device__ __forceinline__ void renew(int& a, int& b) { asm volatile("" : "+v"(a), "+v"(b)); }
// The operand is formed here, not where it is used.
template <int NP>
__device__ __forceinline__ void pin(Op<NP>& s) {
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    u4_t q = __builtin_bit_cast(u4_t, s.p[p]);
    asm volatile("" : "+v"(q));
    s.p[p] = as_bf8(q);
  }
}
__device__ __forceinline__ uint32_t anew(uint32_t a) {
  asm volatile("" : "+v"(a));
  return a;
}

// A wave's 16 columns of the state: a lane has column n and, of each tile of 16 rows, four of them.
template <int KP>
struct State {
  f4_t m[KP / 16];
  // [Dk, Dv] at p, the wave's first column; NULL: zeros
  __device__ __forceinline__ void load(const float* p, int Dk, int Dv, int n, int g, int columns) {
    const Range m(p, p && columns > 0 ? ((int64_t)(Dk - 1) * Dv + columns) * 4 : 0);
    const uint32_t lane = n < columns ? 4 * (8 * g * Dv + n) : NOWHERE;
#pragma unroll
    for (int t = 0; t < KP / 16; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) this->m[t][r] = m.get(p, lane + 4 * row_of(t, r) * Dv);
  }
  __device__ __forceinline__ void store(float* p, int Dk, int Dv, int n, int g, int columns) const {
    const Range m(p, columns > 0 ? ((int64_t)(Dk - 1) * Dv + columns) * 4 : 0);
    const uint32_t lane = n < columns ? 4 * (8 * g * Dv + n) : NOWHERE;
#pragma unroll
    for (int t = 0; t < KP / 16; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) m.put(p, lane + 4 * row_of(t, r) * Dv, this->m[t][r]);
  }
  // [KP, stride] at p, column `col` of lane 0
  __device__ __forceinline__ void keep(float* p, int stride, int col, int n, int g) const {
    const Range m(p, 4 * KP * stride);
    const uint32_t lane = anew(col < stride ? 4 * (8 * g * stride + col + n) : NOWHERE);
#pragma unroll
    for (int t = 0; t < KP / 16; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) m.put(p, lane + 4 * row_of(t, r) * stride, this->m[t][r]);
  }
  // the same [KP, KP], in three parts one after the other
  __device__ __forceinline__ void keep(bf16_t* p, int col, int n, int g) const {
    const Range m(p, 6 * KP * KP);
    const uint32_t lane = anew(2 * (8 * g * KP + col + n));
#pragma unroll
    for (int t = 0; t < KP / 16; ++t) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float left = this->m[t][r];
#pragma unroll
        for (int i = 0; i < 3; ++i) {
          const uint32_t h = pack_bf2_hw(left, 0.f);
          __builtin_amdgcn_raw_buffer_store_b16((uint16_t)h, m.r, lane + 2 * row_of(t, r) * KP, i * 2 * KP * KP, 0);
          left -= __uint_as_float(h << 16);
        }
      }
    }
  }
};

// Workgroups of four waves on a CU that LDS has room for, up to the two that the walks have registers for;
// with one each wave may take 512 (8 x 1,024 tokens, 16 heads, measured with two parts: 256 x 256 in float32 460 us,
// with 256 registers and spills 1,173; in bfloat16 273 and 356; 128 x 128 in float32 162 and 171).
template <typename Lds>
constexpr int WALKS = sizeof(Lds) <= 80 * 1024 ? 2 : 1;

// The grid's `units` by `members` workgroups, the members of a unit on one die, whose L2 then brings
// what they all read once: consecutive workgroups go round the dies. The units behind the last
// multiple of the dies in plain order. Against plain order throughout, with two parts: walks of 2,048 chunks 85 -> 79 us, in
// segments 70 + 69 -> 62 + 60; the backward's 637 -> 619 us in all.
struct Place {
  uint32_t unit, member;
  __device__ __forceinline__ Place(uint32_t units, uint32_t members) {
    const uint32_t x = blockIdx.x, even = units / DIES * DIES, mixed = even * members;
    const uint32_t j = x < mixed ? x / DIES : x - mixed;
    unit = x < mixed ? j / members * DIES + x % DIES : even + j / members;
    member = j % members;
  }
};

// A workgroup of the walks: a segment of a head's chunks by a group of its columns. All that walk the same
// keys are a unit.
struct Part {
  int64_t bh, b, slot;
  uint32_t hv, hk;
  int seg, group;
  int64_t len, chunks, first, last;  // [first, last) of them are this segment's
  __device__ __forceinline__ Part(const DeltaArgs& a, uint32_t groups) {
    const uint32_t NS = (uint32_t)a.NS, Hk = (uint32_t)a.Hk, per = (uint32_t)a.Hv / Hk;
    const Place at((uint32_t)a.B * Hk * NS, per * groups);
    group = (int)(at.member % groups);
    seg = (int)(at.unit % NS);
    b = at.unit / NS / Hk;
    hk = at.unit / NS % Hk;
    hv = hk * per + at.member / groups;
    bh = b * a.Hv + hv;
    slot = bh * NS + seg;
    len = length_of(a.lengths, b, a.S);
    chunks = (len + CH - 1) / CH;
    first = seg * a.SL;
    last = min(chunks, first + a.SL);
  }
  // the sequence ends before this segment; the first one passes an empty sequence's state on
  __device__ __forceinline__ bool empty() const { return seg > 0 && first >= chunks; }
  __device__ __forceinline__ bool ends() const { return last >= chunks; }  // none comes behind it
};

// Four tiles of a chunk's 64 rows, as [CH, stride].
__device__ __forceinline__ void keep_rows(float* p, int stride, int col, int n, int g, const f4_t (&x)[4]) {
  const Range m(p, 4 * CH * stride);
  const uint32_t lane = anew(col < stride ? 4 * (8 * g * stride + col + n) : NOWHERE);
#pragma unroll
  for (int t = 0; t < 4; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r) m.put(p, lane + 4 * row_of(t, r) * stride, x[t][r]);
}

// The decay sums are float64 and their differences float32: a difference between two
// neighbours must not carry the rounding of a long sum. Below -200 a decay is 0 in float32
// whatever it is added to, so that -inf (a fresh start) stays a number here.
__device__ __forceinline__ double clamp_decay(float g) { return g < -200.f ? -200.0 : (double)g; }

// exp(x) of a difference of the sums, off by |x| 2^-23 of itself at most: |x| exp(x) 2^-23 <= 4 x 10^-8 of what
// it decays, however long that has been forgotten.
__device__ __forceinline__ float decay(double x) { return __builtin_amdgcn_exp2f((float)x * 1.44269504f); }

// The running sum over a wave of 64 tokens.
__device__ __forceinline__ double running_sum(double s, int i) {
#pragma unroll
  for (int o = 1; o < CH; o <<= 1) {
    const double up = __shfl_up(s, o, 64);
    if (i >= o) s += up;
  }
  return s;
}

}  // namespace

}  // namespace hc
