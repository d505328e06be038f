// Root-mean-square norm in front of a sublayer function, forward and backward.
//   v = x, x + residual, or the pre-read sum_i h_pre[i] X[i];
//   y = v * w / sqrt(mean_c v^2 + eps), stored in the stream dtype or as 8-bit
//   codes with a scale per row or per group of 32, 64 or 128 channels.
// Each row is read once and stays in float32 registers between the sum of squares
// and the outputs, so the passes are bound by HBM traffic. Per call: 5.8 TB/s for 8,192 x
// 4,096 bfloat16 with residual and e4m3 output (40.5 us), 5.7 for the pre-read form of
// 16,384 x 4 x 7,168 (247 us), 5.5 for the backward of 8,191 x 4,096 (49 us, 4 of them the
// sum of dw's parts). Small calls are bound by the launch (16 x 4,096: 5 us).
#include "hc_sublayer.h"
#include "hc_sublayer_device.h"

namespace hc {

namespace {

constexpr int OUT_STREAM = 0, OUT_E4M3 = 2;  // else int8 codes (the 8-bit forms by their dtype codes in hc.h)

// A row's channels lie in pieces of 8, piece (it * NT + tid) of item it with its NT
// threads: a wave, four rows to a workgroup and no barrier (WAVE, up to 512 channels),
// else a workgroup of as many waves as the row fills (a wave with more pieces a thread
// takes 45 against 35 us backward at 16,384 x 1,024 and 73 against 55 at 2,048 channels;
// forward the two are within 4 %).
constexpr int WAVE_ROWS = 4;

template <bool WAVE>
struct RowThreads {
  int nt, tid, sub;  // threads of a row, this one's number, its row in the workgroup
  __device__ __forceinline__ RowThreads() {
    nt = WAVE ? 64 : blockDim.x;
    tid = WAVE ? threadIdx.x & 63 : threadIdx.x;
    sub = WAVE ? threadIdx.x >> 6 : 0;
  }
  static __device__ __forceinline__ int rows() { return WAVE ? WAVE_ROWS : 1; }
};

// VEC: rows of whole pieces at 16-byte aligned addresses. Otherwise every load is still
// one access (global memory takes any element-aligned address): a row's ragged last
// piece is read as the row's last 8 channels and moved into place when it is opened, so
// that nothing waits for it early.
__device__ __forceinline__ int piece_count(uint32_t c0, uint32_t C) { return c0 < C ? (int)min(8u, C - c0) : 0; }

// 16 bytes at any address of a 2-byte element. bfloat16 rows are streamed, as the aligned
// ones are (ordinary loads are moved down to their first use: 97 against 59 us at 8,192 x
// 4,098); float32 rows, whose lanes skip every other 16 bytes, are not (113 against 120).
typedef uint32_t u4_any __attribute__((ext_vector_type(4), aligned(2)));

// A piece as stored, so that the next row's can be on their way in few registers.
template <typename T> struct Piece;
template <> struct Piece<float> {
  float q[8];
  __device__ __forceinline__ void open(float v[8]) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = q[e];
  }
  __device__ __forceinline__ void close(const float v[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) q[e] = v[e];
  }
};
template <> struct Piece<bf16_t> {
  uint32_t q[4];
  __device__ __forceinline__ void open(float v[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(q[i] << 16);
      v[2 * i + 1] = __uint_as_float(q[i] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ void close(const float v[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = pack_bf2_hw(v[2 * i], v[2 * i + 1]);
  }
};

template <bool VEC, typename T>
__device__ __forceinline__ void row_load(const T* row, uint32_t c0, uint32_t C, Piece<T>& v) {
  typedef uint32_t u4 __attribute__((ext_vector_type(4)));
  const int cnt = piece_count(c0, C);
  if (VEC && cnt > 0) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(v) / 16; ++i) {
      const u4 q = __builtin_nontemporal_load(reinterpret_cast<const u4*>(row + c0) + i);
      __builtin_memcpy((char*)v.q + 16 * i, &q, 16);
    }
  } else if (!VEC && C >= 8) {
    const T* p = row + (cnt == 8 ? c0 : C - 8);
    if (sizeof(T) == 2) {
      const u4_any q = __builtin_nontemporal_load(reinterpret_cast<const u4_any*>(p));
      __builtin_memcpy(v.q, &q, 16);
    } else {
      __builtin_memcpy(v.q, p, sizeof(v));
    }
  } else {
    T e8[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) e8[e] = !VEC && e < cnt ? row[c0 + e] : T(0);
    __builtin_memcpy(v.q, e8, sizeof(v));
  }
}

// The piece as 8 channels, those past the row 0.
template <bool VEC, typename T>
__device__ __forceinline__ void row_open(const Piece<T>& raw, uint32_t c0, uint32_t C, float v[8]) {
  const int cnt = piece_count(c0, C);
  if (VEC || C < 8 || cnt == 8) {
    raw.open(v);
    return;
  }
  const int by = 8 - cnt;  // the piece's first channel is element `by` of what was read
  raw.open(v);
#pragma unroll
  for (int st = 4; st >= 1; st >>= 1)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float up = e + st < 8 ? v[e + st] : 0.f;
      v[e] = (by & st) ? up : v[e];
    }
  if (by == 8) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 0.f;
  }
}

template <bool VEC, typename T>
__device__ __forceinline__ void row_store(T* row, uint32_t c0, uint32_t C, const float v[8]) {
  typedef uint32_t u4 __attribute__((ext_vector_type(4)));
  const int cnt = piece_count(c0, C);
  Piece<T> p;
  p.close(v);
  if (VEC) {
    if (cnt > 0)
#pragma unroll
      for (int i = 0; i < (int)sizeof(p) / 16; ++i) {
        u4 q;
        __builtin_memcpy(&q, (const char*)p.q + 16 * i, 16);
        __builtin_nontemporal_store(q, reinterpret_cast<u4*>(row + c0) + i);
      }
  } else if (cnt == 8) {
    if (sizeof(T) == 2) {
      u4_any q;
      __builtin_memcpy(&q, p.q, 16);
      __builtin_nontemporal_store(q, reinterpret_cast<u4_any*>(row + c0));
    } else {
      __builtin_memcpy(row + c0, p.q, sizeof(p));
    }
  } else {
    T e8[8];
    __builtin_memcpy(e8, p.q, sizeof(p));
#pragma unroll
    for (int e = 0; e < 7; ++e)
      if (e < cnt) row[c0 + e] = e8[e];
  }
}

// The weight is used by every row: ordinary loads, kept in registers over the rows.
template <bool VEC, int ITEMS>
__device__ __forceinline__ void load_weight(const float* w, uint32_t C, uint32_t nt, uint32_t tid, float out[ITEMS][8]) {
#pragma unroll
  for (int it = 0; it < ITEMS; ++it) {
    const uint32_t c0 = (it * nt + tid) * 8;
    if (w == nullptr) {
#pragma unroll
      for (int e = 0; e < 8; ++e) out[it][e] = 1.f;
    } else if (piece_count(c0, C) == 8) {
      if (VEC) load8(w + c0, out[it]);
      else load8_any(w + c0, out[it]);
    } else {
      load8_tail(w + c0, piece_count(c0, C), out[it]);
    }
  }
}

// Sums of NV values over one row's threads, the same in each; `red` is this row parity's
// slice of LDS (the next row uses the other one, so one barrier a row is enough).
template <bool WAVE, int NV>
__device__ __forceinline__ void row_sum(float v[NV], float (*red)[16]) {
#pragma unroll
  for (int i = 0; i < NV; ++i) v[i] = wave_sum(v[i]);
  if (WAVE) return;
  if ((threadIdx.x & 63) == 0)
#pragma unroll
    for (int i = 0; i < NV; ++i) red[i][threadIdx.x >> 6] = v[i];
  lds_barrier();
  const int nw = blockDim.x >> 6;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    v[i] = 0.f;
    for (int w = 0; w < nw; ++w) v[i] += red[i][w];
  }
}

// The largest magnitude as float bits: ordering the bits as unsigned numbers puts
// infinity above every number and NaN above infinity, so a NaN is never lost.
template <int CTRL>
__device__ __forceinline__ uint32_t umax_dpp(uint32_t v) {
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true));
}
constexpr int DPP_HALF_MIRROR = 0x141;  // lane i of 8 takes lane 7 - i

__device__ __forceinline__ uint32_t umax4(uint32_t v) { return umax_dpp<DPP_QXOR2>(umax_dpp<DPP_QXOR1>(v)); }
__device__ __forceinline__ uint32_t umax8(uint32_t v) { return umax_dpp<DPP_HALF_MIRROR>(umax4(v)); }
__device__ __forceinline__ uint32_t umax16(uint32_t v) { return umax_dpp<DPP_ROR8>(umax8(v)); }

// A value that the wave's lanes have in common, in a scalar register.
__device__ __forceinline__ float uniform(float v) {
  return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(v)));
}

template <bool WAVE>
__device__ __forceinline__ uint32_t row_umax(uint32_t v, uint32_t* red) {
  v = umax16(v);
  v = max(v, (uint32_t)__shfl_xor((int)v, 16, 64));
  v = max(v, (uint32_t)__shfl_xor((int)v, 32, 64));
  if (WAVE) return v;
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  lds_barrier();
  const int nw = blockDim.x >> 6;
  uint32_t s = 0;
  for (int i = 0; i < nw; ++i) s = max(s, red[i]);
  return s;
}

__device__ __forceinline__ float rms_factor(float ms) {
  return ms == 0.f ? 0.f : 1.0f / sqrtf(ms);  // the all-zero row without eps normalises to zero
}

// A row whose mean square + eps is in this range has the sum it should have: no square
// passes float32's largest number, and what squares lose below its smallest normal one
// (2^-126 each) is at most 2^-26 of their mean.
__device__ __forceinline__ bool in_range(float ms) { return ms >= 0x1p-100f && ms <= 3.4028235e38f; }

// The others are taken relative to 2^k, the power of two over the row's largest magnitude
// (its bits: `largest`) or sqrt(eps), whichever is more: the norm of v 2^-k with eps 2^-2k
// is that of v with eps, and scaling by a power of two is exact. No such power where the
// row is all zero, or infinite or NaN somewhere.
__device__ __forceinline__ bool scale_of(uint32_t largest, float eps, int& k) {
  if (largest == 0 || largest >= 0x7f800000u) return false;
  k = __builtin_amdgcn_frexp_expf(__uint_as_float(largest));
  if (eps > 0.f) k = max(k, (__builtin_amdgcn_frexp_expf(eps) + 1) >> 1);
  return true;
}

// 8 codes of 8 bits. Clamped first: rounding up at the largest code would overflow.
__device__ __forceinline__ uint2 pack_e4m3(const float v[8], float inv) {
  float c[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float q = v[e] * inv;
    c[e] = q != q ? q : fminf(fmaxf(q, -448.f), 448.f);
  }
  uint2 r;
  int lo = 0, hi = 0;
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(c[0], c[1], lo, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(c[2], c[3], lo, true);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(c[4], c[5], hi, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(c[6], c[7], hi, true);
  r.x = (uint32_t)lo;
  r.y = (uint32_t)hi;
  return r;
}

__device__ __forceinline__ uint2 pack_i8(const float v[8], float inv) {
  uint32_t b[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float q = v[e] * inv;
    b[e] = (uint32_t)(q != q ? 0 : (int)rintf(fminf(fmaxf(q, -127.f), 127.f))) & 0xffu;
  }
  uint2 r;
  r.x = b[0] | (b[1] << 8) | (b[2] << 16) | (b[3] << 24);
  r.y = b[4] | (b[5] << 8) | (b[6] << 16) | (b[7] << 24);
  return r;
}

// MODE 0: v = x; 1: v = x + residual; 2: v = sum_i h[i] x[i] (n streams, four of them on
// their way at once). In modes 0 and 1 the next row is on its way while this one is
// finished (the same for four streams gained nothing: 254 against 248 us).
template <typename T, int MODE, int ITEMS, bool WAVE, bool VEC>
__global__ __launch_bounds__(WAVE ? 64 * WAVE_ROWS : 1024) void rms_norm_kernel(NormArgs a) {
  constexpr int NS = MODE == 1 ? 2 : 1;  // arrays of a row
  __shared__ float red[2][1][16];
  __shared__ uint32_t redm[2][16];
  const RowThreads<WAVE> r;
  const uint32_t tid = r.tid, NT = r.nt, C = (uint32_t)a.C;
  const int64_t step = (int64_t)gridDim.x * r.rows();
  const float inv_c = 1.0f / (float)C;
  float w[ITEMS][8];
  load_weight<VEC, ITEMS>(a.w, C, NT, tid, w);
  int64_t t = (int64_t)blockIdx.x * r.rows() + r.sub;
  Piece<T> raw[NS][ITEMS];
  const auto fetch = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < NS; ++i)
#pragma unroll
      for (int it = 0; it < ITEMS; ++it) {
        row_load<VEC>((const T*)(i == 0 ? a.x : a.res) + row * C, (it * NT + tid) * 8, C, raw[i][it]);
      }
  };
  if (MODE != 2 && t < a.T) fetch(t);
  for (int parity = 0; t < a.T; t += step, parity ^= 1) {
    float v[ITEMS][8];
    float ss = 0.f;
    if (MODE == 2) {
#pragma unroll
      for (int it = 0; it < ITEMS; ++it)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[it][e] = 0.f;
#pragma unroll 4
      for (int i = 0; i < a.n; ++i) {
        const float hi = a.h[t * a.n + i];
#pragma unroll
        for (int it = 0; it < ITEMS; ++it) {
          Piece<T> q;
          float xi[8];
          row_load<VEC>((const T*)a.x + (t * a.n + i) * C, (it * NT + tid) * 8, C, q);
          row_open<VEC>(q, (it * NT + tid) * 8, C, xi);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[it][e] += hi * xi[e];
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < NS; ++i) {
#pragma unroll
        for (int it = 0; it < ITEMS; ++it) {
          float xi[8];
          row_open<VEC>(raw[i][it], (it * NT + tid) * 8, C, xi);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[it][e] = i == 0 ? xi[e] : v[it][e] + xi[e];
        }
      }
      if (t + step < a.T) fetch(t + step);
    }
#pragma unroll
    for (int it = 0; it < ITEMS; ++it) {
      const uint32_t c0 = (it * NT + tid) * 8;
      if (MODE != 0 && a.s) row_store<VEC>((T*)a.s + t * C, c0, C, v[it]);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (MODE != 2 || (VEC ? c0 : c0 + e) < C) ss += v[it][e] * v[it][e];  // 0 * an infinite h is no channel's
    }
    row_sum<WAVE, 1>(&ss, red[parity]);
    float ms = uniform(ss * inv_c + a.eps);
    if (!in_range(ms)) {
      uint32_t top = 0;
#pragma unroll
      for (int it = 0; it < ITEMS; ++it)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (MODE != 2 || (it * NT + tid) * 8 + (VEC ? 0 : e) < C)
            top = max(top, __float_as_uint(v[it][e]) & 0x7fffffffu);
      int k;
      if (scale_of(row_umax<WAVE>(top, redm[parity]), a.eps, k)) {
        ss = 0.f;
#pragma unroll
        for (int it = 0; it < ITEMS; ++it)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            v[it][e] = __builtin_amdgcn_ldexpf(v[it][e], -k);
            if (MODE != 2 || (it * NT + tid) * 8 + (VEC ? 0 : e) < C) ss += v[it][e] * v[it][e];
          }
        row_sum<WAVE, 1>(&ss, red[parity]);
        ms = ss * inv_c + __builtin_amdgcn_ldexpf(a.eps, -2 * k);
      }
    }
    const float rstd = rms_factor(ms);
#pragma unroll
    for (int it = 0; it < ITEMS; ++it)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[it][e] *= rstd * w[it][e];
    if (a.out == OUT_STREAM) {
#pragma unroll
      for (int it = 0; it < ITEMS; ++it)
        row_store<VEC>((T*)a.y + t * C, (it * NT + tid) * 8, C, v[it]);
      continue;
    }
    uint32_t m[ITEMS];
#pragma unroll
    for (int it = 0; it < ITEMS; ++it) {
      m[it] = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const bool in = VEC ? (it * NT + tid) * 8 < C : (it * NT + tid) * 8 + e < C;
        if (in) m[it] = max(m[it], __float_as_uint(v[it][e]) & 0x7fffffffu);
      }
    }
    const float qmax = a.out == OUT_E4M3 ? 448.f : 127.f;
    if (a.group == 0) {
      uint32_t all = 0;
#pragma unroll
      for (int it = 0; it < ITEMS; ++it) all = max(all, m[it]);
      all = row_umax<WAVE>(all, redm[parity]);
#pragma unroll
      for (int it = 0; it < ITEMS; ++it) m[it] = all;
    } else {  // a group's 4, 8 or 16 threads are neighbours in a wave
#pragma unroll
      for (int it = 0; it < ITEMS; ++it)
        m[it] = a.group == 32 ? umax4(m[it]) : a.group == 64 ? umax8(m[it]) : umax16(m[it]);
    }
#pragma unroll
    for (int it = 0; it < ITEMS; ++it) {
      const uint32_t c0 = (it * NT + tid) * 8;
      float scale = __uint_as_float(m[it]) / qmax;
      if (scale < 0x1p-126f) scale = 1.f;
      const float inv = 1.f / scale;
      if (c0 < C) {
        if (a.group == 0) {
          if (c0 == 0) a.scale[t] = scale;
        } else if (c0 % a.group == 0) {
          a.scale[t * a.ngroups + c0 / a.group] = scale;
        }
        const uint2 q = a.out == OUT_E4M3 ? pack_e4m3(v[it], inv) : pack_i8(v[it], inv);
        uint8_t* p = (uint8_t*)a.y + t * C + c0;
        const int cnt = piece_count(c0, C);
        if (VEC) {
          *reinterpret_cast<uint2*>(p) = q;
        } else if (cnt == 8) {
          __builtin_memcpy(p, &q, 8);
        } else {
          for (int e = 0; e < cnt; ++e) p[e] = (uint8_t)((e < 4 ? q.x >> (8 * e) : q.y >> (8 * (e - 4))) & 0xffu);
        }
      }
    }
  }
}

// A thread's eight values of each of its pieces, kept over the rows: in registers with
// one piece, in its own places of LDS (128 KB, one workgroup per CU as its registers leave it)
// with two, where the weight and its gradient beside two rows of operands would spill: 4,096
// rows of 16,384 channels 99 us in bfloat16 and 238 in float32, 152 and 464 from registers.
template <int ITEMS>
struct PieceSums {
  float r[8];
  __device__ __forceinline__ void put(int, const float (&v)[8], int) {
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e] = v[e];
  }
  __device__ __forceinline__ void get(int, float (&v)[8], int) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = r[e];
  }
};
template <>
struct PieceSums<2> {
  static __device__ __forceinline__ float4* at(int it, int array) {
    __shared__ float4 kept[2][4][1024];
    return &kept[array][2 * it][threadIdx.x];
  }
  __device__ __forceinline__ void put(int it, const float (&v)[8], int array) {
    float4* p = at(it, array);
    p[0] = make_float4(v[0], v[1], v[2], v[3]);
    p[1024] = make_float4(v[4], v[5], v[6], v[7]);
  }
  __device__ __forceinline__ void get(int it, float (&v)[8], int array) const {
    const float4 *p = at(it, array), a = p[0], b = p[1024];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
};

// dx = rstd w dy - v rstd^3 mean(w dy v) + ds, and this workgroup's part of
// dw = sum_t dy v rstd, kept in registers over its rows and written once to
// part[workgroup][C] (the parts are added in a fixed order afterwards).
template <typename T, int ITEMS, bool WAVE, bool VEC>
__global__ __launch_bounds__(WAVE ? 64 * WAVE_ROWS : 1024) void rms_norm_backward_kernel(NormBwdArgs a) {
  __shared__ float red[2][2][16];
  __shared__ uint32_t redm[2][16];
  const RowThreads<WAVE> r;
  const uint32_t tid = r.tid, NT = r.nt, C = (uint32_t)a.C;
  const float inv_c = 1.0f / (float)C;
  PieceSums<ITEMS> w, dw;
  {
    float w0[ITEMS][8];
    const float zero[8] = {};
    load_weight<VEC, ITEMS>(a.w, C, NT, tid, w0);
#pragma unroll
    for (int it = 0; it < ITEMS; ++it) {
      w.put(it, w0[it], 0);
      dw.put(it, zero, 1);
    }
  }
  const int64_t step = (int64_t)gridDim.x * r.rows();
  int64_t t = (int64_t)blockIdx.x * r.rows() + r.sub;
  constexpr bool DS_AHEAD = ITEMS == 1 || sizeof(T) == 2;  // two pieces of float32 would spill
  Piece<T> rv[ITEMS], ry[ITEMS], rs[ITEMS];
  const auto fetch = [&](int64_t row) {
#pragma unroll
    for (int it = 0; it < ITEMS; ++it) {
      const uint32_t c0 = (it * NT + tid) * 8;
      row_load<VEC>((const T*)a.s + row * C, c0, C, rv[it]);
      row_load<VEC>((const T*)a.dy + row * C, c0, C, ry[it]);
      if (DS_AHEAD && a.ds) row_load<VEC>((const T*)a.ds + row * C, c0, C, rs[it]);
    }
  };
  if (t < a.T) fetch(t);
  for (int parity = 0; t < a.T; t += step, parity ^= 1) {
    float v[ITEMS][8], dy[ITEMS][8];
    float sums[2] = {0.f, 0.f};
    Piece<T> cs[ITEMS];
#pragma unroll
    for (int it = 0; it < ITEMS; ++it) {
      row_open<VEC>(rv[it], (it * NT + tid) * 8, C, v[it]);
      row_open<VEC>(ry[it], (it * NT + tid) * 8, C, dy[it]);
      if (DS_AHEAD) cs[it] = rs[it];
      else if (a.ds) row_load<VEC>((const T*)a.ds + t * C, (it * NT + tid) * 8, C, cs[it]);
    }
    if (t + step < a.T) fetch(t + step);
#pragma unroll
    for (int it = 0; it < ITEMS; ++it) {
      float wi[8];
      w.get(it, wi, 0);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        sums[0] += v[it][e] * v[it][e];
        sums[1] += v[it][e] * (wi[e] * dy[it][e]);
      }
    }
    row_sum<WAVE, 2>(sums, red[parity]);
    float ms = uniform(sums[0] * inv_c + a.eps);
    float back1 = 1.f, back2 = 1.f;  // dx = ... 2^-k, as a product of two that are in range
    if (!in_range(ms) || !(fabsf(uniform(sums[1])) <= 3.4028235e38f)) {
      uint32_t top = 0;
#pragma unroll
      for (int it = 0; it < ITEMS; ++it)
#pragma unroll
        for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(v[it][e]) & 0x7fffffffu);
      int p;
      if (scale_of(row_umax<WAVE>(top, redm[parity]), a.eps, p)) {
        sums[0] = sums[1] = 0.f;
#pragma unroll
        for (int it = 0; it < ITEMS; ++it) {
          float wi[8];
          w.get(it, wi, 0);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            v[it][e] = __builtin_amdgcn_ldexpf(v[it][e], -p);
            sums[0] += v[it][e] * v[it][e];
            sums[1] += v[it][e] * (wi[e] * dy[it][e]);
          }
        }
        row_sum<WAVE, 2>(sums, red[parity]);
        ms = sums[0] * inv_c + __builtin_amdgcn_ldexpf(a.eps, -2 * p);
        back1 = __builtin_amdgcn_ldexpf(1.f, -(p / 2));
        back2 = __builtin_amdgcn_ldexpf(1.f, -(p - p / 2));
      }
    }
    const float rstd = rms_factor(ms), rstd_dx = rstd * back1;
    const float k = (sums[1] * rstd) * inv_c * rstd;
    if (ITEMS == 2) asm volatile("" ::: "memory");  // the weight is read again, not kept
#pragma unroll
    for (int it = 0; it < ITEMS; ++it) {
      float o[8], ds[8], wi[8], dwi[8];
      row_open<VEC>(cs[it], (it * NT + tid) * 8, C, ds);
      w.get(it, wi, 0);
      dw.get(it, dwi, 1);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        dwi[e] += dy[it][e] * (v[it][e] * rstd);
        o[e] = rstd_dx * ((wi[e] * dy[it][e] - v[it][e] * k) * back2) + (a.ds ? ds[e] : 0.f);
      }
      dw.put(it, dwi, 1);
      row_store<VEC>((T*)a.dx + t * C, (it * NT + tid) * 8, C, o);
    }
  }
  if (a.part == nullptr) return;
  float* p = a.part + (int64_t)blockIdx.x * C;
  float sum[ITEMS][8];
#pragma unroll
  for (int it = 0; it < ITEMS; ++it) dw.get(it, sum[it], 1);
  if constexpr (WAVE) {  // the waves' sums are added here: a fourth of the parts
    __shared__ __attribute__((aligned(16))) float add[WAVE_ROWS][512];
    store8(add[r.sub] + tid * 8, sum[0]);
    __syncthreads();
    for (uint32_t c = threadIdx.x; c < C; c += 64 * WAVE_ROWS) {
      float all = add[0][c];
#pragma unroll
      for (int i = 1; i < WAVE_ROWS; ++i) all += add[i][c];
      p[c] = all;
    }
    return;
  }
#pragma unroll
  for (int it = 0; it < ITEMS; ++it) {
    const uint32_t c0 = (it * NT + tid) * 8;
    if (VEC) {
      if (c0 < C) store8(p + c0, sum[it]);
    } else if (piece_count(c0, C) == 8) {
      store8_any(p + c0, sum[it]);
    } else {
      store8_tail(p + c0, piece_count(c0, C), sum[it]);
    }
  }
}

// out[c] = sum_p part[p][c]: 32 columns by 32 interleaved walks per workgroup, the
// walks added in order.
__global__ __launch_bounds__(1024) void column_sum_kernel(const float* __restrict__ part, int64_t P, int64_t C,
                                                          float* __restrict__ out) {
  __shared__ float s[32][33];
  const int cl = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + cl;
  float v = 0.f;
  if (c < C) {
#pragma unroll 4
    for (int64_t p = g; p < P; p += 32) v += part[p * C + c];
  }
  s[g][cl] = v;
  __syncthreads();
  if (g == 0 && c < C) {
    float r = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) r += s[i][cl];
    out[c] = r;
  }
}

// Launch shape of a pass over T rows of C channels: pieces per thread, threads, and
// the workgroups, bounded so that each keeps the weight in registers over several rows
// and reads ahead. Measured against each other, by events over changing inputs, at 8,192 x
// 4,096 with residual and e4m3 groups / 16,384 x 4 x 7,168: forward with two pieces a
// thread and 16,384 waves 42.8 / 248 us (8,192 waves 43.9 / 261; one piece, 6,144 waves
// 41.6 / 264, 16,384 waves 43.5 / 260). The backward keeps 256 CUs equally busy, with up to
// 16 waves each (bfloat16, 8,192 rows of 2,560 / 4,096 / 7,168 channels: 36 / 50 / 97 us;
// 4,096 waves in all, however they fall, 50 / 51 / 156; one workgroup each 49 / 49 / 98) and
// one piece a thread up to 8,192 channels.
struct RowShape {
  int items;
  bool wave;
  unsigned block, grid;
};

RowShape row_shape(int64_t T, int64_t C, bool bwd) {
  RowShape s;
  const int64_t pieces = (C + 7) / 8;
  s.wave = C <= 512;
  s.items = C <= 2048 || (bwd && C <= 8192) ? 1 : 2;
  s.block = s.wave ? 64 * WAVE_ROWS : (unsigned)((pieces + 64 * s.items - 1) / (64 * s.items) * 64);
  const int64_t need = s.wave ? (T + WAVE_ROWS - 1) / WAVE_ROWS : T;
  const int64_t waves = s.block / 64, most = bwd ? 256 * (waves < 16 ? 16 / waves : 1) : 16384 / waves;
  s.grid = (unsigned)(need < most ? need : most);
  return s;
}

template <typename T, int MODE, int ITEMS, bool WAVE>
void norm_go(bool vec, const RowShape& s, const NormArgs& a, hipStream_t st) {
  if (vec) hipLaunchKernelGGL((rms_norm_kernel<T, MODE, ITEMS, WAVE, true>), dim3(s.grid), dim3(s.block), 0, st, a);
  else hipLaunchKernelGGL((rms_norm_kernel<T, MODE, ITEMS, WAVE, false>), dim3(s.grid), dim3(s.block), 0, st, a);
}

template <typename T, int MODE>
void norm_by_width(bool vec, const NormArgs& a, hipStream_t st) {
  const RowShape s = row_shape(a.T, a.C, false);
  if (s.wave) norm_go<T, MODE, 1, true>(vec, s, a, st);
  else if (s.items == 1) norm_go<T, MODE, 1, false>(vec, s, a, st);
  else norm_go<T, MODE, 2, false>(vec, s, a, st);
}

template <typename T, int ITEMS, bool WAVE>
void norm_bwd_go(bool vec, const RowShape& s, const NormBwdArgs& a, hipStream_t st) {
  if (vec) hipLaunchKernelGGL((rms_norm_backward_kernel<T, ITEMS, WAVE, true>), dim3(s.grid), dim3(s.block), 0, st, a);
  else hipLaunchKernelGGL((rms_norm_backward_kernel<T, ITEMS, WAVE, false>), dim3(s.grid), dim3(s.block), 0, st, a);
}

template <typename T>
void norm_bwd_by_width(bool vec, const NormBwdArgs& a, hipStream_t st) {
  const RowShape s = row_shape(a.T, a.C, true);
  if (s.wave) norm_bwd_go<T, 1, true>(vec, s, a, st);
  else if (s.items == 1) norm_bwd_go<T, 1, false>(vec, s, a, st);
  else norm_bwd_go<T, 2, false>(vec, s, a, st);
}

}  // namespace

int64_t norm_backward_parts(int64_t T, int64_t C) {
  return row_shape(T, C, true).grid;
}

hipError_t launch_rms_norm(int dtype, int mode, bool vec, const NormArgs& a, hipStream_t st) {
  if (dtype == 0) {
    if (mode == 0) norm_by_width<float, 0>(vec, a, st);
    else if (mode == 1) norm_by_width<float, 1>(vec, a, st);
    else norm_by_width<float, 2>(vec, a, st);
  } else {
    if (mode == 0) norm_by_width<bf16_t, 0>(vec, a, st);
    else if (mode == 1) norm_by_width<bf16_t, 1>(vec, a, st);
    else norm_by_width<bf16_t, 2>(vec, a, st);
  }
  return hipGetLastError();
}

hipError_t launch_rms_norm_backward(int dtype, bool vec, const NormBwdArgs& a, float* dw, hipStream_t st) {
  if (a.T > 0 && dtype == 0) norm_bwd_by_width<float>(vec, a, st);
  else if (a.T > 0) norm_bwd_by_width<bf16_t>(vec, a, st);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || dw == nullptr) return e;
  hipLaunchKernelGGL(column_sum_kernel, dim3((unsigned)((a.C + 31) / 32)), dim3(1024), 0, st, a.part,
                     norm_backward_parts(a.T, a.C), a.C, dw);
  return hipGetLastError();
}

}  // namespace hc
