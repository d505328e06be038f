// Layer norm in front of a sublayer function, forward and backward.
//   v = x, x + residual, or the pre-read sum_i h_pre[i] X[i];
//   y = (v - mean) * w / sqrt(var + eps) + b, stored as the root-mean-square norm
//   (hc_norm.hip) stores its own.
// Each row is read once and stays in float32 registers. The variance is that of the
// deviations from the mean, never a difference of two large sums: one exchange over the
// row's threads for the mean, one for the deviations' sums; what rounding leaves in the
// mean is taken off with the scale, in one multiply-add an element.
//   Memory bounds the forward: 8,192 rows of 4,096 bfloat16 with residual, stored as e4m3
// groups, 44 us for 236 MB; the pre-read of 4 streams 67 us for 403 MB. In the backward
// (57 us for 268 MB) a row's two exchanges, and the threads that wait in them, cost as much.
// They were the larger part of both: sums by DPP and lane swaps instead of trips through
// LDS, and one LDS word a lane for the waves' sums instead of a loop over them, took the
// forward from 55 to 45 us, the backward from 69 to 57, and from 159 to 111 us at 7,168
// channels, where 14 waves share a row.
//   Wide rows, 4,096 of them: forward 5.0 TB/s up to 16,384 channels (bfloat16 99 us, float32 216), 3 to 4 at
// odd widths (9,001: 94 and 147 us); backward, whose 16 waves spill above 8,192 channels (8 registers in
// bfloat16, 24 in float32, 131 at odd widths), 4.1 and 4.7 TB/s at 8,192 (66 and 113 us), 3.6 and 3.0 at
// 16,384 (150 and 354), 2.5 and 2.1 at 9,001 (120 and 276).
#include "hc_norm_row.h"

namespace hc {

namespace {

// The sum over a wave's lanes, in every lane: within rows of 16 by DPP, the rows by lane swaps, with no
// trip through LDS (a row takes up to six sums one after the other).
__device__ __forceinline__ float lanes_sum(float v) {
  typedef uint32_t u2 __attribute__((ext_vector_type(2)));
  v = row16_sum(v);
  u2 p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
  p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(p[0]) + __uint_as_float(p[1]);
}

// Sums of NV values over one row's threads, the same in each; `red` is not used again before the
// row's threads have met another barrier.
template <bool WAVE, int NV>
__device__ __forceinline__ void sum_over_row(float (&v)[NV], float (*red)[16]) {
#pragma unroll
  for (int i = 0; i < NV; ++i) v[i] = lanes_sum(v[i]);
  if (WAVE) return;
  if ((threadIdx.x & 63) == 0)
#pragma unroll
    for (int i = 0; i < NV; ++i) red[i][threadIdx.x >> 6] = v[i];
  lds_barrier();
  const uint32_t w = threadIdx.x & 15;  // at most 16 waves
  const bool there = w < blockDim.x >> 6;
#pragma unroll
  for (int i = 0; i < NV; ++i) v[i] = row16_sum(there ? red[i][w] : 0.f);
}

// LDS of one row parity: two slots of up to NV sums, and the words of the row's extremes.
template <int NV>
struct RowRed {
  float sum[2][NV][16];
  uint32_t top[4][16];
};

// Turns a row's values v into their deviations from the mean, but for `rest`, and gives ms, the
// deviations' mean square + eps; of the values u that `up` gives (the backward's w dy) s[0] = sum u
// and s[1] = sum u (v - rest).
//   What rounding leaves in the mean is the deviations' own mean, `rest`, for the caller to take off.
//   Where the deviations are within 2^-15 of the mean, that rounding is no longer small
//   beside them: equal values are found by their bits (their square is 0), others are
//   centred a second time.
//   A row whose magnitudes add up to more than 2^40, whose products might leave float32's
//   range, or with an eps that is no floor to less than 1, so that even a last bit's
//   deviation squared stays a normal number, is taken relative to 2^k (see scale_of): k is
//   returned, 0 otherwise, and v and ms are those of the scaled row.
template <int ITEMS, bool WAVE, bool VEC, bool BWD, typename UP>
__device__ __forceinline__ int row_center(float (&v)[ITEMS][8], const RowThreads<WAVE>& r, uint32_t C, float inv_c,
                                          float eps, RowRed<BWD ? 4 : 2>& red, UP up, float& ms, float& rest, float (&s)[2]) {
  constexpr int NV = BWD ? 4 : 2;
  const auto inside = [&](int it, int e) { return (uint32_t)((it * r.nt + r.tid) * 8 + (VEC ? 0 : e)) < C; };
  float total[2];
  const auto add_up = [&]() {
    total[0] = total[1] = 0.f;
#pragma unroll
    for (int it = 0; it < ITEMS; ++it)
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (inside(it, e)) {
          total[0] += v[it][e];
          total[1] += fabsf(v[it][e]);
        }
    sum_over_row<WAVE, 2>(total, red.sum[0]);
  };
  add_up();
  int k = 0;
  const float all = uniform(total[1]);
  if (!(all <= 0x1p40f) || (all < 1.f && eps < 0x1p-80f)) {
    uint32_t top = 0;
#pragma unroll
    for (int it = 0; it < ITEMS; ++it)
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (inside(it, e)) top = max(top, __float_as_uint(v[it][e]) & 0x7fffffffu);
    if (scale_of(row_umax<WAVE>(top, red.top[0]), eps, k)) {
#pragma unroll
      for (int it = 0; it < ITEMS; ++it)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[it][e] = __builtin_amdgcn_ldexpf(v[it][e], -k);
      add_up();
    } else {
      k = 0;
    }
  }
  const float mean = uniform(total[0] * inv_c);
#pragma unroll
  for (int it = 0; it < ITEMS; ++it)
#pragma unroll
    for (int e = 0; e < 8; ++e) v[it][e] -= inside(it, e) ? mean : 0.f;  // 0 where there is no channel
  float q[NV];
  const auto sums = [&](int slot) {
#pragma unroll
    for (int i = 0; i < NV; ++i) q[i] = 0.f;
#pragma unroll
    for (int it = 0; it < ITEMS; ++it) {
      float u[8];
      if (BWD) up(it, u);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        q[0] += v[it][e];
        q[1] += v[it][e] * v[it][e];
        if (BWD) {
          q[NV - 2] += u[e];
          q[NV - 1] += u[e] * v[it][e];
        }
      }
    }
    sum_over_row<WAVE, NV>(q, red.sum[slot]);
    rest = uniform(q[0] * inv_c);
    ms = uniform(q[1] * inv_c - rest * rest);
  };
  sums(1);
  if (ms < 0x1p-30f * mean * mean) {
    uint32_t top = 0, low = 0;
#pragma unroll
    for (int it = 0; it < ITEMS; ++it)
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (inside(it, e)) {
          top = max(top, __float_as_uint(v[it][e]));
          low = max(low, ~__float_as_uint(v[it][e]));
        }
    top = row_umax<WAVE>(top, red.top[1]);
    low = row_umax<WAVE>(low, red.top[2]);
    const float off = rest;
#pragma unroll
    for (int it = 0; it < ITEMS; ++it)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[it][e] = top == ~low || !inside(it, e) ? 0.f : v[it][e] - off;
    sums(0);
    ms = fmaxf(ms, 0.f);
  }
  if (BWD) {
    s[0] = q[NV - 2];
    s[1] = q[NV - 1] - rest * s[0];
  }
  ms += k == 0 ? eps : __builtin_amdgcn_ldexpf(eps, -2 * k);
  return k;
}

// Modes and reading ahead as in the root-mean-square norm.
template <typename T, int MODE, int ITEMS, bool WAVE, bool VEC>
__global__ __launch_bounds__(WAVE ? 64 * WAVE_ROWS : 1024) void layer_norm_kernel(NormArgs a, const float* bias) {
  constexpr int NS = MODE == 1 ? 2 : 1;  // arrays of a row
  __shared__ RowRed<2> red[2];
  const RowThreads<WAVE> r;
  const uint32_t tid = r.tid, NT = r.nt, C = (uint32_t)a.C;
  const int64_t step = (int64_t)gridDim.x * r.rows();
  const float inv_c = 1.0f / (float)C;
  // kept in registers over the rows with one piece a thread; two would spill and are read
  // again for each row
  float w[8], b[8];
  if (ITEMS == 1) {
    load_piece<VEC>(a.w, C, tid * 8, 1.f, w);
    load_piece<VEC>(bias, C, tid * 8, 0.f, b);
  }
  const auto weight = [&](int it, float* wi, float* bi) {
    if (ITEMS == 1) {
      __builtin_memcpy(wi, w, sizeof(w));
      __builtin_memcpy(bi, b, sizeof(b));
    } else {
      load_piece<VEC>(a.w, C, (it * NT + tid) * 8, 1.f, wi);
      load_piece<VEC>(bias, C, (it * NT + tid) * 8, 0.f, bi);
    }
  };
  int64_t t = (int64_t)blockIdx.x * r.rows() + r.sub;
  Piece<T> raw[NS][ITEMS];
  const auto fetch = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < NS; ++i)
#pragma unroll
      for (int it = 0; it < ITEMS; ++it)
        row_load<VEC>((const T*)(i == 0 ? a.x : a.res) + row * C, (it * NT + tid) * 8, C, raw[i][it]);
  };
  if (MODE != 2 && t < a.T) fetch(t);
  for (int parity = 0; t < a.T; t += step, parity ^= 1) {
    float v[ITEMS][8];
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
      for (int i = 0; i < NS; ++i)
#pragma unroll
        for (int it = 0; it < ITEMS; ++it) {
          float xi[8];
          row_open<VEC>(raw[i][it], (it * NT + tid) * 8, C, xi);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[it][e] = i == 0 ? xi[e] : v[it][e] + xi[e];
        }
      if (t + step < a.T) fetch(t + step);
    }
    if (MODE != 0 && a.s) {
#pragma unroll
      for (int it = 0; it < ITEMS; ++it) row_store<VEC>((T*)a.s + t * C, (it * NT + tid) * 8, C, v[it]);
    }
    float unused[2], ms, rest;
    row_center<ITEMS, WAVE, VEC, false>(v, r, C, inv_c, a.eps, red[parity], [](int, float*) {}, ms, rest, unused);
    const float rstd = rms_factor(ms), off = -rest * rstd;
#pragma unroll
    for (int it = 0; it < ITEMS; ++it) {
      float wi[8], bi[8];
      weight(it, wi, bi);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[it][e] = fmaf(fmaf(v[it][e], rstd, off), wi[e], bi[e]);
    }
    row_write<T, ITEMS, WAVE, VEC>(a, t, NT, tid, v, red[parity].top[3]);
  }
}

// dx = rstd (u - mean(u) - n mean(u n)) + ds with u = w dy and n = (v - mean) rstd, and
// this workgroup's parts of dw = sum_t dy n and db = sum_t dy, kept over its rows as in the
// root-mean-square norm's backward: in registers with one piece a thread; with two the sums
// lie in LDS, and the weight is read again for each row.
template <typename T, int ITEMS, bool WAVE, bool VEC>
__global__ __launch_bounds__(WAVE ? 64 * WAVE_ROWS : 1024) void layer_norm_backward_kernel(NormBwdArgs a) {
  __shared__ RowRed<4> red[2];
  const RowThreads<WAVE> r;
  const uint32_t tid = r.tid, NT = r.nt, C = (uint32_t)a.C;
  const float inv_c = 1.0f / (float)C;
  PieceSums<ITEMS> dw, db;
  float w[8];
  if (ITEMS == 1) load_piece<VEC>(a.w, C, tid * 8, 1.f, w);
  const float zero[8] = {};
#pragma unroll
  for (int it = 0; it < ITEMS; ++it) {
    dw.put(it, zero, 0);
    db.put(it, zero, 1);
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
    float v[ITEMS][8], dy[ITEMS][8], ms, s[2];
    Piece<T> cs[ITEMS];
#pragma unroll
    for (int it = 0; it < ITEMS; ++it) {
      row_open<VEC>(rv[it], (it * NT + tid) * 8, C, v[it]);
      row_open<VEC>(ry[it], (it * NT + tid) * 8, C, dy[it]);
      if (DS_AHEAD) cs[it] = rs[it];
      else if (a.ds) row_load<VEC>((const T*)a.ds + t * C, (it * NT + tid) * 8, C, cs[it]);
    }
    if (t + step < a.T) fetch(t + step);
    const auto up = [&](int it, float* u) {
      float wi[8];
      if (ITEMS == 1) __builtin_memcpy(wi, w, sizeof(wi));
      else load_piece<VEC>(a.w, C, (it * NT + tid) * 8, 1.f, wi);
#pragma unroll
      for (int e = 0; e < 8; ++e) u[e] = wi[e] * dy[it][e];
    };
    float rest;
    const int p = row_center<ITEMS, WAVE, VEC, true>(v, r, C, inv_c, a.eps, red[parity], up, ms, rest, s);
    const float rstd = rms_factor(ms), off = -rest * rstd;
    const float k = (s[1] * rstd) * inv_c * rstd, mean_u = s[0] * inv_c;
    // dx = rstd (u - mean_u - (v - rest) k) 2^-p + ds
    const float by_v = -rstd * k, fixed = -rstd * (mean_u - rest * k);
    const float back1 = __builtin_amdgcn_ldexpf(1.f, -(p / 2)), back2 = __builtin_amdgcn_ldexpf(1.f, -(p - p / 2));
#pragma unroll
    for (int it = 0; it < ITEMS; ++it) {
      float o[8], ds[8], u[8], dwi[8], dbi[8];
      row_open<VEC>(cs[it], (it * NT + tid) * 8, C, ds);
      up(it, u);
      dw.get(it, dwi, 0);
      db.get(it, dbi, 1);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        dwi[e] = fmaf(dy[it][e], fmaf(v[it][e], rstd, off), dwi[e]);
        dbi[e] += dy[it][e];
        if (!a.ds) ds[e] = 0.f;
      }
      if (p == 0) {
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = fmaf(u[e], rstd, fmaf(v[it][e], by_v, ds[e] + fixed));
      } else {  // 2^-p as a product of two that are in range, the second inside
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = (rstd * back1) * ((u[e] - mean_u - (v[it][e] - rest) * k) * back2) + ds[e];
      }
      dw.put(it, dwi, 0);
      db.put(it, dbi, 1);
      row_store<VEC>((T*)a.dx + t * C, (it * NT + tid) * 8, C, o);
    }
  }
  if (a.part == nullptr) return;
  float* pw = a.part + (int64_t)blockIdx.x * C;
  float* pb = a.part + ((int64_t)gridDim.x + blockIdx.x) * C;
  float sw[ITEMS][8], sb[ITEMS][8];
#pragma unroll
  for (int it = 0; it < ITEMS; ++it) {
    dw.get(it, sw[it], 0);
    db.get(it, sb[it], 1);
  }
  if constexpr (WAVE) {  // the waves' sums are added here: a fourth of the parts
    __shared__ __attribute__((aligned(16))) float add[2][WAVE_ROWS][512];
    store8(add[0][r.sub] + tid * 8, sw[0]);
    store8(add[1][r.sub] + tid * 8, sb[0]);
    __syncthreads();
    for (uint32_t c = threadIdx.x; c < C; c += 64 * WAVE_ROWS) {
      float all = add[0][0][c], allb = add[1][0][c];
#pragma unroll
      for (int i = 1; i < WAVE_ROWS; ++i) {
        all += add[0][i][c];
        allb += add[1][i][c];
      }
      pw[c] = all;
      pb[c] = allb;
    }
    return;
  }
#pragma unroll
  for (int it = 0; it < ITEMS; ++it) {
    const uint32_t c0 = (it * NT + tid) * 8;
    if (VEC) {
      if (c0 < C) {
        store8(pw + c0, sw[it]);
        store8(pb + c0, sb[it]);
      }
    } else if (piece_count(c0, C) == 8) {
      store8_any(pw + c0, sw[it]);
      store8_any(pb + c0, sb[it]);
    } else {
      store8_tail(pw + c0, piece_count(c0, C), sw[it]);
      store8_tail(pb + c0, piece_count(c0, C), sb[it]);
    }
  }
}

// Up to this many channels a thread of the forward has one piece and keeps weight and bias in
// registers: 4,096 channels 47 us against 56 with two pieces that read both again, 7,168
// channels 91 against 102 with one piece and 14 waves in step (bfloat16; 6,000 channels of
// float32 84 against 78).
constexpr int64_t ONE_PIECE = 4096;

template <typename T, int MODE, int ITEMS, bool WAVE>
void norm_go(bool vec, const RowShape& s, const NormArgs& a, const float* b, hipStream_t st) {
  if (vec) hipLaunchKernelGGL((layer_norm_kernel<T, MODE, ITEMS, WAVE, true>), dim3(s.grid), dim3(s.block), 0, st, a, b);
  else hipLaunchKernelGGL((layer_norm_kernel<T, MODE, ITEMS, WAVE, false>), dim3(s.grid), dim3(s.block), 0, st, a, b);
}

template <typename T, int MODE>
void norm_by_width(bool vec, const NormArgs& a, const float* b, hipStream_t st) {
  const RowShape s = row_shape(a.T, a.C, false, ONE_PIECE);
  if (s.wave) norm_go<T, MODE, 1, true>(vec, s, a, b, st);
  else if (s.items == 1) norm_go<T, MODE, 1, false>(vec, s, a, b, st);
  else norm_go<T, MODE, 2, false>(vec, s, a, b, st);
}

template <typename T, int ITEMS, bool WAVE>
void norm_bwd_go(bool vec, const RowShape& s, const NormBwdArgs& a, hipStream_t st) {
  if (vec) hipLaunchKernelGGL((layer_norm_backward_kernel<T, ITEMS, WAVE, true>), dim3(s.grid), dim3(s.block), 0, st, a);
  else hipLaunchKernelGGL((layer_norm_backward_kernel<T, ITEMS, WAVE, false>), dim3(s.grid), dim3(s.block), 0, st, a);
}

template <typename T>
void norm_bwd_by_width(bool vec, const NormBwdArgs& a, hipStream_t st) {
  const RowShape s = row_shape(a.T, a.C, true);
  if (s.wave) norm_bwd_go<T, 1, true>(vec, s, a, st);
  else if (s.items == 1) norm_bwd_go<T, 1, false>(vec, s, a, st);
  else norm_bwd_go<T, 2, false>(vec, s, a, st);
}

}  // namespace

hipError_t launch_layer_norm(int dtype, int mode, bool vec, const NormArgs& a, const float* b, hipStream_t st) {
  if (dtype == 0) {
    if (mode == 0) norm_by_width<float, 0>(vec, a, b, st);
    else if (mode == 1) norm_by_width<float, 1>(vec, a, b, st);
    else norm_by_width<float, 2>(vec, a, b, st);
  } else {
    if (mode == 0) norm_by_width<bf16_t, 0>(vec, a, b, st);
    else if (mode == 1) norm_by_width<bf16_t, 1>(vec, a, b, st);
    else norm_by_width<bf16_t, 2>(vec, a, b, st);
  }
  return hipGetLastError();
}

hipError_t launch_layer_norm_backward(int dtype, bool vec, const NormBwdArgs& a, float* dw, float* db, hipStream_t st) {
  if (a.T > 0 && dtype == 0) norm_bwd_by_width<float>(vec, a, st);
  else if (a.T > 0) norm_bwd_by_width<bf16_t>(vec, a, st);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || (dw == nullptr && db == nullptr)) return e;
  return launch_column_sums(a.part, norm_backward_parts(a.T, a.C), a.C, dw, db, st);
}

}  // namespace hc
