// Root-mean-square norm in front of a sublayer function, forward and backward.
//   v = x, x + residual, or the pre-read sum_i h_pre[i] X[i];
//   y = v * w / sqrt(mean_c v^2 + eps), stored in the stream dtype or as 8-bit
//   codes with a scale per row or per group of 32, 64 or 128 channels.
// Each row is read once and stays in float32 registers between the sum of squares
// and the outputs, so the passes are bound by HBM traffic. Per call: 5.8 TB/s for 8,192 x
// 4,096 bfloat16 with residual and e4m3 output (40.5 us), 5.7 for the pre-read form of
// 16,384 x 4 x 7,168 (247 us), 5.5 for the backward of 8,191 x 4,096 (49 us, 4 of them the
// sum of dw's parts). Small calls are bound by the launch (16 x 4,096: 5 us).
#include "hc_norm_row.h"

namespace hc {

namespace {

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
    row_write<T, ITEMS, WAVE, VEC>(a, t, NT, tid, v, redm[parity]);
  }
}

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
// walks added in order. One array of parts for each row of the grid.
__global__ __launch_bounds__(1024) void column_sum_kernel(const float* __restrict__ parts, int64_t P, int64_t C,
                                                          float* __restrict__ out0, float* __restrict__ out1) {
  const float* part = parts + blockIdx.y * P * C;
  float* out = blockIdx.y ? out1 : out0;
  if (out == nullptr) return;
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
  return launch_column_sums(a.part, norm_backward_parts(a.T, a.C), a.C, dw, nullptr, st);
}

hipError_t launch_column_sums(const float* parts, int64_t P, int64_t C, float* out0, float* out1, hipStream_t st) {
  hipLaunchKernelGGL(column_sum_kernel, dim3((unsigned)((C + 31) / 32), out1 ? 2 : 1), dim3(1024), 0, st, parts, P, C,
                     out0, out1);
  return hipGetLastError();
}

}  // namespace hc
