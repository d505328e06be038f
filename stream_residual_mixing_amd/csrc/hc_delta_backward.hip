// Gated delta rule, backward. With the forward's chunk (hc_delta.hip), d = scale dO and N the gradient
// of the state behind the chunk:
//   dX = P^T d + exp(G_end - G) K N,   W = T^T (beta dX) = dV,
//   dM = exp(G_end) N + (exp(G) Q)^T d - (exp(G) K)^T W   (the gradient of the state before it),
//   B = (d X^T) exp(G_i - G_j) (j <= i),   A = -(W X^T) exp(G_i - G_j) (j < i),
//   dQ = exp(G) d M^T + B K,
//   dK = [-exp(G) W M^T + A K] + [exp(G_end - G) X N^T + B^T Q + A^T K]   (as read, as written),
//   dbeta_j = Z_j . dX_j - sum_i exp(G_i - G_j) (k_i . k_j) (W_i . Z_j),
//   dG = q . dq + k . dk_read - k . dk_written, and at the chunk's end
//        sum_j k_j . (X N^T exp(G_end - G))_j + exp(G_end) <M, N>;  dg_t = sum_{i >= t} dG_i.
// The forward's walk is run again and keeps every chunk's M and Z; a second walk from the end back
// keeps N and W and writes dV; then every chunk forms the rest by itself, all value heads of a key
// head in one workgroup, so that dQ and dK are summed in registers and in a fixed order.
#include "hc_delta_device.h"

namespace hc {

namespace {

template <int KP, int NP>
struct BackLds {
  char k[NP][Tokens<KP>::PART];         // keys: rows in row_of's order, then transposed
  char q[NP][KP * Tokens<KP>::COL];     // queries transposed
  char rec[REC_BWD - REC_DEC];
};

template <typename T, int KP, int NT, bool VEC>
__global__ __launch_bounds__(256) void delta_back_kernel(DeltaArgs a) {
  constexpr int NP = Stream<T>::NP, KB = KP / 32, KT = KP / 16;
  constexpr int PIECES = KP / 8, ITEMS = 32 * PIECES / 256;
  constexpr int USED = REC_BWD - REC_DEC, RR = (USED + 4095) / 4096;
  constexpr int PT = REC_P - REC_DEC, TT = REC_TT - REC_DEC;
  extern __shared__ __attribute__((aligned(16))) char lds_raw[];
  typedef BackLds<KP, NP> Lds;
  static_assert(sizeof(Lds) <= 160 * 1024, "LDS of a CU");
  Lds& lds = *reinterpret_cast<Lds*>(lds_raw);
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, n = lane & 15, g = lane >> 4;
  const int64_t groups = (a.Dv + 64 * NT - 1) / (64 * NT);
  const int64_t bh = blockIdx.x / groups, b = bh / a.Hv, hv = bh % a.Hv, hk = hv / (a.Hv / a.Hk);
  const int Dk = (int)a.Dk;
  const int col = (int)(blockIdx.x % groups) * 64 * NT + 16 * NT * w + NT * n, have = max(0, min(NT, (int)a.Dv - col));
  const int64_t len = length_of(a.lengths, b, a.S), chunks = (len + CH - 1) / CH;
  const int64_t qs = a.Hk * a.Dk, vs = a.Hv * a.Dv;
  const T* qp = (const T*)a.q + b * a.S * qs + hk * a.Dk;
  const T* kp = (const T*)a.k + b * a.S * qs + hk * a.Dk;
  const T* dp = (const T*)a.d_o + b * a.S * vs + hv * a.Dv + col;
  T* dvp = (T*)a.dv + b * a.S * vs + hv * a.Dv + col;
  const char* rec = (const char*)a.rec + bh * a.NC * REC_BWD + REC_DEC;

  f4_t D[KT][NT];
  {
    const float* s1 = a.dlast ? a.dlast + bh * a.Dk * a.Dv + col : nullptr;
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = row_of(t, 4 * g + r);
        const Cols<NT> c = load_cols<NT, VEC>(s1 + (int64_t)row * a.Dv, s1 && row < Dk ? have : 0);
#pragma unroll
        for (int h = 0; h < NT; ++h) D[t][h][r] = c.v[h];
      }
  }
  {  // nothing reaches the tokens behind the sequence's length
    Cols<NT> zero;
#pragma unroll
    for (int h = 0; h < NT; ++h) zero.v[h] = 0.f;
    for (int64_t t = len + g; t < a.S; t += 4) store_cols<NT, VEC>(dvp + t * vs, have, zero);
  }

  Raw8<T> kr[ITEMS][2], qr[ITEMS][2];
  u4_t rr[RR];
  Cols<NT> dr[4][4];
  const auto fetch = [&](int64_t c) {
    const int64_t t0 = c * CH;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int x = i * 256 + tid, piece = x % PIECES, pair = x / PIECES;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int64_t t = t0 + 2 * pair + j;
        const int cnt = t < len ? max(0, min(8, Dk - 8 * piece)) : 0;
        kr[i][j] = load_raw8<VEC>(kp + t * qs + 8 * piece, cnt);
        qr[i][j] = load_raw8<VEC>(qp + t * qs + 8 * piece, cnt);
      }
    }
#pragma unroll
    for (int i = 0; i < RR; ++i)
      if (i * 4096 + tid * 16 < USED) rr[i] = *reinterpret_cast<const u4_t*>(rec + c * REC_BWD + i * 4096 + tid * 16);
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int64_t tok = t0 + row_of(t, 4 * g + r);
        dr[t][r] = load_cols<NT, VEC>(dp + tok * vs, tok < len ? have : 0);
      }
  };
  if (chunks > 0) fetch(chunks - 1);
  for (int64_t c = chunks - 1; c >= 0; --c) {
    Op<NP> ko[ITEMS][2];
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int x = i * 256 + tid, piece = x % PIECES, pair = x / PIECES;
      Op<NP> qo[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        ko[i][j] = kr[i][j].op();
        qo[j] = qr[i][j].op();
#pragma unroll
        for (int p = 0; p < NP; ++p)
          *reinterpret_cast<bf8_t*>(lds.k[p] + Tokens<KP>::row_at(place_of(2 * pair + j), 16 * piece)) = ko[i][j].p[p];
      }
#pragma unroll
      for (int p = 0; p < NP; ++p) store_transposed<KP>(lds.q[p], pair, piece, qo[0].p[p], qo[1].p[p]);
    }
#pragma unroll
    for (int i = 0; i < RR; ++i)
      if (i * 4096 + tid * 16 < USED) *reinterpret_cast<u4_t*>(lds.rec + i * 4096 + tid * 16) = rr[i];
    Cols<NT> d[4][4];
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) d[t][r] = dr[t][r];
    if (col < a.VP) {
      bf16_t* keep = (bf16_t*)a.dstates + (bh * a.NC + c) * 2 * KP * a.VP + col;
#pragma unroll
      for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          Cols<NT> y;
#pragma unroll
          for (int h = 0; h < NT; ++h) y.v[h] = D[t][h][r];
          store_parts<NT>(keep + row_of(t, 4 * g + r) * a.VP, KP * a.VP, y);
        }
    }
    __syncthreads();

    f4_t x[4][NT];  // K N
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int h = 0; h < NT; ++h) x[t][h] = f4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      Split sf[NT];
#pragma unroll
      for (int h = 0; h < NT; ++h) sf[h] = split(D[2 * kb][h], D[2 * kb + 1][h]);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        Op<NP> ka;
#pragma unroll
        for (int p = 0; p < NP; ++p)
          ka.p[p] = *reinterpret_cast<const bf8_t*>(lds.k[p] + Tokens<KP>::row_at(16 * t + n, 64 * kb + 16 * g));
#pragma unroll
        for (int h = 0; h < NT; ++h) x[t][h] = mma(ka, sf[h], x[t][h]);
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int it = i * 256 + tid, piece = it % PIECES, pair = it / PIECES;
#pragma unroll
      for (int p = 0; p < NP; ++p) store_transposed<KP>(lds.k[p], pair, piece, ko[i][0].p[p], ko[i][1].p[p]);
    }
    if (c > 0) fetch(c - 1);

    const float* dec = (const float*)lds.rec;
    // beta dX, dX = scale P^T dO + exp(G_end - G) K N
#pragma unroll
    for (int h = 0; h < NT; ++h) {
      Op<NP> df[2];
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = d[2 * kb + (e >> 2)][e & 3].v[h];
        if (NP == 1) {
          df[kb].p[0] = as_bf8(pack8(v));  // exact: they are bfloat16
        } else {
          const Split s = split(v);
          df[kb].p[0] = s.hi;
          df[kb].p[NP - 1] = s.lo;
        }
      }
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        f4_t p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kb = t >> 1; kb < 2; ++kb) p = mma(load_tile(lds.rec + PT, tri_t(t, kb), lane), df[kb], p);
        const f4_t to_end = *reinterpret_cast<const f4_t*>(dec + DEC_TO_END + row_of(t, 4 * g));
        const f4_t beta = *reinterpret_cast<const f4_t*>(dec + DEC_BETA + row_of(t, 4 * g));
        x[t][h] = beta * (a.scale * p + to_end * x[t][h]);
      }
    }
    // W = T^T (beta dX)
    {
      Split xf[2][NT];
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int h = 0; h < NT; ++h) xf[kb][h] = split(x[2 * kb][h], x[2 * kb + 1][h]);
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int h = 0; h < NT; ++h) x[t][h] = f4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int kb = t >> 1; kb < 2; ++kb) {
          const Split ta = load_tile(lds.rec + TT, tri_t(t, kb), lane);
#pragma unroll
          for (int h = 0; h < NT; ++h) x[t][h] = mma(ta, xf[kb][h], x[t][h]);
        }
    }
    {
      bf16_t* keep = (bf16_t*)a.w + (bh * a.NC + c) * 2 * CH * a.VP + col;
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = row_of(t, 4 * g + r);
          Cols<NT> y;
#pragma unroll
          for (int h = 0; h < NT; ++h) y.v[h] = x[t][h][r];
          const int64_t tok = c * CH + row;
          store_cols<NT, VEC>(dvp + tok * vs, tok < len ? have : 0, y);
          if (col < a.VP) store_parts<NT>(keep + row * a.VP, CH * a.VP, y);
        }
    }
    // the gradient of the state before the chunk
    Split df[2][NT], wf[2][NT];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const f4_t ahead = *reinterpret_cast<const f4_t*>(dec + DEC_AHEAD + row_of(t, 4 * g));
#pragma unroll
      for (int h = 0; h < NT; ++h) {
        x[t][h] *= -ahead;
#pragma unroll
        for (int r = 0; r < 4; ++r) d[t][r].v[h] *= a.scale * ahead[r];
      }
    }
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int h = 0; h < NT; ++h) {
        wf[kb][h] = split(x[2 * kb][h], x[2 * kb + 1][h]);
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = d[2 * kb + (e >> 2)][e & 3].v[h];
        df[kb][h] = split(v);
      }
    const float whole = dec[DEC_AHEAD + CH - 1];
    __syncthreads();
#pragma unroll
    for (int t = 0; t < KT; ++t) {
#pragma unroll
      for (int h = 0; h < NT; ++h) D[t][h] *= whole;
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        Op<NP> ka, qa;
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          const int at = Tokens<KP>::col_at(16 * t + n, 64 * kb + 16 * g);
          ka.p[p] = *reinterpret_cast<const bf8_t*>(lds.k[p] + at);
          qa.p[p] = *reinterpret_cast<const bf8_t*>(lds.q[p] + at);
        }
#pragma unroll
        for (int h = 0; h < NT; ++h) {
          D[t][h] = mma(qa, df[kb][h], D[t][h]);
          D[t][h] = mma(ka, wf[kb][h], D[t][h]);
        }
      }
    }
    __syncthreads();
  }
  if (a.dstate0) {
    float* s0 = a.dstate0 + bh * a.Dk * a.Dv + col;
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = row_of(t, 4 * g + r);
        Cols<NT> y;
#pragma unroll
        for (int h = 0; h < NT; ++h) y.v[h] = D[t][h][r];
        store_cols<NT, VEC>(s0 + (int64_t)row * a.Dv, row < Dk ? have : 0, y);
      }
  }
}

// ------------------------------------------------------------- each chunk by itself

template <int KP, int NP>
struct GradLds {
  char k[NP][KP * Tokens<KP>::COL];  // transposed
  char q[NP][KP * Tokens<KP>::COL];
  double G[CH];
  float beta[CH], dG[CH], end[4];
};

template <bool VEC>
__device__ __forceinline__ void store8_some(bf16_t* p, int cnt, const float v[8]) {
  if (VEC) {
    if (cnt > 0) *reinterpret_cast<u4_t*>(p) = pack8(v);
  } else {
    store8_tail(p, cnt, v);
  }
}

template <bool VEC>
__device__ __forceinline__ void store8_some(float* p, int cnt, const float v[8]) {
  if (VEC) {
    if (cnt > 0) store8(p, v);
  } else {
    store8_tail(p, cnt, v);
  }
}

// A row's 32 values from k0 + 8 g of a kept array in two parts.
__device__ __forceinline__ Split kept_op(const bf16_t* p, int64_t lo) {
  return {*reinterpret_cast<const bf8_t*>(p), *reinterpret_cast<const bf8_t*>(p + lo)};
}

__device__ __forceinline__ float sum_groups(float v) {  // over the four lanes of a token
  v += __shfl_xor(v, 16, 64);
  return v + __shfl_xor(v, 32, 64);
}

// SHARED: several value heads read a key head.
template <typename T, int KP, bool VEC, bool SHARED>
__global__ __launch_bounds__(256) void delta_grad_kernel(DeltaArgs a) {
  constexpr int NP = Stream<T>::NP, KB = KP / 32, KT = KP / 16;
  constexpr int PIECES = KP / 8, ITEMS = 32 * PIECES / 256;
  extern __shared__ __attribute__((aligned(16))) char lds_raw[];
  typedef GradLds<KP, NP> Lds;
  static_assert(sizeof(Lds) <= 160 * 1024, "LDS of a CU");
  Lds& lds = *reinterpret_cast<Lds*>(lds_raw);
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, n = lane & 15, g = lane >> 4;
  const int64_t NC = a.NC, chunk = blockIdx.x % NC, bh = blockIdx.x / NC, b = bh / a.Hk, hk = bh % a.Hk;
  const int64_t t0 = chunk * CH, tokens = length_of(a.lengths, b, a.S) - t0, rows = a.S - t0;
  const int Dk = (int)a.Dk, Dv = (int)a.Dv, VP = (int)a.VP;
  const int64_t qs = a.Hk * a.Dk, vs = a.Hv * a.Dv;
  const int64_t q0 = (b * a.S + t0) * qs + hk * a.Dk;
  const T* q = (const T*)a.q + q0;
  const T* k = (const T*)a.k + q0;
  const int tok = 16 * w + n, per = (int)(a.Hv / a.Hk);

  f4_t dqt[KT], dkt[KT];
#pragma unroll
  for (int t = 0; t < KT; ++t) dqt[t] = dkt[t] = f4_t{0.f, 0.f, 0.f, 0.f};
  f4_t kk[4], qk[4];  // rows: the other token in row_of's order, by k_n
  if (tokens > 0) {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int x = i * 256 + tid, piece = x % PIECES, pair = x / PIECES;
      const Op<NP> k0 = token_op<T, VEC>(k, qs, tokens, 2 * pair, 8 * piece, Dk);
      const Op<NP> k1 = token_op<T, VEC>(k, qs, tokens, 2 * pair + 1, 8 * piece, Dk);
      const Op<NP> q0 = token_op<T, VEC>(q, qs, tokens, 2 * pair, 8 * piece, Dk);
      const Op<NP> q1 = token_op<T, VEC>(q, qs, tokens, 2 * pair + 1, 8 * piece, Dk);
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        store_transposed<KP>(lds.k[p], pair, piece, k0.p[p], k1.p[p]);
        store_transposed<KP>(lds.q[p], pair, piece, q0.p[p], q1.p[p]);
      }
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) kk[t] = qk[t] = f4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      const int k0 = 32 * kb + 8 * g;
      const Op<NP> kn = token_op<T, VEC>(k, qs, tokens, tok, k0, Dk);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        if ((t >> 1) < (w >> 1)) continue;
        kk[t] = mma(token_op<T, VEC>(k, qs, tokens, row_of(t, n), k0, Dk), kn, kk[t]);
        qk[t] = mma(token_op<T, VEC>(q, qs, tokens, row_of(t, n), k0, Dk), kn, qk[t]);
      }
    }
  }
  for (int hi = 0; hi < per; ++hi) {
    const int64_t hv = hk * per + hi, at = (b * a.Hv + hv) * NC + chunk;
    const int64_t gat = (b * a.S + t0) * a.Hv + hv;
    if (tokens <= 0) {
      if (tid < CH && tid < rows) a.dg[gat + tid * a.Hv] = a.dbeta[gat + tid * a.Hv] = 0.f;
      continue;
    }
    if (tid < CH) {
      const bool on = tid < tokens;
      lds.G[tid] = running_sum(on ? clamp_decay(a.g[gat + tid * a.Hv]) : 0.0, tid);
      lds.beta[tid] = on ? a.beta[gat + tid * a.Hv] : 0.f;
    }
    __syncthreads();
    const double Gn = lds.G[tok], Gend = lds.G[CH - 1];
    const float beta_n = lds.beta[tok], ahead = expf((float)Gn), to_end = expf((float)(Gend - Gn));

    const T* dop = (const T*)a.d_o + (b * a.S + t0) * vs + hv * a.Dv;
    const bf16_t* zp = (const bf16_t*)a.z + at * 2 * CH * VP;
    const bf16_t* wp = (const bf16_t*)a.w + at * 2 * CH * VP;
    const bf16_t* mp = (const bf16_t*)a.states + at * 2 * KP * VP;
    const bf16_t* np = (const bf16_t*)a.dstates + at * 2 * KP * VP;
    const int vlo = CH * VP, slo = KP * VP;
    // rows j, lane i: Z_j . dO_i and Z_j . W_i; rows i, lane j: dO_i . Z_j and W_i . Z_j
    f4_t zd[4], zw[4], dz[4], wz[4];
    f4_t dq[KT], read[KT], early[KT];
    float mn = 0.f;
#pragma unroll
    for (int t = 0; t < 4; ++t) zd[t] = zw[t] = dz[t] = wz[t] = f4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int t = 0; t < KT; ++t) dq[t] = read[t] = early[t] = f4_t{0.f, 0.f, 0.f, 0.f};
    for (int v0 = 8 * g; v0 < VP; v0 += 32) {
      const Op<NP> dn = token_op<T, VEC>(dop, vs, tokens, tok, v0, Dv);
      const Split zn = kept_op(zp + tok * VP + v0, vlo), wn = kept_op(wp + tok * VP + v0, vlo);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int row = row_of(t, n);
        if ((t >> 1) <= (w >> 1)) {
          const Split zr = kept_op(zp + row * VP + v0, vlo);
          zd[t] = mma(zr, dn, zd[t]);
          zw[t] = mma(zr, wn, zw[t]);
        }
        if ((t >> 1) >= (w >> 1)) {
          dz[t] = mma(token_op<T, VEC>(dop, vs, tokens, row, v0, Dv), zn, dz[t]);
          wz[t] = mma(kept_op(wp + row * VP + v0, vlo), zn, wz[t]);
        }
      }
#pragma unroll
      for (int t = 0; t < KT; ++t) {
        const int row = row_of(t, n);
        const Split m = kept_op(mp + row * VP + v0, slo), nn = kept_op(np + row * VP + v0, slo);
        dq[t] = mma(m, dn, dq[t]);
        read[t] = mma(m, wn, read[t]);
        early[t] = mma(nn, zn, early[t]);
        if ((t & 3) == w)
#pragma unroll
          for (int e = 0; e < 8; ++e) mn += ((float)m.hi[e] + (float)m.lo[e]) * ((float)nn.hi[e] + (float)nn.lo[e]);
      }
    }
    // what each pair of tokens passes on
    float db = 0.f;
    Split bq[2], ar[2], bk[2], aw[2];  // operands: B^T and A^T (lane i), B and A (lane j)
    {
      float vb[2][8], va[2][8];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const f4_t beta = *reinterpret_cast<const f4_t*>(lds.beta + row_of(t, 4 * g));
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int j = row_of(t, 4 * g + r);
          const float d = j <= tok ? beta[r] * expf((float)(Gn - lds.G[j])) : 0.f;
          vb[t >> 1][4 * (t & 1) + r] = j <= tok ? a.scale * d * zd[t][r] : 0.f;
          va[t >> 1][4 * (t & 1) + r] = j < tok ? -d * zw[t][r] : 0.f;
        }
      }
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) bq[kb] = split(vb[kb]), ar[kb] = split(va[kb]);
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int i = row_of(t, 4 * g + r);
          const float d = i >= tok ? expf((float)(lds.G[i] - Gn)) : 0.f;
          const float bz = i >= tok ? a.scale * d * dz[t][r] : 0.f, az = i > tok ? -d * wz[t][r] : 0.f;
          db += (i >= tok ? bz * qk[t][r] : 0.f) + (i > tok ? az * kk[t][r] : 0.f);
          vb[t >> 1][4 * (t & 1) + r] = beta_n * bz;
          va[t >> 1][4 * (t & 1) + r] = beta_n * az;
        }
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) bk[kb] = split(vb[kb]), aw[kb] = split(va[kb]);
    }
    float dot = 0.f, at_end = 0.f;  // q . dq + k . (dk as read - as written); k . early
    const float eb = to_end * beta_n;
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      float kf[8], qf[8];
      {
        const int cnt = tok < tokens ? max(0, min(8, Dk - 32 * kb - 8 * g)) : 0;
        const int64_t o = tok * qs + 32 * kb + 8 * g;
        const Raw8<T> kraw = load_raw8<VEC>(k + o, cnt), qraw = load_raw8<VEC>(q + o, cnt);
        kraw.open(kf);
        qraw.open(qf);
      }
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int t = 2 * kb + half;
        float ke = 0.f;
#pragma unroll
        for (int r = 0; r < 4; ++r) ke += kf[4 * half + r] * early[t][r];
        db += to_end * ke;
        at_end += eb * ke;
        dq[t] *= a.scale * ahead;
        read[t] *= -ahead;
        early[t] *= eb;
#pragma unroll
        for (int b2 = 0; b2 < 2; ++b2) {
          Op<NP> ka, qa;
#pragma unroll
          for (int p = 0; p < NP; ++p) {
            const int o = Tokens<KP>::col_at(16 * t + n, 64 * b2 + 16 * g);
            ka.p[p] = *reinterpret_cast<const bf8_t*>(lds.k[p] + o);
            qa.p[p] = *reinterpret_cast<const bf8_t*>(lds.q[p] + o);
          }
          if (b2 <= (w >> 1)) {
            dq[t] = mma(ka, bq[b2], dq[t]);
            read[t] = mma(ka, ar[b2], read[t]);
          }
          if (b2 >= (w >> 1)) {
            early[t] = mma(qa, bk[b2], early[t]);
            early[t] = mma(ka, aw[b2], early[t]);
          }
        }
#pragma unroll
        for (int r = 0; r < 4; ++r)
          dot += qf[4 * half + r] * dq[t][r] + kf[4 * half + r] * (read[t][r] - early[t][r]);
        dqt[t] = SHARED ? dqt[t] + dq[t] : dq[t];
        dkt[t] = SHARED ? dkt[t] + (read[t] + early[t]) : read[t] + early[t];
      }
    }
    dot = sum_groups(dot);
    db = sum_groups(db);
    // <M, N> and the ends' sum over the chunk
    const float ends = wave_sum(at_end + expf((float)Gend) * mn);
    if (g == 0) {
      lds.dG[tok] = dot;
      if (tok < rows) a.dbeta[gat + tok * a.Hv] = tok < tokens ? db : 0.f;
    }
    if (lane == 0) lds.end[w] = ends;
    __syncthreads();
    if (tid < CH) {
      float s = lds.dG[tid];
#pragma unroll
      for (int o = 1; o < CH; o <<= 1) {
        const float down = __shfl_down(s, o, 64);
        if (tid + o < CH) s += down;
      }
      s += (lds.end[0] + lds.end[1]) + (lds.end[2] + lds.end[3]);
      if (tid < rows) a.dg[gat + tid * a.Hv] = tid < tokens ? s : 0.f;
    }
    __syncthreads();
  }
#pragma unroll
  for (int kb = 0; kb < KB; ++kb) {
    const int cnt = tok < rows ? max(0, min(8, Dk - 32 * kb - 8 * g)) : 0;
    const int64_t o = q0 + tok * qs + 32 * kb + 8 * g;
    float vq[8], vk[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      vq[e] = tok < tokens ? dqt[2 * kb + (e >> 2)][e & 3] : 0.f;
      vk[e] = tok < tokens ? dkt[2 * kb + (e >> 2)][e & 3] : 0.f;
    }
    store8_some<VEC>((T*)a.dq + o, cnt, vq);
    store8_some<VEC>((T*)a.dk + o, cnt, vk);
  }
}

template <typename K>
hipError_t with_lds(K kernel, size_t lds, unsigned grid, const DeltaArgs& a, hipStream_t st) {
  if (lds > 64 * 1024) {
    hipError_t e = hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(kernel, dim3(grid), dim3(256), lds, st, a);
  return hipGetLastError();
}

template <typename T, int KP, int NT>
hipError_t back_go(const DeltaArgs& a, hipStream_t st) {
  const unsigned grid = (unsigned)(a.B * a.Hv * ((a.Dv + 64 * NT - 1) / (64 * NT)));
  const size_t lds = sizeof(BackLds<KP, Stream<T>::NP>);
  return a.vec ? with_lds(delta_back_kernel<T, KP, NT, true>, lds, grid, a, st)
               : with_lds(delta_back_kernel<T, KP, NT, false>, lds, grid, a, st);
}

template <typename T, int KP>
hipError_t grad_go(const DeltaArgs& a, hipStream_t st) {
  const unsigned grid = (unsigned)(a.B * a.Hk * a.NC);
  const size_t lds = sizeof(GradLds<KP, Stream<T>::NP>);
  if (a.Hv == a.Hk)
    return a.vec8 ? with_lds(delta_grad_kernel<T, KP, true, false>, lds, grid, a, st)
                  : with_lds(delta_grad_kernel<T, KP, false, false>, lds, grid, a, st);
  return a.vec8 ? with_lds(delta_grad_kernel<T, KP, true, true>, lds, grid, a, st)
                : with_lds(delta_grad_kernel<T, KP, false, true>, lds, grid, a, st);
}

template <typename T, int KP>
hipError_t backward_go(const DeltaArgs& a, hipStream_t st) {
  hipError_t e;
  if constexpr (KP < 256) e = a.Dv > 64 ? back_go<T, KP, 2>(a, st) : back_go<T, KP, 1>(a, st);
  else e = back_go<T, KP, 1>(a, st);
  return e != hipSuccess || a.NC == 0 ? e : grad_go<T, KP>(a, st);
}

template <typename T>
hipError_t backward_by_width(const DeltaArgs& a, hipStream_t st) {
  if (a.Dk <= 64) return backward_go<T, 64>(a, st);
  if (a.Dk <= 128) return backward_go<T, 128>(a, st);
  return backward_go<T, 256>(a, st);
}

}  // namespace

int64_t delta_backward_ws(DeltaArgs& a, void* ws) {
  const int64_t n = a.B * a.Hv * a.NC, KP = a.Dk <= 64 ? 64 : a.Dk <= 128 ? 128 : 256;
  a.VP = (a.Dv + 31) / 32 * 32;
  int64_t at = 0;
  const auto take = [&](int64_t bytes) {
    char* p = (char*)ws + at;
    at += n * bytes;  // every part is whole kilobytes
    return (void*)p;
  };
  a.states = take(4 * KP * a.VP);
  a.dstates = take(4 * KP * a.VP);
  a.z = take(4 * CH * a.VP);
  a.w = take(4 * CH * a.VP);
  a.rec = take(REC_BWD);
  return at;
}

hipError_t launch_delta_backward(int dtype, const DeltaArgs& a, hipStream_t st) {
  if (a.NC > 0) {
    hipError_t e = launch_delta_keep(dtype, a, st);
    if (e != hipSuccess) return e;
  }
  return dtype == 0 ? backward_by_width<float>(a, st) : backward_by_width<bf16_t>(a, st);
}

}  // namespace hc
