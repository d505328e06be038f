// Gated delta rule, forward. Per head, with the state M [Dk, Dv]:
//   F = exp(g_t) M_{t-1},  z_t = v_t - F^T k_t,  M_t = F + beta_t k_t z_t^T,  o_t = scale M_t^T q_t.
// A chunk of 64 tokens is joined at once: with G the running sum of g in it, M the state before it,
//   A_ij = exp(G_i - G_j) (k_i . k_j) beta_j (j < i),  P_ij = exp(G_i - G_j) (q_i . k_j) (j <= i),
//   Z = (I + A)^-1 (V - exp(G) K M),  X = beta Z,
//   O = scale (exp(G) Q M + P X),  M' = exp(G_end) M + K^T (exp(G_end - G) X).
// Two kernels: every chunk's triangle, its inverse T and P by themselves, and the walk over the
// chunks, whose columns of the state (and of V, Z, O) never meet: a wave keeps its 16 or 32
// columns' state in registers and hands each product's result to the next as its operand.
// Products are bfloat16 matrix instructions with float32 sums; values that are not bfloat16
// already (the state, Z, T, P, float32 streams) enter as two parts, 16 bits, so that the
// state carries errors of 2^-17 of its terms rather than 2^-9.
#include "hc_delta_device.h"

namespace hc {

namespace {

// --------------------------------------------------------------- each chunk by itself

template <typename T, int KP, bool VEC, bool BWD>
__global__ __launch_bounds__(256) void delta_prep_kernel(DeltaArgs a) {
  constexpr int NP = Stream<T>::NP, KB = KP / 32, LS = CH + 4;
  __shared__ __attribute__((aligned(16))) float L[CH][LS], inv[CH][LS];
  __shared__ double G[CH];
  __shared__ __attribute__((aligned(16))) float beta_s[CH];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, n = lane & 15, g = lane >> 4;
  const int64_t NC = a.NC, chunk = blockIdx.x % NC, bh = blockIdx.x / NC, b = bh / a.Hk, hk = bh % a.Hk;
  const int64_t t0 = chunk * CH, tokens = length_of(a.lengths, b, a.S) - t0;
  if (tokens <= 0) return;
  const int Dk = (int)a.Dk;
  const int64_t qs = a.Hk * a.Dk;
  const T* q = (const T*)a.q + (b * a.S + t0) * qs + hk * a.Dk;
  const T* k = (const T*)a.k + (b * a.S + t0) * qs + hk * a.Dk;

  // keys by queries (and keys by keys): lane n is token 16 w + n as the later one, its rows the
  // earlier ones; in the backward also queries (rows) by keys
  f4_t kk[4], qk[4], kq[4];
#pragma unroll
  for (int t = 0; t < 4; ++t) kk[t] = qk[t] = kq[t] = f4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int kb = 0; kb < KB; ++kb) {
    const int k0 = 32 * kb + 8 * g;
    const Op<NP> kn = token_op<T, VEC>(k, qs, tokens, 16 * w + n, k0, Dk);
    const Op<NP> qn = token_op<T, VEC>(q, qs, tokens, 16 * w + n, k0, Dk);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      if ((t >> 1) <= (w >> 1)) {
        const Op<NP> kr = token_op<T, VEC>(k, qs, tokens, row_of(t, n), k0, Dk);
        kk[t] = mma(kr, kn, kk[t]);
        qk[t] = mma(kr, qn, qk[t]);
      }
      if (BWD && (t >> 1) >= (w >> 1)) kq[t] = mma(token_op<T, VEC>(q, qs, tokens, row_of(t, n), k0, Dk), kn, kq[t]);
    }
  }
  // the upper blocks that the inverse's tiles hold stay zero
  {
    const int bl = threadIdx.x >> 7, i = (threadIdx.x & 127) >> 3, c = 2 * (threadIdx.x & 7);
    inv[32 * bl + i][32 * bl + 16 + c] = inv[32 * bl + i][32 * bl + 16 + c + 1] = 0.f;
  }
  const int per = (int)(a.Hv / a.Hk);
  for (int hi = 0; hi < per; ++hi) {
    const int64_t hv = hk * per + hi, rec = (b * a.Hv + hv) * NC + chunk;
    char* out = (char*)a.rec + rec * (BWD ? REC_BWD : REC);
    if (threadIdx.x < CH) {  // one wave
      const int i = threadIdx.x;
      const bool on = i < tokens;
      const int64_t at = (b * a.S + t0 + i) * a.Hv + hv;
      const double s = running_sum(on ? clamp_decay(a.g[at]) : 0.0, i);
      const double end = __shfl(s, CH - 1, 64);
      const float be = on ? a.beta[at] : 0.f;
      G[i] = s;
      beta_s[i] = be;
      float* dec = (float*)(out + REC_DEC);
      dec[DEC_AHEAD + i] = expf((float)s);
      dec[DEC_TO_END + i] = expf((float)(end - s));
      dec[DEC_BETA + i] = be;
    }
    __syncthreads();
    {
      const int i = 16 * w + n;
      const double Gi = G[i];
      float p[2][8];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        if ((t >> 1) > (w >> 1)) continue;
        const int j0 = 32 * (t >> 1) + 8 * g + 4 * (t & 1);
        f4_t l;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float d = j0 + r <= i ? expf((float)(Gi - G[j0 + r])) : 0.f;
          p[t >> 1][4 * (t & 1) + r] = j0 + r <= i ? d * qk[t][r] : 0.f;
          l[r] = j0 + r < i ? d * kk[t][r] * beta_s[j0 + r] : 0.f;
        }
        *reinterpret_cast<f4_t*>(&L[i][j0]) = l;
      }
      if (!BWD) {
        store_tile(out + REC_P, tri(w, 0), lane, p[0]);
        if (w >= 2) store_tile(out + REC_P, tri(w, 1), lane, p[1]);
      }
    }
    if (BWD) {
      const int j = 16 * w + n;
      const double Gj = G[j];
      float p[2][8];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        if ((t >> 1) < (w >> 1)) continue;
        const int i0 = 32 * (t >> 1) + 8 * g + 4 * (t & 1);
#pragma unroll
        for (int r = 0; r < 4; ++r)
          p[t >> 1][4 * (t & 1) + r] = j <= i0 + r ? expf((float)(G[i0 + r] - Gj)) * kq[t][r] : 0.f;
      }
      // lane n holds P^T's row j = 16 w + n: its place in row_of's order
      const int pl = place_of(j), t = pl >> 4, to = (pl & 15) + 16 * g;
      if (w < 2) store_tile(out + REC_P, tri_t(t, 0), to, p[0]);
      store_tile(out + REC_P, tri_t(t, 1), to, p[1]);
    }
    __syncthreads();
    // (I + A)^-1: wave w inverts its 16 x 16 block on the diagonal, a lane a column, ...
    {
      float x[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float s = i == n ? 1.f : 0.f;
#pragma unroll
        for (int m = 0; m < i; ++m) s -= L[16 * w + i][16 * w + m] * x[m];
        x[i] = s;
      }
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if ((i >> 2) == g) inv[16 * w + i][16 * w + n] = x[i];
    }
    __syncthreads();
    // ... then forms the blocks below it: T_iw = -T_ii sum_m A_im T_mw, in float32 products
    {
      f4_t col[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) col[0][r] = inv[16 * w + 4 * g + r][16 * w + n];
#pragma unroll
      for (int d = 1; d < 4; ++d) {  // block row w + d
        if (w + d >= 4) break;
        const int i0 = 16 * (w + d);
        f4_t s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int m = 0; m < d; ++m) {
          const f4_t l = *reinterpret_cast<const f4_t*>(&L[i0 + n][16 * (w + m) + 4 * g]);
#pragma unroll
          for (int r = 0; r < 4; ++r) s = __builtin_amdgcn_mfma_f32_16x16x4f32(l[r], col[m][r], s, 0, 0, 0);
        }
        const f4_t ti = *reinterpret_cast<const f4_t*>(&inv[i0 + n][i0 + 4 * g]);
        f4_t o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int r = 0; r < 4; ++r) o = __builtin_amdgcn_mfma_f32_16x16x4f32(ti[r], -s[r], o, 0, 0, 0);
        col[d] = o;
#pragma unroll
        for (int r = 0; r < 4; ++r) inv[i0 + 4 * g + r][16 * w + n] = o[r];
      }
    }
    __syncthreads();
    {
      const int i = row_of(w, n);
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        if (kb <= (w >> 1)) store_tile(out + REC_T, tri(w, kb), lane, &inv[i][32 * kb + 8 * g]);
        if (BWD && kb >= (w >> 1)) {
          float v[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = inv[32 * kb + 8 * g + e][i];
          store_tile(out + REC_TT, tri_t(w, kb), lane, v);
        }
      }
    }
    __syncthreads();
  }
}

// --------------------------------------------------------------------- the walk

template <int KP, int NP, bool KEEP>
struct WalkLds {
  char k[NP][Tokens<KP>::PART];  // keys: rows in row_of's order, then transposed
  char q[KEEP ? 1 : NP][KEEP ? 16 : Tokens<KP>::ROWS];
  char rec[KEEP ? REC_P : REC];
};

// KEEP: the backward's, which wants every chunk's first state and Z rather than O.
template <typename T, int KP, int NT, bool VEC, bool KEEP>
__global__ __launch_bounds__(256) void delta_walk_kernel(DeltaArgs a) {
  constexpr int NP = Stream<T>::NP, KB = KP / 32, KT = KP / 16;
  static_assert(sizeof(WalkLds<KP, NP, KEEP>) <= 160 * 1024, "LDS of a CU");
  constexpr int PIECES = KP / 8, ITEMS = 32 * PIECES / 256;  // pairs of tokens by pieces of 8, for each thread
  extern __shared__ __attribute__((aligned(16))) char lds_raw[];
  typedef WalkLds<KP, NP, KEEP> Lds;
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
  const T* vp = (const T*)a.v + b * a.S * vs + hv * a.Dv + col;
  T* op = (T*)a.o + b * a.S * vs + hv * a.Dv + col;
  constexpr int REC_STRIDE = KEEP ? REC_BWD : REC, REC_USED = KEEP ? REC_P : REC;
  const char* rec = (const char*)a.rec + bh * a.NC * REC_STRIDE;

  f4_t S[KT][NT];
  {
    const float* s0 = a.state0 ? a.state0 + bh * a.Dk * a.Dv + col : nullptr;
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = row_of(t, 4 * g + r);
        const Cols<NT> c = load_cols<NT, VEC>(s0 + (int64_t)row * a.Dv, s0 && row < Dk ? have : 0);
#pragma unroll
        for (int h = 0; h < NT; ++h) S[t][h][r] = c.v[h];
      }
  }

  // the next chunk's operands on their way
  Raw8<T> kr[ITEMS][2], qr[ITEMS][2];
  u4_t rr[(REC_USED + 4095) / 4096];
  Cols<NT> vr[4][4];
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
        if (!KEEP) qr[i][j] = load_raw8<VEC>(qp + t * qs + 8 * piece, cnt);
      }
    }
#pragma unroll
    for (int i = 0; i < (REC_USED + 4095) / 4096; ++i)
      if (i * 4096 + tid * 16 < REC_USED)
        rr[i] = *reinterpret_cast<const u4_t*>(rec + c * REC_STRIDE + i * 4096 + tid * 16);
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int64_t tok = t0 + row_of(t, 4 * g + r);
        vr[t][r] = load_cols<NT, VEC>(vp + tok * vs, tok < len ? have : 0);
      }
  };
  if (chunks > 0) fetch(0);
  for (int64_t c = 0; c < chunks; ++c) {
    Op<NP> ko[ITEMS][2];
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int x = i * 256 + tid, piece = x % PIECES, pair = x / PIECES;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        ko[i][j] = kr[i][j].op();
#pragma unroll
        for (int p = 0; p < NP; ++p)
          *reinterpret_cast<bf8_t*>(lds.k[p] + Tokens<KP>::row_at(place_of(2 * pair + j), 16 * piece)) = ko[i][j].p[p];
        if (!KEEP) {
          const Op<NP> qo = qr[i][j].op();
#pragma unroll
          for (int p = 0; p < NP; ++p)
            *reinterpret_cast<bf8_t*>(lds.q[p] + Tokens<KP>::row_at(2 * pair + j, 16 * piece)) = qo.p[p];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < (REC_USED + 4095) / 4096; ++i)
      if (i * 4096 + tid * 16 < REC_USED) *reinterpret_cast<u4_t*>(lds.rec + i * 4096 + tid * 16) = rr[i];
    Cols<NT> v[4][4];
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) v[t][r] = vr[t][r];
    __syncthreads();

    if (KEEP && col < a.VP) {
      bf16_t* keep = (bf16_t*)a.states + (bh * a.NC + c) * 2 * KP * a.VP + col;
#pragma unroll
      for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          Cols<NT> y;
#pragma unroll
          for (int h = 0; h < NT; ++h) y.v[h] = S[t][h][r];
          store_parts<NT>(keep + row_of(t, 4 * g + r) * a.VP, KP * a.VP, y);
        }
    }
    // K M and Q M
    f4_t km[4][NT], o[4][NT];
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int h = 0; h < NT; ++h) km[t][h] = o[t][h] = f4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      Split sf[NT];
#pragma unroll
      for (int h = 0; h < NT; ++h) sf[h] = split(S[2 * kb][h], S[2 * kb + 1][h]);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        Op<NP> ka, qa;
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          const int at = Tokens<KP>::row_at(16 * t + n, 64 * kb + 16 * g);
          ka.p[p] = *reinterpret_cast<const bf8_t*>(lds.k[p] + at);
          if (!KEEP) qa.p[p] = *reinterpret_cast<const bf8_t*>(lds.q[p] + at);
        }
#pragma unroll
        for (int h = 0; h < NT; ++h) {
          km[t][h] = mma(ka, sf[h], km[t][h]);
          if (!KEEP) o[t][h] = mma(qa, sf[h], o[t][h]);
        }
      }
    }
    __syncthreads();
    // the keys take the rows' place, transposed, two tokens at a time
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int x = i * 256 + tid, piece = x % PIECES, pair = x / PIECES;
#pragma unroll
      for (int p = 0; p < NP; ++p) store_transposed<KP>(lds.k[p], pair, piece, ko[i][0].p[p], ko[i][1].p[p]);
    }
    if (c + 1 < chunks) fetch(c + 1);

    // R = V - exp(G) K M, Z = T R, X = beta Z
    const float* dec = (const float*)(lds.rec + REC_DEC);
    Split x[2][NT];
    {
      Split rf[2][NT];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const f4_t ahead = *reinterpret_cast<const f4_t*>(dec + DEC_AHEAD + row_of(t, 4 * g));
#pragma unroll
        for (int h = 0; h < NT; ++h)
#pragma unroll
          for (int r = 0; r < 4; ++r) km[t][h][r] = v[t][r].v[h] - ahead[r] * km[t][h][r];
      }
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int h = 0; h < NT; ++h) rf[kb][h] = split(km[2 * kb][h], km[2 * kb + 1][h]);
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int h = 0; h < NT; ++h) km[t][h] = f4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int t = 2 * kb; t < 4; ++t) {
          const Split ta = load_tile(lds.rec + REC_T, tri(t, kb), lane);
#pragma unroll
          for (int h = 0; h < NT; ++h) km[t][h] = mma(ta, rf[kb][h], km[t][h]);
        }
      if (KEEP && col < a.VP) {
        bf16_t* keep = (bf16_t*)a.z + (bh * a.NC + c) * 2 * CH * a.VP + col;
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            Cols<NT> y;
#pragma unroll
            for (int h = 0; h < NT; ++h) y.v[h] = km[t][h][r];
            store_parts<NT>(keep + row_of(t, 4 * g + r) * a.VP, CH * a.VP, y);
          }
      }
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const f4_t beta = *reinterpret_cast<const f4_t*>(dec + DEC_BETA + row_of(t, 4 * g));
#pragma unroll
        for (int h = 0; h < NT; ++h) km[t][h] *= beta;
      }
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int h = 0; h < NT; ++h) x[kb][h] = split(km[2 * kb][h], km[2 * kb + 1][h]);
    }
    if (!KEEP) {  // O = scale (exp(G) Q M + P X)
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const f4_t ahead = *reinterpret_cast<const f4_t*>(dec + DEC_AHEAD + 16 * t + 4 * g);
#pragma unroll
        for (int h = 0; h < NT; ++h) o[t][h] *= ahead;
#pragma unroll
        for (int kb = 0; kb <= (t >> 1); ++kb) {
          const Split pa = load_tile(lds.rec + REC_P, tri(t, kb), lane);
#pragma unroll
          for (int h = 0; h < NT; ++h) o[t][h] = mma(pa, x[kb][h], o[t][h]);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int64_t tok = c * CH + 16 * t + 4 * g + r;
          Cols<NT> y;
#pragma unroll
          for (int h = 0; h < NT; ++h) y.v[h] = a.scale * o[t][h][r];
          store_cols<NT, VEC>(op + tok * vs, tok < len ? have : 0, y);
        }
      }
    }
    // M = exp(G_end) M + K^T (exp(G_end - G) X)
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const f4_t to_end = *reinterpret_cast<const f4_t*>(dec + DEC_TO_END + row_of(t, 4 * g));
#pragma unroll
      for (int h = 0; h < NT; ++h) km[t][h] *= to_end;
    }
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int h = 0; h < NT; ++h) x[kb][h] = split(km[2 * kb][h], km[2 * kb + 1][h]);
    const float whole = dec[DEC_AHEAD + CH - 1];
    __syncthreads();
#pragma unroll
    for (int t = 0; t < KT; ++t) {
#pragma unroll
      for (int h = 0; h < NT; ++h) S[t][h] *= whole;
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        Op<NP> ka;
#pragma unroll
        for (int p = 0; p < NP; ++p)
          ka.p[p] = *reinterpret_cast<const bf8_t*>(lds.k[p] + Tokens<KP>::col_at(16 * t + n, 64 * kb + 16 * g));
#pragma unroll
        for (int h = 0; h < NT; ++h) S[t][h] = mma(ka, x[kb][h], S[t][h]);
      }
    }
    __syncthreads();
  }
  if (a.state1) {
    float* s1 = a.state1 + bh * a.Dk * a.Dv + col;
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = row_of(t, 4 * g + r);
        Cols<NT> y;
#pragma unroll
        for (int h = 0; h < NT; ++h) y.v[h] = S[t][h][r];
        store_cols<NT, VEC>(s1 + (int64_t)row * a.Dv, row < Dk ? have : 0, y);
      }
  }
}

// ---------------------------------------------------------------- token by token

// A few tokens: 32 columns of a head's state in a workgroup's registers, 8 lanes of 4 columns by
// 32 rows at a time. Both products with the state before the token (k and q) are summed at once,
// and o = scale (exp(g) M^T q + (q . k) beta z).
template <typename T, int KP, bool VEC>
__global__ __launch_bounds__(256) void delta_step_kernel(DeltaArgs a) {
  constexpr int R = KP / 32;
  __shared__ float qk_s[2][KP];
  __shared__ float part[2][4][8][12];
  const int tid = threadIdx.x, w = tid >> 6, cl = tid & 7, rg = tid >> 3;
  const int64_t groups = (a.Dv + 31) / 32;
  const int64_t bh = blockIdx.x / groups, b = bh / a.Hv, hv = bh % a.Hv, hk = hv / (a.Hv / a.Hk);
  const int col = (int)(blockIdx.x % groups) * 32 + 4 * cl, have = max(0, min(4, (int)a.Dv - col));
  const int64_t len = length_of(a.lengths, b, a.S);
  f4_t S[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int row = rg + 32 * i;
    S[i] = f4_t{0.f, 0.f, 0.f, 0.f};
    if (a.state0 && row < a.Dk) {
      const float* p = a.state0 + (bh * a.Dk + row) * a.Dv + col;
      if (VEC) {
        if (have > 0) S[i] = *reinterpret_cast<const f4_t*>(p);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (e < have) S[i][e] = p[e];
      }
    }
  }
  for (int64_t t = 0; t < len; ++t) {
    const int64_t qo = ((b * a.S + t) * a.Hk + hk) * a.Dk, vo = ((b * a.S + t) * a.Hv + hv);
    const float decay = expf(a.g[vo]), beta = a.beta[vo];
    for (int i = tid; i < 2 * KP; i += 256) {
      const int row = i & (KP - 1);
      const T* src = i < KP ? (const T*)a.k : (const T*)a.q;
      qk_s[i >= KP][row] = row < a.Dk ? Elem<T>::ld(src + qo + row) : 0.f;
    }
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = e < have ? Elem<T>::ld((const T*)a.v + vo * a.Dv + col + e) : 0.f;
    __syncthreads();
    float s[9] = {};
    float k[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      k[i] = qk_s[0][rg + 32 * i];
      const float q = qk_s[1][rg + 32 * i];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[e] += k[i] * S[i][e];
        s[4 + e] += q * S[i][e];
      }
      s[8] += k[i] * q;
    }
#pragma unroll
    for (int x = 0; x < 9; ++x) {
      s[x] += __shfl_xor(s[x], 8, 64);
      s[x] += __shfl_xor(s[x], 16, 64);
      s[x] += __shfl_xor(s[x], 32, 64);
    }
    if ((tid & 63) < 8)
#pragma unroll
      for (int x = 0; x < 9; ++x) part[t & 1][w][cl][x] = s[x];
    __syncthreads();
#pragma unroll
    for (int x = 0; x < 9; ++x)
      s[x] = (part[t & 1][0][cl][x] + part[t & 1][1][cl][x]) + (part[t & 1][2][cl][x] + part[t & 1][3][cl][x]);
    float add[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) add[e] = beta * (v[e] - decay * s[e]);
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) S[i][e] = decay * S[i][e] + k[i] * add[e];
    if (rg == 0) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < have) Elem<T>::st((T*)a.o + vo * a.Dv + col + e, a.scale * (decay * s[4 + e] + s[8] * add[e]));
    }
  }
  if (a.state1 == nullptr) return;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int row = rg + 32 * i;
    if (row < a.Dk) {
      float* p = a.state1 + (bh * a.Dk + row) * a.Dv + col;
      if (VEC) {
        if (have > 0) *reinterpret_cast<f4_t*>(p) = S[i];
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (e < have) p[e] = S[i][e];
      }
    }
  }
}

constexpr int SHORT = 8;  // tokens up to which they are taken one by one

template <typename T, int KP, int NT, bool KEEP>
hipError_t walk_go(const DeltaArgs& a, hipStream_t st) {
  const size_t lds = sizeof(WalkLds<KP, Stream<T>::NP, KEEP>);
  const dim3 prep((unsigned)(a.B * a.Hk * a.NC)), walk((unsigned)(a.B * a.Hv * ((a.Dv + 64 * NT - 1) / (64 * NT))));
  const auto go = [&](auto prep_k, auto walk_k) {
    if (lds > 64 * 1024) {
      hipError_t e = hipFuncSetAttribute((const void*)walk_k, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
      if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(prep_k, prep, dim3(256), 0, st, a);
    hipLaunchKernelGGL(walk_k, walk, dim3(256), lds, st, a);
    return hipGetLastError();
  };
  if (a.vec) return go(delta_prep_kernel<T, KP, true, KEEP>, delta_walk_kernel<T, KP, NT, true, KEEP>);
  return go(delta_prep_kernel<T, KP, false, KEEP>, delta_walk_kernel<T, KP, NT, false, KEEP>);
}

template <typename T, int KP, bool KEEP>
hipError_t delta_go(const DeltaArgs& a, hipStream_t st) {
  if (!KEEP && a.S <= SHORT) {
    const dim3 grid((unsigned)(a.B * a.Hv * ((a.Dv + 31) / 32)));
    if (a.vec && a.Dv % 4 == 0) hipLaunchKernelGGL((delta_step_kernel<T, KP, true>), grid, dim3(256), 0, st, a);
    else hipLaunchKernelGGL((delta_step_kernel<T, KP, false>), grid, dim3(256), 0, st, a);
    return hipGetLastError();
  }
  if constexpr (KP < 256) {
    if (a.Dv > 64) return walk_go<T, KP, 2, KEEP>(a, st);
  }
  return walk_go<T, KP, 1, KEEP>(a, st);
}

template <typename T, bool KEEP>
hipError_t delta_by_width(const DeltaArgs& a, hipStream_t st) {
  if (a.Dk <= 64) return delta_go<T, 64, KEEP>(a, st);
  if (a.Dk <= 128) return delta_go<T, 128, KEEP>(a, st);
  return delta_go<T, 256, KEEP>(a, st);
}

}  // namespace

int64_t delta_ws_bytes(int64_t B, int64_t S, int64_t Hv) {
  return S <= SHORT ? 0 : B * Hv * ((S + CH - 1) / CH) * (int64_t)REC;
}

hipError_t launch_delta(int dtype, const DeltaArgs& a, hipStream_t st) {
  return dtype == 0 ? delta_by_width<float, false>(a, st) : delta_by_width<bf16_t, false>(a, st);
}

hipError_t launch_delta_keep(int dtype, const DeltaArgs& a, hipStream_t st) {
  return dtype == 0 ? delta_by_width<float, true>(a, st) : delta_by_width<bf16_t, true>(a, st);
}

}  // namespace hc
