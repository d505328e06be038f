// Gated delta rule, forward. Per head, with the state M [Dk, Dv]:
//   F = exp(g_t) M_{t-1},  z_t = v_t - F^T k_t,  M_t = F + beta_t k_t z_t^T,  o_t = scale M_t^T q_t.
// A chunk of 64 tokens is joined at once: with G the running sum of g in it, M the state before it,
//   A_ij = exp(G_i - G_j) (k_i . k_j) beta_j (j < i),  P_ij = exp(G_i - G_j) (q_i . k_j) (j <= i),
//   Z = (I + A)^-1 (V - exp(G) K M),  X = beta Z,
//   O = scale (exp(G) Q M + P X),  M' = exp(G_end) M + K^T (exp(G_end - G) X).
// Two kernels: every chunk's triangle, its inverse T and P by themselves, and the walk over the
// chunks, whose columns of the state (and of V, Z, O) never meet: a wave keeps its 16
// columns' state in registers and hands each product's result to the next as its operand.
// Products are bfloat16 matrix instructions with float32 sums; values that are not bfloat16 already enter
// as three parts, float32's 24 bits, and the six products of parts that matter (with two parts, 16 bits,
// states were off by 7 x 10^-7 of their norm and float32 outputs by 2 to 4 x 10^-6 where a float32 form is by 2
// and 3 x 10^-7; as they are now they are within that, and bfloat16 outputs differ from it in a tenth of the
// roundings. For this a walk takes a tenth longer, of 256 float32 keys a quarter). T and P lie in the record as
// float32, which is smaller than three parts, and are split where they enter LDS, once for all waves.
//   What bounds it: 2,048 chunks of 128 x 128 in bfloat16 (8 sequences of 1,024 tokens, 16 value
// heads on 8 key heads) read and write 118 MB and need 15 GFLOP, 20 us of memory. The chunks
// by themselves take 37 us: each wave reads its tiles of keys and queries from memory between the
// products, four waves the same rows, and nearly every load is waited for by itself; then come the
// triangle's steps. The walk takes 102 us as 16 chunks in a row on 256 workgroups, 6.4 us a chunk of which the
// matrix units work for 1.5. A chunk first waits for the next one's loads, as bfloat16 values are
// widened where they are fetched and loads are waited for in order; then each product waits for the
// one before it and for its operands, which come from LDS just ahead of it. Walks that keep states
// wait for a chunk's stores too. Few heads are walked in segments at once (see delta_plan), and
// what does not depend on the state is done by every chunk for itself.
#include "hc_delta_device.h"

namespace hc {

namespace {

// --------------------------------------------------------------- each chunk by itself

template <typename T, int KP, bool VEC, bool BWD>
__global__ __launch_bounds__(256, 4) void delta_prep_kernel(DeltaArgs a) {
  constexpr int NP = PARTS<T>, KB = KP / 32, LS = CH + 4;
  __shared__ __attribute__((aligned(16))) float L[CH][LS], inv[CH][LS];
  __shared__ double G[CH];
  __shared__ __attribute__((aligned(16))) float beta_s[CH];
  const int lane = threadIdx.x & 63, w = wave_number(), n = lane & 15, g = lane >> 4;
  const uint32_t NC = (uint32_t)a.NC, chunk = blockIdx.x % NC, bh = blockIdx.x / NC, hv = bh % (uint32_t)a.Hv;
  const uint32_t hk = hv / ((uint32_t)a.Hv / (uint32_t)a.Hk);
  const int64_t b = bh / (uint32_t)a.Hv;
  const int64_t t0 = (int64_t)chunk * CH, tokens = length_of(a.lengths, b, a.S) - t0;
  if (tokens <= 0) return;
  const int Dk = (int)a.Dk, qs = (int)(a.Hk * a.Dk), left = (int)min((int64_t)CH, tokens);
  const int64_t at0 = (b * a.S + t0) * qs + hk * Dk;
  const Range q = head_rows((const T*)a.q + at0, left, qs, Dk), k = head_rows((const T*)a.k + at0, left, qs, Dk);

  // keys by queries (and keys by keys): lane n is token 16 w + n as the later one, its rows the
  // earlier ones; in the backward also queries (rows) by keys
  f4_t kk[4], qk[4], kq[4];
#pragma unroll
  for (int t = 0; t < 4; ++t) kk[t] = qk[t] = kq[t] = f4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int kb = 0; kb < KB; ++kb) {
    const int k0 = 32 * kb + 8 * g;
    const Op<NP> kn = token_op<T, VEC, NP>(k, qs, 16 * w + n, k0, Dk);
    const Op<NP> qn = token_op<T, VEC, NP>(q, qs, 16 * w + n, k0, Dk);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      if ((t >> 1) <= (w >> 1)) {
        const Op<NP> kr = token_op<T, VEC, NP>(k, qs, row_of(t, n), k0, Dk);
        kk[t] = mma(kr, kn, kk[t]);
        qk[t] = mma(kr, qn, qk[t]);
      }
      if (BWD && (t >> 1) >= (w >> 1)) kq[t] = mma(token_op<T, VEC, NP>(q, qs, row_of(t, n), k0, Dk), kn, kq[t]);
    }
    keep_order();
  }
  // the upper blocks that the inverse's tiles hold stay zero
  {
    const int bl = threadIdx.x >> 7, i = (threadIdx.x & 127) >> 3, c = 2 * (threadIdx.x & 7);
    inv[32 * bl + i][32 * bl + 16 + c] = inv[32 * bl + i][32 * bl + 16 + c + 1] = 0.f;
  }
  char* out = (char*)a.rec + (int64_t)blockIdx.x * (BWD ? REC_BWD : REC);
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
    dec[DEC_AHEAD + i] = decay(s);
    dec[DEC_TO_END + i] = decay(end - s);
    dec[DEC_BETA + i] = be;
  }
  lds_barrier();
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
        const float d = j0 + r <= i ? decay(Gi - G[j0 + r]) : 0.f;
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
        p[t >> 1][4 * (t & 1) + r] = j <= i0 + r ? decay(G[i0 + r] - Gj) * kq[t][r] : 0.f;
    }
    // lane n holds P^T's row j = 16 w + n: its place in row_of's order
    const int pl = place_of(j), t = pl >> 4, to = (pl & 15) + 16 * g;
    if (w < 2) store_tile(out + REC_P, tri_t(t, 0), to, p[0]);
    store_tile(out + REC_P, tri_t(t, 1), to, p[1]);
  }
  lds_barrier();
  // (I + A)^-1: wave w inverts its 16 x 16 block on the diagonal, a lane a column, ...
  {
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float s = i == n ? 1.f : 0.f;
#pragma unroll
      for (int m = 0; m < i; ++m) s -= L[16 * w + i][16 * w + m] * x[m];
      x[i] = s;
      if (i & 1) keep_order();
    }
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if ((i >> 2) == g) inv[16 * w + i][16 * w + n] = x[i];
  }
  lds_barrier();
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
  lds_barrier();
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
}

// --------------------------------------------------------------------- the walk

constexpr int OUT = 0, KEEP = 1, SUM = 2, SUM_BWD = 3;

template <int KP, int NP, int NW, int MODE>
struct WalkLds {
  static constexpr bool TURN = MODE == OUT && NP == 3 && KP == 256;  // no room for both: keys after queries, in k
  char k[NP][Tokens<KP>::BYTES];  // rows in row_of's order
  char q[MODE == OUT && !TURN ? NP : 1][MODE == OUT && !TURN ? Tokens<KP>::BYTES : 16];
  Record<MODE == OUT ? 2 : 1, 64 * NW> rec;
};

// NW waves of 16 columns over a segment's chunks. OUT: the forward's. KEEP: the backward's, which wants
// every chunk's first state and Z rather than O. SUM: a segment's last state from zeros (the first
// segment's from its own) and, as further columns that start as the unit matrix without values, its
// map of the state; SUM_BWD: the map's transpose too.
template <typename T, int KP, int NW, bool VEC, int MODE>
__global__ __launch_bounds__(64 * NW, (WALKS<WalkLds<KP, PARTS<T>, NW, MODE>>)) void delta_walk_kernel(DeltaArgs a) {
  constexpr int NP = PARTS<T>, KB = KP / 32, KT = KP / 16, THREADS = 64 * NW;
  constexpr int PIECES = KP / 8, ITEMS = (CH * PIECES + THREADS - 1) / THREADS;
  constexpr int STRIDE = MODE == KEEP || MODE == SUM_BWD ? REC_BWD : REC, USED = MODE == OUT ? REC : REC_P;
  extern __shared__ __attribute__((aligned(16))) char lds_raw[];
  typedef WalkLds<KP, NP, NW, MODE> Lds;
  typedef Tokens<KP> Tk;
  constexpr bool TURN = Lds::TURN;
  static_assert(sizeof(Lds) <= 160 * 1024, "LDS of a CU");
  Lds& lds = *reinterpret_cast<Lds*>(lds_raw);
  char(*const lds_q)[Tk::BYTES] = reinterpret_cast<char(*)[Tk::BYTES]>(TURN ? lds.k[0] : lds.q[0]);
  const int tid = threadIdx.x, lane = tid & 63, w = wave_number(), n = lane & 15, g = lane >> 4;
  const int rows_at = Tk::lane_at(n, g), cols_at = Tk::lane_at_t(n, g);
  const int Dk = (int)a.Dk, Dv = (int)a.Dv, VP = (int)a.VP, qs = (int)a.Hk * Dk, vs = (int)a.Hv * Dv;
  const uint32_t v_groups = (Dv + 16 * NW - 1) / (16 * NW);
  const Part part(a, v_groups + (MODE >= SUM ? KP / (16 * NW) : 0));
  const bool unit = MODE >= SUM && part.group >= (int)v_groups;
  if (part.empty() || (MODE >= SUM && (part.ends() || (unit && part.seg == 0)))) return;
  const int64_t bh = part.bh, len = part.len;
  const int col = (part.group - (unit ? (int)v_groups : 0)) * 16 * NW + 16 * w;
  const int have = unit ? 0 : min(16, Dv - col);  // columns of values; may be none
  const int64_t keys = part.b * a.S * qs + part.hk * Dk, values = part.b * a.S * vs + part.hv * Dv + col;
  const char* rec = (const char*)a.rec + bh * a.NC * STRIDE;
  const uint32_t v_lane = n < have ? (8 * g * vs + n) * (uint32_t)sizeof(T) : NOWHERE;
  const uint32_t o_lane = n < have ? (4 * g * vs + n) * (uint32_t)sizeof(T) : NOWHERE;

  State<KP> S;
  if (unit) {
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) S.m[t][r] = row_of(t, 4 * g + r) == col + n ? 1.f : 0.f;
  } else {
    // Where the last state is written over the first, the last segment may end before the first one
    // begins: that one takes the copy that SUM made in the slot of a head's last segment, which has no
    // other use in the forward.
    const bool copied = (MODE == OUT || MODE == SUM) && part.seg == 0 && a.state0 && a.state0 == a.state1 && !part.ends();
    float* copy = a.slots + (copied ? (bh * a.NS + a.NS - 1) * Dk * Dv + col : 0);
    const float* from = part.seg != 0 ? (MODE >= SUM ? nullptr : a.slots + (part.slot - 1) * Dk * Dv + col)
                        : copied && MODE == OUT ? copy : a.state0 ? a.state0 + bh * Dk * Dv + col : nullptr;
    S.load(from, Dk, Dv, n, g, have);
    if (copied && MODE == SUM) S.store(copy, Dk, Dv, n, g, have);
  }

  // the next chunk's operands, which a bfloat16 chunk waits for before it begins (see above)
  Raw8<T> kr[ITEMS], qr[ITEMS];
  typename decltype(lds.rec)::Raw rr;
  float vr[4][4];
  const auto fetch = [&](int64_t c) {
    const int left = (int)min((int64_t)CH, len - c * CH);
    const Range kc = head_rows((const T*)a.k + keys + c * CH * qs, left, qs, Dk);
    const Range qc = head_rows((const T*)a.q + keys + c * CH * qs, left, qs, Dk);
    const Range vc = head_rows((const T*)a.v + values + c * CH * vs, have > 0 ? left : 0, vs, have);
    const Range rc(rec + c * STRIDE, USED);
    const uint32_t vl = anew(v_lane);
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int x = i * THREADS + tid, piece = x % PIECES, row = x / PIECES;
      const uint32_t o = (row * qs + 8 * piece) * (uint32_t)sizeof(T);
      kr[i].template load<VEC>(kc, o, Dk - 8 * piece);
      if (MODE == OUT) qr[i].template load<VEC>(qc, o, Dk - 8 * piece);
    }
    rr.load(rc, REC_T, tid);
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) vr[t][r] = vc.get((const T*)nullptr, vl + row_of(t, r) * vs * (uint32_t)sizeof(T));
  };
  const auto put = [&](char(*m)[Tk::BYTES], const Raw8<T>(&raw)[ITEMS], bool in_order) {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int x = i * THREADS + tid, piece = x % PIECES, row = x / PIECES;
      if (CH * PIECES % THREADS == 0 || row < CH) {
        const Op<NP> o = raw[i].template op<NP>();
#pragma unroll
        for (int p = 0; p < NP; ++p) *reinterpret_cast<bf8_t*>(m[p] + Tk::at(in_order ? row : place_of(row), piece)) = o.p[p];
      }
    }
  };
  if (part.first < part.last) fetch(part.first);
  for (int64_t c = part.first; c < part.last; ++c) {
    if (!TURN) put(lds.k, kr, false);
    if (MODE == OUT) put(lds_q, qr, true);
    lds.rec.put(rr, tid);
    f4_t v[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) v[t] = f4_t{vr[t][0], vr[t][1], vr[t][2], vr[t][3]};
    lds_barrier();
    if (!TURN && c + 1 < part.last) fetch(c + 1);
    if (MODE == KEEP) S.keep((float*)a.states + (bh * a.NC + c) * KP * VP, VP, col, n, g);

    // K M and Q M
    f4_t x[4], o[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) x[t] = o[t] = f4_t{0.f, 0.f, 0.f, 0.f};
    const auto by_state = [&](bool by_k, bool by_q) {
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        const Fine sf = split<3>(S.m[2 * kb], S.m[2 * kb + 1]);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          Op<NP> ka, qa;
#pragma unroll
          for (int p = 0; p < NP; ++p) {
            if (by_k) ka.p[p] = Tk::rows(lds.k[p], rows_at, t, kb);
            if (by_q) qa.p[p] = Tk::rows(lds_q[p], rows_at, t, kb);
          }
          if (by_k) x[t] = mma(ka, sf, x[t]);
          if (by_q) o[t] = mma(qa, sf, o[t]);
        }
        keep_order();
      }
    };
    by_state(!TURN, MODE == OUT);
    if (TURN) {
      lds_barrier();
      put(lds.k, kr, false);
      lds_barrier();
      if (c + 1 < part.last) fetch(c + 1);
      by_state(true, false);
    }
    // R = V - exp(G) K M, Z = T R, X = beta Z
    const float* dec = lds.rec.dec;
    Fine f[2];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      x[t] = v[t] - *reinterpret_cast<const f4_t*>(dec + DEC_AHEAD + row_of(t, 4 * g)) * x[t];
    }
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) f[kb] = split<3>(x[2 * kb], x[2 * kb + 1]);
#pragma unroll
    for (int t = 0; t < 4; ++t) x[t] = f4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
#pragma unroll
      for (int t = 2 * kb; t < 4; ++t) x[t] = mma(lds.rec.tile(0, tri(t, kb), lane), f[kb], x[t]);
      keep_order();
    }
    if (MODE == KEEP) keep_rows((float*)a.z + (bh * a.NC + c) * CH * VP, VP, col, n, g, x);
#pragma unroll
    for (int t = 0; t < 4; ++t) x[t] *= *reinterpret_cast<const f4_t*>(dec + DEC_BETA + row_of(t, 4 * g));
    if (MODE == OUT) {  // O = scale (exp(G) Q M + P X)
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) f[kb] = split<3>(x[2 * kb], x[2 * kb + 1]);
      const Range oc = head_rows((T*)a.o + values + c * CH * vs, have > 0 ? (int)min((int64_t)CH, len - c * CH) : 0, vs, have);
      const uint32_t ol = anew(o_lane);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        o[t] *= *reinterpret_cast<const f4_t*>(dec + DEC_AHEAD + 16 * t + 4 * g);
#pragma unroll
        for (int kb = 0; kb <= (t >> 1); ++kb) o[t] = mma(lds.rec.tile(1, tri(t, kb), lane), f[kb], o[t]);
#pragma unroll
        for (int r = 0; r < 4; ++r)
          oc.put((T*)nullptr, ol + (16 * t + r) * vs * (uint32_t)sizeof(T), a.scale * o[t][r]);
        keep_order();
      }
    }
    // M = exp(G_end) M + K^T (exp(G_end - G) X)
#pragma unroll
    for (int t = 0; t < 4; ++t) x[t] *= *reinterpret_cast<const f4_t*>(dec + DEC_TO_END + row_of(t, 4 * g));
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) f[kb] = split<3>(x[2 * kb], x[2 * kb + 1]);
    const float whole = dec[DEC_AHEAD + CH - 1];
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      S.m[t] *= whole;
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        Op<NP> ka;
#pragma unroll
        for (int p = 0; p < NP; ++p) ka.p[p] = Tk::cols(lds.k[p], cols_at, t, kb);
        S.m[t] = mma(ka, f[kb], S.m[t]);
      }
      if (t & 1) keep_order();
    }
    lds_barrier();
  }
  if (MODE == OUT && a.state1 && part.ends()) S.store(a.state1 + bh * Dk * Dv + col, Dk, Dv, n, g, have);
  if (MODE >= SUM) {
    if (!unit) {
      S.store(a.slots + part.slot * Dk * Dv + col, Dk, Dv, n, g, have);
      return;
    }
    S.keep((bf16_t*)a.phi + part.slot * 3 * KP * KP, col, n, g);
    if (MODE == SUM_BWD) {
      const Range m((bf16_t*)a.phi_t + part.slot * 3 * KP * KP, 6 * KP * KP);
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        const Fine s = split<3>(S.m[2 * kb], S.m[2 * kb + 1]);
        const uint32_t o = 2 * ((col + n) * KP + 32 * kb + 8 * g);
#pragma unroll
        for (int p = 0; p < 3; ++p) m.put_quad(o + p * 2 * KP * KP, __builtin_bit_cast(u4_t, s.p[p]));
      }
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
  const uint32_t groups = ((uint32_t)a.Dv + 31) / 32;
  const int64_t bh = blockIdx.x / groups, b = (uint32_t)bh / (uint32_t)a.Hv;
  const int64_t hv = (uint32_t)bh % (uint32_t)a.Hv, hk = (uint32_t)hv / ((uint32_t)a.Hv / (uint32_t)a.Hk);
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
    lds_barrier();
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
    lds_barrier();
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

// ----------------------------------------------------------------- the segments

// M_{s+1} = Phi_s M_s + N_s over a head's segments, 16 columns of the state by a workgroup; the slots'
// N become the states. A wave has 32 rows of the state, the operand block that the next step's
// products take from all of them through LDS; its rows of the next two steps' Phi and N are on their
// way meanwhile. A chain of products whose maps come from other dies' caches, 96 KB a step in three parts: 51 us
// for 16 heads of 16 segments (128 x 128); of two parts 34, and then 40 with a head's columns spread over the
// dies and one step ahead, 103 with one wave for all rows. BACK: the gradients, from the last segment on, with
// Phi's transpose.
template <int KP, bool BACK>
__global__ __launch_bounds__(2 * KP) void delta_join_kernel(DeltaArgs a) {
  constexpr int KB = KP / 32;
  __shared__ __attribute__((aligned(16))) char lds[2][KB][3][TILE];
  const int lane = threadIdx.x & 63, w = wave_number(), n = lane & 15, g = lane >> 4;
  const int Dk = (int)a.Dk, Dv = (int)a.Dv;
  const Place at((uint32_t)(a.B * a.Hv), ((uint32_t)Dv + 15) / 16);
  const int64_t bh = at.unit, b = at.unit / (uint32_t)a.Hv;
  const int col = (int)at.member * 16, have = min(16, Dv - col);
  const int64_t chunks = (length_of(a.lengths, b, a.S) + CH - 1) / CH, state = (int64_t)Dk * Dv;
  const int segs = (int)((chunks + a.SL - 1) / a.SL);  // that hold tokens
  float* slots = a.slots + bh * a.NS * state + col;
  const bf16_t* maps = (const bf16_t*)(BACK ? a.phi_t : a.phi) + bh * a.NS * 3 * KP * KP;
  if (segs < 3) return;  // the second segment's state is the first's last one
  const auto seg = [&](int i) { return BACK ? segs - 1 - i : i; };
  const uint32_t s_lane = n < have ? 4 * ((32 * w + 8 * g) * Dv + n) : NOWHERE;
  const uint32_t m_lane = 2 * ((8 * (n >> 2) + (n & 3)) * KP + 8 * g);
  constexpr int AHEAD = KP == 256 ? 1 : 2;  // steps whose maps are on their way, as there are registers
  Fine m[AHEAD][2][KB];
  float add[AHEAD][8];
  const auto load_slot = [&](int i, float (&v)[8]) {
    const Range r(slots + seg(i) * state, ((int64_t)(Dk - 1) * Dv + have) * 4);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = r.get((const float*)nullptr, s_lane + 4 * e * Dv);
  };
  const auto fetch = [&](int i, int x) {
    const Range r(maps + seg(i) * (int64_t)3 * KP * KP, 6 * KP * KP);
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) m[x][t][kb] = r.parts(m_lane, 2 * ((32 * w + 4 * t) * KP + 32 * kb), 2 * KP * KP);
    load_slot(i, add[x]);
  };
  float S[8];  // rows 32 w + 8 g + 0 .. 7
  load_slot(0, S);
  const auto step = [&](int i, int x) {
    const Fine own = split<3>(S);
    char* mine = lds[i & 1][w][0] + lane * 16;
#pragma unroll
    for (int p = 0; p < 3; ++p) *reinterpret_cast<bf8_t*>(mine + p * TILE) = own.p[p];
    lds_barrier();
    f4_t o[2] = {{add[x][0], add[x][1], add[x][2], add[x][3]}, {add[x][4], add[x][5], add[x][6], add[x][7]}};
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      const char* p = lds[i & 1][kb][0] + lane * 16;
      const Fine f = {*reinterpret_cast<const bf8_t*>(p), *reinterpret_cast<const bf8_t*>(p + TILE),
                      *reinterpret_cast<const bf8_t*>(p + 2 * TILE)};
#pragma unroll
      for (int t = 0; t < 2; ++t) o[t] = mma(m[x][t][kb], f, o[t]);
    }
    if (i + AHEAD < segs - 1) fetch(i + AHEAD, x);
    const Range r(slots + seg(i) * state, ((int64_t)(Dk - 1) * Dv + have) * 4);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      S[e] = o[e >> 2][e & 3];
      r.put((float*)nullptr, s_lane + 4 * e * Dv, S[e]);
    }
  };
  fetch(1, 0);
  if (AHEAD == 2 && segs > 3) fetch(2, 1);
  for (int i = 1; i < segs - 1; i += AHEAD) {
    step(i, 0);
    if (AHEAD == 2 && i + 1 < segs - 1) step(i + 1, 1);
  }
}

// Tokens up to which they are taken one by one, rather than as a chunk: 6 tokens of 32 heads of 128 x 128
// take 20 us against 24, of 256 heads 21 against 24 and of 2,048 heads 114 against 111; 8 tokens 19
// against 24, 26 against 24 and 144 against 111 (whole calls, bfloat16).
constexpr int SHORT = 6;

// Four waves a workgroup, 64 columns, measured with two parts: 572 us for 8,192 tokens of 16 heads in one walk and 129 for 8 x 1,024
// against 671 and 136 with eight waves, which share keys and queries but wait for each other.
template <typename T, int KP, int MODE>
hipError_t walk_go(const DeltaArgs& a, hipStream_t st) {
  constexpr int NW = 4;
  const size_t lds = sizeof(WalkLds<KP, PARTS<T>, NW, MODE>);
  const unsigned groups = (unsigned)((a.Dv + 16 * NW - 1) / (16 * NW)) + (MODE >= SUM ? KP / (16 * NW) : 0);
  const dim3 grid((unsigned)(a.B * a.Hv * a.NS) * groups);
  const auto go = [&](auto kernel) {
    if (lds > 64 * 1024) {
      hipError_t e = hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
      if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(kernel, grid, dim3(64 * NW), lds, st, a);
    return hipGetLastError();
  };
  return a.vec ? go(delta_walk_kernel<T, KP, NW, true, MODE>) : go(delta_walk_kernel<T, KP, NW, false, MODE>);
}

template <typename T, int KP, int MODE>
hipError_t delta_go(const DeltaArgs& a, hipStream_t st) {
  if (MODE == OUT && a.S <= SHORT) {
    const dim3 grid((unsigned)(a.B * a.Hv * ((a.Dv + 31) / 32)));
    if (a.vec4) hipLaunchKernelGGL((delta_step_kernel<T, KP, true>), grid, dim3(256), 0, st, a);
    else hipLaunchKernelGGL((delta_step_kernel<T, KP, false>), grid, dim3(256), 0, st, a);
    return hipGetLastError();
  }
  const dim3 prep((unsigned)(a.B * a.Hv * a.NC));
  if (a.vec) hipLaunchKernelGGL((delta_prep_kernel<T, KP, true, MODE == KEEP>), prep, dim3(256), 0, st, a);
  else hipLaunchKernelGGL((delta_prep_kernel<T, KP, false, MODE == KEEP>), prep, dim3(256), 0, st, a);
  hipError_t e = hipGetLastError();
  if (e == hipSuccess && a.NS > 1) {
    e = walk_go<T, KP, MODE == KEEP ? SUM_BWD : SUM>(a, st);
    if (e == hipSuccess) e = launch_delta_join(false, a, st);
  }
  return e == hipSuccess ? walk_go<T, KP, MODE>(a, st) : e;
}

template <typename T, int MODE>
hipError_t delta_by_width(const DeltaArgs& a, hipStream_t st) {
  if (a.Dk <= 64) return delta_go<T, 64, MODE>(a, st);
  if (a.Dk <= 128) return delta_go<T, 128, MODE>(a, st);
  return delta_go<T, 256, MODE>(a, st);
}

template <bool BACK>
void join_go(const DeltaArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)(a.B * a.Hv * ((a.Dv + 15) / 16)));
  if (a.Dk <= 64) hipLaunchKernelGGL((delta_join_kernel<64, BACK>), grid, dim3(128), 0, st, a);
  else if (a.Dk <= 128) hipLaunchKernelGGL((delta_join_kernel<128, BACK>), grid, dim3(256), 0, st, a);
  else hipLaunchKernelGGL((delta_join_kernel<256, BACK>), grid, dim3(512), 0, st, a);
}

}  // namespace

int64_t delta_plan(DeltaArgs& a, bool backward, void* ws) {
  const int64_t KP = a.Dk <= 64 ? 64 : a.Dk <= 128 ? 128 : 256, heads = a.B * a.Hv;
  a.NC = (a.S + CH - 1) / CH;
  a.VP = (a.Dv + 31) / 32 * 32;
  a.NS = 1;
  a.SL = a.NC;
  // Workgroups that walk whole sequences. Where they are few for 256 CUs of two each, every sequence is cut
  // into segments of 4 chunks and more, as many as fill the CUs, walked at once from zeros, with their maps
  // of the state, joined, and walked again from their own states: twice the work and the join. One walk
  // against segments, us, forward and backward (bfloat16, whole calls):
  //   eight segments and more fill the CUs: 1,024 tokens of 16 heads of 128 x 128 97 : 68 and 205 : 161, of 32
  //   heads 101 : 80 and 236 : 207, 16 heads of 256 x 256 142 : 119 and 388 : 355; at 512 tokens 55 : 55 and
  //   128 : 137;
  //   four to seven: 1,024 tokens of 64 heads 108 : 119 and 328 : 368, 2,048 208 : 203 and 668 : 663, 4,096
  //   450 : 395 and 1,332 : 1,220; maps of 256 keys cost more: 24 heads, 2,048 tokens 277 : 312 and 1,004 : 1,068,
  //   4,096 557 : 506 and 2,009 : 1,893; 32 heads (four) 588 : 644 and 2,254 : 2,353;
  //   two or three: 128 heads of 128 x 128, 2,048 tokens 275 : 370 and 1,011 : 1,197.
  const int64_t wide = heads * ((a.Dv + 63) / 64), fill = wide > 0 ? 512 / wide : 0;
  if (fill >= (KP == 256 ? 5 : 4) && a.NC >= (fill >= 8 ? 16 : KP == 256 ? 64 : 32)) {
    const int64_t most = fill < a.NC / 4 ? fill : a.NC / 4;
    a.SL = (a.NC + most - 1) / most;
    a.NS = (a.NC + a.SL - 1) / a.SL;
  }
  if (!backward && a.S <= SHORT) return 0;
  int64_t at = 0;
  const auto take = [&](int64_t bytes) {
    char* p = (char*)ws + at;
    at += (bytes + 255) / 256 * 256;
    return (void*)p;
  };
  a.rec = take(heads * a.NC * (backward ? REC_BWD : REC));
  if (a.NS > 1) {
    a.slots = (float*)take(heads * a.NS * a.Dk * a.Dv * 4);
    a.phi = take(heads * a.NS * 6 * KP * KP);
    if (backward) a.phi_t = take(heads * a.NS * 6 * KP * KP);
  }
  if (backward) {
    const int64_t n = heads * a.NC;
    a.states = take(n * 4 * KP * a.VP);
    a.dstates = take(n * 4 * KP * a.VP);
    a.z = take(n * 4 * CH * a.VP);
    a.w = take(n * 4 * CH * a.VP);
  }
  return at;
}

hipError_t launch_delta(int dtype, const DeltaArgs& a, hipStream_t st) {
  return dtype == 0 ? delta_by_width<float, OUT>(a, st) : delta_by_width<bf16_t, OUT>(a, st);
}

hipError_t launch_delta_keep(int dtype, const DeltaArgs& a, hipStream_t st) {
  return dtype == 0 ? delta_by_width<float, KEEP>(a, st) : delta_by_width<bf16_t, KEEP>(a, st);
}

hipError_t launch_delta_join(bool back, const DeltaArgs& a, hipStream_t st) {
  if (back) join_go<true>(a, st);
  else join_go<false>(a, st);
  return hipGetLastError();
}

}  // namespace hc
