// Gated delta rule, backward. With the forward's chunk (hc_delta.hip), d = scale dO and N the gradient
// of the state behind the chunk:
//   dX = P^T d + exp(G_end - G) K N,   W = T^T (beta dX) = dV,
//   dM = exp(G_end) N + (exp(G) Q)^T d - (exp(G) K)^T W   (the gradient of the state before it),
//   B = (d X^T) exp(G_i - G_j) (j <= i),   A = -(W X^T) exp(G_i - G_j) (j < i),
//   dQ = exp(G) d M^T + B K,
//   dK = [-exp(G) W M^T + A K] + [exp(G_end - G) X N^T + B^T Q + A^T K]   (as read, as written),
//   dbeta_j = Z_j . dX_j - sum_i exp(G_i - G_j) (k_i . k_j) (W_i . Z_j),
//   dg_t = sum_{i >= t} exp(G_i) [d_i . (M^T q_i) - W_i . (M^T k_i)] + sum_{j < t} exp(G_end - G_j) X_j . (N^T k_j)
//        + exp(G_end) <M, N> + sum_{i >= t > j} c_ij,  c_ij = (P_ij d_i - exp(G_i - G_j) (k_i . k_j) W_i) . X_j:
//        all that passes over token t, each with its own decay, so that what is forgotten leaves no
//        rounding behind. (q . dq - v . dv summed over the later tokens is the same, and was off by
//        4 x 10^-5 in heads that forget fast.) The pairs as a running sum of what starts at a token less what
//        ends there, the same c_ij in both.
// The forward's walk is run again and keeps every chunk's M and Z; a second walk from the end back
// keeps N and W and writes dV; then every chunk forms the rest by itself, all value heads of a key
// head in one workgroup, so that dQ and dK are summed in registers and in a fixed order.
// Every factor keeps float32's 24 bits, in three bfloat16 parts: gradients are as near the definition as a float32
// form's (2 to 4 x 10^-7 of their norm; with two parts 3 to 6 x 10^-6, the whole call 5 % faster).
//   2,048 chunks of 128 x 128 (2 x 4,096 tokens, 16 value heads on 8 key heads, bfloat16), with segments: the
// forward's part 255 us (the chunks 52, segments from zeros 96, joins 26, the walk that keeps states 80), the walks
// back 218 (80, 28, 110), the chunks' own part 262. That one reads the states that the
// walks kept, 64 KB a chunk and direction in float32, and Z and W three times, for the pairs and for each 64 keys (400 MB
// kept, 600 MB of reads at 2.4 TB/s), on one workgroup a CU, whose registers hold dQ and dK; its
// steps wait for memory and barriers.
#include "hc_delta_device.h"

namespace hc {

namespace {

template <int KP, int NP, int NW>
struct BackLds {
  static constexpr bool TURN = NP == 3 && KP == 256;  // no room for both: queries after keys, in k
  char k[NP][Tokens<KP>::BYTES], q[TURN ? 1 : NP][TURN ? 16 : Tokens<KP>::BYTES];  // rows in row_of's order
  Record<2, 64 * NW> rec;  // P's transpose and T's
};

// FULL: as above, over a segment's chunks. Otherwise a segment's first gradient from zeros (the last
// segment's from its own), nothing else.
template <typename T, int KP, int NW, bool VEC, bool FULL>
__global__ __launch_bounds__(64 * NW, (WALKS<BackLds<KP, PARTS<T>, NW>>)) void delta_back_kernel(DeltaArgs a) {
  constexpr int NP = PARTS<T>, KB = KP / 32, KT = KP / 16, THREADS = 64 * NW;
  constexpr int PIECES = KP / 8, ITEMS = (CH * PIECES + THREADS - 1) / THREADS;
  extern __shared__ __attribute__((aligned(16))) char lds_raw[];
  typedef BackLds<KP, NP, NW> Lds;
  typedef Tokens<KP> Tk;
  constexpr bool TURN = Lds::TURN;
  static_assert(sizeof(Lds) <= 160 * 1024, "LDS of a CU");
  Lds& lds = *reinterpret_cast<Lds*>(lds_raw);
  char(*const lds_q)[Tk::BYTES] = reinterpret_cast<char(*)[Tk::BYTES]>(TURN ? lds.k[0] : lds.q[0]);
  const int tid = threadIdx.x, lane = tid & 63, w = wave_number(), n = lane & 15, g = lane >> 4;
  const int rows_at = Tk::lane_at(n, g), cols_at = Tk::lane_at_t(n, g);
  const int Dk = (int)a.Dk, Dv = (int)a.Dv, VP = (int)a.VP, qs = (int)a.Hk * Dk, vs = (int)a.Hv * Dv;
  const Part part(a, ((uint32_t)Dv + 16 * NW - 1) / (16 * NW));
  const int64_t bh = part.bh, len = part.len;
  const int col = part.group * 16 * NW + 16 * w, have = min(16, Dv - col);  // columns; may be none
  const int64_t keys = part.b * a.S * qs + part.hk * Dk, values = part.b * a.S * vs + part.hv * Dv + col;
  if (FULL && part.ends() && n < have) {  // nothing reaches the tokens behind the sequence's length
    const int64_t from = max(len, part.first * CH), to = min(a.S, (part.first + a.SL) * CH);
    for (int64_t t = from + g; t < to; t += 4) Elem<T>::st((T*)a.dv + values + t * vs + n, 0.f);
  }
  if (part.empty() || (!FULL && part.seg == 0)) return;
  const char* rec = (const char*)a.rec + bh * a.NC * REC_BWD;
  const uint32_t v_lane = n < have ? (8 * g * vs + n) * (uint32_t)sizeof(T) : NOWHERE;

  State<KP> D;
  {
    const float* from = part.ends() ? a.dlast + (a.dlast ? bh * Dk * Dv : 0) : FULL ? a.slots + (part.slot + 1) * Dk * Dv : nullptr;
    D.load(from ? from + col : nullptr, Dk, Dv, n, g, have);
  }

  Raw8<T> kr[ITEMS], qr[ITEMS];
  typename decltype(lds.rec)::Raw rr;
  float dr[4][4];
  const auto fetch_tokens = [&](Raw8<T>(&raw)[ITEMS], const void* from, int64_t c) {
    const Range m = head_rows((const T*)from + keys + c * CH * qs, (int)min((int64_t)CH, len - c * CH), qs, Dk);
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int x = i * THREADS + tid, piece = x % PIECES, row = x / PIECES;
      raw[i].template load<VEC>(m, (row * qs + 8 * piece) * (uint32_t)sizeof(T), Dk - 8 * piece);
    }
  };
  const auto fetch = [&](int64_t c) {  // all but the queries
    const int left = (int)min((int64_t)CH, len - c * CH);
    const Range dc = head_rows((const T*)a.d_o + values + c * CH * vs, have > 0 ? left : 0, vs, have);
    const uint32_t vl = anew(v_lane);
    fetch_tokens(kr, a.k, c);
    rr.load(Range(rec + c * REC_BWD, REC_BWD), REC_P, tid);
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) dr[t][r] = dc.get((const T*)nullptr, vl + row_of(t, r) * vs * (uint32_t)sizeof(T));
  };
  const auto put = [&](char(*m)[Tk::BYTES], const Raw8<T>(&raw)[ITEMS]) {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int x = i * THREADS + tid, piece = x % PIECES, row = x / PIECES;
      if (CH * PIECES % THREADS == 0 || row < CH) {
        const Op<NP> o = raw[i].template op<NP>();
#pragma unroll
        for (int p = 0; p < NP; ++p) *reinterpret_cast<bf8_t*>(m[p] + Tk::at(place_of(row), piece)) = o.p[p];
      }
    }
  };
  if (part.first < part.last) {
    fetch_tokens(qr, a.q, part.last - 1);
    fetch(part.last - 1);
  }
  for (int64_t c = part.last - 1; c >= part.first; --c) {
    put(lds.k, kr);
    if (!TURN) put(lds_q, qr);
    lds.rec.put(rr, tid);
    f4_t d[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) d[t] = f4_t{dr[t][0], dr[t][1], dr[t][2], dr[t][3]};
    lds_barrier();
    if (c > part.first) {
      if (!TURN) fetch_tokens(qr, a.q, c - 1);
      fetch(c - 1);
    }
    if (FULL) D.keep((float*)a.dstates + (bh * a.NC + c) * KP * VP, VP, col, n, g);

    f4_t x[4];  // K N
#pragma unroll
    for (int t = 0; t < 4; ++t) x[t] = f4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      const Fine sf = split<3>(D.m[2 * kb], D.m[2 * kb + 1]);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        Op<NP> ka;
#pragma unroll
        for (int p = 0; p < NP; ++p) ka.p[p] = Tk::rows(lds.k[p], rows_at, t, kb);
        x[t] = mma(ka, sf, x[t]);
      }
      keep_order();
    }
    const float* dec = lds.rec.dec;
    // beta dX, dX = scale P^T dO + exp(G_end - G) K N
    {
      Op<NP> df[2];
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) df[kb] = split<NP>(d[2 * kb], d[2 * kb + 1]);  // bfloat16 is its own high part
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        f4_t p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kb = t >> 1; kb < 2; ++kb) p = mma(lds.rec.tile(0, tri_t(t, kb), lane), df[kb], p);
        const f4_t to_end = *reinterpret_cast<const f4_t*>(dec + DEC_TO_END + row_of(t, 4 * g));
        const f4_t beta = *reinterpret_cast<const f4_t*>(dec + DEC_BETA + row_of(t, 4 * g));
        x[t] = beta * (a.scale * p + to_end * x[t]);
      }
      keep_order();
    }
    // W = T^T (beta dX)
    Fine f[2], wf[2];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) f[kb] = split<3>(x[2 * kb], x[2 * kb + 1]);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      x[t] = f4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int kb = t >> 1; kb < 2; ++kb) x[t] = mma(lds.rec.tile(1, tri_t(t, kb), lane), f[kb], x[t]);
    }
    keep_order();
    if (FULL) {
      const Range vc = head_rows((T*)a.dv + values + c * CH * vs, have > 0 ? (int)min((int64_t)CH, len - c * CH) : 0, vs, have);
      const uint32_t vl = anew(v_lane);
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) vc.put((T*)nullptr, vl + row_of(t, r) * vs * (uint32_t)sizeof(T), x[t][r]);
      keep_rows((float*)a.w + (bh * a.NC + c) * CH * VP, VP, col, n, g, x);
    }
    // the gradient of the state before the chunk
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const f4_t ahead = *reinterpret_cast<const f4_t*>(dec + DEC_AHEAD + row_of(t, 4 * g));
      x[t] *= -ahead;
      d[t] *= a.scale * ahead;
    }
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      wf[kb] = split<3>(x[2 * kb], x[2 * kb + 1]);
      f[kb] = split<3>(d[2 * kb], d[2 * kb + 1]);
    }
    const float whole = dec[DEC_AHEAD + CH - 1];
    keep_order();
    const auto add = [&](bool by_q, bool by_k) {  // (exp(G) Q)^T dO, -(exp(G) K)^T W
#pragma unroll
      for (int t = 0; t < KT; ++t) {
        if (by_k) D.m[t] *= whole;
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
          Op<NP> ka, qa;
#pragma unroll
          for (int p = 0; p < NP; ++p) {
            if (by_k) ka.p[p] = Tk::cols(lds.k[p], cols_at, t, kb);
            if (by_q) qa.p[p] = Tk::cols(lds_q[p], cols_at, t, kb);
          }
          if (by_q) D.m[t] = mma(qa, f[kb], D.m[t]);
          if (by_k) D.m[t] = mma(ka, wf[kb], D.m[t]);
        }
        keep_order();
      }
    };
    add(!TURN, true);
    if (TURN) {
      lds_barrier();
      put(lds_q, qr);
      lds_barrier();
      if (c > part.first) fetch_tokens(qr, a.q, c - 1);
      add(true, false);
    }
    lds_barrier();
  }
  float* to = !FULL ? a.slots + part.slot * Dk * Dv : part.seg == 0 && a.dstate0 ? a.dstate0 + bh * Dk * Dv : nullptr;
  if (to) D.store(to + col, Dk, Dv, n, g, have);
}

// ------------------------------------------------------------- each chunk by itself

// What each chunk's workgroup of four waves, 16 tokens each, brings through LDS, in turn in NBUF
// buffers: Z, W (three parts each) and dO, 64 tokens by COLS columns, and then the state and its gradient
// (three parts each), 64 keys by COLS columns. Each step waits for memory once: steps of 32 columns
// took 277 us for 2,048 chunks of 128 x 128 where 64 took 226 (with two parts), so these where there is room.
// Of 256 float32 keys and queries LDS holds KL = 128 at a time.
template <int KP, int NP>
struct GradLds {
  static constexpr int KL = NP == 3 && KP == 256 ? 128 : KP;
  static constexpr int COLS = KL == 128 && NP == 3 ? 32 : 64, PIECES = COLS / 8, PART = CH * COLS * 2;
  static constexpr int NBUF = NP == 1 && KP <= 128 ? 2 : 1;
  char k[NP][Tokens<KL>::BYTES], q[NP][Tokens<KL>::BYTES];  // rows in row_of's order
  char buf[NBUF][(6 + NP) * PART];
  double G[CH];
  float beta[CH], read[CH], late[CH], row[4][CH], end[4];
  // a row's place in row_of's order, its 16-byte pieces exchanged so that 16 lanes reading a piece of 16 rows
  // reach all banks
  static __device__ __forceinline__ int at(int place, int piece) {
    return COLS == 64 ? Tokens<64>::at(place, piece) : place * 64 + ((piece ^ ((place >> 2) & 3)) << 4);
  }
  // an operand of tile `tile` (64-byte k block kb), the lane's own part at `at`
  static __device__ __forceinline__ bf8_t one(const char* m, int part, int at, int tile, int kb) {
    return *reinterpret_cast<const bf8_t*>(m + part * PART + 32 * COLS * tile + (at ^ (kb << 6)));
  }
  static __device__ __forceinline__ void put(char* m, int part, int at, const F8& v) {
    const Fine s = split<3>(v.a, v.b);
#pragma unroll
    for (int p = 0; p < 3; ++p) *reinterpret_cast<bf8_t*>(m + (part + p) * PART + at) = s.p[p];
  }
  static __device__ __forceinline__ Fine fine(const char* m, int part, int at, int tile, int kb) {
    return {one(m, part, at, tile, kb), one(m, part + 1, at, tile, kb), one(m, part + 2, at, tile, kb)};
  }
  static __device__ __forceinline__ Op<NP> stream(const char* m, int part, int at, int tile, int kb) {
    Op<NP> d;
#pragma unroll
    for (int p = 0; p < NP; ++p) d.p[p] = one(m, part + p, at, tile, kb);
    return d;
  }
};

// Eight elements at byte offset o, the first `cnt` of them (VEC: all or none).
template <bool VEC>
__device__ __forceinline__ void put_row8(bf16_t* p, const Range& m, uint32_t o, int cnt, const float v[8]) {
  if (VEC) {
    m.put_quad(cnt > 0 ? o : NOWHERE, pack8(v));
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) m.put(p, e < cnt ? o + 2 * e : NOWHERE, v[e]);
  }
}

template <bool VEC>
__device__ __forceinline__ void put_row8(float* p, const Range& m, uint32_t o, int cnt, const float v[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (VEC) {
      m.put_quad(cnt > 0 ? o + 16 * h : NOWHERE, __builtin_bit_cast(u4_t, f4_t{v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]}));
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) m.put(p, 4 * h + e < cnt ? o + 16 * h + 4 * e : NOWHERE, v[4 * h + e]);
    }
  }
}

__device__ __forceinline__ float sum_groups(float v) {  // over the four lanes of a token
  v += __shfl_xor(v, 16, 64);
  return v + __shfl_xor(v, 32, 64);
}

// SHARED: several value heads read a key head. Up to 128 keys at a time, for which there are registers:
// wider heads take two passes, the second of which adds to the first's dg and dbeta.
template <typename T, int KP, bool VEC, bool SHARED>
__global__ __launch_bounds__(256) void delta_grad_kernel(DeltaArgs a) {
  constexpr int NP = PARTS<T>, QUADS = KP == 64 ? 1 : 2, PASSES = KP / 64 / QUADS;
  typedef GradLds<KP, NP> Lds;
  constexpr int KL = Lds::KL, PIECES = KL / 8, ITEMS = CH * PIECES / 256;
  constexpr int KB = KL / 32;
  constexpr bool HALVES = KL < KP;
  typedef Tokens<KL> Tk;
  extern __shared__ __attribute__((aligned(16))) char lds_raw[];
  static_assert(sizeof(Lds) <= 160 * 1024, "LDS of a CU");
  Lds& lds = *reinterpret_cast<Lds*>(lds_raw);
  const int tid = threadIdx.x, lane = tid & 63, w = wave_number(), h = w >> 1;
  int n = lane & 15, g = lane >> 4;
  const uint32_t NC = (uint32_t)a.NC, chunk = blockIdx.x % NC, bh = blockIdx.x / NC, hk = bh % (uint32_t)a.Hk;
  const int64_t b = bh / (uint32_t)a.Hk, t0 = (int64_t)chunk * CH, tokens = length_of(a.lengths, b, a.S) - t0;
  const int rows = (int)min((int64_t)CH, a.S - t0), left = (int)max((int64_t)0, min((int64_t)CH, tokens));
  const int Dk = (int)a.Dk, Dv = (int)a.Dv, VP = (int)a.VP, qs = (int)a.Hk * Dk, vs = (int)a.Hv * Dv;
  const int per = (int)((uint32_t)a.Hv / (uint32_t)a.Hk);
  const int64_t keys = (b * a.S + t0) * qs + hk * Dk;
  const auto bring = [&](int key0) {
    const Range q = head_rows((const T*)a.q + keys, left, qs, Dk), k = head_rows((const T*)a.k + keys, left, qs, Dk);
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int x = i * 256 + tid, piece = x % PIECES, row = x / PIECES;
      const Op<NP> ko = token_op<T, VEC>(k, qs, row, key0 + 8 * piece, Dk), qo = token_op<T, VEC>(q, qs, row, key0 + 8 * piece, Dk);
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        const int at = Tk::at(place_of(row), piece);
        *reinterpret_cast<bf8_t*>(lds.k[p] + at) = ko.p[p];
        *reinterpret_cast<bf8_t*>(lds.q[p] + at) = qo.p[p];
      }
    }
  };
  // rows i: k_i . k_j and q_i . k_j of the keys in LDS, j the wave's tokens; x: the other half's rows (h = 0)
  struct Dots {
    f4_t kk[2], qk[2], xk[2], xq[2];
  };
  const auto dots = [&](Dots& o) {
    const int k_rows = Tk::lane_at(n, g) + 32 * h * Tk::ROW, k_own = Tk::at(place_of(16 * w + n), g);
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      Op<NP> kn;
#pragma unroll
      for (int p = 0; p < NP; ++p) kn.p[p] = *reinterpret_cast<const bf8_t*>(lds.k[p] + (k_own ^ (kb << 6)));
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        Op<NP> ka, qa;
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          ka.p[p] = Tk::rows(lds.k[p], k_rows, t, kb);
          qa.p[p] = Tk::rows(lds.q[p], k_rows, t, kb);
        }
        o.kk[t] = mma(ka, kn, o.kk[t]);
        o.qk[t] = mma(qa, kn, o.qk[t]);
      }
      if (h == 0) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          Op<NP> ka, qa;
#pragma unroll
          for (int p = 0; p < NP; ++p) {
            ka.p[p] = Tk::rows(lds.k[p], k_rows, 2 + t, kb);
            qa.p[p] = Tk::rows(lds.q[p], k_rows, 2 + t, kb);
          }
          o.xk[t] = mma(ka, kn, o.xk[t]);
          o.xq[t] = mma(qa, kn, o.xq[t]);
        }
      }
      keep_order();
    }
  };
  Dots of_halves = {};
  if (HALVES) {
    bring(KL);
    lds_barrier();
    dots(of_halves);
    lds_barrier();
  }
  bring(0);
  if (HALVES) {
    lds_barrier();
    dots(of_halves);
  }
  const Range dqp = head_rows((T*)a.dq + keys, rows, qs, Dk), dkp = head_rows((T*)a.dk + keys, rows, qs, Dk);
  const auto put = [&](int tok, int key0, const f4_t* dq, const f4_t* dk) {  // 64 keys of the wave's tokens
#pragma unroll
    for (int t2 = 0; t2 < 2; ++t2) {
      const int k0 = key0 + 32 * t2 + 8 * g;
      float vq[8], vk[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        vq[e] = tok < left ? dq[2 * t2 + (e >> 2)][e & 3] : 0.f;
        vk[e] = tok < left ? dk[2 * t2 + (e >> 2)][e & 3] : 0.f;
      }
      put_row8<VEC>((T*)nullptr, dqp, (tok * qs + k0) * (uint32_t)sizeof(T), Dk - k0, vq);
      put_row8<VEC>((T*)nullptr, dkp, (tok * qs + k0) * (uint32_t)sizeof(T), Dk - k0, vk);
    }
  };
#pragma unroll 1
  for (int pass = 0; pass < PASSES; ++pass) {
    if (HALVES && pass) {
      of_halves = {};
      bring(KL);  // every wave has passed the last head's last barrier
    }
    f4_t dqt[4 * QUADS], dkt[4 * QUADS];
#pragma unroll
    for (int t = 0; t < 4 * QUADS; ++t) dqt[t] = dkt[t] = f4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
    for (int hi = 0; hi < per; ++hi) {
      renew(n, g);
      const int tok = 16 * w + n;
      const int64_t hv = hk * per + hi, at = (b * a.Hv + hv) * NC + chunk;
      const int64_t gat = (b * a.S + t0) * a.Hv + hv;
      if (left == 0) {
        if (tid < rows) a.dg[gat + tid * a.Hv] = a.dbeta[gat + tid * a.Hv] = 0.f;
        continue;
      }
      if (tid < CH) {
        const bool on = tid < left;
        lds.G[tid] = running_sum(on ? clamp_decay(a.g[gat + tid * a.Hv]) : 0.0, tid);
        lds.beta[tid] = on ? a.beta[gat + tid * a.Hv] : 0.f;
      }
      const Range dop = head_rows((const T*)a.d_o + (b * a.S + t0) * vs + hv * Dv, left, vs, Dv);
      const Range zp((const float*)a.z + at * CH * VP, 4 * CH * VP);
      const Range wp((const float*)a.w + at * CH * VP, 4 * CH * VP);
      // a thread brings eight columns of a row, or of two, of each array
      constexpr int COLS = Lds::COLS, N = COLS / 32, M_ROWS = 256 / Lds::PIECES;
      const int m_row = tid / Lds::PIECES, m_piece = tid % Lds::PIECES, m_col = 8 * m_piece;
      const int own_at = Lds::at(place_of(tok), g), rows_at = Lds::at(n, g);

      // What each pair of tokens passes on. The wave's tokens lie in half h of the chunk; with those of the
      // same half a token is the earlier or the later one, with the other half's only one of them.
      // Lane j = tok. Rows i >= j: B_ij and A_ij (it is the earlier one); rows j' <= tok: B and A of
      // (tok, j'), the later one. As operands: bq by K for dQ, bk by Q and aa by K for dK; x is the
      // other half's bk (h = 0) or bq (h = 1), ax its aa.
      float db = 0.f, late = 0.f;  // late: of the token as the earlier one of pairs and of the chunk's end
      Fine bq, bk, aa, x, ax;
      {
        F8 zs[N], ws[N];
        Raw8<T> ds[N];
        const auto fetch = [&](int vb) {
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const int row = M_ROWS * i + m_row, c = vb + m_col;
            const uint32_t o = c < VP ? 4 * (row * VP + c) : NOWHERE;
            zs[i] = zp.floats(o, 0);
            ws[i] = wp.floats(o, 0);
            ds[i].template load<VEC>(dop, (row * vs + c) * (uint32_t)sizeof(T), Dv - c);
          }
        };
        f4_t zd[2], zw[2], dz[2], wz[2];  // Z_row . dO, Z_row . W, dO_row . Z, W_row . Z with the wave's tokens
        f4_t xd[2], xw[2];                // the other half's: the last two (h = 0) or the first two
#pragma unroll
        for (int t = 0; t < 2; ++t) zd[t] = zw[t] = dz[t] = wz[t] = xd[t] = xw[t] = f4_t{0.f, 0.f, 0.f, 0.f};
        fetch(0);
        for (int vb = 0, turn = 0; vb < VP; vb += COLS, turn ^= 1) {
          char* m = lds.buf[Lds::NBUF == 2 ? turn : 0];
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const int o = Lds::at(place_of(M_ROWS * i + m_row), m_piece);
            const Op<NP> d = ds[i].template op<NP>();
            Lds::put(m, 0, o, zs[i]);
            Lds::put(m, 3, o, ws[i]);
#pragma unroll
            for (int p = 0; p < NP; ++p) *reinterpret_cast<bf8_t*>(m + (6 + p) * Lds::PART + o) = d.p[p];
          }
          if (vb + COLS < VP) fetch(vb + COLS);
          lds_barrier();
#pragma unroll
          for (int kb = 0; kb < N; ++kb) {
            const Op<NP> dn = Lds::stream(m, 6, own_at, 0, kb);
            const Fine zn = Lds::fine(m, 0, own_at, 0, kb), wn = Lds::fine(m, 3, own_at, 0, kb);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              const int r = 2 * h + t, o = 2 - 2 * h + t;
              const Fine zr = Lds::fine(m, 0, rows_at, r, kb);
              zd[t] = mma(zr, dn, zd[t]);
              zw[t] = mma(zr, wn, zw[t]);
              dz[t] = mma(Lds::stream(m, 6, rows_at, r, kb), zn, dz[t]);
              wz[t] = mma(Lds::fine(m, 3, rows_at, r, kb), zn, wz[t]);
              if (h == 0) {
                xd[t] = mma(Lds::stream(m, 6, rows_at, o, kb), zn, xd[t]);
                xw[t] = mma(Lds::fine(m, 3, rows_at, o, kb), zn, xw[t]);
              } else {
                const Fine zo = Lds::fine(m, 0, rows_at, o, kb);
                xd[t] = mma(zo, dn, xd[t]);
                xw[t] = mma(zo, wn, xw[t]);
              }
              keep_order();
            }
          }
          if (Lds::NBUF == 1) lds_barrier();
        }
        keep_order();
        Dots both_of = of_halves;
        if (!HALVES && pass == 0) dots(both_of);
        const f4_t(&kk)[2] = both_of.kk, (&qk)[2] = both_of.qk, (&xk)[2] = both_of.xk, (&xq)[2] = both_of.xq;
        const double Gn = lds.G[tok];
        const float beta_n = lds.beta[tok];
        float vq[8], vk[8], va[8], c[8];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int r0 = 32 * h + 8 * g + 4 * t;
          const f4_t beta = *reinterpret_cast<const f4_t*>(lds.beta + r0);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int row = r0 + r;
            const double G = lds.G[row];
            const float d = decay(row >= tok ? G - Gn : Gn - G);
            const float bz = row >= tok ? a.scale * d * dz[t][r] : 0.f, az = row > tok ? -d * wz[t][r] : 0.f;
            vq[4 * t + r] = row <= tok ? a.scale * beta[r] * d * zd[t][r] : 0.f;
            vk[4 * t + r] = beta_n * bz;
            va[4 * t + r] = row < tok ? -beta[r] * d * zw[t][r] : beta_n * az;
            const float both = bz * qk[t][r] + az * kk[t][r];
            db += both;
            c[4 * t + r] = row > tok ? beta_n * both : 0.f;
          }
        }
        const auto ends_at = [&](int row0) {  // the pairs' parts by the later token, over the wave's earlier ones
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            late += c[e];
            c[e] = row16_sum(c[e]);
          }
          if (n == 0) store8(lds.row[w] + row0, c);
        };
        ends_at(32 * h + 8 * g);
        bq = split<3>(vq);
        bk = split<3>(vk);
        aa = split<3>(va);
        pin(bq);
        pin(bk);
        pin(aa);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int r0 = 32 - 32 * h + 8 * g + 4 * t;
          const f4_t beta = *reinterpret_cast<const f4_t*>(lds.beta + r0);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const double G = lds.G[r0 + r];
            const float d = decay(h == 0 ? G - Gn : Gn - G);
            const float bx = a.scale * d * xd[t][r], axx = -d * xw[t][r], be = h == 0 ? beta_n : beta[r];
            const float both = h == 0 ? bx * xq[t][r] + axx * xk[t][r] : 0.f;
            db += both;
            c[4 * t + r] = beta_n * both;
            vq[4 * t + r] = be * bx;
            va[4 * t + r] = be * axx;
          }
        }
        if (h == 0) ends_at(32 + 8 * g);
        x = split<3>(vq);
        ax = split<3>(va);
        pin(x);
        pin(ax);
        keep_order();
      }
      // What the states pass on, 64 keys at a time.
      const Range mp((const float*)a.states + at * KP * VP, 4 * KP * VP);
      const Range np((const float*)a.dstates + at * KP * VP, 4 * KP * VP);
      F8 mr[N], nr[N], zn_next[N], wn_next[N];
      Op<NP> dn_next[N];
      const auto fetch = [&](int key0, int vb) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const uint32_t o = vb + m_col < VP ? 4 * ((M_ROWS * i + m_row) * VP + m_col) : NOWHERE;
          mr[i] = mp.floats(o, 4 * (key0 * VP + vb));
          nr[i] = np.floats(o, 4 * (key0 * VP + vb));
          const int c = vb + 32 * i + 8 * g;
          const uint32_t own = c < VP ? 4 * (tok * VP + c) : NOWHERE;
          dn_next[i] = token_op<T, VEC>(dop, vs, tok, c, Dv);
          zn_next[i] = zp.floats(own, 0);
          wn_next[i] = wp.floats(own, 0);
        }
      };
      fetch(64 * QUADS * pass, 0);
      const double Gend = lds.G[CH - 1], Gown = lds.G[tok];
      const float ahead = decay(Gown), to_end = decay(Gend - Gown), eb = to_end * lds.beta[tok];
      float mn = 0.f, from_start = 0.f;  // <M, N>; what the token reads of M
      lds_barrier();  // the buffers held Z, W and dO until here
#pragma unroll
      for (int quad = 0; quad < QUADS; ++quad) {
        const int key0 = 64 * (QUADS * pass + quad);
        f4_t dq[4], read[4], early[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) dq[t] = read[t] = early[t] = f4_t{0.f, 0.f, 0.f, 0.f};
        for (int vb = 0, turn = 0; vb < VP; vb += COLS, turn ^= 1) {
          char* m = lds.buf[Lds::NBUF == 2 ? turn : 0];
          Op<NP> dn[N];
          Fine zn[N], wn[N];
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const int o = Lds::at(place_of(M_ROWS * i + m_row), m_piece);
            Lds::put(m, 0, o, mr[i]);
            Lds::put(m, 3, o, nr[i]);
#pragma unroll
            for (int e = 0; e < 4; ++e) mn += mr[i].a[e] * nr[i].a[e] + mr[i].b[e] * nr[i].b[e];
            dn[i] = dn_next[i];
            zn[i] = split<3>(zn_next[i].a, zn_next[i].b);
            wn[i] = split<3>(wn_next[i].a, wn_next[i].b);
          }
          if (vb + COLS < VP) fetch(key0, vb + COLS);
          else if (quad + 1 < QUADS) fetch(key0 + 64, 0);
          lds_barrier();
#pragma unroll
          for (int kb = 0; kb < N; ++kb) {
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              const Fine ms = Lds::fine(m, 0, rows_at, t, kb), ns = Lds::fine(m, 3, rows_at, t, kb);
              dq[t] = mma(ms, dn[kb], dq[t]);
              read[t] = mma(ms, wn[kb], read[t]);
              early[t] = mma(ns, zn[kb], early[t]);
              if (t & 1) keep_order();
            }
          }
          if (Lds::NBUF == 1) lds_barrier();
        }
        // after an odd number of steps the next one takes the same buffer
        if (Lds::NBUF == 2 && ((VP + COLS - 1) / COLS & 1)) lds_barrier();
        const int held = HALVES ? 64 * quad : key0;  // their place in LDS
        const int cols_at = Tk::lane_at_t(n, g) ^ (2 * held);
        f4_t dk[4];
#pragma unroll
        for (int t2 = 0; t2 < 2; ++t2) {
          float kf[8], qf[8];
          {
            const int o = Tk::at(place_of(tok), (held >> 3) + 4 * t2 + g);
#pragma unroll
            for (int e = 0; e < 8; ++e) kf[e] = qf[e] = 0.f;
#pragma unroll
            for (int p = NP - 1; p >= 0; --p) {
              const bf8_t kp = *reinterpret_cast<const bf8_t*>(lds.k[p] + o), qp = *reinterpret_cast<const bf8_t*>(lds.q[p] + o);
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                kf[e] += (float)kp[e];
                qf[e] += (float)qp[e];
              }
            }
          }
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int t = 2 * t2 + u;
            float ke = 0.f;
#pragma unroll
            for (int r = 0; r < 4; ++r) ke += kf[4 * u + r] * early[t][r];
            db += to_end * ke;
            late += eb * ke;
            dq[t] *= a.scale * ahead;
#pragma unroll
            for (int r = 0; r < 4; ++r) from_start += qf[4 * u + r] * dq[t][r] - kf[4 * u + r] * (ahead * read[t][r]);
            dk[t] = eb * early[t] - ahead * read[t];
            Op<NP> ko, qo, kx, qx;
#pragma unroll
            for (int p = 0; p < NP; ++p) {
              ko.p[p] = Tk::cols(lds.k[p], cols_at, t, h);
              qo.p[p] = Tk::cols(lds.q[p], cols_at, t, h);
              kx.p[p] = Tk::cols(lds.k[p], cols_at, t, 1 - h);
              if (h == 0) qx.p[p] = Tk::cols(lds.q[p], cols_at, t, 1);
            }
            dq[t] = mma(ko, bq, dq[t]);
            dk[t] = mma(qo, bk, dk[t]);
            dk[t] = mma(ko, aa, dk[t]);
            dk[t] = mma(kx, ax, dk[t]);
            if (h == 0) dk[t] = mma(qx, x, dk[t]);
            else dq[t] = mma(kx, x, dq[t]);
            if (SHARED) {
              dqt[4 * quad + t] += dq[t];
              dkt[4 * quad + t] += dk[t];
            }
            keep_order();
          }
        }
        if (!SHARED) put(tok, key0, dq, dk);
      }
      db = sum_groups(db);
      late = sum_groups(late);
      from_start = sum_groups(from_start);
      const float whole = wave_sum(decay(Gend) * mn);
      if (g == 0) {
        lds.read[tok] = from_start;
        lds.late[tok] = late;
        float* p = a.dbeta + gat + tok * a.Hv;
        if (tok < rows) *p = tok < left ? (pass ? *p + db : db) : 0.f;
      }
      if (lane == 0) lds.end[w] = whole;
      lds_barrier();
      if (tid < CH) {
        float s = lds.read[tid], open = lds.late[tid] - (lds.row[0][tid] + lds.row[1][tid]);
        if (tid >= CH / 2) open -= lds.row[2][tid] + lds.row[3][tid];
#pragma unroll
        for (int o = 1; o < CH; o <<= 1) {
          const float down = __shfl_down(s, o, 64), up = __shfl_up(open, o, 64);
          if (tid + o < CH) s += down;
          if (tid >= o) open += up;
        }
        const float before = __shfl_up(open, 1, 64);
        s += (tid > 0 ? before : 0.f) + ((lds.end[0] + lds.end[1]) + (lds.end[2] + lds.end[3]));
        float* p = a.dg + gat + tid * a.Hv;
        if (tid < rows) *p = tid < left ? (pass ? *p + s : s) : 0.f;
      }
      lds_barrier();
    }
    if (SHARED || left == 0)
#pragma unroll
      for (int quad = 0; quad < QUADS; ++quad) put(16 * w + n, 64 * (QUADS * pass + quad), dqt + 4 * quad, dkt + 4 * quad);
  }
}

template <typename K>
hipError_t with_lds(K kernel, size_t lds, unsigned grid, unsigned block, const DeltaArgs& a, hipStream_t st) {
  if (lds > 64 * 1024) {
    hipError_t e = hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(kernel, dim3(grid), dim3(block), lds, st, a);
  return hipGetLastError();
}

template <typename T, int KP, bool FULL>
hipError_t back_go(const DeltaArgs& a, hipStream_t st) {
  constexpr int NW = 4;
  const unsigned grid = (unsigned)(a.B * a.Hv * a.NS * ((a.Dv + 16 * NW - 1) / (16 * NW)));
  const size_t lds = sizeof(BackLds<KP, PARTS<T>, NW>);
  return a.vec ? with_lds(delta_back_kernel<T, KP, NW, true, FULL>, lds, grid, 64 * NW, a, st)
               : with_lds(delta_back_kernel<T, KP, NW, false, FULL>, lds, grid, 64 * NW, a, st);
}

template <typename T, int KP>
hipError_t grad_go(const DeltaArgs& a, hipStream_t st) {
  typedef GradLds<KP, PARTS<T>> Lds;
  const unsigned grid = (unsigned)(a.B * a.Hk * a.NC), block = 256;
  if (a.Hv == a.Hk)
    return a.vec8 ? with_lds(delta_grad_kernel<T, KP, true, false>, sizeof(Lds), grid, block, a, st)
                  : with_lds(delta_grad_kernel<T, KP, false, false>, sizeof(Lds), grid, block, a, st);
  return a.vec8 ? with_lds(delta_grad_kernel<T, KP, true, true>, sizeof(Lds), grid, block, a, st)
                : with_lds(delta_grad_kernel<T, KP, false, true>, sizeof(Lds), grid, block, a, st);
}

template <typename T, int KP>
hipError_t backward_go(const DeltaArgs& a, hipStream_t st) {
  hipError_t e = hipSuccess;
  if (a.NS > 1) {
    e = back_go<T, KP, false>(a, st);
    if (e == hipSuccess) e = launch_delta_join(true, a, st);
  }
  if (e == hipSuccess) e = back_go<T, KP, true>(a, st);
  return e != hipSuccess || a.NC == 0 ? e : grad_go<T, KP>(a, st);
}

template <typename T>
hipError_t backward_by_width(const DeltaArgs& a, hipStream_t st) {
  if (a.Dk <= 64) return backward_go<T, 64>(a, st);
  if (a.Dk <= 128) return backward_go<T, 128>(a, st);
  return backward_go<T, 256>(a, st);
}

}  // namespace

hipError_t launch_delta_backward(int dtype, const DeltaArgs& a, hipStream_t st) {
  if (a.NC > 0) {
    hipError_t e = launch_delta_keep(dtype, a, st);
    if (e != hipSuccess) return e;
  }
  return dtype == 0 ? backward_by_width<float>(a, st) : backward_by_width<bf16_t>(a, st);
}

}  // namespace hc
