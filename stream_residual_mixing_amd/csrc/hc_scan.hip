// The diagonal gated linear recurrence over the sequence, forward and backward:
//   a_t = sigmoid(gate_t),  u_t = 1 - a_t (tied) or 1,
//   h_t = a_t h_{t-1} + u_t x_t,  y_t = h_t.
// Backward, with R_t the gradient that reaches h_t from later tokens (R = dh_last
// behind the last token): dh_t = dy_t + R_t, R_{t-1} = a_t dh_t, dx_t = u_t dh_t,
// dgate_t = dh_t (h_{t-1} - x_t (tied) or h_{t-1}) a_t (1 - a_t), dh0 = R before token 0.
// Both directions walk an affine map per token and channel, s -> a s + b (the
// backward with b = a dy, from the last token). Maps compose, so a long sequence is
// cut along time and the pieces' composed maps (A, H): s -> A s + H are joined.
//
// Two forms. Up to 32 tokens (16 backward) one thread walks the whole sequence of its channels.
// Longer ones run in one pass over the data: a workgroup holds a tile of tokens in
// registers, publishes the tile's composed map, joins the maps of the few tiles before
// it to the state that an earlier group of tiles left, and walks its tokens again from
// registers.
// A column's tiles (128 channels of a sequence) are taken from its counter in walk
// order, so that every tile waited for belongs to a workgroup that already runs and
// waits for earlier tiles only.
// Bound by HBM. Per call, the clearing launch included: 8,192 x 4,096 bfloat16 forward in
// 47 us (5 of them the clearing, 5 the joining), the backward of 2 x 4,096 x 4,096 in 82 (5
// the clearing, part of which the launch before it hides; a trace, which hides nothing, has
// 82 to 87 + 6). One counter for all columns took 51 and 87; reading the data twice (chunk
// maps, a walk over them, the outputs) 135 and 176.
// Rows behind a sequence's length are read like the others and then dropped: 5 x 1,021 x
// 1,100 float32 takes 17.5 us with 43 to 66 % of the rows live.
#include "hc_sublayer.h"
#include "hc_sublayer_device.h"

namespace hc {

namespace {

constexpr int V = 2;          // channels of one thread: 128 of a wave, one full access a row
constexpr int WAVES = 8;      // waves of a tile, one after another in time
constexpr int TILE_C = 64 * V;
constexpr int COUNTER = 32;   // words of a counter: a cache line of its own
// Sequences that one thread walks alone: 16 us against 24 in tiles for 64 x 32 x 4,096
// forward; backward 14.0 against 13.9 for 16 x 16 x 4,096 and 24 against 14 for 32 tokens.
constexpr int SHORT_FWD = 32, SHORT_BWD = 16;

// Tokens of one wave's walk in registers: 16 forward (8: 73 against 57 us at 8,192 x
// 4,096, twice the tiles to join), 8 backward, which keeps four values of each.
template <typename T, bool BWD>
struct Tile {
  static constexpr int LW = BWD ? 8 : 16;
  static constexpr int TOKENS = LW * WAVES;
};

// V channels of a row as stored. VEC: C is even and every row is aligned to two
// elements. Otherwise two channels are still one access where the row has them (any();
// global memory takes any element-aligned address), streamed where that measured better:
// float32 of 2 x 4,096 x 2,049 in 58 against 66 us, bfloat16 in 40 against 39.
template <typename T> struct Pair;
template <> struct Pair<float> {
  typedef float2 raw;
  static __device__ __forceinline__ void open(raw q, float v[V]) { v[0] = q.x; v[1] = q.y; }
  static __device__ __forceinline__ raw close(const float v[V]) { return make_float2(v[0], v[1]); }
  static __device__ __forceinline__ raw any(const float* p) {
    typedef float f2 __attribute__((ext_vector_type(2), aligned(4)));
    const f2 q = __builtin_nontemporal_load(reinterpret_cast<const f2*>(p));
    return make_float2(q.x, q.y);
  }
  static __device__ __forceinline__ raw stream(const float* p) {
    typedef float f2 __attribute__((ext_vector_type(2)));
    const f2 q = __builtin_nontemporal_load(reinterpret_cast<const f2*>(p));
    return make_float2(q.x, q.y);
  }
  static __device__ __forceinline__ void stream_out(float* p, raw q) {
    typedef float f2 __attribute__((ext_vector_type(2)));
    __builtin_nontemporal_store(f2{q.x, q.y}, reinterpret_cast<f2*>(p));
  }
  static __device__ __forceinline__ raw one(float e) { return make_float2(e, 0.f); }
  static __device__ __forceinline__ raw zero() { return make_float2(0.f, 0.f); }
  static __device__ __forceinline__ raw inf() { return make_float2(INFINITY, INFINITY); }
};
template <> struct Pair<bf16_t> {
  typedef uint32_t raw;
  static __device__ __forceinline__ void open(raw q, float v[V]) {
    v[0] = __uint_as_float(q << 16);
    v[1] = __uint_as_float(q & 0xffff0000u);
  }
  static __device__ __forceinline__ raw close(const float v[V]) { return pack_bf2_hw(v[0], v[1]); }
  static __device__ __forceinline__ raw any(const bf16_t* p) {
    raw q;
    __builtin_memcpy(&q, p, sizeof(q));
    return q;
  }
  static __device__ __forceinline__ raw stream(const bf16_t* p) {
    return __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(p));
  }
  static __device__ __forceinline__ void stream_out(bf16_t* p, raw q) {
    __builtin_nontemporal_store(q, reinterpret_cast<uint32_t*>(p));
  }
  static __device__ __forceinline__ raw one(bf16_t e) { return e; }
  static __device__ __forceinline__ raw zero() { return 0u; }
  static __device__ __forceinline__ raw inf() { return 0x7f807f80u; }
};

// OLD: the backward's arrays were written long before and are not kept in the caches
// (98 -> 94 us at 2 x 4096 x 4096); the forward's were just produced, and keeping them
// costs nothing where they are not (22 -> 19.5 us where they fit).
template <bool VEC, bool OLD = false, typename T>
__device__ __forceinline__ typename Pair<T>::raw ld2(const T* p, int cnt) {
  typename Pair<T>::raw q;
  if (VEC && OLD) {
    q = Pair<T>::stream(p);
  } else if (VEC) {
    q = *reinterpret_cast<const typename Pair<T>::raw*>(p);
  } else if (cnt >= V) {
    q = Pair<T>::any(p);
  } else {
    q = Pair<T>::one(p[0]);
  }
  return q;
}

// PAST: the forward's y goes past the caches (54.8 -> 53.4 us at 8,192 x 4,096, 30 -> 27
// at 64 x 128 x 2,048); the backward's two gradients do better without (92 against 95).
template <bool VEC, bool PAST = false, typename T>
__device__ __forceinline__ void st2(T* p, int cnt, const float v[V]) {
  const typename Pair<T>::raw q = Pair<T>::close(v);
  if (VEC && PAST) {
    Pair<T>::stream_out(p, q);
  } else if (VEC) {
    *reinterpret_cast<typename Pair<T>::raw*>(p) = q;
  } else if (cnt >= V) {
    __builtin_memcpy(p, &q, sizeof(q));
  } else {
    __builtin_memcpy(p, &q, sizeof(T));
  }
}

template <bool VEC>
__device__ __forceinline__ void ld2f(const float* p, int cnt, float v[V]) {
  Pair<float>::open(ld2<VEC>(p, cnt), v);
}

// a = sigmoid(g), u = 1 - a. The smaller of the two is q = e / (1 + e) with e =
// exp(-|g|), free of cancellation; the larger is 1 - q, which rounds once (from the
// reciprocal itself a would carry its error through every token of a long memory).
// q is kept with the sign of g: one register per token for both.
__device__ __forceinline__ float gate_q(float g) {
  const float e = __builtin_amdgcn_exp2f(-1.44269504f * fabsf(g));
  return copysignf(e * __builtin_amdgcn_rcpf(1.f + e), g);
}

__device__ __forceinline__ void gate_au(float q, float& a, float& u) {
  const float lo = fabsf(q), hi = 1.f - lo;
  const bool neg = (int)__float_as_uint(q) < 0;
  a = neg ? lo : hi;
  u = neg ? hi : lo;
}

__device__ __forceinline__ int64_t seq_len(const int32_t* lengths, int64_t b, int64_t S) {
  if (!lengths) return S;
  const int64_t n = lengths[b];
  return n < 0 ? 0 : (n > S ? S : n);
}

// The backward's outputs of one token from the state s (R_t), which becomes R_{t-1}.
__device__ __forceinline__ void back_step(bool tied, float a, float u, float dy, float x, float hp, float& s,
                                          float& dx, float& dg) {
  const float dh = dy + s;
  dx = tied ? u * dh : dh;
  dg = dh * (tied ? hp - x : hp) * (a * u);
  s = a * dh;
}

// ------------------------------------------------ short sequences: one walk

template <typename T, bool VEC, bool BWD>
__global__ __launch_bounds__(256) void scan_short_kernel(ScanArgs a) {
  const int64_t ncg = (a.C + V - 1) / V;
  const int64_t g = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (g >= a.B * ncg) return;
  const int64_t b = g / ncg, c = (g - b * ncg) * V;
  const int cnt = (int)(a.C - c < V ? a.C - c : V);
  const int64_t len = seq_len(a.lengths, b, a.S);
  const float* first = BWD ? a.dlast : a.state0;
  float s[V] = {0.f, 0.f};
  if (first) ld2f<VEC>(first + b * a.C + c, cnt, s);
  const int64_t row0 = b * a.S * a.C + c;
#pragma unroll 4
  for (int64_t i = 0; i < len; ++i) {
    const int64_t t = BWD ? len - 1 - i : i;
    const int64_t at = row0 + t * a.C;
    float gv[V], x[V], d[V], u[V];
    Pair<T>::open(ld2<VEC>((const T*)a.gate + at, cnt), gv);
    Pair<T>::open(ld2<VEC>((const T*)a.x + at, cnt), x);
#pragma unroll
    for (int e = 0; e < V; ++e) gate_au(gate_q(gv[e]), d[e], u[e]);
    if (!BWD) {
#pragma unroll
      for (int e = 0; e < V; ++e) s[e] = d[e] * s[e] + (a.tied ? u[e] * x[e] : x[e]);
      st2<VEC>((T*)a.y + at, cnt, s);
    } else {
      float dy[V], hp[V] = {0.f, 0.f}, dx[V], dg[V];
      Pair<T>::open(ld2<VEC>((const T*)a.dy + at, cnt), dy);
      if (t > 0) Pair<T>::open(ld2<VEC>((const T*)a.y_in + at - a.C, cnt), hp);
      else if (a.state0) ld2f<VEC>(a.state0 + b * a.C + c, cnt, hp);
#pragma unroll
      for (int e = 0; e < V; ++e) back_step(a.tied, d[e], u[e], dy[e], x[e], hp[e], s[e], dx[e], dg[e]);
      st2<VEC>((T*)a.y + at, cnt, dx);
      st2<VEC>((T*)a.dgate + at, cnt, dg);
    }
  }
  if (BWD) {  // padding receives no gradient
    const float zero[V] = {0.f, 0.f};
    for (int64_t t = len; t < a.S; ++t) {
      st2<VEC>((T*)a.y + row0 + t * a.C, cnt, zero);
      st2<VEC>((T*)a.dgate + row0 + t * a.C, cnt, zero);
    }
  }
  if (a.state1) st2<VEC>(a.state1 + b * a.C + c, cnt, s);
}

// ---------------------------------------------- long sequences: joined tiles

// The product A of many a that are all above 0 may fall below float32's smallest number.
// To a finite state 0 is as good, but an infinite one stays infinite: such a product is
// kept as -0, apart from the +0 of a gate that closed fully (or of a constant map).
constexpr uint32_t FADED = 0x80000000u;

// A with its zero's sign by `least`, the smallest of its factors' bits (-0 and NaN are
// above every number there).
__device__ __forceinline__ float product_of(float A, uint32_t least) {
  return A == 0.f ? __uint_as_float(least ? FADED : 0u) : A;
}

// s -> A s + H of an infinite state as well.
__device__ __forceinline__ float apply_map(float A, float s, float H) {
  return (__float_as_uint(A) == FADED && fabsf(s) == INFINITY ? 1.f : A) * s + H;
}

// A published map is one 64-bit word per channel, so no word is ever seen half
// written: A in the low half, H in the high half. All ones: not there yet (a value
// of that pattern, a NaN, is published as another NaN).
constexpr uint64_t ABSENT = ~0ull;

__device__ __forceinline__ uint64_t word_of(float A, float H) {
  const uint32_t a = __float_as_uint(A);
  uint32_t h = __float_as_uint(H);
  if (h == 0xffffffffu) h = 0x7fc00000u;
  return (uint64_t)h << 32 | a;
}

__device__ __forceinline__ void publish(uint64_t* p, uint64_t w) {
  __hip_atomic_store(p, w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

__device__ __forceinline__ uint64_t peek(const uint64_t* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Waits for a word. The tile waited for is running (see the counter), so the wait
// ends; the bound (some seconds) turns a workspace that another call writes meanwhile into
// NaN outputs instead of a hang.
constexpr int MOST_POLLS = 1 << 22;

__device__ __forceinline__ uint64_t await(const uint64_t* p) {
  uint64_t w = peek(p);
  for (int i = 0; w == ABSENT && i < MOST_POLLS; ++i) {
    __builtin_amdgcn_s_sleep(1);
    w = peek(p);
  }
  return w;
}

// The words of all tiles absent, the counters zero.
__global__ __launch_bounds__(256) void scan_clear_kernel(uint4* ws, int64_t counters16, int64_t n16) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n16) return;
  const uint32_t v = i < counters16 ? 0u : 0xffffffffu;
  ws[i] = make_uint4(v, v, v, v);
}

__device__ __forceinline__ void forget(float& v) { asm volatile("" : "+v"(v)); }
__device__ __forceinline__ void forget(uint32_t& v) { asm volatile("" : "+v"(v)); }
__device__ __forceinline__ void forget(float2& v) {
  forget(v.x);
  forget(v.y);
}

// ONE: the sequences are one tile long, and nothing is joined.
template <typename T, bool VEC, bool BWD, bool ONE>
__global__ __launch_bounds__(64 * WAVES, 4) void scan_tile_kernel(ScanArgs a, int64_t ntile, int64_t nct) {
  constexpr int LW = Tile<T, BWD>::LW, TOKENS = Tile<T, BWD>::TOKENS;
  typedef typename Pair<T>::raw raw;
  __shared__ float sA[WAVES][TILE_C], sH[WAVES][TILE_C];   // the waves' maps
  __shared__ float lA[WAVES][TILE_C], lH[WAVES][TILE_C];   // earlier tiles' maps
  __shared__ unsigned ticket;
  // what the whole wave shares is kept in scalar registers: every row is then one scalar
  // base and a 32-bit lane offset
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // A column is one channel tile of one sequence; its tiles in walk order, by its counter.
  // The columns move on by one from one row of workgroups to the next, or with a multiple
  // of 8 of them each would stay on one of the 8 dies (53 against 49 us at 8,192 x 4,096).
  const uint32_t ncol = (uint32_t)nct * (uint32_t)a.B, col = (blockIdx.x + blockIdx.x / ncol) % ncol;
  if (!ONE) {
    if (threadIdx.x == 0) ticket = atomicAdd((unsigned*)a.ws + (int64_t)col * COUNTER, 1u);
    lds_barrier();
  }
  // A counter that another call spoils meanwhile must not lead out of the workspace.
  const uint32_t j = ONE ? 0u : min((uint32_t)__builtin_amdgcn_readfirstlane(ticket), (uint32_t)ntile - 1);
  const uint32_t ct = col % (uint32_t)nct, b = col / (uint32_t)nct;
  const int64_t c0 = (int64_t)ct * TILE_C;
  const bool in = lane * V < a.C - c0;
  const uint32_t lo = in ? lane * V : 0;  // lanes past the row read its tile's first channels and store nothing
  const int cnt = (int)min((int64_t)V, a.C - c0 - lo);
  const int64_t len = seq_len(a.lengths, b, a.S);
  const int64_t seq0 = b * a.S * a.C + c0, st0 = b * a.C + c0;
  const int64_t i0 = (int64_t)j * TOKENS + wv * LW;  // this wave's first step of the walk
  const bool tied = a.tied;

  // token of step k, and the row that is read for it (a real one for every step)
#define HC_TOKEN(k) (BWD ? a.S - 1 - (i0 + (k)) : i0 + (k))
  raw rg[LW], rx[LW], rd[BWD ? LW : 1], ry[BWD ? LW : 1];
#pragma unroll
  for (int k = 0; k < LW; ++k) {
    int64_t t = HC_TOKEN(k);
    t = t < 0 ? 0 : (t >= a.S ? a.S - 1 : t);
    const int64_t at = seq0 + t * a.C;
    rg[k] = ld2<VEC, BWD>((const T*)a.gate + at + lo, cnt);
    rx[k] = ld2<VEC, BWD>((const T*)a.x + at + lo, cnt);
    if (BWD) {
      rd[k] = ld2<VEC, BWD>((const T*)a.dy + at + lo, cnt);
      ry[k] = ld2<VEC, BWD>((const T*)a.y_in + (at - (t > 0 ? a.C : 0)) + lo, cnt);
    }
  }

  // steps past the end and behind a sequence's length leave the state as it is: a = 1, b = 0
  if (BWD ? i0 + LW > a.S || a.S - i0 > len : i0 + LW > len)
#pragma unroll
    for (int k = 0; k < LW; ++k) {
      const int64_t t = HC_TOKEN(k);
      if (t < 0 || t >= len) {
        rg[k] = Pair<T>::inf();
        if (BWD) rd[BWD ? k : 0] = Pair<T>::zero();
        else rx[k] = Pair<T>::zero();
      }
    }

  // this wave's composed map; the forward keeps a and b, the backward the signed q
  float ka[LW][V], kb[BWD ? 1 : LW][V];
  float A[V] = {1.f, 1.f}, H[V] = {0.f, 0.f};
  uint32_t least[V] = {~0u, ~0u};
#pragma unroll
  for (int k = 0; k < LW; ++k) {
    float g[V], x[V];
    Pair<T>::open(rg[k], g);
    Pair<T>::open(BWD ? rd[BWD ? k : 0] : rx[k], x);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float q = gate_q(g[e]);
      float d, u;
      gate_au(q, d, u);
      const float bb = BWD ? d * x[e] : (tied ? u * x[e] : x[e]);
      H[e] = d * H[e] + bb;
      A[e] *= d;
      least[e] = min(least[e], __float_as_uint(d));
      ka[k][e] = BWD ? q : d;
      if (!BWD) kb[BWD ? 0 : k][e] = bb;
    }
  }
  // The caller's state is read here and nowhere else, by the walk's first wave, which
  // makes its map constant: whoever writes the last state (it may be the same array) has
  // waited for that map or for one composed from it.
  float init[V] = {0.f, 0.f};
#pragma unroll
  for (int e = 0; e < V; ++e) A[e] = product_of(A[e], least[e]);
  const float* first = BWD ? a.dlast : a.state0;
  if (i0 == 0 && first) {
    ld2f<VEC>(first + st0 + lo, cnt, init);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      H[e] = apply_map(A[e], init[e], H[e]);
      A[e] = 0.f;
    }
  }
#pragma unroll
  for (int e = 0; e < V; ++e) {
    sA[wv][lane * V + e] = A[e];
    sH[wv][lane * V + e] = H[e];
  }
  lds_barrier();
  // the waves before this one (pA, pH), and the whole tile's map
  float pA[V] = {1.f, 1.f}, pH[V] = {0.f, 0.f}, tA[V] = {1.f, 1.f}, tH[V] = {0.f, 0.f};
#pragma unroll BWD ? 2 : WAVES
  for (int w = 0; w < WAVES; ++w)
#pragma unroll
    for (int e = 0; e < V; ++e) {
      if (w == wv) {
        pA[e] = tA[e];
        pH[e] = tH[e];
      }
      const float wa = sA[w][lane * V + e];
      tH[e] = wa * tH[e] + sH[w][lane * V + e];
      tA[e] *= wa;
    }
  if (__any(tA[0] == 0.f || tA[1] == 0.f || pA[0] == 0.f || pA[1] == 0.f))
#pragma unroll
    for (int e = 0; e < V; ++e) {
      uint32_t least = ~0u;
#pragma unroll 1
      for (int w = 0; w < WAVES; ++w) {
        if (w == wv) pA[e] = product_of(pA[e], least);
        least = min(least, __float_as_uint(sA[w][lane * V + e]));
      }
      tA[e] = product_of(tA[e], least);
    }
  // A NaN may be what 0 made of an infinite state: the sums again, with care.
  if (__any(tH[0] != tH[0] || tH[1] != tH[1]))
#pragma unroll
    for (int e = 0; e < V; ++e) {
      tH[e] = 0.f;
#pragma unroll 1
      for (int w = 0; w < WAVES; ++w) {
        if (w == wv) pH[e] = tH[e];
        tH[e] = apply_map(sA[w][lane * V + e], tH[e], sH[w][lane * V + e]);
      }
    }

  // one word per lane's channel, inside the row or not
  uint64_t* words = (uint64_t*)((unsigned*)a.ws + (int64_t)ncol * COUNTER) + (int64_t)col * TILE_C + lane * V;
  const int64_t wstep = (int64_t)ncol * TILE_C;  // from one tile of the walk to the next
  // The state before the tile. Tiles are joined in groups of WAVES, always in the same
  // order (what is ready first makes no difference to a sum's rounding): from the state
  // that the group before left, through the maps of the group's earlier tiles (in the
  // first group, the first tile's map is constant). Each wave fetches one of these words;
  // the group's last tile publishes the state, the others their maps.
  const uint32_t gj = j % WAVES, g0 = j - gj;  // place in the group, its first tile
  const bool leaves = !ONE && wv == WAVES - 1 && j + 1 < ntile;
  if (leaves && gj < WAVES - 1)
#pragma unroll
    for (int e = 0; e < V; ++e) publish(words + (int64_t)j * wstep + e, word_of(tA[e], tH[e]));
  float s[V] = {0.f, 0.f};
  if (!ONE && j > 0) {
    // wave i: the map of the group's i-th tile; the last wave: the state before the group
    const bool state = wv == WAVES - 1;
    const bool want = state ? g0 > 0 : (uint32_t)wv < gj;
    const uint64_t* p = words + (int64_t)(state ? g0 - 1 : g0 + wv) * wstep;
    uint64_t w[V];
#pragma unroll
    for (int e = 0; e < V; ++e) w[e] = want ? peek(p + e) : word_of(1.f, 0.f);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      if (w[e] == ABSENT) w[e] = await(p + e);
      lA[wv][lane * V + e] = __uint_as_float((uint32_t)w[e]);
      lH[wv][lane * V + e] = __uint_as_float((uint32_t)(w[e] >> 32));
    }
    lds_barrier();
#pragma unroll
    for (int e = 0; e < V; ++e) s[e] = lH[WAVES - 1][lane * V + e];
#pragma unroll 4
    for (uint32_t i = 0; i < gj; ++i)
#pragma unroll
      for (int e = 0; e < V; ++e) s[e] = lA[i][lane * V + e] * s[e] + lH[i][lane * V + e];
    if (__any(s[0] != s[0] || s[1] != s[1]))  // as above
#pragma unroll
      for (int e = 0; e < V; ++e) {
        s[e] = lH[WAVES - 1][lane * V + e];
#pragma unroll 1
        for (uint32_t i = 0; i < gj; ++i) s[e] = apply_map(lA[i][lane * V + e], s[e], lH[i][lane * V + e]);
      }
  }
  if (leaves && gj == WAVES - 1)
#pragma unroll
    for (int e = 0; e < V; ++e) publish(words + (int64_t)j * wstep + e, word_of(0.f, apply_map(tA[e], s[e], tH[e])));

  // what the waves before this one make of it (one tile's first wave's map is constant, or of 0)
#pragma unroll
  for (int e = 0; e < V; ++e) s[e] = i0 == 0 ? init[e] : ONE ? pH[e] : apply_map(pA[e], s[e], pH[e]);

  // The backward's walk opens q and the rows again: without this the compiler keeps what
  // it made of them, four registers for one.
  if (BWD)
#pragma unroll
    for (int k = 0; k < LW; ++k) {
#pragma unroll
      for (int e = 0; e < V; ++e) forget(ka[k][e]);
      forget(rx[k]);
      forget(rd[BWD ? k : 0]);
    }

  // the walk itself
#pragma unroll
  for (int k = 0; k < LW; ++k) {
    const int64_t t = HC_TOKEN(k);
    const bool live = t >= 0 && t < len;
    const int64_t at = seq0 + t * a.C;
    if (!BWD) {
#pragma unroll
      for (int e = 0; e < V; ++e) s[e] = ka[k][e] * s[e] + kb[BWD ? 0 : k][e];
      if (live && in) st2<VEC, true>((T*)a.y + at + lo, cnt, s);
    } else if (t >= 0 && t < a.S) {
      float x[V], dy[V], hp[V], dx[V] = {0.f, 0.f}, dg[V] = {0.f, 0.f};
      if (live) {
        Pair<T>::open(rx[k], x);
        Pair<T>::open(rd[BWD ? k : 0], dy);
        Pair<T>::open(ry[BWD ? k : 0], hp);
        if (t == 0) {
          hp[0] = hp[1] = 0.f;
          if (a.state0) ld2f<VEC>(a.state0 + st0 + lo, cnt, hp);
        }
#pragma unroll
        for (int e = 0; e < V; ++e) {
          float d, u;
          gate_au(ka[k][e], d, u);
          back_step(tied, d, u, dy[e], x[e], hp[e], s[e], dx[e], dg[e]);
        }
      }
      if (in) {  // padding receives no gradient
        st2<VEC>((T*)a.y + at + lo, cnt, dx);
        st2<VEC>((T*)a.dgate + at + lo, cnt, dg);
      }
    }
  }
  // the wave of the walk's last step ends in the state that goes on
  if (a.state1 && in && i0 <= a.S - 1 && a.S - 1 < i0 + LW) st2<VEC>(a.state1 + st0 + lo, cnt, s);
#undef HC_TOKEN
}

template <typename T, bool VEC, bool BWD>
hipError_t scan_go(const ScanArgs& a, hipStream_t st) {
  if (a.S <= (BWD ? SHORT_BWD : SHORT_FWD)) {
    const int64_t threads = a.B * ((a.C + V - 1) / V);
    hipLaunchKernelGGL((scan_short_kernel<T, VEC, BWD>), dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, st, a);
    return hipGetLastError();
  }
  constexpr int TOKENS = Tile<T, BWD>::TOKENS;
  const int64_t ntile = (a.S + TOKENS - 1) / TOKENS, nct = (a.C + TILE_C - 1) / TILE_C;
  const dim3 g((unsigned)(ntile * a.B * nct)), b(64 * WAVES);
  if (ntile == 1) {
    hipLaunchKernelGGL((scan_tile_kernel<T, VEC, BWD, true>), g, b, 0, st, a, ntile, nct);
    return hipGetLastError();
  }
  const int64_t counters16 = a.B * nct * COUNTER / 4, n16 = counters16 + ntile * a.B * nct * TILE_C / 2;
  hipLaunchKernelGGL(scan_clear_kernel, dim3((unsigned)((n16 + 255) / 256)), dim3(256), 0, st, (uint4*)a.ws, counters16,
                     n16);
  hipLaunchKernelGGL((scan_tile_kernel<T, VEC, BWD, false>), g, b, 0, st, a, ntile, nct);
  return hipGetLastError();
}

template <bool BWD>
hipError_t scan_by_type(int dtype, bool vec, const ScanArgs& a, hipStream_t st) {
  if (dtype == 0) return vec ? scan_go<float, true, BWD>(a, st) : scan_go<float, false, BWD>(a, st);
  return vec ? scan_go<bf16_t, true, BWD>(a, st) : scan_go<bf16_t, false, BWD>(a, st);
}

}  // namespace

// The counter and the words of the finest tiling (both directions and types).
int64_t scan_ws_bytes(int64_t B, int64_t S, int64_t C) {
  constexpr int TOKENS = Tile<float, true>::TOKENS;
  if (S <= TOKENS) return 0;
  const int64_t ntile = (S + TOKENS - 1) / TOKENS, nct = (C + TILE_C - 1) / TILE_C;
  return B * nct * (COUNTER * 4 + ntile * TILE_C * 8);
}

hipError_t launch_scan(int dtype, bool bwd, bool vec, const ScanArgs& a, hipStream_t st) {
  return bwd ? scan_by_type<true>(dtype, vec, a, st) : scan_by_type<false>(dtype, vec, a, st);
}

}  // namespace hc
