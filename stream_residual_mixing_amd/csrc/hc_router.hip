// Training of the xHC stream router: the balance loss over the active sets, with
// its gradient to the scores, and the backward of the router's projection.
//   balance, per sequence b of n_b unmasked tokens: count_i = tokens whose active
//   set holds stream i, p_tj = s_tj / sum_j s_tj, P_j = mean_t p_tj,
//   f_j = E / ((k - m) n_b) count_{m+j};  loss = coef / B sum_b sum_j f_j P_j.
//   router: z_t = (vec X_t @ W) / r_t, s = sigmoid(z), r = ||vec X|| / sqrt(NC).
#include "hc_sublayer.h"
#include "hc_sublayer_device.h"

namespace hc {

namespace {

// W lanes of a wave share a token (lane j: candidate j, or stream j for the
// counts), so the scores are read once, in order, and the row's sum is a DPP sum.
template <int W>
__device__ __forceinline__ float lanes_sum(float v) {
  return W == 16 ? row16_sum(v) : wave_sum(v);
}

// Tokens of one workgroup's part, and the most that one workgroup takes alone: above,
// the loads of more workgroups pay for a second launch. With 16 lanes a token, loss and
// gradient take 24.9 us alone and 27.5 in parts at 4,096 tokens, 42 and 27 at 8,192; with
// 64 lanes 58 and 27 at 2,048.
constexpr int BAL_TOKENS = 128;
inline int64_t balance_alone(int W) { return W == 16 ? 4096 : 512; }

__device__ __forceinline__ float share(float s, float total) { return total == 0.f ? 0.f : s / total; }

// Token `at` of a lane group: adds its share, its streams (LDS counts: integer sums do
// not depend on their order) and itself.
template <int W>
__device__ __forceinline__ void balance_token(const float* __restrict__ score, const int32_t* __restrict__ idx,
                                              const uint8_t* __restrict__ mask, int64_t at, int E, int k, int j,
                                              int32_t* hist, float& p, int32_t& n) {
  const bool live = !mask || mask[at];
  float s = j < E ? score[at * E + j] : 0.f;
  const int32_t i = j < k ? idx[at * k + j] : -1;
  if (!live) s = 0.f;
  p += share(s, lanes_sum<W>(s));
  if (live) {
    if (i >= 0 && i < W) atomicAdd(&hist[i], 1);
    ++n;
  }
}

// Per (sequence, BAL_TOKENS tokens): counts [W], sums of p [W] and the unmasked tokens.
template <int W>
__global__ __launch_bounds__(256) void balance_part_kernel(const float* __restrict__ score,
                                                           const int32_t* __restrict__ idx,
                                                           const uint8_t* __restrict__ mask, int64_t S, int64_t nblk,
                                                           int E, int k, float* __restrict__ psum,
                                                           int32_t* __restrict__ cnt, int32_t* __restrict__ tok) {
  constexpr int SLOTS = 256 / W;
  __shared__ float sp[SLOTS][W];
  __shared__ int32_t sn[SLOTS], hist[W];
  const int j = threadIdx.x % W, slot = threadIdx.x / W;
  const int64_t part = blockIdx.x, b = part / nblk, t0 = (part - b * nblk) * BAL_TOKENS;
  const int64_t t1 = t0 + BAL_TOKENS < S ? t0 + BAL_TOKENS : S;
  if (threadIdx.x < W) hist[threadIdx.x] = 0;
  __syncthreads();
  float p = 0.f;
  int32_t n = 0;
#pragma unroll 4
  for (int64_t t = t0 + slot; t < t1; t += SLOTS)
    balance_token<W>(score, idx, mask, b * S + t, E, k, j, hist, p, n);
  sp[slot][j] = p;
  if (j == 0) sn[slot] = n;
  __syncthreads();
  if (slot == 0) {
    float ps = 0.f;
    int32_t ns = 0;
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) {
      ps += sp[i][j];
      ns += sn[i];
    }
    psum[part * W + j] = ps;
    cnt[part * W + j] = hist[j];
    if (j == 0) tok[part] = ns;
  }
}

// One workgroup adds up each sequence, in a fixed order, and forms the loss: from the
// parts, or (ALONE) from the tokens themselves. `subs` lane groups share a sequence.
template <int W, bool ALONE>
__global__ __launch_bounds__(1024) void balance_finish_kernel(
    const float* __restrict__ psum, const int32_t* __restrict__ cnt, const int32_t* __restrict__ tok,
    const float* __restrict__ score, const int32_t* __restrict__ idx, const uint8_t* __restrict__ mask, int64_t B,
    int64_t S, int64_t nblk, int subs, int N, int k, int m, float coef, float* __restrict__ loss,
    int32_t* __restrict__ count, int32_t* __restrict__ tokens, float* __restrict__ mean_p) {
  constexpr int SLOTS = 1024 / W;
  __shared__ float red[16], sp[SLOTS][W];
  __shared__ int32_t sn[SLOTS], hist[SLOTS][W];
  const int j = threadIdx.x % W, slot = threadIdx.x / W, sub = slot % subs, own = slot - sub;
  const int E = N - m, per = SLOTS / subs;  // sequences at once
  float sum = 0.f;
  for (int64_t b0 = 0; b0 < B; b0 += per) {
    const int64_t b = b0 + slot / subs;
    hist[slot][j] = 0;
    __syncthreads();
    float ps = 0.f;
    int32_t ns = 0;
    if (b < B && slot < per * subs) {
      if (ALONE) {
#pragma unroll 4
        for (int64_t t = sub; t < S; t += subs)
          balance_token<W>(score, idx, mask, b * S + t, E, k, j, hist[own], ps, ns);
      } else {
        int32_t cs = 0;
#pragma unroll 4
        for (int64_t i = sub; i < nblk; i += subs) {
          const int64_t part = b * nblk + i;
          ps += psum[part * W + j];
          cs += cnt[part * W + j];
          ns += tok[part];
        }
        if (cs) atomicAdd(&hist[own][j], cs);
      }
    }
    sp[slot][j] = ps;
    if (j == 0) sn[slot] = ns;
    __syncthreads();
    if (b < B && sub == 0 && slot < per * subs) {
      ps = 0.f;
      ns = 0;
      for (int i = 0; i < subs; ++i) {
        ps += sp[slot + i][j];
        ns += sn[slot + i];
      }
      if (j < N) count[b * N + j] = hist[slot][j];
      if (j == 0) tokens[b] = ns;
      if (j < E) {
        const float n = (float)(ns > 0 ? ns : 1);
        const float mp = ps / n;
        const float f = (float)hist[slot][m + j] * ((float)E / (float)(k - m)) / n;
        mean_p[b * E + j] = mp;
        sum += f * mp;
      }
    }
    __syncthreads();
  }
  const float all = block_sum(sum, red);
  if (threadIdx.x == 0) *loss = B > 0 ? coef * (all / (float)B) : 0.f;
}

// dscore_tj = dloss coef / (B n) (f_j - sum_i f_i p_ti) / sum_i s_ti; 0 for masked tokens.
template <int W>
__global__ __launch_bounds__(256) void balance_backward_kernel(const float* __restrict__ score,
                                                               const int32_t* __restrict__ count,
                                                               const int32_t* __restrict__ tokens,
                                                               const uint8_t* __restrict__ mask, int64_t B, int64_t S,
                                                               int N, int k, int m, float coef,
                                                               const float* __restrict__ dloss,
                                                               float* __restrict__ dscore) {
  const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) / W;
  const int j = threadIdx.x % W;
  const int E = N - m;
  if (at >= B * S) return;
  const int64_t b = at / S;
  const bool live = !mask || mask[at];
  float g = 0.f;
  if (live) {  // uniform over the token's lanes
    const int32_t ns = tokens[b];
    const float n = (float)(ns > 0 ? ns : 1);
    const float s = j < E ? score[at * E + j] : 0.f;
    const float f = j < E ? (float)count[b * N + m + j] * ((float)E / (float)(k - m)) / n : 0.f;
    const float total = lanes_sum<W>(s);
    const float dot = lanes_sum<W>(f * share(s, total));
    const float w = (dloss ? *dloss : 1.f) * coef / ((float)B * n);
    g = total == 0.f ? 0.f : w * (f - dot) / total;
  }
  if (j < E) dscore[at * E + j] = g;
}

// ---------------------------------------------------- the router's projection

// The apply pass multiplies on the matrix cores (v_mfma_f32_16x16x32_bf16), 32 tokens
// and 64 channels of a wave at a time, so that the 2 E products per value of X hide
// behind its memory traffic (on the vector units they took half as long as the traffic:
// 845 against 768 us at N = 16, C = 4096, T = 8192). X is bfloat16 as it is; the float32
// factors P = dz / r and the weights are split into bfloat16 parts: P into three (24 bits,
// all of it) for dw, and P and w into two each (16 bits) for dX, which is rounded to 8.
// Lane 16 q + m of a wave holds channels 4 m .. 4 m + 3 of tokens 4 q + i and 16 + 4 q +
// i, i < 4: what it loads is its part of both operands and of both results,
//   dX:  D[token][channel] += [P_hi | P_lo] [w_part | w_part]^T, k = 16 part + j,
//   dw:  D[channel][j] += x^T P_part, k = 8 q + kk the lane's kk-th token.
// Factors of one group of 32 tokens, written by the pass before in the operands' layout.
struct Group {
  uint16_t a[2][64][8];   // dX's operand of each 16 tokens: lane, k
  uint16_t b[3][64][8];   // dw's operand of each part of P: lane (16 q + j), kk
  float c[32];            // the factor of x; NO_PART for a token that takes no part
};
constexpr uint32_t NO_PART = 0x80000000u;  // -0; a token that does take part has +0
constexpr int GT = 32;

__device__ __forceinline__ uint16_t bf_part(float& v) {  // the leading bfloat16 of v, taken off
  const uint32_t h = f2bf(v);
  v -= bf2f(h);
  return (uint16_t)h;
}

// One workgroup per token (and for the places behind the last one, which are cleared):
// r from the whole row, then the token's factors. A token whose dscore is all zero takes
// part in nothing: its row is not read.
__global__ __launch_bounds__(256) void router_factors_kernel(const bf16_t* __restrict__ X, int64_t T, int64_t NC,
                                                             int E, const float* __restrict__ score,
                                                             const float* __restrict__ dscore,
                                                             Group* __restrict__ G) {
  __shared__ float red[4];
  const int64_t t = blockIdx.x;
  const int j = threadIdx.x;
  bool any = false;
  if (t < T)
    for (int i = 0; i < E; ++i) any |= dscore[t * E + i] != 0.f;
  float ss = 0.f;
  if (any) {
    const bf16_t* x = X + t * NC;
    for (int64_t c = (int64_t)threadIdx.x * 8; c < NC; c += 2048) {
      float v[8];
      load8(x + c, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) ss += v[e] * v[e];
    }
    ss = block_sum(ss, red);
  }
  if (j >= 16) return;
  float dz = 0.f, along = 0.f;
  if (any && j < E) {
    const float s = score[t * E + j];
    dz = dscore[t * E + j] * (s * (1.f - s));
    along = dz == 0.f ? 0.f : dz * (logf(s) - logf(1.f - s));  // z from its sigmoid
  }
  along = row16_sum(along);
  const float ms = ss / (float)NC;
  const float inv_r = ms == 0.f ? 0.f : 1.f / sqrtf(ms);
  float p = dz * inv_r;
  Group& g = G[t / GT];
  const int tau = (int)(t % GT), tile = tau / 16, m = tau % 16, q = m / 4, kk = 4 * tile + m % 4;
  uint16_t part[3];
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    part[i] = bf_part(p);
    g.b[i][16 * q + j][kk] = part[i];
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) g.a[tile][16 * (2 * i + j / 8) + m][j % 8] = part[i];
  if (j == 0) g.c[tau] = any ? along * inv_r * inv_r / (float)NC + 0.f : __uint_as_float(NO_PART);  // -0 + 0 = +0
}

typedef __bf16 bfv8 __attribute__((ext_vector_type(8)));
typedef float fv4 __attribute__((ext_vector_type(4)));
typedef uint32_t u2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ bfv8 as_bf8(uint4 v) { return __builtin_bit_cast(bfv8, v); }

// 8 weights of one channel, column j0 on, their bfloat16 parts packed.
template <int E>
__device__ __forceinline__ void weight_parts(const float* __restrict__ w, int64_t ch, int j0, uint4& hi, uint4& lo) {
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = j0 + 2 * i < E ? w[ch * E + j0 + 2 * i] : 0.f;
    const float b = j0 + 2 * i + 1 < E ? w[ch * E + j0 + 2 * i + 1] : 0.f;
    h[i] = pack_bf2_hw(a, b);
    l[i] = pack_bf2_hw(a - __uint_as_float(h[i] << 16), b - __uint_as_float(h[i] & 0xffff0000u));
  }
  hi = make_uint4(h[0], h[1], h[2], h[3]);
  lo = make_uint4(l[0], l[1], l[2], l[3]);
}

// The groups are taken from the last one back, the splits in turns: the pass before has
// just read the last rows. KEPT: all of X may still be in the last-level cache (256 MB)
// and is read through it (T = 240 of 16 x 4,096: 43 against 49 us; 1 GB: 776 against 770).
template <int E, bool KEPT>
__global__ __launch_bounds__(256, 3) void router_apply_kernel(const bf16_t* __restrict__ X, int64_t T, int64_t NC,
                                                              const float* __restrict__ w,
                                                              const Group* __restrict__ G, const bf16_t* dX_in,
                                                              bf16_t* dX_out, float* __restrict__ part) {
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m = lane & 15, q = lane >> 4;
  const int64_t c0 = (int64_t)blockIdx.x * 256 + wv * 64;  // this wave's channels
  if (c0 >= NC) return;
  const bool in = c0 + 4 * m < NC;  // NC is a multiple of 32; lanes past it read channel c0 on and store nothing
  const uint32_t ch = in ? 4 * m : 0;
  uint4 wh[4], wl[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) weight_parts<E>(w, c0 + ch + e, 8 * (q & 1), wh[e], wl[e]);
  fv4 dw[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) dw[e] = fv4{0.f, 0.f, 0.f, 0.f};
  const uint32_t row = (uint32_t)NC;

  for (int64_t g = (T + GT - 1) / GT - 1 - blockIdx.y; g >= 0; g -= gridDim.y) {
    const int64_t t0 = g * GT;
    const int live = (int)min((int64_t)GT, T - t0);
    const bf16_t* xb = X + t0 * NC + c0;
    const bf16_t* db = dX_in + t0 * NC + c0;
    u2 x[8], d[8];
    uint32_t off[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int tau = 16 * (i >> 2) + 4 * q + (i & 3);
      off[i] = (uint32_t)min(tau, live - 1) * row + ch;  // past the end: the last token's row again
      const u2* xp = reinterpret_cast<const u2*>(xb + off[i]);
      x[i] = KEPT ? *xp : __builtin_nontemporal_load(xp);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) d[i] = __builtin_nontemporal_load(reinterpret_cast<const u2*>(db + off[i]));
    const Group& f = G[g];
    uint4 pa[2], pb[3];
#pragma unroll
    for (int i = 0; i < 2; ++i) pa[i] = reinterpret_cast<const uint4*>(f.a[i])[lane];
#pragma unroll
    for (int i = 0; i < 3; ++i) pb[i] = reinterpret_cast<const uint4*>(f.b[i])[lane];
    float c[8];
    {
      const float4 u = reinterpret_cast<const float4*>(f.c)[q], v = reinterpret_cast<const float4*>(f.c)[4 + q];
      c[0] = u.x; c[1] = u.y; c[2] = u.z; c[3] = u.w;
      c[4] = v.x; c[5] = v.y; c[6] = v.z; c[7] = v.w;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (__float_as_uint(c[i]) == NO_PART) x[i] = u2{0u, 0u};  // such a token may hold anything
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      uint32_t k[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // channel e of tokens 2 i, 2 i + 1
        const uint32_t u = e < 2 ? x[2 * i].x : x[2 * i].y, v = e < 2 ? x[2 * i + 1].x : x[2 * i + 1].y;
        k[i] = (e & 1) ? __builtin_amdgcn_perm(v, u, 0x07060302) : __builtin_amdgcn_perm(v, u, 0x05040100);
      }
      const bfv8 xa = as_bf8(make_uint4(k[0], k[1], k[2], k[3]));
#pragma unroll
      for (int i = 0; i < 3; ++i) dw[e] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xa, as_bf8(pb[i]), dw[e], 0, 0, 0);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // 16 tokens each
      fv4 s[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[e] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf8(pa[h]), as_bf8(wl[e]), fv4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
        s[e] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf8(pa[h]), as_bf8(wh[e]), s[e], 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const u2 xq = x[4 * h + i], dq = d[4 * h + i];
        const float cf = c[4 * h + i];
        const float o0 = __uint_as_float(dq.x << 16) + (s[0][i] - cf * __uint_as_float(xq.x << 16));
        const float o1 = __uint_as_float(dq.x & 0xffff0000u) + (s[1][i] - cf * __uint_as_float(xq.x & 0xffff0000u));
        const float o2 = __uint_as_float(dq.y << 16) + (s[2][i] - cf * __uint_as_float(xq.y << 16));
        const float o3 = __uint_as_float(dq.y & 0xffff0000u) + (s[3][i] - cf * __uint_as_float(xq.y & 0xffff0000u));
        if (in && 16 * h + 4 * q + i < live)
          __builtin_nontemporal_store(u2{pack_bf2_hw(o0, o1), pack_bf2_hw(o2, o3)},
                                      reinterpret_cast<u2*>(dX_out + t0 * NC + c0 + off[4 * h + i]));
      }
    }
  }
  // D row 4 q + i, column m: channel 4 (4 q + i) + e, j = m
  float* p = part + ((int64_t)blockIdx.y * NC + c0) * E;
#pragma unroll
  for (int e = 0; e < 4; ++e)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int cc = 4 * (4 * q + i) + e;
      if (m < E && c0 + cc < NC) p[(int64_t)cc * E + m] = dw[e][i];
    }
}

__global__ __launch_bounds__(256) void split_sum_kernel(const float* __restrict__ part, int64_t n, int splits,
                                                        float* __restrict__ out) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  float s = 0.f;
#pragma unroll 8
  for (int k = 0; k < splits; ++k) s += part[k * n + i];
  out[i] = s;
}

// Token splits of the apply pass: one round of the workgroups that are resident at
// once, three a CU.
int64_t router_splits(int64_t T, int64_t NC) {
  const int64_t blocks = (NC + 255) / 256;
  int64_t s = 768 / blocks;
  const int64_t most = (T + GT - 1) / GT;
  if (s > most) s = most;
  return s < 1 ? 1 : s;
}

inline int64_t router_groups(int64_t T) { return (T + GT - 1) / GT; }

inline int64_t al256(int64_t b) { return (b + 255) & ~(int64_t)255; }

inline int64_t bal_blocks(int64_t S) { return (S + BAL_TOKENS - 1) / BAL_TOKENS; }

template <int W>
hipError_t balance_go(const float* score, const int32_t* idx, const uint8_t* mask, int64_t B, int64_t S, int N, int k,
                      int m, float coef, float* loss, int32_t* count, int32_t* tokens, float* mean_p, void* ws,
                      hipStream_t st) {
  const int64_t nblk = bal_blocks(S), parts = B * nblk;
  int subs = 1024 / W;  // lane groups of one sequence: all of them, halved while sequences go without
  while (subs > 1 && (1024 / W) / subs < B) subs /= 2;
  if (B * S <= balance_alone(W)) {
    hipLaunchKernelGGL((balance_finish_kernel<W, true>), dim3(1), dim3(1024), 0, st, nullptr, nullptr, nullptr, score,
                       idx, mask, B, S, nblk, subs, N, k, m, coef, loss, count, tokens, mean_p);
    return hipGetLastError();
  }
  char* q = (char*)ws;
  float* psum = (float*)q;
  q += al256(parts * W * 4);
  int32_t* cnt = (int32_t*)q;
  q += al256(parts * W * 4);
  int32_t* tok = (int32_t*)q;
  hipLaunchKernelGGL((balance_part_kernel<W>), dim3((unsigned)parts), dim3(256), 0, st, score, idx, mask, S, nblk,
                     N - m, k, psum, cnt, tok);
  hipLaunchKernelGGL((balance_finish_kernel<W, false>), dim3(1), dim3(1024), 0, st, psum, cnt, tok, score, idx, mask,
                     B, S, nblk, subs, N, k, m, coef, loss, count, tokens, mean_p);
  return hipGetLastError();
}

template <int E>
void router_apply(const void* X, int64_t T, int64_t NC, int64_t splits, const float* w, const Group* G,
                  const void* dX_in, void* dX_out, float* part, hipStream_t st) {
  const dim3 g((unsigned)((NC + 255) / 256), (unsigned)splits), b(256);
  if (T * NC * 2 <= (256ll << 20))
    hipLaunchKernelGGL((router_apply_kernel<E, true>), g, b, 0, st, (const bf16_t*)X, T, NC, w, G,
                       (const bf16_t*)dX_in, (bf16_t*)dX_out, part);
  else
    hipLaunchKernelGGL((router_apply_kernel<E, false>), g, b, 0, st, (const bf16_t*)X, T, NC, w, G,
                       (const bf16_t*)dX_in, (bf16_t*)dX_out, part);
}

}  // namespace

int64_t balance_ws_bytes(int64_t B, int64_t S, int N, int m) {
  const int W = N <= 16 ? 16 : 64;
  const int64_t parts = B * bal_blocks(S);
  if (B * S <= balance_alone(W)) return 0;
  return 2 * al256(parts * W * 4) + al256(parts * 4);
}

hipError_t launch_balance(const float* score, const int32_t* idx, const uint8_t* mask, int64_t B, int64_t S, int N,
                          int k, int m, float coef, float* loss, int32_t* count, int32_t* tokens, float* mean_p,
                          void* ws, hipStream_t st) {
  return N <= 16 ? balance_go<16>(score, idx, mask, B, S, N, k, m, coef, loss, count, tokens, mean_p, ws, st)
                 : balance_go<64>(score, idx, mask, B, S, N, k, m, coef, loss, count, tokens, mean_p, ws, st);
}

hipError_t launch_balance_backward(const float* score, const int32_t* count, const int32_t* tokens,
                                   const uint8_t* mask, int64_t B, int64_t S, int N, int k, int m, float coef,
                                   const float* dloss, float* dscore, hipStream_t st) {
  const int W = N <= 16 ? 16 : 64;
  const dim3 g((unsigned)((B * S * W + 255) / 256)), b(256);
  if (W == 16)
    hipLaunchKernelGGL((balance_backward_kernel<16>), g, b, 0, st, score, count, tokens, mask, B, S, N, k, m, coef,
                       dloss, dscore);
  else
    hipLaunchKernelGGL((balance_backward_kernel<64>), g, b, 0, st, score, count, tokens, mask, B, S, N, k, m, coef,
                       dloss, dscore);
  return hipGetLastError();
}

int64_t router_backward_ws_bytes(int64_t T, int N, int64_t C, int m) {
  if (T == 0) return 0;
  const int64_t NC = (int64_t)N * C;
  return al256(router_groups(T) * sizeof(Group)) + al256(router_splits(T, NC) * NC * (N - m) * 4);
}

hipError_t launch_router_backward(const void* X, int64_t T, int N, int64_t C, int m, const float* w,
                                  const float* score, const float* dscore, const void* dX_in, void* dX_out, float* dw,
                                  void* ws, hipStream_t st) {
  const int E = N - m;
  const int64_t NC = (int64_t)N * C, splits = router_splits(T, NC);
  Group* G = (Group*)ws;
  // one split's part is dw itself
  float* part = splits == 1 ? dw : (float*)((char*)ws + al256(router_groups(T) * sizeof(Group)));
  const int64_t n = NC * E;
  if (T == 0) {
    hipLaunchKernelGGL(split_sum_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, st, part, n, 0, dw);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(router_factors_kernel, dim3((unsigned)(router_groups(T) * GT)), dim3(256), 0, st,
                     (const bf16_t*)X, T, NC, E, score, dscore, G);
  switch (E) {
#define HC_ROUTER_CASE(e) \
  case e: router_apply<e>(X, T, NC, splits, w, G, dX_in, dX_out, part, st); break;
    HC_ROUTER_CASE(1) HC_ROUTER_CASE(2) HC_ROUTER_CASE(3) HC_ROUTER_CASE(4) HC_ROUTER_CASE(5)
    HC_ROUTER_CASE(6) HC_ROUTER_CASE(7) HC_ROUTER_CASE(8) HC_ROUTER_CASE(9) HC_ROUTER_CASE(10)
    HC_ROUTER_CASE(11) HC_ROUTER_CASE(12) HC_ROUTER_CASE(13) HC_ROUTER_CASE(14) HC_ROUTER_CASE(15)
#undef HC_ROUTER_CASE
    default: break;
  }
  if (splits == 1) return hipGetLastError();
  hipLaunchKernelGGL(split_sum_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, st, part, n, (int)splits, dw);
  return hipGetLastError();
}

}  // namespace hc
