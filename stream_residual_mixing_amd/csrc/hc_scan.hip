// The diagonal gated linear recurrence over the sequence, forward and backward:
//   a_t = sigmoid(gate_t),  u_t = 1 - a_t (tied) or 1,
//   h_t = a_t h_{t-1} + u_t x_t,  y_t = h_t.
// Backward, with R_t the gradient that reaches h_t from later tokens (R = dh_last
// behind the last token): dh_t = dy_t + R_t, R_{t-1} = a_t dh_t, dx_t = u_t dh_t,
// dgate_t = dh_t (h_{t-1} - x_t (tied) or h_{t-1}) a_t (1 - a_t), dh0 = R before token 0.
// Both directions walk an affine map per token and channel, s -> a s + b; maps
// compose, so the sequence is cut into chunks: each chunk's composed map, a walk
// over the chunks for each chunk's first state, and a second walk inside the
// chunks that writes the outputs.
#include "hc_device.h"
#include "hc_launch.h"

namespace hc {

namespace {

constexpr int CHUNK = 64;  // tokens of one thread's walk

constexpr int V = 4;       // channels of one thread

// V consecutive channels of one row. VEC: C is a multiple of V and every row is
// aligned to V elements. Otherwise four channels are still one access where the row
// has them (global memory takes any element-aligned address); `cnt` of them at its end.
template <bool VEC>
__device__ __forceinline__ void ld4(const float* p, int cnt, float v[V]) {
  if (VEC) {
    const float4 q = *reinterpret_cast<const float4*>(p);
    v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
  } else if (cnt == V) {
    __builtin_memcpy(v, p, 16);
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = e < cnt ? p[e] : 0.f;
  }
}

template <bool VEC>
__device__ __forceinline__ void ld4(const bf16_t* p, int cnt, float v[V]) {
  uint2 q;
  if (VEC) {
    q = *reinterpret_cast<const uint2*>(p);
  } else if (cnt == V) {
    __builtin_memcpy(&q, p, 8);
  } else {
    q.x = (uint32_t)p[0] | (cnt > 1 ? (uint32_t)p[1] << 16 : 0u);
    q.y = cnt > 2 ? (uint32_t)p[2] : 0u;
  }
  v[0] = bf2f(q.x & 0xffffu); v[1] = __uint_as_float(q.x & 0xffff0000u);
  v[2] = bf2f(q.y & 0xffffu); v[3] = __uint_as_float(q.y & 0xffff0000u);
}

template <bool VEC>
__device__ __forceinline__ void st4(float* p, int cnt, const float v[V]) {
  if (VEC) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  } else if (cnt == V) {
    __builtin_memcpy(p, v, 16);
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (e < cnt) p[e] = v[e];
  }
}

template <bool VEC>
__device__ __forceinline__ void st4(bf16_t* p, int cnt, const float v[V]) {
  const uint2 q = make_uint2(pack_bf2(v[0], v[1]), pack_bf2(v[2], v[3]));
  if (VEC) {
    *reinterpret_cast<uint2*>(p) = q;
  } else if (cnt == V) {
    __builtin_memcpy(p, &q, 8);
  } else {
    p[0] = (bf16_t)q.x;
    if (cnt > 1) p[1] = (bf16_t)(q.x >> 16);
    if (cnt > 2) p[2] = (bf16_t)q.y;
  }
}

// a = sigmoid(g) and u = 1 - a, each from exp(-|g|) so that neither cancels.
__device__ __forceinline__ void gates(float g, float& a, float& u) {
  const float e = __expf(-fabsf(g));
  const float s = __builtin_amdgcn_rcpf(1.f + e);
  a = g >= 0.f ? s : e * s;
  u = g >= 0.f ? e * s : s;
}

__device__ __forceinline__ int64_t seq_len(const int32_t* lengths, int64_t b, int64_t S) {
  if (!lengths) return S;
  const int64_t n = lengths[b];
  return n < 0 ? 0 : (n > S ? S : n);
}

// Thread -> (sequence, chunk, V channels); tokens t0 .. t1 - 1.
struct Place {
  int64_t b, j, c, t0, t1;
  int cnt;
};

__device__ __forceinline__ bool place(const ScanArgs& a, int64_t nchunk, Place& p) {
  const int64_t ncg = (a.C + V - 1) / V;
  const int64_t g = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (g >= a.B * nchunk * ncg) return false;
  p.c = (g % ncg) * V;
  p.cnt = (int)(a.C - p.c < V ? a.C - p.c : V);
  const int64_t r = g / ncg;
  p.j = r % nchunk;
  p.b = r / nchunk;
  const int64_t len = seq_len(a.lengths, p.b, a.S);
  p.t0 = p.j * CHUNK < len ? p.j * CHUNK : len;
  p.t1 = (p.j + 1) * CHUNK < len ? (p.j + 1) * CHUNK : len;
  return true;
}

// The composed map of one chunk, (A, H): s -> A s + H, at ws[(b, j)][2][C].
template <typename T, bool VEC, bool BWD>
__global__ __launch_bounds__(256) void scan_chunk_kernel(ScanArgs a, int64_t nchunk) {
  Place p;
  if (!place(a, nchunk, p)) return;
  float A[V], H[V];
#pragma unroll
  for (int e = 0; e < V; ++e) { A[e] = 1.f; H[e] = 0.f; }
  const int64_t n = p.t1 - p.t0;
#pragma unroll 8
  for (int64_t i = 0; i < n; ++i) {
    const int64_t t = BWD ? p.t1 - 1 - i : p.t0 + i;
    const int64_t at = (p.b * a.S + t) * a.C + p.c;
    float g[V], x[V];
    ld4<VEC>((const T*)a.gate + at, p.cnt, g);
    ld4<VEC>((const T*)(BWD ? a.dy : a.x) + at, p.cnt, x);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      float d, u;
      gates(g[e], d, u);
      H[e] = BWD ? d * (H[e] + x[e]) : d * H[e] + (a.tied ? u * x[e] : x[e]);
      A[e] *= d;
    }
  }
  float* w = (float*)a.ws + (p.b * nchunk + p.j) * 2 * a.C + p.c;
  st4<VEC>(w, p.cnt, A);
  st4<VEC>(w + a.C, p.cnt, H);
}

// The state before each chunk, in place of the chunk's A.
template <bool BWD>
__global__ __launch_bounds__(64) void scan_carry_kernel(ScanArgs a, int64_t nchunk) {
  const int64_t g = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (g >= a.B * a.C) return;
  const int64_t b = g / a.C, c = g - b * a.C;
  const float* first = BWD ? a.dlast : a.state0;
  float s = first ? first[g] : 0.f;
  float* w = (float*)a.ws + b * nchunk * 2 * a.C + c;
#pragma unroll 8
  for (int64_t i = 0; i < nchunk; ++i) {
    float* q = w + (BWD ? nchunk - 1 - i : i) * 2 * a.C;
    const float A = q[0], H = q[a.C];
    q[0] = s;
    s = A * s + H;
  }
}

// The walk inside each chunk from its first state; with one chunk the state comes
// from and goes to the caller's arrays.
template <typename T, bool VEC, bool BWD>
__global__ __launch_bounds__(256) void scan_apply_kernel(ScanArgs a, int64_t nchunk) {
  Place p;
  if (!place(a, nchunk, p)) return;
  float s[V];
#pragma unroll
  for (int e = 0; e < V; ++e) s[e] = 0.f;
  if (nchunk > 1) {
    ld4<VEC>((const float*)a.ws + (p.b * nchunk + p.j) * 2 * a.C + p.c, p.cnt, s);
  } else {
    const float* first = BWD ? a.dlast : a.state0;
    if (first) ld4<VEC>(first + p.b * a.C + p.c, p.cnt, s);
  }
  const int64_t n = p.t1 - p.t0;
#pragma unroll 4
  for (int64_t i = 0; i < n; ++i) {
    const int64_t t = BWD ? p.t1 - 1 - i : p.t0 + i;
    const int64_t at = (p.b * a.S + t) * a.C + p.c;
    float g[V], x[V];
    ld4<VEC>((const T*)a.gate + at, p.cnt, g);
    ld4<VEC>((const T*)a.x + at, p.cnt, x);
    if (!BWD) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float d, u;
        gates(g[e], d, u);
        s[e] = d * s[e] + (a.tied ? u * x[e] : x[e]);
      }
      st4<VEC>((T*)a.y + at, p.cnt, s);
    } else {
      float dy[V], hp[V], dx[V], dg[V];
      ld4<VEC>((const T*)a.dy + at, p.cnt, dy);
      if (t > 0) {
        ld4<VEC>((const T*)a.y_in + at - a.C, p.cnt, hp);
      } else if (a.state0) {
        ld4<VEC>(a.state0 + p.b * a.C + p.c, p.cnt, hp);
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) hp[e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float d, u;
        gates(g[e], d, u);
        const float dh = dy[e] + s[e];
        dx[e] = a.tied ? u * dh : dh;
        dg[e] = dh * (a.tied ? hp[e] - x[e] : hp[e]) * (d * u);
        s[e] = d * dh;
      }
      st4<VEC>((T*)a.y + at, p.cnt, dx);
      st4<VEC>((T*)a.dgate + at, p.cnt, dg);
    }
  }
  if (BWD) {  // padding receives no gradient
    const int64_t end = (p.j + 1) * CHUNK < a.S ? (p.j + 1) * CHUNK : a.S;
    const float zero[4] = {0.f, 0.f, 0.f, 0.f};
    for (int64_t t = p.t1 > p.j * CHUNK ? p.t1 : p.j * CHUNK; t < end; ++t) {
      const int64_t at = (p.b * a.S + t) * a.C + p.c;
      st4<VEC>((T*)a.y + at, p.cnt, zero);
      st4<VEC>((T*)a.dgate + at, p.cnt, zero);
    }
  }
  // the last chunk's walk ends in the state that goes on, the same value as its last y
  if (p.j == (BWD ? 0 : nchunk - 1) && a.state1) st4<VEC>(a.state1 + p.b * a.C + p.c, p.cnt, s);
}

// at least one, whose walk also passes the state on when there is no token
int64_t chunks_of(int64_t S) { return S > CHUNK ? (S + CHUNK - 1) / CHUNK : 1; }

template <typename T, bool VEC, bool BWD>
hipError_t scan_go(const ScanArgs& a, hipStream_t st) {
  const int64_t nchunk = chunks_of(a.S);
  const int64_t threads = a.B * nchunk * ((a.C + V - 1) / V);
  const dim3 g((unsigned)((threads + 255) / 256)), b(256);
  if (nchunk > 1) {
    hipLaunchKernelGGL((scan_chunk_kernel<T, VEC, BWD>), g, b, 0, st, a, nchunk);
    hipLaunchKernelGGL((scan_carry_kernel<BWD>), dim3((unsigned)((a.B * a.C + 63) / 64)), dim3(64), 0, st, a, nchunk);
  }
  hipLaunchKernelGGL((scan_apply_kernel<T, VEC, BWD>), g, b, 0, st, a, nchunk);
  return hipGetLastError();
}

template <bool BWD>
hipError_t scan_by_type(int dtype, bool vec, const ScanArgs& a, hipStream_t st) {
  if (dtype == 0) return vec ? scan_go<float, true, BWD>(a, st) : scan_go<float, false, BWD>(a, st);
  return vec ? scan_go<bf16_t, true, BWD>(a, st) : scan_go<bf16_t, false, BWD>(a, st);
}

}  // namespace

int64_t scan_ws_bytes(int64_t B, int64_t S, int64_t C) {
  const int64_t n = chunks_of(S);
  return n > 1 ? B * n * 2 * C * 4 : 0;
}

hipError_t launch_scan(int dtype, bool bwd, bool vec, const ScanArgs& a, hipStream_t st) {
  return bwd ? scan_by_type<true>(dtype, vec, a, st) : scan_by_type<false>(dtype, vec, a, st);
}

}  // namespace hc
