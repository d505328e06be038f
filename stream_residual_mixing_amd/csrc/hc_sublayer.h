// Launch functions of the operators beside the stream mixing: the norm, the gated
// scan and the training of the router (internal; the public ABI is include/hc.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace hc {

// ---- norm (hc_norm.hip)
// mode 0: v = x; 1: v = x + res; 2: v = sum_i h[i] x[i]. s: v rounded to the stream
// dtype (mode 0 has none; may be NULL). out: 0 stream dtype, 2 e4m3, 3 int8 with
// scale [T, ngroups] (group 0: one scale a row). vec: C % 8 == 0 with 16-byte
// aligned arrays (8 bytes for 8-bit y). C <= 16384.
struct NormArgs {
  const void* x;
  const void* res;
  const float* h;
  const float* w;
  void* s;
  void* y;
  float* scale;
  int64_t T, C, ngroups;
  int n, out, group;
  float eps;
};
hipError_t launch_rms_norm(int dtype, int mode, bool vec, const NormArgs& a, hipStream_t st);
// ds and part (then dw too) may be NULL; part [norm_backward_parts(T, C), C].
struct NormBwdArgs {
  const void* s;
  const float* w;
  const void* dy;
  const void* ds;
  void* dx;
  float* part;
  int64_t T, C;
  float eps;
};
int64_t norm_backward_parts(int64_t T, int64_t C);
hipError_t launch_rms_norm_backward(int dtype, bool vec, const NormBwdArgs& a, float* dw, hipStream_t st);
// out0[c], out1[c] = the sums over P parts of [P, C], the second array's parts behind the
// first's; either may be NULL
hipError_t launch_column_sums(const float* parts, int64_t P, int64_t C, float* out0, float* out1, hipStream_t st);

// ---- layer norm (hc_layer_norm.hip): as above, b the bias (may be NULL)
hipError_t launch_layer_norm(int dtype, int mode, bool vec, const NormArgs& a, const float* b, hipStream_t st);
// dw, db may be NULL; part (NULL when both are) [2, norm_backward_parts(T, C), C]
hipError_t launch_layer_norm_backward(int dtype, bool vec, const NormBwdArgs& a, float* dw, float* db, hipStream_t st);

// ---- gated linear recurrence (hc_scan.hip)
// Forward: y, last from x, gate, h0. Backward (bwd): dx, dgate, dh0 from x, gate, y,
// dy, h0, dh_last. vec: C even, the stream arrays aligned to 2 elements and the state
// arrays to 8 bytes.
struct ScanArgs {
  const void* x;
  const void* gate;
  const void* y_in;      // backward: the forward's output
  const void* dy;        // backward
  const float* state0;   // h0 (may be NULL: zeros)
  const float* dlast;    // backward: the last state's gradient (may be NULL: zeros)
  const int32_t* lengths;  // may be NULL: S tokens each
  void* y;               // forward: y; backward: dx
  void* dgate;           // backward
  float* state1;         // forward: the last state; backward: dh0 (may be NULL)
  void* ws;
  int64_t B, S, C;
  int tied;
};
int64_t scan_ws_bytes(int64_t B, int64_t S, int64_t C);
hipError_t launch_scan(int dtype, bool bwd, bool vec, const ScanArgs& a, hipStream_t st);

// ---- gated delta rule (hc_delta.hip, hc_delta_backward.hip)
// vec: Dk % 8 == 0 with q, k and their gradients 16-byte aligned; vec8: also Dv % 8 == 0 with v and
// d_o 16-byte aligned; vec4: Dv % 4 == 0 with the states 16-byte aligned.
struct DeltaArgs {
  const void* q;
  const void* k;
  const void* v;
  const float* g;
  const float* beta;
  const float* state0;     // may be NULL: zeros
  const int32_t* lengths;  // may be NULL: S tokens each
  void* o;
  float* state1;           // may be NULL
  int64_t B, S, Hk, Hv, Dk, Dv;
  float scale;
  bool vec, vec8, vec4;
  // backward
  const void* d_o;
  const float* dlast;      // may be NULL: zeros
  void* dq;
  void* dk;
  void* dv;
  float* dg;
  float* dbeta;
  float* dstate0;          // may be NULL
  // set by delta_plan: NC = ceil(S / 64) chunks in segments of SL, NS segments at most; VP is Dv in
  // whole 32s; the arrays in the workspace
  int64_t NC, SL, NS, VP;
  void* rec;               // the chunks' records
  float* slots;            // [B, Hv, NS, Dk, Dv] a segment's last state (backward: the gradient of its first)
  void* phi;               // [B, Hv, NS, 3, KP, KP] its map of the state, in three bfloat16 parts
  void* phi_t;             // the same transposed; KP is Dk as 64, 128 or 256
  void* states;            // backward: every chunk's first state [KP, VP] and Z [64, VP], and the gradient
  void* z;                 // of the state behind it and W of the same shapes, float32
  void* dstates;
  void* w;
};
// lays the call out and returns the bytes of its workspace; ws may be NULL
int64_t delta_plan(DeltaArgs& a, bool backward, void* ws);
hipError_t launch_delta(int dtype, const DeltaArgs& a, hipStream_t st);
// the backward's first part: records, segments' maps, states and z
hipError_t launch_delta_keep(int dtype, const DeltaArgs& a, hipStream_t st);
hipError_t launch_delta_backward(int dtype, const DeltaArgs& a, hipStream_t st);
// joins the segments' states (back: their gradients, from the last one)
hipError_t launch_delta_join(bool back, const DeltaArgs& a, hipStream_t st);

// ---- balance loss and the router's backward (hc_router.hip)
int64_t balance_ws_bytes(int64_t B, int64_t S, int N, int m);
hipError_t launch_balance(const float* score, const int32_t* idx, const uint8_t* mask, int64_t B, int64_t S, int N,
                          int k, int m, float coef, float* loss, int32_t* count, int32_t* tokens, float* mean_p,
                          void* ws, hipStream_t st);
hipError_t launch_balance_backward(const float* score, const int32_t* count, const int32_t* tokens,
                                   const uint8_t* mask, int64_t B, int64_t S, int N, int k, int m, float coef,
                                   const float* dloss, float* dscore, hipStream_t st);
int64_t router_backward_ws_bytes(int64_t T, int N, int64_t C, int m);
hipError_t launch_router_backward(const void* X, int64_t T, int N, int64_t C, int m, const float* w,
                                  const float* score, const float* dscore, const void* dX_in, void* dX_out, float* dw,
                                  void* ws, hipStream_t st);

}  // namespace hc
