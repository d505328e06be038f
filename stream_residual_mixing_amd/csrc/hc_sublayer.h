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
