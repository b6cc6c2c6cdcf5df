// Internal interface between the C ABI of the sequence-mixer operators
// (gdn_mixer_api.cpp: validation, workspace carving) and their kernels: the
// short causal convolution, the selective scan, the single-token steps and
// the layer norm.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime.h>

namespace gdn {

// Records the thread's error text and returns `code` (gdn_api.cpp).
int set_error(int code, const char *fmt, ...);
void clear_error();
int64_t compute_units();

// ---- packed sequences
// N sequences over `tokens` = B * T tokens in a row.  cu: device [N + 1]
// (packed batch, B = 1) or null (N = B rows of T tokens).
struct Seqs {
  const int32_t *cu;
  int N;
  int64_t T, tokens;
};

struct ConvArgs {
  Seqs s;
  int D, W, dtype, wdtype, silu;
  int64_t xs;  // elements from one token of x to the next
  const void *x, *w, *bias, *h0, *dy, *dht;
  void *y, *ht, *dx, *dw, *db, *dh0;
  float *partial;  // backward: [conv_bwd_tiles][W + 1][D]
};
int64_t conv_bwd_tiles(int64_t tokens, int D);
hipError_t launch_conv_fwd(const ConvArgs &a, hipStream_t st);
hipError_t launch_conv_bwd(const ConvArgs &a, hipStream_t st);

struct ConvStepArgs {
  int B, D, W, dtype, wdtype, silu, slots;
  int64_t xs;
  const void *x, *w, *bias;
  void *state, *y;
  const int32_t *index;
};
hipError_t launch_conv_step(const ConvStepArgs &a, hipStream_t st);

struct NormArgs {
  int64_t rows;
  int D, dtype, wdtype, rms;
  float eps;
  const void *x, *w, *b, *gate, *dy;
  void *y, *dx, *dw, *db, *dgate;
  float *mean, *rstd;  // written by the forward, read by the backward
  float *partial;      // backward: [norm_bwd_parts][2][D], then the rows' sums where a row is wider than a workgroup holds
};
int64_t norm_bwd_parts(int64_t rows);
size_t norm_bwd_floats(int64_t rows, int D);
hipError_t launch_norm_fwd(const NormArgs &a, hipStream_t st);
hipError_t launch_norm_bwd(const NormArgs &a, hipStream_t st);

// One token of the recurrences: state [slots][Hv][K][V] fp32, updated in
// place.  delta: the gated delta rule (g, beta, scale, l2), else the
// selective scan (dt, A, D, dt_bias, softplus).
struct StepArgs {
  int B, Hq, Hv, K, V, dtype, delta, l2, softplus, slots;
  float scale;
  int64_t qs, ks, vs;  // elements from one batch row of q (c), k (b), v (x) to the next
  const void *q, *k, *v, *beta;  // beta: dt of the scan
  const float *g, *A, *D, *dt_bias;
  float *state;
  const int32_t *index;
  void *o;
};
hipError_t launch_step(const StepArgs &a, hipStream_t st);

// The selective scan over whole sequences, cut into segments of `seg` tokens;
// each has a slot in the workspace (gdn_scan.hpp).
struct ScanArgs {
  Seqs s;
  int Hq, Hv, K, V, dtype, softplus;
  int seg;
  int64_t slots;
  bool one_seg;             // no sequence has two segments
  int64_t cs, bs, xs;       // elements from one token to the next of c, b, x
  const void *c, *b, *x, *dt, *dy;
  const float *A, *D, *dt_bias, *h0, *dht;
  void *y, *dc, *db, *dx, *ddt;
  float *ht, *dA, *dD, *ddt_bias, *dh0;
  char *ws;
};
struct ScanPlan {
  int seg;
  int64_t slots;
  bool one_seg;
  size_t ws;
};
ScanPlan scan_plan(const ScanArgs &a, bool bwd);
hipError_t launch_scan_fwd(const ScanArgs &a, hipStream_t st);
hipError_t launch_scan_bwd(const ScanArgs &a, hipStream_t st);

}  // namespace gdn
