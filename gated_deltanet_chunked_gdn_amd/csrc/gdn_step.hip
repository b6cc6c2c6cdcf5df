// One token of a recurrence for each row of a batch, the K x V fp32 state of
// every head read, updated and written in place:
//
//   gated delta rule   S = e^g S;  u = beta (v - S^T k);  S += k u^T;  o = scale S^T q
//   selective scan     S = e^(delta A) S + b (delta x)^T;  y = S^T c + D x
//   linear attention   S = e^g S + k v^T;  o = scale S^T q      (g: a head's)
//
// All are S' = a S + k u^T, o = s (a S^T q + (q . k) u), so the two dot
// products of every column with k and q are taken in one pass over the old
// state, before u is known: the state is read once, held in registers and
// written once.  8 K V bytes a head set the time.
//
// A wave owns 32 columns of one head: 8 lanes of 4 columns (128 bytes of a
// row) times 8 lanes of K / 8 rows, K / 2 registers a lane, no LDS and no
// barrier; the row lanes' sums meet by lane exchange.  64 rows x 64 heads x
// 128 x 64 (270 MB): 45 us, 6.0 TB/s; 250 rows x 32 heads x 128 x 128 (1.03
// GB): 200 us, 5.2 TB/s, and the same for linear attention (a large copy: 5.1 to 5.4).
#include "gdn_internal.h"
#include "gdn_mixer.hpp"

namespace gdn {
namespace {

constexpr int kMostWaves = 4;  // of a workgroup

// Sum over the 8 row lanes (lane bits 3, 4, 5).
__device__ __forceinline__ float rows_sum(float v) {
  v += dpp_mov<0x128>(v);  // row_ror:8
  v += __shfl_xor(v, 16);
  v += __shfl_xor(v, 32);
  return v;
}

// N consecutive elements of type E as floats (N * sizeof(E) bytes, aligned to
// the smaller of that and 16)
template <typename E, int N>
__device__ __forceinline__ void load_n(float (&r)[N], const E *p) {
  constexpr int PER = N * (int)sizeof(E) < 16 ? N : 16 / (int)sizeof(E);
  typedef E piece __attribute__((ext_vector_type(PER)));
#pragma unroll
  for (int i = 0; i < N / PER; ++i) {
    const piece x = reinterpret_cast<const piece *>(p)[i];
#pragma unroll
    for (int j = 0; j < PER; ++j) r[i * PER + j] = to_f32(x[j]);
  }
}

template <typename E, int K, int RULE>
__global__ __launch_bounds__(64 * kMostWaves) void step_kernel(StepArgs a) {
  constexpr int R = K / 8;  // rows a lane
  constexpr bool DELTA = RULE == kStepDelta;
  const int lane = threadIdx.x & 63, cl = lane & 7, rl = lane >> 3;
  const int slices = a.V >> 5;
  const int64_t unit = (int64_t)blockIdx.x * (blockDim.x >> 6) + wave_of(threadIdx.x);
  const int sl = (int)(unit % slices), h = (int)(unit / slices % a.Hv);
  const int64_t row = unit / slices / a.Hv;
  if (row >= a.B) return;
  const int hq = h / (a.Hv / a.Hq);
  const int col = 32 * sl + 4 * cl;
  E *o = static_cast<E *>(a.o) + (row * a.Hv + h) * a.V + col;
  int64_t slot = row;
  bool live = true;
  if (a.index) {
    slot = a.index[row];
    live = slot >= 0 && slot < a.slots;
    // a slot named twice belongs to the first row that names it
    bool twice = false;
    for (int64_t j = lane; j < row; j += 64) twice |= a.index[j] == slot;
    live = live && !__any(twice);
  }
  if (!live) {
    if (rl == 0) st4(o, 0.f, 0.f, 0.f, 0.f);
    return;
  }
  float *S = a.state + ((slot * a.Hv + h) * K + rl * R) * (int64_t)a.V + col;
  f32x4 s[R];
#pragma unroll
  for (int r = 0; r < R; ++r) s[r] = *reinterpret_cast<const f32x4 *>(S + (int64_t)r * a.V);
  float q[R], k[R], v[4];
  load_n<E, R>(q, static_cast<const E *>(a.q) + row * a.qs + hq * K + rl * R);
  load_n<E, R>(k, static_cast<const E *>(a.k) + row * a.ks + hq * K + rl * R);
  load_n<E, 4>(v, static_cast<const E *>(a.v) + row * a.vs + (int64_t)h * a.V + col);
  const float be = RULE == kStepDecay ? 0.f : to_f32(static_cast<const E *>(a.beta)[row * a.Hv + h]);

  if (DELTA && a.l2) {
    float qq = 0.f, kk = 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      qq += q[r] * q[r];
      kk += k[r] * k[r];
    }
    const float fq = 1.f / __builtin_sqrtf(rows_sum(qq) + 1e-6f);
    const float fk = 1.f / __builtin_sqrtf(rows_sum(kk) + 1e-6f);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      q[r] *= fq;
      k[r] *= fk;
    }
  }
  float qk = 0.f;
  f32x4 sq = zero4(), sk = zero4();
#pragma unroll
  for (int r = 0; r < R; ++r) {
    qk += q[r] * k[r];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      sq[i] += q[r] * s[r][i];
      if (DELTA) sk[i] += k[r] * s[r][i];
    }
  }
  qk = rows_sum(qk);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    sq[i] = rows_sum(sq[i]);
    if (DELTA) sk[i] = rows_sum(sk[i]);
  }
  float decay, u[4], out[4];
  if (DELTA) {
    decay = expf(a.g[row * a.Hv + h]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      u[i] = be * (v[i] - decay * sk[i]);
      out[i] = a.scale * (decay * sq[i] + qk * u[i]);
    }
  } else if (RULE == kStepDecay) {
    const float most = expf(a.g[h]);
    decay = most > __FLT_MAX__ ? __FLT_MAX__ : most;  // a state of 0 stays 0
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      u[i] = v[i];
      out[i] = a.scale * (decay * sq[i] + qk * u[i]);
    }
  } else {
    const float z = be + (a.dt_bias ? a.dt_bias[h] : 0.f);
    const float delta = a.softplus ? softplusf(z) : z;
    const float skip = a.D ? a.D[h] : 0.f;
    decay = expf(delta * a.A[h]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      u[i] = delta * v[i];
      out[i] = decay * sq[i] + qk * u[i] + skip * v[i];
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    f32x4 n;
#pragma unroll
    for (int i = 0; i < 4; ++i) n[i] = decay * s[r][i] + k[r] * u[i];
    *reinterpret_cast<f32x4 *>(S + (int64_t)r * a.V) = n;
  }
  if (rl == 0) st4(o, out[0], out[1], out[2], out[3]);
}

template <typename E, int K>
hipError_t go(const StepArgs &a, hipStream_t st) {
  const int64_t units = (int64_t)a.B * a.Hv * (a.V / 32);
  // a compute unit each while there are no more waves than those
  const int waves = units > compute_units() ? kMostWaves : 1;
  const unsigned blocks = (unsigned)((units + waves - 1) / waves);
  if (a.rule == kStepDelta) {
    KernelTimer kt("delta_step", st);
    step_kernel<E, K, kStepDelta><<<blocks, 64 * waves, 0, st>>>(a);
  } else if (a.rule == kStepDecay) {
    KernelTimer kt("attn_step", st);
    step_kernel<E, K, kStepDecay><<<blocks, 64 * waves, 0, st>>>(a);
  } else {
    KernelTimer kt("scan_step", st);
    step_kernel<E, K, kStepScan><<<blocks, 64 * waves, 0, st>>>(a);
  }
  return hipGetLastError();
}
template <typename E>
hipError_t go_k(const StepArgs &a, hipStream_t st) {
  return a.K == 32 ? go<E, 32>(a, st) : a.K == 64 ? go<E, 64>(a, st) : go<E, 128>(a, st);
}

}  // namespace

hipError_t launch_step(const StepArgs &a, hipStream_t st) {
  return a.dtype == 1 ? go_k<bf16>(a, st) : go_k<float>(a, st);
}

}  // namespace gdn
