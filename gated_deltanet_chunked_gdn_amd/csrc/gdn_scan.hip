// The selective state-space scan over whole sequences, and its backward.  Per
// v-head, with the state S (K x V, fp32), delta_t = softplus(dt_t + dt_bias)
// (or dt_t + dt_bias) and g_t = delta_t A:
//
//   S_t = e^{g_t} S_{t-1} + delta_t b_t x_t^T,   y_t = S_t^T c_t + D x_t
//
// Backward, with Z_t the gradient of S_t (all that follows from it, token t's
// own output included):
//
//   Z_t = c_t dy_t^T + Z'_t,  Z'_t = e^{g_{t+1}} Z_{t+1}
//   dc_t = S_t dy_t,  db_t = delta_t Z_t x_t,  dx_t = delta_t Z_t^T b_t + D dy_t
//   dg_t = <e^{g_t} S_{t-1}, Z_t>
//   d delta_t = r_t + m_t + A dg_t,
//     r_t = x_t . Z'_t^T b_t,  m_t = (c_t . b_t)(x_t . dy_t)
//
// Sequences are cut into segments that run side by side: a pass over every
// segment from a zero state, a scan of the segments' ends, and the pass that
// writes the results from the true start states (backward: the same in
// reverse order for Z).
//
// The kernels of this file hold the state in fp32 registers, one column (or
// row) of it a lane, and walk token by token: they are the form for fp32
// problems.
#include "gdn_internal.h"
#include "gdn_scan.hpp"

namespace gdn {
namespace scan {
namespace {

constexpr int TB = 16;      // tokens staged at a time
constexpr int kAhead = 8;  // segments whose states a carry has in flight

// What a sweep does.  Lane operand L (one value a lane and token), uniform
// operands U (the update's other factor) and P (the output's factor):
//   kOut  forward, lanes over V:  L = delta x, U = b, P = c, out = y
//   kDc   forward, lanes over K:  L = delta b, U = x, P = dy, out = dc
//   kDx   reverse, lanes over V:  L = dy, U = c, P = b, out -> dx, r, dD
//   kDb   reverse, lanes over K:  L = c, U = dy, P = x, out -> db
//   kLocal / kRLocal: the state alone, from zero (lanes over V)
enum Mode { kLocal, kOut, kDc, kRLocal, kDx, kDb };

struct Sweep {
  const void *L, *U, *P;
  int64_t ls, us, ps;  // elements from one token to the next
  int l_v, u_v, p_v;   // operand lies with the v-heads (else the c/b heads)
  int LD;              // lane dimension (K or V, 64 at the most)
};

template <int RD, int MODE>
__global__ __launch_bounds__(64) void sweep_kernel(ScanArgs a, Layout w, Sweep s) {
  constexpr bool REV = MODE == kRLocal || MODE == kDx || MODE == kDb;
  constexpr bool OUT = MODE != kLocal && MODE != kRLocal;
  constexpr bool LANE_V = MODE != kDc && MODE != kDb;
  __shared__ __align__(16) float us[TB][RD], ps[OUT ? TB : 1][RD];
  __shared__ float del[TB], dec[TB];
  const int lane = threadIdx.x, h = blockIdx.x % a.Hv;
  const int64_t slot = blockIdx.x / a.Hv;
  const SlotLoc loc = locate(a, slot);
  if (!loc.used || (MODE == kLocal && loc.last)) return;
  const int hq = h / (a.Hv / a.Hq);
  const bool on = lane < s.LD;
  const int lc = on ? lane : s.LD - 1;  // idle lanes of a 32-wide operand read along, and write nothing
  const float *L = static_cast<const float *>(s.L) + (int64_t)(s.l_v ? h : hq) * s.LD + lc;
  const float *U = static_cast<const float *>(s.U) + (int64_t)(s.u_v ? h : hq) * RD;
  const float *P = OUT ? static_cast<const float *>(s.P) + (int64_t)(s.p_v ? h : hq) * RD : nullptr;
  const float A = a.A[h], bias = a.dt_bias ? a.dt_bias[h] : 0.f, skip = a.D ? a.D[h] : 0.f;
  const int64_t kv = (int64_t)a.K * a.V;
  const int64_t sr = LANE_V ? a.V : 1, so = LANE_V ? lc : (int64_t)lc * a.V;

  float S[RD];
  const float *src = nullptr;
  if (MODE == kOut || MODE == kDc)
    src = a.one_seg && MODE == kOut ? (a.h0 ? a.h0 + (loc.n * (int64_t)a.Hv + h) * kv : nullptr)
                                    : w.start(a) + (slot * a.Hv + h) * kv;
  if (MODE == kDx || MODE == kDb) src = w.zend(a) + (slot * a.Hv + h) * kv;
#pragma unroll
  for (int r = 0; r < RD; ++r) S[r] = src ? src[r * sr + so] : 0.f;

  float total = 0.f, dD = 0.f;
  const int64_t nt = loc.t1 - loc.t0;
  for (int64_t b0 = 0; b0 < nt; b0 += TB) {
    // token j of the block is t0 + b0 + j, or counted back from the end
    const int nb = (int)(nt - b0 < TB ? nt - b0 : TB);
    __syncthreads();
    for (int i = lane; i < TB * RD; i += 64) {
      const int j = i / RD, r = i % RD;
      const int jc = j < nb ? j : nb - 1;
      const int64_t t = REV ? loc.t1 - 1 - (b0 + jc) : loc.t0 + b0 + jc;
      us[j][r] = U[t * s.us + r];
      if (OUT) ps[j][r] = P[t * s.ps + r];
    }
    if (lane < nb) {
      const int64_t t = REV ? loc.t1 - 1 - (b0 + lane) : loc.t0 + b0 + lane;
      const float z = static_cast<const float *>(a.dt)[t * a.Hv + h] + bias;
      const float d = a.softplus ? softplusf(z) : z;
      del[lane] = d;
      dec[lane] = d * A;
    }
    float lv[TB];
#pragma unroll
    for (int j = 0; j < TB; ++j) {
      const int jc = j < nb ? j : nb - 1;
      const int64_t t = REV ? loc.t1 - 1 - (b0 + jc) : loc.t0 + b0 + jc;
      lv[j] = L[t * s.ls];
    }
    __syncthreads();
#pragma unroll 1
    for (int j = 0; j < nb; ++j) {
      const int64_t t = REV ? loc.t1 - 1 - (b0 + j) : loc.t0 + b0 + j;
      const float delta = del[j], decay = expf(dec[j]);
      total += dec[j];
      float mine = 0.f;  // lv[j] with j in a register index the compiler can see
#pragma unroll
      for (int i = 0; i < TB; ++i) mine = i == j ? lv[i] : mine;
      const float f = REV ? mine : delta * mine;
      // kDc, kDx: the output without the token's own update, and u . p
      constexpr bool OWN = MODE == kDc || MODE == kDx;
      float out = 0.f, up = 0.f;
#pragma unroll
      for (int r = 0; r < RD; r += 4) {
        const f32x4 u = *reinterpret_cast<const f32x4 *>(&us[j][r]);
        f32x4 p = zero4();
        if (OUT) p = *reinterpret_cast<const f32x4 *>(&ps[j][r]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float old = REV ? S[r + i] : decay * S[r + i], now = old + f * u[i];
          if (OUT) out += (OWN ? old : now) * p[i];
          if (OWN) up += u[i] * p[i];
          S[r + i] = REV ? decay * now : now;
        }
      }
      if (MODE == kOut) {
        const float x = mine;
        if (on) static_cast<float *>(a.y)[(t * a.Hv + h) * a.V + lane] = out + skip * x;
      } else if (MODE == kDc || MODE == kDb) {
        float *part = MODE == kDc ? w.dc_part(a) : w.db_part(a);
        if (on) part[(t * a.Hv + h) * a.K + lane] = MODE == kDc ? out + f * up : delta * out;
      } else if (MODE == kDx) {
        const float x = static_cast<const float *>(a.x)[t * a.xs + (int64_t)h * a.V + lc];
        if (on) static_cast<float *>(a.dx)[(t * a.Hv + h) * a.V + lane] = delta * (out + f * up) + skip * mine;
        const float v = wave_sum(on ? x * out : 0.f), xd = wave_sum(on ? x * mine : 0.f);
        if (lane == 0) {
          const int64_t i = (int64_t)h * a.s.tokens + t;
          w.r_part(a)[i] = v;
          w.m_part(a)[i] = xd * up;
        }
        dD += xd;
      }
    }
  }
  if (MODE == kLocal || MODE == kRLocal) {
    float *dst = (MODE == kLocal ? w.start(a) : w.zend(a)) + (slot * a.Hv + h) * kv;
    if (on)
      for (int r = 0; r < RD; ++r) dst[r * sr + so] = S[r];
    // (in the backward the reverse pass, which has every segment: one writer)
    if ((MODE == kRLocal || !a.dy) && lane == 0) w.decay(a)[slot * a.Hv + h] = total;
  }
  if (MODE == kOut && loc.last && a.ht && on) {
    float *dst = a.ht + (loc.n * (int64_t)a.Hv + h) * kv;
    for (int r = 0; r < RD; ++r) dst[r * sr + so] = S[r];
  }
  if (MODE == kDx) {
    if (lane == 0) w.dd_part(a)[slot * a.Hv + h] = dD;
  }
}

// The segments' local ends -> every segment's start state (in place).  One
// thread has 4 elements of one head's state.
__device__ __forceinline__ void carry(const ScanArgs &a, const Layout &w, int64_t i) {
  const int64_t kv4 = (int64_t)a.K * a.V / 4;
  const int64_t e = i % kv4, h = i / kv4 % a.Hv, n = i / kv4 / a.Hv;
  if (n >= a.s.N) return;
  const Span sp = seq_span(a.s, (int)n);
  const int64_t slot = first_slot(a.s, sp, (int)n, a.seg), ns = segs_of(sp, a.seg);
  f32x4 cur = zero4();
  const int64_t own = (n * a.Hv + h) * kv4 + e;
  if (a.h0) cur = reinterpret_cast<const f32x4 *>(a.h0)[own];
  f32x4 *H = reinterpret_cast<f32x4 *>(w.start(a)) + (slot * a.Hv + h) * kv4 + e;
  const float *g = w.decay(a) + slot * a.Hv + h;
  const int64_t step = a.Hv * kv4, read = ns - 1;  // segments whose own state is there
  for (int64_t s = 0; s < ns; s += kAhead) {
    f32x4 x[kAhead];
    float d[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int64_t t = s + j < read ? s + j : 0;
      x[j] = H[t * step];
      d[j] = g[t * a.Hv];
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (s + j >= ns) break;
      H[(s + j) * step] = cur;
      if (s + j >= read) break;
      const float f = expf(d[j]);
#pragma unroll
      for (int k = 0; k < 4; ++k) cur[k] = f * cur[k] + x[j][k];
    }
  }
}

// In reverse: every segment's local gradient of its start state -> the
// gradient of its last state from what follows it (in place), and dh0.
__device__ __forceinline__ void rcarry(const ScanArgs &a, const Layout &w, int64_t i) {
  const int64_t kv4 = (int64_t)a.K * a.V / 4;
  const int64_t e = i % kv4, h = i / kv4 % a.Hv, n = i / kv4 / a.Hv;
  if (n >= a.s.N) return;
  const Span sp = seq_span(a.s, (int)n);
  const int64_t slot = first_slot(a.s, sp, (int)n, a.seg), ns = segs_of(sp, a.seg);
  f32x4 cur = zero4();
  const int64_t own = (n * a.Hv + h) * kv4 + e;
  if (a.dht) cur = reinterpret_cast<const f32x4 *>(a.dht)[own];
  f32x4 *Z = reinterpret_cast<f32x4 *>(w.zend(a)) + (slot * a.Hv + h) * kv4 + e;
  const float *g = w.decay(a) + slot * a.Hv + h;
  const int64_t step = a.Hv * kv4;
  for (int64_t s = ns - 1; s >= 0; s -= kAhead) {
    f32x4 x[kAhead];
    float d[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int64_t t = s - j > 0 ? s - j : 0;
      x[j] = Z[t * step];
      d[j] = g[t * a.Hv];
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (s - j < 0) break;
      Z[(s - j) * step] = cur;
      const float f = expf(d[j]);
#pragma unroll
      for (int k = 0; k < 4; ++k) cur[k] = f * cur[k] + x[j][k];
    }
  }
  if (a.dh0) reinterpret_cast<f32x4 *>(a.dh0)[own] = cur;
}

// Both in one launch where there are both (`blocks` workgroups each).
__global__ __launch_bounds__(256) void carry_kernel(ScanArgs a, Layout w, int64_t blocks) {
  const int64_t b = blockIdx.x;
  if (b < blocks)
    carry(a, w, b * 256 + threadIdx.x);
  else
    rcarry(a, w, (b - blocks) * 256 + threadIdx.x);
}

// dg, then ddt and the segment's part of dA, ddt_bias and dD.
//
// dg_t = <e^{g_t} S_{t-1}, Z_t> of a segment whose first state is S0 and whose
// last state has the gradient Z1, with E_ij the decay from token j to i, p_t
// that from the segment's start to t and w_t that from t to its end:
//
//   dg_t = p_end <S0, Z1> + sum_{i >= t} p_i c_i . S0 dy_i + sum_{j < t} delta_j w_j b_j . Z1 x_j
//          + sum_{j < t <= i} E_ij delta_j (c_i . b_j)(dy_i . x_j)
//
// which is the product taken apart: nothing cancels that does not cancel in it.
// (As the chain dg_{t+1} + c_t . e^{g_t} S_{t-1} dy_t - delta_t r_t it was off by
// 3e-3 of dA where tokens forget to e^-9 and dg is far below both terms.)
//
// A workgroup has one segment (64 tokens at the most) of one head, a wave 16 of
// its tokens: their rows of C B^T and DY X^T, S0 dy and Z1 x, all by fp32
// matrix instructions.  Log decays are summed in 64 bits, so that the decay
// between two tokens is as good as its own logarithm.
//
// 2 x 4096 tokens x 16 heads, K = V = 64: 83 us (the chain: 19, of a backward of
// 590), three workgroups a compute unit by registers and latency of the steps.
template <int K, int V>
__global__ __launch_bounds__(256, 3) void gates_kernel(ScanArgs a, Layout w) {
  constexpr int KF = K / 16, VF = V / 16, P = V + 4, WP = 65;
  __shared__ __align__(16) float mats[2 * K * P > 64 * WP ? 2 * K * P : 64 * WP];  // S0 and Z1, then the pairs
  __shared__ double gam[64];
  __shared__ float del[64], own[2][64], pairs[64];
  float *const s0 = mats, *const z1 = mats + K * P;
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_of(tid), l16 = lane & 15, q = lane >> 4;
  const int64_t units = a.slots * a.Hv;
  for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const int h = (int)(unit % a.Hv), hq = h / (a.Hv / a.Hq);
    const SlotLoc loc = locate(a, unit / a.Hv);
    float *part = w.head_part(a) + unit * 3;
    const int nt = loc.used ? (int)(loc.t1 - loc.t0) : 0;
    if (nt <= 0) {
      if (tid < 3) part[tid] = 0.f;
      continue;
    }
    const float A = a.A[h], bias = a.dt_bias ? a.dt_bias[h] : 0.f;
    auto dt_at = [&](int tok) { return static_cast<const float *>(a.dt)[(loc.t0 + tok) * a.Hv + h] + bias; };
    __syncthreads();  // the unit before is done with LDS
    for (int i = tid; i < K * V / 4; i += 256) {
      const int at = i / (V / 4) * P + i % (V / 4) * 4;
      *reinterpret_cast<f32x4 *>(s0 + at) = reinterpret_cast<const f32x4 *>(w.start(a) + unit * K * V)[i];
      *reinterpret_cast<f32x4 *>(z1 + at) = reinterpret_cast<const f32x4 *>(w.zend(a) + unit * K * V)[i];
    }
    if (wave == 0) {
      const float z = dt_at(lane < nt ? lane : nt - 1);
      const float delta = lane < nt ? (a.softplus ? softplusf(z) : z) : 0.f, g = delta * A;
      gam[lane] = sum_upto(g < -1e4f ? -1e4f : g, lane);  // (e^-1e4 is 0; an infinity would leave no difference)
      del[lane] = delta;
    }
    __syncthreads();
    // rows of the tokens 16 blk + l16, elements 16 s + 4 q ..
    auto rows = [&](f32x4 *r, const void *p, int64_t stride, int col, int blk, int frags) {
      const int tok = 16 * blk + l16 < nt ? 16 * blk + l16 : nt - 1;
      const float *e = static_cast<const float *>(p) + (loc.t0 + tok) * stride + col + 4 * q;
      for (int s = 0; s < frags; ++s) r[s] = *reinterpret_cast<const f32x4 *>(e + 16 * s);
    };
    auto prod = [](const f32x4 &x, const f32x4 &y, f32x4 c) {
#pragma unroll
      for (int k = 0; k < 4; ++k) c = Mma<float>::mma(x[k], y[k], c);
      return c;
    };
    const int64_t ys = (int64_t)a.Hv * V;
    const double end = gam[nt - 1];
    f32x4 pt[4];  // this wave's tokens i (rows), all j before the block's end
    if (16 * wave < nt) {
      f32x4 cf[KF], bf[KF], df[VF], xf[VF];
      rows(cf, a.c, a.cs, hq * K, wave, KF);
      rows(df, a.dy, ys, h * V, wave, VF);
#pragma unroll 1
      for (int jb = 0; jb <= wave; ++jb) {
        rows(bf, a.b, a.bs, hq * K, jb, KF);
        rows(xf, a.x, a.xs, h * V, jb, VF);
        f32x4 g = zero4(), m = zero4();
#pragma unroll
        for (int s = 0; s < KF; ++s) g = prod(cf[s], bf[s], g);
#pragma unroll
        for (int s = 0; s < VF; ++s) m = prod(df[s], xf[s], m);
        const int j = 16 * jb + l16;
        f32x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = 16 * wave + 4 * q + e;
          const bool in = j < i && i < nt;
          const float decay = expf(in ? (float)(gam[i] - gam[j]) : 0.f);
          v[e] = in ? decay * g[e] * (m[e] * del[j]) : 0.f;
        }
#pragma unroll
        for (int b = 0; b < 4; ++b) pt[b] = b == jb ? v : pt[b];
      }
      // (bf, xf: of the wave's own tokens)
      float sa = 0.f, sb = 0.f;
#pragma unroll
      for (int k = 0; k < KF; ++k) {
        f32x4 u = zero4(), v = zero4();  // rows 16 k + 4 q .. of S0 dy^T and Z1 x^T, columns the tokens
        const int at = (16 * k + l16) * P + 4 * q;
#pragma unroll
        for (int s = 0; s < VF; ++s) {
          u = prod(*reinterpret_cast<const f32x4 *>(s0 + at + 16 * s), df[s], u);
          v = prod(*reinterpret_cast<const f32x4 *>(z1 + at + 16 * s), xf[s], v);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          sa += cf[k][e] * u[e];
          sb += bf[k][e] * v[e];
        }
      }
      sa += __shfl_xor(sa, 16);
      sb += __shfl_xor(sb, 16);
      sa += __shfl_xor(sa, 32);
      sb += __shfl_xor(sb, 32);
      const int tok = 16 * wave + l16;
      if (q == 0 && tok < nt) {
        own[0][tok] = sa * expf((float)gam[tok]);
        own[1][tok] = sb * (del[tok] * expf((float)(end - gam[tok])));
      }
    }
    double sz = 0.;
    if (wave == 0)
      for (int i = lane; i < K * V; i += 64) {
        const int at = i / V * P + i % V;
        sz += (double)s0[at] * z1[at];
      }
    __syncthreads();
    float *const tri = mats;  // [i][j], j < i
    if (16 * wave < nt) {
#pragma unroll
      for (int jb = 0; jb < 4; ++jb)
        if (jb <= wave)
#pragma unroll
          for (int e = 0; e < 4; ++e) tri[(16 * wave + 4 * q + e) * WP + 16 * jb + l16] = pt[jb][e];
    }
    __syncthreads();
    // the pairs j < t <= i: a lane sums its row i up to t, the lanes from t on are added.
    // (Rows i < t, and with them what no wave wrote, stay out.)
    if (16 * wave < nt) {
      float row = 0.f;
      for (int j = 0; j < 16 * wave; ++j) row += tri[lane * WP + j];
      for (int t = 16 * wave; t < 16 * wave + 16 && t < nt; ++t) {
        const float v = wave_sum(lane >= t && lane < nt ? row : 0.f);
        if (lane == 0) pairs[t] = v;
        row += tri[lane * WP + t];
      }
    }
    __syncthreads();
    if (wave) continue;
    // lane 0 the last token
    const bool on = lane < nt;
    const int tok = on ? nt - 1 - lane : 0;
    const int64_t t = loc.t0 + tok, i = (int64_t)h * a.s.tokens + t;
    const float z = dt_at(tok);
    const double rv = on ? w.r_part(a)[i] : 0.f, mv = on ? w.m_part(a)[i] : 0.f;
    const double dg = wave_sum64(sz) * expf((float)end) + sum_upto(on ? own[0][tok] : 0.f, lane) +
                      sum_before(on ? own[1][tok] : 0.f, lane) + pairs[tok];
    double dd = rv + mv + A * dg;
    if (a.softplus) dd *= 1.f / (1.f + expf(-z));
    if (on) static_cast<float *>(a.ddt)[t * a.Hv + h] = (float)dd;
    const double dA = wave_sum64(on ? del[tok] * dg : 0.), dbias = wave_sum64(on ? dd : 0.);
    if (lane == 0) {
      part[0] = (float)dA;
      part[1] = (float)dbias;
      part[2] = w.dd_part(a)[unit];
    }
  }
}

// dA, ddt_bias, dD of a head: the segments' parts, 64 interleaved sums joined
// in a fixed order.
__global__ __launch_bounds__(64) void heads_kernel(ScanArgs a, Layout w) {
  const int h = blockIdx.x;
  double v[3] = {0., 0., 0.};
  for (int64_t s = threadIdx.x; s < a.slots; s += 64)
    for (int k = 0; k < 3; ++k) v[k] += w.head_part(a)[(s * a.Hv + h) * 3 + k];
  float *out[3] = {a.dA, a.ddt_bias, a.dD};
  for (int k = 0; k < 3; ++k) {
    const double t = wave_sum64(v[k]);
    if (threadIdx.x == 0 && out[k]) out[k][h] = (float)t;
  }
}

// dc, db: the sum over the heads of a group, 4 elements a thread.  (Tokens that
// no sequence has have no parts, and their rows are not the kernel's.)
__global__ __launch_bounds__(256) void group_kernel(ScanArgs a, Layout w) {
  const int64_t k4 = a.K / 4, n = a.s.tokens * a.Hq * k4;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  const int R = a.Hv / a.Hq;
  const int64_t e = i % k4, th = i / k4;  // th = token * Hq + hq
  if (a.s.cu) {
    const int64_t t = th / a.Hq;
    const Span sp = seq_span(a.s, seq_of(a.s, t));
    if (t < sp.first || t >= sp.end) return;
  }
  const f32x4 *pc = reinterpret_cast<const f32x4 *>(w.dc_part(a)) + th * R * k4 + e;
  const f32x4 *pb = reinterpret_cast<const f32x4 *>(w.db_part(a)) + th * R * k4 + e;
  f32x4 c = zero4(), b = zero4();
  for (int r = 0; r < R; ++r) {
    c += pc[r * k4];
    b += pb[r * k4];
  }
  reinterpret_cast<f32x4 *>(a.dc)[i] = c;
  reinterpret_cast<f32x4 *>(a.db)[i] = b;
}

template <int MODE>
hipError_t sweep(const char *name, const ScanArgs &a, const Layout &w, const Sweep &s, int rd, hipStream_t st) {
  const unsigned blocks = (unsigned)(a.slots * a.Hv);
  KernelTimer kt(name, st);
  if (rd == 32)
    sweep_kernel<32, MODE><<<blocks, 64, 0, st>>>(a, w, s);
  else
    sweep_kernel<64, MODE><<<blocks, 64, 0, st>>>(a, w, s);
  return hipGetLastError();
}

void gates(const ScanArgs &a, const Layout &w, hipStream_t st) {
  // (a launch has fewer than 2^32 threads; a workgroup takes more units beyond that)
  const unsigned blocks = (unsigned)(a.slots * a.Hv < (1 << 22) ? a.slots * a.Hv : 1 << 22);
  switch (a.K * 1000 + a.V) {
    case 32032: gates_kernel<32, 32><<<blocks, 256, 0, st>>>(a, w); break;
    case 32064: gates_kernel<32, 64><<<blocks, 256, 0, st>>>(a, w); break;
    case 64032: gates_kernel<64, 32><<<blocks, 256, 0, st>>>(a, w); break;
    default: gates_kernel<64, 64><<<blocks, 256, 0, st>>>(a, w);
  }
}

unsigned carry_blocks(const ScanArgs &a) {
  return (unsigned)(((int64_t)a.s.N * a.Hv * a.K * a.V / 4 + 255) / 256);
}

hipError_t fwd(const ScanArgs &a, hipStream_t st) {
  const Layout w = layout(a, false);
  hipError_t e = hipSuccess;
  const Sweep out{a.x, a.b, a.c, a.xs, a.bs, a.cs, 1, 0, 0, a.V};
  if (!a.one_seg) {
    e = sweep<kLocal>("scan_local", a, w, out, a.K, st);
    if (e != hipSuccess) return e;
    KernelTimer kt("scan_carry", st);
    carry_kernel<<<carry_blocks(a), 256, 0, st>>>(a, w, carry_blocks(a));
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  return sweep<kOut>("scan_out", a, w, out, a.K, st);
}

hipError_t fwd_mma(const ScanArgs &a, hipStream_t st) {
  const Layout w = layout(a, false);
  if (!a.one_seg) {
    hipError_t e = launch_mma_local(a, w, st);
    if (e != hipSuccess) return e;
    KernelTimer kt("scan_carry", st);
    carry_kernel<<<carry_blocks(a), 256, 0, st>>>(a, w, carry_blocks(a));
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  return launch_mma_out(a, w, st);
}

hipError_t bwd_mma(const ScanArgs &a, hipStream_t st) {
  const Layout w = layout(a, true);
  hipError_t e;
  if (!a.one_seg) {
    if ((e = launch_mma_locals(a, w, st)) != hipSuccess) return e;
    KernelTimer kt("scan_carry", st);
    carry_kernel<<<2 * carry_blocks(a), 256, 0, st>>>(a, w, carry_blocks(a));
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if ((e = launch_mma_states(a, w, st)) != hipSuccess) return e;
  return launch_mma_grad(a, w, st);
}

hipError_t bwd(const ScanArgs &a, hipStream_t st) {
  const Layout w = layout(a, true);
  const int64_t qs = (int64_t)a.Hv * a.V;  // dy is contiguous
  const Sweep out{a.x, a.b, a.c, a.xs, a.bs, a.cs, 1, 0, 0, a.V};
  const Sweep dc{a.b, a.x, a.dy, a.bs, a.xs, qs, 0, 1, 1, a.K};
  const Sweep dx{a.dy, a.c, a.b, qs, a.cs, a.bs, 1, 0, 0, a.V};
  const Sweep db{a.c, a.dy, a.x, a.cs, qs, a.xs, 0, 1, 1, a.K};
  hipError_t e;
#define GDN_DO(x) \
  if ((e = (x)) != hipSuccess) return e
  GDN_DO((sweep<kLocal>("scan_local", a, w, out, a.K, st)));
  GDN_DO((sweep<kRLocal>("scan_rlocal", a, w, dx, a.K, st)));
  {
    KernelTimer kt("scan_carry", st);
    carry_kernel<<<2 * carry_blocks(a), 256, 0, st>>>(a, w, carry_blocks(a));
    GDN_DO(hipGetLastError());
  }
  GDN_DO((sweep<kDc>("scan_dc", a, w, dc, a.V, st)));
  GDN_DO((sweep<kDx>("scan_dx", a, w, dx, a.K, st)));
  GDN_DO((sweep<kDb>("scan_db", a, w, db, a.V, st)));
  {
    KernelTimer kt("scan_gates", st);
    gates(a, w, st);
    heads_kernel<<<a.Hv, 64, 0, st>>>(a, w);
    GDN_DO(hipGetLastError());
  }
  if (a.s.tokens) {
    KernelTimer kt("scan_group", st);
    const int64_t n = a.s.tokens * a.Hq * (a.K / 4);
    group_kernel<<<(unsigned)((n + 255) / 256), 256, 0, st>>>(a, w);
    GDN_DO(hipGetLastError());
  }
#undef GDN_DO
  return hipSuccess;
}

}  // namespace
}  // namespace scan

// Segments: as long as the whole sequence unless that leaves compute units
// without work, then as many as give each a workgroup of the matrix kernels
// (bf16, whole chunks of 64) or eight waves of the sweeps (fp32, which walk token
// by token: down to 16 tokens).  fp32 backward: 64 tokens at the most,
// what a workgroup of the gates' kernel has.
ScanPlan scan_plan(const ScanArgs &a0, bool bwd) {
  ScanArgs a = a0;
  // workgroups a segment
  const int slices = a.Hv / a.Hq * (a.V / 32);
  const int64_t per = a.dtype == 1 ? (int64_t)a.Hq * (slices / scan::slices_per_block(slices)) : a.Hv;
  int64_t want = (compute_units() * (a.dtype == 1 ? 1 : 8) + per - 1) / per;  // segments over the whole batch
  if (want < a.s.N) want = a.s.N;
  int64_t seg = (a.s.tokens + want - 1) / want;
  const int64_t unit = a.dtype == 1 ? 64 : scan::TB;
  seg = (seg + unit - 1) / unit * unit;
  if (seg < unit) seg = unit;
  if (bwd && a.dtype != 1 && seg > 64) seg = 64;
  ScanPlan p;
  p.seg = (int)seg;
  a.slots = p.slots = scan::slots_of(a.s, p.seg);
  a.one_seg = p.one_seg = (!bwd || a.dtype == 1) && a.s.T <= seg;
  p.ws = scan::layout(a, bwd).total;
  return p;
}

hipError_t launch_scan_fwd(const ScanArgs &a, hipStream_t st) {
  return a.dtype == 1 ? scan::fwd_mma(a, st) : scan::fwd(a, st);
}
hipError_t launch_scan_bwd(const ScanArgs &a, hipStream_t st) {
  return a.dtype == 1 ? scan::bwd_mma(a, st) : scan::bwd(a, st);
}

}  // namespace gdn
