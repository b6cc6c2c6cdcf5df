// The selective scan of bf16 problems on matrix instructions: chunks of 64
// tokens, the state of a head in MFMA accumulators.  With gamma_t the sum of
// log2 decays from the chunk's first token to t and S the state entering it,
//
//   y_i = 2^{gamma_i} S^T c_i + sum_{j <= i} (c_i . b_j) 2^{gamma_i - gamma_j} delta_j x_j + D x_i
//   S'  = 2^{gamma_L} S + sum_j b_j (2^{gamma_L - gamma_j} delta_j x_j)^T
//
// A wave owns VW = min(V, 64) columns of one head's state and a segment's
// chunks in order; the waves of a workgroup are column slices that share c
// and b (the v-heads of a group, and the halves of a head of 128), which the
// workgroup stages for the next chunk while it works on this one.  No wave
// waits for another but at the one barrier a chunk.
//
// Everything is arranged so that accumulators are operands without moving
// (gdn_slice.hpp): S tiles (rows k, lane v) give S^T for c; C B^T is formed
// as (B C^T) with rows j and lane i, which is P^T as the second operand of
// X^T P^T, and y comes out transposed, lane i, four consecutive v a quad:
// 16-byte stores after one exchange between the wave's halves.
//
// Roundings to bf16: P and the state as operands of y (y itself is bf16).
// The state is held to fp32: its update takes b as it is and the weighted x
// as the sum of two bf16 parts (2^-18 of it is lost).
#include "gdn_internal.h"
#include "gdn_scan.hpp"
#include "gdn_slice.hpp"

namespace gdn {
namespace scan {
namespace {

using slice::f32x16;
using slice::lds16;
using slice::mma32;
using slice::pi_pos;
using slice::put_pi;
using slice::slots;
using slice::TrA;
using slice::zero16;

constexpr float kLog2e = 1.44269504088896340736f;

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// Inclusive prefix sums inside each half (32 lanes) of the wave.
__device__ __forceinline__ float half_incl_scan(float x) {
  x += dpp_mov<0x111>(x);       // row_shr:1
  x += dpp_mov<0x112>(x);       // row_shr:2
  x += dpp_mov<0x114>(x);       // row_shr:4
  x += dpp_mov<0x118>(x);       // row_shr:8
  x += dpp_mov<0x142, 0xA>(x);  // row_bcast:15 into rows 1 and 3
  return x;
}
__device__ __forceinline__ float lane_f(float x, int l) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), l));
}

// Pieces of 16 bytes of one chunk's rows (64 x COLS bf16) in the registers of
// THREADS threads; rows past the sequence read as zeros.
template <int COLS, int THREADS>
struct Rows {
  static constexpr int N = 64 * COLS / 8 / THREADS;
  uint4 r[N];
  __device__ __forceinline__ void load(const bf16 *p, int64_t stride, int rows, int tid) {
    const uint32_t bytes = rows > 0 ? (uint32_t)(((rows - 1) * stride + COLS) * 2) : 0u;
    const auto rsrc = raw_buffer(p, bytes);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int pc = tid + i * THREADS, row = pc / (COLS / 8), col = pc % (COLS / 8);
      // (a row past the end may still lie inside the byte range of the last
      // row's neighbours in a wider tensor: it is sent past the range)
      r[i] = buf_load16(rsrc, row < rows ? (uint32_t)(row * stride * 2 + col * 16) : 0xFFFFFFF0u);
    }
  }
  __device__ __forceinline__ void store_pi(bf16 *lds, int pitch, int tid) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int pc = tid + i * THREADS, row = pc / (COLS / 8), col = pc % (COLS / 8);
      put_pi(lds + row * pitch, col, r[i]);
    }
  }
};

// What a wave keeps of a chunk's steps in LDS, by token: log2 decays summed
// from the token's half (32 tokens), delta, the weight of the token in the
// chunk's last state, and (first half) in the half's last state.
//
// A token whose own decay is below 2^kForget ends all that is before it to
// fp32 (2^-27 of a term is an eighth of its half step).  It counts as an
// exact 0 and stays out of the sums, where it would cost the differences
// between later tokens their digits; m0, m1 mark such tokens of the halves.
constexpr float kForget = -27.f;
struct Gates {
  float gam[64], del[64], w[64], u[32];
};
struct GateTotals {
  float t0, t1;     // the halves' sums of log2 decays
  uint32_t m0, m1;  // tokens that forget
  __device__ __forceinline__ float all() const { return m0 | m1 ? 0.f : exp2_hw(t0 + t1); }
};
// bits 0 .. i, and the bits above i
__device__ __forceinline__ uint32_t upto(uint32_t m, int i) { return m & (0xFFFFFFFFu >> (31 - i)); }
__device__ __forceinline__ uint32_t above(uint32_t m, int i) { return m & ~(0xFFFFFFFFu >> (31 - i)); }
__device__ __forceinline__ int last_bit(uint32_t m) { return m ? 31 - __builtin_clz(m) : 0; }

__device__ __forceinline__ GateTotals gates(Gates &s, float z, float A2, bool softplus, bool live, int lane) {
  const float d = live ? (softplus ? softplusf(z) : z) : 0.f;
  const float g = d * A2;
  const bool cut = g < kForget;
  const unsigned long long m = __ballot(cut);
  const float gam = half_incl_scan(cut ? 0.f : g);
  GateTotals t{lane_f(gam, 31), lane_f(gam, 63), (uint32_t)m, (uint32_t)(m >> 32)};
  const int i = lane & 31;
  const uint32_t later = lane < 32 ? above(t.m0, i) : above(t.m1, i);
  s.gam[lane] = gam;
  s.del[lane] = d;
  s.w[lane] = later | (lane < 32 ? t.m1 : 0u) ? 0.f : exp2_hw(lane < 32 ? (t.t0 - gam) + t.t1 : t.t1 - gam) * d;
  if (lane < 32) s.u[lane] = later ? 0.f : exp2_hw(t.t0 - gam) * d;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  return t;
}

// bf16 parts hi + lo of x[e] * w[e]
struct Split {
  bf16x8 hi, lo;
};
__device__ __forceinline__ Split split_scaled(const bf16x8 &x, const float *w) {
  const f32x4 w0 = *reinterpret_cast<const f32x4 *>(w), w1 = *reinterpret_cast<const f32x4 *>(w + 8);
  Split r;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float f = (float)x[e] * (e < 4 ? w0[e & 3] : w1[e & 3]);
    r.hi[e] = (bf16)f;
    r.lo[e] = (bf16)(f - (float)r.hi[e]);
  }
  return r;
}

template <int K, int V>
struct Dims {
  static constexpr int VW = V < 64 ? V : 64, VT = VW / 32, KT = K / 32;
  static constexpr int KP = K + 16, VP = VW + 16;  // LDS row pitches
  typedef f32x16 State[VT][KT];                    // rows k, lane v
};

template <int K, int V>
__device__ __forceinline__ void state_io(typename Dims<K, V>::State &S, float *p, bool store, int lane) {
  using D = Dims<K, V>;
  const int h = lane >> 5, c = lane & 31;
#pragma unroll
  for (int vt = 0; vt < D::VT; ++vt)
#pragma unroll
    for (int kt = 0; kt < D::KT; ++kt)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float *e = p + (32 * kt + 8 * (i >> 2) + 4 * h + (i & 3)) * V + 32 * vt + c;
        if (store)
          *e = S[vt][kt][i];
        else
          S[vt][kt][i] = *e;
      }
}

// OUT: y, from the segment's start state (and the sequence's last state);
// else a segment's last state from zero and its decay, kept for carry_kernel.
template <int K, int V, int NW, bool OUT>
__global__ __launch_bounds__(64 * NW, 1) void mma_kernel(ScanArgs a, Layout w, int blocks_per_group) {
  using D = Dims<K, V>;
  constexpr int VW = D::VW, VT = D::VT, KT = D::KT, KP = D::KP, VP = D::VP, THREADS = 64 * NW;
  __shared__ __align__(16) bf16 Kl[2][64 * KP], Ql[OUT ? 2 : 1][OUT ? 64 * KP : 8], Vl[NW][64 * VP];
  __shared__ __align__(16) Gates G[NW];
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_of(tid), h2 = lane >> 5, r32 = lane & 31;
  const int64_t item = xcd_remap(blockIdx.x, gridDim.x);
  const int blk = (int)(item % blocks_per_group), hq = (int)(item / blocks_per_group % a.Hq);
  const int64_t slot = item / blocks_per_group / a.Hq;
  const SlotLoc loc = locate(a, slot);
  if (!loc.used || (!OUT && loc.last && !w.need_last)) return;
  const int slice = blk * NW + wave;  // of the group's columns
  const int h = hq * (a.Hv / a.Hq) + slice * VW / V, v0 = slice * VW % V;
  const int64_t kv = (int64_t)K * V;
  const float A2 = a.A[h] * kLog2e, bias = a.dt_bias ? a.dt_bias[h] : 0.f, skip = a.D ? a.D[h] : 0.f;
  const bf16 *cp = static_cast<const bf16 *>(a.c) + hq * K, *bp = static_cast<const bf16 *>(a.b) + hq * K;
  const bf16 *xp = static_cast<const bf16 *>(a.x) + (int64_t)h * V + v0;
  const bf16 *dtp = static_cast<const bf16 *>(a.dt) + h;

  typename D::State S;
  const float *src = nullptr;
  if (OUT)
    src = a.one_seg ? (a.h0 ? a.h0 + (loc.n * (int64_t)a.Hv + h) * kv : nullptr) : w.start(a) + (slot * a.Hv + h) * kv;
  if (src) {
    state_io<K, V>(S, const_cast<float *>(src) + v0, false, lane);
  } else {
#pragma unroll
    for (int i = 0; i < VT; ++i)
#pragma unroll
      for (int j = 0; j < KT; ++j) S[i][j] = zero16();
  }

  const int nt = (int)(loc.t1 - loc.t0), nc = (nt + 63) >> 6;
  Rows<K, THREADS> kr, qr;
  Rows<VW, 64> vr;
  float z = 0.f;
  auto fetch = [&](int c) {
    const int64_t t = loc.t0 + 64 * (int64_t)c;
    const int rows = nt - 64 * c < 64 ? nt - 64 * c : 64;
    kr.load(bp + t * a.bs, a.bs, rows, tid);
    if (OUT) qr.load(cp + t * a.cs, a.cs, rows, tid);
    vr.load(xp + t * a.xs, a.xs, rows, lane);
    z = lane < rows ? (float)dtp[(t + lane) * a.Hv] : 0.f;
  };
  auto commit = [&](int buf) {
    kr.store_pi(Kl[buf], KP, tid);
    if (OUT) qr.store_pi(Ql[buf], KP, tid);
    vr.store_pi(Vl[wave], VP, lane);
  };
  if (nc > 0) {
    fetch(0);
    commit(0);
  }
  __syncthreads();
  float total = 0.f;
  for (int c = 0; c < nc; ++c) {
    const int rows = nt - 64 * c < 64 ? nt - 64 * c : 64;
    Gates &g = G[wave];
    const GateTotals gt = gates(g, z + bias, A2, a.softplus, lane < rows, lane);
    total += gt.m0 | gt.m1 ? -INFINITY : gt.t0 + gt.t1;
    if (c + 1 < nc) fetch(c + 1);
    const bf16 *k = Kl[c & 1], *q = Ql[OUT ? c & 1 : 0], *v = Vl[wave];
    bf16x8 vf[VT][4];
    {
      const TrA tv(v, VP, lane);
#pragma unroll
      for (int vt = 0; vt < VT; ++vt)
#pragma unroll
        for (int s = 0; s < 4; ++s) vf[vt][s] = tv.at(s, vt, VP);
    }
    if (OUT) {
      // Y^T = S^T C^T and (B C^T) of the three tiles with j <= i
      f32x16 Y[2][VT], P00 = zero16(), P01 = zero16(), P11 = zero16();
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int vt = 0; vt < VT; ++vt) Y[i][vt] = zero16();
#pragma unroll
      for (int s = 0; s < K / 16; ++s) {
        const bf16x8 q0 = lds16(q + r32 * KP + 16 * s + 8 * h2), q1 = lds16(q + (32 + r32) * KP + 16 * s + 8 * h2);
        const bf16x8 k0 = lds16(k + r32 * KP + 16 * s + 8 * h2), k1 = lds16(k + (32 + r32) * KP + 16 * s + 8 * h2);
#pragma unroll
        for (int vt = 0; vt < VT; ++vt) {
          const bf16x8 sf = slots(S[vt][s >> 1], s & 1);
          Y[0][vt] = mma32(sf, q0, Y[0][vt]);
          Y[1][vt] = mma32(sf, q1, Y[1][vt]);
        }
        P00 = mma32(k0, q0, P00);
        P01 = mma32(k0, q1, P01);  // j in the first half, i in the second
        P11 = mma32(k1, q1, P11);
      }
      const float g0 = g.gam[r32], g1 = g.gam[32 + r32];  // of token i in each half
      const uint32_t f0 = upto(gt.m0, r32), f1 = upto(gt.m1, r32);
      const float e0 = f0 ? 0.f : exp2_hw(g0), e1 = f1 ? 0.f : exp2_hw(g1), e01 = gt.m0 | f1 ? 0.f : exp2_hw(gt.t0 + g1);
      const int l0 = last_bit(f0), l1 = last_bit(f1);  // the first token that token i sees
#pragma unroll
      for (int vt = 0; vt < VT; ++vt)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          Y[0][vt][i] *= e0;
          Y[1][vt][i] *= e01;
        }
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int j0 = 8 * b + 4 * h2;
        const f32x4 ga = *reinterpret_cast<const f32x4 *>(&g.gam[j0]), de = *reinterpret_cast<const f32x4 *>(&g.del[j0]);
        const f32x4 gb = *reinterpret_cast<const f32x4 *>(&g.gam[32 + j0]), df = *reinterpret_cast<const f32x4 *>(&g.del[32 + j0]);
        const f32x4 u = *reinterpret_cast<const f32x4 *>(&g.u[j0]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int j = j0 + i;
          P00[4 * b + i] = j <= r32 && j >= l0 ? P00[4 * b + i] * (exp2_hw(g0 - ga[i]) * de[i]) : 0.f;
          P11[4 * b + i] = j <= r32 && j >= l1 ? P11[4 * b + i] * (exp2_hw(g1 - gb[i]) * df[i]) : 0.f;
          P01[4 * b + i] *= e1 * u[i];
        }
      }
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const bf16x8 p00 = slots(P00, s), p01 = slots(P01, s), p11 = slots(P11, s);
#pragma unroll
        for (int vt = 0; vt < VT; ++vt) {
          Y[0][vt] = mma32(vf[vt][s], p00, Y[0][vt]);
          Y[1][vt] = mma32(vf[vt][s], p01, Y[1][vt]);
          Y[1][vt] = mma32(vf[vt][2 + s], p11, Y[1][vt]);
        }
      }
      const int64_t t = loc.t0 + 64 * (int64_t)c;
      bf16 *yp = static_cast<bf16 *>(a.y) + (t * a.Hv + h) * V + v0;
      const int64_t ys = (int64_t)a.Hv * V;
      const auto yr = raw_buffer(yp, (uint32_t)(((rows - 1) * ys + VW) * 2));
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int row = 32 * i + r32;
        const bf16 *xrow = v + row * VP;
#pragma unroll
        for (int vt = 0; vt < VT; ++vt) {
          uint2 o[4];
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            // columns 32 vt + 8 b + 4 h: in the pi layout 8 h past those of h = 0
            const bf16x4 xv = *reinterpret_cast<const bf16x4 *>(xrow + pi_pos(32 * vt + 8 * b) + 8 * h2);
            bf16x4 r;
#pragma unroll
            for (int e = 0; e < 4; ++e) r[e] = (bf16)(Y[i][vt][4 * b + e] + skip * (float)xv[e]);
            o[b] = __builtin_bit_cast(uint2, r);
          }
#pragma unroll
          for (int b = 0; b < 4; b += 2) {
            // halves: lanes h = 0 get columns 8 b .. 8 b + 7, lanes h = 1 the next 8
            const auto p = __builtin_amdgcn_permlane32_swap(o[b].x, o[b + 1].x, false, false);
            const auto r = __builtin_amdgcn_permlane32_swap(o[b].y, o[b + 1].y, false, false);
            buf_store16(make_uint4(p[0], r[0], p[1], r[1]), yr,
                        row < rows ? (uint32_t)(row * ys * 2 + (32 * vt + 8 * b + 8 * h2) * 2) : 0xFFFFFFF0u);
          }
        }
      }
    }
    // S = 2^{gamma_L} S + B^T (w X)
    const float eL = gt.all();
#pragma unroll
    for (int vt = 0; vt < VT; ++vt)
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
#pragma unroll
        for (int i = 0; i < 16; ++i) S[vt][kt][i] *= eL;
    const TrA tk(k, KP, lane);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      Split x[VT];
#pragma unroll
      for (int vt = 0; vt < VT; ++vt) x[vt] = split_scaled(vf[vt][s], &g.w[16 * s + 4 * h2]);
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) {
        const bf16x8 kf = tk.at(s, kt, KP);
#pragma unroll
        for (int vt = 0; vt < VT; ++vt) {
          S[vt][kt] = mma32(kf, x[vt].hi, S[vt][kt]);
          S[vt][kt] = mma32(kf, x[vt].lo, S[vt][kt]);
        }
      }
    }
    if (c + 1 < nc) commit((c + 1) & 1);
    __syncthreads();
  }
  if (!OUT) {
    state_io<K, V>(S, w.start(a) + (slot * a.Hv + h) * kv + v0, true, lane);
    if (lane == 0 && v0 == 0) w.decay(a)[slot * a.Hv + h] = total / kLog2e;
  } else if (a.ht && loc.last) {
    state_io<K, V>(S, a.ht + (loc.n * (int64_t)a.Hv + h) * kv + v0, true, lane);
  }
}

template <int K, int V, bool OUT>
hipError_t go(const char *name, const ScanArgs &a, const Layout &w, hipStream_t st) {
  const int per = a.Hv / a.Hq * (V / Dims<K, V>::VW);  // column slices of a group
  const int nw = slices_per_block(per);
  const unsigned blocks = (unsigned)(a.slots * a.Hq * (per / nw));
  KernelTimer kt(name, st);
  if (nw == 4)
    mma_kernel<K, V, 4, OUT><<<blocks, 256, 0, st>>>(a, w, per / 4);
  else if (nw == 2)
    mma_kernel<K, V, 2, OUT><<<blocks, 128, 0, st>>>(a, w, per / 2);
  else
    mma_kernel<K, V, 1, OUT><<<blocks, 64, 0, st>>>(a, w, per);
  return hipGetLastError();
}
template <bool OUT>
hipError_t pick(const char *name, const ScanArgs &a, const Layout &w, hipStream_t st) {
  switch (a.K * 1000 + a.V) {
    case 32032: return go<32, 32, OUT>(name, a, w, st);
    case 32064: return go<32, 64, OUT>(name, a, w, st);
    case 32128: return go<32, 128, OUT>(name, a, w, st);
    case 64032: return go<64, 32, OUT>(name, a, w, st);
    case 64064: return go<64, 64, OUT>(name, a, w, st);
    case 64128: return go<64, 128, OUT>(name, a, w, st);
    case 128032: return go<128, 32, OUT>(name, a, w, st);
    case 128064: return go<128, 64, OUT>(name, a, w, st);
    default: return go<128, 128, OUT>(name, a, w, st);
  }
}

}  // namespace

hipError_t launch_mma_local(const ScanArgs &a, const Layout &w, hipStream_t st) {
  return pick<false>("scan_local", a, w, st);
}
hipError_t launch_mma_out(const ScanArgs &a, const Layout &w, hipStream_t st) {
  return pick<true>("scan_out", a, w, st);
}

}  // namespace scan
}  // namespace gdn
