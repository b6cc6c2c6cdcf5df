// The selective scan of bf16 problems on matrix instructions: chunks of 64
// tokens, the state of a head in MFMA accumulators.  With gamma_t the sum of
// log2 decays from the chunk's first token to t and S the state entering it,
//
//   y_i = 2^{gamma_i} S^T c_i + sum_{j <= i} (c_i . b_j) 2^{gamma_i - gamma_j} delta_j x_j + D x_i
//   S'  = 2^{gamma_L} S + sum_j b_j (2^{gamma_L - gamma_j} delta_j x_j)^T
//
// A wave owns 32 columns of one head's state and a segment's chunks in order;
// the waves of a workgroup (eight where the group has as many) are column
// slices of a head group, which share c and b in LDS, the next chunk's rows on
// their way while one is worked on.  (One wave a SIMD with 64 columns: 171 us
// for the out pass at 8192 tokens x 64 heads, K 128, V 64, the state in
// accumulation registers that vector instructions reach only by moves; this
// form 68 us, and 75 with the exact state updates below.)  The pass from zero
// takes 42 us there.  Both have one workgroup a compute unit, whose waves go in
// step from barrier to barrier.
//
// Everything is arranged so that accumulators are operands without moving
// (gdn_slice.hpp): S tiles (rows k, lane v) give S^T for c; C B^T is formed
// as (B C^T) with rows j and lane i, which is P^T as the second operand of
// X^T P^T, and y comes out transposed, lane i, four consecutive v a quad:
// 16-byte stores after one exchange between the wave's halves.
//
// Roundings to bf16: P and the state as operands of y (y itself is bf16).
// The state is held to fp32: its update takes b as it is and the weighted x,
// an fp32 number, as the sum of three bf16 parts, which lose nothing.  (Two
// parts lose 2^-18 of it: 2e-6 of a final state, 2e-6 of dA and ddt_bias.)
#include "gdn_internal.h"
#include "gdn_scan_mma.hpp"

namespace gdn {
namespace scan {
namespace {

// What a pass over a segment's chunks does:
//   kLocal   the segment's last state from zero and its decay (for carry_kernel)
//   kOut     y, from the segment's start state, and the sequence's last state
//   kStates  the state entering every chunk, as bf16 and what fp32 has below
//            it, and a_i = p_i c_i . S dy_i (backward)
//   kRLocal  reverse: the gradient of the segment's first state from its own
//            outputs; a.b, a.x hold c and dy: Z = 2^{gamma_L} Z + C^T (2^{gamma} dY)
enum { kLocal, kOut, kStates, kRLocal };

template <int K, int NW, bool QROWS>
struct Lds {
  bf16 k[64 * (K + 8)], q[QROWS ? 64 * (K + 8) : 8], v[NW][64 * 40];
  Gates g[NW];
};

template <int K, int V, int NW, int MODE, typename L>
__device__ __forceinline__ void chunks(const ScanArgs &a, const Layout &w, int blocks_per_group, int64_t item, L &lds) {
  constexpr bool OUT = MODE == kOut, REV = MODE == kRLocal, QROWS = OUT || MODE == kStates;
  using D = Dims<K, V>;
  constexpr int VW = D::VW, KT = D::KT, KP = D::KP, VP = D::VP, THREADS = 64 * NW;
  static_assert(KP == K + 8 && VP == 40, "row pitches of Lds");
  bf16 *const Kl = lds.k, *const Ql = lds.q;
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_of(tid), h2 = lane >> 5, r32 = lane & 31;
  const int blk = (int)(item % blocks_per_group), hq = (int)(item / blocks_per_group % a.Hq);
  const int64_t slot = item / blocks_per_group / a.Hq;
  const SlotLoc loc = locate(a, slot);
  if (!loc.used || (MODE == kLocal && loc.last)) return;
  const int slice = blk * NW + wave;  // of the group's columns
  const int h = hq * (a.Hv / a.Hq) + slice * VW / V, v0 = slice * VW % V;
  const int64_t kv = (int64_t)K * V;
  const float A2 = a.A[h] * kLog2e, bias = a.dt_bias ? a.dt_bias[h] : 0.f, skip = a.D ? a.D[h] : 0.f;
  const bf16 *cp = static_cast<const bf16 *>(a.c) + hq * K, *bp = static_cast<const bf16 *>(a.b) + hq * K;
  const bf16 *xp = static_cast<const bf16 *>(a.x) + (int64_t)h * V + v0;
  const bf16 *dtp = static_cast<const bf16 *>(a.dt) + h;

  typename D::State S;
  const float *src = nullptr;
  if (OUT || MODE == kStates)
    src = a.one_seg ? (a.h0 ? a.h0 + (loc.n * (int64_t)a.Hv + h) * kv : nullptr) : w.start(a) + (slot * a.Hv + h) * kv;
  if (src) {
    state_io<K, V>(S, const_cast<float *>(src) + v0, false, lane);
    if (MODE == kStates) {
#pragma unroll
      for (int j = 0; j < KT; ++j)
#pragma unroll
        for (int i = 0; i < 16; ++i) S[j][i] = quiet(S[j][i]) * Turn(loc.index * (a.seg / 64)).begins();
    }
  } else {
#pragma unroll
    for (int j = 0; j < KT; ++j) S[j] = zero16();
  }

  const int nt = (int)(loc.t1 - loc.t0), nc = (nt + 63) >> 6;
  // one chunk's rows on their way to LDS.  (An object of the loop's body: one
  // outside it, loaded under a condition, would hold its registers throughout.)
  struct In {
    Rows<K, THREADS> k, q;
    Rows<VW, 64> v;
    bf16 dt;  // of this lane's token
  };
  float z = 0.f;
  auto fetch = [&](In &r, int step, int tid) {
    const int lane = tid & 63, c = REV ? nc - 1 - step : step;
    const int64_t t = loc.t0 + 64 * (int64_t)c;
    const int rows = nt - 64 * c < 64 ? nt - 64 * c : 64;
    r.k.load(bp + t * a.bs, a.bs, rows, tid);
    if (QROWS) r.q.load(cp + t * a.cs, a.cs, rows, tid);
    r.v.load(xp + t * a.xs, a.xs, rows, lane);
    r.dt = load_dt(dtp + t * a.Hv, a.Hv, rows, lane);
  };
  auto commit = [&](const In &r, int tid) {
    const int lane = tid & 63;
    r.k.store_pi(Kl, KP, tid);
    if (QROWS) r.q.store_pi(Ql, KP, tid);
    r.v.store_pi(lds.v[wave], VP, lane);
    z = settle((float)r.dt);
  };
  if (nc > 0) {
    In r;
    fetch(r, 0, tid);
    commit(r, tid);
  }
  __syncthreads();
  float total = 0.f, ends = 1.f;
  for (int step = 0; step < nc; ++step) {
    const int c = REV ? nc - 1 - step : step;
    const int tid = opaque_tid(), lane = tid & 63, h2 = lane >> 5, r32 = lane & 31;
    const int rows = nt - 64 * c < 64 ? nt - 64 * c : 64;
    const Turn turn(loc.index * (a.seg / 64) + c);
    Gates &g = lds.g[wave];
    const GateTotals gt = gates(g, z + bias, A2, a.softplus, lane < rows, lane, REV ? turn.of(lane) : 1.f,
                                OUT ? 1.f : turn.of(lane));
    total += gt.m0 | gt.m1 ? -INFINITY : gt.t0 + gt.t1;
    In in;
    fetch(in, step + 1 < nc ? step + 1 : step, tid);
    const bf16 *k = Kl, *q = Ql, *v = lds.v[wave];
    if (MODE == kStates) {
      const int64_t at = ((w.chunk(a, loc, c) * a.Hv + h) * (V / 32) + v0 / 32) * (K * 32) + lane * 8;
      bf16x4 dyv[2][4];  // dy of this lane's tokens, columns 8 b + 4 h ..
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int tok = 32 * i + r32 < rows ? 32 * i + r32 : rows - 1;
        const bf16 *p = static_cast<const bf16 *>(a.dy) + ((loc.t0 + 64 * (int64_t)c + tok) * a.Hv + h) * V + v0 + 4 * h2;
#pragma unroll
        for (int b = 0; b < 4; ++b) dyv[i][b] = *reinterpret_cast<const bf16x4 *>(p + 8 * b);
      }
      f32x16 U[2] = {zero16(), zero16()};  // U^T = S^T C^T
#pragma unroll
      for (int s = 0; s < K / 16; ++s) {
        const SplitHalves x = split_halves(S[s >> 1], s & 1);
        *reinterpret_cast<uint4 *>(w.s_hi(a) + at + s * 512) = turn.right(x.hi);
        *reinterpret_cast<uint4 *>(w.s_low(a) + at + s * 512) = x.low;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const bf16x8 qf = lds16(q + (32 * i + r32) * KP + 16 * s + 8 * h2);
          U[i] = mma32(x.lo, qf, U[i]);
          U[i] = mma32(x.mid, qf, U[i]);
          U[i] = mma32(x.hi, qf, U[i]);
        }
        if (s & 1) __builtin_amdgcn_sched_barrier(0);
      }
      const int64_t t0 = loc.t0 + 64 * (int64_t)c;
      float *ai = w.ai_part(a) + ((int64_t)(v0 / 32) * a.Hv + h) * a.s.tokens + t0;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float v = acc_dot(U[i], dyv[i]) * (g.p[32 * i + r32] * turn.begins());
        if (h2 == 0 && 32 * i + r32 < rows) ai[32 * i + r32] = v;
      }
    }
    bf16x8 vf[4];
    const TrA tv(v, VP, lane);
#pragma unroll
    for (int s = 0; s < 4; ++s) vf[s] = tv.at(s, 0, VP);
    if (OUT) {
      bf16 *yp = static_cast<bf16 *>(a.y) + ((loc.t0 + 64 * (int64_t)c) * a.Hv + h) * V + v0;
      const int64_t ys = (int64_t)a.Hv * V;
      const auto yr = raw_buffer(yp, (uint32_t)(((rows - 1) * ys + VW) * 2));
      // 32 tokens i at a time: Y^T = S^T C^T and (B C^T) of the tiles with j <= i
#pragma unroll
      for (int it = 0; it < 2; ++it) {
        f32x16 Y = zero16(), Pd = zero16(), Po = zero16();  // diagonal tile; j in the first half, i in the second
        const bf16 *qi = q + (32 * it + r32) * KP + 8 * h2, *kd = k + (32 * it + r32) * KP + 8 * h2,
                   *ko = k + r32 * KP + 8 * h2;
#pragma unroll
        for (int s = 0; s < K / 16; ++s) {
          const bf16x8 qf = lds16(qi + 16 * s);
          Y = mma32(slots(S[s >> 1], s & 1), qf, Y);
          Pd = mma32(lds16(kd + 16 * s), qf, Pd);
          if (it) Po = mma32(lds16(ko + 16 * s), qf, Po);
          if ((s & 3) == 3) __builtin_amdgcn_sched_barrier(0);
        }
        const float gi = g.gam[32 * it + r32];  // of token i, from its half's start
        const uint32_t f = upto(it ? gt.m1 : gt.m0, r32);
        const float ei = it ? g.e[r32] : 0.f, e0 = g.p[32 * it + r32];
        const int first = last_bit(f);  // the first token of the half that token i sees
#pragma unroll
        for (int i = 0; i < 16; ++i) Y[i] *= e0;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const int j0 = 8 * b + 4 * h2;
          const f32x4 gj = *reinterpret_cast<const f32x4 *>(&g.gam[32 * it + j0]);
          const f32x4 dj = *reinterpret_cast<const f32x4 *>(&g.del[32 * it + j0]);
          const f32x4 uj = *reinterpret_cast<const f32x4 *>(&g.u[j0]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int j = j0 + i;
            Pd[4 * b + i] *= exp2_if(j <= r32 && j >= first, gi - gj[i]) * dj[i];
            if (it) Po[4 * b + i] *= ei * uj[i];
          }
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if (it) Y = mma32(vf[s], slots(Po, s), Y);
          Y = mma32(vf[2 * it + s], slots(Pd, s), Y);
        }
        const int row = 32 * it + r32;
        const bf16 *xrow = v + row * VP;
        uint2 o[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          // columns 8 b + 4 h: in the pi layout 8 h past those of h = 0
          const bf16x4 xv = *reinterpret_cast<const bf16x4 *>(xrow + pi_pos(8 * b) + 8 * h2);
          bf16x4 r;
#pragma unroll
          for (int e = 0; e < 4; ++e) r[e] = (bf16)(Y[4 * b + e] + skip * (float)xv[e]);
          o[b] = __builtin_bit_cast(uint2, r);
        }
#pragma unroll
        for (int b = 0; b < 4; b += 2) {
          // halves: lanes h = 0 get columns 8 b .. 8 b + 7, lanes h = 1 the next 8
          const auto p = __builtin_amdgcn_permlane32_swap(o[b].x, o[b + 1].x, false, false);
          const auto r = __builtin_amdgcn_permlane32_swap(o[b].y, o[b + 1].y, false, false);
          buf_store16(make_uint4(p[0], r[0], p[1], r[1]), yr,
                      row < rows ? (uint32_t)(row * ys * 2 + (8 * b + 8 * h2) * 2) : kOutside);
        }
        // (the second half's reads, moved up into the first, would spill in every
        // form; as it is, two-wave workgroups with K = 128 spill 36 registers, and
        // <64, 64> with one wave 4)
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    // S = 2^{gamma_L} S + B^T (w X)
    const float eL = gt.all();
    scale(S, eL);
    const TrA tk(k, KP, lane);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const Split3 x = split_scaled(vf[s], (REV ? g.p : g.w) + 16 * s + 4 * h2);
      if (!OUT && s == 1) scale(S, -1.f);
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) {
        const bf16x8 kf = tk.at(s, kt, KP);
        S[kt] = mma32(kf, x.lo, S[kt]);
        S[kt] = mma32(kf, x.mid, S[kt]);
        S[kt] = mma32(kf, x.hi, S[kt]);
      }
    }
    ends = turn.ends();
    __syncthreads();  // every wave is done with b and c
    commit(in, tid);
    __syncthreads();
  }
  if (MODE == kLocal || REV) {
    if (REV && lane == 0 && v0 == 0) w.decay(a)[slot * a.Hv + h] = total / kLog2e;
    float *dst = (REV ? w.zend(a) : w.start(a)) + (slot * a.Hv + h) * kv + v0;
    scale(S, ends);
    state_io<K, V>(S, dst, true, lane);
    // (in the backward the reverse pass has the decays: one writer)
    if (MODE == kLocal && w.chunks == 0 && lane == 0 && v0 == 0) w.decay(a)[slot * a.Hv + h] = total / kLog2e;
  } else if (OUT && a.ht && loc.last) {
    state_io<K, V>(S, a.ht + (loc.n * (int64_t)a.Hv + h) * kv + v0, true, lane);
  }
}

template <int K, int V, int NW, int MODE>
__global__ __launch_bounds__(64 * NW, 2) void mma_kernel(ScanArgs a, Layout w, int blocks_per_group) {
  __shared__ __align__(16) Lds<K, NW, MODE == kOut || MODE == kStates> lds;
  chunks<K, V, NW, MODE>(a, w, blocks_per_group, xcd_remap(blockIdx.x, gridDim.x), lds);
}

// The backward's two passes from zero, which need nothing of each other, in
// one launch: the first half of the workgroups has kLocal, the other kRLocal
// (`r`: the arguments with c and dy in b's and x's place).
template <int K, int V, int NW>
__global__ __launch_bounds__(64 * NW, 2) void mma_locals_kernel(ScanArgs a, ScanArgs r, Layout w, int blocks_per_group) {
  __shared__ __align__(16) Lds<K, NW, false> lds;
  const int64_t half = gridDim.x / 2, b = blockIdx.x;
  if (b < half)
    chunks<K, V, NW, kLocal>(a, w, blocks_per_group, xcd_remap(b, half), lds);
  else
    chunks<K, V, NW, kRLocal>(r, w, blocks_per_group, xcd_remap(b - half, half), lds);
}

template <int K, int V, int MODE, int NW>
void launch(const ScanArgs &a, const Layout &w, unsigned blocks, int per, hipStream_t st) {
  if constexpr (MODE == kRLocal) {  // both passes from zero
    ScanArgs r = a;
    r.b = a.c;
    r.bs = a.cs;
    r.x = a.dy;
    r.xs = (int64_t)a.Hv * a.V;
    mma_locals_kernel<K, V, NW><<<2 * blocks, 64 * NW, 0, st>>>(a, r, w, per / NW);
  } else {
    mma_kernel<K, V, NW, MODE><<<blocks, 64 * NW, 0, st>>>(a, w, per / NW);
  }
}

template <int K, int V, int MODE>
hipError_t go(const char *name, const ScanArgs &a, const Layout &w, hipStream_t st) {
  const int per = a.Hv / a.Hq * (V / Dims<K, V>::VW);  // column slices of a group
  const int nw = slices_per_block(per);
  const unsigned blocks = (unsigned)(a.slots * a.Hq * (per / nw));
  KernelTimer kt(name, st);
  if (nw == 8)
    launch<K, V, MODE, 8>(a, w, blocks, per, st);
  else if (nw == 4)
    launch<K, V, MODE, 4>(a, w, blocks, per, st);
  else if (nw == 2)
    launch<K, V, MODE, 2>(a, w, blocks, per, st);
  else
    launch<K, V, MODE, 1>(a, w, blocks, per, st);
  return hipGetLastError();
}
template <int MODE>
hipError_t pick(const char *name, const ScanArgs &a, const Layout &w, hipStream_t st) {
  switch (a.K * 1000 + a.V) {
    case 32032: return go<32, 32, MODE>(name, a, w, st);
    case 32064: return go<32, 64, MODE>(name, a, w, st);
    case 32128: return go<32, 128, MODE>(name, a, w, st);
    case 64032: return go<64, 32, MODE>(name, a, w, st);
    case 64064: return go<64, 64, MODE>(name, a, w, st);
    case 64128: return go<64, 128, MODE>(name, a, w, st);
    case 128032: return go<128, 32, MODE>(name, a, w, st);
    case 128064: return go<128, 64, MODE>(name, a, w, st);
    default: return go<128, 128, MODE>(name, a, w, st);
  }
}

}  // namespace

hipError_t launch_mma_local(const ScanArgs &a, const Layout &w, hipStream_t st) {
  return pick<kLocal>("scan_local", a, w, st);
}
hipError_t launch_mma_out(const ScanArgs &a, const Layout &w, hipStream_t st) {
  return pick<kOut>("scan_out", a, w, st);
}
hipError_t launch_mma_states(const ScanArgs &a, const Layout &w, hipStream_t st) {
  return pick<kStates>("scan_states", a, w, st);
}
hipError_t launch_mma_locals(const ScanArgs &a, const Layout &w, hipStream_t st) {
  return pick<kRLocal>("scan_locals", a, w, st);
}

}  // namespace scan
}  // namespace gdn
