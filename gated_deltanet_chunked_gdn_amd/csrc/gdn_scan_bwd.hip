// Backward of the selective scan for bf16 problems, on matrix instructions.
//
// With S the state entering a chunk of 64 tokens, Z the gradient of the state
// leaving it, gamma the log2 decays summed from the chunk's first token,
// E_ij = 2^{gamma_i - gamma_j}, G_ij = c_i . b_j, M_ij = dy_i . x_j, p_i =
// 2^{gamma_i}, w_j = 2^{gamma_L - gamma_j}, and all sums over j <= i:
//
//   dx_j = delta_j (sum_i E_ij G_ij dy_i + w_j Z^T b_j) + D dy_j
//   dc_i = sum_heads (sum_j E_ij delta_j M_ij b_j + p_i S dy_i)
//   db_j = sum_heads delta_j (sum_i E_ij M_ij c_i + w_j Z x_j)
//   Z_in = 2^{gamma_L} Z + sum_i p_i c_i dy_i^T          (the chunk before's Z)
//
// and for the gates, with W_ij = E_ij G_ij M_ij,
//
//   a_i = p_i c_i . S dy_i,   z_j = w_j b_j . Z x_j
//   r_j = sum_{i > j} W_ij,   m_j = W_jj
//   dg_t = 2^{gamma_L} <S, Z> + sum_{i >= t} a_i + sum_{j < t} delta_j z_j
//          + sum_{j < t <= i} W_ij delta_j
//   d delta_t = r_t + z_t + m_t + A dg_t
//
// The pass that forms the states (kStates, gdn_scan_mma.hip) also has a_i.  Two
// kernels share the rest.  grad_kernel walks a segment's chunks from its end with
// Z in accumulators (32 columns of a head a wave, as the forward): dx, the gates'
// sums, and Z of every chunk, rounded to bf16, for the other.  pair_kernel has dc
// and db: one chunk of one head group a workgroup, the heads in turn, so that
// their sums stay in registers.
//
// The gates' sums reach dA and ddt_bias, fp32 sums over all tokens, so what
// enters them is held to fp32: the recurrences of S and Z, S and Z as
// operands in three bf16 parts, G and M from the inputs as they are, <S, Z>
// afresh in every chunk from both in fp32, and the pairs' sum of dg_t by halves
// and quarters of the chunk, so that every pair enters only where it counts:
// pairs from both halves by i (t in the second) or by j (t in the first), pairs
// from both quarters of a half likewise, pairs inside a quarter by the sum over
// their rectangle j < t <= i.  (As sums of all pairs to t less those behind t,
// the pairs inside a quarter put dA up to 2e-5 off where strong decays lie among
// mild ones.  S and Z in two bf16 parts would leave dA of a short sequence with
// states 3e-5 off; <S, Z> carried along over two chunks, ddt_bias 3e-5.)
// dx, dc and db are bf16 themselves and take their operands rounded.
//
// 2 x 4096 tokens x 64 heads, K 128, V 64: passes from zero 78 us, carries 24,
// states 119, grad_kernel 194, pair_kernel 130, gates 24 (of which the exactness
// of the gates' sums takes 7 in the states and 20 in grad_kernel).  S and Z of
// every chunk, 0.8 GB written and read again, are what the middle three move
// beside the tensors, at 3.0 to 3.5 TB/s.
#include "gdn_internal.h"
#include "gdn_scan_mma.hpp"

namespace gdn {
namespace scan {
namespace {

// Sums over the 16 lanes of a quarter of 16 registers each: lane l ends with
// the sum of register l & 15.
__device__ __forceinline__ float fold16(float (&r)[16], int lane) {
#pragma unroll
  for (int n = 0; n < 8; ++n) {
    const bool b = lane & 1;
    r[n] = (b ? r[2 * n + 1] : r[2 * n]) + dpp_mov<0xB1>(b ? r[2 * n] : r[2 * n + 1]);
  }
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    const bool b = lane & 2;
    r[n] = (b ? r[2 * n + 1] : r[2 * n]) + dpp_mov<0x4E>(b ? r[2 * n] : r[2 * n + 1]);
  }
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    const bool b = lane & 4;
    r[n] = (b ? r[2 * n + 1] : r[2 * n]) + __shfl_xor(b ? r[2 * n] : r[2 * n + 1], 4);
  }
  const bool b = lane & 8;
  return (b ? r[1] : r[0]) + __shfl_xor(b ? r[0] : r[1], 8);
}

// Token of this lane's tile: sum over the 32 columns of acc (rows column,
// lane token) times the token's row of a pi-layout matrix.
__device__ __forceinline__ float row_dot(const f32x16 &acc, const bf16 *row, int h2) {
  bf16x4 x[4];
#pragma unroll
  for (int b = 0; b < 4; ++b) x[b] = *reinterpret_cast<const bf16x4 *>(row + pi_pos(8 * b) + 8 * h2);
  return acc_dot(acc, x);
}

// Writes rows of 32 columns (acc + skip * row of `add`, rows column, lane
// token) as 16-byte pieces.
__device__ __forceinline__ void put_rows(const f32x16 &acc, float skip, const bf16 *add, __amdgpu_buffer_rsrc_t out,
                                         uint32_t off, int h2) {
  uint2 o[4];
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    bf16x4 x = {};
    if (add) x = *reinterpret_cast<const bf16x4 *>(add + pi_pos(8 * b) + 8 * h2);
    bf16x4 r;
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] = (bf16)(acc[4 * b + e] + skip * (float)x[e]);
    o[b] = __builtin_bit_cast(uint2, r);
  }
#pragma unroll
  for (int b = 0; b < 4; b += 2) {
    // halves: lanes h = 0 get columns 8 b .. 8 b + 7, lanes h = 1 the next 8
    const auto p = __builtin_amdgcn_permlane32_swap(o[b].x, o[b + 1].x, false, false);
    const auto r = __builtin_amdgcn_permlane32_swap(o[b].y, o[b + 1].y, false, false);
    buf_store16(make_uint4(p[0], r[0], p[1], r[1]), out, off + (off == kOutside ? 0u : (uint32_t)(16 * b + 16 * h2)));
  }
}

// v[4 b + e]: W_ij delta_j of the row i = 8 b + 4 h2 + e and this lane's column j
// of a diagonal tile.  Where i and j are of one quarter it becomes, for j < i, the
// sum of the column from row i to the quarter's end: the sum of these over the
// quarter's columns is that of the pairs j < t <= i at t = i.
__device__ __forceinline__ void own_rectangles(float (&v)[16], int j, int h2) {
  const bool late = j & 16;
  float s[16];
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    s[4 * b + 3] = v[4 * b + 3];
#pragma unroll
    for (int e = 2; e >= 0; --e) s[4 * b + e] = v[4 * b + e] + s[4 * b + e + 1];
  }
  // the quarter's rows in fours: this lane's first, the other half's, again each
  const float second = late ? s[12] : s[4];
  const float o0 = __shfl_xor(late ? s[8] : s[0], 32), o1 = __shfl_xor(second, 32);
  const float after[2] = {second + o1 + (h2 ? 0.f : o0), h2 ? 0.f : o1};
#pragma unroll
  for (int b = 0; b < 4; ++b)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int k = 4 * b + e;
      const float sum = 8 * b + 4 * h2 + e > j ? s[k] + after[b & 1] : 0.f;
      v[k] = (b >> 1) == late ? sum : v[k];
    }
}

// The next forgetting token of the half above j (32: none)
__device__ __forceinline__ int next_bit(uint32_t m) { return m ? __builtin_ctz(m) : 32; }

template <int K, int V, int NW>
__global__ __launch_bounds__(64 * NW, 2) void grad_kernel(ScanArgs a, Layout w, int blocks_per_group) {
  using D = Dims<K, V>;
  constexpr int VW = D::VW, KT = D::KT, KP = D::KP, VP = D::VP, THREADS = 64 * NW;
  __shared__ __align__(16) bf16 Ql[64 * KP], Kl[64 * KP], Xl[NW][64 * VP], Dl[NW][64 * VP];
  __shared__ __align__(16) FineGates G[NW];
  const int tid0 = threadIdx.x, wave = wave_of(tid0);
  const int64_t item = xcd_remap(blockIdx.x, gridDim.x);
  const int blk = (int)(item % blocks_per_group), hq = (int)(item / blocks_per_group % a.Hq);
  const int64_t slot = item / blocks_per_group / a.Hq;
  const SlotLoc loc = locate(a, slot);
  if (!loc.used) return;
  const int slice = blk * NW + wave;
  const int h = hq * (a.Hv / a.Hq) + slice * VW / V, v0 = slice * VW % V, vs = v0 / 32;
  const int64_t kv = (int64_t)K * V, ys = (int64_t)a.Hv * V;
  const float A2 = a.A[h] * kLog2e, bias = a.dt_bias ? a.dt_bias[h] : 0.f, skip = a.D ? a.D[h] : 0.f;
  const bf16 *cp = static_cast<const bf16 *>(a.c) + hq * K, *bp = static_cast<const bf16 *>(a.b) + hq * K;
  const int64_t col0 = (int64_t)hq * (a.Hv / a.Hq) * V + blk * NW * VW;  // the workgroup's first column
  const bf16 *xp = static_cast<const bf16 *>(a.x) + col0, *dp = static_cast<const bf16 *>(a.dy) + col0;
  const bf16 *dtp = static_cast<const bf16 *>(a.dt) + h;
  const int nt = (int)(loc.t1 - loc.t0), nc = (nt + 63) >> 6;

  typename D::State Z;
  const int64_t seq = (loc.n * (int64_t)a.Hv + h) * kv + v0;
  const float *src = a.one_seg ? (a.dht ? a.dht + seq : nullptr) : w.zend(a) + (slot * a.Hv + h) * kv + v0;
  float *const dh0 = a.one_seg && a.dh0 ? a.dh0 + seq : nullptr;  // (else the carries have it)
  if (nc == 0) {
    if (dh0)
      for (int i = tid0 & 63; i < K * VW; i += 64) {
        const int64_t at = (int64_t)(i / VW) * V + i % VW;
        dh0[at] = src ? src[at] : 0.f;
      }
    return;
  }
  bf16x8 sh[K / 16];
  uint4 sl[K / 16];
  // one chunk's rows on their way to LDS.  (An object of the loop's body: one
  // outside it, loaded under a condition, would hold its registers throughout.)
  struct In {
    Rows<K, THREADS> k, q;
    Rows<NW * VW, THREADS> x, dy;  // of all the slices, which lie side by side: whole lines of memory
    bf16 dt;  // of this lane's token
  };
  float z = 0.f;
  const int64_t first_chunk = w.chunk(a, loc, 0);
  auto state_at = [&](int c, int lane) {
    return (((first_chunk + c) * a.Hv + h) * (V / 32) + vs) * (K * 32) + lane * 8;
  };
  auto fetch = [&](In &r, int c, int tid) {
    const int lane = tid & 63;
    const int64_t t = loc.t0 + 64 * (int64_t)c;
    const int rows = nt - 64 * c < 64 ? nt - 64 * c : 64;
    r.k.load(bp + t * a.bs, a.bs, rows, tid);
    r.q.load(cp + t * a.cs, a.cs, rows, tid);
    r.x.load(xp + t * a.xs, a.xs, rows, tid);
    r.dy.load(dp + t * ys, ys, rows, tid);
    r.dt = load_dt(dtp + t * a.Hv, a.Hv, rows, lane);
  };
  auto fetch_state = [&](int c, int lane) {
    const int64_t at = state_at(c, lane);
#pragma unroll
    for (int s = 0; s < K / 16; ++s) {
      sh[s] = *reinterpret_cast<const bf16x8 *>(w.s_hi(a) + at + s * 512);
      sl[s] = *reinterpret_cast<const uint4 *>(w.s_low(a) + at + s * 512);
    }
  };
  auto commit = [&](const In &r, int tid) {
    const int lane = tid & 63;
    r.k.store_pi(Kl, KP, tid);
    r.q.store_pi(Ql, KP, tid);
    r.x.store_slices_pi(Xl[0], VP, tid);
    r.dy.store_slices_pi(Dl[0], VP, tid);
    z = settle((float)r.dt);
  };
  {
    In r;
    fetch(r, nc - 1, tid0);
    commit(r, tid0);
  }
  fetch_state(nc - 1, tid0 & 63);
  if (src) {
    state_io<K, V>(Z, const_cast<float *>(src), false, tid0 & 63);
    scale(Z, Turn(loc.index * (a.seg / 64) + nc - 1).begins());
  } else {
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) Z[kt] = zero16();
  }
  __syncthreads();
  for (int c = nc - 1; c >= 0; --c) {
    const int tid = opaque_tid(), lane = tid & 63, h2 = lane >> 5, r32 = lane & 31;
    const int rows = nt - 64 * c < 64 ? nt - 64 * c : 64;
    const int64_t t0 = loc.t0 + 64 * (int64_t)c;
    const Turn turn(loc.index * (a.seg / 64) + c);
    FineGates &g = G[wave];
    const GateTotals gt = gates(g, z + bias, A2, a.softplus, lane < rows, lane, turn.of(lane));
    const bf16 *q = Ql, *k = Kl, *x = Xl[wave], *dy = Dl[wave];
    const int64_t sums = ((int64_t)vs * a.Hv + h) * a.s.tokens + t0;  // of a_part, r_part, m_part
    const float eL = gt.all();
    // Y^T = Z^T B^T (rows v, lane token), <S, Z>, and Z out
    f32x16 Y[2] = {zero16(), zero16()};
    float xd = 0.f;
    {
      const int64_t at = state_at(c, lane);
      const bf16 *k0 = k + r32 * KP + 8 * h2;
#pragma unroll
      for (int s = 0; s < K / 16; ++s) {
        const Split3 zf = split(Z[s >> 1], s & 1);
        *reinterpret_cast<uint4 *>(w.z(a) + at + s * 512) = turn.right(zf.hi);
        xd = dot_halves(sh[s], sl[s], Z[s >> 1], s & 1, xd);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const bf16x8 kf = lds16(k0 + 32 * i * KP + 16 * s);
          Y[i] = mma32(zf.lo, kf, Y[i]);
          Y[i] = mma32(zf.mid, kf, Y[i]);
          Y[i] = mma32(zf.hi, kf, Y[i]);
        }
        if (s & 1) __builtin_amdgcn_sched_barrier(0);
      }
    }
    const float xo = wave_sum(xd) * (eL * turn.begins());
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int tok = 32 * i + r32;
      const float v = row_dot(Y[i], x + tok * VP, h2) * (g.w1[tok] * turn.begins());
      if (h2 == 0 && tok < rows) w.ri_part(a)[sums + tok] = v;
    }
    __builtin_amdgcn_sched_barrier(0);
    bf16x8 df[4];  // dy^T: lane v, tokens
    {
      const TrA td(dy, VP, lane);
#pragma unroll
      for (int s = 0; s < 4; ++s) df[s] = td.at(s, 0, VP);
    }
    float dD = 0.f;
    const auto out = raw_buffer(static_cast<bf16 *>(a.dx) + (t0 * a.Hv + h) * V + v0, (uint32_t)(((rows - 1) * ys + VW) * 2));
#pragma unroll
    for (int jt = 0; jt < 2; ++jt) {
      const int tj = 32 * jt + r32;  // token j of this lane
      const float gj = g.gam[tj], lj = g.rest[tj], dj = g.del[tj];
      const int lim = next_bit(above(jt ? gt.m1 : gt.m0, r32));  // the first token of the half that no longer sees j
      f32x16 T = Y[jt];
      const float wj = g.w1[tj] * turn.begins();
#pragma unroll
      for (int i = 0; i < 16; ++i) T[i] *= wj;
      float ms = 0.f;
#pragma unroll
      for (int it = jt; it < 2; ++it) {
        float rs[2] = {0.f, 0.f}, ar[16];  // (rs: of i in the tile's first and second 16 rows)
        f32x16 P = zero16(), M = zero16();
        const bf16 *qi = q + (32 * it + r32) * KP + 8 * h2, *kj = k + tj * KP + 8 * h2;
#pragma unroll
        for (int s = 0; s < K / 16; ++s) {
          P = mma32(lds16(qi + 16 * s), lds16(kj + 16 * s), P);
          if ((s & 3) == 3) __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int s = 0; s < 2; ++s)
          M = mma32(lds16(dy + (32 * it + r32) * VP + 8 * h2 + 16 * s), lds16(x + tj * VP + 8 * h2 + 16 * s), M);
        const float uj = it == jt ? 0.f : g.u1[r32];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const int i0 = 8 * b + 4 * h2;
          // rows i: log2 decays (diagonal tile) or decays from the second half's start
          const f32x4 gi = *reinterpret_cast<const f32x4 *>(it == jt ? &g.gam[32 * it + i0] : &g.e[i0]);
          const f32x4 li = *reinterpret_cast<const f32x4 *>(&g.rest[32 * it + i0]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int i = i0 + e;
            float E;
            if (it == jt)
              E = exp2_if(i >= r32 && i < lim, (gi[e] - gj) + (li[e] - lj));
            else
              E = gi[e] * uj;
            const float p = P[4 * b + e] * E, wm = p * M[4 * b + e];
            P[4 * b + e] = p;
            const bool diag = it == jt && i == r32;
            if (it == jt) {
              ms += diag ? wm : 0.f;
              dD += diag ? M[4 * b + e] : 0.f;
            }
            const float wx = diag ? 0.f : wm;
            rs[b >> 1] += wx;
            ar[4 * b + e] = wx * dj;
          }
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) T = mma32(df[2 * it + s], slots(P, s), T);
        if (it == jt) own_rectangles(ar, r32, h2);
        rs[0] += __shfl_xor(rs[0], 32);
        rs[1] += __shfl_xor(rs[1], 32);
        const float lo = fold16(ar, lane), hi = __shfl_xor(lo, 16);  // j in the tile's first, second 16 columns (lanes of the first)
        const int i = 32 * it + 8 * ((lane & 15) >> 2) + 4 * h2 + (lane & 3);
        const bool put_r = h2 == 0 && tj < rows, put_a = !(lane & 16) && i < rows;
        if (it != jt) {
          if (put_r) w.half_part(a)[sums + tj] = rs[0] + rs[1];
          if (put_a) w.half_part(a)[sums + i] = lo + hi;
        } else {
          if (put_r) w.r_part(a)[sums + tj] = r32 & 16 ? rs[1] : rs[0];
          if (put_r && !(r32 & 16)) w.quarter_part(a)[sums + tj] = rs[1];
          if (put_a) w.a_part(a)[sums + i] = i & 16 ? hi : lo;
          if (put_a && (i & 16)) w.quarter_part(a)[sums + i] = lo;
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      ms += __shfl_xor(ms, 32);
      if (h2 == 0 && tj < rows) w.m_part(a)[sums + tj] = ms;
#pragma unroll
      for (int i = 0; i < 16; ++i) T[i] *= dj;
      put_rows(T, skip, dy + tj * VP, out, tj < rows ? (uint32_t)(tj * ys * 2) : kOutside, h2);
      __builtin_amdgcn_sched_barrier(0);
    }
    dD = wave_sum(dD);
    if (lane == 0) {
      const int64_t i = ((int64_t)vs * w.chunks + first_chunk + c) * a.Hv + h;
      w.x_part(a)[i] = xo;
      w.dd_part(a)[i] = dD;
    }
    In in;
    fetch(in, c > 0 ? c - 1 : 0, tid);
    __builtin_amdgcn_sched_barrier(0);
    // Z = 2^{gamma_L} Z + C^T (p dY)
    scale(Z, eL);
    const TrA tq(q, KP, lane);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const Split3 y = split_scaled(df[s], &g.p[16 * s + 4 * h2]);
      if (s == 1) scale(Z, -1.f);
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) {
        const bf16x8 qf = tq.at(s, kt, KP);
        Z[kt] = mma32(qf, y.lo, Z[kt]);
        Z[kt] = mma32(qf, y.mid, Z[kt]);
        Z[kt] = mma32(qf, y.hi, Z[kt]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    // (before the update, the state's registers would not fit beside it)
    fetch_state(c > 0 ? c - 1 : 0, lane);
    if (c > 0) {
      __syncthreads();  // every wave is done with c and b
      commit(in, tid);
      __syncthreads();
    }
  }
  scale(Z, Turn(loc.index * (a.seg / 64)).ends());
  if (dh0) state_io<K, V>(Z, dh0, true, opaque_tid() & 63);
}

// dc and db of one chunk and head group.  Waves are (k tile, dc or db), units
// are 64 (or 32) columns of a head, one after the other; six of the waves also
// gather sum_heads E delta M, a tile each for every second unit, which meets
// the tokens of the chunk at the end.
template <int K, int V>
struct Pair {
  static constexpr int KT = K / 32, WAVES = 8, THREADS = 512;
  static constexpr int UC = V < 64 ? V : 64;  // columns of a unit
  static constexpr int KP = K + 16, UP = UC + 16, NP = 64 + 16;
};

// One unit is worked on in one LDS buffer, the next is written into the other
// (its gates by a wave that has no tile of N), the two after it are on their
// way in registers: one barrier a unit.  With one unit ahead and one buffer
// every unit waited for its own loads and gates (180 us at 2 x 4096 tokens x
// 64 heads, 2.2 TB/s).
template <int K, int V>
__global__ __launch_bounds__(512, 2) void pair_kernel(ScanArgs a, Layout w) {
  using C = Pair<K, V>;
  constexpr int KT = C::KT, UC = C::UC, KP = C::KP, UP = C::UP, NP = C::NP, THREADS = C::THREADS;
  struct Buf {
    bf16 s[UC * KP], z[UC * KP], x[64 * UP], dy[64 * UP];
  };
  struct Tiles {  // after the units
    bf16 n[2][64 * NP];
    float part[3][16][64];
  };
  __shared__ __align__(16) bf16 Ql[64 * KP], Kl[64 * KP];
  __shared__ __align__(16) char room[2 * sizeof(Buf) > sizeof(Tiles) ? 2 * sizeof(Buf) : sizeof(Tiles)];
  __shared__ __align__(16) Gates G[2];
  __shared__ uint32_t Gm[2][2];
  Buf *const B = reinterpret_cast<Buf *>(room);
  Tiles &Tl = *reinterpret_cast<Tiles *>(room);
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_of(tid), h2 = lane >> 5, r32 = lane & 31;
  const int64_t item = xcd_remap(blockIdx.x, gridDim.x);
  const int hq = (int)(item % a.Hq);
  const int64_t slot = item / a.Hq;
  const SlotLoc loc = locate(a, slot);  // (a.seg = 64 here)
  const int rows = (int)(loc.t1 - loc.t0);
  if (!loc.used || rows <= 0) return;
  const int64_t t0 = loc.t0, ys = (int64_t)a.Hv * V;
  const int R = a.Hv / a.Hq, units = R * (V / UC);

  constexpr int PIECES = UC * K / 8;  // of a state
  constexpr int SP = (PIECES + THREADS - 1) / THREADS;
  constexpr int XT = 64 * UC / 8;  // threads that move x and dy pieces
  static_assert(XT <= THREADS, "one piece a thread");
  struct In {
    uint4 s[SP], z[SP], x, dy;
    bf16 dt;
    float A, bias;
  };
  const int xrow = tid / (UC / 8), xcol = tid % (UC / 8);
  auto fetch = [&](In &r, int u) {
    const int h = hq * R + u * UC / V, v0 = u * UC % V;
    const int64_t st = ((slot * a.Hv + h) * (V / 32) + v0 / 32) * (K * 32);
    const auto rs = raw_buffer(w.s_hi(a) + st, PIECES * 16), rz = raw_buffer(w.z(a) + st, PIECES * 16);
#pragma unroll
    for (int i = 0; i < SP; ++i) {
      r.s[i] = buf_load16(rs, (tid + i * THREADS) * 16);
      r.z[i] = buf_load16(rz, (tid + i * THREADS) * 16);
    }
    const auto rx = raw_buffer(static_cast<const bf16 *>(a.x) + t0 * a.xs + (int64_t)h * V + v0, (uint32_t)(((rows - 1) * a.xs + UC) * 2));
    const auto ry = raw_buffer(static_cast<const bf16 *>(a.dy) + t0 * ys + (int64_t)h * V + v0, (uint32_t)(((rows - 1) * ys + UC) * 2));
    const bool in = xrow < rows;  // (rows < 64: threads past XT have xrow >= 64)
    r.x = buf_load16(rx, in ? (uint32_t)(xrow * a.xs * 2 + xcol * 16) : kOutside);
    r.dy = buf_load16(ry, in ? (uint32_t)(xrow * ys * 2 + xcol * 16) : kOutside);
    r.dt = load_dt(static_cast<const bf16 *>(a.dt) + t0 * a.Hv + h, a.Hv, rows, lane);
    r.A = a.A[h];
    r.bias = a.dt_bias ? a.dt_bias[h] : 0.f;
  };
  // unit u into its buffer, and its gates
  auto commit = [&](const In &r, int u) {
    Buf &b = B[u & 1];
    if (wave == 7) {
      const GateTotals t = gates(G[u & 1], (float)r.dt + r.bias, r.A * kLog2e, a.softplus, lane < rows, lane);
      if (lane == 0) {
        Gm[u & 1][0] = t.m0;
        Gm[u & 1][1] = t.m1;
      }
    }
#pragma unroll
    for (int i = 0; i < SP; ++i) {
      // piece (column slice, s, lane): column, and its place in the column's row of k
      const int pc = tid + i * THREADS, l = pc & 63, s = pc / 64 % (K / 16), cs = pc / 64 / (K / 16);
      if (PIECES % THREADS == 0 || pc < PIECES) {
        const int at = (32 * cs + (l & 31)) * KP + 16 * s + 8 * (l >> 5);
        *reinterpret_cast<uint4 *>(b.s + at) = r.s[i];
        *reinterpret_cast<uint4 *>(b.z + at) = r.z[i];
      }
    }
    if (tid < XT) {
      put_pi(b.x + xrow * UP, xcol, r.x);
      put_pi(b.dy + xrow * UP, xcol, r.dy);
    }
  };

  const bool has_out = wave < 2 * KT, is_db = wave >= KT;
  const int kt = wave % KT;
  f32x16 acc[2] = {zero16(), zero16()};  // rows k, lane token
  // wave 0..5: tile (it, jt) of N (rows i, lane j), units of one parity
  const int nt = wave % 3, it = nt > 0, jt = nt > 1;
  f32x16 Nacc = zero16();
  // unit u; `in` holds u + 1 and takes u + 3
  auto work = [&](In &in, int u) {
    __syncthreads();  // unit u is in LDS, the other buffer's reads are done
    if (u + 1 < units) commit(in, u + 1);
    fetch(in, u + 3 < units ? u + 3 : units - 1);
    const Buf &b_ = B[u & 1];
    const Gates &g = G[u & 1];
    const bf16 *Sl = b_.s, *Zl = b_.z, *Xl = b_.x, *Dl = b_.dy;
    if (has_out) {
      const TrA ts((is_db ? Zl : Sl), KP, lane);
      const bf16 *y = (is_db ? Xl : Dl) + r32 * UP + 8 * h2;
      f32x16 P[2] = {zero16(), zero16()};
#pragma unroll
      for (int s = 0; s < UC / 16; ++s) {
        const bf16x8 sf = ts.at(s, kt, KP);
#pragma unroll
        for (int i = 0; i < 2; ++i) P[i] = mma32(sf, lds16(y + 32 * i * UP + 16 * s), P[i]);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float f = is_db ? g.w[32 * i + r32] : g.p[32 * i + r32];
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][e] += f * P[i][e];
      }
    }
    if (wave < 6 && (u & 1) == (wave >= 3)) {
      f32x16 M = zero16();
      const bf16 *yi = Dl + (32 * it + r32) * UP + 8 * h2, *xj = Xl + (32 * jt + r32) * UP + 8 * h2;
#pragma unroll
      for (int s = 0; s < UC / 16; ++s) M = mma32(lds16(yi + 16 * s), lds16(xj + 16 * s), M);
      const float gj = g.gam[32 * jt + r32], dj = g.del[32 * jt + r32], uj = g.u[r32];
      const int lim = next_bit(above(Gm[u & 1][jt], r32));
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int i0 = 8 * b + 4 * h2;
        const f32x4 gi = *reinterpret_cast<const f32x4 *>(it == jt ? &g.gam[32 * it + i0] : &g.e[i0]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = i0 + e;
          float E;
          if (it == jt)
            E = exp2_if(i >= r32 && i < lim, gi[e] - gj) * dj;
          else
            E = gi[e] * uj;
          Nacc[4 * b + e] += E * M[4 * b + e];
        }
      }
    }
  };
  {
    In in0, in1;
    fetch(in0, 0);
    fetch(in1, units > 1 ? 1 : 0);
    Rows<K, THREADS> kr, qr;
    kr.load(static_cast<const bf16 *>(a.b) + t0 * a.bs + hq * K, a.bs, rows, tid);
    qr.load(static_cast<const bf16 *>(a.c) + t0 * a.cs + hq * K, a.cs, rows, tid);
    kr.store_pi(Kl, KP, tid);
    qr.store_pi(Ql, KP, tid);
    commit(in0, 0);
    fetch(in0, units > 2 ? 2 : units - 1);
    for (int u = 0; u < units; u += 2) {
      work(in1, u);
      if (u + 1 < units) work(in0, u + 1);
    }
  }
  // N of all heads, rounded to bf16, by rows i and by rows j
  __syncthreads();
  if (wave >= 3 && wave < 6) {
#pragma unroll
    for (int e = 0; e < 16; ++e) Tl.part[nt][e][lane] = Nacc[e];
  }
  for (int i = tid; i < 32 * NP; i += THREADS) {  // the tile with j > i
    Tl.n[0][i] = (bf16)0.f;
    Tl.n[1][32 * NP + i] = (bf16)0.f;
  }
  __syncthreads();
  if (wave < 3) {
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      bf16x4 r;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float v = Nacc[4 * b + e] + Tl.part[nt][4 * b + e][lane];
        r[e] = (bf16)v;
        const int i = 32 * it + 8 * b + 4 * h2 + e, j = 32 * jt + r32;
        // N[0]: rows i, position of j in the pi layout
        Tl.n[0][i * NP + pi_pos(j & ~3) + (j & 3)] = r[e];
      }
      // N[1]: rows j, four consecutive i
      *reinterpret_cast<bf16x4 *>(&Tl.n[1][(32 * jt + r32) * NP + pi_pos(32 * it + 8 * b) + 8 * h2]) = r;
    }
  }
  __syncthreads();
  if (!has_out) return;
  // dc^T += B^T N^T (lane i, over j <= i); db^T += C^T N (lane j, over i >= j)
  const TrA tb(is_db ? Ql : Kl, KP, lane);
  const bf16 *nr = Tl.n[is_db ? 1 : 0] + r32 * NP + 8 * h2;
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const bf16x8 f = tb.at(s, kt, KP);
#pragma unroll
    for (int i = 0; i < 2; ++i) acc[i] = mma32(f, lds16(nr + 32 * i * NP + 16 * s), acc[i]);
  }
  bf16 *dst = static_cast<bf16 *>(is_db ? a.db : a.dc) + (t0 * a.Hq + hq) * K + 32 * kt;
  const int64_t qs = (int64_t)a.Hq * K;
  const auto out = raw_buffer(dst, (uint32_t)(((rows - 1) * qs + 32) * 2));
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int tok = 32 * i + r32;
    put_rows(acc[i], 0.f, nullptr, out, tok < rows ? (uint32_t)(tok * qs * 2) : kOutside, h2);
  }
}

// Tokens of `width` in a row, tok = rows - 1 - lane, and the pairs from two such
// neighbours: for t in the second, the sum of v over its tokens from t on (a_i);
// in the first, over its tokens before t (delta_j r_j).  (The terms are 0 where a
// token between i and j forgets all.)
__device__ __forceinline__ double outer_sum(double v, int tok, int lane, int width) {
  const bool second = tok & width;
  const double prior = __shfl_down(v, 1);
  if (!second) v = lane < 63 && (tok & (width - 1)) ? prior : 0.;
  for (int d = 1; d < width; d <<= 1) {
    const int from = second ? lane - d : lane + d, at = second ? tok + d : tok - d;
    const double more = __shfl(v, from & 63);
    if (from >= 0 && from < 64 && (at ^ tok) < width && at >= 0) v += more;
  }
  return v;
}
// The gates of one chunk and head: dg from the chunk's <S, Z>, its a, z and
// pairs (in 64 bits, since dg cancels against r and m in the sums over all
// tokens), then ddt and the chunk's parts of dA, ddt_bias, dD.  Lanes are tokens, lane
// 0 the last.
__global__ __launch_bounds__(256) void chunk_gates_kernel(ScanArgs a, Layout w) {
  const int lane = threadIdx.x & 63;
  const int64_t unit = (int64_t)blockIdx.x * 4 + wave_of(threadIdx.x);
  const int h = (int)(unit % a.Hv);
  const int64_t slot = unit / a.Hv;
  if (slot >= w.chunks) return;
  const SlotLoc loc = locate(a, slot);  // (a.seg = 64 here)
  float *part = w.head_part(a) + (slot * a.Hv + h) * 3;
  const int rows = (int)(loc.t1 - loc.t0);
  if (!loc.used || rows <= 0) {
    if (lane < 3) part[lane] = 0.f;
    return;
  }
  const int slices = a.V / 32;
  const bool on = lane < rows;
  const int64_t t = loc.t1 - 1 - (on ? lane : 0);
  double av = 0., ai = 0., rv = 0., ri = 0., half = 0., quarter = 0., mv = 0., x = 0., dD = 0.;
  for (int s = 0; s < slices; ++s) {
    const int64_t i = ((int64_t)s * a.Hv + h) * a.s.tokens + t;
    av += w.a_part(a)[i];
    ai += w.ai_part(a)[i];
    half += w.half_part(a)[i];
    quarter += w.quarter_part(a)[i];
    rv += w.r_part(a)[i];
    ri += w.ri_part(a)[i];
    mv += w.m_part(a)[i];
    const int64_t j = ((int64_t)s * w.chunks + slot) * a.Hv + h;
    x += w.x_part(a)[j];
    dD += w.dd_part(a)[j];
  }
  const float A = a.A[h];
  const float z = (float)static_cast<const bf16 *>(a.dt)[t * a.Hv + h] + (a.dt_bias ? a.dt_bias[h] : 0.f);
  const float delta = a.softplus ? softplusf(z) : z;
  const int tok = rows - 1 - lane;
  const bool late32 = tok & 32, late16 = tok & 16;
  const double dg = x + sum_upto(on ? ai : 0., lane) + sum_before(on ? delta * ri : 0., lane) +
                    outer_sum(on ? (late32 ? half : delta * half) : 0., tok, lane, 32) +
                    outer_sum(on ? (late16 ? quarter : delta * quarter) : 0., tok, lane, 16) +
                    (on ? av : 0.);
  double dd = rv + (late16 ? 0. : quarter) + (late32 ? 0. : half) + ri + mv + A * dg;
  if (a.softplus) dd *= 1.f / (1.f + expf(-z));
  if (on) static_cast<bf16 *>(a.ddt)[t * a.Hv + h] = (bf16)(float)dd;
  const float dA = (float)wave_sum64(on ? delta * dg : 0.), dbias = (float)wave_sum64(on ? dd : 0.);
  if (lane == 0) {
    part[0] = dA;
    part[1] = dbias;
    part[2] = (float)dD;
  }
}

// dA, ddt_bias, dD of a head: the chunks' parts in a fixed order.
__global__ __launch_bounds__(256) void chunk_heads_kernel(ScanArgs a, Layout w) {
  __shared__ double red[3][4];
  const int h = blockIdx.x, lane = threadIdx.x & 63;
  double v[3] = {0., 0., 0.};
  for (int64_t s = threadIdx.x; s < w.chunks; s += 256)
    for (int k = 0; k < 3; ++k) v[k] += w.head_part(a)[(s * a.Hv + h) * 3 + k];
  for (int k = 0; k < 3; ++k) {
    const double t = wave_sum64(v[k]);
    if (lane == 0) red[k][threadIdx.x >> 6] = t;
  }
  __syncthreads();
  float *out[3] = {a.dA, a.ddt_bias, a.dD};
  if (threadIdx.x < 3 && out[threadIdx.x]) {
    const double *r = red[threadIdx.x];
    out[threadIdx.x][h] = (float)((r[0] + r[1]) + (r[2] + r[3]));
  }
}

template <int K, int V>
hipError_t go(const ScanArgs &a, const Layout &w, hipStream_t st) {
  const int per = a.Hv / a.Hq * (V / 32);  // column slices of a group
  // (four waves: with eight 173 us against 167 at 2 x 4096 tokens x 64 heads)
  const int nw = slices_per_block(per) < 4 ? slices_per_block(per) : 4;
  const unsigned blocks = (unsigned)(a.slots * a.Hq * (per / nw));
  {
    KernelTimer kt("scan_grad", st);
    if (nw == 4)
      grad_kernel<K, V, 4><<<blocks, 256, 0, st>>>(a, w, per / 4);
    else if (nw == 2)
      grad_kernel<K, V, 2><<<blocks, 128, 0, st>>>(a, w, per / 2);
    else
      grad_kernel<K, V, 1><<<blocks, 64, 0, st>>>(a, w, per);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  ScanArgs c = a;
  c.seg = 64;
  c.slots = w.chunks;
  {
    KernelTimer kt("scan_pair", st);
    pair_kernel<K, V><<<(unsigned)(w.chunks * a.Hq), 512, 0, st>>>(c, w);
  }
  if ((e = hipGetLastError()) != hipSuccess) return e;
  KernelTimer kt("scan_gates", st);
  chunk_gates_kernel<<<(unsigned)((w.chunks * a.Hv + 3) / 4), 256, 0, st>>>(c, w);
  chunk_heads_kernel<<<a.Hv, 256, 0, st>>>(c, w);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mma_grad(const ScanArgs &a, const Layout &w, hipStream_t st) {
  switch (a.K * 1000 + a.V) {
    case 32032: return go<32, 32>(a, w, st);
    case 32064: return go<32, 64>(a, w, st);
    case 32128: return go<32, 128>(a, w, st);
    case 64032: return go<64, 32>(a, w, st);
    case 64064: return go<64, 64>(a, w, st);
    case 64128: return go<64, 128>(a, w, st);
    case 128032: return go<128, 32>(a, w, st);
    case 128064: return go<128, 64>(a, w, st);
    default: return go<128, 128>(a, w, st);
  }
}

}  // namespace scan
}  // namespace gdn
