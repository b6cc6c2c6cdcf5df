// Pieces shared by the selective scan's matrix kernels (forward and local
// passes in gdn_scan_mma.hip, the backward in gdn_scan_bwd.hip).
#pragma once

#include "gdn_scan.hpp"
#include "gdn_slice.hpp"

namespace gdn {
namespace scan {

using slice::f32x16;
using slice::lds16;
using slice::mma32;
using slice::pi_pos;
using slice::put_pi;
using slice::slots;
using slice::TrA;
using slice::zero16;

// A byte offset that lies past every buffer: loads read 0, stores are dropped.
constexpr uint32_t kOutside = 0xFFFFFFF0u;
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
  static constexpr int PIECES = 64 * COLS / 8;
  static constexpr int N = (PIECES + THREADS - 1) / THREADS;
  uint4 r[N];
  __device__ __forceinline__ void load(const bf16 *p, int64_t stride, int rows, int tid) {
    const uint32_t bytes = rows > 0 ? (uint32_t)(((rows - 1) * stride + COLS) * 2) : 0u;
    const auto rsrc = raw_buffer(p, bytes);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int pc = tid + i * THREADS, row = pc / (COLS / 8), col = pc % (COLS / 8);
      // (a row past the end may still lie inside the byte range of the last
      // row's neighbours in a wider tensor: it is sent past the range)
      // (so are pieces past the chunk's, where THREADS are more)
      r[i] = buf_load16(rsrc, row < rows ? (uint32_t)(row * stride * 2 + col * 16) : kOutside);
    }
  }
  // rows of COLS / 32 slices of 32 columns, each slice's to its own 64 rows
  __device__ __forceinline__ void store_slices_pi(bf16 *lds, int pitch, int tid) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int pc = tid + i * THREADS, row = pc / (COLS / 8), col = pc % (COLS / 8);
      put_pi(lds + ((col >> 2) * 64 + row) * pitch, col & 3, r[i]);
    }
  }
  __device__ __forceinline__ void store_pi(bf16 *lds, int pitch, int tid) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int pc = tid + i * THREADS, row = pc / (COLS / 8), col = pc % (COLS / 8);
      if (PIECES % THREADS == 0 || pc < PIECES) put_pi(lds + row * pitch, col, r[i]);
    }
  }
};

// 2^x where `in`, else 0, without a branch (the compiler makes one of a
// select around the exponential: 32 a chunk, each a wait of its own).
__device__ __forceinline__ float exp2_if(bool in, float x) { return exp2_hw(in ? x : -1000.f); }
// x, ready here: a value on its way from memory is waited for where it is
// next to the loads it came with, not in the next round of a loop, where the
// wait would cover every store since.
__device__ __forceinline__ float settle(float x) {
  asm volatile("" : "+v"(x));
  return x;
}

// LDS written by a wave is read by other lanes of it after this.
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}
// dt of lane's token of a chunk (0 past its rows), as it is: converted where
// it is loaded, or loaded under a branch, it would be waited for there, and
// with it every load issued before.
__device__ __forceinline__ bf16 load_dt(const bf16 *dt, int64_t stride, int rows, int lane) {
  const auto r = raw_buffer(dt, (uint32_t)(((rows - 1) * stride + 1) * 2));
  return buf_load_elem<bf16>(r, (uint32_t)(lane * stride * 2));
}

// What a wave keeps of a chunk's steps in LDS, by token: log2 decays summed
// from the token's half (32 tokens), delta, the decay from the token to the
// chunk's last (w1) and times delta (w), that of the first half's tokens to
// the half's last (u1) and times delta (u), from the second half's first token
// to its tokens (e), and from the chunk's first token to the token (p).
//
// The last digits of gamma are the relative error of 2^{gamma_i - gamma_j}, and
// a chunk's log decays can add up to thousands: each is taken as a multiple of
// 2^-12 (gam, whose sums and differences are exact up to 2^12) and the rest
// (rest, below 2^-13 each).  A token whose own decay is below 2^kForget ends
// all that is before it; it counts as an exact 0 and stays out of the sums, so
// that a half's stays below 2^12.  m0, m1 mark such tokens of the halves.
//
// The reverse pass, whose pairs' decays reach fp32 gradients, keeps gam and
// rest apart (FineGates); where only bf16 outputs see them (Gates) gam is the
// sum of both, off by 2^-25 of itself (8192 tokens x 64 heads, both apart: out
// pass 76 us against 73).
constexpr float kForget = -126.f;
struct GatesCore {
  float gam[64], del[64], w1[64], p[64], u1[32], e[32];
};
struct FineGates : GatesCore {
  float rest[64];
};
struct Gates : GatesCore {
  float w[64], u[32];
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

// The bf16 matrix instructions round what lies below their sum's last bit down,
// not to nearest: of random operands -0.02 to -0.06 of 2^-24 of the summands'
// sizes an instruction, whatever their sign.  A state that forgets little gathers
// that for as long as it lives, and <S, Z> over all K V elements: dA came out 1e-6
// low in every head.  So the backward's updates of S and Z turn signs over: a
// chunk's first 16 tokens (where a sum from zero loses most) with one sign, the
// other 48 with the other, and the chunks of a sequence in turn with either first
// (dA 2e-7 off, of either sign, for 5 % of the reverse pass).
struct Turn {
  bool odd;  // chunk, uniform
  __device__ __forceinline__ Turn(int64_t chunk) : odd(__builtin_amdgcn_readfirstlane((int)chunk) & 1) {}
  // An odd chunk begins with the state and ends with its negative, an even one the
  // other way round.
  __device__ __forceinline__ float begins() const { return odd ? 1.f : -1.f; }
  __device__ __forceinline__ float ends() const { return odd ? -1.f : 1.f; }
  // of a token's weight (p or w of its gates); the state turns over behind the first 16
  __device__ __forceinline__ float of(int token) const { return odd == (token < 16) ? 1.f : -1.f; }
  // eight bf16 numbers of the state that the chunk begins with
  __device__ __forceinline__ uint4 right(const bf16x8 &x) const {
    const uint32_t m = odd ? 0u : 0x80008000u;
    const uint4 u = __builtin_bit_cast(uint4, x);
    return make_uint4(u.x ^ m, u.y ^ m, u.z ^ m, u.w ^ m);
  }
};
template <int KT>
__device__ __forceinline__ void scale(f32x16 (&S)[KT], float f) {
#pragma unroll
  for (int kt = 0; kt < KT; ++kt)
#pragma unroll
    for (int i = 0; i < 16; ++i) S[kt][i] *= f;
}

template <typename G>
__device__ __forceinline__ GateTotals gates(G &s, float z, float A2, bool softplus, bool live, int lane, float psign = 1.f,
                                                  float wsign = 1.f) {
  const float d = live ? (softplus ? softplusf(z) : z) : 0.f;
  const float g = d * A2;
  const bool cut = g < kForget;
  const unsigned long long m = __ballot(cut);
  const float gh = cut ? 0.f : __builtin_rintf(g * 4096.f) * (1.f / 4096.f), gl = cut ? 0.f : g - gh;
  const float gam = half_incl_scan(gh), rest = half_incl_scan(gl);
  const float h0 = lane_f(gam, 31), h1 = lane_f(gam, 63), r0 = lane_f(rest, 31), r1 = lane_f(rest, 63);
  GateTotals t{h0 + r0, h1 + r1, (uint32_t)m, (uint32_t)(m >> 32)};
  const int i = lane & 31;
  const uint32_t later = lane < 32 ? above(t.m0, i) : above(t.m1, i);
  constexpr bool fine = __is_same(G, FineGates);
  s.gam[lane] = fine ? gam : gam + rest;
  if constexpr (fine) s.rest[lane] = rest;
  s.del[lane] = d;
  const uint32_t before = upto(lane < 32 ? t.m0 : t.m1, i) | (lane < 32 ? 0u : t.m0);
  s.p[lane] = before ? 0.f : psign * exp2_hw(lane < 32 ? gam + rest : (h0 + gam) + (r0 + rest));
  const float w1 = later | (lane < 32 ? t.m1 : 0u) ? 0.f : exp2_hw(lane < 32 ? ((h0 - gam) + h1) + ((r0 - rest) + r1) : (h1 - gam) + (r1 - rest));
  s.w1[lane] = w1;
  if constexpr (!fine) s.w[lane] = w1 * d * wsign;
  if (lane < 32) {
    const float u1 = later ? 0.f : exp2_hw((h0 - gam) + (r0 - rest));
    s.u1[lane] = u1;
    if constexpr (!fine) s.u[lane] = u1 * d;
  } else {
    s.e[lane - 32] = upto(t.m1, i) ? 0.f : exp2_hw(gam + rest);
  }
  wave_lds_fence();
  return t;
}

// x[e] * w[e], rounded to fp32, as the sum of three bf16 numbers: its upper 8
// bits, the next 8 and the last (each cut off by a mask, so exactly).
struct Split3 {
  bf16x8 hi, mid, lo;
};
__device__ __forceinline__ Split3 split_scaled(const bf16x8 &x, const float *w) {
  const f32x4 w0 = *reinterpret_cast<const f32x4 *>(w), w1 = *reinterpret_cast<const f32x4 *>(w + 8);
  typedef uint32_t u32x4_ __attribute__((ext_vector_type(4)));
  u32x4_ hi, mid;
  Split3 r;
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    uint32_t u[2], m[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float f = (float)x[e + k] * (e < 4 ? w0[(e + k) & 3] : w1[(e + k) & 3]);
      u[k] = __builtin_bit_cast(uint32_t, f);
      const float r1 = f - __builtin_bit_cast(float, u[k] & 0xFFFF0000u);
      m[k] = __builtin_bit_cast(uint32_t, r1);
      r.lo[e + k] = (bf16)(r1 - __builtin_bit_cast(float, m[k] & 0xFFFF0000u));
    }
    hi[e / 2] = __builtin_amdgcn_perm(u[1], u[0], 0x07060302);
    mid[e / 2] = __builtin_amdgcn_perm(m[1], m[0], 0x07060302);
  }
  r.hi = __builtin_bit_cast(bf16x8, hi);
  r.mid = __builtin_bit_cast(bf16x8, mid);
  return r;
}

// Operand slots 8 s .. 8 s + 7 of an accumulator tile as the sum of three bf16
// numbers, each rounded to nearest: exact but for fp32's last bit or so.
__device__ __forceinline__ Split3 split(const f32x16 &x, int s) {
  Split3 r;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    r.hi[e] = (bf16)x[8 * s + e];
    const float r1 = x[8 * s + e] - (float)r.hi[e];
    r.mid[e] = (bf16)r1;
    r.lo[e] = (bf16)(r1 - (float)r.mid[e]);
  }
  return r;
}
// The same, hi rounded by an integer sum (halves away from 0), and the fp32
// numbers' lower 16 bits: these and hi are the numbers again (dot_halves), in
// the room of two bf16 parts.  (A NaN whose upper bits are all ones would
// round to 0: quiet() first.)
struct SplitHalves : Split3 {
  uint4 low;
};
__device__ __forceinline__ SplitHalves split_halves(const f32x16 &x, int s) {
  SplitHalves r;
  uint32_t hi[4], low[4];
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    uint32_t u[2], b[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float f = x[8 * s + e + k];
      b[k] = __builtin_bit_cast(uint32_t, f);
      u[k] = b[k] + 0x8000u;
      const float r1 = f - __builtin_bit_cast(float, u[k] & 0xFFFF0000u);
      r.mid[e + k] = (bf16)r1;
      r.lo[e + k] = (bf16)(r1 - (float)r.mid[e + k]);
    }
    hi[e / 2] = __builtin_amdgcn_perm(u[1], u[0], 0x07060302);
    low[e / 2] = __builtin_amdgcn_perm(b[1], b[0], 0x05040100);
  }
  r.hi = __builtin_bit_cast(bf16x8, make_uint4(hi[0], hi[1], hi[2], hi[3]));
  r.low = make_uint4(low[0], low[1], low[2], low[3]);
  return r;
}
__device__ __forceinline__ float quiet(float x) {
  return x == x ? x : __builtin_bit_cast(float, 0x7FC00000u);
}
// c plus the products of such numbers and slots 8 s .. of a tile, in fp32.
__device__ __forceinline__ float dot_halves(const bf16x8 &hi, const uint4 &low, const f32x16 &z, int s, float c) {
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  const uint4 h4 = __builtin_bit_cast(uint4, hi);
  const uint32_t h[4] = {h4.x, h4.y, h4.z, h4.w}, l[4] = {low.x, low.y, low.z, low.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // (hi is one more where the lower half is 0x8000 or above)
    const uint32_t up = (l[i] >> 15) & 0x00010001u;
    const uint32_t b = __builtin_bit_cast(uint32_t, __builtin_bit_cast(u16x2, h[i]) - __builtin_bit_cast(u16x2, up));
    c += __builtin_bit_cast(float, __builtin_amdgcn_perm(b, l[i], 0x05040100)) * z[8 * s + 2 * i];
    c += __builtin_bit_cast(float, __builtin_amdgcn_perm(b, l[i], 0x07060302)) * z[8 * s + 2 * i + 1];
  }
  return c;
}

// Sum over the 32 columns of an accumulator tile (rows column, lane token)
// times the token's values of columns 8 b + 4 h ..
__device__ __forceinline__ float acc_dot(const f32x16 &acc, const bf16x4 (&x)[4]) {
  float v = 0.f;
#pragma unroll
  for (int b = 0; b < 4; ++b)
#pragma unroll
    for (int e = 0; e < 4; ++e) v += acc[4 * b + e] * (float)x[b][e];
  return v + __shfl_xor(v, 32);
}

template <int K, int V>
struct Dims {
  static constexpr int VW = 32, KT = K / 32;
  // LDS row pitches: 16-byte reads of 16 consecutive rows meet every bank once
  static constexpr int KP = K + 8, VP = VW + 8;
  typedef f32x16 State[KT];                        // rows k, lane v
};

template <int K, int V>
__device__ __forceinline__ void state_io(typename Dims<K, V>::State &S, float *p, bool store, int lane) {
  using D = Dims<K, V>;
  const int h = lane >> 5, c = lane & 31;
#pragma unroll
  for (int kt = 0; kt < D::KT; ++kt)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float *e = p + (32 * kt + 8 * (i >> 2) + 4 * h + (i & 3)) * V + c;
      if (store)
        *e = S[kt][i];
      else
        S[kt][i] = *e;
    }
}

}  // namespace scan
}  // namespace gdn
