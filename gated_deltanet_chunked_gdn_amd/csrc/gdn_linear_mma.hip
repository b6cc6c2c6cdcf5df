// Linear attention with a decay for each head, bf16 (gdn_linear.hpp has the
// passes): chunks of 64 tokens, the state in MFMA accumulators.
//
// A workgroup has a segment of one head and VS = 32 or 64 of the output's
// columns (gdn_linear.hip, plan_mma).  Its twelve waves work side by side on a
// chunk: four on the outputs, 16 tokens i each,
//
//   O^T = l^{i+1} S^T A^T + C^T P^T,   P^T = (B A^T) l^{i-j}, rows j, lanes i
//
// and eight on the state, which lies in their accumulators by tiles of 16 x 16,
//
//   S' = l^64 S + B^T (u C),   u_j = l^{63-j}
//
// so that a chunk costs one barrier: b, c, u C and the state (as bf16,
// transposed) lie in LDS twice, the next chunk's written under the present
// one's products, and the loads run two chunks ahead.  a goes from memory to the
// lanes that multiply it; a pass reads a, b, c once for each VS columns and
// writes its output once, S never.  P^T's accumulators are the next product's
// operand as they are, its tokens in the order 16 t + 4 g + e in which C^T is then
// read (g: the lane's group of 16).  The columns of an output tile are dealt so
// that a lane ends with eight in a row.
//
// Roundings to bf16: P and the state as operands of the outputs, which are bf16
// themselves; o is 1.25 times, dq and dk 1.4 times as far from 64 bits as rounding
// the output alone.  Not so for a way of one chunk, whose P may be few numbers (one
// for a token alone: dq and dk up to 3.2 times): there both are taken as two bf16
// parts, off by 2^-17, the state's second one in the buffer that no second chunk
// needs.  (P in two parts throughout: 1.14 and 1.3 times, the passes 2 to 4 % longer.)
// The state is held in fp32.  Its update takes the weighted c, an fp32 number, as
// two bf16 parts (off by 2^-17), and as three, which lose nothing, where a returned
// or carried state sees the step; one part left dq and dk 1.6 times as far from 64
// bits as rounding the output alone.
//
// What bounds it: the chunks of a sequence follow one another, one workgroup a
// compute unit (LDS), 1.2 us a chunk of 32 columns and 1.6 of 64, between the
// barriers LDS reads, products and the commits of the next chunk, each waited for;
// HBM would take half of that.  One workgroup, because b, c, u c and the state lie
// in LDS twice; a step moves some 280 KB through it at 64 columns.  K = V = 128: 8192
// tokens x 64 heads forward 160 to 164 us (3.3 TB/s of its inputs and outputs once
// each); 16384 packed tokens x 32 heads in 16 sequences 167 us, at their end the
// longest prompts of the last heads alone; backward of 2 x 4096 x 32 heads 187 us, its
// three passes side by side in one launch, 384 workgroups, one and a half rounds.
// Waves of their own for P (sixteen, a read twice) 210 us against 161; a through LDS
// the same within noise.
#include <type_traits>

#include "gdn_internal.h"
#include "gdn_linear.hpp"

namespace gdn {
namespace attn {
namespace {

// Row pitches in LDS: 32 bytes over a multiple of 64.  16-byte reads of 16 rows
// then take 4 clocks and transpose reads of 32 bytes of 16 rows 1.4 (with 16
// bytes over: 8 and 2.1).
constexpr int pitch(int columns) { return columns + 16; }
typedef Mma<bf16> M;
typedef __attribute__((address_space(3))) bf16x4 lds_bf16x4;
__device__ __forceinline__ bf16x4 tr4(const bf16 *p) { return __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4 *)p); }
__device__ __forceinline__ bf16x8 join(const bf16x4 &a, const bf16x4 &b) {
  return bf16x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}

// The output's columns, VS of them, are dealt to a tile's rows: row 4 q + e of tile
// t is column 32 (t / 2) + 8 q + 4 (t % 2) + e, so that a lane ends with runs of
// eight.  Row of a column in this order:
__device__ __forceinline__ int dealt(int v) { return 32 * (v >> 5) + 16 * ((v >> 2) & 1) + 4 * ((v >> 3) & 3) + (v & 3); }

// What bf16 leaves of x (nothing of an infinity).
__device__ __forceinline__ float left_of(float x) {
  const float l = x - (float)(bf16)x;
  return __builtin_isfinite(l) ? l : 0.f;
}

// A pass's two chunks.  s: the state that enters it, a column a row, dealt; w: u c
// in PARTS bf16 numbers.
template <int DA, int VS, bool OUT, int PARTS_>
struct Lds {
  static constexpr int PARTS = PARTS_, P = pitch(DA), VP = pitch(VS), BUFS = OUT ? 2 : 1;
  bf16 b[BUFS][64 * P], c[2][OUT ? 64 * VP : 8], s[2][OUT ? VS * P : 8], w[BUFS][PARTS][64 * VP];
};

// A segment's chunks in the order of a pass.
struct Way {
  int64_t t0;
  int nt, nc;
  bool rev;
  __device__ __forceinline__ int rest() const { return nt - 64 * (nc - 1); }  // tokens of the last chunk
  __device__ __forceinline__ int64_t first() const { return t0 + (rev ? 64 * (int64_t)(nc - 1) : 0); }
  // whether a step's chunk has `rest` tokens; none past the last
  __device__ __forceinline__ bool part(int step) const { return step == (rev ? 0 : nc - 1); }
};
// Rows of a tensor, chunk after chunk: a buffer that ends with the chunk's last
// row, so that what lies past it (at least a row's distance from that row's
// start) reads as zeros and is not written.  All scalar: a 64-bit product a
// step made address arithmetic a third of the loops' instructions.
struct Stream {
  char *at;
  int64_t step_bytes;
  uint32_t whole, rest;
  int left;  // steps with a chunk
  bool part_now, rev;
  __device__ __forceinline__ Stream(const Way &w, const void *p, int64_t stride, int64_t column, int width, int elem) {
    at = static_cast<char *>(const_cast<void *>(p)) + (w.first() * stride + column) * elem;
    step_bytes = (w.rev ? -64 : 64) * stride * elem;
    whole = (uint32_t)((63 * stride + width) * elem);
    rest = (uint32_t)(((w.rest() - 1) * stride + width) * elem);
    left = w.nc;
    rev = w.rev;
    part_now = rev || left == 1;
  }
  __device__ __forceinline__ __amdgpu_buffer_rsrc_t next() {
    const auto r = raw_buffer(static_cast<void *>(at), left <= 0 ? 0u : part_now ? rest : whole);
    at += step_bytes;
    --left;
    part_now = !rev && left == 1;
    return r;
  }
};

// ---- the outputs' waves

// ND: blocks of 16 tokens j that the wave's tokens see.
// PART: the output is fp32, a v-head's part (a branch around stores, which may
// then be none, makes the compiler wait for loads of the step after).
template <int DA, int VS, int ND, bool PART, typename L>
__device__ __forceinline__ void outputs(const Pass &p, const Way &way, float g2, int c0, int ib, const L &lds) {
  constexpr int P = L::P, VP = L::VP, KS = DA / 32, OT = VS / 16;
  const int lane = threadIdx.x & 63, l16 = lane & 15, g = lane >> 4, i = 16 * ib + l16;
  const bool rev = way.rev;
  float wt[ND][4];  // l^{|i-j|} of the blocks at 0, 1, .. from the wave's own
#pragma unroll
  for (int d = 0; d < ND; ++d)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int far = 16 * d + (rev ? 4 * g + r - l16 : l16 - 4 * g - r);
      wt[d][r] = far >= 0 ? finite(power(g2, far) * p.scale_p) : 0.f;
    }
  struct In {
    uint4 q[KS];
  };
  Stream from(way, p.a, p.as, 0, DA, 2), to(way, p.out, p.os, c0, VS, PART ? 4 : 2);
  const int a_off = (int)(i * p.as * 2 + 16 * g), o_off = (int)((i * p.os + 8 * g) * (PART ? 4 : 2));
  const int o_line = (int)(((16 * ib + (l16 & 7)) * p.os + 8 * g) * 2 + (l16 & 8 ? 64 : 0));
  auto fetch = [&](In &in) {
    const auto r = from.next();
#pragma unroll
    for (int s = 0; s < KS; ++s) in.q[s] = buf_load16(r, (uint32_t)(a_off + 64 * s));
  };
  // the state's decay to token i: of a whole chunk, and of the last
  const float in_whole = finite(power(g2, rev ? 63 - i : i + 1) * p.scale_in);
  const float in_rest = rev ? finite(power(g2, way.rest() - 1 - i > 0 ? way.rest() - 1 - i : 0) * p.scale_in) : in_whole;
  auto work = [&](In &in, int step, auto lone) {
    constexpr bool LONE = decltype(lone)::value;  // the way's one chunk
    const bf16 *b = lds.b[step & 1], *c = lds.c[step & 1], *s = lds.s[step & 1];
    f32x4 O[OT], pd[ND];
#pragma unroll
    for (int t = 0; t < OT; ++t) O[t] = zero4();
#pragma unroll
    for (int d = 0; d < ND; ++d) pd[d] = zero4();
    // operands from LDS, a step ahead of the products that take them (left to
    // itself the compiler reads one after the other, each waited for)
    bf16x8 m[2][ND + OT], cf[(ND + 1) / 2][OT];
    auto read = [&](int k) {
#pragma unroll
      for (int d = 0; d < ND; ++d) m[k & 1][d] = M::ld(b + (16 * (rev ? ib + d : ib - d) + l16) * P + 32 * k + 8 * g);
#pragma unroll
      for (int t = 0; t < OT; ++t) m[k & 1][ND + t] = M::ld(s + (16 * t + l16) * P + 32 * k + 8 * g);
    };
    read(0);
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      if (k + 1 < KS) {
        read(k + 1);
      } else {
        const bf16 *at = c + (4 * g + (l16 >> 2)) * VP + 8 * (l16 & 3);
#pragma unroll
        for (int d = 0; d < ND; d += 2) {
          const int j0 = rev ? ib + d : ib - d, j1 = d + 1 == ND ? j0 : rev ? j0 + 1 : j0 - 1;
#pragma unroll
          for (int t = 0; t < OT; ++t) {
            const int col = 32 * (t >> 1) + 4 * (t & 1);
            cf[d / 2][t] = join(tr4(at + 16 * j0 * VP + col), tr4(at + 16 * j1 * VP + col));
          }
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      const bf16x8 q = __builtin_bit_cast(bf16x8, in.q[k]);
#pragma unroll
      for (int d = 0; d < ND; ++d) pd[d] = M::mma(m[k & 1][d], q, pd[d]);
#pragma unroll
      for (int t = 0; t < OT; ++t) O[t] = M::mma(m[k & 1][ND + t], q, O[t]);
      __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (LONE) {  // the rest of the state
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int t = 0; t < OT; ++t)
          O[t] = M::mma(M::ld(lds.s[1] + (16 * t + l16) * P + 32 * k + 8 * g), __builtin_bit_cast(bf16x8, in.q[k]), O[t]);
    } else {
      fetch(in);
    }
    const float pin = way.part(step) ? in_rest : in_whole;
#pragma unroll
    for (int t = 0; t < OT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) O[t][r] *= pin;
#pragma unroll
    for (int d = 0; d < ND; d += 2) {
      bf16x8 w;
      float f[8];
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        const int e = d + (r >> 2);
        f[r] = e < ND ? pd[e < ND ? e : d][r & 3] * wt[e < ND ? e : d][r & 3] : 0.f;
        w[r] = (bf16)f[r];
      }
#pragma unroll
      for (int t = 0; t < OT; ++t) O[t] = M::mma(cf[d / 2][t], w, O[t]);
      if constexpr (LONE) {
#pragma unroll
        for (int r = 0; r < 8; ++r) w[r] = (bf16)left_of(f[r]);
#pragma unroll
        for (int t = 0; t < OT; ++t) O[t] = M::mma(cf[d / 2][t], w, O[t]);
      }
    }
    const auto r = to.next();
    if constexpr (PART) {
#pragma unroll
      for (int t = 0; t < OT; ++t)
        buf_store16(__builtin_bit_cast(uint4, O[t]), r, (uint32_t)(o_off + 128 * (t >> 1) + 16 * (t & 1)));
      return;
    }
    uint4 o[OT / 2];
#pragma unroll
    for (int v = 0; v < OT / 2; ++v) {
      bf16x8 x;
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = (bf16)O[2 * v + (e >> 2)][e & 3];
      o[v] = __builtin_bit_cast(uint4, x);
    }
    if constexpr (OT == 2) {
      buf_store16(o[0], r, (uint32_t)o_off);
    } else {
      // lanes i and i + 8 of a group exchange halves of their rows, so that a store
      // writes whole 128-byte lines of eight rows
      const bool low = l16 < 8;
      uint4 give, own, got;
      const uint32_t *a0 = &o[0].x, *a1 = &o[1].x;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        (&own.x)[e] = low ? a0[e] : a1[e];
        (&give.x)[e] = low ? a1[e] : a0[e];
        (&got.x)[e] = __builtin_bit_cast(uint32_t, dpp_mov<0x128>(__builtin_bit_cast(float, (&give.x)[e])));  // row_ror:8
      }
      buf_store16(low ? own : got, r, (uint32_t)o_line);
      buf_store16(low ? got : own, r, (uint32_t)(o_line + 16 * p.os));
    }
  };
  In x, y;
  fetch(x);
  fetch(y);
  __syncthreads();
  // (with a way out between the two, the compiler sees one back to the loop's
  // head there too, and waits at the head for the loads of the second half)
  for (int step = 0; step + 1 < way.nc; step += 2) {
    work(x, step, std::false_type());
    __syncthreads();
    work(y, step + 1, std::false_type());
    __syncthreads();
  }
  if (way.nc == 1) {
    work(x, 0, std::true_type());
    __syncthreads();
  } else if (way.nc & 1) {
    work(x, way.nc - 1, std::false_type());
    __syncthreads();
  }
}

// ---- the state's waves

// OUT: beside the outputs' waves, which read the state of every chunk.  From step
// `exact` on the state is held to fp32, by three parts of u c instead of two
// (L::PARTS = 2: never; one part left dq and dk 1.6 times as far from 64 bits as
// rounding the output alone, two 1.4).
template <int DA, int VS, bool OUT, typename L>
__device__ __forceinline__ void states(const Pass &p, const Way &way, float g2, int DC, int c0, int exact, int tid, float *dst, L &lds) {
  constexpr int P = L::P, VP = L::VP, PARTS = L::PARTS, NS = 8, T = 64 * NS;
  // tiles of 16 x 16: KT rows by CT columns of them a wave, KW waves side by side
  // over the rows
  constexpr int CT = VS == 64 && DA >= 64 ? 2 : 1, CW = VS / 16 / CT, KW = NS / CW, KT = (DA / 16 + KW - 1) / KW;
  constexpr int NB = (64 * DA / 8 + T - 1) / T;            // pieces of b's rows, 8 elements each
  constexpr int NC = 64 * VS / T;                          // elements of c
  typedef uint32_t piece __attribute__((ext_vector_type(NC / 2)));
  static_assert(NC == 4 || NC == 8, "of one row");
  const int lane = tid & 63, wave = wave_of(tid), l16 = lane & 15, g = lane >> 4, ct = wave % CW * CT;
  const bool rev = way.rev, tiles = wave / CW < DA / 16;
  // this wave's tiles: rows 16 kt(i) + 4 g + e of column 16 (ct + j) + l16
  auto kt = [&](int i) { return wave / CW + KW * i; };
  auto state_io = [&](f32x4(&S)[KT][CT], float *ptr, bool store) {
    const int64_t sr = p.tr ? 1 : DC, sc = p.tr ? DA : 1;
    if (!tiles) return;
#pragma unroll
    for (int i = 0; i < KT; ++i)
#pragma unroll
      for (int j = 0; j < CT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float *at = ptr + (16 * kt(i) + 4 * g + e) * sr + (c0 + 16 * (ct + j) + l16) * sc;
          if (store)
            *at = S[i][j][e];
          else
            S[i][j][e] = *at;
        }
  };
  struct In {
    uint4 b[NB];
    piece c;
  };
  const int crow = tid * NC / VS, ccol = tid * NC % VS;
  Stream from_b(way, p.b, p.bs, 0, DA, 2), from_c(way, p.c, p.cs, c0, VS, 2);
  int b_off[NB];
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    const int pc = tid + T * i, row = pc / (DA / 8), col = pc % (DA / 8);
    b_off[i] = (int)(row * p.bs * 2 + col * 16);
  }
  const int c_off = (int)((crow * p.cs + ccol) * 2);
  auto fetch = [&](In &in) {
    const auto rb = from_b.next(), rc = from_c.next();
#pragma unroll
    for (int i = 0; i < NB; ++i) in.b[i] = buf_load16(rb, (uint32_t)b_off[i]);
    if constexpr (NC == 8)
      in.c = __builtin_amdgcn_raw_buffer_load_b128(rc, c_off, 0, 0);
    else
      in.c = __builtin_amdgcn_raw_buffer_load_b64(rc, c_off, 0, 0);
  };
  // from this thread's token of c to the state behind the chunk, whole or last; of all the chunk
  const int up = rev ? crow + 1 : 63 - crow, up_rest = rev ? up : up - (64 - way.rest());
  const float u_whole = finite(power(g2, up) * p.scale_up), u_rest = finite(power(g2, up_rest > 0 ? up_rest : 0) * p.scale_up);
  const float all_whole = power(g2, 64), all_rest = power(g2, way.rest());
  auto commit = [&](const In &in, int step) {
    const int buf = OUT ? step & 1 : 0;
    const float u = way.part(step) ? u_rest : u_whole;
    bf16 *at = lds.w[buf][0] + crow * VP + ccol;
    typedef bf16 els __attribute__((ext_vector_type(NC)));
    const els c = __builtin_bit_cast(els, in.c);
    els w;
    float f[NC];
#pragma unroll
    for (int e = 0; e < NC; ++e) {
      f[e] = (float)c[e] * u;
      w[e] = (bf16)f[e];
    }
    *reinterpret_cast<els *>(at) = w;
    auto rest = [&](int k) {
#pragma unroll
      for (int e = 0; e < NC; ++e) {
        f[e] -= (float)w[e];
        w[e] = (bf16)f[e];
      }
      *reinterpret_cast<els *>(at + k * 64 * VP) = w;
    };
    rest(1);
    if (PARTS > 2 && step >= exact) rest(2);
    if (OUT) *reinterpret_cast<els *>(lds.c[buf] + crow * VP + ccol) = c;
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int pc = tid + T * i, row = pc / (DA / 8), col = pc % (DA / 8);
      if (64 * DA / 8 % T == 0 || pc < 64 * DA / 8) *reinterpret_cast<uint4 *>(lds.b[buf] + row * P + col * 8) = in.b[i];
    }
  };
  f32x4 S[KT][CT];
  auto show = [&](const f32x4(&S)[KT][CT], int buf) {
    if (!OUT || !tiles) return;
#pragma unroll
    for (int j = 0; j < CT; ++j) {
      bf16 *at = lds.s[buf] + dealt(16 * (ct + j) + l16) * P + 4 * g;
#pragma unroll
      for (int i = 0; i < KT; ++i) st4(at + 16 * kt(i), S[i][j][0], S[i][j][1], S[i][j][2], S[i][j][3]);
    }
  };
  In x, y;
  fetch(x);
  fetch(y);
#pragma unroll
  for (int i = 0; i < KT; ++i)
#pragma unroll
    for (int j = 0; j < CT; ++j) S[i][j] = zero4();
  if (OUT && p.start) state_io(S, const_cast<float *>(p.start), false);
  commit(x, 0);
  show(S, 0);
  if (OUT && way.nc == 1) {  // and what bf16 leaves of it, where the next state would lie
    f32x4 low[KT][CT];
#pragma unroll
    for (int i = 0; i < KT; ++i)
#pragma unroll
      for (int j = 0; j < CT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) low[i][j][e] = left_of(S[i][j][e]);
    show(low, 1);
  }
  __syncthreads();
  // `in` is free, `next` has the chunk after this one
  auto work = [&](In &in, const In &next, int step) {
    fetch(in);
    const bf16 *b = lds.b[OUT ? step & 1 : 0], *w = lds.w[OUT ? step & 1 : 0][0];
    const float all = way.part(step) ? all_rest : all_whole;
    const int row = 4 * g + (l16 >> 2);  // of this lane's share of a transpose read
    auto tr = [&](const bf16 *m, int pitch, int s, int tile) {
      const bf16 *at = m + (32 * s + row) * pitch + 16 * tile + 4 * (l16 & 3);
      return join(tr4(at), tr4(at + 16 * pitch));
    };
    bf16x8 wf[2][PARTS][CT], bf[2][KT];
    if (tiles) {
#pragma unroll
      for (int s = 0; s < 2; ++s) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int j = 0; j < CT; ++j) wf[s][k][j] = tr(w + k * 64 * VP, VP, s, ct + j);
#pragma unroll
        for (int i = 0; i < KT; ++i) bf[s][i] = tr(b, P, s, kt(i));
      }
      if (PARTS > 2 && step >= exact) {
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int j = 0; j < CT; ++j) wf[s][PARTS - 1][j] = tr(w + 2 * 64 * VP, VP, s, ct + j);
      }
    }
    if (!OUT) __syncthreads();  // one set of rows: more workgroups a compute unit instead
    __builtin_amdgcn_sched_barrier(0);
    commit(next, step + 1);  // under the reads
    __builtin_amdgcn_sched_barrier(0);
    if (tiles) {
#pragma unroll
      for (int i = 0; i < KT; ++i)
#pragma unroll
        for (int j = 0; j < CT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) S[i][j][e] *= all;
      auto add = [&](int k) {
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int i = 0; i < KT; ++i)
#pragma unroll
            for (int j = 0; j < CT; ++j) S[i][j] = M::mma(bf[s][i], wf[s][k][j], S[i][j]);
      };
      if (PARTS > 2 && step >= exact) add(2);
      add(1);
      add(0);
    }
    if (way.nc > 1) show(S, (step + 1) & 1);
  };
  for (int step = 0; step + 1 < way.nc; step += 2) {
    work(x, y, step);
    __syncthreads();
    work(y, x, step + 1);
    __syncthreads();
  }
  if (way.nc & 1) {
    work(x, y, way.nc - 1);
    __syncthreads();
  }
  if (!OUT)
    state_io(S, dst, true);
  else if (p.last)
    state_io(S, p.last, true);
}

struct Place {
  SlotLoc loc;
  int64_t slot;
  int h, c0, kind;
};
// Items in the order (head, slot, pass, columns): what shares rows runs together
// on one XCD, and every XCD has all sequences (with slots first, those of one
// length, or the parts that nothing is asked of, were an XCD's own).
__device__ __forceinline__ Place place(const AttnArgs &a, int seg, int64_t slots, int first, int kinds, int slices, int VS) {
  int64_t item = xcd_remap(blockIdx.x, gridDim.x);
  Place p;
  p.c0 = (int)(item % slices) * VS;
  item /= slices;
  p.kind = first + (int)(item % kinds);
  item /= kinds;
  p.slot = item % slots;
  p.h = (int)(item / slots);
  // the q-heads dealt to the XCDs in turn: neighbours often decay alike, and what
  // a head costs goes by its decay
  if (a.Hq % 8 == 0) {
    const int per = a.Hv / 8, R = a.Hv / a.Hq, l = p.h % per;
    p.h = (l / R * 8 + p.h / per) * R + l % R;
  }
  p.loc = locate(a.s, seg, p.slot);
  return p;
}
__device__ __forceinline__ Way way_of(const SlotLoc &loc, bool rev) {
  Way w;
  w.t0 = loc.t0;
  w.nt = (int)(loc.t1 - loc.t0);
  w.nc = (w.nt + 63) >> 6;
  w.rev = rev;
  return w;
}

// The step from which a pass whose state is returned at the sequence's end holds
// it to fp32: what comes before is left to 2^-10 there, and its own error of 2^-18
// to 2^-28.
__device__ __forceinline__ int exact_from(const AttnArgs &a, const SlotLoc &loc, const Way &way, float g2) {
  const Span sp = seq_span(a.s, loc.n);
  const float near = 10.f / fmaxf(-g2, 1e-7f);  // tokens from the end
  // from the pass's first token to the sequence's end on its way
  const int64_t all = way.rev ? way.t0 + way.nt - sp.first : sp.end - way.t0;
  if (!(near < (float)all)) return 0;
  const int64_t step = (all - (int64_t)near) / 64 - 1;
  return step < 0 ? 0 : step < way.nc ? (int)step : way.nc;
}

// The passes first .. first + kinds - 1, whose a and b are DA wide and whose
// output is DC.  EXACT: some return their state.
template <int DA, int VS, bool EXACT, bool PART>
__global__ __launch_bounds__(768, 3) void mma_kernel(AttnArgs a, Layout w, int first, int kinds, int DC) {
  __shared__ __align__(16) Lds<DA, VS, true, EXACT ? 3 : 2> lds;
  const Place at = place(a, a.seg, a.slots, first, kinds, DC / VS, VS);
  if (!at.loc.used) return;
  const Pass p = make_pass<bf16>(a, w, at.kind, at.loc, at.h);
  const Way way = way_of(at.loc, p.rev);
  const float g2 = log2_decay(a.g[at.h]);
  const int wave = wave_of(threadIdx.x);
  if (wave >= 4) {
    states<DA, VS, true>(p, way, g2, DC, at.c0, p.last ? exact_from(a, at.loc, way, g2) : way.nc, threadIdx.x - 256, nullptr, lds);
    return;
  }
  switch (p.rev ? 4 - wave : wave + 1) {
    case 1: outputs<DA, VS, 1, PART>(p, way, g2, at.c0, wave, lds); break;
    case 2: outputs<DA, VS, 2, PART>(p, way, g2, at.c0, wave, lds); break;
    case 3: outputs<DA, VS, 3, PART>(p, way, g2, at.c0, wave, lds); break;
    default: outputs<DA, VS, 4, PART>(p, way, g2, at.c0, wave, lds);
  }
}

// What a part of a segment adds to S (o's pass) and, with two kinds, to Z (dv's).
// Tokens whose decay to the next segment is 0 in fp32 add nothing and are not read.
template <int DA, int VS>
__global__ __launch_bounds__(512, 4) void mma_local_kernel(AttnArgs a, Layout w, int64_t slots, int kinds) {
  __shared__ __align__(16) Lds<DA, VS, false, 3> lds;
  Place at = place(a, a.seg / a.parts, slots, 0, kinds, a.V / VS, VS);
  if (!at.loc.used) return;
  const Pass p = make_pass<bf16>(a, w, at.kind ? kDv : kO, at.loc, at.h);
  if (!carried(a, at.loc, p.rev)) return;
  float *dst = (p.rev ? w.zend(a) : w.start(a)) + (at.slot * a.Hv + at.h) * (int64_t)DA * a.V;
  const float g2 = log2_decay(a.g[at.h]);
  // tokens between the part and the segment's border, and how far it sees
  const int sub = a.seg / a.parts, part = (int)(at.loc.index % a.parts);
  const int64_t n = at.loc.t1 - at.loc.t0, past = (int64_t)sub * (p.rev ? part : a.parts - 1 - part);
  if (g2 * (float)(n + past) < -151.f) {
    const int64_t seen = (int64_t)(151.f / -g2) + 1 - past, most = seen < 0 ? 0 : seen < n ? seen : n;
    if (p.rev)
      at.loc.t1 = at.loc.t0 + most;
    else
      at.loc.t0 += (n - most) / 64 * 64;
  }
  const Way way = way_of(at.loc, p.rev);
  states<DA, VS, false>(p, way, g2, a.V, at.c0, (p.rev ? a.dh0 : a.ht) ? exact_from(a, at.loc, way, g2) : way.nc, threadIdx.x, dst, lds);
}

template <typename F>
void with_sizes(int DA, int DC, int cols, F f) {
  auto wide = [&](auto da) {
    if (DC == 32 || cols == 32)
      f(da, std::integral_constant<int, 32>());
    else
      f(da, std::integral_constant<int, 64>());
  };
  if (DA == 32)
    wide(std::integral_constant<int, 32>());
  else if (DA == 64)
    wide(std::integral_constant<int, 64>());
  else
    wide(std::integral_constant<int, 128>());
}

// exact: a state of these passes is returned; part: they write v-heads' parts
hipError_t run(const char *name, const AttnArgs &a, const Layout &w, int DA, int DC, int first, int kinds, bool exact, bool part, hipStream_t st) {
  KernelTimer kt(name, st);
  with_sizes(DA, DC, a.cols, [&](auto da, auto vs) {
    const unsigned blocks = (unsigned)(a.slots * a.Hv * kinds * (DC / vs));
    if (part)
      mma_kernel<da, vs, false, true><<<blocks, 768, 0, st>>>(a, w, first, kinds, DC);
    else if (exact)
      mma_kernel<da, vs, true, false><<<blocks, 768, 0, st>>>(a, w, first, kinds, DC);
    else
      mma_kernel<da, vs, false, false><<<blocks, 768, 0, st>>>(a, w, first, kinds, DC);
  });
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mma_local(const AttnArgs &a, const Layout &w, bool both, hipStream_t st) {
  const int kinds = both ? 2 : 1;
  KernelTimer kt("attn_local", st);
  with_sizes(a.K, a.V, 64, [&](auto da, auto vs) {
    const int64_t slots = scan::slots_of(a.s, a.seg / a.parts);
    mma_local_kernel<da, vs><<<(unsigned)(slots * a.Hv * kinds * (a.V / vs)), 512, 0, st>>>(a, w, slots, kinds);
  });
  return hipGetLastError();
}
hipError_t launch_mma_out(const AttnArgs &a, const Layout &w, hipStream_t st) {
  return run("attn_out", a, w, a.K, a.V, kO, 1, a.ht != nullptr, false, st);
}
hipError_t launch_mma_grads(const AttnArgs &a, const Layout &w, hipStream_t st) {
  const bool exact = a.dh0 != nullptr, part = a.Hv != a.Hq;
  if (a.K == a.V && !exact && !part) return run("attn_grads", a, w, a.K, a.V, kDq, 3, false, false, st);
  const hipError_t e = run("attn_grads", a, w, a.V, a.K, kDq, 2, false, part, st);
  return e != hipSuccess ? e : run("attn_grads", a, w, a.K, a.V, kDv, 1, exact, false, st);
}

}  // namespace attn
}  // namespace gdn
