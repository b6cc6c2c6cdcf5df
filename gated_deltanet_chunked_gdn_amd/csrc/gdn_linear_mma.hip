// Linear attention with a decay for each head, bf16 (gdn_linear.hpp has the
// passes): chunks of 64 tokens, the state in MFMA accumulators.
//
// A workgroup has a segment of one head and 32 of the output's columns.  Its
// waves work side by side on a chunk: four on the outputs, 16 tokens i each,
//
//   O^T = l^{i+1} S^T A^T + C^T P^T,   P^T = (B A^T) l^{i-j}, rows j, lanes i
//
// and four on the state, a tile of 16 rows and 16 columns after the other,
//
//   S' = l^64 S + B^T (u C),   u_j = l^{63-j}
//
// so that a chunk costs one barrier: b, c and the state (as bf16, transposed)
// lie in LDS twice, the next chunk's written under the present one's products,
// and the loads run two chunks ahead.  a goes from memory to the lanes that
// multiply it.  P^T's accumulators are the next product's operand as they
// are, its tokens in the order 16 t + 4 g + e in which C^T is then read (g: the
// lane's group of 16).  The columns of an output tile are dealt so that a lane
// ends with eight in a row.
//
// Roundings to bf16: P and the state as operands of the outputs, which are bf16
// themselves.  The state is held in fp32; where it is returned or carried to
// another segment its update takes the weighted c, an fp32 number, as three
// bf16 parts, which lose nothing, elsewhere as one.
#include <type_traits>

#include "gdn_internal.h"
#include "gdn_linear.hpp"

namespace gdn {
namespace attn {
namespace {

// Row pitches in LDS: 32 bytes over a multiple of 64.  16-byte reads of 16 rows
// then take 4 clocks and transpose reads of 32 bytes of 16 rows 1.4 (with 16
// bytes over: 8 and 2.1).
constexpr int VP = 48;  // of c's 32 columns
typedef Mma<bf16> M;
typedef __attribute__((address_space(3))) bf16x4 lds_bf16x4;
__device__ __forceinline__ bf16x4 tr4(const bf16 *p) { return __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4 *)p); }
__device__ __forceinline__ bf16x8 join(const bf16x4 &a, const bf16x4 &b) {
  return bf16x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}

// A pass's two chunks.  s: the state that enters it, a column a row, in the order
// 16 ((v >> 2) & 1) + 4 (v >> 3) + (v & 3) (what the lanes of an output tile
// take); w: u c in PARTS bf16 numbers.
template <int DA, bool OUT, int PARTS>
struct Lds {
  static constexpr int P = DA + 16;
  bf16 b[2][64 * P], c[2][OUT ? 64 * VP : 8], s[2][OUT ? 32 * P : 8], w[2][PARTS][64 * VP];
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
template <int DA, int ND, typename L>
__device__ __forceinline__ void outputs(const Pass &p, const Way &way, float g2, int c0, int ib, const L &lds) {
  constexpr int P = L::P, KS = DA / 32;
  const int lane = threadIdx.x & 63, l16 = lane & 15, g = lane >> 4, i = 16 * ib + l16;
  const bool rev = way.rev;
  float wt[ND][4];  // l^{|i-j|} of the blocks at 0, 1, .. from the wave's own
#pragma unroll
  for (int d = 0; d < ND; ++d)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int far = 16 * d + (rev ? 4 * g + r - l16 : l16 - 4 * g - r);
      wt[d][r] = far >= 0 ? power(g2, far) * p.scale_p : 0.f;
    }
  struct In {
    uint4 q[KS];
  };
  Stream from(way, p.a, p.as, 0, DA, 2), to(way, p.out, p.os, c0, 32, p.part ? 4 : 2);
  const int a_off = (int)(i * p.as * 2 + 16 * g), o_off = (int)((i * p.os + 8 * g) * (p.part ? 4 : 2));
  auto fetch = [&](In &in) {
    const auto r = from.next();
#pragma unroll
    for (int s = 0; s < KS; ++s) in.q[s] = buf_load16(r, (uint32_t)(a_off + 64 * s));
  };
  // the state's decay to token i: of a whole chunk, and of the last
  const float in_whole = power(g2, rev ? 63 - i : i + 1) * p.scale_in;
  const float in_rest = rev ? power(g2, way.rest() - 1 - i > 0 ? way.rest() - 1 - i : 0) * p.scale_in : in_whole;
  auto work = [&](In &in, int step) {
    const bf16 *b = lds.b[step & 1], *c = lds.c[step & 1], *s = lds.s[step & 1];
    f32x4 O[2] = {zero4(), zero4()}, pd[ND];
#pragma unroll
    for (int d = 0; d < ND; ++d) pd[d] = zero4();
    // operands from LDS, a step ahead of the products that take them (left to
    // itself the compiler reads one after the other, each waited for)
    bf16x8 m[2][ND + 2], cf[(ND + 1) / 2][2];
    auto read = [&](int k) {
#pragma unroll
      for (int d = 0; d < ND; ++d) m[k & 1][d] = M::ld(b + (16 * (rev ? ib + d : ib - d) + l16) * P + 32 * k + 8 * g);
#pragma unroll
      for (int t = 0; t < 2; ++t) m[k & 1][ND + t] = M::ld(s + (16 * t + l16) * P + 32 * k + 8 * g);
    };
    read(0);
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      if (k + 1 < KS) {
        read(k + 1);
      } else {
        // row 4 q + e of tile t: column 8 q + 4 t + e
        const bf16 *at = c + (4 * g + (l16 >> 2)) * VP + 8 * (l16 & 3);
#pragma unroll
        for (int d = 0; d < ND; d += 2) {
          const int j0 = rev ? ib + d : ib - d, j1 = d + 1 == ND ? j0 : rev ? j0 + 1 : j0 - 1;
#pragma unroll
          for (int t = 0; t < 2; ++t) cf[d / 2][t] = join(tr4(at + 16 * j0 * VP + 4 * t), tr4(at + 16 * j1 * VP + 4 * t));
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      const bf16x8 q = __builtin_bit_cast(bf16x8, in.q[k]);
#pragma unroll
      for (int d = 0; d < ND; ++d) pd[d] = M::mma(m[k & 1][d], q, pd[d]);
#pragma unroll
      for (int t = 0; t < 2; ++t) O[t] = M::mma(m[k & 1][ND + t], q, O[t]);
      __builtin_amdgcn_sched_barrier(0);
    }
    fetch(in);
    const float pin = way.part(step) ? in_rest : in_whole;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) O[t][r] *= pin;
#pragma unroll
    for (int d = 0; d < ND; d += 2) {
      bf16x8 w;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        w[r] = (bf16)(pd[d][r] * wt[d][r]);
        w[4 + r] = d + 1 < ND ? (bf16)(pd[d + 1 < ND ? d + 1 : d][r] * wt[d + 1 < ND ? d + 1 : d][r]) : (bf16)0.f;
      }
#pragma unroll
      for (int t = 0; t < 2; ++t) O[t] = M::mma(cf[d / 2][t], w, O[t]);
    }
    const auto r = to.next();
    if (p.part) {
#pragma unroll
      for (int t = 0; t < 2; ++t) buf_store16(__builtin_bit_cast(uint4, O[t]), r, (uint32_t)(o_off + 16 * t));
    } else {
      bf16x8 o;
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = (bf16)O[e >> 2][e & 3];
      buf_store16(__builtin_bit_cast(uint4, o), r, (uint32_t)o_off);
    }
  };
  In x, y;
  fetch(x);
  fetch(y);
  __syncthreads();
  // (with a way out between the two, the compiler sees one back to the loop's
  // head there too, and waits at the head for the loads of the second half)
  for (int step = 0; step + 1 < way.nc; step += 2) {
    work(x, step);
    __syncthreads();
    work(y, step + 1);
    __syncthreads();
  }
  if (way.nc & 1) {
    work(x, way.nc - 1);
    __syncthreads();
  }
}

// ---- the state's waves

// OUT: beside the outputs' waves, which read the state of every chunk.  EXACT:
// the state is wanted to fp32.  NS waves.
template <int DA, int NS, bool OUT, bool EXACT>
__device__ __forceinline__ void states(const Pass &p, const Way &way, float g2, int DC, int c0, int tid, float *dst,
                                       Lds<DA, OUT, EXACT ? 3 : 1> &lds) {
  constexpr int P = Lds<DA, OUT, EXACT ? 3 : 1>::P, PARTS = EXACT ? 3 : 1, T = 64 * NS;
  constexpr int KT = (DA / 8 + NS - 1) / NS;               // tiles of 16 x 16
  constexpr int NB = (64 * DA / 8 + T - 1) / T;            // pieces of b's rows, 8 elements each
  constexpr int NC = 2048 / T;                             // elements of c
  typedef uint32_t piece __attribute__((ext_vector_type(NC / 2)));
  static_assert(NC == 4 || NC == 8, "of one row");
  const int lane = tid & 63, wave = wave_of(tid), l16 = lane & 15, g = lane >> 4, ct = wave & 1;
  const bool rev = way.rev, tiles = wave < DA / 8;
  // this wave's tiles: rows 16 kt + 4 g + e of column 16 ct + l16
  auto kt = [&](int i) { return (wave + NS * i) >> 1; };
  auto state_io = [&](f32x4(&S)[KT], float *ptr, bool store) {
    const int64_t sr = p.tr ? 1 : DC, sc = p.tr ? DA : 1;
    ptr += (c0 + 16 * ct + l16) * sc;
    if (!tiles) return;
#pragma unroll
    for (int i = 0; i < KT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float *at = ptr + (16 * kt(i) + 4 * g + e) * sr;
        if (store)
          *at = S[i][e];
        else
          S[i][e] = *at;
      }
  };
  struct In {
    uint4 b[NB];
    piece c;
  };
  const int crow = tid * NC / 32, ccol = tid * NC % 32;
  Stream from_b(way, p.b, p.bs, 0, DA, 2), from_c(way, p.c, p.cs, c0, 32, 2);
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
  const float u_whole = power(g2, up) * p.scale_up, u_rest = power(g2, up_rest > 0 ? up_rest : 0) * p.scale_up;
  const float all_whole = power(g2, 64), all_rest = power(g2, way.rest());
  auto commit = [&](const In &in, int step) {
    const int buf = step & 1;
    const float u = way.part(step) ? u_rest : u_whole;
    bf16 *at = lds.w[buf][0] + crow * VP + ccol;
    typedef bf16 els __attribute__((ext_vector_type(NC)));
    const els c = __builtin_bit_cast(els, in.c);
    els w[PARTS];
#pragma unroll
    for (int e = 0; e < NC; ++e) {
      float f = (float)c[e] * u;
#pragma unroll
      for (int k = 0; k < PARTS; ++k) {
        w[k][e] = (bf16)f;
        f -= (float)w[k][e];
      }
    }
#pragma unroll
    for (int k = 0; k < PARTS; ++k) *reinterpret_cast<els *>(at + k * 64 * VP) = w[k];
    if (OUT) *reinterpret_cast<els *>(lds.c[buf] + crow * VP + ccol) = c;
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int pc = tid + T * i, row = pc / (DA / 8), col = pc % (DA / 8);
      if (64 * DA / 8 % T == 0 || pc < 64 * DA / 8) *reinterpret_cast<uint4 *>(lds.b[buf] + row * P + col * 8) = in.b[i];
    }
  };
  f32x4 S[KT];
  auto show = [&](int buf) {
    if (!OUT || !tiles) return;
#pragma unroll
    for (int i = 0; i < KT; ++i) {
      const int v = 16 * ct + l16, row = 16 * ((v >> 2) & 1) + 4 * (v >> 3) + (v & 3);
      st4(lds.s[buf] + row * P + 16 * kt(i) + 4 * g, S[i][0], S[i][1], S[i][2], S[i][3]);
    }
  };
  In x, y;
  fetch(x);
  fetch(y);
#pragma unroll
  for (int i = 0; i < KT; ++i) S[i] = zero4();
  if (OUT && p.start) state_io(S, const_cast<float *>(p.start), false);
  commit(x, 0);
  show(0);
  __syncthreads();
  // `in` is free, `next` has the chunk after this one
  auto work = [&](In &in, const In &next, int step) {
    fetch(in);
    const bf16 *b = lds.b[step & 1], *w = lds.w[step & 1][0];
    const float all = way.part(step) ? all_rest : all_whole;
    const int row = 4 * g + (l16 >> 2);  // of this lane's share of a transpose read
    auto tr = [&](const bf16 *m, int pitch, int s, int tile) {
      const bf16 *at = m + (32 * s + row) * pitch + 16 * tile + 4 * (l16 & 3);
      return join(tr4(at), tr4(at + 16 * pitch));
    };
    if (tiles) {
#pragma unroll
      for (int i = 0; i < KT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) S[i][e] *= all;
      bf16x8 wf[2][PARTS], bf[2][KT];
#pragma unroll
      for (int s = 0; s < 2; ++s) {
#pragma unroll
        for (int k = 0; k < PARTS; ++k) wf[s][k] = tr(w + k * 64 * VP, VP, s, ct);
#pragma unroll
        for (int i = 0; i < KT; ++i) bf[s][i] = tr(b, P, s, kt(i));
      }
      __builtin_amdgcn_sched_barrier(0);
      commit(next, step + 1);  // under the reads
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int k = PARTS - 1; k >= 0; --k)
#pragma unroll
          for (int i = 0; i < KT; ++i) S[i] = M::mma(bf[s][i], wf[s][k], S[i]);
    } else {
      commit(next, step + 1);
    }
    show((step + 1) & 1);
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
  bool out;  // past the work
};
// Items in the order (slot, head, pass, columns): what shares rows runs together
// on one XCD.
__device__ __forceinline__ Place place(const AttnArgs &a, int first, int kinds, int slices) {
  int64_t item = xcd_remap(blockIdx.x, gridDim.x);
  Place p;
  p.c0 = (int)(item % slices) * 32;
  item /= slices;
  p.kind = first + (int)(item % kinds);
  item /= kinds;
  p.h = (int)(item % a.Hv);
  p.slot = item / a.Hv;
  p.loc = locate(a.s, a.seg, p.slot);
  p.out = !p.loc.used;
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

// The passes first .. first + kinds - 1, whose a and b are DA wide and whose
// output is DC.
template <int DA, bool EXACT>
__global__ __launch_bounds__(768, 3) void mma_kernel(AttnArgs a, Layout w, int first, int kinds, int DC) {
  __shared__ __align__(16) Lds<DA, true, EXACT ? 3 : 1> lds;
  const Place at = place(a, first, kinds, DC / 32);
  if (at.out) return;
  const Pass p = make_pass<bf16>(a, w, at.kind, at.loc, at.slot, at.h);
  const Way way = way_of(at.loc, p.rev);
  const float g2 = log2_decay(a.g[at.h]);
  const int wave = wave_of(threadIdx.x);
  if (wave >= 4) {
    states<DA, 8, true, EXACT>(p, way, g2, DC, at.c0, threadIdx.x - 256, nullptr, lds);
    return;
  }
  switch (p.rev ? 4 - wave : wave + 1) {
    case 1: outputs<DA, 1>(p, way, g2, at.c0, wave, lds); break;
    case 2: outputs<DA, 2>(p, way, g2, at.c0, wave, lds); break;
    case 3: outputs<DA, 3>(p, way, g2, at.c0, wave, lds); break;
    default: outputs<DA, 4>(p, way, g2, at.c0, wave, lds);
  }
}

// What a segment adds to S (o's pass) and, with two kinds, to Z (dv's).
template <int DA>
__global__ __launch_bounds__(256) void mma_local_kernel(AttnArgs a, Layout w, int kinds) {
  __shared__ __align__(16) Lds<DA, false, 3> lds;
  const Place at = place(a, 0, kinds, a.V / 32);
  if (at.out) return;
  const Pass p = make_pass<bf16>(a, w, at.kind ? kDv : kO, at.loc, at.slot, at.h);
  if (p.rev ? at.loc.index == 0 : at.loc.last) return;
  float *dst = (p.rev ? w.zend(a) : w.start(a)) + (at.slot * a.Hv + at.h) * (int64_t)DA * a.V;
  states<DA, 4, false, true>(p, way_of(at.loc, p.rev), log2_decay(a.g[at.h]), a.V, at.c0, threadIdx.x, dst, lds);
}

// exact: a state of these passes is returned
hipError_t run(const char *name, const AttnArgs &a, const Layout &w, int DA, int DC, int first, int kinds, bool exact, hipStream_t st) {
  const unsigned blocks = (unsigned)(a.slots * a.Hv * kinds * (DC / 32));
  KernelTimer kt(name, st);
  auto go = [&](auto exact) {
    constexpr bool X = decltype(exact)::value;
    if (DA == 32)
      mma_kernel<32, X><<<blocks, 768, 0, st>>>(a, w, first, kinds, DC);
    else if (DA == 64)
      mma_kernel<64, X><<<blocks, 768, 0, st>>>(a, w, first, kinds, DC);
    else
      mma_kernel<128, X><<<blocks, 768, 0, st>>>(a, w, first, kinds, DC);
  };
  if (exact)
    go(std::true_type());
  else
    go(std::false_type());
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mma_local(const AttnArgs &a, const Layout &w, bool both, hipStream_t st) {
  const int kinds = both ? 2 : 1;
  const unsigned blocks = (unsigned)(a.slots * a.Hv * kinds * (a.V / 32));
  KernelTimer kt("attn_local", st);
  if (a.K == 32)
    mma_local_kernel<32><<<blocks, 256, 0, st>>>(a, w, kinds);
  else if (a.K == 64)
    mma_local_kernel<64><<<blocks, 256, 0, st>>>(a, w, kinds);
  else
    mma_local_kernel<128><<<blocks, 256, 0, st>>>(a, w, kinds);
  return hipGetLastError();
}
hipError_t launch_mma_out(const AttnArgs &a, const Layout &w, hipStream_t st) {
  return run("attn_out", a, w, a.K, a.V, kO, 1, a.ht != nullptr, st);
}
hipError_t launch_mma_grads(const AttnArgs &a, const Layout &w, hipStream_t st) {
  const bool exact = a.dh0 != nullptr;
  if (a.K == a.V && !exact) return run("attn_grads", a, w, a.K, a.V, kDq, 3, false, st);
  const hipError_t e = run("attn_grads", a, w, a.V, a.K, kDq, 2, false, st);
  return e != hipSuccess ? e : run("attn_grads", a, w, a.K, a.V, kDv, 1, exact, st);
}

}  // namespace attn
}  // namespace gdn
