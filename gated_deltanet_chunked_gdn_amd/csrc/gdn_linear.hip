// Linear attention with a decay for each head (gdn_linear.hpp has the
// formulas): the passes of fp32 problems, in fp32 matrix instructions, and what
// joins segments and heads.
//
// A workgroup has a segment of one head and 32 of the output's columns; chunks
// of 32 tokens.  The state is in accumulators and, for the chunk that reads
// it, in LDS.  Operands and sums are fp32 throughout.  Short batches are bound by launches
// and by the chain of chunks: segments as short as gives each compute unit two
// workgroups, their states summed up by the outputs' pass itself where they are few
// (plan_f32).  7 packed prompts, 1277 tokens, 8 heads, K = V = 64: 18 us a call (5
// more with a carry between); backward of 5, 1901 tokens, 8 heads (4 of q and k): 47
// a call, in a trace states 12, carry 7.5, gradients 27.5, shared heads 4.5.
#include "gdn_internal.h"
#include "gdn_linear.hpp"

namespace gdn {
namespace attn {
namespace {

constexpr int C = 32;        // tokens a chunk
constexpr int kAhead = 8;    // segments whose states a carry has in flight
constexpr int kThreads = 256;
constexpr int kJoinAhead = 4;  // segments whose states the outputs' pass has in flight where it joins them

// What a launch does: the state a segment adds (forwards; or forwards and
// backwards, for the backward), o, or the three gradients.
enum { kLocal, kLocals, kForward, kGrads };

template <int D>
struct Lds {
  static constexpr int P = D + 4;  // row pitches: a column of 16 rows meets every bank once
  float a[C * P], b[C * P], c[C * 36], p[C * 36], s[32 * P], pw[C + 1];
};

// A chunk's rows of COLS columns in the registers of a workgroup; rows past
// its end lie past the buffer's, and read as zeros.
template <int COLS>
struct Rows {
  static constexpr int PER = 4, PIECES = C * COLS / PER, N = (PIECES + kThreads - 1) / kThreads;
  uint4 r[N];
  __device__ __forceinline__ void load(const float *p, int64_t stride, int rows, int tid) {
    const uint32_t bytes = rows > 0 ? (uint32_t)(((rows - 1) * stride + COLS) * 4) : 0u;
    const auto rsrc = raw_buffer(p, bytes);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int pc = tid + i * kThreads, row = pc / (COLS / PER), col = pc % (COLS / PER);
      r[i] = buf_load16(rsrc, (uint32_t)(row * stride * 4 + col * 16));
    }
  }
  __device__ __forceinline__ void store(float *lds, int pitch, int tid) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int pc = tid + i * kThreads, row = pc / (COLS / PER), col = pc % (COLS / PER);
      if (PIECES % kThreads != 0 && pc >= PIECES) continue;
      *reinterpret_cast<uint4 *>(lds + row * pitch + col * PER) = r[i];
    }
  }
};

__device__ __forceinline__ f32x4 prod(const f32x4 &x, const f32x4 &y, f32x4 c) {
#pragma unroll
  for (int k = 0; k < 4; ++k) c = Mma<float>::mma(x[k], y[k], c);
  return c;
}

// DA: width of a and b, DC: of c and the output, of which the workgroup has
// 32 columns from c0.
template <int DA, int DC, bool OUT>
__device__ __forceinline__ void sweep(const AttnArgs &args, const Pass &p, const SlotLoc &loc, float *state, int h, int c0, Lds<DA> &lds) {
  constexpr int P = Lds<DA>::P, KT = DA / 32;
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_of(tid), l16 = lane & 15, q = lane >> 4;
  const float g2 = log2_decay(args.g[h]);
  // (finite with the pass's scale as well)
  if (tid <= C) lds.pw[tid] = finite(power(g2, tid), 0.9999f * __FLT_MAX__ / fmaxf(1.f, fabsf(args.scale)));

  // this wave's tiles of the state: rows 16 kt + 4 q + e of column 16 ct + l16
  auto kt = [&](int i) { return (wave + 4 * i) >> 1; };
  const int ct = wave & 1;
  auto state_io = [&](f32x4(&S)[KT], float *ptr, bool store) {
#pragma unroll
    for (int i = 0; i < KT; ++i) {
      const int r = 16 * kt(i) + 4 * q, c = c0 + 16 * ct + l16;
      if (p.tr) {  // never stored: dq and dk return no state
        S[i] = *reinterpret_cast<const f32x4 *>(ptr + (int64_t)c * DA + r);
        continue;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float *at = ptr + (int64_t)(r + e) * DC + c;
        if (store)
          *at = S[i][e];
        else
          S[i][e] = *at;
      }
    }
  };
  f32x4 S[KT];
  if (OUT && p.start) {
    state_io(S, const_cast<float *>(p.start), false);
  } else {
#pragma unroll
    for (int i = 0; i < KT; ++i) S[i] = zero4();
  }
  if (OUT) {
    for (int s0 = 0; s0 < p.before; s0 += kJoinAhead) {
      f32x4 add[kJoinAhead][KT];
#pragma unroll
      for (int j = 0; j < kJoinAhead; ++j)
        if (s0 + j < p.before) state_io(add[j], const_cast<float *>(p.added + (s0 + j) * p.step), false);
#pragma unroll
      for (int j = 0; j < kJoinAhead; ++j) {
        if (s0 + j >= p.before) break;
        const float d = power(g2, s0 + j == 0 ? p.nt0 : args.seg);
#pragma unroll
        for (int i = 0; i < KT; ++i) S[i] = S[i] * d + add[j][i];
      }
    }
  }
  const int nt = (int)(loc.t1 - loc.t0), nc = (nt + C - 1) / C;
  struct In {
    Rows<DA> a, b;
    Rows<32> c;
  };
  auto fetch = [&](In &r, int step) {
    const int ch = p.rev ? nc - 1 - step : step;
    const int64_t t = loc.t0 + (int64_t)C * ch;
    const int rows = nt - C * ch < C ? nt - C * ch : C;
    if (OUT) r.a.load(static_cast<const float *>(p.a) + t * p.as, p.as, rows, tid);
    r.b.load(static_cast<const float *>(p.b) + t * p.bs, p.bs, rows, tid);
    r.c.load(static_cast<const float *>(p.c) + t * p.cs + c0, p.cs, rows, tid);
  };
  In in;
  if (nc > 0) fetch(in, 0);
  for (int step = 0; step < nc; ++step) {
    const int ch = p.rev ? nc - 1 - step : step;
    const int n = nt - C * ch < C ? nt - C * ch : C;
    __syncthreads();  // the chunk before is done with LDS
    if (OUT) in.a.store(lds.a, P, tid);
    in.b.store(lds.b, P, tid);
    in.c.store(lds.c, 36, tid);
    if (OUT) {
#pragma unroll
      for (int i = 0; i < KT; ++i)
        *reinterpret_cast<f32x4 *>(lds.s + (16 * ct + l16) * P + 16 * kt(i) + 4 * q) = S[i];
    }
    __syncthreads();
    if (step + 1 < nc) fetch(in, step + 1);
    // decays of the token from the state before the chunk, and from it to the state behind
    auto w_in = [&](int i) { return p.rev ? lds.pw[n - 1 - i > 0 ? n - 1 - i : 0] : lds.pw[i + 1]; };
    auto w_up = [&](int j) { return p.rev ? lds.pw[j + 1] : lds.pw[n - 1 - j > 0 ? n - 1 - j : 0]; };
    f32x4 O = zero4();
    const int it = wave >> 1, jt = wave & 1;
    if (OUT) {
      // a wave's 16 x 16 of the pairs, and of the state's share of the output
      f32x4 pair = zero4();
#pragma unroll
      for (int s = 0; s < DA / 16; ++s) {
        const f32x4 x = *reinterpret_cast<const f32x4 *>(lds.a + (16 * it + l16) * P + 16 * s + 4 * q);
        const f32x4 y = *reinterpret_cast<const f32x4 *>(lds.b + (16 * jt + l16) * P + 16 * s + 4 * q);
        const f32x4 z = *reinterpret_cast<const f32x4 *>(lds.s + (16 * jt + l16) * P + 16 * s + 4 * q);
        pair = prod(x, y, pair);
        O = prod(x, z, O);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = 16 * it + 4 * q + e, d = p.rev ? 16 * jt + l16 - i : i - (16 * jt + l16);
        lds.p[i * 36 + 16 * jt + l16] = d >= 0 ? pair[e] * (lds.pw[d >= 0 ? d : 0] * p.scale_p) : 0.f;
        O[e] *= w_in(i) * p.scale_in;
      }
      __syncthreads();
#pragma unroll
      for (int s = 0; s < C / 16; ++s) {
        const f32x4 x = *reinterpret_cast<const f32x4 *>(lds.p + (16 * it + l16) * 36 + 16 * s + 4 * q);
        f32x4 y;
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = lds.c[(16 * s + 4 * q + e) * 36 + 16 * jt + l16];
        O = prod(x, y, O);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = 16 * it + 4 * q + e;
        const int64_t at = (loc.t0 + (int64_t)C * ch + i) * p.os + c0 + 16 * jt + l16;
        if (i < n) static_cast<float *>(p.out)[at] = O[e];
      }
    }
    // S = l^n S + sum_j u_j b_j c_j^T
    const float all = lds.pw[n];
    f32x4 cw[C / 16];
#pragma unroll
    for (int s = 0; s < C / 16; ++s)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = 16 * s + 4 * q + e;
        cw[s][e] = lds.c[j * 36 + 16 * ct + l16] * (w_up(j) * p.scale_up);
      }
#pragma unroll
    for (int i = 0; i < KT; ++i) {
#pragma unroll
      for (int e = 0; e < 4; ++e) S[i][e] *= all;
#pragma unroll
      for (int s = 0; s < C / 16; ++s) {
        f32x4 x;
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = lds.b[(16 * s + 4 * q + e) * P + 16 * kt(i) + l16];
        S[i] = prod(x, cw[s], S[i]);
      }
    }
  }
  if (!OUT)
    state_io(S, state, true);
  else if (p.last)
    state_io(S, p.last, true);
}

template <int K, int V, int WHAT>
__global__ __launch_bounds__(kThreads) void pass_kernel(AttnArgs a, Layout w, int64_t slots, int64_t per) {
  constexpr int D = K > V ? K : V;
  __shared__ __align__(16) char mem[sizeof(Lds<(WHAT == kGrads ? D : K)>)];
  const int64_t part = blockIdx.x / per, item = blockIdx.x % per;
  int kind = kO;
  if (WHAT == kLocals) kind = part ? kDv : kO;
  int64_t unit = item;  // (slot, head, 32 columns)
  if (WHAT == kGrads) kind = part == 0 ? kDv : part == 1 ? kDk : kDq;
  const bool tr = WHAT == kGrads && kind != kDv;
  const int slices = (tr ? K : V) / 32;
  const int64_t head = unit / slices;
  const int c0 = (int)(unit % slices) * 32, h = (int)(head % a.Hv);
  const int64_t slot = head / a.Hv;
  if (slot >= slots) return;
  constexpr bool LOCAL = WHAT == kLocal || WHAT == kLocals;
  const SlotLoc loc = locate(a.s, LOCAL ? a.seg / a.parts : a.seg, slot);
  if (!loc.used) return;
  Pass p = make_pass<float>(a, w, kind, loc, h);
  if constexpr (LOCAL) {
    if (!carried(a, loc, p.rev)) return;
    // the state is built of b and c
    float *dst = (p.rev ? w.zend(a) : w.start(a)) + (slot * a.Hv + h) * (int64_t)K * V;
    sweep<K, V, false>(a, p, loc, dst, h, c0, *reinterpret_cast<Lds<K> *>(mem));
  } else if constexpr (WHAT == kForward) {
    sweep<K, V, true>(a, p, loc, nullptr, h, c0, *reinterpret_cast<Lds<K> *>(mem));
  } else {
    if (tr)
      sweep<V, K, true>(a, p, loc, nullptr, h, c0, *reinterpret_cast<Lds<V> *>(mem));
    else
      sweep<K, V, true>(a, p, loc, nullptr, h, c0, *reinterpret_cast<Lds<K> *>(mem));
  }
}

// The parts of a sequence's segments in order, 4 elements of the state a thread:
// where a segment but the sequence's first begins (backwards: but its last ends),
// its part gets the state there.
template <bool REV>
__device__ __forceinline__ void carry(const AttnArgs &a, const Layout &w, int64_t i) {
  const int64_t kv4 = (int64_t)a.K * a.V / 4, heads = i / kv4;
  const int h = (int)(heads % a.Hv), n = (int)(heads / a.Hv), sub = a.seg / a.parts;
  const Span sp = seq_span(a.s, n);
  const int64_t segs = segs_of(sp, a.seg), ns = segs_of(sp, sub), step = (REV ? -1 : 1) * a.Hv * kv4;
  // parts on the way, and the last that a state is written to
  const int64_t last = REV ? ns - a.parts : (segs - 1) * a.parts;
  if (segs == 1) return;
  f32x4 *at = reinterpret_cast<f32x4 *>(REV ? w.zend(a) : w.start(a)) + (first_slot(a.s, sp, n, sub) * a.Hv + h) * kv4 + i % kv4;
  if (REV) at -= (ns - 1) * step;
  const f32x4 *given = reinterpret_cast<const f32x4 *>(REV ? a.dht : a.h0);
  f32x4 cur = given ? given[i] : zero4();
  const float g2 = log2_decay(a.g[h]), whole = power(g2, sub);
  // of the first part on the way: backwards the sequence's last
  float d = REV ? power(g2, (int)(sp.end - sp.first - (ns - 1) * sub)) : whole;
  // a part is read before a state takes its place (reading on at the last one past
  // it: branches around loads make each waited for)
  f32x4 add[kAhead + 1];
  add[kAhead] = at[0];
  for (int64_t s0 = 0; s0 < last; s0 += kAhead) {
    add[0] = add[kAhead];
#pragma unroll
    for (int j = 1; j <= kAhead; ++j) add[j] = at[(s0 + j < last ? s0 + j : last) * step];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int64_t s = s0 + j + 1;  // the part that follows
      if (s > last) break;
      cur = cur * d + add[j];
      if (((REV ? ns - s : s) & (a.parts - 1)) == 0) at[s * step] = cur;
      d = whole;
    }
  }
}
__global__ __launch_bounds__(256) void carry_kernel(AttnArgs a, Layout w, int64_t blocks) {
  const int64_t b = blockIdx.x, i = b % blocks * 256 + threadIdx.x;
  if (i >= (int64_t)a.s.N * a.Hv * a.K * a.V / 4) return;
  if (b < blocks)
    carry<false>(a, w, i);
  else
    carry<true>(a, w, i);
}

// dq, dk of a q-head: the sum over its v-heads, 4 elements a thread.  (Tokens
// that no sequence has have no parts, and their rows are not the kernel's.)
template <typename E>
__global__ __launch_bounds__(256) void group_kernel(AttnArgs a, Layout w) {
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
  const f32x4 *pq = reinterpret_cast<const f32x4 *>(w.dq_part(a)) + th * R * k4 + e;
  const f32x4 *pk = reinterpret_cast<const f32x4 *>(w.dk_part(a)) + th * R * k4 + e;
  f32x4 q = zero4(), k = zero4();
  for (int r = 0; r < R; ++r) {
    q += pq[r * k4];
    k += pk[r * k4];
  }
  st4(static_cast<E *>(a.dq) + 4 * i, q[0], q[1], q[2], q[3]);
  st4(static_cast<E *>(a.dk) + 4 * i, k[0], k[1], k[2], k[3]);
}

template <int K, int V, int WHAT>
hipError_t go(const AttnArgs &a, const Layout &w, hipStream_t st) {
  const int most = WHAT == kGrads && K > V ? K : V;
  const int64_t slots = WHAT == kLocal || WHAT == kLocals ? scan::slots_of(a.s, a.seg / a.parts) : a.slots;
  const int64_t per = slots * a.Hv * (most / 32);
  const int parts = WHAT == kGrads ? 3 : WHAT == kLocals ? 2 : 1;
  KernelTimer kt(WHAT == kGrads ? "attn_grads" : WHAT == kForward ? "attn_out" : "attn_local", st);
  pass_kernel<K, V, WHAT><<<(unsigned)(per * parts), kThreads, 0, st>>>(a, w, slots, per);
  return hipGetLastError();
}
template <int WHAT>
hipError_t pick(const AttnArgs &a, const Layout &w, hipStream_t st) {
  switch (a.K * 1000 + a.V) {
    case 32032: return go<32, 32, WHAT>(a, w, st);
    case 32064: return go<32, 64, WHAT>(a, w, st);
    case 32128: return go<32, 128, WHAT>(a, w, st);
    case 64032: return go<64, 32, WHAT>(a, w, st);
    case 64064: return go<64, 64, WHAT>(a, w, st);
    case 64128: return go<64, 128, WHAT>(a, w, st);
    case 128032: return go<128, 32, WHAT>(a, w, st);
    case 128064: return go<128, 64, WHAT>(a, w, st);
    default: return go<128, 128, WHAT>(a, w, st);
  }
}
template <int WHAT>
hipError_t pass(const AttnArgs &a, const Layout &w, hipStream_t st) {
  if (a.dtype != 1) return pick<WHAT>(a, w, st);
  if (WHAT == kForward) return launch_mma_out(a, w, st);
  if (WHAT == kGrads) return launch_mma_grads(a, w, st);
  return launch_mma_local(a, w, WHAT == kLocals, st);
}

// of S, and with two ways of Z
hipError_t run_carry(const AttnArgs &a, const Layout &w, int ways, hipStream_t st) {
  const int64_t blocks = ((int64_t)a.s.N * a.Hv * a.K * a.V / 4 + 255) / 256;
  KernelTimer kt("attn_carry", st);
  carry_kernel<<<(unsigned)(ways * blocks), 256, 0, st>>>(a, w, blocks);
  return hipGetLastError();
}

// Segments of bf16 problems, and the columns that a workgroup has: what takes the
// least by a model of the passes' time in us.  A step of 64 tokens takes a
// workgroup, one a compute unit, 1.6 with 64 columns and 1.2 with 32, as long as the
// longest segment has steps or the work fills the chip; cutting sequences costs the
// launches for the states and reading k and v again.  The four numbers are of K = V
// = 128 and taken for the smaller heads too.  The work is spread evenly: whole
// rounds of workgroups are not counted, nor what long sequences leave at a round's
// end, so that a few heads more than fill the chip are modelled too short.
// (8192 tokens, 64 heads: 64 columns, one segment 185 and two 171, 32 columns one
// segment 162, two 222.  2 x 4096 tokens, 32 heads, backward: 64 columns, one
// segment 178 and two 223, 32 columns 229.  Packed, 16 sequences, 32 heads: 64
// columns 170, 32 columns 226.)  Where the device alone knows the sequences'
// lengths, the longest is taken to be four times the mean.
AttnPlan plan_mma(const AttnArgs &a, bool bwd) {
  const double cus = (double)compute_units(), steps = (double)a.s.tokens / 64, passes = bwd ? 3 : 1;
  double longest = (double)a.longest;
  if (!a.known && longest > 4. * a.s.T / a.s.N) longest = 4. * a.s.T / a.s.N;
  AttnPlan best = {};
  double least = 1e300;
  for (int cols = a.V < 64 ? 32 : 64; cols >= 32; cols /= 2) {
    const double wgs = (double)a.Hv * (a.V / cols);
    for (int64_t cuts = 1; cuts == 1 || cuts < 2 * a.longest / 64; cuts *= 2) {
      int64_t seg = (a.longest + cuts - 1) / cuts;
      const int parts = cuts > 1 && seg >= 512 ? 4 : 1;
      const int64_t unit = 64 * parts;
      seg = (seg + unit - 1) / unit * unit;
      if (seg < unit) seg = unit;
      if (seg > INT32_MAX) continue;
      const double segment = longest < (double)seg ? longest : (double)seg;
      const double full = steps * wgs * passes / cus, most = segment / 64 > full ? segment / 64 : full;
      double t = most * (cols == 64 ? 1.6 : 1.2);
      if (cuts > 1) t += 12 + (bwd ? 2 : 1) * steps * a.Hv * a.V / 64 / cus * (1. - 1. / cuts) * 1.3;
      if (t < least) {
        least = t;
        best.seg = (int)seg;
        best.parts = parts;
        best.cols = cols;
        best.one_seg = cuts == 1;
      }
    }
  }
  return best;
}
// fp32: segments as long as the whole batch unless that leaves compute units
// without two workgroups each.  The outputs' pass sums up the segments before its
// own where they are few, and no carry is launched; backwards three passes do so
// with less work beside it, and lose sooner.  (8 heads, K = V = 64, joined and
// with a carry, us a call: forward of 16 segments 19 and 22, of 32 23 and 27; backward
// of 8 segments 25 and 28, of 32 54 and 43.  K = V = 128: forward of 8 segments 20
// and 24, of 16 28 and 32; backward of 8 39 and 40, of 16 75 and 67.)
AttnPlan plan_f32(const AttnArgs &a, bool bwd) {
  const int64_t per = (int64_t)a.Hv * (a.V / 32);  // workgroups a segment
  const int64_t want = (compute_units() * 2 + per - 1) / per;
  int64_t seg = ((a.s.tokens + want - 1) / want + 63) / 64 * 64;
  AttnPlan p;
  p.seg = seg < 64 ? 64 : seg > INT32_MAX - 63 ? INT32_MAX / 64 * 64 : (int)seg;
  p.parts = 1;
  p.cols = 32;
  p.one_seg = a.longest <= p.seg;
  p.joined = a.longest <= (int64_t)(bwd ? 8 : 32) * p.seg;
  return p;
}

}  // namespace
}  // namespace attn

AttnPlan attn_plan(const AttnArgs &a0, bool bwd) {
  AttnArgs a = a0;
  AttnPlan p = a.dtype == 1 ? attn::plan_mma(a, bwd) : attn::plan_f32(a, bwd);
  a.seg = p.seg;
  a.parts = p.parts;
  a.slots = p.slots = scan::slots_of(a.s, p.seg);
  a.one_seg = p.one_seg;
  a.joined = p.joined;
  p.ws = attn::layout(a, bwd).total;
  return p;
}

hipError_t launch_attn_fwd(const AttnArgs &a, hipStream_t st) {
  using namespace attn;
  const Layout w = layout(a, false);
  if (!a.one_seg) {
    hipError_t e = pass<kLocal>(a, w, st);
    if (e != hipSuccess) return e;
    if (!a.joined && (e = run_carry(a, w, 1, st)) != hipSuccess) return e;
  }
  return pass<kForward>(a, w, st);
}

hipError_t launch_attn_bwd(const AttnArgs &a, hipStream_t st) {
  using namespace attn;
  const Layout w = layout(a, true);
  hipError_t e;
  if (!a.one_seg) {
    if ((e = pass<kLocals>(a, w, st)) != hipSuccess) return e;
    if (!a.joined && (e = run_carry(a, w, 2, st)) != hipSuccess) return e;
  }
  if ((e = pass<kGrads>(a, w, st)) != hipSuccess) return e;
  if (a.Hv == a.Hq || a.s.tokens == 0) return hipSuccess;
  KernelTimer kt("attn_group", st);
  const unsigned blocks = (unsigned)((a.s.tokens * a.Hq * (a.K / 4) + 255) / 256);
  if (a.dtype == 1)
    group_kernel<bf16><<<blocks, 256, 0, st>>>(a, w);
  else
    group_kernel<float><<<blocks, 256, 0, st>>>(a, w);
  return hipGetLastError();
}

}  // namespace gdn
