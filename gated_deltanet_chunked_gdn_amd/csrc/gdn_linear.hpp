// Linear attention with a decay for each head: the passes that its forward and
// backward are made of, their workspace, and what their kernels share.
//
// With l = exp(log decay) and s the scale,
//
//   S_t = l S_{t-1} + k_t v_t^T,   o_t = s S_t^T q_t
//
// so that o_i = s (sum_{j <= i} l^{i-j} (q_i . k_j) v_j + l^{i+1} S_0^T q_i),
// counted from the tokens of a chunk and the state before it.  The gradients
// have the same form with the operands in other places; with Z_j the gradient
// of S_j by the tokens behind j, Z_{t-1} = l (Z_t + s q_t do_t^T):
//
//   pass   out_i    a    b    c    state (a x c)   tokens
//   o      o        q    k    v    S               forwards
//   dq     dq       do   v    k    S^T             forwards
//   dk     dk       v    do   q    Z^T             backwards
//   dv     dv       k    q    do   Z               backwards
//
// Each pass takes sum (a_i . b_j) l^{|i-j|} c_j over the tokens j on its side of
// i (i among them) and the state times a_i.
#pragma once

#include "gdn_scan.hpp"

namespace gdn {
namespace attn {

using scan::first_slot;
using scan::locate;
using scan::segs_of;
using scan::SlotLoc;

struct Layout {
  size_t o_start = 0, o_zend = 0, o_dq = 0, o_dk = 0, total = 0;
  __host__ __device__ float *at(const AttnArgs &a, size_t o) const { return reinterpret_cast<float *>(a.ws + o); }
  // fp32 [sub slots][Hv][K][V], a sub slot a part of a segment: what it adds to
  // the state; then, in a segment's first but not a sequence's, the state that the
  // segment begins with
  __host__ __device__ float *start(const AttnArgs &a) const { return at(a, o_start); }
  // the same of Z; then, in a segment's last part but not a sequence's, Z behind it
  __host__ __device__ float *zend(const AttnArgs &a) const { return at(a, o_zend); }
  // fp32 [tokens][Hv][K] each: the v-heads' parts of dq and dk where they share heads
  __host__ __device__ float *dq_part(const AttnArgs &a) const { return at(a, o_dq); }
  __host__ __device__ float *dk_part(const AttnArgs &a) const { return at(a, o_dk); }
};

inline Layout layout(const AttnArgs &a, bool bwd) {
  Layout w;
  size_t off = 0;
  auto piece = [&](size_t bytes) {
    const size_t o = off;
    off = (off + bytes + 255) & ~(size_t)255;
    return o;
  };
  const size_t states = a.one_seg ? 0 : (size_t)scan::slots_of(a.s, a.seg / a.parts) * a.Hv * a.K * a.V * 4;
  if (!a.one_seg) {
    w.o_start = piece(states);
    if (bwd) w.o_zend = piece(states);
  }
  if (bwd && a.Hv != a.Hq) {
    const size_t part = (size_t)a.s.tokens * a.Hv * a.K * 4;
    w.o_dq = piece(part);
    w.o_dk = piece(part);
  }
  w.total = off ? off : 256;
  return w;
}

// l^n as 2^(g2 n), g2 = log2 of the decay.  (A decay of 0 is as good as one of
// e^-10000, whose powers but the 0th are 0; -inf would give NaN there, as inf would.)
__device__ __forceinline__ float log2_decay(float g) { return (g < -1e4f ? -1e4f : g > 1e4f ? 1e4f : g) * 1.44269504088896340736f; }
// x within +-`most`, NaN as it is.  No factor is infinite: chunks are multiplied
// out whole, and what is 0 there (rows behind a sequence's end, tokens of zeros, a
// state that has not begun) stays 0 under any power of a decay that grows.
__device__ __forceinline__ float finite(float x, float most = __FLT_MAX__) { return x > most ? most : x < -most ? -most : x; }
__device__ __forceinline__ float power(float g2, int n) { return finite(__builtin_amdgcn_exp2f(g2 * (float)n)); }

enum PassKind { kO, kDq, kDk, kDv };

// Whether a part of a segment goes into the carry: of S those before a sequence's
// last segment, of Z those behind its first.
__device__ __forceinline__ bool carried(const AttnArgs &a, const SlotLoc &sub, bool rev) {
  if (rev) return sub.index >= a.parts;
  const Span sp = seq_span(a.s, sub.n);
  return sub.index < (segs_of(sp, a.seg) - 1) * a.parts;
}

// One pass, for one v-head and segment.
struct Pass {
  const void *a, *b, *c;      // at the head's first element of token 0
  int64_t as, bs, cs;         // elements from one token to the next
  void *out;                  // likewise
  int64_t os;
  bool part;                  // out is fp32, a v-head's part
  bool rev;                   // tokens backwards
  bool tr;                    // the state is stored [c][a]
  float scale_p, scale_in, scale_up;  // of the pairs, the state's share and its update
  const float *start;         // the state to begin with, or null: 0
  float *last;                // where the sequence's last state goes, or null
  // without a carry: what the segments before this one add, `before` of them from
  // `added` on in steps of `step`, the first of `nt0` tokens
  const float *added;
  int64_t step;
  int before, nt0;
};

template <typename E>
__device__ __forceinline__ Pass make_pass(const AttnArgs &a, const Layout &w, int kind, const SlotLoc &loc, int h) {
  const int hq = h / (a.Hv / a.Hq);
  const int64_t kv = (int64_t)a.K * a.V, os = (int64_t)a.Hv * a.V;
  const E *q = static_cast<const E *>(a.q) + (int64_t)hq * a.K, *k = static_cast<const E *>(a.k) + (int64_t)hq * a.K;
  const E *v = static_cast<const E *>(a.v) + (int64_t)h * a.V, *dO = static_cast<const E *>(a.dO) + (int64_t)h * a.V;
  const int64_t state = (loc.n * (int64_t)a.Hv + h) * kv;
  Pass p;
  p.part = a.Hv != a.Hq;
  p.rev = kind == kDk || kind == kDv;
  p.tr = kind == kDq || kind == kDk;
  p.scale_p = a.scale;
  p.scale_in = p.rev ? 1.f : a.scale;
  p.scale_up = p.rev ? a.scale : 1.f;
  const float *given = p.rev ? a.dht : a.h0;
  // (where the sequence begins, what the call gives; the carry writes the others'.
  // With one segment there is none, whatever the device's lengths say.)
  p.before = 0;
  if (a.one_seg || (p.rev ? loc.last : loc.index == 0)) {
    p.start = given ? given + state : nullptr;
  } else if (a.joined) {
    const Span sp = seq_span(a.s, loc.n);
    const int64_t ns = segs_of(sp, a.seg), first = first_slot(a.s, sp, loc.n, a.seg) + (p.rev ? ns - 1 : 0);
    p.start = given ? given + state : nullptr;
    p.added = (p.rev ? w.zend(a) : w.start(a)) + (first * a.Hv + h) * kv;
    p.step = (p.rev ? -1 : 1) * a.Hv * kv;
    p.before = (int)(p.rev ? ns - 1 - loc.index : loc.index);
    p.nt0 = p.rev ? (int)(sp.end - sp.first - (ns - 1) * a.seg) : a.seg;
  } else {
    const int sub = a.seg / a.parts;
    const int64_t at = first_slot(a.s, seq_span(a.s, loc.n), loc.n, sub) + (p.rev ? (loc.index + 1) * a.parts - 1 : loc.index * a.parts);
    p.start = (p.rev ? w.zend(a) : w.start(a)) + (at * a.Hv + h) * kv;
  }
  p.last = nullptr;
  // a v-head's part of a q-head's gradient, or the gradient itself
  auto shared = [&](void *d, float *parts) {
    p.out = p.part ? static_cast<void *>(parts + (int64_t)h * a.K) : static_cast<void *>(static_cast<E *>(d) + (int64_t)hq * a.K);
    p.os = p.part ? (int64_t)a.Hv * a.K : (int64_t)a.Hq * a.K;
  };
  auto own = [&](void *d) {
    p.part = false;
    p.out = static_cast<E *>(d) + (int64_t)h * a.V;
    p.os = os;
  };
  switch (kind) {
    case kO:
      p.a = q, p.as = a.qs, p.b = k, p.bs = a.ks, p.c = v, p.cs = a.vs;
      own(a.o);
      if (a.ht && loc.last) p.last = a.ht + state;
      break;
    case kDq:
      p.a = dO, p.as = os, p.b = v, p.bs = a.vs, p.c = k, p.cs = a.ks;
      shared(a.dq, w.dq_part(a));
      break;
    case kDk:
      p.a = v, p.as = a.vs, p.b = dO, p.bs = os, p.c = q, p.cs = a.qs;
      shared(a.dk, w.dk_part(a));
      break;
    default:
      p.a = k, p.as = a.ks, p.b = q, p.bs = a.qs, p.c = dO, p.cs = os;
      own(a.dv);
      if (a.dh0 && loc.index == 0) p.last = a.dh0 + state;
  }
  return p;
}

// bf16, gdn_linear_mma.hip
hipError_t launch_mma_local(const AttnArgs &a, const Layout &w, bool both, hipStream_t st);
hipError_t launch_mma_out(const AttnArgs &a, const Layout &w, hipStream_t st);
hipError_t launch_mma_grads(const AttnArgs &a, const Layout &w, hipStream_t st);

}  // namespace attn
}  // namespace gdn
