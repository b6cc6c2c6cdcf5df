// The short causal convolution over a sequence's channels (depthwise, W taps):
//
//   pre_t = bias + sum_j w[:, j] x_{t - (W - 1) + j},   y_t = act(pre_t)
//
// over packed or padded-free batches, with the last W - 1 inputs as the state
// that goes in and comes out; its backward, and its form for single tokens.
// All of it moves data far longer than it computes: x and y once (the
// backward: x, dy and dx), so each kernel is one pass with the window in
// registers.  16384 tokens x 8192 channels in bf16 forward: 108 us, 5.0 TB/s
// (a large copy here: 5.4); 2 x 4096 x 8192 backward with the sums: 106 to 114
// us a call by what ran before it (114 to 119 + 5 in kernel traces), 3.3 to 3.8 TB/s
// (three streams, half the waves by registers).  A token's step is a launch: 9 us
// a call at 32 x 8192.
#include <initializer_list>

#include "gdn_internal.h"
#include "gdn_mixer.hpp"

namespace gdn {
namespace {

constexpr int kThreads = 256;

// silu(z) and its derivative s (1 + z (1 - s)), s = sigmoid(z)
__device__ __forceinline__ float silu(float z) { return z * sigmoidf(z); }
__device__ __forceinline__ float dsilu(float z) {
  const float s = sigmoidf(z);
  return s * (1.f + z * (1.f - s));
}

// Row `t` of the inputs of sequence n as the convolution sees it: a token, or
// a row of the incoming state, or zeros.
template <typename E, int VEC>
__device__ __forceinline__ void load_row(Vec<E, VEC> &r, const ConvArgs &a, const Span &sp, int n,
                                         int64_t t, int c0) {
  if (t >= sp.first)
    r.load(static_cast<const E *>(a.x) + t * a.xs + c0);
  else if (a.h0)
    r.load(static_cast<const E *>(a.h0) +
           ((int64_t)n * (a.W - 1) + (a.W - 1) + (t - sp.first)) * a.D + c0);
  else
    r.zero();
}

template <typename E, int VEC, int W>
struct Taps {
  float w[W][VEC], b[VEC];
  __device__ __forceinline__ Taps(const ConvArgs &a, int c0) { load_taps(w, b, a.w, a.bias, c0, a.wdtype); }
};

// A workgroup is `subs` token tiles of `tt` tokens times 256 / subs groups of
// VEC channels (a wave reads 1 KB of one token, or 512 B of two).  Workgroups
// past the tiles write the outgoing state, one sequence each.
struct Geo {
  int cg_bits;    // log2 of channel groups per workgroup
  int tt;         // tokens per thread
  int64_t tiles;  // workgroups along the tokens
  int cblocks;    // workgroups along the channels
};

template <typename E, int VEC, int W>
__global__ __launch_bounds__(kThreads) void conv_fwd_kernel(ConvArgs a, Geo g) {
  const int cgs = 1 << g.cg_bits, subs = kThreads >> g.cg_bits;
  const int64_t tile = blockIdx.x / g.cblocks;
  const int c0 = ((int)(blockIdx.x % g.cblocks) * cgs + (threadIdx.x & (cgs - 1))) * VEC;
  if (c0 >= a.D) return;
  const int sub = threadIdx.x >> g.cg_bits;
  if (tile >= g.tiles) {
    if (sub) return;
    const int n = (int)(tile - g.tiles);
    const Span sp = seq_span(a.s, n);
#pragma unroll
    for (int i = 0; i < W - 1; ++i) {
      Vec<E, VEC> r;
      load_row<E, VEC>(r, a, sp, n, sp.end - (W - 1) + i, c0);
      r.store(static_cast<E *>(a.ht) + ((int64_t)n * (W - 1) + i) * a.D + c0);
    }
    return;
  }
  const int64_t t0 = (tile * subs + sub) * g.tt;
  const int64_t t1 = t0 + g.tt < a.s.tokens ? t0 + g.tt : a.s.tokens;
  if (t0 >= t1) return;
  const Taps<E, VEC, W> tp(a, c0);
  const E *x = static_cast<const E *>(a.x) + c0;
  E *y = static_cast<E *>(a.y) + c0;
  int64_t at = t0;
  for (int n = seq_of(a.s, t0); n < a.s.N && at < t1; ++n) {
    const Span sp = seq_span(a.s, n);
    if (sp.end <= at) continue;
    at = at > sp.first ? at : sp.first;
    const int64_t b = t1 < sp.end ? t1 : sp.end;
    if (at >= b) continue;
    Vec<E, VEC> win[W - 1];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) load_row<E, VEC>(win[j], a, sp, n, at - (W - 1) + j, c0);
    constexpr int U = 4;  // rows in flight per thread, while as many are worked on
    Raw<E, VEC> next[U];
    auto fetch = [&](int64_t t) {
#pragma unroll
      for (int u = 0; u < U; ++u) next[u].load(x + (t + u < b ? t + u : b - 1) * a.xs);
    };
    fetch(at);
    for (int64_t t = at; t < b; t += U) {
      Raw<E, VEC> raw[U];
#pragma unroll
      for (int u = 0; u < U; ++u) raw[u] = next[u];
      if (t + U < b) fetch(t + U);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const Vec<E, VEC> cur = raw[u].f();
        Vec<E, VEC> out;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          float p = tp.b[i];
#pragma unroll
          for (int j = 0; j < W - 1; ++j) p += tp.w[j][i] * win[j].v[i];
          p += tp.w[W - 1][i] * cur.v[i];
          out.v[i] = a.silu ? silu(p) : p;
        }
        if (t + u < b) out.store(y + (t + u) * a.D);
#pragma unroll
        for (int j = 0; j + 1 < W - 1; ++j) win[j] = win[j + 1];
        win[W - 2] = cur;
      }
    }
    at = b;
  }
}

// Backward in one walk up the tokens: with d_t = dy_t act'(pre_t), token t
// adds w_j d_t to dx_{t - (W - 1) + j}, so W - 1 unfinished rows of dx travel
// along in registers; a tile runs W - 1 tokens past its end for the rows it
// owns.  dw_j = sum_t d_t x_{t - (W - 1) + j} and dbias stay in registers,
// are added over a workgroup's token tiles in LDS and leave as one partial
// per workgroup (no atomics: the result does not depend on the order).
template <typename E, int VEC, int W>
__global__ __launch_bounds__(kThreads) void conv_bwd_kernel(ConvArgs a, Geo g) {
  const int cgs = 1 << g.cg_bits, subs = kThreads >> g.cg_bits;
  const int64_t tile = blockIdx.x / g.cblocks;
  const int cg = threadIdx.x & (cgs - 1);
  const int c0 = ((int)(blockIdx.x % g.cblocks) * cgs + cg) * VEC;
  const int sub = threadIdx.x >> g.cg_bits;
  const bool live = c0 < a.D;
  const E *x = static_cast<const E *>(a.x) + c0;
  const E *dy = static_cast<const E *>(a.dy) + c0;
  if (tile >= g.tiles) {  // the gradient of one sequence's incoming state
    if (sub || !live) return;
    const Taps<E, VEC, W> tp(a, c0);
    const int n = (int)(tile - g.tiles);
    const Span sp = seq_span(a.s, n);
    const int64_t len = sp.end - sp.first;
    Vec<E, VEC> win[2 * W - 2], dh[W - 1];
#pragma unroll
    for (int j = 0; j < 2 * W - 2; ++j) {
      win[j].zero();
      if (j < W - 1 + len) load_row<E, VEC>(win[j], a, sp, n, sp.first - (W - 1) + j, c0);
    }
#pragma unroll
    for (int i = 0; i < W - 1; ++i) {
      dh[i].zero();
      if (a.dht && i >= len)
        dh[i].load(static_cast<const E *>(a.dht) + ((int64_t)n * (W - 1) + (i - len)) * a.D + c0);
    }
#pragma unroll
    for (int u = 0; u < W - 1; ++u) {  // token first + u
      if (u >= len) break;
      Vec<E, VEC> d;
      d.load(dy + (sp.first + u) * (int64_t)a.D);
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        if (a.silu) {
          float p = tp.b[i];
#pragma unroll
          for (int j = 0; j < W; ++j) p += tp.w[j][i] * win[u + j].v[i];
          d.v[i] *= dsilu(p);
        }
#pragma unroll
        for (int j = 0; j + u < W - 1; ++j) dh[u + j].v[i] += tp.w[j][i] * d.v[i];
      }
    }
#pragma unroll
    for (int i = 0; i < W - 1; ++i)
      dh[i].store(static_cast<E *>(a.dh0) + ((int64_t)n * (W - 1) + i) * a.D + c0);
    return;
  }
  float dw[W][VEC], db[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    db[i] = 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) dw[j][i] = 0.f;
  }
  const int64_t t0 = (tile * subs + sub) * g.tt;
  const int64_t t1 = t0 + g.tt < a.s.tokens ? t0 + g.tt : a.s.tokens;
  if (live && t0 < t1) {
    const Taps<E, VEC, W> tp(a, c0);
    E *dx = static_cast<E *>(a.dx) + c0;
    int64_t at = t0;
    for (int n = seq_of(a.s, t0); n < a.s.N && at < t1; ++n) {
      const Span sp = seq_span(a.s, n);
      if (sp.end <= at) continue;
      at = at > sp.first ? at : sp.first;
      const int64_t b = t1 < sp.end ? t1 : sp.end;
      if (at >= b) continue;
      const int64_t stop = b + (W - 1) < sp.end ? b + (W - 1) : sp.end;
      Vec<E, VEC> win[W - 1];
      float acc[W - 1][VEC];
#pragma unroll
      for (int j = 0; j < W - 1; ++j) {
        load_row<E, VEC>(win[j], a, sp, n, at - (W - 1) + j, c0);
#pragma unroll
        for (int i = 0; i < VEC; ++i) acc[j][i] = 0.f;
      }
      constexpr int U = 4;
      Raw<E, VEC> nx[U], nd[U];
      auto fetch = [&](int64_t t) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int64_t tu = t + u < stop ? t + u : stop - 1;
          nx[u].load(x + tu * a.xs);
          nd[u].load(dy + tu * (int64_t)a.D);
        }
      };
      fetch(at);
      for (int64_t t = at; t < stop; t += U) {
        Raw<E, VEC> rx[U], rd[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          rx[u] = nx[u];
          rd[u] = nd[u];
        }
        if (t + U < stop) fetch(t + U);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (t + u >= stop) break;
          const Vec<E, VEC> cur = rx[u].f();
          Vec<E, VEC> d = rd[u].f(), out;
          const bool mine = t + u < b;
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            if (a.silu) {
              float p = tp.b[i];
#pragma unroll
              for (int j = 0; j < W - 1; ++j) p += tp.w[j][i] * win[j].v[i];
              p += tp.w[W - 1][i] * cur.v[i];
              d.v[i] *= dsilu(p);
            }
            const float dm = mine ? d.v[i] : 0.f;
            db[i] += dm;
#pragma unroll
            for (int j = 0; j < W - 1; ++j) dw[j][i] += dm * win[j].v[i];
            dw[W - 1][i] += dm * cur.v[i];
            out.v[i] = acc[0][i] + tp.w[0][i] * d.v[i];
#pragma unroll
            for (int j = 0; j + 1 < W - 1; ++j) acc[j][i] = acc[j + 1][i] + tp.w[j + 1][i] * d.v[i];
            acc[W - 2][i] = tp.w[W - 1][i] * d.v[i];
          }
          // (W = 2: the row before t is finished by tap 0, the row t begun by tap 1)
          if (t + u - (W - 1) >= at) out.store(dx + (t + u - (W - 1)) * (int64_t)a.D);
#pragma unroll
          for (int j = 0; j + 1 < W - 1; ++j) win[j] = win[j + 1];
          win[W - 2] = cur;
        }
      }
      if (stop == sp.end) {  // the rows that no later token of the sequence reaches
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
          const int64_t t = stop - (W - 1) + j;
          if (t < at || t >= b) continue;
          Vec<E, VEC> out;
          out.zero();
          if (a.dht) out.load(static_cast<const E *>(a.dht) + ((int64_t)n * (W - 1) + j) * a.D + c0);
#pragma unroll
          for (int i = 0; i < VEC; ++i) out.v[i] += acc[j][i];
          out.store(dx + t * (int64_t)a.D);
        }
      }
      at = b;
    }
  }
  __shared__ float red[kThreads * VEC];
  for (int j = 0; j <= W; ++j) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      float v = db[i];
#pragma unroll
      for (int k = 0; k < W; ++k) v = j == k ? dw[k][i] : v;
      red[i * kThreads + threadIdx.x] = v;
    }
    __syncthreads();
    if (sub == 0 && live) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        float v = 0.f;
        for (int s = 0; s < subs; ++s) v += red[i * kThreads + s * cgs + cg];
        a.partial[(tile * (W + 1) + j) * a.D + c0 + i] = v;
      }
    }
  }
}

// dw, dbias: the partials of all workgroups, added in order.
__global__ __launch_bounds__(kSumThreads) void conv_sum_kernel(ConvArgs a, int64_t tiles) {
  sum_parts(a.partial, tiles, (int64_t)(a.W + 1) * a.D, [&](int64_t i, float v) {
    const int j = (int)(i / a.D);
    const int64_t c = i % a.D;
    if (j < a.W)
      store_w(a.dw, c * a.W + j, v, a.wdtype);
    else if (a.db)
      store_w(a.db, c, v, a.wdtype);
  });
}

// One token: y from the state's rows and x, the state moved on by one row.
// A workgroup has one batch row and blockDim.x groups of VEC channels.
template <typename E, int VEC, int W>
__global__ void conv_step_kernel(ConvStepArgs a, int cblocks) {
  const int64_t row = blockIdx.x / cblocks;
  const int c0 = ((int)(blockIdx.x % cblocks) * (int)blockDim.x + (int)threadIdx.x) * VEC;
  int64_t slot = row;
  bool live = true;
  if (a.index) {
    slot = a.index[row];
    live = slot >= 0 && slot < a.slots;
    // a slot named twice belongs to the first row that names it
    int twice = 0;
    for (int64_t j = threadIdx.x; j < row; j += blockDim.x) twice |= a.index[j] == slot;
    live = !__syncthreads_or(twice) && live;
  }
  if (c0 >= a.D) return;
  E *y = static_cast<E *>(a.y) + row * a.D + c0;
  if (!live) {
    Vec<E, VEC> z;
    z.zero();
    z.store(y);
    return;
  }
  E *st = static_cast<E *>(a.state) + slot * (W - 1) * a.D + c0;
  Vec<E, VEC> win[W], out;
  float w[W][VEC], b[VEC];
  load_taps(w, b, a.w, a.bias, c0, a.wdtype);
#pragma unroll
  for (int j = 0; j < W - 1; ++j) win[j].load(st + (int64_t)j * a.D);
  win[W - 1].load(static_cast<const E *>(a.x) + row * a.xs + c0);
#pragma unroll
  for (int k = 0; k < VEC; ++k) {
    float p = b[k];
#pragma unroll
    for (int j = 0; j < W; ++j) p += w[j][k] * win[j].v[k];
    out.v[k] = a.silu ? silu(p) : p;
  }
  out.store(y);
#pragma unroll
  for (int j = 0; j < W - 1; ++j) win[j + 1].store(st + (int64_t)j * a.D);
}

int log2_up(int64_t x) {
  int b = 0;
  while (((int64_t)1 << b) < x) ++b;
  return b;
}

bool rows16(const void *p) { return ((uintptr_t)p & 15) == 0; }

Geo conv_geo(const ConvArgs &a, int vec, bool bwd) {
  Geo g;
  const int64_t groups = (a.D + vec - 1) / vec;
  if (bwd) {
    g.cg_bits = log2_up(groups) < 5 ? log2_up(groups) : 5;
    g.tiles = conv_bwd_tiles(a.s.tokens, a.D);
    const int64_t per = g.tiles ? (a.s.tokens + g.tiles - 1) / g.tiles : 1;
    const int subs = kThreads >> g.cg_bits;
    g.tt = (int)((per + subs - 1) / subs);
    if (g.tt < 1) g.tt = 1;
  } else {
    g.cg_bits = log2_up(groups) < 8 ? log2_up(groups) : 8;
    const int subs = kThreads >> g.cg_bits;
    // enough threads for 16 waves a compute unit before a thread takes more tokens
    int64_t tt = groups * a.s.tokens / (compute_units() * 1024);
    g.tt = tt < 8 ? 8 : tt > 64 ? 64 : (int)(tt & ~(int64_t)7);
    g.tiles = (a.s.tokens + (int64_t)g.tt * subs - 1) / ((int64_t)g.tt * subs);
  }
  g.cblocks = (int)((groups + (1 << g.cg_bits) - 1) >> g.cg_bits);
  return g;
}

template <template <typename, int, int> class F, int VB, typename... A>
hipError_t dispatch(int dtype, bool vec, int W, A &&...args) {
#define GDN_W(E, VEC)                                   \
  switch (W) {                                          \
    case 2: return F<E, VEC, 2>::go(args...);           \
    case 3: return F<E, VEC, 3>::go(args...);           \
    default: return F<E, VEC, 4>::go(args...);          \
  }
  if (dtype == 1) {
    if (vec) { GDN_W(bf16, VB) }
    GDN_W(bf16, 1)
  }
  if (vec) { GDN_W(float, 4) }
  GDN_W(float, 1)
#undef GDN_W
}

template <typename E, int VEC, int W>
struct GoFwd {
  static hipError_t go(const ConvArgs &a, hipStream_t st) {
    const Geo g = conv_geo(a, VEC, false);
    const int64_t blocks = (g.tiles + (a.ht ? a.s.N : 0)) * g.cblocks;
    if (blocks) {
      KernelTimer kt("conv_fwd", st);
      conv_fwd_kernel<E, VEC, W><<<(unsigned)blocks, kThreads, 0, st>>>(a, g);
    }
    return hipGetLastError();
  }
};
template <typename E, int VEC, int W>
struct GoBwd {
  static hipError_t go(const ConvArgs &a, hipStream_t st) {
    const Geo g = conv_geo(a, VEC, true);
    const int64_t blocks = (g.tiles + (a.dh0 ? a.s.N : 0)) * g.cblocks;
    if (blocks) {
      KernelTimer kt("conv_bwd", st);
      conv_bwd_kernel<E, VEC, W><<<(unsigned)blocks, kThreads, 0, st>>>(a, g);
    }
    KernelTimer kt("conv_bwd_sum", st);
    const int64_t n = (int64_t)(W + 1) * a.D;
    conv_sum_kernel<<<sum_blocks(n), kSumThreads, 0, st>>>(a, g.tiles);
    return hipGetLastError();
  }
};
template <typename E, int VEC, int W>
struct GoStep {
  static hipError_t go(const ConvStepArgs &a, hipStream_t st) {
    const int cgs = (a.D + VEC - 1) / VEC;
    const int threads = cgs <= 64 ? 64 : 128;
    const int cblocks = (cgs + threads - 1) / threads;
    KernelTimer kt("conv_step", st);
    conv_step_kernel<E, VEC, W><<<(unsigned)((int64_t)a.B * cblocks), threads, 0, st>>>(a, cblocks);
    return hipGetLastError();
  }
};

}  // namespace

// Tokens of one workgroup of the backward: as many as leave four workgroups a
// compute unit (their partials are written and read again), 32 to 512.
int64_t conv_bwd_tiles(int64_t tokens, int D) {
  int64_t per = tokens * D / (compute_units() * 1024);
  per = per < 32 ? 32 : per > 512 ? 512 : per;
  return (tokens + per - 1) / per;
}

// Whole sequences: four channels a thread (8 bytes in bf16).  Eight, 16 bytes,
// leave 3 waves a SIMD (backward: 1) and are 6 % slower in both directions at
// 16384 x 8192 (2 x 4096 x 8192), both timed in turn.
static bool wide4(const ConvArgs &a, std::initializer_list<const void *> rows) {
  const uintptr_t mask = a.dtype == 1 ? 7 : 15;
  for (const void *p : rows)
    if ((uintptr_t)p & mask) return false;
  return a.D % 4 == 0 && a.xs % 4 == 0 && rows16(a.w) && rows16(a.bias);
}
hipError_t launch_conv_fwd(const ConvArgs &a, hipStream_t st) {
  return dispatch<GoFwd, 4>(a.dtype, wide4(a, {a.x, a.y, a.h0, a.ht}), a.W, a, st);
}
hipError_t launch_conv_bwd(const ConvArgs &a, hipStream_t st) {
  return dispatch<GoBwd, 4>(a.dtype, wide4(a, {a.x, a.dy, a.h0, a.dht, a.dx, a.dh0}), a.W, a, st);
}
hipError_t launch_conv_step(const ConvStepArgs &a, hipStream_t st) {
  const int vec = a.dtype == 1 ? 8 : 4;
  const bool wide = a.D % vec == 0 && a.xs % vec == 0 && rows16(a.x) && rows16(a.y) && rows16(a.state) &&
                    rows16(a.w) && rows16(a.bias);
  return dispatch<GoStep, 8>(a.dtype, wide, a.W, a, st);
}

}  // namespace gdn
