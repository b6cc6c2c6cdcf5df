// Group norm of channels-last tensors [N][S][C], C = G Dg, with an activation
// or an output gate, and its backward:
//
//   xh = (x - mean) rstd,  z = xh w + b,  y = z, silu(z) or z silu(gate)
//
// mean and rstd over the S Dg values of a sample's group.  With dz the gradient
// of z and t = dz w:
//
//   dx = rstd (t - mean(t) - xh mean(t xh))
//   dw = sum dz xh,  db = sum dz  over samples and positions
//
// Memory decides.  Where a workgroup's registers hold a group (S Dg values)
// it is read once: the lanes that share it take the mean, then the variance of
// the centred values, then write.  Larger ones take two passes over the tensor
// by rows of all channels, a thread its own channels: sums of each channel over
// a block of rows, joined by group in 64 bits, and the outputs.  The variance's
// sums are of eight rows at a time, about the first of them: sum d^2 is at most 9
// times their squares about their mean, wherever that lies; eights are joined by
// their means (which are taken from the thread's first value of the channel, so
// that a mean far from zero costs them no bits).
//
// Measured (a large copy: 5.1 TB/s; kernels in a trace, calls that follow each
// other).  Held, 8192 tokens, 64 heads of 128, bf16 with a gate: forward 81 us, 5.0
// TB/s; backward 135 and 5 for dw and db, the call 140, 4.8 TB/s.  By rows, bf16 with
// SiLU: 8 maps of 9216 x 320, 32 groups, sums 13, join 4, outputs 17, the call 32;
// backward of 6 maps of 4096 x 512 14 + 6 + 15, the call 33.  The second reading
// comes from the last-level cache; the launch between the two large ones is as long
// as small launches are.  Which groups are held goes by what registers hold; with
// several positions of few channels the rows' form was not measured against it.
#include "gdn_internal.h"
#include "gdn_mixer.hpp"

namespace gdn {
namespace group {
namespace {

constexpr int kHeld = 8192;  // values of a group that a workgroup holds: 8 a lane

// Sum over the TPG lanes of a group, the same value in each (gdn_norm.hip).
template <int TPG>
__device__ __forceinline__ void sum2(float &u, float &v, float *red) {
  u = group_sum<(TPG < 16 ? TPG : 16)>(u);
  v = group_sum<(TPG < 16 ? TPG : 16)>(v);
  if constexpr (TPG >= 64) {
    u += __shfl_xor(u, 16), v += __shfl_xor(v, 16);
    u += __shfl_xor(u, 32), v += __shfl_xor(v, 32);
  }
  if constexpr (TPG > 64) {
    const int w = threadIdx.x >> 6;
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[2 * w] = u, red[2 * w + 1] = v;
    __syncthreads();
    u = v = 0.f;
#pragma unroll
    for (int i = 0; i < TPG / 64; ++i) u += red[2 * i], v += red[2 * i + 1];
  }
}
template <int TPG>
__device__ __forceinline__ float sum1(float u, float *red) {
  float v = 0.f;
  sum2<TPG>(u, v, red);
  return u;
}

__device__ __forceinline__ float activate(float z, bool silu, bool gated, float gate) {
  return silu ? z * sigmoidf(z) : gated ? z * (gate * sigmoidf(gate)) : z;
}
// The gradients of z and of the gate.
__device__ __forceinline__ float back(float dy, float z, bool silu, bool gated, float gate, float &dgate) {
  if (silu) {
    const float s = sigmoidf(z);
    return dy * (s * (1.f + z * (1.f - s)));
  }
  if (!gated) return dy;
  const float s = sigmoidf(gate);
  dgate = dy * z * (s * (1.f + gate * (1.f - s)));
  return dy * (gate * s);
}

// ---- groups held in registers

// The lanes of a group and where their values lie: piece v of a lane has VEC
// channels of one position.
template <int VEC, int TPG, int NV>
struct Held {
  static constexpr int T = TPG > 256 ? TPG : 256, RPB = T / TPG;
  int lane, sub, g;
  int64_t row, rows;  // of this lane group's first sample, and from one to the next
  int off[NV], col[NV];
  bool in[NV];
  __device__ __forceinline__ Held(const GroupArgs &a) {
    lane = threadIdx.x % TPG;
    sub = threadIdx.x / TPG;
    // (the grid's lane groups are a multiple of G: each keeps its channels)
    const int64_t first = (int64_t)blockIdx.x * RPB + sub;
    g = (int)(first % a.G);
    row = first / a.G;
    rows = (int64_t)gridDim.x * RPB / a.G;
    const int pd = a.Dg / VEC, C = a.G * a.Dg;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int p = v * TPG + lane, s = p / pd;
      in[v] = s < a.S;
      col[v] = g * a.Dg + (p - s * pd) * VEC;
      off[v] = s * C + col[v];
    }
  }
};

template <typename E, int VEC, int TPG, int NV>
__global__ __launch_bounds__(TPG > 256 ? TPG : 256) void fwd_kernel(GroupArgs a) {
  __shared__ float red[32];
  const Held<VEC, TPG, NV> at(a);
  const int64_t sample = a.S * a.G * a.Dg;
  const float inv = 1.f / ((float)a.S * (float)a.Dg);
  const E *x = static_cast<const E *>(a.x), *gate = static_cast<const E *>(a.gate);
  float w[NV][VEC], b[NV][VEC];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    if (!at.in[v]) continue;
    load_ws(w[v], a.w, at.col[v], a.wdtype, 1.f);
    load_ws(b[v], a.b, at.col[v], a.wdtype, 0.f);
  }
  Raw<E, VEC> xr[NV], gr[NV];
  auto fetch = [&](int64_t n) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (!at.in[v]) continue;
      xr[v].load(x + n * sample + at.off[v]);
      if (gate) gr[v].load(gate + n * sample + at.off[v]);
    }
  };
  int64_t n = at.row;
  if (n >= a.N) return;  // (TPG > 64: a workgroup has one group)
  fetch(n);
  for (;;) {
    float xv[NV][VEC], g[NV][VEC], s = 0.f, q = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        xv[v][i] = at.in[v] ? to_f32(xr[v].e[i]) : 0.f;
        g[v][i] = at.in[v] && gate ? to_f32(gr[v].e[i]) : 0.f;
        s += xv[v][i];
      }
    const int64_t next = n + at.rows;
    if (next < a.N) fetch(next);
    const float mean = sum1<TPG>(s, red) * inv;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        xv[v][i] -= mean;
        q += at.in[v] ? xv[v][i] * xv[v][i] : 0.f;
      }
    const float rstd = 1.f / __builtin_sqrtf(sum1<TPG>(q, red) * inv + a.eps);
    if (at.lane == 0) {
      a.mean[n * a.G + at.g] = mean;
      a.rstd[n * a.G + at.g] = rstd;
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (!at.in[v]) continue;
      Vec<E, VEC> out;
#pragma unroll
      for (int i = 0; i < VEC; ++i) out.v[i] = activate(xv[v][i] * rstd * w[v][i] + b[v][i], a.silu, gate != nullptr, g[v][i]);
      out.store(static_cast<E *>(a.y) + n * sample + at.off[v]);
    }
    if (next >= a.N) break;
    n = next;
  }
}

template <typename E, int VEC, int TPG, int NV>
__global__ __launch_bounds__(TPG > 256 ? TPG : 256) void bwd_kernel(GroupArgs a) {
  using H = Held<VEC, TPG, NV>;
  __shared__ float red[32];
  __shared__ float cols[H::T * NV * VEC], more[H::T];
  const H at(a);
  const int64_t sample = a.S * a.G * a.Dg;
  const float inv = 1.f / ((float)a.S * (float)a.Dg);
  const E *x = static_cast<const E *>(a.x), *dy = static_cast<const E *>(a.dy), *gate = static_cast<const E *>(a.gate);
  float w[NV][VEC], b[NV][VEC], dw[NV][VEC], db[NV][VEC];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) w[v][i] = b[v][i] = dw[v][i] = db[v][i] = 0.f;
    if (!at.in[v]) continue;
    load_ws(w[v], a.w, at.col[v], a.wdtype, 1.f);
    load_ws(b[v], a.b, at.col[v], a.wdtype, 0.f);
  }
  Raw<E, VEC> xr[NV], yr[NV], gr[NV];
  float nmean = 0.f, nrstd = 0.f;
  auto fetch = [&](int64_t n) {
    nmean = a.mean[n * a.G + at.g];
    nrstd = a.rstd[n * a.G + at.g];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (!at.in[v]) continue;
      xr[v].load(x + n * sample + at.off[v]);
      yr[v].load(dy + n * sample + at.off[v]);
      if (gate) gr[v].load(gate + n * sample + at.off[v]);
    }
  };
  if (at.row < a.N) fetch(at.row);
  for (int64_t n = at.row; n < a.N; n += at.rows) {
    const float mean = nmean, rstd = nrstd;
    float xh[NV][VEC], t[NV][VEC], s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      Vec<E, VEC> dgate;
      dgate.zero();
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        xh[v][i] = at.in[v] ? (to_f32(xr[v].e[i]) - mean) * rstd : 0.f;
        const float dz = at.in[v] ? back(to_f32(yr[v].e[i]), xh[v][i] * w[v][i] + b[v][i], a.silu, gate != nullptr,
                                         gate ? to_f32(gr[v].e[i]) : 0.f, dgate.v[i])
                                  : 0.f;
        t[v][i] = dz * w[v][i];
        s1 += t[v][i];
        s2 += t[v][i] * xh[v][i];
        dw[v][i] += dz * xh[v][i];
        db[v][i] += dz;
      }
      if (gate && at.in[v]) dgate.store(static_cast<E *>(a.dgate) + n * sample + at.off[v]);
    }
    if (n + at.rows < a.N) fetch(n + at.rows);
    sum2<TPG>(s1, s2, red);
    s1 *= inv;
    s2 *= inv;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (!at.in[v]) continue;
      Vec<E, VEC> out;
#pragma unroll
      for (int i = 0; i < VEC; ++i) out.v[i] = rstd * (t[v][i] - s1 - xh[v][i] * s2);
      out.store(static_cast<E *>(a.dx) + n * sample + at.off[v]);
    }
  }
  if (!a.dw && !a.db) return;
  // [lane groups / G][2][C]: a lane group's sums over its samples and the positions
  const int64_t C = (int64_t)a.G * a.Dg;
  float *part = reinterpret_cast<float *>(a.ws) + at.row * 2 * C + (int64_t)at.g * a.Dg;
  if (a.S == 1) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (!at.in[v]) continue;
      float *p = part + (at.col[v] - at.g * a.Dg);
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        p[i] = dw[v][i];
        p[C + i] = db[v][i];
      }
    }
    return;
  }
  constexpr int W = TPG * NV * VEC;  // a group's values, in the order of its positions
  // a channel's positions are shared by up to 32 lanes (one: 9 of 22 us with 333
  // positions of 7 channels), whose sums are added in order
  int share = TPG / a.Dg;
  share = share < 1 ? 1 : share > 32 ? 32 : share;
  const int d0 = at.lane / share, q = at.lane - d0 * share, step = TPG / share;
  float *own = cols + at.sub * W;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    __syncthreads();
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int i = 0; i < VEC; ++i) own[(v * TPG + at.lane) * VEC + i] = k ? db[v][i] : dw[v][i];
    __syncthreads();
    for (int d = d0; d < a.Dg && d0 < step; d += step) {
      float s = 0.f;
      for (int p = q; p < a.S; p += share) s += own[p * a.Dg + d];
      if (share == 1)
        part[k * C + d] = s;
      else
        more[at.sub * TPG + d * share + q] = s;  // (share > 1: a lane has one channel)
    }
    if (share == 1) continue;
    __syncthreads();
    if (at.lane < a.Dg) {
      const int n = share < a.S ? share : (int)a.S;
      float s = 0.f;
      for (int j = 0; j < n; ++j) s += more[at.sub * TPG + at.lane * share + j];
      part[k * C + at.lane] = s;
    }
  }
}

// ---- larger groups: by rows of all channels

// A thread's channels [c, c + VEC) and rows; PX pieces of a row side by side.
struct Tile {
  int px, ty_n, tx, ty, c;
  int64_t n, r0, r1;
  bool in;
};
template <int VEC>
__device__ __forceinline__ Tile tile_of(const GroupArgs &a, int64_t blocks, int64_t per) {
  const int C = a.G * a.Dg, pieces = C / VEC;
  Tile t;
  t.px = pieces < 256 ? pieces : 256;
  t.ty_n = 256 / t.px;
  t.tx = threadIdx.x % t.px;
  t.ty = threadIdx.x / t.px;
  t.c = (int)(blockIdx.y * t.px + t.tx) * VEC;
  t.in = t.ty < t.ty_n && t.c < C;
  t.n = blockIdx.x / blocks;
  t.r0 = blockIdx.x % blocks * per;
  t.r1 = t.r0 + per < a.S ? t.r0 + per : a.S;
  return t;
}
// What the threads have of their channels into LDS, in the order [row of threads][channel]
template <int VEC>
__device__ __forceinline__ void to_lds(const Tile &t, const float (&u)[VEC], const float (&v)[VEC], float *lu, float *lv) {
  if (t.ty < t.ty_n) {
    const int at = (t.ty * t.px + t.tx) * VEC;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      lu[at + i] = u[i];
      lv[at + i] = v[i];
    }
  }
  __syncthreads();
}

constexpr int kRows = 4;  // rows a thread has in flight

// [N blocks][2][C]: mean of a block's rows, and the squares about it; by_group:
// [N blocks][2][G], of all channels of a group
// (six workgroups a compute unit, as row_blocks asks: 82 registers would be five)
template <typename E, int VEC>
__global__ __launch_bounds__(256, 6) void stats_kernel(GroupArgs a, int64_t blocks, int64_t per, bool by_group) {
  constexpr int ROWS = 2 * kRows;
  __shared__ float lu[VEC * 256], lv[VEC * 256];
  const Tile t = tile_of<VEC>(a, blocks, per);
  const int64_t C = (int64_t)a.G * a.Dg;
  const E *x = static_cast<const E *>(a.x) + t.n * a.S * C + t.c;
  float first[VEC], mean[VEC], m2[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) first[i] = mean[i] = m2[i] = 0.f;
  const int64_t own = t.in && t.r0 + t.ty < t.r1 ? (t.r1 - t.r0 - t.ty + t.ty_n - 1) / t.ty_n : 0;
  for (int64_t k = 0; k < own; k += ROWS) {
    Raw<E, VEC> r[ROWS];
#pragma unroll
    for (int j = 0; j < ROWS; ++j) r[j].load(x + (t.r0 + t.ty + (k + j < own ? k + j : own - 1) * t.ty_n) * C);
    // eight rows, or the last ones: their share of the mean of all so far
    const int n = own - k < ROWS ? (int)(own - k) : ROWS;
    const float inv = 1.f / (float)n, share = (float)n / (float)(k + n), both = share * (float)k;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const float own0 = to_f32(r[0].e[i]);
      if (k == 0) first[i] = own0;
      float m = 0.f, q = 0.f;
#pragma unroll
      for (int j = 1; j < ROWS; ++j) {
        const float d = j < n ? to_f32(r[j].e[i]) - own0 : 0.f;
        m += d;
        q += d * d;
      }
      q -= m * (m * inv);
      m = m * inv + (own0 - first[i] - mean[i]);
      mean[i] += m * share;
      m2[i] += q + m * m * both;
    }
  }
#pragma unroll
  for (int i = 0; i < VEC; ++i) mean[i] += first[i];
  to_lds<VEC>(t, mean, m2, lu, lv);
  // a thread a channel: the mean of the threads' means, then the squares about it
  const int width = t.px * VEC, rows = (int)(t.r1 - t.r0), even = rows / t.ty_n, odd = rows - even * t.ty_n;
  const float inv_rows = 1.f / (float)rows;
  float *part = reinterpret_cast<float *>(a.ws) + (int64_t)blockIdx.x * 2 * (by_group ? a.G : C);
  for (int c = threadIdx.x; c < width; c += 256) {
    float m = 0.f, q = 0.f;
    for (int y = 0; y < t.ty_n; ++y) m += (float)(even + (y < odd)) * lu[y * width + c];
    m *= inv_rows;
    for (int y = 0; y < t.ty_n; ++y) {
      const float d = lu[y * width + c] - m;
      q += lv[y * width + c] + (float)(even + (y < odd)) * d * d;
    }
    if (by_group) {
      lu[c] = m;  // (row 0 of its own channel)
      lv[c] = q;
    } else {
      const int64_t at = (int64_t)blockIdx.y * width + c;
      if (at < C) part[at] = m, part[C + at] = q;
    }
  }
  if (!by_group) return;
  // (one workgroup has all channels: C <= 256 VEC.)  They have as many rows each:
  // the group's mean is that of their means.
  __syncthreads();
  const float inv_ch = 1.f / (float)a.Dg;
  for (int g = threadIdx.x; g < a.G; g += 256) {
    float m = 0.f, q = 0.f;
    for (int d = 0; d < a.Dg; ++d) m += lu[g * a.Dg + d];
    m *= inv_ch;
    for (int d = 0; d < a.Dg; ++d) {
      const float e = lu[g * a.Dg + d] - m;
      q += lv[g * a.Dg + d] + (float)rows * e * e;
    }
    part[g] = m;
    part[a.G + g] = q;
  }
}

// The sum over a workgroup of 256, in 64 bits, in every thread.
__device__ __forceinline__ double block_sum(double v, double *red) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  return (red[0] + red[1]) + (red[2] + red[3]);
}

// mean and rstd of a sample's group from its blocks, each with `width` of its
// values (Dg, or 1 of all channels)
__global__ __launch_bounds__(256) void stats_join_kernel(GroupArgs a, int64_t blocks, int64_t per, int width) {
  __shared__ double red[4];
  const int g = blockIdx.x % a.G;
  const int64_t n = blockIdx.x / a.G, C = (int64_t)a.G * width;
  const uint32_t items = (uint32_t)(blocks * width);
  const float *part = reinterpret_cast<const float *>(a.ws) + n * blocks * 2 * C + (int64_t)g * width;
  const double count = (double)a.S * width;
  auto rows = [&](int64_t b) { return (double)((b + 1) * per < a.S ? per : a.S - b * per); };
  double s = 0.;
  for (uint32_t i = threadIdx.x; i < items; i += 256) {
    const uint32_t b = i / (uint32_t)width;
    s += rows(b) * part[b * 2 * C + (i - b * width)];
  }
  const double mean = block_sum(s, red) / count;
  double q = 0.;
  for (uint32_t i = threadIdx.x; i < items; i += 256) {
    const uint32_t b = i / (uint32_t)width;
    const float *p = part + b * 2 * C + (i - b * width);
    const double d = p[0] - mean;
    q += p[C] + rows(b) * d * d * (width == 1 ? (double)a.Dg : 1.);
  }
  q = block_sum(q, red) / ((double)a.S * a.Dg);
  if (threadIdx.x == 0) {
    a.mean[blockIdx.x] = (float)mean;
    a.rstd[blockIdx.x] = (float)(1. / sqrt(q + (double)a.eps));
  }
}

// What a thread's channels need of every row.
template <int VEC>
struct Chan {
  float mean[VEC], rstd[VEC], w[VEC], b[VEC];
  __device__ __forceinline__ Chan(const GroupArgs &a, const Tile &t) {
    load_ws(w, a.w, t.c, a.wdtype, 1.f);
    load_ws(b, a.b, t.c, a.wdtype, 0.f);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const int64_t g = t.n * a.G + (t.c + i) / a.Dg;
      mean[i] = a.mean[g];
      rstd[i] = a.rstd[g];
    }
  }
};

template <typename E, int VEC>
__global__ __launch_bounds__(256) void apply_kernel(GroupArgs a, int64_t blocks, int64_t per) {
  const Tile t = tile_of<VEC>(a, blocks, per);
  if (!t.in) return;
  const int64_t C = (int64_t)a.G * a.Dg, base = t.n * a.S * C + t.c;
  const E *x = static_cast<const E *>(a.x) + base, *gate = a.gate ? static_cast<const E *>(a.gate) + base : nullptr;
  E *y = static_cast<E *>(a.y) + base;
  const Chan<VEC> ch(a, t);
  for (int64_t r = t.r0 + t.ty; r < t.r1; r += kRows * t.ty_n) {
    Raw<E, VEC> xr[kRows], gr[kRows];
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const int64_t at = r + j * t.ty_n < t.r1 ? r + j * t.ty_n : r;
      xr[j].load(x + at * C);
      if (gate) gr[j].load(gate + at * C);
    }
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      if (r + j * t.ty_n >= t.r1) break;
      Vec<E, VEC> out;
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        out.v[i] = activate((to_f32(xr[j].e[i]) - ch.mean[i]) * ch.rstd[i] * ch.w[i] + ch.b[i], a.silu, gate != nullptr,
                            gate ? to_f32(gr[j].e[i]) : 0.f);
      out.store(y + (r + j * t.ty_n) * C);
    }
  }
}

// dw, db of 32 columns from the partials, added in order
__device__ __forceinline__ void sum_columns(const GroupArgs &a, int64_t parts, int64_t block) {
  const int64_t C = (int64_t)a.G * a.Dg;
  sum_parts(reinterpret_cast<const float *>(a.ws), parts, 2 * C, [&](int64_t i, float v) {
    if (i < C) {
      if (a.dw) store_w(a.dw, i, v, a.wdtype);
    } else if (a.db) {
      store_w(a.db, i - C, v, a.wdtype);
    }
  }, block);
}

// [N blocks][2][C]: sums of dz xh and dz over a block's rows
template <typename E, int VEC>
__global__ __launch_bounds__(256) void sums_kernel(GroupArgs a, int64_t blocks, int64_t per) {
  __shared__ float lu[VEC * 256], lv[VEC * 256];
  const Tile t = tile_of<VEC>(a, blocks, per);
  const int64_t C = (int64_t)a.G * a.Dg, base = t.n * a.S * C + t.c;
  float dw[VEC], db[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) dw[i] = db[i] = 0.f;
  if (t.in) {
    const E *x = static_cast<const E *>(a.x) + base, *gate = a.gate ? static_cast<const E *>(a.gate) + base : nullptr;
    const E *dy = static_cast<const E *>(a.dy) + base;
    const Chan<VEC> ch(a, t);
    for (int64_t r = t.r0 + t.ty; r < t.r1; r += kRows * t.ty_n) {
      Raw<E, VEC> xr[kRows], yr[kRows], gr[kRows];
#pragma unroll
      for (int j = 0; j < kRows; ++j) {
        const int64_t at = r + j * t.ty_n < t.r1 ? r + j * t.ty_n : r;
        xr[j].load(x + at * C);
        yr[j].load(dy + at * C);
        if (gate) gr[j].load(gate + at * C);
      }
#pragma unroll
      for (int j = 0; j < kRows; ++j) {
        if (r + j * t.ty_n >= t.r1) break;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const float xh = (to_f32(xr[j].e[i]) - ch.mean[i]) * ch.rstd[i];
          float dgate;
          const float dz = back(to_f32(yr[j].e[i]), xh * ch.w[i] + ch.b[i], a.silu, gate != nullptr,
                                gate ? to_f32(gr[j].e[i]) : 0.f, dgate);
          dw[i] += dz * xh;
          db[i] += dz;
        }
      }
    }
  }
  to_lds<VEC>(t, dw, db, lu, lv);
  const int width = t.px * VEC;
  float *part = reinterpret_cast<float *>(a.ws) + (int64_t)blockIdx.x * 2 * C;
  for (int c = threadIdx.x; c < width; c += 256) {
    float u = 0.f, v = 0.f;
    for (int y = 0; y < t.ty_n; ++y) {
      u += lu[y * width + c];
      v += lv[y * width + c];
    }
    const int64_t at = (int64_t)blockIdx.y * width + c;
    if (at < C) part[at] = u, part[C + at] = v;
  }
}

// [N][G][2]: the means of t and t xh of a sample's group, behind the partials; the
// workgroups past them have 32 columns of dw and db each (kSumThreads threads all)
__global__ __launch_bounds__(kSumThreads) void sums_join_kernel(GroupArgs a, float *sums, int64_t blocks, int64_t groups) {
  __shared__ double red[kSumThreads / 64][2];
  const int64_t C = (int64_t)a.G * a.Dg;
  if (blockIdx.x >= groups) {
    sum_columns(a, a.N * blocks, blockIdx.x - groups);
    return;
  }
  const int g = blockIdx.x % a.G;
  const int64_t n = blockIdx.x / a.G;
  const uint32_t items = (uint32_t)(blocks * a.Dg);
  const float *part = reinterpret_cast<const float *>(a.ws) + n * blocks * 2 * C + (int64_t)g * a.Dg;
  double s1 = 0., s2 = 0.;
  for (uint32_t i = threadIdx.x; i < items; i += kSumThreads) {
    const uint32_t b = i / (uint32_t)a.Dg, d = i - b * a.Dg;
    const float *p = part + b * 2 * C + d;
    const double w = a.w ? load_w(a.w, (int64_t)g * a.Dg + d, a.wdtype) : 1.f;
    s1 += w * p[C];
    s2 += w * p[0];
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    s1 += __shfl_xor(s1, d);
    s2 += __shfl_xor(s2, d);
  }
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6][0] = s1, red[threadIdx.x >> 6][1] = s2;
  __syncthreads();
  if (threadIdx.x < 2) {
    double s = 0.;
    for (int i = 0; i < kSumThreads / 64; ++i) s += red[i][threadIdx.x];
    sums[2 * (int64_t)blockIdx.x + threadIdx.x] = (float)(s / ((double)a.S * a.Dg));
  }
}

template <typename E, int VEC>
__global__ __launch_bounds__(256) void grads_kernel(GroupArgs a, const float *sums, int64_t blocks, int64_t per) {
  const Tile t = tile_of<VEC>(a, blocks, per);
  if (!t.in) return;
  const int64_t C = (int64_t)a.G * a.Dg, base = t.n * a.S * C + t.c;
  const E *x = static_cast<const E *>(a.x) + base, *gate = a.gate ? static_cast<const E *>(a.gate) + base : nullptr;
  const E *dy = static_cast<const E *>(a.dy) + base;
  E *dx = static_cast<E *>(a.dx) + base, *dg = a.gate ? static_cast<E *>(a.dgate) + base : nullptr;
  const Chan<VEC> ch(a, t);
  float m1[VEC], m2[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    const int64_t g = t.n * a.G + (t.c + i) / a.Dg;
    m1[i] = sums[2 * g];
    m2[i] = sums[2 * g + 1];
  }
  constexpr int ROWS = 2;
  for (int64_t r = t.r0 + t.ty; r < t.r1; r += ROWS * t.ty_n) {
    Raw<E, VEC> xr[ROWS], yr[ROWS], gr[ROWS];
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
      const int64_t at = r + j * t.ty_n < t.r1 ? r + j * t.ty_n : r;
      xr[j].load(x + at * C);
      yr[j].load(dy + at * C);
      if (gate) gr[j].load(gate + at * C);
    }
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
      if (r + j * t.ty_n >= t.r1) break;
      Vec<E, VEC> out, og;
      og.zero();
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float xh = (to_f32(xr[j].e[i]) - ch.mean[i]) * ch.rstd[i];
        const float dz = back(to_f32(yr[j].e[i]), xh * ch.w[i] + ch.b[i], a.silu, gate != nullptr,
                              gate ? to_f32(gr[j].e[i]) : 0.f, og.v[i]);
        out.v[i] = ch.rstd[i] * (dz * ch.w[i] - m1[i] - xh * m2[i]);
      }
      out.store(dx + (r + j * t.ty_n) * C);
      if (gate) og.store(dg + (r + j * t.ty_n) * C);
    }
  }
}

__global__ __launch_bounds__(kSumThreads) void sum_kernel(GroupArgs a, int64_t parts) { sum_columns(a, parts, blockIdx.x); }

bool al16(const void *p) { return ((uintptr_t)p & 15) == 0; }

// Groups that registers hold (offsets inside a sample are 32-bit there).
bool held(const GroupArgs &a) {
  return a.S <= kHeld && a.S * a.Dg <= kHeld && a.S * a.G * a.Dg < ((int64_t)1 << 31) - 1024;
}
int lanes_for(int64_t values) {  // 8 a lane
  return values <= 32 ? 4 : values <= 128 ? 16 : values <= 512 ? 64 : values <= 2048 ? 256 : 1024;
}
// Workgroups whose lane groups are a multiple of G, so that each keeps its
// channels from sample to sample: `want`, or as many as there is work for.
int64_t held_blocks(const GroupArgs &a, int64_t want) {
  const int lanes = lanes_for(a.S * a.Dg), rpb = (lanes > 256 ? lanes : 256) / lanes;
  int64_t g = a.G, r = rpb;
  while (r) {
    const int64_t m = g % r;
    g = r;
    r = m;
  }
  const int64_t unit = a.G / g, most = (a.N * a.G + rpb - 1) / rpb;
  int64_t blocks = want < most ? want : most;
  blocks = (blocks + unit - 1) / unit * unit;
  return blocks ? blocks : unit;
}
int64_t fwd_want(const GroupArgs &a) { return compute_units() * (lanes_for(a.S * a.Dg) > 256 ? 2 : 8); }
int64_t bwd_want(const GroupArgs &a) { return compute_units() * (lanes_for(a.S * a.Dg) > 256 ? 1 : 4); }
int64_t held_parts(const GroupArgs &a) {
  const int lanes = lanes_for(a.S * a.Dg);
  return held_blocks(a, bwd_want(a)) * ((lanes > 256 ? lanes : 256) / lanes) / a.G;
}

// Blocks of a sample's rows in the two-pass form: six workgroups a compute unit,
// in whole rounds of their threads' rows in flight.
int64_t row_blocks(const GroupArgs &a, int64_t *per) {
  const int64_t pieces = (int64_t)a.G * a.Dg / (a.G * a.Dg % 8 == 0 ? 8 : 1);  // (as if aligned: the same workspace)
  const int64_t unit = 2 * kRows * (pieces < 256 ? 256 / pieces : 1), cols = (pieces + 255) / 256;
  int64_t want = (compute_units() * 6 + a.N * cols - 1) / (a.N * cols);
  if (want < 1) want = 1;
  *per = ((a.S + want - 1) / want + unit - 1) / unit * unit;
  return (a.S + *per - 1) / *per;
}
size_t part_bytes(const GroupArgs &a) {
  int64_t per;
  return (size_t)(a.N * row_blocks(a, &per)) * 2 * a.G * a.Dg * 4;
}

template <typename E, int VEC, int TPG, int NV>
hipError_t go_fwd(const GroupArgs &a, hipStream_t st) {
  KernelTimer kt("group_fwd", st);
  fwd_kernel<E, VEC, TPG, NV><<<(unsigned)held_blocks(a, fwd_want(a)), Held<VEC, TPG, NV>::T, 0, st>>>(a);
  return hipGetLastError();
}
template <typename E, int VEC, int TPG, int NV>
hipError_t go_bwd(const GroupArgs &a, hipStream_t st) {
  KernelTimer kt("group_bwd", st);
  bwd_kernel<E, VEC, TPG, NV><<<(unsigned)held_blocks(a, bwd_want(a)), Held<VEC, TPG, NV>::T, 0, st>>>(a);
  return hipGetLastError();
}

#define GDN_GROUP(GO, E, VEC)                                   \
  switch (lanes_for(a.S * a.Dg)) {                              \
    case 4: return GO<E, VEC, 4, 8 / VEC>(a, st);               \
    case 16: return GO<E, VEC, 16, 8 / VEC>(a, st);             \
    case 64: return GO<E, VEC, 64, 8 / VEC>(a, st);             \
    case 256: return GO<E, VEC, 256, 8 / VEC>(a, st);           \
    default: return GO<E, VEC, 1024, 8 / VEC>(a, st);           \
  }
hipError_t held_fwd(const GroupArgs &a, bool wide, hipStream_t st) {
  if (a.dtype == 1) {
    if (wide) { GDN_GROUP(go_fwd, bf16, 8) }
    GDN_GROUP(go_fwd, bf16, 1)
  }
  if (wide) { GDN_GROUP(go_fwd, float, 4) }
  GDN_GROUP(go_fwd, float, 1)
}
hipError_t held_bwd(const GroupArgs &a, bool wide, hipStream_t st) {
  if (a.dtype == 1) {
    if (wide) { GDN_GROUP(go_bwd, bf16, 8) }
    GDN_GROUP(go_bwd, bf16, 1)
  }
  if (wide) { GDN_GROUP(go_bwd, float, 4) }
  GDN_GROUP(go_bwd, float, 1)
}

template <typename E, int VEC>
hipError_t tall_fwd(const GroupArgs &a, hipStream_t st) {
  int64_t per;
  const int64_t blocks = row_blocks(a, &per);
  const int pieces = a.G * a.Dg / VEC;
  const dim3 grid((unsigned)(a.N * blocks), (unsigned)((pieces + 255) / 256));
  {
    KernelTimer kt("group_stats", st);
    const bool by_group = grid.y == 1;
    stats_kernel<E, VEC><<<grid, 256, 0, st>>>(a, blocks, per, by_group);
    stats_join_kernel<<<(unsigned)(a.N * a.G), 256, 0, st>>>(a, blocks, per, by_group ? 1 : a.Dg);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  KernelTimer kt("group_apply", st);
  apply_kernel<E, VEC><<<grid, 256, 0, st>>>(a, blocks, per);
  return hipGetLastError();
}
template <typename E, int VEC>
hipError_t tall_bwd(const GroupArgs &a, hipStream_t st) {
  int64_t per;
  const int64_t blocks = row_blocks(a, &per);
  const int pieces = a.G * a.Dg / VEC;
  const dim3 grid((unsigned)(a.N * blocks), (unsigned)((pieces + 255) / 256));
  float *sums = reinterpret_cast<float *>(a.ws + part_bytes(a));
  {
    KernelTimer kt("group_sums", st);
    sums_kernel<E, VEC><<<grid, 256, 0, st>>>(a, blocks, per);
    const int64_t groups = a.N * a.G;
    sums_join_kernel<<<(unsigned)(groups + (a.dw || a.db ? sum_blocks(2 * (int64_t)a.G * a.Dg) : 0)), kSumThreads, 0, st>>>(a, sums, blocks, groups);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  KernelTimer kt("group_grads", st);
  grads_kernel<E, VEC><<<grid, 256, 0, st>>>(a, sums, blocks, per);
  return hipGetLastError();
}

}  // namespace
}  // namespace group

bool group_fits(const GroupArgs &a, bool bwd) {
  if (a.N == 0 || group::held(a)) return true;
  int64_t per;
  const int64_t blocks = a.N * group::row_blocks(a, &per), channels = (int64_t)a.G * a.Dg, cols = (channels + 255) / 256;
  constexpr int64_t most = (int64_t)1 << 24;  // workgroups of 256
  // a workgroup joins each group's blocks; the backward's have kSumThreads, and sum up dw and db beside that
  const int64_t joins = bwd ? (a.N * a.G + sum_blocks(2 * channels)) * (kSumThreads / 256) : a.N * a.G;
  return cols < 65536 && blocks < most && blocks * cols < most && joins < most;
}
size_t group_fwd_bytes(const GroupArgs &a) {
  const size_t n = group::held(a) || a.N == 0 ? 0 : group::part_bytes(a);
  return n ? n : 256;
}
size_t group_bwd_bytes(const GroupArgs &a) {
  if (a.N == 0) return 256;
  if (group::held(a)) return (size_t)group::held_parts(a) * 2 * a.G * a.Dg * 4;
  return group::part_bytes(a) + (size_t)a.N * a.G * 8;
}

hipError_t launch_group_fwd(const GroupArgs &a, hipStream_t st) {
  using namespace group;
  if (a.N == 0) return hipSuccess;
  const int vec = a.dtype == 1 ? 8 : 4;
  const bool to16 = al16(a.x) && al16(a.w) && al16(a.b) && al16(a.y) && al16(a.gate);
  if (held(a)) return held_fwd(a, to16 && a.Dg % vec == 0, st);
  const bool wide = to16 && a.G * a.Dg % vec == 0;
  if (a.dtype == 1) return wide ? tall_fwd<bf16, 8>(a, st) : tall_fwd<bf16, 1>(a, st);
  return wide ? tall_fwd<float, 4>(a, st) : tall_fwd<float, 1>(a, st);
}

hipError_t launch_group_bwd(const GroupArgs &a, hipStream_t st) {
  using namespace group;
  int64_t parts = 0;
  if (a.N) {
    const int vec = a.dtype == 1 ? 8 : 4;
    const bool to16 = al16(a.x) && al16(a.w) && al16(a.b) && al16(a.dy) && al16(a.gate) && al16(a.dx) && al16(a.dgate);
    if (!held(a)) {
      const bool wide = to16 && a.G * a.Dg % vec == 0;
      if (a.dtype == 1) return wide ? tall_bwd<bf16, 8>(a, st) : tall_bwd<bf16, 1>(a, st);
      return wide ? tall_bwd<float, 4>(a, st) : tall_bwd<float, 1>(a, st);
    }
    parts = held_parts(a);
    const hipError_t e = held_bwd(a, to16 && a.Dg % vec == 0, st);
    if (e != hipSuccess) return e;
  }
  if (!a.dw && !a.db) return hipSuccess;
  KernelTimer kt("group_sum", st);
  sum_kernel<<<sum_blocks(2 * (int64_t)a.G * a.Dg), kSumThreads, 0, st>>>(a, parts);
  return hipGetLastError();
}

}  // namespace gdn
