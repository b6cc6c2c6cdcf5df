// Layer norm over the last dimension, with an optional output gate, and its
// backward with the reduction of the weight's gradient:
//
//   xh = (x - mean) rstd,  z = xh w + b,  y = z silu(gate)
//
// (rms: mean = 0 and rstd from the mean square).  With t = dy silu(gate) w:
//
//   dx = rstd (t - mean_D(t) - xh mean_D(t xh))      (rms: no mean_D(t))
//   dw = sum_rows dy silu(gate) xh,  db = sum_rows dy silu(gate),
//   dgate = dy z silu'(gate)
//
// Memory decides: a row is read once and held in registers by the TPR lanes
// that share it, so the variance is taken from the centred values.  Column
// sums stay in the registers of the lanes that own the columns while a
// workgroup walks its rows; one partial per workgroup is written and a second
// kernel adds them in order (no atomics, the same bits on every run).
// 16384 x 4096 bf16 forward: 44 us, 6.1 TB/s; gated RMS backward of 2^19 rows
// of 128: 140 us, 4.8 TB/s, and 6 for the sums; 1500 x 5003 fp32 backward: 22
// and 6 us.
#include "gdn_internal.h"
#include "gdn_mixer.hpp"

namespace gdn {
namespace {

// Sum over the TPR lanes of a row, the same value in each: inside 16 lanes by
// DPP, across the wave by lane exchange, across waves through LDS (TPR > 64,
// where the row has the whole workgroup).
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float *red) {
  v = group_sum<(TPR < 16 ? TPR : 16)>(v);
  if constexpr (TPR >= 32) v += __shfl_xor(v, 16);
  if constexpr (TPR >= 64) v += __shfl_xor(v, 32);
  if constexpr (TPR > 64) {
    const int w = threadIdx.x >> 6;
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[w] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < TPR / 64; ++i) v += red[i];
  }
  return v;
}

// Two such sums at once.
template <int TPR>
__device__ __forceinline__ void row_sum2(float &u, float &v, float *red) {
  u = group_sum<(TPR < 16 ? TPR : 16)>(u);
  v = group_sum<(TPR < 16 ? TPR : 16)>(v);
  if constexpr (TPR >= 32) u += __shfl_xor(u, 16), v += __shfl_xor(v, 16);
  if constexpr (TPR >= 64) u += __shfl_xor(u, 32), v += __shfl_xor(v, 32);
  if constexpr (TPR > 64) {
    const int w = threadIdx.x >> 6;
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[2 * w] = u, red[2 * w + 1] = v;
    __syncthreads();
    u = v = 0.f;
#pragma unroll
    for (int i = 0; i < TPR / 64; ++i) u += red[2 * i], v += red[2 * i + 1];
  }
}

__device__ __forceinline__ float silu_of(float z, float &s) {
  s = sigmoidf(z);
  return z * s;
}

// TPR lanes hold a row, NV pieces of VEC elements each: piece v of lane l is
// columns (v TPR + l) VEC ...  A workgroup walks rows with its columns'
// weights in registers (read again for every row, one by one, they took five
// times the row's own time), the next row's loads under the current one's sums.
template <typename E, int VEC, int TPR, int NV>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void norm_fwd_kernel(NormArgs a) {
  constexpr int RPB = (TPR > 256 ? TPR : 256) / TPR;
  __shared__ float red[16];
  const int lane = threadIdx.x % TPR;
  const int64_t step = (int64_t)gridDim.x * RPB;
  const E *x = static_cast<const E *>(a.x), *gate = static_cast<const E *>(a.gate);
  const float inv = 1.f / (float)a.D;
  float w[NV][VEC], b[NV][VEC];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = (v * TPR + lane) * VEC;
    if (c >= a.D) continue;
    load_ws(w[v], a.w, c, a.wdtype, 1.f);
    load_ws(b[v], a.b, c, a.wdtype, 0.f);
  }
  Raw<E, VEC> xr[NV], gr[NV];
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * TPR + lane) * VEC;
      if (c >= a.D) continue;
      xr[v].load(x + row * a.D + c);
      if (gate) gr[v].load(gate + row * a.D + c);
    }
  };
  int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
  if (row >= a.rows) return;  // (TPR > 64: a workgroup has one row)
  fetch(row);
  for (;;) {
    Vec<E, VEC> xv[NV], g[NV];
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const bool in = (v * TPR + lane) * VEC < a.D;
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        xv[v].v[i] = in ? to_f32(xr[v].e[i]) : 0.f;
        g[v].v[i] = in && gate ? to_f32(gr[v].e[i]) : 0.f;
        s += xv[v].v[i];
      }
    }
    const int64_t next = row + step;
    if (next < a.rows) fetch(next);
    const float mean = a.rms ? 0.f : row_sum<TPR>(s, red) * inv;
    float q = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const bool in = (v * TPR + lane) * VEC < a.D;
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float d = in ? xv[v].v[i] - mean : 0.f;
        q += d * d;
      }
    }
    const float rstd = 1.f / __builtin_sqrtf(row_sum<TPR>(q, red) * inv + a.eps);
    if (lane == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * TPR + lane) * VEC;
      if (c >= a.D) continue;
      Vec<E, VEC> out;
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        float z = (xv[v].v[i] - mean) * rstd * w[v][i] + b[v][i];
        if (gate) z *= g[v].v[i] * sigmoidf(g[v].v[i]);
        out.v[i] = z;
      }
      out.store(static_cast<E *>(a.y) + row * a.D + c);
    }
    if (next >= a.rows) break;
    row = next;
  }
}

// Rows wider than a workgroup's registers hold: the row is read three times
// (mean, centred squares, output), the later ones from the caches.
template <typename E>
__global__ __launch_bounds__(1024) void norm_fwd_wide_kernel(NormArgs a) {
  __shared__ float red[16];
  const int64_t row = blockIdx.x;
  const E *x = static_cast<const E *>(a.x) + row * a.D;
  float s = 0.f;
  if (!a.rms)
    for (int c = threadIdx.x; c < a.D; c += 1024) s += to_f32(x[c]);
  const float inv = 1.f / (float)a.D;
  const float mean = a.rms ? 0.f : row_sum<1024>(s, red) * inv;
  float q = 0.f;
  for (int c = threadIdx.x; c < a.D; c += 1024) {
    const float d = to_f32(x[c]) - mean;
    q += d * d;
  }
  const float rstd = 1.f / __builtin_sqrtf(row_sum<1024>(q, red) * inv + a.eps);
  if (threadIdx.x == 0) {
    if (a.mean) a.mean[row] = mean;
    if (a.rstd) a.rstd[row] = rstd;
  }
  for (int c = threadIdx.x; c < a.D; c += 1024) {
    float z = (to_f32(x[c]) - mean) * rstd;
    if (a.w) z *= load_w(a.w, c, a.wdtype);
    if (a.b) z += load_w(a.b, c, a.wdtype);
    if (a.gate) {
      const float g = to_f32(static_cast<const E *>(a.gate)[row * a.D + c]);
      z *= g * sigmoidf(g);
    }
    static_cast<E *>(a.y)[row * a.D + c] = from_f32<E>(z);
  }
}

// One element of the backward before its row's sums: t = dz w, and xh.
struct Elem {
  float xh, t, dz, dgate;
};
__device__ __forceinline__ Elem elem(const NormArgs &a, float x, float dy, float gate, float w,
                                     float b, float mean, float rstd) {
  Elem e;
  e.xh = (x - mean) * rstd;
  e.dz = dy;
  e.dgate = 0.f;
  if (a.gate) {
    float s;
    const float g = silu_of(gate, s);
    e.dgate = dy * (e.xh * w + b) * (s * (1.f + gate * (1.f - s)));
    e.dz = dy * g;
  }
  e.t = e.dz * w;
  return e;
}

template <typename E, int VEC, int TPR, int NV>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void norm_bwd_kernel(NormArgs a, int64_t per) {
  constexpr int THREADS = TPR > 256 ? TPR : 256;
  constexpr int RPB = THREADS / TPR;
  __shared__ float red[32];
  __shared__ float cols[RPB > 1 ? THREADS : 1];
  const int lane = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const float inv = 1.f / (float)a.D;
  float w[NV][VEC], b[NV][VEC], dw[NV][VEC], db[NV][VEC];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = (v * TPR + lane) * VEC;
#pragma unroll
    for (int i = 0; i < VEC; ++i) w[v][i] = b[v][i] = dw[v][i] = db[v][i] = 0.f;
    if (c >= a.D) continue;
    load_ws(w[v], a.w, c, a.wdtype, 1.f);
    load_ws(b[v], a.b, c, a.wdtype, 0.f);
  }
  const int64_t r0 = (int64_t)blockIdx.x * per;
  const int64_t r1 = r0 + per < a.rows ? r0 + per : a.rows;
  Raw<E, VEC> xr[NV], yr[NV], gr[NV];
  float nmean = 0.f, nrstd = 0.f;
  auto fetch = [&](int64_t rb) {
    const int64_t row = rb + sub < r1 ? rb + sub : r1 - 1;
    nmean = a.rms ? 0.f : a.mean[row];
    nrstd = a.rstd[row];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * TPR + lane) * VEC;
      if (c >= a.D) continue;
      xr[v].load(static_cast<const E *>(a.x) + row * a.D + c);
      yr[v].load(static_cast<const E *>(a.dy) + row * a.D + c);
      if (a.gate) gr[v].load(static_cast<const E *>(a.gate) + row * a.D + c);
    }
  };
  fetch(r0);
  for (int64_t rb = r0; rb < r1; rb += RPB) {
    const bool live = rb + sub < r1;
    const int64_t row = live ? rb + sub : r1 - 1;
    const float mean = nmean, rstd = nrstd;
    Vec<E, VEC> xh[NV], t[NV];
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * TPR + lane) * VEC;
      xh[v].zero();
      t[v].zero();
      if (c >= a.D) continue;
      Vec<E, VEC> dgate;
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const Elem e = elem(a, to_f32(xr[v].e[i]), to_f32(yr[v].e[i]), a.gate ? to_f32(gr[v].e[i]) : 0.f, w[v][i], b[v][i],
                            mean, rstd);
        xh[v].v[i] = e.xh;
        t[v].v[i] = e.t;
        dgate.v[i] = e.dgate;
        s1 += e.t;
        s2 += e.t * e.xh;
        dw[v][i] += live ? e.dz * e.xh : 0.f;
        db[v][i] += live ? e.dz : 0.f;
      }
      if (a.gate && live) dgate.store(static_cast<E *>(a.dgate) + row * a.D + c);
    }
    if (rb + RPB < r1) fetch(rb + RPB);
    row_sum2<TPR>(s1, s2, red);
    s1 = a.rms ? 0.f : s1 * inv;
    s2 *= inv;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * TPR + lane) * VEC;
      if (c >= a.D || !live) continue;
      Vec<E, VEC> out;
#pragma unroll
      for (int i = 0; i < VEC; ++i) out.v[i] = rstd * (t[v].v[i] - s1 - xh[v].v[i] * s2);
      out.store(static_cast<E *>(a.dx) + row * a.D + c);
    }
  }
  if (!a.dw && !a.db) return;
  float *part = a.partial + (int64_t)blockIdx.x * 2 * a.D;
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int i = 0; i < VEC; ++i)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float s = k ? db[v][i] : dw[v][i];
        if constexpr (RPB > 1) {
          __syncthreads();
          cols[threadIdx.x] = s;
          __syncthreads();
          s = 0.f;
          if (sub == 0)
            for (int j = 0; j < RPB; ++j) s += cols[j * TPR + lane];
        }
        const int c = (v * TPR + lane) * VEC + i;
        if (sub == 0 && c < a.D) part[k * a.D + c] = s;
      }
}

// Wide rows, first kernel: a row's two sums.
template <typename E>
__global__ __launch_bounds__(1024) void norm_bwd_rows_kernel(NormArgs a, float *sums) {
  __shared__ float red[16];
  const int64_t row = blockIdx.x;
  const float mean = a.rms ? 0.f : a.mean[row], rstd = a.rstd[row];
  float s1 = 0.f, s2 = 0.f;
  for (int c = threadIdx.x; c < a.D; c += 1024) {
    const int64_t i = row * a.D + c;
    const Elem e = elem(a, to_f32(static_cast<const E *>(a.x)[i]), to_f32(static_cast<const E *>(a.dy)[i]),
                        a.gate ? to_f32(static_cast<const E *>(a.gate)[i]) : 0.f,
                        a.w ? load_w(a.w, c, a.wdtype) : 1.f, a.b ? load_w(a.b, c, a.wdtype) : 0.f, mean, rstd);
    s1 += e.t;
    s2 += e.t * e.xh;
  }
  const float inv = 1.f / (float)a.D;
  s1 = a.rms ? 0.f : row_sum<1024>(s1, red) * inv;
  s2 = row_sum<1024>(s2, red) * inv;
  if (threadIdx.x == 0) {
    sums[2 * row] = s1;
    sums[2 * row + 1] = s2;
  }
}
// Wide rows, second kernel: a thread owns a column over `per` rows.
template <typename E>
__global__ __launch_bounds__(256) void norm_bwd_cols_kernel(NormArgs a, const float *sums, int64_t per) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= a.D) return;
  const float w = a.w ? load_w(a.w, c, a.wdtype) : 1.f, b = a.b ? load_w(a.b, c, a.wdtype) : 0.f;
  const int64_t r0 = (int64_t)blockIdx.y * per;
  const int64_t r1 = r0 + per < a.rows ? r0 + per : a.rows;
  float dw = 0.f, db = 0.f;
  for (int64_t row = r0; row < r1; ++row) {
    const int64_t i = row * a.D + c;
    const float mean = a.rms ? 0.f : a.mean[row], rstd = a.rstd[row];
    const Elem e = elem(a, to_f32(static_cast<const E *>(a.x)[i]), to_f32(static_cast<const E *>(a.dy)[i]),
                        a.gate ? to_f32(static_cast<const E *>(a.gate)[i]) : 0.f, w, b, mean, rstd);
    dw += e.dz * e.xh;
    db += e.dz;
    static_cast<E *>(a.dx)[i] = from_f32<E>(rstd * (e.t - sums[2 * row] - e.xh * sums[2 * row + 1]));
    if (a.gate) static_cast<E *>(a.dgate)[i] = from_f32<E>(e.dgate);
  }
  float *part = a.partial + (int64_t)blockIdx.y * 2 * a.D;
  part[c] = dw;
  part[a.D + c] = db;
}

// dw, db from the workgroups' partials, added in order.
__global__ __launch_bounds__(kSumThreads) void norm_sum_kernel(NormArgs a, int64_t parts) {
  sum_parts(a.partial, parts, 2 * (int64_t)a.D, [&](int64_t i, float v) {
    if (i < a.D) {
      if (a.dw) store_w(a.dw, i, v, a.wdtype);
    } else if (a.db) {
      store_w(a.db, i - a.D, v, a.wdtype);
    }
  });
}

// The widest row whose pieces a workgroup holds in registers (16 elements of
// bf16 or fp32 a lane at 1024 lanes).
constexpr int kHeld = 16384;
int lanes_for(int D) {  // 16 elements a lane at the most
  return D <= 256 ? 16 : D <= 1024 ? 64 : D <= 4096 ? 256 : 1024;
}
bool al16(const void *p) { return ((uintptr_t)p & 15) == 0; }

template <typename E, int VEC, int TPR, int NV>
hipError_t go_fwd(const NormArgs &a, hipStream_t st) {
  constexpr int T = TPR > 256 ? TPR : 256, RPB = T / TPR;
  KernelTimer kt("norm_fwd", st);
  // as many workgroups as the compute units hold at once (2048 threads each)
  int64_t blocks = compute_units() * (2048 / T);
  const int64_t most = (a.rows + RPB - 1) / RPB;
  if (blocks > most) blocks = most;
  norm_fwd_kernel<E, VEC, TPR, NV><<<(unsigned)blocks, T, 0, st>>>(a);
  return hipGetLastError();
}
template <typename E, int VEC, int TPR, int NV>
hipError_t go_bwd(const NormArgs &a, hipStream_t st) {
  constexpr int T = TPR > 256 ? TPR : 256;
  const int64_t parts = norm_bwd_parts(a.rows), per = (a.rows + parts - 1) / parts;
  KernelTimer kt("norm_bwd", st);
  norm_bwd_kernel<E, VEC, TPR, NV><<<(unsigned)parts, T, 0, st>>>(a, per);
  return hipGetLastError();
}

#define GDN_NORM(GO, E, VEC, N1, N2)                                                        \
  switch (lanes_for(a.D)) {                                                                 \
    case 16: return a.D <= 16 * VEC * N1 ? GO<E, VEC, 16, N1>(a, st) : GO<E, VEC, 16, N2>(a, st); \
    case 64: return a.D <= 64 * VEC * N1 ? GO<E, VEC, 64, N1>(a, st) : GO<E, VEC, 64, N2>(a, st); \
    case 256: return a.D <= 256 * VEC * N1 ? GO<E, VEC, 256, N1>(a, st) : GO<E, VEC, 256, N2>(a, st); \
    default: return a.D <= 1024 * VEC * N1 ? GO<E, VEC, 1024, N1>(a, st) : GO<E, VEC, 1024, N2>(a, st); \
  }

hipError_t held_fwd(const NormArgs &a, bool wide, hipStream_t st) {
  if (a.dtype == 1) {
    if (wide) { GDN_NORM(go_fwd, bf16, 8, 1, 2) }
    GDN_NORM(go_fwd, bf16, 1, 8, 16)
  }
  if (wide) { GDN_NORM(go_fwd, float, 4, 2, 4) }
  GDN_NORM(go_fwd, float, 1, 8, 16)
}
hipError_t held_bwd(const NormArgs &a, bool wide, hipStream_t st) {
  if (a.dtype == 1) {
    if (wide) { GDN_NORM(go_bwd, bf16, 8, 1, 2) }
    GDN_NORM(go_bwd, bf16, 1, 8, 16)
  }
  if (wide) { GDN_NORM(go_bwd, float, 4, 2, 4) }
  GDN_NORM(go_bwd, float, 1, 8, 16)
}

}  // namespace

// Workgroups of the backward, each with its partial of the column sums: four
// a compute unit, but at least 16 rows each while every compute unit has one,
// so that the partials stay small.
int64_t norm_bwd_parts(int64_t rows) {
  int64_t p = compute_units() * 4;
  int64_t most = (rows + 15) / 16;
  if (most < compute_units()) most = rows < compute_units() ? rows : compute_units();
  p = p < most ? p : most;
  if (p < 1) p = 1;
  const int64_t per = (rows + p - 1) / p;
  return per ? (rows + per - 1) / per : 1;
}
size_t norm_bwd_floats(int64_t rows, int D) {
  return (size_t)norm_bwd_parts(rows) * 2 * D + (D > kHeld ? (size_t)rows * 2 : 0);
}

hipError_t launch_norm_fwd(const NormArgs &a, hipStream_t st) {
  if (a.rows == 0) return hipSuccess;
  if (a.D > kHeld) {
    KernelTimer kt("norm_fwd", st);
    if (a.dtype == 1)
      norm_fwd_wide_kernel<bf16><<<(unsigned)a.rows, 1024, 0, st>>>(a);
    else
      norm_fwd_wide_kernel<float><<<(unsigned)a.rows, 1024, 0, st>>>(a);
    return hipGetLastError();
  }
  const int vec = a.dtype == 1 ? 8 : 4;
  return held_fwd(a, a.D % vec == 0 && al16(a.x) && al16(a.w) && al16(a.b) && al16(a.y) && al16(a.gate), st);
}

hipError_t launch_norm_bwd(const NormArgs &a, hipStream_t st) {
  const int64_t parts = norm_bwd_parts(a.rows);
  hipError_t e = hipSuccess;
  if (a.rows) {
    if (a.D > kHeld) {
      float *sums = a.partial + parts * 2 * a.D;
      const int64_t per = (a.rows + parts - 1) / parts;
      const dim3 grid((unsigned)((a.D + 255) / 256), (unsigned)parts);
      KernelTimer kt("norm_bwd", st);
      if (a.dtype == 1) {
        norm_bwd_rows_kernel<bf16><<<(unsigned)a.rows, 1024, 0, st>>>(a, sums);
        norm_bwd_cols_kernel<bf16><<<grid, 256, 0, st>>>(a, sums, per);
      } else {
        norm_bwd_rows_kernel<float><<<(unsigned)a.rows, 1024, 0, st>>>(a, sums);
        norm_bwd_cols_kernel<float><<<grid, 256, 0, st>>>(a, sums, per);
      }
      e = hipGetLastError();
    } else {
      const int vec = a.dtype == 1 ? 8 : 4;
      e = held_bwd(a, a.D % vec == 0 && al16(a.x) && al16(a.w) && al16(a.b) && al16(a.dy) && al16(a.gate) && al16(a.dx) && al16(a.dgate), st);
    }
  }
  if (e != hipSuccess || (!a.dw && !a.db)) return e;
  KernelTimer kt("norm_bwd_sum", st);
  norm_sum_kernel<<<sum_blocks(2 * (int64_t)a.D), kSumThreads, 0, st>>>(a, a.rows ? parts : 0);
  return hipGetLastError();
}

}  // namespace gdn
