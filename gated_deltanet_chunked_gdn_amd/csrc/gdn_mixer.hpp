// Device helpers of the sequence-mixer kernels.
#pragma once

#include "gdn_common.hpp"
#include "gdn_mixer.h"

namespace gdn {

// Sequence n's tokens [first, end), clamped to the batch, so that a bad
// cu_seqlens on the device cannot lead a kernel out of its buffers.
struct Span {
  int64_t first, end;
};
__device__ __forceinline__ Span seq_span(const Seqs &s, int n) {
  if (!s.cu) return Span{(int64_t)n * s.T, (int64_t)(n + 1) * s.T};
  int64_t a = s.cu[n], b = s.cu[n + 1];
  a = a < 0 ? 0 : (a > s.tokens ? s.tokens : a);
  b = b < a ? a : (b > s.tokens ? s.tokens : b);
  return Span{a, b};
}

// The last sequence n with first(n) <= t (empty sequences in front of the one
// that holds t are passed over).
__device__ __forceinline__ int seq_of(const Seqs &s, int64_t t) {
  if (!s.cu) return (int)(t / s.T);
  return find_seq(s.cu, s.N, t);
}

// The raw form of VEC elements (one, or 8 or 16 bytes of them).
template <int BYTES>
struct RawOf;
template <>
struct RawOf<16> {
  typedef uint4 type;
};
template <>
struct RawOf<8> {
  typedef uint2 type;
};

// VEC elements as floats.
template <typename E, int VEC>
struct Vec {
  float v[VEC];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = 0.f;
  }
  __device__ __forceinline__ void load(const E *p) {
    if constexpr (VEC == 1) {
      v[0] = to_f32(*p);
    } else {
      typedef typename RawOf<VEC * (int)sizeof(E)>::type R;
      const R r = *reinterpret_cast<const R *>(p);
      const E *e = reinterpret_cast<const E *>(&r);
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[i] = to_f32(e[i]);
    }
  }
  __device__ __forceinline__ void store(E *p) const {
    if constexpr (VEC == 1) {
      *p = from_f32<E>(v[0]);
    } else {
      typedef typename RawOf<VEC * (int)sizeof(E)>::type R;
      R r;
      E *e = reinterpret_cast<E *>(&r);
#pragma unroll
      for (int i = 0; i < VEC; ++i) e[i] = from_f32<E>(v[i]);
      *reinterpret_cast<R *>(p) = r;
    }
  }
};
// one raw load, converted later: a batch of these
// stays in flight without holding its fp32 form
template <typename E, int VEC>
struct Raw {
  E e[VEC];
  __device__ __forceinline__ void load(const E *p) {
    if constexpr (VEC == 1) {
      e[0] = *p;
    } else {
      typedef typename RawOf<VEC * (int)sizeof(E)>::type R;
      *reinterpret_cast<R *>(e) = *reinterpret_cast<const R *>(p);
    }
  }
  __device__ __forceinline__ Vec<E, VEC> f() const {
    Vec<E, VEC> r;
#pragma unroll
    for (int i = 0; i < VEC; ++i) r.v[i] = to_f32(e[i]);
    return r;
  }
} __attribute__((aligned(sizeof(E) * VEC)));

// 1 / (1 + exp(-z)): v_exp_f32 of a rounded -z log2(e) (off by |z| 2^-24) and
// v_rcp_f32; 0 and 1 at the ends, since exp(-z) runs to infinity and to 0.
__device__ __forceinline__ float sigmoidf(float z) {
  return __builtin_amdgcn_rcpf(1.f + __expf(-z));
}
// log(1 + exp(z)) = max(z, 0) + log1p(t), t = exp(-|z|): finite for every finite
// z and right to fp32's relative accuracy where it is small (the step sizes of
// a state-space layer begin at 0.001): an exponential of full accuracy, and
// log1p(t) = 2 artanh(s), s = t / (2 + t) <= 1/3, as its power series (nine
// terms leave 1e-10).  The hardware's exponential and logarithm left 7e-7 at
// 0.001, all of one sign.
__device__ __forceinline__ float softplusf(float z) {
  const float t = expf(-fabsf(z)), d = 2.f + t;
  float r = __builtin_amdgcn_rcpf(d);
  r = r * (2.f - d * r);
  const float s = t * r, q = s * s;
  float p = 1.f / 17.f;
#pragma unroll
  for (int n = 15; n >= 3; n -= 2) p = p * q + 1.f / (float)n;
  return fmaxf(z, 0.f) + 2.f * (s + s * q * p);
}

// a weight held in the problem's type or in fp32
__device__ __forceinline__ float load_w(const void *p, int64_t i, int wdtype) {
  return wdtype == 0 ? static_cast<const float *>(p)[i] : (float)static_cast<const bf16 *>(p)[i];
}
__device__ __forceinline__ void store_w(void *p, int64_t i, float v, int wdtype) {
  if (wdtype == 0)
    static_cast<float *>(p)[i] = v;
  else
    static_cast<bf16 *>(p)[i] = (bf16)v;
}

// VEC weights from column c on (1 or 0, `def`, without a weight)
template <int VEC>
__device__ __forceinline__ void load_ws(float (&r)[VEC], const void *p, int64_t c, int wdtype, float def) {
  if (!p) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) r[i] = def;
  } else if constexpr (VEC == 1) {
    r[0] = load_w(p, c, wdtype);
  } else if (wdtype == 0) {
#pragma unroll
    for (int i = 0; i < VEC; i += 4) {
      const f32x4 x = *reinterpret_cast<const f32x4 *>(static_cast<const float *>(p) + c + i);
#pragma unroll
      for (int j = 0; j < 4; ++j) r[i + j] = x[j];
    }
  } else {
#pragma unroll
    for (int i = 0; i < VEC; i += 4) {
      const bf16x4 x = *reinterpret_cast<const bf16x4 *>(static_cast<const bf16 *>(p) + c + i);
#pragma unroll
      for (int j = 0; j < 4; ++j) r[i + j] = (float)x[j];
    }
  }
}

// The W taps and the bias of VEC channels from c0 on ([D, W] and [D]), by
// channel.
template <int VEC, int W>
__device__ __forceinline__ void load_taps(float (&w)[W][VEC], float (&b)[VEC], const void *wp, const void *bp, int c0,
                                          int wdtype) {
  load_ws<VEC>(b, bp, c0, wdtype, 0.f);
  if constexpr (VEC == 1) {
#pragma unroll
    for (int j = 0; j < W; ++j) w[j][0] = load_w(wp, (int64_t)c0 * W + j, wdtype);
  } else {
    float t[VEC * W];
    load_ws<VEC * W>(t, wp, (int64_t)c0 * W, wdtype, 0.f);
#pragma unroll
    for (int i = 0; i < VEC; ++i)
#pragma unroll
      for (int j = 0; j < W; ++j) w[j][i] = t[i * W + j];
  }
}

// Sums of `n` columns over `parts` rows, in an order that does not depend on
// the launch: a workgroup of 512 has 32 columns, 16 rows at a time (a single
// thread a column takes a load's latency for every row: 234 us for 1024 rows
// of 256 columns), and joins its 16 sums in LDS.  put(column, sum).
constexpr int kSumThreads = 512;
__host__ __device__ inline unsigned sum_blocks(int64_t n) { return (unsigned)((n + 31) / 32); }
template <typename F>
__device__ __forceinline__ void sum_parts(const float *part, int64_t parts, int64_t n, F put) {
  __shared__ float red[16][32];
  const int col = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int64_t i = (int64_t)blockIdx.x * 32 + col;
  float v = 0.f;
  if (i < n) {
#pragma unroll 4
    for (int64_t p = g; p < parts; p += 16) v += part[p * n + i];
  }
  red[g][col] = v;
  __syncthreads();
  if (g == 0 && i < n) {
    v = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) v += red[k][col];
    put(i, v);
  }
}

}  // namespace gdn
