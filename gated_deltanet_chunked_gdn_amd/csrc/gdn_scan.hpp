// Segments, slots and the workspace of the selective scan's kernels.
#pragma once

#include "gdn_mixer.hpp"

namespace gdn {
namespace scan {

__host__ __device__ inline int64_t segs_of(const Span &sp, int seg) {
  const int64_t n = (sp.end - sp.first + seg - 1) / seg;
  return n > 0 ? n : 1;  // an empty sequence has one empty segment
}
// The first slot of sequence n.  Packed: first / seg + n, distinct without a
// table, since floor(x / seg) + n grows by at least ceil(len / seg) and at
// least 1 from one sequence to the next.
__host__ __device__ inline int64_t first_slot(const Seqs &s, const Span &sp, int n, int seg) {
  return s.cu ? sp.first / seg + n : (int64_t)n * segs_of(sp, seg);
}
// Slots of the whole batch.
inline int64_t slots_of(const Seqs &s, int seg) {
  return s.cu ? s.tokens / seg + s.N : s.N * segs_of(Span{0, s.T}, seg);
}

struct SlotLoc {
  int n;
  int64_t t0, t1;  // tokens of the segment
  int64_t index;   // of the segment in its sequence
  bool used, last;
};

// Byte offsets of the workspace's pieces (each at a 256-byte boundary).
struct Layout {
  size_t o_start = 0, o_decay = 0, o_zend = 0, o_a = 0, o_r = 0, o_ri = 0, o_half = 0, o_quarter = 0, o_m = 0, o_dd = 0, o_x = 0, o_head = 0,
         o_dc = 0, o_db = 0, o_ai = 0, o_shi = 0, o_slow = 0, o_z = 0, total = 0;
  int64_t chunks = 0;      // slots of 64-token chunks (bf16 backward)
  __host__ __device__ float *at(const ScanArgs &a, size_t o) const { return reinterpret_cast<float *>(a.ws + o); }
  __host__ __device__ bf16 *bat(const ScanArgs &a, size_t o) const { return reinterpret_cast<bf16 *>(a.ws + o); }
  // fp32 [slots][Hv][K][V]: a segment's state from zero, then its start state
  __host__ __device__ float *start(const ScanArgs &a) const { return at(a, o_start); }
  // [slots][Hv]: the sum of g over a segment
  __host__ __device__ float *decay(const ScanArgs &a) const { return at(a, o_decay); }
  // [slots][Hv][K][V]: the gradient of a segment's first state from its own
  // tokens, then of its last state from what follows
  __host__ __device__ float *zend(const ScanArgs &a) const { return at(a, o_zend); }
  // [slices (fp32: 1)][Hv][tokens] each: parts of the pairs inside token t's
  // quarter of a chunk that count for dg_t (bf16), of r_t and m_t
  __host__ __device__ float *a_part(const ScanArgs &a) const { return at(a, o_a); }
  __host__ __device__ float *r_part(const ScanArgs &a) const { return at(a, o_r); }
  __host__ __device__ float *m_part(const ScanArgs &a) const { return at(a, o_m); }
  // bf16, the same: a_t, and what of r_t comes from the gradient of the state
  // leaving the chunk
  __host__ __device__ float *ai_part(const ScanArgs &a) const { return at(a, o_ai); }
  __host__ __device__ float *ri_part(const ScanArgs &a) const { return at(a, o_ri); }
  // and the pairs of tokens from both halves of a chunk, by the earlier token (in
  // r) in the first half, by the later in the second; from both quarters of a half
  // likewise
  __host__ __device__ float *half_part(const ScanArgs &a) const { return at(a, o_half); }
  __host__ __device__ float *quarter_part(const ScanArgs &a) const { return at(a, o_quarter); }
  // parts of dD: [slices][slots, bf16: chunks][Hv]
  __host__ __device__ float *dd_part(const ScanArgs &a) const { return at(a, o_dd); }
  // [slices][chunks][Hv]: parts of 2^{gamma_L} <S, Z>, S entering the chunk, Z
  // of the state leaving it (bf16)
  __host__ __device__ float *x_part(const ScanArgs &a) const { return at(a, o_x); }
  // [slots or chunks][Hv][3]: parts of dA, ddt_bias, dD
  __host__ __device__ float *head_part(const ScanArgs &a) const { return at(a, o_head); }
  // fp32 problems, [tokens][Hv][K] each: the heads' parts of dc and db
  __host__ __device__ float *dc_part(const ScanArgs &a) const { return at(a, o_dc); }
  __host__ __device__ float *db_part(const ScanArgs &a) const { return at(a, o_db); }
  // bf16 problems, [chunks][Hv][V / 32][K / 16][64][8] each: the state entering
  // a chunk as bf16 and as the lower 16 bits of its fp32 form (split_halves), and
  // the gradient of the state leaving it.  Piece
  // (s, lane) holds rows 16 s + rho(lane >> 5, e) of column lane & 31: what a
  // lane of the passes has in its accumulators, 1 KB a store.
  __host__ __device__ bf16 *s_hi(const ScanArgs &a) const { return bat(a, o_shi); }
  __host__ __device__ bf16 *s_low(const ScanArgs &a) const { return bat(a, o_slow); }
  __host__ __device__ bf16 *z(const ScanArgs &a) const { return bat(a, o_z); }
  // slot of chunk c of a segment
  __device__ int64_t chunk(const ScanArgs &a, const SlotLoc &l, int c) const {
    return first_slot(a.s, seq_span(a.s, l.n), l.n, 64) + l.index * (a.seg / 64) + c;
  }
};

inline Layout layout(const ScanArgs &a, bool bwd) {
  Layout w;
  size_t off = 0;
  auto piece = [&](size_t bytes) {
    const size_t o = off;
    off = (off + bytes + 255) & ~(size_t)255;
    return o;
  };
  const size_t heads = (size_t)a.slots * a.Hv, kv = (size_t)a.K * a.V;
  const size_t tok = (size_t)a.s.tokens * a.Hv;
  if (!a.one_seg) {
    w.o_start = piece(heads * kv * 4);
    w.o_decay = piece(heads * 4);
  }
  if (bwd && !a.one_seg) w.o_zend = piece(heads * kv * 4);
  if (bwd && a.dtype != 1) {
    w.o_r = piece(tok * 4);
    w.o_m = piece(tok * 4);
    w.o_dd = piece(heads * 4);
    w.o_head = piece(heads * 3 * 4);
    w.o_dc = piece(tok * a.K * 4);
    w.o_db = piece(tok * a.K * 4);
  }
  if (bwd && a.dtype == 1) {
    const size_t slices = a.V / 32;
    w.chunks = slots_of(a.s, 64);
    const size_t ch = (size_t)w.chunks * a.Hv;
    w.o_a = piece(tok * slices * 4);
    w.o_r = piece(tok * slices * 4);
    w.o_m = piece(tok * slices * 4);
    w.o_ai = piece(tok * slices * 4);
    w.o_ri = piece(tok * slices * 4);
    w.o_half = piece(tok * slices * 4);
    w.o_quarter = piece(tok * slices * 4);
    w.o_dd = piece(ch * slices * 4);
    w.o_x = piece(ch * slices * 4);
    w.o_head = piece(ch * 3 * 4);
    w.o_shi = piece(ch * kv * 2);
    w.o_slow = piece(ch * kv * 2);
    w.o_z = piece(ch * kv * 2);
  }
  w.total = off ? off : 256;
  return w;
}

// Column slices of a head group that a workgroup of the matrix kernels has.
// Eight hold a compute unit; with four, two workgroups of them, c and b come
// in twice (8192 tokens x 64 heads, with the updates in two parts: out pass 71
// us against 68, the backward's passes from zero 78 against 70).
inline int slices_per_block(int per) { return per % 8 == 0 ? 8 : per % 4 == 0 ? 4 : per % 2 == 0 ? 2 : 1; }
// bf16, gdn_scan_mma.hip
hipError_t launch_mma_local(const ScanArgs &a, const Layout &w, hipStream_t st);
hipError_t launch_mma_out(const ScanArgs &a, const Layout &w, hipStream_t st);
hipError_t launch_mma_states(const ScanArgs &a, const Layout &w, hipStream_t st);
hipError_t launch_mma_locals(const ScanArgs &a, const Layout &w, hipStream_t st);
// bf16, gdn_scan_bwd.hip
hipError_t launch_mma_grad(const ScanArgs &a, const Layout &w, hipStream_t st);

// Lane 0 the last token: the sum of v from a lane's token on, and over the
// tokens before it.
__device__ __forceinline__ double sum_upto(double v, int lane) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const double o = __shfl_up(v, d);
    if (lane >= d) v += o;
  }
  return v;
}
__device__ __forceinline__ double sum_before(double v, int lane) {
  v = __shfl_down(v, 1);
  if (lane == 63) v = 0.;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const double o = __shfl_down(v, d);
    if (lane + d < 64) v += o;
  }
  return v;
}
__device__ __forceinline__ double wave_sum64(double v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
  return v;
}

__device__ __forceinline__ SlotLoc locate(const ScanArgs &a, int64_t slot) {
  int lo = 0, hi = a.s.N - 1;
  if (!a.s.cu) {
    lo = (int)(slot / segs_of(Span{0, a.s.T}, a.seg));
  } else {
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (first_slot(a.s, seq_span(a.s, mid), mid, a.seg) <= slot)
        lo = mid;
      else
        hi = mid - 1;
    }
  }
  const Span sp = seq_span(a.s, lo);
  const int64_t s = slot - first_slot(a.s, sp, lo, a.seg), ns = segs_of(sp, a.seg);
  SlotLoc l;
  l.n = lo;
  l.used = s >= 0 && s < ns;
  l.index = s;
  l.last = s == ns - 1;
  l.t0 = sp.first + s * a.seg;
  l.t1 = l.t0 + a.seg < sp.end ? l.t0 + a.seg : sp.end;
  return l;
}

}  // namespace scan
}  // namespace gdn
