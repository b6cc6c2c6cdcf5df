// Segments, slots and the workspace of the selective scan's kernels.
#pragma once

#include "gdn_mixer.hpp"

namespace gdn {
namespace scan {

// Byte offsets of the workspace's pieces (each at a 256-byte boundary).
struct Layout {
  size_t o_start = 0, o_decay = 0, o_zend = 0, o_hend = 0, o_a = 0, o_r = 0, o_m = 0, o_dd = 0, o_head = 0, o_dc = 0, o_db = 0,
         total = 0;
  bool need_last = false;  // the local pass runs a sequence's last segment too
  __host__ __device__ float *at(const ScanArgs &a, size_t o) const { return reinterpret_cast<float *>(a.ws + o); }
  // fp32 [slots][Hv][K][V]: a segment's state from zero, then its start state
  __host__ __device__ float *start(const ScanArgs &a) const { return at(a, o_start); }
  // [slots][Hv]: the sum of g over a segment
  __host__ __device__ float *decay(const ScanArgs &a) const { return at(a, o_decay); }
  // [slots][Hv][K][V]: the gradient of a segment's first state from its own
  // tokens, then of its last state from what follows
  __host__ __device__ float *zend(const ScanArgs &a) const { return at(a, o_zend); }
  // [N][Hv][K][V]: a sequence's last state
  __host__ __device__ float *hend(const ScanArgs &a) const { return at(a, o_hend); }
  // [slices][Hv][tokens] each: parts of a_t, r_t and m_t
  __host__ __device__ float *a_part(const ScanArgs &a) const { return at(a, o_a); }
  __host__ __device__ float *r_part(const ScanArgs &a) const { return at(a, o_r); }
  __host__ __device__ float *m_part(const ScanArgs &a) const { return at(a, o_m); }
  // [slices][slots][Hv]: parts of dD; [slots][Hv][3]: of dA, ddt_bias, dD
  __host__ __device__ float *dd_part(const ScanArgs &a) const { return at(a, o_dd); }
  __host__ __device__ float *head_part(const ScanArgs &a) const { return at(a, o_head); }
  // [tokens][Hv][K] each: the heads' parts of dc and db
  __host__ __device__ float *dc_part(const ScanArgs &a) const { return at(a, o_dc); }
  __host__ __device__ float *db_part(const ScanArgs &a) const { return at(a, o_db); }
};

inline Layout layout(const ScanArgs &a, bool bwd) {
  Layout w;
  size_t off = 0;
  auto piece = [&](size_t floats) {
    const size_t o = off;
    off = (off + floats * 4 + 255) & ~(size_t)255;
    return o;
  };
  const size_t heads = (size_t)a.slots * a.Hv, kv = (size_t)a.K * a.V;
  const size_t tok = (size_t)a.s.tokens * a.Hv;
  if (!a.one_seg) {
    w.o_start = piece(heads * kv);
    w.o_decay = piece(heads);
  }
  if (bwd) {
    w.o_zend = piece(heads * kv);
    w.o_hend = piece((size_t)a.s.N * a.Hv * kv);
    w.o_a = piece(tok * ((a.K + 63) / 64));
    w.o_r = piece(tok * ((a.V + 63) / 64));
    w.o_m = piece(tok * ((a.V + 63) / 64));
    w.o_dd = piece(heads * ((a.V + 63) / 64));
    w.o_head = piece(heads * 3);
    w.o_dc = piece(tok * a.K);
    w.o_db = piece(tok * a.K);
  }
  w.need_last = bwd;
  w.total = off ? off : 256;
  return w;
}

// Column slices of a head group that a workgroup of the matrix kernels has.
inline int slices_per_block(int per) { return per % 8 == 0 ? 8 : per % 4 == 0 ? 4 : per % 2 == 0 ? 2 : 1; }
// bf16, gdn_scan_mma.hip
hipError_t launch_mma_local(const ScanArgs &a, const Layout &w, hipStream_t st);
hipError_t launch_mma_out(const ScanArgs &a, const Layout &w, hipStream_t st);

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

struct SlotLoc {
  int n;
  int64_t t0, t1;  // tokens of the segment
  bool used, last;
};
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
  l.last = s == ns - 1;
  l.t0 = sp.first + s * a.seg;
  l.t1 = l.t0 + a.seg < sp.end ? l.t0 + a.seg : sp.end;
  return l;
}

}  // namespace scan
}  // namespace gdn
