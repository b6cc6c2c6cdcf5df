// C ABI of the sequence-mixer operators: argument validation and kernel
// dispatch.  All checks run before any HIP launch.
#include <cstdint>

#include "../../include/gdn.h"
#include "gdn_internal.h"
#include "gdn_mixer.h"

namespace {

using gdn::set_error;

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }
size_t elem(int dtype) { return dtype == GDN_BF16 ? 2 : 4; }
bool known(int dtype) { return dtype == GDN_F32 || dtype == GDN_BF16; }

// Sequences of a packed or plain batch; the host copy is checked if given.
int check_seqs(int B, int T, int N, const int32_t *cu, const int32_t *host) {
  if (!cu) {
    if (host) return set_error(GDN_ERR_INVALID_ARG, "cu_seqlens_host given without cu_seqlens");
    if (N != B)
      return set_error(GDN_ERR_INVALID_ARG, "N must equal B without cu_seqlens (N=%d B=%d)", N, B);
    return GDN_OK;
  }
  if (B != 1) return set_error(GDN_ERR_INVALID_ARG, "B must be 1 with cu_seqlens (got %d)", B);
  if (N <= 0) return set_error(GDN_ERR_INVALID_ARG, "N must be positive (got %d)", N);
  if (!host) return GDN_OK;
  if (host[0] != 0) return set_error(GDN_ERR_INVALID_ARG, "cu_seqlens[0] = %d, must be 0", host[0]);
  for (int n = 0; n < N; ++n)
    if (host[n + 1] < host[n])
      return set_error(GDN_ERR_INVALID_ARG, "cu_seqlens decreases at %d (%d -> %d)", n, host[n], host[n + 1]);
  if (host[N] != T) return set_error(GDN_ERR_INVALID_ARG, "cu_seqlens[N] = %d but T = %d", host[N], T);
  return GDN_OK;
}

int hip(hipError_t e, const char *what) {
  if (e == hipSuccess) return GDN_OK;
  return set_error(GDN_ERR_HIP, "%s launch failed: %s", what, hipGetErrorString(e));
}

int check_ws(const void *ws, size_t have, size_t need) {
  if (!ws || have < need)
    return set_error(GDN_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, ws ? have : (size_t)0);
  if (!aligned(ws, 256)) return set_error(GDN_ERR_WORKSPACE, "workspace not 256-byte aligned");
  return GDN_OK;
}

int check_slots(const int32_t *idx, int slots, int B) {
  if (slots <= 0 || (!idx && slots < B))
    return set_error(GDN_ERR_INVALID_ARG, "%d state slots for %d batch rows", slots, B);
  if (!aligned(idx, 4)) return set_error(GDN_ERR_LAYOUT, "state_indices must be 4-byte aligned");
  return GDN_OK;
}

constexpr int64_t kGrid = (int64_t)1 << 31;  // workgroups of a launch

// A step has a wave for 32 columns of a row's head, up to four a workgroup (and a
// launch has fewer than 2^32 threads).
bool step_fits(int B, int Hv, int V) { return (double)B * Hv * (V / 32) <= (double)((1 << 26) - 4); }

// ---- convolution
int check_conv(const gdn_conv_t *p, gdn::ConvArgs *a) {
  if (!p) return set_error(GDN_ERR_INVALID_ARG, "problem descriptor is NULL");
  if (p->B <= 0 || p->T < 0 || p->D <= 0)
    return set_error(GDN_ERR_INVALID_ARG, "dimensions must be positive (B=%d T=%d D=%d)", p->B, p->T, p->D);
  if (p->W < 2 || p->W > 4)
    return set_error(GDN_ERR_UNSUPPORTED, "W=%d taps: 2, 3 and 4 are supported", p->W);
  if (!known(p->dtype)) return set_error(GDN_ERR_UNSUPPORTED, "dtype %d is not GDN_F32 or GDN_BF16", p->dtype);
  if (p->weight_dtype != GDN_F32 && p->weight_dtype != p->dtype)
    return set_error(GDN_ERR_UNSUPPORTED, "weight_dtype %d is neither fp32 nor the problem's", p->weight_dtype);
  if (p->silu != 0 && p->silu != 1) return set_error(GDN_ERR_INVALID_ARG, "silu must be 0 or 1 (got %d)", p->silu);
  const int64_t xs = p->x_stride ? p->x_stride : p->D;
  if (xs < p->D) return set_error(GDN_ERR_INVALID_ARG, "x_stride %lld below D = %d", (long long)xs, p->D);
  const int rc = check_seqs(p->B, p->T, p->N, p->cu_seqlens, p->cu_seqlens_host);
  if (rc != GDN_OK) return rc;
  const int64_t tokens = (int64_t)p->B * p->T;
  // (channel indices are 32-bit, the last workgroup's among them: up to 1024 channels each)
  if (p->D > INT32_MAX - 1023 || tokens >= kGrid || ((tokens + 7) / 8 + p->N) * (((int64_t)p->D + 31) / 32) >= kGrid)
    return set_error(GDN_ERR_UNSUPPORTED, "problem too large for the launch grid");
  *a = gdn::ConvArgs{};
  a->s = gdn::Seqs{p->cu_seqlens, p->cu_seqlens ? p->N : p->B, p->T, tokens};
  a->D = p->D;
  a->W = p->W;
  a->dtype = p->dtype;
  a->wdtype = p->weight_dtype;
  a->silu = p->silu;
  a->xs = xs;
  return GDN_OK;
}

// The sums over the tokens' parts take 16 threads a column
// (and a launch has fewer than 2^32 threads)
int check_conv_bwd(const gdn_conv_t *p, gdn::ConvArgs *a) {
  const int rc = check_conv(p, a);
  if (rc == GDN_OK && (int64_t)(p->W + 1) * p->D >= ((int64_t)1 << 28))
    return set_error(GDN_ERR_UNSUPPORTED, "problem too large for the launch grid");
  return rc;
}
size_t conv_bwd_bytes(const gdn::ConvArgs &a) {
  const size_t n = (size_t)gdn::conv_bwd_tiles(a.s.tokens, a.D) * (a.W + 1) * a.D * 4;
  return n ? n : 256;
}

// ---- scan
int check_scan(const gdn_scan_t *p, bool step, gdn::ScanArgs *a) {
  if (!p) return set_error(GDN_ERR_INVALID_ARG, "problem descriptor is NULL");
  if (p->B <= 0 || p->T < 0 || p->Hq <= 0 || p->Hv <= 0 || p->K <= 0 || p->V <= 0)
    return set_error(GDN_ERR_INVALID_ARG, "dimensions must be positive (B=%d T=%d Hq=%d Hv=%d K=%d V=%d)", p->B,
                     p->T, p->Hq, p->Hv, p->K, p->V);
  if (!known(p->dtype)) return set_error(GDN_ERR_UNSUPPORTED, "dtype %d is not GDN_F32 or GDN_BF16", p->dtype);
  if (p->Hv % p->Hq != 0)
    return set_error(GDN_ERR_UNSUPPORTED, "Hv=%d is not a multiple of Hq=%d", p->Hv, p->Hq);
  const int most = p->dtype == GDN_BF16 || step ? 128 : 64;
  auto ok = [most](int d) { return d == 32 || d == 64 || (d == 128 && most == 128); };
  if (!ok(p->K) || !ok(p->V))
    return set_error(GDN_ERR_UNSUPPORTED, "K=%d V=%d not supported: 32, 64%s", p->K, p->V,
                     most == 128 ? " and 128 are" : " are in fp32");
  if (p->dt_softplus != 0 && p->dt_softplus != 1)
    return set_error(GDN_ERR_INVALID_ARG, "dt_softplus must be 0 or 1 (got %d)", p->dt_softplus);
  if (step && (p->T != 1 || p->cu_seqlens))
    return set_error(GDN_ERR_INVALID_ARG, "a step has T = 1 and no cu_seqlens (T=%d)", p->T);
  const int rc = check_seqs(p->B, p->T, p->N, p->cu_seqlens, p->cu_seqlens_host);
  if (rc != GDN_OK) return rc;
  const int64_t qs = (int64_t)p->Hq * p->K, vs = (int64_t)p->Hv * p->V;
  const int64_t cs = p->c_stride ? p->c_stride : qs, bs = p->b_stride ? p->b_stride : qs,
                xs = p->x_stride ? p->x_stride : vs;
  if (cs < qs || bs < qs || xs < vs)
    return set_error(GDN_ERR_INVALID_ARG, "a stride is below its row (c %lld b %lld x %lld)", (long long)cs,
                     (long long)bs, (long long)xs);
  const int64_t per = 16 / (int64_t)elem(p->dtype);
  // (the scan's kernels address 64 rows by 32-bit byte offsets, the step's one row by itself)
  constexpr int64_t kRow = (int64_t)1 << 24;
  if (!step && (cs >= kRow || bs >= kRow || xs >= kRow))
    return set_error(GDN_ERR_UNSUPPORTED, "c, b and x rows must lie less than 2^24 elements apart");
  if (cs % per || bs % per || xs % per)
    return set_error(GDN_ERR_LAYOUT, "c, b and x strides must be multiples of 16 bytes");
  const int64_t tokens = (int64_t)p->B * p->T;
  if (tokens * (p->Hv > p->Hq ? p->Hv : p->Hq) * 128 > ((int64_t)1 << 40) ||
      (tokens / 16 + p->N) * p->Hv * 4 >= kGrid || (step && !step_fits(p->B, p->Hv, p->V)))
    return set_error(GDN_ERR_UNSUPPORTED, "problem too large");
  *a = gdn::ScanArgs{};
  a->s = gdn::Seqs{p->cu_seqlens, p->cu_seqlens ? p->N : p->B, p->T, tokens};
  a->Hq = p->Hq;
  a->Hv = p->Hv;
  a->K = p->K;
  a->V = p->V;
  a->dtype = p->dtype;
  a->softplus = p->dt_softplus;
  a->cs = cs;
  a->bs = bs;
  a->xs = xs;
  return GDN_OK;
}

// ---- norm
int check_norm(const gdn_norm_t *p, gdn::NormArgs *a) {
  if (!p) return set_error(GDN_ERR_INVALID_ARG, "problem descriptor is NULL");
  if (p->rows < 0 || p->D <= 0)
    return set_error(GDN_ERR_INVALID_ARG, "dimensions must be positive (rows=%lld D=%d)", (long long)p->rows, p->D);
  if (!known(p->dtype)) return set_error(GDN_ERR_UNSUPPORTED, "dtype %d is not GDN_F32 or GDN_BF16", p->dtype);
  if (p->weight_dtype != GDN_F32 && p->weight_dtype != p->dtype)
    return set_error(GDN_ERR_UNSUPPORTED, "weight_dtype %d is neither fp32 nor the problem's", p->weight_dtype);
  if (p->rms != 0 && p->rms != 1) return set_error(GDN_ERR_INVALID_ARG, "rms must be 0 or 1 (got %d)", p->rms);
  if (!(p->eps >= 0)) return set_error(GDN_ERR_INVALID_ARG, "eps must not be negative");
  if (p->rows >= kGrid || p->D > (1 << 24)) return set_error(GDN_ERR_UNSUPPORTED, "problem too large");
  *a = gdn::NormArgs{};
  a->rows = p->rows;
  a->D = p->D;
  a->dtype = p->dtype;
  a->wdtype = p->weight_dtype;
  a->rms = p->rms;
  a->eps = p->eps;
  return GDN_OK;
}

// ---- linear attention
int check_attn(const gdn_attn_t *p, bool step, bool bwd, gdn::AttnArgs *a) {
  if (!p) return set_error(GDN_ERR_INVALID_ARG, "problem descriptor is NULL");
  if (p->B <= 0 || p->T < 0 || p->Hq <= 0 || p->Hv <= 0 || p->K <= 0 || p->V <= 0)
    return set_error(GDN_ERR_INVALID_ARG, "dimensions must be positive (B=%d T=%d Hq=%d Hv=%d K=%d V=%d)", p->B,
                     p->T, p->Hq, p->Hv, p->K, p->V);
  if (!known(p->dtype)) return set_error(GDN_ERR_UNSUPPORTED, "dtype %d is not GDN_F32 or GDN_BF16", p->dtype);
  if (p->Hv % p->Hq != 0)
    return set_error(GDN_ERR_UNSUPPORTED, "Hv=%d is not a multiple of Hq=%d", p->Hv, p->Hq);
  auto ok = [](int d) { return d == 32 || d == 64 || d == 128; };
  if (!ok(p->K) || !ok(p->V))
    return set_error(GDN_ERR_UNSUPPORTED, "K=%d V=%d not supported: 32, 64 and 128 are", p->K, p->V);
  if (!(p->scale == p->scale)) return set_error(GDN_ERR_INVALID_ARG, "scale is NaN");
  if (step && (p->T != 1 || p->cu_seqlens))
    return set_error(GDN_ERR_INVALID_ARG, "a step has T = 1 and no cu_seqlens (T=%d)", p->T);
  const int rc = check_seqs(p->B, p->T, p->N, p->cu_seqlens, p->cu_seqlens_host);
  if (rc != GDN_OK) return rc;
  const int64_t qw = (int64_t)p->Hq * p->K, vw = (int64_t)p->Hv * p->V;
  const int64_t qs = p->q_stride ? p->q_stride : qw, ks = p->k_stride ? p->k_stride : qw,
                vs = p->v_stride ? p->v_stride : vw;
  if (qs < qw || ks < qw || vs < vw)
    return set_error(GDN_ERR_INVALID_ARG, "a stride is below its row (q %lld k %lld v %lld)", (long long)qs,
                     (long long)ks, (long long)vs);
  const int64_t per = 16 / (int64_t)elem(p->dtype);
  // (the passes address a chunk's rows, contiguous ones among them, by 32-bit
  // byte offsets, the step its one row by itself)
  constexpr int64_t kRow = (int64_t)1 << 24;
  if (!step && (qs >= kRow || ks >= kRow || vs >= kRow || (int64_t)p->Hv * p->K >= kRow))
    return set_error(GDN_ERR_UNSUPPORTED, "q, k and v rows must lie less than 2^24 elements apart");
  if (qs % per || ks % per || vs % per)
    return set_error(GDN_ERR_LAYOUT, "q, k and v strides must be multiples of 16 bytes");
  *a = gdn::AttnArgs{};
  a->s = gdn::Seqs{p->cu_seqlens, p->cu_seqlens ? p->N : p->B, p->T, (int64_t)p->B * p->T};
  a->Hq = p->Hq;
  a->Hv = p->Hv;
  a->K = p->K;
  a->V = p->V;
  a->dtype = p->dtype;
  a->scale = p->scale;
  a->qs = qs;
  a->ks = ks;
  a->vs = vs;
  a->longest = p->T;
  a->known = !p->cu_seqlens || p->cu_seqlens_host;
  if (p->cu_seqlens_host) {
    a->longest = 0;
    for (int n = 0; n < p->N; ++n) {
      const int64_t len = (int64_t)p->cu_seqlens_host[n + 1] - p->cu_seqlens_host[n];
      if (len > a->longest) a->longest = len;
    }
  }
  // (a launch has fewer than 2^32 threads: up to twelve workgroups of 768 a
  // slot and head, two threads for four elements of a state, one for four of dq)
  constexpr int64_t kBlocks = (int64_t)1 << 24;
  const int64_t heads = (int64_t)p->Hv * (step ? 0 : gdn::attn_plan(*a, bwd).slots);
  if (a->s.tokens * p->Hv * 128 > ((int64_t)1 << 40) || (int64_t)a->s.N * p->Hv >= kGrid || heads * 36 >= kBlocks ||
      (step && !step_fits(p->B, p->Hv, p->V)) ||
      (!step && ((int64_t)a->s.N * p->Hv * p->K * p->V / 512 >= kBlocks || (bwd && a->s.tokens * p->Hq * p->K / 1024 >= kBlocks))))
    return set_error(GDN_ERR_UNSUPPORTED, "problem too large");
  return GDN_OK;
}

// ---- group norm
int check_group(const gdn_group_t *p, bool bwd, gdn::GroupArgs *a) {
  if (!p) return set_error(GDN_ERR_INVALID_ARG, "problem descriptor is NULL");
  if (p->N < 0 || p->S <= 0 || p->G <= 0 || p->Dg <= 0)
    return set_error(GDN_ERR_INVALID_ARG, "dimensions must be positive (N=%lld S=%lld G=%d Dg=%d)", (long long)p->N,
                     (long long)p->S, p->G, p->Dg);
  if (!known(p->dtype)) return set_error(GDN_ERR_UNSUPPORTED, "dtype %d is not GDN_F32 or GDN_BF16", p->dtype);
  if (p->weight_dtype != GDN_F32 && p->weight_dtype != p->dtype)
    return set_error(GDN_ERR_UNSUPPORTED, "weight_dtype %d is neither fp32 nor the problem's", p->weight_dtype);
  if (p->silu != 0 && p->silu != 1) return set_error(GDN_ERR_INVALID_ARG, "silu must be 0 or 1 (got %d)", p->silu);
  if (!(p->eps >= 0)) return set_error(GDN_ERR_INVALID_ARG, "eps must not be negative");
  if ((int64_t)p->G * p->Dg >= (1 << 24) || p->S >= kGrid || p->N >= kGrid || p->N * p->G >= kGrid ||
      (double)p->N * (double)p->S * p->G * p->Dg >= 1e12)
    return set_error(GDN_ERR_UNSUPPORTED, "problem too large");
  *a = gdn::GroupArgs{};
  a->N = p->N;
  a->S = p->S;
  a->G = p->G;
  a->Dg = p->Dg;
  a->dtype = p->dtype;
  a->wdtype = p->weight_dtype;
  a->silu = p->silu;
  a->eps = p->eps;
  if (!gdn::group_fits(*a, bwd)) return set_error(GDN_ERR_UNSUPPORTED, "problem too large for the launch grid");
  return GDN_OK;
}

}  // namespace

extern "C" {

int gdn_causal_conv_fwd(const gdn_conv_t *p, const void *x, const void *weight, const void *bias,
                        const void *h0, void *y, void *ht, void *stream) {
  gdn::clear_error();
  gdn::ConvArgs a;
  const int rc = check_conv(p, &a);
  if (rc != GDN_OK) return rc;
  if (!weight || (a.s.tokens > 0 && (!x || !y)))
    return set_error(GDN_ERR_INVALID_ARG, "x, weight and y are required");
  const size_t e = elem(p->dtype), we = elem(p->weight_dtype);
  if (!aligned(x, e) || !aligned(y, e) || !aligned(h0, e) || !aligned(ht, e) || !aligned(weight, we) || !aligned(bias, we))
    return set_error(GDN_ERR_LAYOUT, "a buffer is not aligned to its elements");
  a.x = x;
  a.w = weight;
  a.bias = bias;
  a.h0 = h0;
  a.y = y;
  a.ht = ht;
  return hip(gdn::launch_conv_fwd(a, static_cast<hipStream_t>(stream)), "convolution");
}

size_t gdn_causal_conv_bwd_workspace_size(const gdn_conv_t *p) {
  gdn::clear_error();
  gdn::ConvArgs a;
  return check_conv_bwd(p, &a) == GDN_OK ? conv_bwd_bytes(a) : 0;
}

int gdn_causal_conv_bwd(const gdn_conv_t *p, const void *x, const void *weight, const void *bias, const void *dy,
                        const void *h0, const void *dht, void *dx, void *dweight, void *dbias, void *dh0,
                        void *workspace, size_t ws_bytes, void *stream) {
  gdn::clear_error();
  gdn::ConvArgs a;
  int rc = check_conv_bwd(p, &a);
  if (rc != GDN_OK) return rc;
  if (!weight || !dweight || (a.s.tokens > 0 && (!x || !dy || !dx)))
    return set_error(GDN_ERR_INVALID_ARG, "x, weight, dy, dx and dweight are required");
  if (dbias && !bias) return set_error(GDN_ERR_INVALID_ARG, "dbias given without bias");
  const size_t e = elem(p->dtype), we = elem(p->weight_dtype);
  if (!aligned(x, e) || !aligned(dy, e) || !aligned(h0, e) || !aligned(dht, e) || !aligned(dx, e) || !aligned(dh0, e) ||
      !aligned(weight, we) || !aligned(bias, we) || !aligned(dweight, we) || !aligned(dbias, we))
    return set_error(GDN_ERR_LAYOUT, "a buffer is not aligned to its elements");
  if ((rc = check_ws(workspace, ws_bytes, conv_bwd_bytes(a))) != GDN_OK) return rc;
  a.x = x;
  a.w = weight;
  a.bias = bias;
  a.dy = dy;
  a.h0 = h0;
  a.dht = dht;
  a.dx = dx;
  a.dw = dweight;
  a.db = dbias;
  a.dh0 = dh0;
  a.partial = static_cast<float *>(workspace);
  return hip(gdn::launch_conv_bwd(a, static_cast<hipStream_t>(stream)), "convolution backward");
}

int gdn_causal_conv_step(const gdn_conv_t *p, const void *x, void *state, const void *weight, const void *bias,
                         const int32_t *state_indices, int32_t slots, void *y, void *stream) {
  gdn::clear_error();
  gdn::ConvArgs c;
  int rc = check_conv(p, &c);
  if (rc != GDN_OK) return rc;
  if (p->T != 1 || p->cu_seqlens)
    return set_error(GDN_ERR_INVALID_ARG, "a step has T = 1 and no cu_seqlens (T=%d)", p->T);
  if (!x || !state || !weight || !y) return set_error(GDN_ERR_INVALID_ARG, "x, state, weight and y are required");
  if ((rc = check_slots(state_indices, slots, p->B)) != GDN_OK) return rc;
  const size_t e = elem(p->dtype), we = elem(p->weight_dtype);
  if (!aligned(x, e) || !aligned(y, e) || !aligned(state, e) || !aligned(weight, we) || !aligned(bias, we))
    return set_error(GDN_ERR_LAYOUT, "a buffer is not aligned to its elements");
  gdn::ConvStepArgs a{p->B, p->D, p->W, p->dtype, p->weight_dtype, p->silu, slots, c.xs,
                      x,    weight, bias, state,    y,               state_indices};
  return hip(gdn::launch_conv_step(a, static_cast<hipStream_t>(stream)), "convolution step");
}

size_t gdn_selective_scan_fwd_workspace_size(const gdn_scan_t *p) {
  gdn::clear_error();
  gdn::ScanArgs a;
  return check_scan(p, false, &a) == GDN_OK ? gdn::scan_plan(a, false).ws : 0;
}
size_t gdn_selective_scan_bwd_workspace_size(const gdn_scan_t *p) {
  gdn::clear_error();
  gdn::ScanArgs a;
  return check_scan(p, false, &a) == GDN_OK ? gdn::scan_plan(a, true).ws : 0;
}

int gdn_selective_scan_fwd(const gdn_scan_t *p, const void *c, const void *b, const void *x, const void *dt,
                           const float *A, const float *D, const float *dt_bias, const float *h0, void *y, float *ht,
                           void *workspace, size_t ws_bytes, void *stream) {
  gdn::clear_error();
  gdn::ScanArgs a;
  int rc = check_scan(p, false, &a);
  if (rc != GDN_OK) return rc;
  if (!A || (a.s.tokens > 0 && (!c || !b || !x || !dt || !y)))
    return set_error(GDN_ERR_INVALID_ARG, "c, b, x, dt, A and y are required");
  if (!aligned(c, 16) || !aligned(b, 16) || !aligned(x, 16) || !aligned(y, 16) || !aligned(h0, 16) || !aligned(ht, 16) ||
      !aligned(dt, elem(p->dtype)) || !aligned(A, 4) || !aligned(D, 4) || !aligned(dt_bias, 4))
    return set_error(GDN_ERR_LAYOUT, "c, b, x, y and the states must be 16-byte aligned; the rest to their elements");
  const gdn::ScanPlan pl = gdn::scan_plan(a, false);
  if ((rc = check_ws(workspace, ws_bytes, pl.ws)) != GDN_OK) return rc;
  a.seg = pl.seg;
  a.slots = pl.slots;
  a.one_seg = pl.one_seg;
  a.c = c;
  a.b = b;
  a.x = x;
  a.dt = dt;
  a.A = A;
  a.D = D;
  a.dt_bias = dt_bias;
  a.h0 = h0;
  a.y = y;
  a.ht = ht;
  a.ws = static_cast<char *>(workspace);
  return hip(gdn::launch_scan_fwd(a, static_cast<hipStream_t>(stream)), "scan");
}

int gdn_selective_scan_bwd(const gdn_scan_t *p, const void *c, const void *b, const void *x, const void *dt,
                           const float *A, const float *D, const float *dt_bias, const float *h0, const void *dy,
                           const float *dht, void *dc, void *db, void *dx, void *ddt, float *dA, float *dD,
                           float *ddt_bias, float *dh0, void *workspace, size_t ws_bytes, void *stream) {
  gdn::clear_error();
  gdn::ScanArgs a;
  int rc = check_scan(p, false, &a);
  if (rc != GDN_OK) return rc;
  if (!A || !dA || (a.s.tokens > 0 && (!c || !b || !x || !dt || !dy || !dc || !db || !dx || !ddt)))
    return set_error(GDN_ERR_INVALID_ARG, "c, b, x, dt, A, dy, dc, db, dx, ddt and dA are required");
  if (!aligned(c, 16) || !aligned(b, 16) || !aligned(x, 16) || !aligned(dy, 16) || !aligned(dc, 16) || !aligned(db, 16) ||
      !aligned(dx, 16) || !aligned(h0, 16) || !aligned(dht, 16) || !aligned(dh0, 16) || !aligned(dt, elem(p->dtype)) ||
      !aligned(ddt, elem(p->dtype)) || !aligned(A, 4) || !aligned(D, 4) || !aligned(dt_bias, 4) || !aligned(dA, 4) ||
      !aligned(dD, 4) || !aligned(ddt_bias, 4))
    return set_error(GDN_ERR_LAYOUT,
                     "c, b, x, dy, dc, db, dx and the states must be 16-byte aligned; the rest to their elements");
  const gdn::ScanPlan pl = gdn::scan_plan(a, true);
  if ((rc = check_ws(workspace, ws_bytes, pl.ws)) != GDN_OK) return rc;
  a.seg = pl.seg;
  a.slots = pl.slots;
  a.one_seg = pl.one_seg;
  a.c = c;
  a.b = b;
  a.x = x;
  a.dt = dt;
  a.dy = dy;
  a.A = A;
  a.D = D;
  a.dt_bias = dt_bias;
  a.h0 = h0;
  a.dht = dht;
  a.dc = dc;
  a.db = db;
  a.dx = dx;
  a.ddt = ddt;
  a.dA = dA;
  a.dD = dD;
  a.ddt_bias = ddt_bias;
  a.dh0 = dh0;
  a.ws = static_cast<char *>(workspace);
  return hip(gdn::launch_scan_bwd(a, static_cast<hipStream_t>(stream)), "scan backward");
}

int gdn_selective_scan_step(const gdn_scan_t *p, const void *c, const void *b, const void *x, const void *dt,
                            const float *A, const float *D, const float *dt_bias, float *state,
                            const int32_t *state_indices, int32_t slots, void *y, void *stream) {
  gdn::clear_error();
  gdn::ScanArgs s;
  int rc = check_scan(p, true, &s);
  if (rc != GDN_OK) return rc;
  if (!c || !b || !x || !dt || !A || !state || !y)
    return set_error(GDN_ERR_INVALID_ARG, "c, b, x, dt, A, state and y are required");
  if ((rc = check_slots(state_indices, slots, p->B)) != GDN_OK) return rc;
  if (!aligned(c, 16) || !aligned(b, 16) || !aligned(x, 16) || !aligned(y, 16) || !aligned(state, 16) ||
      !aligned(dt, elem(p->dtype)) || !aligned(A, 4) || !aligned(D, 4) || !aligned(dt_bias, 4))
    return set_error(GDN_ERR_LAYOUT, "c, b, x, y and state must be 16-byte aligned; the rest to their elements");
  gdn::StepArgs a = {};
  a.B = p->B;
  a.Hq = p->Hq;
  a.Hv = p->Hv;
  a.K = p->K;
  a.V = p->V;
  a.dtype = p->dtype;
  a.softplus = p->dt_softplus;
  a.slots = slots;
  a.qs = s.cs;
  a.ks = s.bs;
  a.vs = s.xs;
  a.q = c;
  a.k = b;
  a.v = x;
  a.beta = dt;
  a.A = A;
  a.D = D;
  a.dt_bias = dt_bias;
  a.state = state;
  a.index = state_indices;
  a.o = y;
  return hip(gdn::launch_step(a, static_cast<hipStream_t>(stream)), "scan step");
}

int gdn_delta_rule_step(const gdn_problem_t *p, const void *q, const void *k, const void *v, const float *g,
                        const void *beta, int64_t q_stride, int64_t k_stride, int64_t v_stride, float *state,
                        const int32_t *state_indices, int32_t slots, void *o, void *stream) {
  gdn::clear_error();
  if (!p) return set_error(GDN_ERR_INVALID_ARG, "problem descriptor is NULL");
  if (!(p->scale == p->scale)) return set_error(GDN_ERR_INVALID_ARG, "scale is NaN");
  if (p->qk_l2norm != 0 && p->qk_l2norm != 1)
    return set_error(GDN_ERR_INVALID_ARG, "qk_l2norm must be 0 or 1 (got %d)", p->qk_l2norm);
  const gdn_scan_t sp{p->B, p->T, p->Hq, p->Hv, p->K, p->V, p->N, p->dtype, 0, q_stride, k_stride, v_stride,
                      p->cu_seqlens, p->cu_seqlens_host};
  gdn::ScanArgs s;
  int rc = check_scan(&sp, true, &s);
  if (rc != GDN_OK) return rc;
  if (!q || !k || !v || !g || !beta || !state || !o)
    return set_error(GDN_ERR_INVALID_ARG, "q, k, v, g, beta, state and o are required");
  if ((rc = check_slots(state_indices, slots, p->B)) != GDN_OK) return rc;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) || !aligned(state, 16) ||
      !aligned(beta, elem(p->dtype)) || !aligned(g, 4))
    return set_error(GDN_ERR_LAYOUT, "q, k, v, o and state must be 16-byte aligned; g and beta to their elements");
  gdn::StepArgs a = {};
  a.B = p->B;
  a.Hq = p->Hq;
  a.Hv = p->Hv;
  a.K = p->K;
  a.V = p->V;
  a.dtype = p->dtype;
  a.rule = gdn::kStepDelta;
  a.l2 = p->qk_l2norm;
  a.slots = slots;
  a.scale = p->scale;
  a.qs = s.cs;
  a.ks = s.bs;
  a.vs = s.xs;
  a.q = q;
  a.k = k;
  a.v = v;
  a.beta = beta;
  a.g = g;
  a.state = state;
  a.index = state_indices;
  a.o = o;
  return hip(gdn::launch_step(a, static_cast<hipStream_t>(stream)), "delta rule step");
}

int gdn_layer_norm_fwd(const gdn_norm_t *p, const void *x, const void *weight, const void *bias, const void *gate,
                       void *y, float *mean, float *rstd, void *stream) {
  gdn::clear_error();
  gdn::NormArgs a;
  const int rc = check_norm(p, &a);
  if (rc != GDN_OK) return rc;
  if (p->rows > 0 && (!x || !y)) return set_error(GDN_ERR_INVALID_ARG, "x and y are required");
  const size_t e = elem(p->dtype), we = elem(p->weight_dtype);
  if (!aligned(x, e) || !aligned(y, e) || !aligned(gate, e) || !aligned(weight, we) || !aligned(bias, we) ||
      !aligned(mean, 4) || !aligned(rstd, 4))
    return set_error(GDN_ERR_LAYOUT, "a buffer is not aligned to its elements");
  a.x = x;
  a.w = weight;
  a.b = bias;
  a.gate = gate;
  a.y = y;
  a.mean = mean;
  a.rstd = rstd;
  return hip(gdn::launch_norm_fwd(a, static_cast<hipStream_t>(stream)), "layer norm");
}

size_t gdn_layer_norm_bwd_workspace_size(const gdn_norm_t *p) {
  gdn::clear_error();
  gdn::NormArgs a;
  return check_norm(p, &a) == GDN_OK ? gdn::norm_bwd_floats(a.rows, a.D) * 4 : 0;
}

int gdn_layer_norm_bwd(const gdn_norm_t *p, const void *dy, const void *x, const void *weight, const void *bias,
                       const void *gate, const float *mean, const float *rstd, void *dx, void *dweight, void *dbias,
                       void *dgate, void *workspace, size_t ws_bytes, void *stream) {
  gdn::clear_error();
  gdn::NormArgs a;
  int rc = check_norm(p, &a);
  if (rc != GDN_OK) return rc;
  if (p->rows > 0 && (!dy || !x || !rstd || !dx || (!p->rms && !mean) || (gate && !dgate)))
    return set_error(GDN_ERR_INVALID_ARG, "dy, x, rstd, dx, mean (without rms) and dgate (with gate) are required");
  if ((dweight && !weight) || (dbias && !bias) || (dgate && !gate))
    return set_error(GDN_ERR_INVALID_ARG, "a gradient is asked for without its weight, bias or gate");
  const size_t e = elem(p->dtype), we = elem(p->weight_dtype);
  if (!aligned(dy, e) || !aligned(x, e) || !aligned(gate, e) || !aligned(dx, e) || !aligned(dgate, e) ||
      !aligned(weight, we) || !aligned(bias, we) || !aligned(dweight, we) || !aligned(dbias, we) || !aligned(mean, 4) ||
      !aligned(rstd, 4))
    return set_error(GDN_ERR_LAYOUT, "a buffer is not aligned to its elements");
  if ((rc = check_ws(workspace, ws_bytes, gdn::norm_bwd_floats(a.rows, a.D) * 4)) != GDN_OK) return rc;
  a.dy = dy;
  a.x = x;
  a.w = weight;
  a.b = bias;
  a.gate = gate;
  a.mean = const_cast<float *>(mean);
  a.rstd = const_cast<float *>(rstd);
  a.dx = dx;
  a.dw = dweight;
  a.db = dbias;
  a.dgate = dgate;
  a.partial = static_cast<float *>(workspace);
  return hip(gdn::launch_norm_bwd(a, static_cast<hipStream_t>(stream)), "layer norm backward");
}

size_t gdn_linear_attention_fwd_workspace_size(const gdn_attn_t *p) {
  gdn::clear_error();
  gdn::AttnArgs a;
  return check_attn(p, false, false, &a) == GDN_OK ? gdn::attn_plan(a, false).ws : 0;
}
size_t gdn_linear_attention_bwd_workspace_size(const gdn_attn_t *p) {
  gdn::clear_error();
  gdn::AttnArgs a;
  return check_attn(p, false, true, &a) == GDN_OK ? gdn::attn_plan(a, true).ws : 0;
}

int gdn_linear_attention_fwd(const gdn_attn_t *p, const void *q, const void *k, const void *v, const float *log_decay,
                             const float *h0, void *o, float *ht, void *workspace, size_t ws_bytes, void *stream) {
  gdn::clear_error();
  gdn::AttnArgs a;
  int rc = check_attn(p, false, false, &a);
  if (rc != GDN_OK) return rc;
  if (!log_decay || (a.s.tokens > 0 && (!q || !k || !v || !o)))
    return set_error(GDN_ERR_INVALID_ARG, "q, k, v, log_decay and o are required");
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) || !aligned(h0, 16) || !aligned(ht, 16) ||
      !aligned(log_decay, 4))
    return set_error(GDN_ERR_LAYOUT, "q, k, v, o and the states must be 16-byte aligned; log_decay to its elements");
  const gdn::AttnPlan pl = gdn::attn_plan(a, false);
  if ((rc = check_ws(workspace, ws_bytes, pl.ws)) != GDN_OK) return rc;
  a.seg = pl.seg;
  a.parts = pl.parts;
  a.cols = pl.cols;
  a.slots = pl.slots;
  a.one_seg = pl.one_seg;
  a.joined = pl.joined;
  a.q = q;
  a.k = k;
  a.v = v;
  a.g = log_decay;
  a.h0 = h0;
  a.o = o;
  a.ht = ht;
  a.ws = static_cast<char *>(workspace);
  return hip(gdn::launch_attn_fwd(a, static_cast<hipStream_t>(stream)), "linear attention");
}

int gdn_linear_attention_bwd(const gdn_attn_t *p, const void *q, const void *k, const void *v, const float *log_decay,
                             const float *h0, const void *d_o, const float *dht, void *dq, void *dk, void *dv, float *dh0,
                             void *workspace, size_t ws_bytes, void *stream) {
  gdn::clear_error();
  gdn::AttnArgs a;
  int rc = check_attn(p, false, true, &a);
  if (rc != GDN_OK) return rc;
  if (!log_decay || (a.s.tokens > 0 && (!q || !k || !v || !d_o || !dq || !dk || !dv)))
    return set_error(GDN_ERR_INVALID_ARG, "q, k, v, log_decay, do, dq, dk and dv are required");
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(d_o, 16) || !aligned(dq, 16) || !aligned(dk, 16) ||
      !aligned(dv, 16) || !aligned(h0, 16) || !aligned(dht, 16) || !aligned(dh0, 16) || !aligned(log_decay, 4))
    return set_error(GDN_ERR_LAYOUT,
                     "q, k, v, do, dq, dk, dv and the states must be 16-byte aligned; log_decay to its elements");
  const gdn::AttnPlan pl = gdn::attn_plan(a, true);
  if ((rc = check_ws(workspace, ws_bytes, pl.ws)) != GDN_OK) return rc;
  a.seg = pl.seg;
  a.parts = pl.parts;
  a.cols = pl.cols;
  a.slots = pl.slots;
  a.one_seg = pl.one_seg;
  a.joined = pl.joined;
  a.q = q;
  a.k = k;
  a.v = v;
  a.dO = d_o;
  a.g = log_decay;
  a.h0 = h0;
  a.dht = dht;
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  a.dh0 = dh0;
  a.ws = static_cast<char *>(workspace);
  return hip(gdn::launch_attn_bwd(a, static_cast<hipStream_t>(stream)), "linear attention backward");
}

int gdn_linear_attention_step(const gdn_attn_t *p, const void *q, const void *k, const void *v, const float *log_decay,
                              float *state, const int32_t *state_indices, int32_t slots, void *o, void *stream) {
  gdn::clear_error();
  gdn::AttnArgs s;
  int rc = check_attn(p, true, false, &s);
  if (rc != GDN_OK) return rc;
  if (!q || !k || !v || !log_decay || !state || !o)
    return set_error(GDN_ERR_INVALID_ARG, "q, k, v, log_decay, state and o are required");
  if ((rc = check_slots(state_indices, slots, p->B)) != GDN_OK) return rc;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) || !aligned(state, 16) || !aligned(log_decay, 4))
    return set_error(GDN_ERR_LAYOUT, "q, k, v, o and state must be 16-byte aligned; log_decay to its elements");
  gdn::StepArgs a = {};
  a.B = p->B;
  a.Hq = p->Hq;
  a.Hv = p->Hv;
  a.K = p->K;
  a.V = p->V;
  a.dtype = p->dtype;
  a.rule = gdn::kStepDecay;
  a.slots = slots;
  a.scale = p->scale;
  a.qs = s.qs;
  a.ks = s.ks;
  a.vs = s.vs;
  a.q = q;
  a.k = k;
  a.v = v;
  a.g = log_decay;
  a.state = state;
  a.index = state_indices;
  a.o = o;
  return hip(gdn::launch_step(a, static_cast<hipStream_t>(stream)), "linear attention step");
}

size_t gdn_group_norm_fwd_workspace_size(const gdn_group_t *p) {
  gdn::clear_error();
  gdn::GroupArgs a;
  return check_group(p, false, &a) == GDN_OK ? gdn::group_fwd_bytes(a) : 0;
}
size_t gdn_group_norm_bwd_workspace_size(const gdn_group_t *p) {
  gdn::clear_error();
  gdn::GroupArgs a;
  return check_group(p, true, &a) == GDN_OK ? gdn::group_bwd_bytes(a) : 0;
}

int gdn_group_norm_fwd(const gdn_group_t *p, const void *x, const void *weight, const void *bias, const void *gate,
                       void *y, float *mean, float *rstd, void *workspace, size_t ws_bytes, void *stream) {
  gdn::clear_error();
  gdn::GroupArgs a;
  int rc = check_group(p, false, &a);
  if (rc != GDN_OK) return rc;
  if (p->N > 0 && (!x || !y || !mean || !rstd))
    return set_error(GDN_ERR_INVALID_ARG, "x, y, mean and rstd are required");
  if (gate && p->silu) return set_error(GDN_ERR_INVALID_ARG, "silu and a gate exclude each other");
  const size_t e = elem(p->dtype), we = elem(p->weight_dtype);
  if (!aligned(x, e) || !aligned(y, e) || !aligned(gate, e) || !aligned(weight, we) || !aligned(bias, we) ||
      !aligned(mean, 4) || !aligned(rstd, 4))
    return set_error(GDN_ERR_LAYOUT, "a buffer is not aligned to its elements");
  if ((rc = check_ws(workspace, ws_bytes, gdn::group_fwd_bytes(a))) != GDN_OK) return rc;
  a.x = x;
  a.w = weight;
  a.b = bias;
  a.gate = gate;
  a.y = y;
  a.mean = mean;
  a.rstd = rstd;
  a.ws = static_cast<char *>(workspace);
  return hip(gdn::launch_group_fwd(a, static_cast<hipStream_t>(stream)), "group norm");
}

int gdn_group_norm_bwd(const gdn_group_t *p, const void *dy, const void *x, const void *weight, const void *bias,
                       const void *gate, const float *mean, const float *rstd, void *dx, void *dweight, void *dbias,
                       void *dgate, void *workspace, size_t ws_bytes, void *stream) {
  gdn::clear_error();
  gdn::GroupArgs a;
  int rc = check_group(p, true, &a);
  if (rc != GDN_OK) return rc;
  if (p->N > 0 && (!dy || !x || !mean || !rstd || !dx || (gate && !dgate)))
    return set_error(GDN_ERR_INVALID_ARG, "dy, x, mean, rstd, dx and dgate (with gate) are required");
  if ((dweight && !weight) || (dbias && !bias) || (dgate && !gate))
    return set_error(GDN_ERR_INVALID_ARG, "a gradient is asked for without its weight, bias or gate");
  if (gate && p->silu) return set_error(GDN_ERR_INVALID_ARG, "silu and a gate exclude each other");
  const size_t e = elem(p->dtype), we = elem(p->weight_dtype);
  if (!aligned(dy, e) || !aligned(x, e) || !aligned(gate, e) || !aligned(dx, e) || !aligned(dgate, e) ||
      !aligned(weight, we) || !aligned(bias, we) || !aligned(dweight, we) || !aligned(dbias, we) || !aligned(mean, 4) ||
      !aligned(rstd, 4))
    return set_error(GDN_ERR_LAYOUT, "a buffer is not aligned to its elements");
  if ((rc = check_ws(workspace, ws_bytes, gdn::group_bwd_bytes(a))) != GDN_OK) return rc;
  a.dy = dy;
  a.x = x;
  a.w = weight;
  a.b = bias;
  a.gate = gate;
  a.mean = const_cast<float *>(mean);
  a.rstd = const_cast<float *>(rstd);
  a.dx = dx;
  a.dw = dweight;
  a.db = dbias;
  a.dgate = dgate;
  a.ws = static_cast<char *>(workspace);
  return hip(gdn::launch_group_bwd(a, static_cast<hipStream_t>(stream)), "group norm backward");
}

}  // extern "C"
