"""The operators around the chunked gated delta rule in a sequence mixer.

  causal_conv_fwd / _bwd / _step     short causal convolution (with SiLU)
  selective_scan_fwd / _bwd / _step  selective state-space scan
  gated_delta_rule_step              the gated delta rule for single tokens
  layer_norm_fwd / _bwd              layer norm (or RMS norm), optional output gate

Argument marshalling over libgdn.so (include/gdn.h) like the chunked entry
points: torch supplies outputs, workspace and the current stream of the
inputs' device; nothing here computes.  Tensors are [B, T, ...]; a packed batch
has B = 1 and cu_seqlens (int32 [N + 1]).  With check_cu_seqlens=False a device
cu_seqlens is not copied to the host for checking, so the call does not wait
for the device and can be captured into a graph; its last entry may then be
below T, and the rows of the outputs past it are not written (they hold what
torch.empty left).
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import GDN_BF16, GDN_F32, GdnError, GdnProblem, _check, _check_device, _check_state, _contig, last_error
from . import lib as _base_lib

_I32, _I64, _P, _S = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t


class ConvProblem(ctypes.Structure):
    _fields_ = [(n, _I32) for n in ("B", "T", "D", "W", "N", "dtype", "weight_dtype", "silu")] + [
        ("x_stride", _I64), ("cu_seqlens", _P), ("cu_seqlens_host", _P)]


class ScanProblem(ctypes.Structure):
    _fields_ = [(n, _I32) for n in ("B", "T", "Hq", "Hv", "K", "V", "N", "dtype", "dt_softplus")] + [
        ("c_stride", _I64), ("b_stride", _I64), ("x_stride", _I64), ("cu_seqlens", _P), ("cu_seqlens_host", _P)]


class NormProblem(ctypes.Structure):
    _fields_ = [("rows", _I64)] + [(n, _I32) for n in ("D", "dtype", "weight_dtype", "rms")] + [("eps", ctypes.c_float)]


_ready = None


def lib():
    """libgdn.so with these entry points' argument types."""
    global _ready
    if _ready is None:
        L = _base_lib()
        cp, sp, np_, pp = (ctypes.POINTER(t) for t in (ConvProblem, ScanProblem, NormProblem, GdnProblem))
        for name, args in (
                ("gdn_causal_conv_fwd", [cp] + [_P] * 7),
                ("gdn_causal_conv_bwd", [cp] + [_P] * 11 + [_S, _P]),
                ("gdn_causal_conv_step", [cp] + [_P] * 5 + [_I32, _P, _P]),
                ("gdn_selective_scan_fwd", [sp] + [_P] * 11 + [_S, _P]),
                ("gdn_selective_scan_bwd", [sp] + [_P] * 19 + [_S, _P]),
                ("gdn_selective_scan_step", [sp] + [_P] * 9 + [_I32, _P, _P]),
                ("gdn_delta_rule_step", [pp] + [_P] * 5 + [_I64] * 3 + [_P, _P, _I32, _P, _P]),
                ("gdn_layer_norm_fwd", [np_] + [_P] * 8),
                ("gdn_layer_norm_bwd", [np_] + [_P] * 12 + [_S, _P])):
            f = getattr(L, name)
            f.argtypes, f.restype = args, ctypes.c_int
        for name, arg in (("gdn_causal_conv_bwd_workspace_size", cp), ("gdn_selective_scan_fwd_workspace_size", sp),
                          ("gdn_selective_scan_bwd_workspace_size", sp), ("gdn_layer_norm_bwd_workspace_size", np_)):
            f = getattr(L, name)
            f.argtypes, f.restype = [arg], _S
        _ready = L
    return _ready


def _dtype(t, name):
    if t.dtype == torch.bfloat16:
        return GDN_BF16
    if t.dtype == torch.float32:
        return GDN_F32
    raise TypeError(f"{name} must be bfloat16 or float32, got {t.dtype}")


def _sizes(*sizes):
    """The descriptors and slot counts are 32-bit; ctypes would cut a larger one."""
    if max(sizes) > 0x7FFFFFFF:
        raise ValueError(f"a size is beyond 32 bits: {sizes}")


def _weight_dtype(x, *weights):
    """GDN dtype of the weights that are given (one type, x's or float32)."""
    given = [w for w in weights if w is not None]
    for w in given:
        if w.dtype not in (x.dtype, torch.float32) or w.dtype != given[0].dtype:
            raise TypeError(f"weight and bias must share one type, {x.dtype} or float32")
    return _dtype(given[0], "weight") if given else GDN_F32


class _Seqs:
    """N and the two copies of cu_seqlens (which must outlive the call)."""

    def __init__(self, cu, B, T, device, check):
        self.dev = self.host = None
        self.N = B
        if cu is None:
            return
        if cu.dim() != 1 or cu.numel() < 2 or cu.dtype not in (torch.int32, torch.int64):
            raise ValueError("cu_seqlens must be an integer tensor [N + 1]")
        if B != 1:
            raise ValueError(f"B must be 1 with cu_seqlens (got {B})")
        self.N = cu.numel() - 1
        if check or not cu.is_cuda:
            host = cu.detach().to("cpu", torch.int64)
            lens = host[1:] - host[:-1]
            if int(host[0]) != 0 or int(host[-1]) != T or bool((lens < 0).any()):
                raise ValueError(f"cu_seqlens must run from 0 to T = {T} without decreasing, got {host.tolist()[:8]}")
            self.host = host.to(torch.int32).contiguous()
        self.dev = cu.detach().to(device, torch.int32).contiguous()

    def ptrs(self):
        return (None if self.dev is None else self.dev.data_ptr(), None if self.host is None else self.host.data_ptr())


def _aligned(t):
    """t, contiguous and at a 16-byte boundary (a copy where it is not)."""
    if t is None:
        return None
    t = t.contiguous()
    return t.clone() if t.data_ptr() % 16 else t


def _rows(t, lead: int, aligned: bool = False, most: int = 1 << 62):
    """(tensor, elements from one row to the next) of t, whose first `lead`
    dimensions count rows: t itself where its rows lie at one distance (`most`
    at the most) and each is contiguous, in whole 16-byte pieces; a contiguous
    copy elsewhere.  A contiguous tensor is taken at any address unless
    `aligned`."""
    inner = 1
    for n in t.shape[lead:]:
        inner *= n
    if t.is_contiguous():
        return _aligned(t) if aligned else t, inner
    want, ok = 1, True
    for n, s in zip(reversed(t.shape[lead:]), reversed(t.stride()[lead:])):
        ok = ok and (n == 1 or s == want)
        want *= n
    dims = [(n, s) for n, s in zip(t.shape[:lead], t.stride()[:lead]) if n != 1]
    step = dims[-1][1] if dims else inner
    if len(dims) == 2:
        ok = ok and dims[0][1] == dims[1][0] * dims[1][1]
    per = 16 // t.element_size()
    if ok and inner <= step <= most and step % per == 0 and t.data_ptr() % 16 == 0:
        return t, step
    return t.contiguous(), inner


def _p(t):
    return None if t is None else t.data_ptr()


def _call(f, device, *args):
    """f(*args, stream) on the current stream of `device`, which is made current if it is not."""
    i = device.index
    if i == torch._C._cuda_getDevice():
        rc = f(*args, torch._C._cuda_getCurrentRawStream(i))
    else:
        with torch.cuda.device(device):
            rc = f(*args, torch._C._cuda_getCurrentRawStream(i))
    if rc:
        _check(rc)


def _workspace(n, device):
    if n == 0:
        raise GdnError(1, last_error())
    return torch.empty(n, device=device, dtype=torch.uint8)


def _like(t, shape, dtype, name):
    """An optional tensor of one shape and dtype, contiguous."""
    if t is None:
        return None
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype} {list(shape)}, got {t.dtype} {list(t.shape)}")
    return t.contiguous()


def _indices(idx, B, state, name="state_indices"):
    _sizes(state.shape[0])
    if idx is None:
        if state.shape[0] < B:
            raise ValueError(f"state has {state.shape[0]} slots for {B} batch rows")
        return None
    if tuple(idx.shape) != (B,) or idx.dtype != torch.int32:
        raise ValueError(f"{name} must be int32 [{B}], got {idx.dtype} {list(idx.shape)}")
    return idx.contiguous()


# ---------------------------------------------------------------- convolution


def _conv_problem(x, weight, bias, activation, lead):
    if weight.dim() != 2 or weight.shape[0] != x.shape[-1]:
        raise ValueError(f"weight must be [D, W] with D = {x.shape[-1]}, got {list(weight.shape)}")
    if bias is not None and tuple(bias.shape) != (x.shape[-1],):
        raise ValueError(f"bias must be [{x.shape[-1]}], got {list(bias.shape)}")
    if activation not in (None, "silu"):
        raise ValueError(f"activation must be None or 'silu', got {activation!r}")
    D, W = weight.shape
    _sizes(*x.shape, W)
    dt, wd = _dtype(x, "x"), _weight_dtype(x, weight, bias)
    xr, xs = _rows(x, lead)
    return ConvProblem(x.shape[0], x.shape[1] if lead == 2 else 1, D, W, x.shape[0], dt, wd,
                       int(activation == "silu"), xs, None, None), xr, weight.contiguous(), _contig(bias)


def causal_conv_fwd(x, weight, bias=None, initial_state=None, cu_seqlens=None, activation: Optional[str] = "silu",
                    output_final_state: bool = True, check_cu_seqlens: bool = True):
    """Depthwise causal convolution over tokens.  Returns (y, final_state).

    x [B, T, D] (its token rows may be a slice of a wider tensor), weight [D, W]
    with W in {2, 3, 4}, bias [D]; weight[:, W - 1] meets the current token.
    initial_state and final_state are the last W - 1 inputs [N, W - 1, D] in
    x's dtype.  activation: "silu" or None."""
    if x.dim() != 3:
        raise ValueError(f"x must be [B, T, D], got {list(x.shape)}")
    p, xr, weight, bias = _conv_problem(x, weight, bias, activation, 2)
    B, T, D = x.shape
    dev = x.device
    sq = _Seqs(cu_seqlens, B, T, dev, check_cu_seqlens)
    h0 = _like(initial_state, (sq.N, p.W - 1, D), x.dtype, "initial_state")
    _check_device(x, weight, bias, h0)
    p.N = sq.N
    p.cu_seqlens, p.cu_seqlens_host = sq.ptrs()
    y = torch.empty(B, T, D, device=dev, dtype=x.dtype)
    ht = torch.empty(sq.N, p.W - 1, D, device=dev, dtype=x.dtype) if output_final_state else None
    _call(lib().gdn_causal_conv_fwd, dev, ctypes.byref(p), _p(xr), _p(weight), _p(bias), _p(h0), _p(y), _p(ht))
    return y, ht


def causal_conv_bwd(x, weight, bias, dy, initial_state=None, dfinal_state=None, cu_seqlens=None,
                    activation: Optional[str] = "silu", check_cu_seqlens: bool = True):
    """Backward of causal_conv_fwd.  Returns (dx, dweight, dbias,
    dinitial_state), the last two None without bias and initial_state."""
    if x.dim() != 3:
        raise ValueError(f"x must be [B, T, D], got {list(x.shape)}")
    p, xr, weight, bias = _conv_problem(x, weight, bias, activation, 2)
    B, T, D = x.shape
    dev = x.device
    if dy is None or dy.shape != x.shape or dy.dtype != x.dtype:
        raise ValueError(f"dy must have x's shape {list(x.shape)} and dtype {x.dtype}")
    sq = _Seqs(cu_seqlens, B, T, dev, check_cu_seqlens)
    dy = dy.contiguous()
    h0 = _like(initial_state, (sq.N, p.W - 1, D), x.dtype, "initial_state")
    dht = _like(dfinal_state, (sq.N, p.W - 1, D), x.dtype, "dfinal_state")
    _check_device(x, weight, bias, dy, h0, dht)
    p.N = sq.N
    p.cu_seqlens, p.cu_seqlens_host = sq.ptrs()
    dx = torch.empty(B, T, D, device=dev, dtype=x.dtype)
    dw = torch.empty_like(weight)
    db = None if bias is None else torch.empty_like(bias)
    dh0 = None if h0 is None else torch.empty_like(h0)
    L = lib()
    n = L.gdn_causal_conv_bwd_workspace_size(ctypes.byref(p))
    ws = _workspace(n, dev)
    _call(L.gdn_causal_conv_bwd, dev, ctypes.byref(p), _p(xr), _p(weight), _p(bias), _p(dy), _p(h0), _p(dht),
          _p(dx), _p(dw), _p(db), _p(dh0), _p(ws), n)
    return dx, dw, db, dh0


def causal_conv_step(x, state, weight, bias=None, activation: Optional[str] = "silu", state_indices=None):
    """One token: x [B, D] -> y [B, D]; state [slots, W - 1, D] (x's dtype) is
    moved on in place.  state_indices (int32 [B]): the slot of each row; a row
    with an index outside the slots, or one that an earlier row names, is
    padding (y = 0, no state changes)."""
    if x.dim() != 2:
        raise ValueError(f"x must be [B, D], got {list(x.shape)}")
    p, xr, weight, bias = _conv_problem(x, weight, bias, activation, 1)
    B, D = x.shape
    if state.dim() != 3 or tuple(state.shape[1:]) != (p.W - 1, D) or state.dtype != x.dtype or not state.is_contiguous():
        raise ValueError(f"state must be a contiguous {x.dtype} [slots, {p.W - 1}, {D}], got {state.dtype} {list(state.shape)}")
    idx = _indices(state_indices, B, state)
    _check_device(x, state, weight, bias, idx)
    dev = x.device
    y = torch.empty(B, D, device=dev, dtype=x.dtype)
    _call(lib().gdn_causal_conv_step, dev, ctypes.byref(p), _p(xr), _p(state), _p(weight), _p(bias), _p(idx),
          state.shape[0], _p(y))
    return y


# ---------------------------------------------------------------- selective scan


def _scan_problem(c, b, x, dt, A, D, dt_bias, dt_softplus, lead):
    what = "[B, T, H, K]" if lead == 2 else "[B, H, K]"
    if c.dim() != lead + 2 or b.shape != c.shape or x.dim() != lead + 2 or x.shape[:lead] != c.shape[:lead]:
        raise ValueError(f"c, b must be {what} and x as them over the v-heads")
    if dt.shape != x.shape[:lead + 1]:
        raise ValueError(f"dt must be {list(x.shape[:lead + 1])}, got {list(dt.shape)}")
    if not (c.dtype == b.dtype == x.dtype == dt.dtype):
        raise TypeError("c, b, x and dt must share one dtype")
    _sizes(*x.shape, *c.shape)
    Hv = x.shape[lead]
    for t, name in ((A, "A"), (D, "D"), (dt_bias, "dt_bias")):
        if t is None and name != "A":
            continue
        if t is None or t.dtype != torch.float32 or tuple(t.shape) != (Hv,):
            raise ValueError(f"{name} must be float32 [{Hv}]")
    most = (1 << 24) - 1 if lead == 2 else 1 << 62
    (cr, cs), (br, bs), (xr, xs) = (_rows(t, lead, True, most) for t in (c, b, x))
    p = ScanProblem(x.shape[0], x.shape[1] if lead == 2 else 1, c.shape[lead], Hv, c.shape[lead + 1], x.shape[lead + 1],
                    x.shape[0], _dtype(x, "c, b, x and dt"), int(bool(dt_softplus)), cs, bs, xs, None, None)
    return p, cr, br, xr, dt.contiguous(), A.contiguous(), _contig(D), _contig(dt_bias)


def selective_scan_fwd(c, b, x, dt, A, D=None, dt_bias=None, dt_softplus: bool = True, initial_state=None,
                       cu_seqlens=None, output_final_state: bool = True, check_cu_seqlens: bool = True):
    """Selective state-space scan.  Returns (y, final_state).

    Per v-head h, with delta = softplus(dt + dt_bias) (dt + dt_bias without
    dt_softplus): S_t = exp(delta_t A) S_{t-1} + delta_t b_t x_t^T and
    y_t = S_t^T c_t + D x_t.  c, b [B, T, Hq, K] (read by v-head h at head
    h // (Hv // Hq)), x [B, T, Hv, V], dt [B, T, Hv] in one dtype; A, D,
    dt_bias float32 [Hv]; states float32 [N, Hv, K, V]; K, V in {32, 64, 128}
    in bfloat16, {32, 64} in float32 (the step: all three).  The token rows of
    c, b and x may be slices of a wider tensor.  A state that grows (A > 0) is
    computed as it is, up to what float32 holds.  A NaN or an infinity in a
    token reaches the tokens of its 64-token chunk, earlier ones too, and all
    later ones of its sequence; no other sequence."""
    p, c, b, x, dt, A, D, dt_bias = _scan_problem(c, b, x, dt, A, D, dt_bias, dt_softplus, 2)
    dev = x.device
    sq = _Seqs(cu_seqlens, p.B, p.T, dev, check_cu_seqlens)
    shape = (sq.N, p.Hv, p.K, p.V)
    h0 = _aligned(initial_state)
    _check_state(h0, "initial_state", shape)
    _check_device(x, c, b, dt, A, D, dt_bias, h0)
    p.N = sq.N
    p.cu_seqlens, p.cu_seqlens_host = sq.ptrs()
    y = torch.empty(x.shape, device=dev, dtype=x.dtype)
    ht = torch.empty(shape, device=dev, dtype=torch.float32) if output_final_state else None
    L = lib()
    n = L.gdn_selective_scan_fwd_workspace_size(ctypes.byref(p))
    ws = _workspace(n, dev)
    _call(L.gdn_selective_scan_fwd, dev, ctypes.byref(p), _p(c), _p(b), _p(x), _p(dt), _p(A), _p(D),
          _p(dt_bias), _p(h0), _p(y), _p(ht), _p(ws), n)
    return y, ht


def selective_scan_bwd(c, b, x, dt, A, dy, dht=None, D=None, dt_bias=None, dt_softplus: bool = True, initial_state=None,
                       cu_seqlens=None, check_cu_seqlens: bool = True):
    """Backward of selective_scan_fwd.  Returns (dc, db, dx, ddt, dA, dD,
    ddt_bias, dh0): dc, db summed over the v-heads of a group, ddt with
    respect to dt as given (before bias and softplus); dD, ddt_bias and dh0
    None where D, dt_bias and initial_state are."""
    p, c, b, x, dt, A, D, dt_bias = _scan_problem(c, b, x, dt, A, D, dt_bias, dt_softplus, 2)
    if dy is None or dy.shape != x.shape or dy.dtype != x.dtype:
        raise ValueError(f"dy must have x's shape {list(x.shape)} and dtype {x.dtype}")
    dev = x.device
    sq = _Seqs(cu_seqlens, p.B, p.T, dev, check_cu_seqlens)
    shape = (sq.N, p.Hv, p.K, p.V)
    dy, dht, h0 = _aligned(dy), _aligned(dht), _aligned(initial_state)
    _check_state(dht, "dht", shape)
    _check_state(h0, "initial_state", shape)
    _check_device(x, c, b, dt, A, D, dt_bias, dy, dht, h0)
    p.N = sq.N
    p.cu_seqlens, p.cu_seqlens_host = sq.ptrs()
    new = lambda t: torch.empty(t.shape, device=dev, dtype=t.dtype)  # noqa: E731
    dc, db, dx, ddt, dA = new(c), new(b), new(x), new(dt), new(A)
    dD, dbias, dh0 = (None if t is None else new(t) for t in (D, dt_bias, h0))
    L = lib()
    n = L.gdn_selective_scan_bwd_workspace_size(ctypes.byref(p))
    ws = _workspace(n, dev)
    _call(L.gdn_selective_scan_bwd, dev, ctypes.byref(p), _p(c), _p(b), _p(x), _p(dt), _p(A), _p(D),
          _p(dt_bias), _p(h0), _p(dy), _p(dht), _p(dc), _p(db), _p(dx), _p(ddt), _p(dA), _p(dD), _p(dbias),
          _p(dh0), _p(ws), n)
    return dc, db, dx, ddt, dA, dD, dbias, dh0


def _step_state(state, Hv, K, V):
    if state.dim() != 4 or tuple(state.shape[1:]) != (Hv, K, V) or state.dtype != torch.float32 or not state.is_contiguous():
        raise ValueError(f"state must be a contiguous float32 [slots, {Hv}, {K}, {V}], got {state.dtype} {list(state.shape)}")


def selective_scan_step(c, b, x, dt, A, state, D=None, dt_bias=None, dt_softplus: bool = True, state_indices=None):
    """One token of the selective scan: c, b [B, Hq, K], x [B, Hv, V], dt
    [B, Hv] -> y [B, Hv, V]; state [slots, Hv, K, V] (float32) is updated in
    place.  state_indices as for causal_conv_step."""
    p, c, b, x, dt, A, D, dt_bias = _scan_problem(c, b, x, dt, A, D, dt_bias, dt_softplus, 1)
    _step_state(state, p.Hv, p.K, p.V)
    idx = _indices(state_indices, p.B, state)
    _check_device(x, c, b, dt, A, D, dt_bias, state, idx)
    dev = x.device
    y = torch.empty(x.shape, device=dev, dtype=x.dtype)
    _call(lib().gdn_selective_scan_step, dev, ctypes.byref(p), _p(c), _p(b), _p(x), _p(dt), _p(A), _p(D),
          _p(dt_bias), _p(state), _p(idx), state.shape[0], _p(y))
    return y


def gated_delta_rule_step(q, k, v, g, beta, state, scale=None, use_qk_l2norm_in_kernel: bool = False,
                          state_indices=None):
    """One token of the gated delta rule (the recurrence of
    chunk_gated_delta_rule): q, k [B, Hq, K], v [B, Hv, V], g (float32) and
    beta [B, Hv] -> o [B, Hv, V]; state [slots, Hv, K, V] (float32, such as
    the prefill's final state) is updated in place.  state_indices as for
    causal_conv_step."""
    if q.dim() != 3 or k.shape != q.shape or v.dim() != 3 or v.shape[0] != q.shape[0]:
        raise ValueError("q, k must be [B,Hq,K] and v [B,Hv,V]")
    B, Hq, K = q.shape
    Hv, V = v.shape[1:]
    _sizes(*q.shape, Hv, V)
    if tuple(g.shape) != (B, Hv) or tuple(beta.shape) != (B, Hv):
        raise ValueError("g and beta must be [B,Hv]")
    if k.dtype != q.dtype or v.dtype != q.dtype or beta.dtype != q.dtype:
        raise TypeError("q, k, v and beta must share one dtype")
    if g.dtype != torch.float32:
        raise TypeError("g must be float32")
    dt = _dtype(q, "q, k, v and beta")
    _step_state(state, Hv, K, V)
    idx = _indices(state_indices, B, state)
    (q, qs), (k, ks), (v, vs) = (_rows(t, 1, True) for t in (q, k, v))
    g, beta = g.contiguous(), beta.contiguous()
    _check_device(q, k, v, g, beta, state, idx)
    dev = q.device
    o = torch.empty(B, Hv, V, device=dev, dtype=v.dtype)
    p = GdnProblem(B, 1, Hq, Hv, K, V, B, dt, float(K ** -0.5 if scale is None else scale), None, None, -1,
                   int(bool(use_qk_l2norm_in_kernel)))
    _call(lib().gdn_delta_rule_step, dev, ctypes.byref(p), _p(q), _p(k), _p(v), _p(g), _p(beta), qs, ks, vs,
          _p(state), _p(idx), state.shape[0], _p(o))
    return o


# ---------------------------------------------------------------- layer norm


def _norm_problem(x, weight, bias, gate, eps, rms):
    D = x.shape[-1] if x.dim() else 0
    if D == 0:
        raise ValueError(f"x must be [..., D] with D > 0, got {list(x.shape)}")
    _sizes(D)
    for t, name in ((weight, "weight"), (bias, "bias")):
        if t is not None and tuple(t.shape) != (D,):
            raise ValueError(f"{name} must be [{D}], got {list(t.shape)}")
    if gate is not None and (gate.shape != x.shape or gate.dtype != x.dtype):
        raise ValueError(f"gate must have x's shape {list(x.shape)} and dtype {x.dtype}")
    return NormProblem(x.numel() // D, D, _dtype(x, "x"), _weight_dtype(x, weight, bias), int(bool(rms)), float(eps))


def layer_norm_fwd(x, weight=None, bias=None, gate=None, eps: float = 1e-5, rms: bool = False):
    """Layer norm over the last dimension.  Returns (y, mean, rstd).

    z = (x - mean) rstd weight + bias and y = z silu(gate) (y = z without
    gate).  rms=True: RMS norm, mean is taken as 0 and returned as None.  x
    and gate [..., D]; weight, bias [D] in x's dtype or float32; mean, rstd
    float32 [...], for the backward."""
    p = _norm_problem(x, weight, bias, gate, eps, rms)
    x, weight, bias, gate = _contig(x), _contig(weight), _contig(bias), _contig(gate)
    _check_device(x, weight, bias, gate)
    dev = x.device
    y = torch.empty_like(x)
    mean = None if rms else torch.empty(x.shape[:-1], device=dev, dtype=torch.float32)
    rstd = torch.empty(x.shape[:-1], device=dev, dtype=torch.float32)
    _call(lib().gdn_layer_norm_fwd, dev, ctypes.byref(p), _p(x), _p(weight), _p(bias), _p(gate), _p(y),
          _p(mean), _p(rstd))
    return y, mean, rstd


def layer_norm_bwd(dy, x, weight, bias, mean, rstd, gate=None, rms: bool = False):
    """Backward of layer_norm_fwd, from its mean and rstd.  Returns (dx,
    dweight, dbias, dgate), each None where its tensor is."""
    p = _norm_problem(x, weight, bias, gate, 0.0, rms)
    if dy is None or dy.shape != x.shape or dy.dtype != x.dtype:
        raise ValueError(f"dy must have x's shape {list(x.shape)} and dtype {x.dtype}")
    mean = None if rms else _like(mean, x.shape[:-1], torch.float32, "mean")
    if (mean is None) != bool(rms):
        raise ValueError("mean is required without rms")
    if rstd is None:
        raise ValueError("rstd is required")
    rstd = _like(rstd, x.shape[:-1], torch.float32, "rstd")
    x, dy, weight, bias, gate = (_contig(t) for t in (x, dy, weight, bias, gate))
    _check_device(x, dy, weight, bias, gate, mean, rstd)
    dev = x.device
    dx, dw, db, dgate = (None if t is None else torch.empty_like(t) for t in (x, weight, bias, gate))
    L = lib()
    n = L.gdn_layer_norm_bwd_workspace_size(ctypes.byref(p))
    ws = _workspace(n, dev)
    _call(L.gdn_layer_norm_bwd, dev, ctypes.byref(p), _p(dy), _p(x), _p(weight), _p(bias), _p(gate), _p(mean),
          _p(rstd), _p(dx), _p(dw), _p(db), _p(dgate), _p(ws), n)
    return dx, dw, db, dgate
