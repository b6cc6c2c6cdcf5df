"""GPU parity of the sequence-mixer operators on the paths that larger problems
take, at sizes whose 64-bit value is still quick: segments of several chunks,
sequences of one segment, every decay regime in both types, masked tokens,
padded batches, rows at odd addresses and distances.

The 64-bit form of the scan runs over all sequences at once on the GPU (one
elementwise step a token).  Tolerances as in test_gpu_mixer.py."""
import pytest
import torch

from tests.mixer_ref import DT, delta_of, near, near_sum
from tests.gpu_util import announce
from tests.test_gpu_mixer import F32, SCAN, SCAN_OUT, cu_of, gdn, gen, randn  # noqa: F401  (gdn: the fixture)

pytestmark = pytest.mark.gpu


def rows_of(lens, B, T):
    """Tokens of every sequence side by side: places [N, longest] in the batch's rows, and which of them are there."""
    lens = torch.tensor(lens if lens is not None else [T] * B)
    first = torch.cumsum(lens, 0) - lens
    at = torch.arange(max(int(lens.max()), 1))
    live = at < lens[:, None]
    return torch.where(live, first[:, None] + at, 0).cuda(), live.cuda()


def scan64(lens, c, b, x, dt, A, D, bias, h0, softplus):
    """tests.mixer_ref.scan for all sequences at once; A, D, bias [B, T, Hv] or None.  (A token that is not there
    leaves the state as it is.)"""
    B, T, Hv, V = x.shape
    K = c.shape[3]
    at, live = rows_of(lens, B, T)
    of = torch.arange(Hv, device="cuda") // (Hv // c.shape[2])
    pick = lambda t: t.reshape(B * T, *t.shape[2:])[at]  # noqa: E731
    delta = pick(delta_of(dt, bias, softplus)) * live[..., None]
    g = delta * pick(A)
    c, b, xs = pick(c)[:, :, of], pick(b)[:, :, of], pick(x)
    S = torch.zeros(len(at), Hv, K, V, dtype=torch.float64, device="cuda") if h0 is None else h0
    ys = []
    for t in range(at.shape[1]):
        S = torch.exp(g[:, t])[..., None, None] * S + (delta[:, t, :, None] * b[:, t])[..., None] * xs[:, t, :, None]
        ys.append((S * c[:, t][..., None]).sum(2))
    y = torch.stack(ys, 1)
    y = y if D is None else y + pick(D)[..., None] * xs
    return y[live].reshape(B, T, Hv, V), S


def d64(t):
    return None if t is None else t.detach().double()


def near_dA(got, terms, decays):
    """near_sum of dA's terms delta_t dg_t, dg_t = e^{g_t} <S_{t-1}, Z_t>.  A decay e^{g_t} below 2^-126 is below the
    normal numbers of fp32, where an exponential may give 0: such a term may be missing, which is off by the term."""
    lost = terms.abs() * (decays < 2.0 ** -126)
    off, most = (d64(got) - terms.sum((0, 1))).abs(), F32 * terms.abs().sum((0, 1)) + lost.sum((0, 1))
    assert bool((off <= most).all()), f"dA: {(off / most).tolist()} of the bound"


def check_scan(gdn, dtype, lens, c, b, x, dt, A, D, bias, h0, dy, dht, softplus):  # noqa: F811
    """Both directions against 64 bits."""
    heads = x.shape[:3]
    leaves = [d64(t) for t in (c, b, x, dt, A, D, bias, h0)]
    leaves = [t.expand(heads).clone() if t is not None and i in (4, 5, 6) else t for i, t in enumerate(leaves)]
    leaves = [None if t is None else t.requires_grad_() for t in leaves]
    ry, rht = scan64(lens, *leaves, softplus)
    kw = dict(D=D, dt_bias=bias, dt_softplus=softplus, initial_state=h0, cu_seqlens=cu_of(lens))
    y, ht = gdn.selective_scan_fwd(c, b, x, dt, A, **kw)
    near("y", y, ry, SCAN[dtype])
    near("ht", ht, rht, F32)
    value = (ry * d64(dy)).sum() if dht is None else (ry * d64(dy)).sum() + (rht * d64(dht)).sum()
    want = iter(torch.autograd.grad(value, [t for t in leaves if t is not None]))
    want = [None if t is None else next(want) for t in leaves]
    got = gdn.selective_scan_bwd(c, b, x, dt, A, dy, dht=dht, **kw)
    for n, a, r in zip(SCAN_OUT, got, want):
        if n == "dA":
            near_dA(a, r, torch.exp(delta_of(d64(dt), d64(bias), softplus) * d64(A)))
        elif n in ("dD", "ddt_bias"):
            near_sum(n, a, r if r is None else r.cpu(), F32)
        else:
            near(n, a, r, F32 if n == "dh0" else SCAN[dtype])


def inputs(dtype, B, T, Hq, Hv, K, V, lens=None, state=True, seed=1):
    g, dt = gen(seed), DT[dtype]
    T = sum(lens) if lens is not None else T
    N = len(lens) if lens is not None else B
    c, b, x = randn(g, B, T, Hq, K, dt=dt), randn(g, B, T, Hq, K, dt=dt), randn(g, B, T, Hv, V, dt=dt)
    A = -(0.5 + 8 * torch.rand(Hv, generator=g)).cuda()
    D, bias = randn(g, Hv), randn(g, Hv, s=0.5) - 3
    dtv = randn(g, B, T, Hv, s=0.7, dt=dt)
    h0, dht = (randn(g, N, Hv, K, V, s=0.3), randn(g, N, Hv, K, V, s=0.3)) if state else (None, None)
    return dict(c=c, b=b, x=x, dt=dtv, A=A, D=D, bias=bias, h0=h0, dy=randn(g, B, T, Hv, V, dt=dt), dht=dht, softplus=True)


def segment(gdn, dtype, B, T, Hq, Hv, K, V, lens, bwd):  # noqa: F811
    """Tokens of a segment by the planner's rule, held against the workspace that the forward asks for."""
    T = sum(lens) if lens is not None else T
    N = len(lens) if lens is not None else B
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    if dtype == "bf16":
        slices = Hv // Hq * (V // 32)
        each = next(n for n in (8, 4, 2, 1) if slices % n == 0)
        want, unit = -(-cus // (Hq * (slices // each))), 64
    else:
        want, unit = -(-cus * 8 // (Hv * -(-V // 64))), 16
    seg = max(unit, -(-(-(-B * T // max(want, N))) // unit) * unit)
    slots = B * T // seg + N if lens is not None else N * -(-T // seg)
    up = lambda n: -(-n // 256) * 256  # noqa: E731
    ws = 256 if T <= seg else up(slots * Hv * K * V * 4) + up(slots * Hv * 4)
    cu = 16 if lens is not None else None
    p = gdn.mixer.ScanProblem(B, T, Hq, Hv, K, V, N, int(dtype == "bf16"), 1, 0, 0, 0, cu, None)
    import ctypes
    assert gdn.mixer.lib().gdn_selective_scan_fwd_workspace_size(ctypes.byref(p)) == ws
    return min(seg, 64) if bwd and dtype == "f32" else seg


# The fp32 backward's segments are 64 tokens at the most.
STEPS = [1e-4, 0.3, 2.0, 9.0, 18.0, 25.0, 40.0, 120.0, "mixed", "mostly mild"]


@pytest.mark.parametrize("state", [False, True])
@pytest.mark.parametrize("K,V", [(32, 32), (64, 64), (64, 32)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_scan_decay_regimes_of_long_segments(gdn, dtype, K, V, state):  # noqa: F811
    """Log decays a token from nothing to all, a regime a head, in segments of 64 tokens and a short one."""
    Hv, B, T = 40, 52, 70
    announce(f"scan regimes {dtype} {K} {V} state={state}")
    assert dtype == "bf16" or segment(gdn, dtype, B, T, 1, Hv, K, V, None, True) == 64
    i = inputs(dtype, B, T, 1, Hv, K, V, state=state, seed=17)
    g = gen(18)
    step = torch.empty(B, T, Hv)
    for h in range(Hv):
        s = STEPS[h % len(STEPS)]
        if s == "mixed":
            step[..., h] = torch.tensor([1e-4, 0.3, 2.0, 9.0, 18.0, 40.0, 200.0])[torch.randint(0, 7, (B, T), generator=g)]
        elif s == "mostly mild":
            step[..., h] = torch.tensor([0.001, 0.01, 0.3, 19.0])[torch.randint(0, 4, (B, T), generator=g)]
        else:
            step[..., h] = s * (0.8 + 0.4 * torch.rand(B, T, generator=g))
    i["A"] = -torch.tensor([1.0, 0.5])[torch.arange(Hv) % 2].cuda()
    i["dt"] = (step / torch.tensor([1.0, 0.5])[torch.arange(Hv) % 2]).to(DT[dtype]).cuda()
    i["bias"], i["softplus"] = None, False
    check_scan(gdn, dtype, None, **i)


# ---------------------------------------------------------------- buffers of the C entries


class Buffers:
    """Outputs and workspace of a C entry, each the middle of a wider buffer
    whose ends hold a pattern, and the entry's inputs, which stay as they are.
    Outputs start as 7, the workspace as NaN."""

    BAND = 4096  # bytes

    def __init__(self, inputs):  # noqa: F811
        self.inputs = [(t, t.clone()) for t in inputs if t is not None]
        self.bands = []

    def bytes(self, n, fill):
        whole = torch.full((n + 2 * self.BAND,), 0xA5, dtype=torch.uint8, device="cuda")
        whole[self.BAND:self.BAND + n] = fill
        self.bands.append((whole, n))
        return whole[self.BAND:self.BAND + n]

    def new(self, shape, dt):
        n = torch.Size(shape).numel()
        return self.bytes(n * dt.itemsize, 0).view(dt).view(shape).fill_(7)

    def like(self, t):
        return None if t is None else self.new(t.shape, t.dtype)

    def check(self):
        torch.cuda.synchronize()
        for whole, n in self.bands:
            assert bool((whole[:self.BAND] == 0xA5).all()) and bool((whole[self.BAND + n:] == 0xA5).all())
        for t, was in self.inputs:
            assert torch.equal(t.reshape(-1).view(torch.uint8), was.reshape(-1).view(torch.uint8))


def raw_call(f, *args):
    import ctypes
    args = [a.data_ptr() if isinstance(a, torch.Tensor) else ctypes.byref(a) if isinstance(a, ctypes.Structure) else a
            for a in args]
    assert f(*args, torch.cuda.current_stream().cuda_stream) == 0


def raw_conv(gdn, x, w, b, h0, dy, dht, cu):  # noqa: F811
    """(y, ht), (dx, dw, db, dh0) of the C entries, cu on the device, unchecked."""
    import ctypes
    m, N = gdn.mixer, cu.numel() - 1
    p = m.ConvProblem(1, x.shape[1], x.shape[2], w.shape[1], N, int(x.dtype == torch.bfloat16), int(w.dtype == torch.bfloat16),
                      1, 0, cu.data_ptr(), None)
    o = Buffers((x, w, b, h0, dy, dht, cu))
    y, ht = o.like(x), o.new((N, w.shape[1] - 1, x.shape[2]), x.dtype)
    raw_call(m.lib().gdn_causal_conv_fwd, p, x, w, b, h0, y, ht)
    grads = [o.like(t) for t in (x, w, b, h0)]
    n = m.lib().gdn_causal_conv_bwd_workspace_size(ctypes.byref(p))
    raw_call(m.lib().gdn_causal_conv_bwd, p, x, w, b, dy, h0, dht, *grads, o.bytes(n, 0xFF), n)
    o.check()
    return (y, ht), grads


def raw_scan(gdn, i, cu):  # noqa: F811
    """(y, ht), (dc, db, dx, ddt, dA, dD, ddt_bias, dh0) likewise."""
    import ctypes
    m, N, x, c = gdn.mixer, cu.numel() - 1, i["x"], i["c"]
    p = m.ScanProblem(1, x.shape[1], c.shape[2], x.shape[2], c.shape[3], x.shape[3], N, int(x.dtype == torch.bfloat16),
                      int(i["softplus"]), 0, 0, 0, cu.data_ptr(), None)
    ins = [i[k] for k in ("c", "b", "x", "dt", "A", "D", "bias", "h0")]
    o = Buffers(ins + [i["dy"], i["dht"], cu])
    y, ht = o.like(x), o.new((N, x.shape[2], c.shape[3], x.shape[3]), torch.float32)
    n = m.lib().gdn_selective_scan_fwd_workspace_size(ctypes.byref(p))
    raw_call(m.lib().gdn_selective_scan_fwd, p, *ins, y, ht, o.bytes(n, 0xFF), n)
    grads = [o.like(t) for t in ins]
    n = m.lib().gdn_selective_scan_bwd_workspace_size(ctypes.byref(p))
    raw_call(m.lib().gdn_selective_scan_bwd, p, *ins, i["dy"], i["dht"], *grads, o.bytes(n, 0xFF), n)
    o.check()
    return (y, ht), grads


# tokens of the sequences, rows behind them
PADDED = [([30, 0, 30], 40), ([70, 1, 64], 1), ([200], 100), ([5], 3), ([0, 0], 20)]


@pytest.mark.parametrize("lens,pad", PADDED)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_behind_the_last_sequence_stay(gdn, dtype, lens, pad):  # noqa: F811
    """They hold NaN, no result sees them, and nothing is written to theirs."""
    announce(f"padded {dtype} {lens} {pad}")
    T, cu = sum(lens), cu_of(lens).cuda()

    def padded(t):
        return torch.cat([t, torch.full((1, pad, *t.shape[2:]), float("nan"), dtype=t.dtype, device="cuda")], 1)

    def rows(got, T):
        assert bool((got[:, T:] == 7).all())
        return got[:, :T]

    g, dt = gen(41), DT[dtype]
    x, w, b, dy = randn(g, 1, T, 40, dt=dt), randn(g, 40, 4, dt=dt), randn(g, 40, dt=dt), randn(g, 1, T, 40, dt=dt)
    h0, dht = randn(g, len(lens), 3, 40, dt=dt), randn(g, len(lens), 3, 40, dt=dt)
    (y, ht), (dx, dw, db, dh0) = raw_conv(gdn, padded(x), w, b, h0, padded(dy), dht, cu)
    ry, rht = gdn.causal_conv_fwd(x, w, b, initial_state=h0, cu_seqlens=cu)
    want = gdn.causal_conv_bwd(x, w, b, dy, initial_state=h0, dfinal_state=dht, cu_seqlens=cu)
    assert torch.equal(rows(y, T), ry) and torch.equal(ht, rht) and torch.equal(rows(dx, T), want[0]) and torch.equal(dh0, want[3])
    near("dw", dw, want[1], SCAN[dtype])
    near("db", db, want[2], SCAN[dtype])

    i = inputs(dtype, 1, 0, 2, 4, 64, 32, lens=lens, seed=42)
    j = {k: padded(t) if k in ("c", "b", "x", "dt", "dy") else t for k, t in i.items()}
    (y, ht), got = raw_scan(gdn, j, cu)
    kw = dict(D=i["D"], dt_bias=i["bias"], initial_state=i["h0"], cu_seqlens=cu)
    ins = [i[k] for k in ("c", "b", "x", "dt", "A")]
    ry, rht = gdn.selective_scan_fwd(*ins, **kw)
    near("y", rows(y, T), ry, SCAN[dtype])
    near("ht", ht, rht, 2 * F32)  # (two results, each with its own segments)
    want = gdn.selective_scan_bwd(*ins, i["dy"], dht=i["dht"], **kw)
    for n, a, r in zip(SCAN_OUT, got, want):
        a = rows(a, T) if a.dim() > 2 and n != "dh0" else a
        if n in ("dA", "dD", "ddt_bias"):
            assert bool(torch.isfinite(a).all())
        else:
            near(n, a, r, 2 * F32 if n == "dh0" else 2 * SCAN[dtype])


# ---------------------------------------------------------------- rows as they lie


def test_steps_on_a_token_of_a_long_sequence(gdn):  # noqa: F811
    """q[:, t] of a [B, T, H, K]: rows 2^24 elements and more apart."""
    g = gen(51)
    B, T, Hq, Hv, K, V, t = 2, 16390, 8, 16, 128, 64, 16389
    q, k, v = (torch.zeros(B, T, h, n, dtype=torch.bfloat16, device="cuda") for h, n in ((Hq, K), (Hq, K), (Hv, V)))
    for x in (q, k, v):
        x[:, t] = randn(g, B, *x.shape[2:], dt=torch.bfloat16)
    beta, gate, A = torch.rand(B, Hv, generator=g).bfloat16().cuda(), -torch.rand(B, Hv, generator=g).cuda(), -torch.rand(Hv, generator=g).cuda()
    st = randn(g, B, Hv, K, V)
    for f in (lambda q, k, v, s: gdn.gated_delta_rule_step(q, k, v, gate, beta, s, use_qk_l2norm_in_kernel=True),
              lambda q, k, v, s: gdn.selective_scan_step(q, k, v, beta, A, s)):
        s1, s2 = st.clone(), st.clone()
        assert torch.equal(f(q[:, t], k[:, t], v[:, t], s1), f(*(x[:, t].clone() for x in (q, k, v)), s2))
        assert torch.equal(s1, s2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_tensors_off_a_16_byte_boundary(gdn, dtype):  # noqa: F811
    """Contiguous and one element off: the same bits as from a boundary, in every operator."""
    def off(t):
        if t is None:
            return None
        o = torch.cat([t.new_zeros(1), t.reshape(-1)])[1:].view(t.shape)
        assert o.is_contiguous() and o.data_ptr() % 16
        return o

    def same(a, b):
        for x, y in zip(a, b):
            assert (x is None and y is None) or torch.equal(x, y)

    i = inputs(dtype, 2, 70, 1, 2, 64, 32, seed=52)
    o = {k: off(t) if isinstance(t, torch.Tensor) else t for k, t in i.items()}
    fwd = lambda i: gdn.selective_scan_fwd(i["c"], i["b"], i["x"], i["dt"], i["A"], D=i["D"], dt_bias=i["bias"],  # noqa: E731
                                           initial_state=i["h0"])
    bwd = lambda i: gdn.selective_scan_bwd(i["c"], i["b"], i["x"], i["dt"], i["A"], i["dy"], dht=i["dht"], D=i["D"],  # noqa: E731
                                           dt_bias=i["bias"], initial_state=i["h0"])
    same(fwd(o), fwd(i))
    same(bwd(o), bwd(i))
    one = lambda i: [i[k][:, 0].contiguous() for k in ("c", "b", "x", "dt")]  # noqa: E731
    s1, s2 = i["h0"].clone(), i["h0"].clone()
    args = one(i)
    gate = -args[3].float().abs()
    same([gdn.selective_scan_step(*map(off, args), off(i["A"]), s1), s1], [gdn.selective_scan_step(*args, i["A"], s2), s2])
    same([gdn.gated_delta_rule_step(*map(off, args[:3]), off(gate), off(args[3]), s1), s1],
         [gdn.gated_delta_rule_step(*args[:3], gate, args[3], s2), s2])
