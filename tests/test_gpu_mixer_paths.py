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


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("act", ["silu", None])
def test_convolution_off_a_boundary(gdn, dtype, act):  # noqa: F811
    """D a multiple of 4, rows off: the form of single channels gives the bits of the wide one's outputs."""
    g, dt = gen(53), DT[dtype]
    lens = [40, 0, 1, 90]
    x, dy = randn(g, 1, sum(lens), 64, dt=dt), randn(g, 1, sum(lens), 64, dt=dt)
    w, b, h0, dht = randn(g, 64, 4, dt=dt), randn(g, 64, dt=dt), randn(g, 4, 3, 64, dt=dt), randn(g, 4, 3, 64, dt=dt)
    off = lambda t: torch.cat([t.new_zeros(1), t.reshape(-1)])[1:].view(t.shape)  # noqa: E731
    kw = dict(cu_seqlens=cu_of(lens), activation=act)
    for a, r in zip(gdn.causal_conv_fwd(off(x), off(w), off(b), initial_state=off(h0), **kw),
                    gdn.causal_conv_fwd(x, w, b, initial_state=h0, **kw)):
        assert torch.equal(a, r)
    got = gdn.causal_conv_bwd(off(x), off(w), off(b), off(dy), initial_state=off(h0), dfinal_state=off(dht), **kw)
    want = gdn.causal_conv_bwd(x, w, b, dy, initial_state=h0, dfinal_state=dht, **kw)
    assert torch.equal(got[0], want[0]) and torch.equal(got[3], want[3])
    for a, r in zip(got[1:3], want[1:3]):  # sums, in another order
        near("sum", a, r, 2 * SCAN[dtype])
    s1, s2 = h0.clone(), off(h0)
    assert torch.equal(gdn.causal_conv_step(x[0, :4], s1, w, b, activation=act),
                       gdn.causal_conv_step(off(x[0, :4]), s2, off(w), off(b), activation=act)) and torch.equal(s1, s2)


# ---------------------------------------------------------------- unchecked cu_seqlens

# (sequences that decrease, run past the batch, overlap, begin late, are negative; 200 tokens)
BAD = [[0, 500, 3, 10, 190, 7, 90, 200, 100], [-5, 1, 3, 3, 6, 150, 200, 200, 100000], [200, 150, 100, 64, 63, 20, 1, 0, -1],
       [0, 200, 0, 200, 0, 200, 0, 200, 0], [-2 ** 31, 2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1, 5, 9, 8, 7, 2 ** 31 - 1],
       [100, 100, 100, 120, 120, 130, 131, 140, 150]]


@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_bad_cu_seqlens_on_the_device_writes_into_the_outputs_only(gdn, dtype, bad):  # noqa: F811
    """Results are unspecified; inputs, and what lies beside outputs and workspace, stay as they were."""
    announce(f"bad cu {dtype} {bad}")
    cu, N, T = torch.tensor(bad, dtype=torch.int64).to(torch.int32).cuda(), len(bad) - 1, 200
    g, dt = gen(61), DT[dtype]
    x, w, b, dy = randn(g, 1, T, 40, dt=dt), randn(g, 40, 4, dt=dt), randn(g, 40, dt=dt), randn(g, 1, T, 40, dt=dt)
    raw_conv(gdn, x, w, b, randn(g, N, 3, 40, dt=dt), dy, randn(g, N, 3, 40, dt=dt), cu)
    i = inputs(dtype, 1, 0, 2, 4, 64, 32, lens=[T] + [0] * (N - 1), seed=62)
    raw_scan(gdn, i, cu)
    i["h0"] = i["dht"] = None
    raw_scan(gdn, i, cu)


# ---------------------------------------------------------------- segments


def test_scan_segments_of_several_chunks_in_one_segment(gdn):  # noqa: F811
    """As many sequences as workgroups: a segment is a sequence, of three chunks, with its states."""
    B, T = 260, 150
    assert segment(gdn, "bf16", B, T, 1, 1, 32, 32, None, True) == 192
    check_scan(gdn, "bf16", None, **inputs("bf16", B, T, 1, 1, 32, 32, seed=71))


@pytest.mark.parametrize("Hq,Hv,K,V,N,seg", [(1, 1, 32, 64, 300, 128), (4, 8, 32, 32, 64, 192), (2, 16, 64, 32, 128, 128),
                                             (8, 16, 128, 64, 32, 192)])
@pytest.mark.parametrize("state", [False, True])
def test_scan_segments_of_several_chunks_joined(gdn, Hq, Hv, K, V, N, seg, state):  # noqa: F811
    """A packed batch whose segments have two or three chunks, one sequence of several of them."""
    announce(f"segments {Hq} {Hv} {K} {V} {N} {state}")
    lens = [int(v) for v in torch.randint(0, 2 * (seg - 64), (N,), generator=gen(72))]
    lens[N // 2], lens[3] = 5 * seg - 7, 0
    most = seg * N if N > 128 else seg * max(N, -(-torch.cuda.get_device_properties(0).multi_processor_count // Hq))
    while sum(lens) > most - 8:
        lens[lens.index(max(lens[:N // 2]))] //= 2
    n = N - 1
    while sum(lens) <= most * (seg - 64) // seg:
        lens[n], n = seg, n - 1
    assert segment(gdn, "bf16", 1, 0, Hq, Hv, K, V, lens, True) == seg, sum(lens)
    check_scan(gdn, "bf16", lens, **inputs("bf16", 1, 0, Hq, Hv, K, V, lens=lens, state=state, seed=73))


@pytest.mark.parametrize("dtype,T", [("bf16", 1), ("bf16", 40), ("bf16", 64), ("f32", 1), ("f32", 16), ("f32", 17)])
@pytest.mark.parametrize("Hq,Hv,K,V", [(1, 1, 32, 32), (2, 6, 64, 64)])
def test_scan_of_one_short_segment_with_states(gdn, dtype, T, Hq, Hv, K, V):  # noqa: F811
    assert segment(gdn, dtype, 3, T, Hq, Hv, K, V, None, False) == {("f32", 17): 16}.get((dtype, T), 64 if dtype == "bf16" else 16)
    check_scan(gdn, dtype, None, **inputs(dtype, 3, T, Hq, Hv, K, V, seed=74))
    lens = [T, 0, 1]
    check_scan(gdn, dtype, lens, **inputs(dtype, 1, 0, Hq, Hv, K, V, lens=lens, seed=75))


@pytest.mark.parametrize("dtype,T", [("bf16", 700), ("f32", 700), ("f32", 2100)])
def test_scan_long(gdn, dtype, T):  # noqa: F811
    check_scan(gdn, dtype, None, **inputs(dtype, 1, T, 2, 4, 64, 64, seed=76))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scan_backward_of_a_growing_state(gdn, dtype):  # noqa: F811
    i = inputs(dtype, 2, 150, 1, 2, 64, 32, seed=77)
    i["A"] = i["A"].abs() * 0.02
    check_scan(gdn, dtype, None, **i)


# ---------------------------------------------------------------- masked tokens and infinities


@pytest.mark.parametrize("mask", [float("-inf"), "lowest"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_step_of_minus_infinity_masks_its_token(gdn, dtype, mask):  # noqa: F811
    """softplus(-inf) = 0: the token adds nothing and forgets nothing, in whole chunks and single places; its output
    is the state's as it stands.  So does the type's lowest value."""
    i = inputs(dtype, 2, 200, 1, 2, 64, 32, seed=81)
    low = mask if mask != "lowest" else torch.finfo(DT[dtype]).min
    i["dt"][0, 40:140] = low
    i["dt"][1, ::3] = low
    i["dt"][1, :64] = low
    j = dict(i, dt=torch.where(i["dt"] == low, -200.0, i["dt"].float()).to(DT[dtype]))  # e^-200: 0 in fp32
    check_scan(gdn, dtype, None, **j)
    kw = dict(D=i["D"], dt_bias=i["bias"], initial_state=i["h0"])
    ins = lambda i: [i[k] for k in ("c", "b", "x", "dt", "A")]  # noqa: E731
    for a, r in zip(gdn.selective_scan_fwd(*ins(i), **kw), gdn.selective_scan_fwd(*ins(j), **kw)):
        assert torch.equal(a, r)
    for a, r in zip(gdn.selective_scan_bwd(*ins(i), i["dy"], dht=i["dht"], **kw),
                    gdn.selective_scan_bwd(*ins(j), i["dy"], dht=i["dht"], **kw)):
        assert torch.equal(a, r)
    s = i["h0"].clone()
    args = [i[k][:, 60] for k in ("c", "b", "x", "dt")]
    args[3] = torch.full_like(args[3], low)
    y = gdn.selective_scan_step(*args, i["A"], s, D=i["D"], dt_bias=i["bias"])
    assert torch.equal(s, i["h0"]) and bool(torch.isfinite(y).all())


@pytest.mark.parametrize("what", ["c", "b", "x", "dt", "dy"])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_an_infinity_stays_in_its_sequence(gdn, dtype, what, value):  # noqa: F811
    lens = [70, 30, 64, 5]
    i = inputs(dtype, 1, 0, 1, 2, 64, 32, lens=lens, seed=82)
    j = dict(i, **{what: i[what].clone()})
    j[what][0, 75] = value
    keep, rows = torch.ones(sum(lens), dtype=torch.bool), [0, 2, 3]
    keep[70:100] = False

    def run(i):
        kw = dict(D=i["D"], dt_bias=i["bias"], initial_state=i["h0"], cu_seqlens=cu_of(lens))
        ins = [i[k] for k in ("c", "b", "x", "dt", "A")]
        return gdn.selective_scan_fwd(*ins, **kw) + gdn.selective_scan_bwd(*ins, i["dy"], dht=i["dht"], **kw)

    for n, a, r in zip(("y", "ht") + SCAN_OUT, run(j), run(i)):
        if n in ("ht", "dh0"):
            assert torch.equal(a[rows], r[rows]), n
        elif n not in ("dA", "dD", "ddt_bias"):
            assert torch.equal(a[0, keep], r[0, keep]), n


# ---------------------------------------------------------------- precision of the gates' gradients


@pytest.mark.parametrize("part", ["S Z", "c S dy", "b Z x"])
@pytest.mark.parametrize("dtype,K,V", [("bf16", 32, 32), ("bf16", 64, 64), ("bf16", 128, 64), ("bf16", 32, 128), ("f32", 32, 32),
                                       ("f32", 64, 64)])
def test_scan_gate_sums_take_states_as_they_are(gdn, dtype, K, V, part):  # noqa: F811
    """dA of sequences of two tokens, from a state, a state's gradient, or both.  dg_t = e^{g_t} <S_{t-1}, Z_t> is a
    sum of K V products; with random signs it is about e^{g_t} |S| |Z| / sqrt(K V), and so is each factor's rounding
    to a part u of itself about u times that.  fp32's u is 2^-24; the sums' own roundings and those of delta and the
    decays are a few of those, 2^-20 leaves 16.  (A factor in two bf16 parts has u = 2^-18.)"""
    announce(f"gate sums {dtype} {K} {V} {part}")
    N, Hv = 40, 8
    i = inputs(dtype, N, 2, 1, Hv, K, V, seed=91)
    i["A"] = -torch.ones(Hv, device="cuda")
    if part == "c S dy":
        i["dht"] = None
    if part == "b Z x":
        i["h0"] = None
    if part != "c S dy":
        i["dy"].zero_()
    x, b, c, dy = (d64(i[k]) for k in ("x", "b", "c", "dy"))
    delta = delta_of(d64(i["dt"]), d64(i["bias"]), True)
    dec = torch.exp(delta * d64(i["A"]))[..., None, None]
    zero = torch.zeros(N, Hv, K, V, dtype=torch.float64, device="cuda")
    S0, Z2 = (zero if t is None else d64(t) for t in (i["h0"], i["dht"]))
    S1 = dec[:, 0] * S0 + delta[:, 0, :, None, None] * b[:, 0, :, :, None] * x[:, 0, :, None]
    Z1 = c[:, 1, :, :, None] * dy[:, 1, :, None] + Z2
    Z0 = c[:, 0, :, :, None] * dy[:, 0, :, None] + dec[:, 1] * Z1
    dg = torch.stack([(dec[:, 0] * S0 * Z0).sum((2, 3)), (dec[:, 1] * S1 * Z1).sum((2, 3))], 1)
    size = torch.stack([dec[:, 0, :, 0, 0] * S0.norm(dim=(2, 3)) * Z0.norm(dim=(2, 3)),
                        dec[:, 1, :, 0, 0] * S1.norm(dim=(2, 3)) * Z1.norm(dim=(2, 3))], 1) / (K * V) ** 0.5
    got = gdn.selective_scan_bwd(i["c"], i["b"], i["x"], i["dt"], i["A"], i["dy"], dht=i["dht"], dt_bias=i["bias"],
                                 initial_state=i["h0"])[4]
    off = (d64(got) - (delta * dg).sum((0, 1))).abs()
    most = 2.0 ** -20 * ((delta * size) ** 2).sum((0, 1)).sqrt()
    assert bool((off <= most).all()), f"dA: {(off / most).tolist()} of the bound"


@pytest.mark.parametrize("K,V", [(32, 32), (64, 64)])
@pytest.mark.parametrize("T", [5, 16, 64])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scan_gate_sums_of_a_few_tokens(gdn, dtype, T, K, V):  # noqa: F811
    """dA where tokens that forget nearly all lie among tokens that forget little: theirs is the longest step and the
    least dg, far below the products of the pairs on either side.  The bound is the one above, 2^-20 of
    delta_t e^{g_t} |S_{t-1}| |Z_t| / sqrt(K V) for each token, joined as independent errors are."""
    announce(f"gate sums of {T} tokens {dtype} {K} {V}")
    N, Hv = 40, 6
    i = inputs(dtype, N, T, 1, Hv, K, V, state=False, seed=92)
    i["A"] = -torch.ones(Hv, device="cuda")
    step = torch.tensor([0.001, 0.001, 0.02, 0.3, 9.0, 14.0])[torch.randint(0, 6, (N, T, Hv), generator=gen(93))]
    i["dt"] = step.to(DT[dtype]).cuda()
    x, b, c, dy, delta = (d64(i[k]) for k in ("x", "b", "c", "dy", "dt"))
    dec = torch.exp(-delta)[..., None, None]
    S, Z = [torch.zeros(N, Hv, K, V, dtype=torch.float64, device="cuda")], [None] * T
    for t in range(T):
        S.append(dec[:, t] * S[t] + delta[:, t, :, None, None] * b[:, t, :, :, None] * x[:, t, :, None])
    after = torch.zeros_like(S[0])
    for t in range(T - 1, -1, -1):
        Z[t] = c[:, t, :, :, None] * dy[:, t, :, None] + after
        after = dec[:, t] * Z[t]
    want = sum((delta[:, t] * (dec[:, t] * S[t] * Z[t]).sum((2, 3))).sum(0) for t in range(T))
    size = sum(((delta[:, t] * dec[:, t, :, 0, 0] * S[t].norm(dim=(2, 3)) * Z[t].norm(dim=(2, 3))) ** 2).sum(0) for t in range(T))
    got = gdn.selective_scan_bwd(i["c"], i["b"], i["x"], i["dt"], i["A"], i["dy"], dt_softplus=False)[4]
    off, most = (d64(got) - want).abs(), 2.0 ** -20 * (size / (K * V)).sqrt()
    assert bool((off <= most).all()), f"dA: {(off / most).tolist()} of the bound"


@pytest.mark.parametrize("dtype,K,V", [("bf16", 128, 64), ("bf16", 64, 64), ("f32", 64, 64)])
def test_scan_gate_sums_of_long_memory(gdn, dtype, K, V):  # noqa: F811
    """dA of tokens that forget little, with the operands that a SiLU leaves (of positive mean): a rounding to one side
    in the states' sums would add up over the tokens that it lives for and over the K V elements of <S, Z>.  A state
    carries roundings of a few 2^-24 of itself, for as long as it lives, so that dA's terms are off together, and all
    by 2^-22 of their sizes at the most."""
    announce(f"gate sums of long memory {dtype} {K} {V}")
    T, Hv = 2048, 8
    i = inputs(dtype, 1, T, 1, Hv, K, V, state=False, seed=94)
    g = gen(95)
    for k in ("c", "b", "x"):
        i[k] = torch.nn.functional.silu(i[k].float()).to(DT[dtype])
    i["A"], i["bias"], i["softplus"] = -torch.ones(Hv, device="cuda"), None, False
    step = torch.logspace(-3, -2, Hv) * torch.exp(0.5 * torch.randn(1, T, Hv, generator=g))
    i["dt"] = step.to(DT[dtype]).cuda()
    leaves = [d64(i[k]) for k in ("c", "b", "x", "dt", "A")]
    A = leaves[4].expand(1, T, Hv).clone().requires_grad_()
    y, _ = scan64(None, *leaves[:4], A, None, None, None, False)
    terms, = torch.autograd.grad((y * d64(i["dy"])).sum(), [A])
    got = gdn.selective_scan_bwd(*[i[k] for k in ("c", "b", "x", "dt", "A")], i["dy"], dt_softplus=False)[4]
    off, most = (d64(got) - terms.sum((0, 1))).abs(), 2.0 ** -22 * terms.abs().sum((0, 1))
    assert bool((off <= most).all()), f"dA: {(off / most).tolist()} of the bound"


# ---------------------------------------------------------------- the step sizes


@pytest.mark.parametrize("lo,hi", [(-85, -30), (-30, -12), (-12, -6), (-6, -2), (-2, 2), (2, 60)])
def test_softplus_is_exact_to_a_few_steps_of_fp32(gdn, lo, hi):  # noqa: F811
    """delta = softplus(dt) as a step leaves it in a zero state (b = x = 1).  An exponential within an ulp (two half
    steps) and a few roundings of a half step each behind it: 8 half steps, 2^-21, at the most.  (dt of -7 is a step
    of 0.001, where such layers begin.)"""
    Hv, B = 64, 512
    z = (lo + (hi - lo) * torch.rand(B, Hv, generator=gen(96))).cuda()
    st = torch.zeros(B, Hv, 32, 32, device="cuda")
    one = torch.ones(B, 1, 32, device="cuda")
    gdn.selective_scan_step(one, one, torch.ones(B, Hv, 32, device="cuda"), z, torch.zeros(Hv, device="cuda"), st)
    want = torch.clamp(z.double(), min=0) + torch.log1p(torch.exp(-z.double().abs()))
    off = ((st[:, :, 0, 0].double() - want) / want).abs().max()
    assert bool(off <= 2.0 ** -21), float(off)
    for dtype in (torch.float32, torch.bfloat16):  # the prompts' forms
        dt = z.view(B, 1, Hv).to(dtype)
        e = torch.ones(B, 1, 1, 32, device="cuda", dtype=dt.dtype)
        _, ht = gdn.selective_scan_fwd(e, e, torch.ones(B, 1, Hv, 32, device="cuda", dtype=dt.dtype), dt, torch.zeros(Hv, device="cuda"))
        want = torch.clamp(dt.double(), min=0) + torch.log1p(torch.exp(-dt.double().abs()))
        # (bf16: delta x enters the products as three bf16 numbers, and a part below 2^-126, which is no normal number,
        # counts as 0 there: the second and the third may be missing, at most 2^-126 each)
        tiny = 2.0 ** -125 if dtype == torch.bfloat16 else 0.0
        off, most = (ht[:, :, 0, 0].double() - want[:, 0]).abs(), 2.0 ** -21 * want[:, 0] + tiny
        assert bool((off <= most).all()), float((off / most).max())


# ---------------------------------------------------------------- again, and in graphs


@pytest.mark.parametrize("dtype,T", [("f32", 400), ("bf16", 700)])
def test_scan_replayed_from_two_graphs_gives_the_eager_bits(gdn, dtype, T):  # noqa: F811
    """Both directions over segments that a carry joins, on two sets of inputs, replayed in turn with eager calls
    between (each graph has its own workspace)."""
    lens = [T, 0, 1, T // 3]
    cu = cu_of(lens).cuda()

    def call(seed):
        i = inputs(dtype, 1, 0, 2, 4, 64, 64, lens=lens, seed=seed)
        kw = dict(D=i["D"], dt_bias=i["bias"], initial_state=i["h0"], cu_seqlens=cu, check_cu_seqlens=False)
        ins = [i[k] for k in ("c", "b", "x", "dt", "A")]
        return lambda: gdn.selective_scan_fwd(*ins, **kw) + gdn.selective_scan_bwd(*ins, i["dy"], dht=i["dht"], **kw)

    runs = [call(98), call(99)]
    want = [f() for f in runs]
    torch.cuda.synchronize()
    graphs = []
    for f in runs:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs = f()
        graphs.append((gr, outs))
    for _ in range(4):
        for (gr, outs), w in zip(graphs, want):
            for t in outs:
                t.zero_()
            gr.replay()
            eager = runs[0]()
            torch.cuda.synchronize()
            assert all(torch.equal(a, r) for a, r in zip(outs, w)) and all(torch.equal(a, r) for a, r in zip(eager, want[0]))
