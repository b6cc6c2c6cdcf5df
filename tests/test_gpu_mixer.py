"""GPU parity of the sequence-mixer operators (short convolution, selective
scan, single-token steps, layer norm) against plain 64-bit forms.

Tolerances, as relative Frobenius errors: ONE[dtype] for an output that is
computed in fp32 and rounded once (half a step, plus fp32 sums); SCAN[dtype]
for the bf16 scan's products, whose operands are rounded as well (the weighted
products inside a chunk and the state, each by half a step at the most, and
the output); F32 for whatever is held in fp32 (the library's bound for fp32)."""
import numpy as np
import pytest
import torch

from tests import mixer_ref as ref
from tests.mixer_ref import DT, dbl, near, near_sum
from tests.gpu_util import announce

pytestmark = pytest.mark.gpu

F32 = 1e-5
ONE = {"bf16": 2.0 ** -8 + F32, "f32": F32}
SCAN = {"bf16": 2 * 2.0 ** -8, "f32": F32}


@pytest.fixture(scope="module")
def gdn():
    import gated_deltanet_chunked_gdn_amd as g
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    g.lib()
    return g


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape, dt=torch.float32, s=1.0):
    return (s * torch.randn(*shape, generator=g)).to(dt).cuda()


def cu_of(lens):
    return None if lens is None else torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32)


# ---------------------------------------------------------------- convolution

CONV = [
    # dtype, B, T, D, W, lens, bias, state, act, weights in fp32
    ("bf16", 1, 1, 8, 4, None, True, True, "silu", False),
    ("bf16", 2, 3, 33, 4, None, False, False, "silu", False),
    ("bf16", 2, 130, 264, 3, None, True, False, None, True),
    ("f32", 1, 77, 36, 2, None, True, True, "silu", True),
    ("f32", 3, 65, 5, 4, None, False, True, "silu", True),
    ("bf16", 1, 0, 64, 4, [0, 1, 2, 0, 3, 200, 70, 0], True, True, "silu", False),
    ("f32", 1, 0, 129, 3, [5, 0, 1, 1, 90], True, True, "silu", True),
    ("bf16", 1, 0, 16, 4, [0, 0], True, True, "silu", False),
    ("bf16", 1, 3000, 2056, 4, None, True, False, "silu", False),
]


def conv_inputs(case, seed=0, wide=False):
    dtype, B, T, D, W, lens, bias, state, act, wf = case
    g = gen(seed)
    dt = DT[dtype]
    wd = torch.float32 if wf else dt
    T = sum(lens) if lens is not None else T
    N = len(lens) if lens is not None else B
    x = randn(g, B, T, D + (24 if wide else 0), dt=dt)
    x = x[..., 8:8 + D] if wide else x
    w = randn(g, D, W, dt=wd, s=W ** -0.5)
    b = randn(g, D, dt=wd, s=0.3) if bias else None
    h0 = randn(g, N, W - 1, D, dt=dt) if state else None
    dy = randn(g, B, T, D, dt=dt)
    dht = randn(g, N, W - 1, D, dt=dt) if state else None
    return x, w, b, h0, dy, dht, cu_of(lens), act


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("case", CONV)
def test_conv(gdn, case, wide):
    announce(f"conv {case} wide={wide}")
    dtype = case[0]
    x, w, b, h0, dy, dht, cu, act = conv_inputs(case, wide=wide)
    y, ht = gdn.causal_conv_fwd(x, w, b, initial_state=h0, cu_seqlens=cu, activation=act)
    f = lambda x, w, b, h0: ref.conv(x, w, b, h0, cu, act)  # noqa: E731
    ry, rht = f(dbl(x), dbl(w), dbl(b), dbl(h0))
    near("y", y, ry, ONE[dtype])
    assert torch.equal(ht.cpu().double(), rht)  # copies of inputs
    got = gdn.causal_conv_bwd(x, w, b, dy, initial_state=h0, dfinal_state=dht, cu_seqlens=cu, activation=act)
    if x.numel() == 0:
        assert not got[1].any() and not got[2].any()
        near("dh0", got[3], dbl(dht), 0)
        return
    want = ref.grads(f, [x, w, b, h0], [dy, dht])
    for n, a, r in zip(("dx", "dw", "db", "dh0"), got, want):
        near(n, a, r, ONE[dtype])


def test_conv_gradient_against_differences(gdn):
    """The directional derivative of sum(y dy) + sum(ht dht), by central differences of the 64-bit form."""
    case = ("f32", 1, 0, 20, 4, [9, 0, 2, 30], True, True, "silu", True)
    x, w, b, h0, dy, dht, cu, act = conv_inputs(case, seed=3)
    got = gdn.causal_conv_bwd(x, w, b, dy, initial_state=h0, dfinal_state=dht, cu_seqlens=cu, activation=act)
    args = [dbl(t) for t in (x, w, b, h0)]
    g = gen(9)
    dirs = [torch.randn(t.shape, generator=g, dtype=torch.float64) for t in args]

    def value(e):
        y, ht = ref.conv(*[t + e * d for t, d in zip(args, dirs)], cu, act)
        return float((y * dbl(dy)).sum() + (ht * dbl(dht)).sum())

    want = (value(1e-5) - value(-1e-5)) / 2e-5
    have = sum(float((dbl(a) * d).sum()) for a, d in zip(got, dirs))
    size = sum(float((dbl(a) * d).abs().sum()) for a, d in zip(got, dirs))
    assert abs(have - want) <= 1e-6 * size


@pytest.mark.parametrize("dtype,B,D,W,act", [("bf16", 1, 33, 4, "silu"), ("bf16", 37, 256, 2, None), ("f32", 5, 132, 3, "silu"),
                                             ("bf16", 3, 1032, 4, "silu")])
@pytest.mark.parametrize("pool", [False, True])
def test_conv_step(gdn, dtype, B, D, W, act, pool):
    announce(f"conv_step {dtype} {B} {D} {W} pool={pool}")
    g, dt = gen(5), DT[dtype]
    slots = B + 4 if pool else B
    x, w, b = randn(g, B, D, dt=dt), randn(g, D, W, dt=dt), randn(g, D, dt=dt)
    st = randn(g, slots, W - 1, D, dt=dt)
    idx = torch.randperm(slots, generator=g)[:B].int().cuda() if pool else None
    live = torch.ones(B, dtype=torch.bool)
    if pool and B > 3:
        idx[1], idx[2], idx[3] = -1, slots, idx[0]  # outside, outside, named before
        live[1:4] = False
    at = idx.cpu().long()[live] if pool else torch.arange(B)
    old = st.clone()
    y = gdn.causal_conv_step(x, st, w, b, activation=act, state_indices=idx)
    z = torch.cat([dbl(old)[at], dbl(x)[live][:, None]], 1)
    pre = (z * dbl(w).t()).sum(1) + dbl(b)
    want = torch.zeros(B, D, dtype=torch.float64)
    want[live] = ref.silu(pre) if act else pre
    near("y", y, want, ONE[dtype])
    new = dbl(old)
    new[at] = z[:, 1:]
    assert torch.equal(st.cpu().double(), new)


# ---------------------------------------------------------------- scan

SCANS = [
    # dtype, B, T, Hq, Hv, K, V, lens, state, softplus, skip, bias
    ("bf16", 1, 1, 1, 1, 32, 32, None, False, True, True, True),
    ("bf16", 2, 65, 1, 2, 64, 64, None, True, True, True, True),
    ("bf16", 1, 200, 2, 6, 128, 64, None, True, False, False, False),
    ("bf16", 1, 130, 1, 4, 64, 128, None, False, True, True, False),
    ("bf16", 1, 96, 1, 1, 128, 128, None, True, True, False, True),
    ("bf16", 1, 0, 1, 8, 128, 64, [0, 1, 63, 64, 65, 0, 129, 0], True, True, True, True),
    ("bf16", 1, 0, 2, 2, 32, 128, [70, 3], False, True, True, True),
    ("bf16", 1, 0, 2, 10, 128, 32, [5, 0, 170], True, True, True, True),
    ("f32", 1, 70, 1, 2, 32, 64, None, True, True, True, True),
    ("f32", 1, 0, 2, 2, 64, 32, [0, 1, 64, 90], True, True, True, True),
    ("f32", 2, 33, 1, 3, 64, 64, None, False, False, True, False),
    ("bf16", 1, 1100, 1, 2, 64, 32, None, True, True, True, True),
    ("bf16", 1, 150, 2, 8, 32, 64, None, True, True, True, True),
    ("bf16", 1, 0, 1, 3, 32, 32, [64, 0, 2, 31], False, True, True, False),
]


def scan_inputs(case, seed=1, wide=False):
    dtype, B, T, Hq, Hv, K, V, lens, state, softplus, skip, bias = case
    g, dt = gen(seed), DT[dtype]
    T = sum(lens) if lens is not None else T
    N = len(lens) if lens is not None else B
    if wide:  # c, b, x as slices of one projection
        all_ = randn(g, B, T, 2 * Hq * K + Hv * V + 16, dt=dt)
        c = all_[..., :Hq * K].unflatten(-1, (Hq, K))
        b = all_[..., Hq * K:2 * Hq * K].unflatten(-1, (Hq, K))
        x = all_[..., 2 * Hq * K:2 * Hq * K + Hv * V].unflatten(-1, (Hv, V))
    else:
        c, b, x = randn(g, B, T, Hq, K, dt=dt), randn(g, B, T, Hq, K, dt=dt), randn(g, B, T, Hv, V, dt=dt)
    A = -(0.5 + 8 * torch.rand(Hv, generator=g)).cuda()
    D = randn(g, Hv) if skip else None
    dt_bias = randn(g, Hv, s=0.5) - 3 if bias else None
    z = randn(g, B, T, Hv, s=0.7)
    dtv = (z if softplus else z.abs() * 0.05).to(dt)
    h0 = randn(g, N, Hv, K, V, s=0.3) if state else None
    dy = randn(g, B, T, Hv, V, dt=dt)
    dht = randn(g, N, Hv, K, V, s=0.3) if state else None
    return c, b, x, dtv, A, D, dt_bias, h0, dy, dht, cu_of(lens), softplus


SCAN_OUT = ("dc", "db", "dx", "ddt", "dA", "dD", "ddt_bias", "dh0")


def check_scan_grads(got, inputs, dy, dht, cu, sp, dtype):
    heads = inputs[3].shape  # [B, T, Hv]: A, D and dt_bias token by token, for the terms of their sums
    inputs = [t.expand(heads) if t is not None and i in (4, 5, 6) else t for i, t in enumerate(inputs)]
    want = ref.grads(lambda *a: ref.scan(*a, cu, sp), inputs, [dy, dht])
    for n, a, r in zip(SCAN_OUT, got, want):
        if n in ("dA", "dD", "ddt_bias"):
            near_sum(n, a, r, F32)
        else:
            near(n, a, r, F32 if n == "dh0" else SCAN[dtype])


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("case", SCANS)
def test_scan_fwd(gdn, case, wide):
    announce(f"scan_fwd {case} wide={wide}")
    c, b, x, dt, A, D, bias, h0, _, _, cu, sp = scan_inputs(case, wide=wide)
    y, ht = gdn.selective_scan_fwd(c, b, x, dt, A, D=D, dt_bias=bias, dt_softplus=sp, initial_state=h0, cu_seqlens=cu)
    ry, rht = ref.scan(*[dbl(t) for t in (c, b, x, dt, A, D, bias, h0)], cu, sp)
    near("y", y, ry, SCAN[case[0]])
    near("ht", ht, rht, F32)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("case", SCANS)
def test_scan_bwd(gdn, case, wide):
    announce(f"scan_bwd {case} wide={wide}")
    c, b, x, dt, A, D, bias, h0, dy, dht, cu, sp = scan_inputs(case, seed=2, wide=wide)
    got = gdn.selective_scan_bwd(c, b, x, dt, A, dy, dht=dht, D=D, dt_bias=bias, dt_softplus=sp, initial_state=h0,
                                 cu_seqlens=cu)
    check_scan_grads(got, (c, b, x, dt, A, D, bias, h0), dy, dht, cu, sp, case[0])


def test_scan_gradient_against_differences(gdn):
    case = ("f32", 1, 0, 1, 2, 32, 32, [40, 0, 1, 70], True, True, True, True)
    c, b, x, dt, A, D, bias, h0, dy, dht, cu, sp = scan_inputs(case, seed=4)
    got = gdn.selective_scan_bwd(c, b, x, dt, A, dy, dht=dht, D=D, dt_bias=bias, dt_softplus=sp, initial_state=h0,
                                 cu_seqlens=cu)
    args = [dbl(t) for t in (c, b, x, dt, A, D, bias, h0)]
    g = gen(11)
    for k, name in enumerate(SCAN_OUT):  # one input moved at a time
        d = torch.randn(args[k].shape, generator=g, dtype=torch.float64)

        def value(e):
            y, ht = ref.scan(*[t + e * d if i == k else t for i, t in enumerate(args)], cu, sp)
            return float((y * dbl(dy)).sum() + (ht * dbl(dht)).sum())

        want = (value(1e-6) - value(-1e-6)) / 2e-6
        have, size = float((dbl(got[k]) * d).sum()), float((dbl(got[k]) * d).abs().sum())
        # fp32 sums on our side, cancellation in the difference (1e-16 of the value over 2e-6) on the other
        assert abs(have - want) <= F32 * size + 1e-10 * abs(value(0.0)), name


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scan_growing_state(gdn, dtype):
    """A > 0: the state grows; nothing divides by a decay."""
    c, b, x, dt, A, D, bias, h0, dy, dht, cu, sp = scan_inputs((dtype, 1, 150, 1, 2, 32, 32, None, True, True, True, True))
    A = A.abs() * 0.02
    y, ht = gdn.selective_scan_fwd(c, b, x, dt, A, D=D, dt_bias=bias, initial_state=h0)
    ry, rht = ref.scan(*[dbl(t) for t in (c, b, x, dt, A, D, bias, h0)], cu, sp)
    near("y", y, ry, SCAN[dtype])
    near("ht", ht, rht, F32)


def test_scan_extreme_steps(gdn):
    """Steps so long that a token forgets everything, and so short that it adds nothing."""
    c, b, x, dt, A, D, bias, h0, dy, dht, cu, sp = scan_inputs(("bf16", 1, 140, 1, 2, 64, 64, None, True, True, True, True))
    dt[:, ::7] = 300.0
    dt[:, 3::7] = -300.0
    y, ht = gdn.selective_scan_fwd(c, b, x, dt, A, D=D, dt_bias=bias, initial_state=h0)
    ry, rht = ref.scan(*[dbl(t) for t in (c, b, x, dt, A, D, bias, h0)], cu, sp)
    near("y", y, ry, SCAN["bf16"])
    near("ht", ht, rht, F32)
    got = gdn.selective_scan_bwd(c, b, x, dt, A, dy, dht=dht, D=D, dt_bias=bias, initial_state=h0)
    check_scan_grads(got, (c, b, x, dt, A, D, bias, h0), dy, dht, cu, sp, "bf16")


@pytest.mark.parametrize("step", [1e-4, 0.3, 2.0, 9.0, 18.0, 40.0, "mixed"])
def test_scan_decay_regimes(gdn, step):
    """Log decays a token from nothing to all (18 is just short of what counts
    as all), and each kind beside the others in one chunk."""
    announce(f"scan decays {step}")
    g = gen(17)
    c, b, x, _, _, D, _, h0, dy, dht, _, _ = scan_inputs(("bf16", 1, 150, 1, 2, 64, 64, None, True, True, True, True))
    if step == "mixed":
        d = torch.tensor([1e-4, 0.3, 2.0, 9.0, 18.0, 40.0, 200.0])[torch.randint(0, 7, (1, 150, 2), generator=g)]
    else:
        d = step * (0.8 + 0.4 * torch.rand(1, 150, 2, generator=g))
    A = torch.tensor([-1.0, -0.5]).cuda()
    dt = (d / torch.tensor([1.0, 0.5])).bfloat16().cuda()
    y, ht = gdn.selective_scan_fwd(c, b, x, dt, A, D=D, dt_softplus=False, initial_state=h0)
    ry, rht = ref.scan(*[dbl(t) for t in (c, b, x, dt, A, D)], None, dbl(h0), None, False)
    near("y", y, ry, SCAN["bf16"])
    near("ht", ht, rht, F32)
    got = gdn.selective_scan_bwd(c, b, x, dt, A, dy, dht=dht, D=D, dt_softplus=False, initial_state=h0)
    check_scan_grads(got, (c, b, x, dt, A, D, None, h0), dy, dht, None, False, "bf16")


def test_scan_many_short_sequences(gdn):
    """More sequences than segments would need, single tokens and empty ones."""
    lens = [int(v) for v in torch.randint(0, 5, (300,), generator=gen(23))] + [200]
    case = ("bf16", 1, 0, 2, 4, 32, 32, lens, True, True, True, True)
    c, b, x, dt, A, D, bias, h0, dy, dht, cu, sp = scan_inputs(case)
    y, ht = gdn.selective_scan_fwd(c, b, x, dt, A, D=D, dt_bias=bias, initial_state=h0, cu_seqlens=cu)
    ry, rht = ref.scan(*[dbl(t) for t in (c, b, x, dt, A, D, bias, h0)], cu, sp)
    near("y", y, ry, SCAN["bf16"])
    near("ht", ht, rht, F32)
    got = gdn.selective_scan_bwd(c, b, x, dt, A, dy, dht=dht, D=D, dt_bias=bias, initial_state=h0, cu_seqlens=cu)
    check_scan_grads(got, (c, b, x, dt, A, D, bias, h0), dy, dht, cu, sp, "bf16")


def test_scan_batch_by_batch_is_the_batch(gdn):
    """Rows of a batch do not meet: each alone gives the batch's values, cut into
    other segments."""
    case = ("bf16", 2, 130, 1, 8, 64, 64, None, True, True, True, True)
    c, b, x, dt, A, D, bias, h0, *_ = scan_inputs(case)
    y, ht = gdn.selective_scan_fwd(c, b, x, dt, A, D=D, dt_bias=bias, initial_state=h0)
    for i in range(2):
        r = slice(i, i + 1)
        y1, ht1 = gdn.selective_scan_fwd(c[r], b[r], x[r], dt[r], A, D=D, dt_bias=bias, initial_state=h0[r])
        near("y", y1, dbl(y[r]), SCAN["bf16"])
        near("ht", ht1, dbl(ht[r]), F32)


def test_scan_a_nan_stays_in_its_sequence(gdn):
    lens = [70, 30, 64]
    c, b, x, dt, A, D, bias, h0, dy, dht, cu, sp = scan_inputs(("bf16", 1, 0, 1, 2, 64, 64, lens, True, True, True, True))
    clean = gdn.selective_scan_fwd(c, b, x, dt, A, D=D, dt_bias=bias, initial_state=h0, cu_seqlens=cu)
    x2 = x.clone()
    x2[0, 75] = float("nan")
    y, ht = gdn.selective_scan_fwd(c, b, x2, dt, A, D=D, dt_bias=bias, initial_state=h0, cu_seqlens=cu)
    keep = torch.ones(164, dtype=torch.bool)
    keep[70:100] = False
    assert torch.equal(y[0, keep], clean[0][0, keep]) and torch.equal(ht[[0, 2]], clean[1][[0, 2]])
    assert bool(torch.isnan(y[0, 75:100]).all())


# ---------------------------------------------------------------- steps


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,Hq,Hv,K,V", [(1, 1, 1, 32, 32), (3, 2, 6, 64, 128), (5, 2, 4, 128, 64), (70, 1, 1, 128, 128)])
@pytest.mark.parametrize("pool", [False, True])
def test_steps(gdn, dtype, B, Hq, Hv, K, V, pool):
    announce(f"steps {dtype} {B} {Hq} {Hv} {K} {V} pool={pool}")
    g, dt = gen(7), DT[dtype]
    slots = B + 3 if pool else B
    q, k, v = randn(g, B, Hq, K, dt=dt, s=K ** -0.5), randn(g, B, Hq, K, dt=dt, s=K ** -0.5), randn(g, B, Hv, V, dt=dt)
    gate, beta = -torch.rand(B, Hv, generator=g).cuda(), torch.rand(B, Hv, generator=g).to(dt).cuda()
    st = randn(g, slots, Hv, K, V)
    idx = torch.randperm(slots, generator=g)[:B].int().cuda() if pool else None
    live = torch.ones(B, dtype=torch.bool)
    if pool and B > 3:
        idx[1], idx[2], idx[B - 1] = -1, slots + 5, idx[0]
        live[1:3] = False
        live[B - 1] = False
    at = idx.cpu().long()[live] if pool else torch.arange(B)

    def check(run, want_of):
        s = st.clone()
        o = run(s)
        ro, rs = want_of(dbl(st)[at])
        want, new = torch.zeros(B, Hv, V, dtype=torch.float64), dbl(st)
        want[live], new[at] = ro, rs
        near("o", o, want, ONE[dtype])
        near("state", s, new, F32)

    for l2 in (False, True):
        check(lambda s: gdn.gated_delta_rule_step(q, k, v, gate, beta, s, use_qk_l2norm_in_kernel=l2, state_indices=idx),
              lambda s: ref.delta_step(*[dbl(t)[live] for t in (q, k, v, gate, beta)], s, K ** -0.5, l2))
    A, D, bias = -torch.rand(Hv, generator=g).cuda() * 4, randn(g, Hv), randn(g, Hv)
    for sp, Dv, bv in ((True, D, bias), (False, None, None)):
        def want_of(s):
            y, ht = ref.scan(*[dbl(t)[live][:, None] for t in (q, k, v, beta)], dbl(A), dbl(Dv), dbl(bv), s, None, sp)
            return y[:, 0], ht
        check(lambda s: gdn.selective_scan_step(q, k, v, beta, A, s, D=Dv, dt_bias=bv, dt_softplus=sp, state_indices=idx),
              want_of)


# ---------------------------------------------------------------- layer norm

NORMS = [
    # dtype, rows, D, weight, bias, gate, rms, weights in fp32
    ("bf16", 1, 1, True, True, False, False, True),
    ("bf16", 3, 7, True, True, True, False, False),
    ("f32", 17, 33, True, False, True, True, True),
    ("bf16", 300, 128, True, False, True, True, True),
    ("bf16", 65, 256, True, True, False, False, False),
    ("f32", 9, 257, False, False, False, False, True),
    ("bf16", 40, 1000, True, True, True, False, True),
    ("f32", 33, 1024, True, True, True, False, True),
    ("bf16", 2100, 264, True, True, True, False, True),
    ("bf16", 10, 4096, True, True, False, False, True),
    ("f32", 21, 5003, True, True, False, False, True),
    ("bf16", 5, 16384, True, True, True, False, True),
    ("bf16", 5, 16385, True, True, True, False, True),
    ("f32", 34, 20001, True, False, False, True, True),
    ("bf16", 40000, 72, True, True, True, False, True),
    ("f32", 3000, 1500, True, True, False, False, True),
]


@pytest.mark.parametrize("case", NORMS)
def test_norm(gdn, case):
    announce(f"norm {case}")
    dtype, rows, D, hw, hb, hg, rms, wf = case
    g, dt = gen(13), DT[dtype]
    wd = torch.float32 if wf else dt
    x = (randn(g, rows, D) * torch.exp(randn(g, rows, 1)) + 0.5).to(dt)
    w = (1 + randn(g, D, s=0.2)).to(wd) if hw else None
    b = randn(g, D, dt=wd, s=0.2) if hb else None
    gate = randn(g, rows, D, dt=dt) if hg else None
    dy = randn(g, rows, D, dt=dt)
    y, mean, rstd = gdn.layer_norm_fwd(x, w, b, gate=gate, eps=1e-5, rms=rms)
    f = lambda *a: ref.norm(*a, 1e-5, rms)  # noqa: E731
    ry, rm, rr = f(dbl(x), dbl(w), dbl(b), dbl(gate))
    near("y", y, ry, ONE[dtype])
    near("rstd", rstd, rr, F32)
    if rms:
        assert mean is None
    else:
        near("mean", mean, rm, F32)
    got = gdn.layer_norm_bwd(dy, x, w, b, mean, rstd, gate=gate, rms=rms)
    want = ref.grads(lambda *a: f(*a)[:1], [x, w, b, gate], [dy])
    for n, a, r in zip(("dx", "dw", "db", "dgate"), got, want):
        if n == "dx" and D == 1 and not rms:  # a row of one element is its own mean
            assert not a.any()
            continue
        if D == 1 and n == "dw":
            continue
        near(n, a, r, ONE["f32"] if n in ("dw", "db") and wf else ONE[dtype])


def test_norm_constant_and_empty_rows(gdn):
    x = torch.full((3, 100), 7.0, device="cuda")
    y, mean, rstd = gdn.layer_norm_fwd(x, eps=1e-5)
    assert not y.any() and torch.equal(mean, torch.full((3,), 7.0, device="cuda"))
    near("rstd", rstd, torch.full((3,), 1e-5 ** -0.5), F32)
    w = torch.ones(64, device="cuda")
    x = torch.zeros(0, 64, device="cuda")
    y, mean, rstd = gdn.layer_norm_fwd(x, w)
    dx, dw, _, _ = gdn.layer_norm_bwd(x, x, w, None, mean, rstd)
    assert y.shape == dx.shape == (0, 64) and not dw.any()


# ---------------------------------------------------------------- together


@pytest.mark.parametrize("kind", ["delta", "scan"])
def test_mixer_prompt_then_tokens(gdn, kind):
    """convolution -> recurrence -> gated norm over a packed prompt, then token
    by token from the states it left, against the whole sequences at once."""
    announce(f"mixer {kind}")
    g, dt = gen(21), torch.bfloat16
    Hq, Hv, K, V, W = 2, 4, 64, 64, 4
    ch = 2 * Hq * K + Hv * V
    lens, more = [70, 1, 129], 5
    whole = [n + more for n in lens]
    x = randn(g, 1, sum(whole), ch, dt=dt)
    w, bias = randn(g, ch, W, dt=dt, s=0.5), randn(g, ch, dt=dt, s=0.1)
    extra = randn(g, 1, sum(whole), Hv, dt=dt)
    A, dtb, gate, nw = -torch.rand(Hv, generator=g).cuda(), randn(g, Hv), randn(g, 1, sum(whole), Hv, V, dt=dt), \
        1 + randn(g, V, s=0.1)

    def split(z):
        lead = z.shape[:-1]
        q, k, v = z.split([Hq * K, Hq * K, Hv * V], -1)
        return q.reshape(*lead, Hq, K), k.reshape(*lead, Hq, K), v.reshape(*lead, Hv, V)

    def prompt(idx, cu):
        z, cs = gdn.causal_conv_fwd(x[:, idx], w, bias, cu_seqlens=cu)
        q, k, v = split(z)
        if kind == "delta":
            gg = -torch.nn.functional.softplus(extra[:, idx].float())
            o, st = gdn.chunk_gated_delta_rule(q, k, v, gg, torch.sigmoid(extra[:, idx]), output_final_state=True,
                                               cu_seqlens=cu, use_qk_l2norm_in_kernel=True)
        else:
            o, st = gdn.selective_scan_fwd(q, k, v, extra[:, idx], A, dt_bias=dtb, cu_seqlens=cu)
        return gdn.layer_norm_fwd(o, nw, gate=gate[:, idx], rms=True)[0], cs, st

    starts = np.concatenate([[0], np.cumsum(whole)])
    first = torch.cat([torch.arange(a, a + n) for a, n in zip(starts, lens)]).cuda()
    want, _, _ = prompt(torch.arange(sum(whole)).cuda(), cu_of(whole))
    y, cs, st = prompt(first, cu_of(lens))
    near("prompt", y, want[:, first], 2 ** -6)  # two bf16 paths of one value
    for i in range(more):
        at = torch.tensor([a + n + i for a, n in zip(starts, lens)]).cuda()
        z = gdn.causal_conv_step(x[0, at], cs, w, bias)
        q, k, v = split(z)
        e = extra[0, at]
        if kind == "delta":
            o = gdn.gated_delta_rule_step(q, k, v, -torch.nn.functional.softplus(e.float()), torch.sigmoid(e), st,
                                          use_qk_l2norm_in_kernel=True)
        else:
            o = gdn.selective_scan_step(q, k, v, e, A, st, dt_bias=dtb)
        o = gdn.layer_norm_fwd(o, nw, gate=gate[0, at], rms=True)[0]
        near(f"token {i}", o, want[0, at], 2 ** -6)


def test_the_same_bits_again(gdn):
    c, b, x, dt, A, D, bias, h0, dy, dht, cu, sp = scan_inputs(SCANS[5])
    run = lambda: gdn.selective_scan_bwd(c, b, x, dt, A, dy, dht=dht, D=D, dt_bias=bias, initial_state=h0,  # noqa: E731
                                         cu_seqlens=cu)
    for a, r in zip(run(), run()):
        assert torch.equal(a, r)
    x, w, b, h0, dy, dht, cu, act = conv_inputs(CONV[8])
    run = lambda: gdn.causal_conv_bwd(x, w, b, dy)  # noqa: E731
    for a, r in zip(run(), run()):
        assert a is None or torch.equal(a, r)


def all_calls(gdn, seed):
    """A call of every operator on inputs of one seed, device cu_seqlens unchecked: () -> list of outputs."""
    cs = conv_inputs(CONV[5], seed)
    sc = scan_inputs(SCANS[5], seed)
    g = gen(seed)
    ccu, scu = cs[6].cuda(), sc[10].cuda()
    B, Hq, Hv, K, V = 3, 1, 2, 64, 64
    q, k, v = randn(g, B, Hq, K, dt=torch.bfloat16, s=0.1), randn(g, B, Hq, K, dt=torch.bfloat16, s=0.1), \
        randn(g, B, Hv, V, dt=torch.bfloat16)
    beta, gg, st0 = torch.rand(B, Hv, generator=g).bfloat16().cuda(), -torch.rand(B, Hv, generator=g).cuda(), randn(g, B, Hv, K, V)
    xn, wn = randn(g, 50, 256, dt=torch.bfloat16), randn(g, 256)
    cst = randn(g, B, 3, 64, dt=torch.bfloat16)
    xc = randn(g, B, 64, dt=torch.bfloat16)

    def run():
        x, w, b, h0, dy, dht, _, act = cs
        out = list(gdn.causal_conv_fwd(x, w, b, initial_state=h0, cu_seqlens=ccu, check_cu_seqlens=False))
        out += gdn.causal_conv_bwd(x, w, b, dy, initial_state=h0, dfinal_state=dht, cu_seqlens=ccu, check_cu_seqlens=False)
        c, b_, x, dt, A, D, bias, h0, dy, dht, _, sp = sc
        out += gdn.selective_scan_fwd(c, b_, x, dt, A, D=D, dt_bias=bias, initial_state=h0, cu_seqlens=scu,
                                      check_cu_seqlens=False)
        out += gdn.selective_scan_bwd(c, b_, x, dt, A, dy, dht=dht, D=D, dt_bias=bias, initial_state=h0, cu_seqlens=scu,
                                      check_cu_seqlens=False)
        st, cv = st0.clone(), cst.clone()
        out += [gdn.gated_delta_rule_step(q, k, v, gg, beta, st), gdn.selective_scan_step(q, k, v, beta, A[:Hv], st), st]
        out += [gdn.causal_conv_step(xc, cv, w, b), cv]
        y, mean, rstd = gdn.layer_norm_fwd(xn, wn)
        out += [y, mean, rstd] + [t for t in gdn.layer_norm_bwd(y, xn, wn, None, mean, rstd) if t is not None]
        return [t for t in out if t is not None]

    return run


def test_graph_replays_and_other_streams(gdn):
    """Every operator captured into a graph and replayed several times between
    eager calls, and run on a stream of its own, gives the eager bits."""
    run, other = all_calls(gdn, 31), all_calls(gdn, 32)
    want, want2 = run(), other()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = run()
    s.synchronize()
    for a, r in zip(got, want):
        assert torch.equal(a, r)
    graphs = []
    for f in (run, other):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs = f()
        graphs.append((gr, outs))
    for _ in range(4):
        for (gr, outs), w in zip(graphs, (want, want2)):
            for t in outs:
                t.zero_()
            gr.replay()
            eager = other()
            torch.cuda.synchronize()
            for a, r in zip(outs, w):
                assert torch.equal(a, r)
            for a, r in zip(eager, want2):
                assert torch.equal(a, r)


def test_a_bad_device_cu_seqlens_stays_in_bounds(gdn):
    """Unchecked cu_seqlens that decrease or run past the batch: results are
    unspecified, buffers behind the batch stay as they were."""
    x, w, b, h0, dy, dht, cu, act = conv_inputs(CONV[5])
    c, b_, xs, dt, A, D, bias, sh0, sdy, sdht, scu, sp = scan_inputs(SCANS[5])
    for bad in ([0, 500, 3, 10, 400, 7, 90, 276, 100], [-5, 1, 3, 3, 6, 206, 276, 276, 100000]):
        cu = torch.tensor(bad, dtype=torch.int32).cuda()
        gdn.causal_conv_fwd(x, w, b, initial_state=h0, cu_seqlens=cu, check_cu_seqlens=False)
        gdn.causal_conv_bwd(x, w, b, dy, initial_state=h0, dfinal_state=dht, cu_seqlens=cu, check_cu_seqlens=False)
        cu = torch.tensor(bad, dtype=torch.int32).cuda()
        gdn.selective_scan_fwd(c, b_, xs, dt, A, initial_state=sh0, cu_seqlens=cu, check_cu_seqlens=False)
        gdn.selective_scan_bwd(c, b_, xs, dt, A, sdy, dht=sdht, initial_state=sh0, cu_seqlens=cu, check_cu_seqlens=False)
    torch.cuda.synchronize()
    y, ht = gdn.selective_scan_fwd(c, b_, xs, dt, A, D=D, dt_bias=bias, initial_state=sh0, cu_seqlens=scu)
    ry, rht = ref.scan(*[dbl(t) for t in (c, b_, xs, dt, A, D, bias, sh0)], scu, sp)
    near("ht", ht, rht, F32)


def test_fewer_tokens_than_the_batch(gdn):
    """Rows behind the last sequence of an unchecked packed batch are left as they were."""
    x, w, b, h0, dy, dht, cu, act = conv_inputs(("bf16", 1, 100, 64, 4, None, True, False, "silu", False))
    cu = torch.tensor([0, 30, 60], dtype=torch.int32).cuda()
    y = torch.full_like(x, 7.0)
    p, xr, w_, b_ = gdn.mixer._conv_problem(x, w, b, "silu", 2)
    p.N, p.cu_seqlens = 2, cu.data_ptr()
    import ctypes
    rc = gdn.mixer.lib().gdn_causal_conv_fwd(ctypes.byref(p), xr.data_ptr(), w_.data_ptr(), b_.data_ptr(), None, y.data_ptr(),
                                             None, torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    assert bool((y[:, 60:] == 7).all()) and not bool((y[:, :60] == 7).all())


def test_offsets_past_32_bits(gdn):
    """The last rows of tensors of more than 2^31 elements are what the same
    rows give alone."""
    g = torch.Generator(device="cuda").manual_seed(31)
    rnd = lambda *shape, dt=torch.bfloat16: torch.randn(*shape, generator=g, device="cuda", dtype=dt)  # noqa: E731
    T, D = 270_000, 8192
    x, w = rnd(1, T, D), rnd(D, 4)
    announce("offsets conv")
    y, _ = gdn.causal_conv_fwd(x, w)
    one, _ = gdn.causal_conv_fwd(x[:, -40:].clone(), w, initial_state=x[:, -43:-40].clone())
    assert torch.equal(y[:, -40:], one)
    dy = y
    dx, _, _, _ = gdn.causal_conv_bwd(x, w, None, dy)
    one, _, _, _ = gdn.causal_conv_bwd(x[:, -40:].clone(), w, None, dy[:, -40:].clone(),
                                       initial_state=x[:, -43:-40].clone())
    assert torch.equal(dx[:, -40:], one)
    del y, dy, dx
    announce("offsets norm")
    rows = x.view(T * 2, D // 2)
    y, mean, rstd = gdn.layer_norm_fwd(rows, gate=rows)
    dx, _, _, dg = gdn.layer_norm_bwd(rows, rows, None, None, mean, rstd, gate=rows)
    last = rows[-50:].clone()
    yl, ml, rl = gdn.layer_norm_fwd(last, gate=last)
    dxl, _, _, dgl = gdn.layer_norm_bwd(last, last, None, None, ml, rl, gate=last)
    for u, v in ((y, yl), (mean, ml), (rstd, rl), (dx, dxl), (dg, dgl)):
        assert torch.equal(u[-50:], v)
    del y, dx, dg, rows
    announce("offsets scan")
    x = x.view(1, T, 128, 64)
    c, b = rnd(1, T, 2, 32), rnd(1, T, 2, 32)
    dt, A = rnd(1, T, 128), -torch.ones(128, device="cuda")
    cut = T - 200
    cu = torch.tensor([0, cut, T], dtype=torch.int32)
    y, ht = gdn.selective_scan_fwd(c, b, x, dt, A, cu_seqlens=cu)
    tail = [t[:, cut:].clone() for t in (c, b, x, dt)]
    yl, hl = gdn.selective_scan_fwd(*tail, A)
    near("y", y[:, cut:], dbl(yl), SCAN["bf16"])
    near("ht", ht[1:], dbl(hl), F32)
    del y, ht, x
    announce("offsets step")
    slots = 4200  # 4200 x 32 x 128 x 128: 2.2e9 elements
    state = torch.zeros(slots, 32, 128, 128, device="cuda")
    q, k, v = rnd(2, 16, 128), rnd(2, 16, 128), rnd(2, 32, 128)
    gg, beta = -torch.rand(2, 32, generator=g, device="cuda"), rnd(2, 32)
    o = gdn.gated_delta_rule_step(q, k, v, gg, beta, state, state_indices=torch.tensor([slots - 1, 0], dtype=torch.int32).cuda())
    small = torch.zeros(2, 32, 128, 128, device="cuda")
    assert torch.equal(o, gdn.gated_delta_rule_step(q, k, v, gg, beta, small))
    assert torch.equal(state[-1], small[0]) and torch.equal(state[0], small[1])
    assert not state[1:-1].any()
