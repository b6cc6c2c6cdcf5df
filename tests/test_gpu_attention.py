"""GPU parity of linear attention with a decay for each head and of the
channels-last group norm against plain 64-bit forms.

Tolerances, as relative Frobenius errors: ONE[dtype] for an output that is
computed in fp32 and rounded once (half a step, plus fp32 sums); PAIRS[dtype]
for the bf16 passes, whose operands are rounded as well (the weighted products
inside a chunk and the state, each by half a step at the most, and the output);
F32 for whatever is held in fp32 (the library's bound for fp32)."""
import numpy as np
import pytest
import torch

from tests import attention_ref as ref
from tests.gpu_util import announce
from tests.mixer_ref import DT, dbl, grads, near

pytestmark = pytest.mark.gpu

F32 = 1e-5
ONE = {"bf16": 2.0 ** -8 + F32, "f32": F32}
PAIRS = {"bf16": 2 * 2.0 ** -8, "f32": F32}


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


# ---------------------------------------------------------------- linear attention

ATTN = [
    # B, T, Hq, Hv, K, V, lens, state, scale, log decays from .. to
    (1, 1, 1, 1, 32, 32, None, True, None, -0.1, -0.1),
    (2, 3, 1, 2, 64, 32, None, False, None, -1.0, -0.01),
    (1, 64, 2, 2, 128, 128, None, True, 1.0, -0.5, -0.002),
    (3, 65, 1, 3, 32, 128, None, True, -0.3, -2.0, 0.0),
    (1, 33, 2, 4, 128, 64, None, False, None, -0.1, -0.01),
    (1, 700, 1, 2, 128, 128, None, True, None, -0.2, -0.0005),
    (2, 300, 2, 2, 64, 64, None, True, None, -40.0, -3.0),
    (1, 0, 2, 4, 64, 128, [0, 1, 2, 0, 3, 200, 70, 0], True, None, -0.3, -0.003),
    (1, 0, 3, 3, 32, 64, [64, 128, 1, 63, 65], True, 0.5, -0.05, -0.001),
    (1, 0, 1, 8, 128, 32, [400, 0, 17], False, None, -0.05, -0.001),
    (1, 0, 2, 2, 32, 32, [0, 0], True, None, -0.1, -0.1),
    (1, 450, 2, 2, 64, 64, None, True, None, 0.004, 0.001),
]


def attn_inputs(dtype, case, seed=0, wide=False):
    B, T, Hq, Hv, K, V, lens, state, scale, lo, hi = case
    g, dt = gen(seed), DT[dtype]
    T = sum(lens) if lens is not None else T
    N = len(lens) if lens is not None else B
    if wide:  # slices of one projection
        W = (2 * Hq * K + Hv * V)
        x = randn(g, B, T, W + 16, dt=dt)
        q, k, v = x[..., 8:8 + Hq * K], x[..., 8 + Hq * K:8 + 2 * Hq * K], x[..., 8 + 2 * Hq * K:8 + W]
        q, k, v = q.unflatten(-1, (Hq, K)), k.unflatten(-1, (Hq, K)), v.unflatten(-1, (Hv, V))
    else:
        q, k, v = randn(g, B, T, Hq, K, dt=dt), randn(g, B, T, Hq, K, dt=dt), randn(g, B, T, Hv, V, dt=dt)
    decay = torch.linspace(lo, hi, Hv).cuda()
    h0 = randn(g, N, Hv, K, V) if state else None
    do = randn(g, B, T, Hv, V, dt=dt)
    dht = randn(g, N, Hv, K, V, s=0.3) if state else None
    return q, k, v, decay, h0, do, dht, cu_of(lens), scale


def form(decay, cu, scale, K):
    s = K ** -0.5 if scale is None else scale
    return lambda q, k, v, h0: ref.attention(q, k, v, dbl(decay), h0, cu, s)


def check_attention(gdn, dtype, args):
    q, k, v, decay, h0, do, dht, cu, scale = args
    o, ht = gdn.linear_attention_fwd(q, k, v, decay, scale=scale, initial_state=h0, cu_seqlens=cu)
    f = form(decay, cu, scale, q.shape[-1])
    ro, rht = f(dbl(q), dbl(k), dbl(v), dbl(h0))
    near("o", o, ro, PAIRS[dtype])
    near("ht", ht, rht, F32)
    got = gdn.linear_attention_bwd(q, k, v, decay, do, dht=dht, scale=scale, initial_state=h0, cu_seqlens=cu)
    want = grads(f, [q, k, v, h0], [do, dht])
    for n, a, r in zip(("dq", "dk", "dv", "dh0"), got, want):
        near(n, a, r, F32 if n == "dh0" else PAIRS[dtype])


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("case", ATTN)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention(gdn, dtype, case, wide):
    announce(f"attention {dtype} {case} wide={wide}")
    check_attention(gdn, dtype, attn_inputs(dtype, case, wide=wide))


@pytest.mark.parametrize("K", [32, 64, 128])
@pytest.mark.parametrize("V", [32, 64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_of_every_head_size(gdn, dtype, K, V):
    announce(f"attention {dtype} K={K} V={V}")
    check_attention(gdn, dtype, attn_inputs(dtype, (1, 0, 2, 4, K, V, [150, 30, 0, 129], True, None, -0.2, -0.002), seed=K + V))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_without_final_state_or_gradients_of_it(gdn, dtype):
    announce(f"attention {dtype} without states")
    q, k, v, decay, h0, do, dht, cu, scale = attn_inputs(dtype, ATTN[8])
    o, ht = gdn.linear_attention_fwd(q, k, v, decay, scale=scale, cu_seqlens=cu, output_final_state=False)
    assert ht is None
    f = form(decay, cu, scale, q.shape[-1])
    near("o", o, f(dbl(q), dbl(k), dbl(v), None)[0], PAIRS[dtype])
    got = gdn.linear_attention_bwd(q, k, v, decay, do, scale=scale, initial_state=h0, cu_seqlens=cu)  # no dht
    want = grads(f, [q, k, v, h0], [do, None])
    for n, a, r in zip(("dq", "dk", "dv", "dh0"), got, want):
        near(n, a, r, F32 if n == "dh0" else PAIRS[dtype])


def test_attention_gradient_against_differences(gdn):
    """The directional derivative of sum(o do) + sum(ht dht), by central differences of the 64-bit form."""
    q, k, v, decay, h0, do, dht, cu, scale = attn_inputs("f32", ATTN[7], seed=3)
    got = gdn.linear_attention_bwd(q, k, v, decay, do, dht=dht, scale=scale, initial_state=h0, cu_seqlens=cu)
    args = [dbl(t) for t in (q, k, v, h0)]
    g = gen(9)
    dirs = [torch.randn(t.shape, generator=g, dtype=torch.float64) for t in args]
    f = form(decay, cu, scale, q.shape[-1])

    def value(e):
        o, ht = f(*[t + e * d for t, d in zip(args, dirs)])
        return float((o * dbl(do)).sum() + (ht * dbl(dht)).sum())

    want = (value(1e-5) - value(-1e-5)) / 2e-5
    have = sum(float((dbl(a) * d).sum()) for a, d in zip(got, dirs))
    size = sum(float((dbl(a) * d).abs().sum()) for a, d in zip(got, dirs))
    assert abs(have - want) <= 1e-6 * size


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_that_forgets_or_keeps_everything(gdn, dtype):
    """Log decays of -inf, of float32's lowest value, of 0 and in between."""
    announce(f"attention {dtype} decays at the ends")
    args = list(attn_inputs(dtype, (1, 0, 4, 4, 32, 64, [130, 1, 90], True, None, 0, 0), seed=4))
    args[3] = torch.tensor([float("-inf"), torch.finfo(torch.float32).min, 0.0, -87.0]).cuda()
    check_attention(gdn, dtype, args)


@pytest.mark.parametrize("what", ["q", "k", "v", "do"])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_an_infinity_stays_in_its_sequence(gdn, dtype, what, value):
    announce(f"attention {dtype} {what}={value}")
    case = (1, 0, 2, 2, 64, 64, [100, 200, 80], True, None, -0.1, -0.01)
    q, k, v, decay, h0, do, dht, cu, scale = attn_inputs(dtype, case, seed=6)
    run = lambda: (*gdn.linear_attention_fwd(q, k, v, decay, initial_state=h0, cu_seqlens=cu),  # noqa: E731
                   *gdn.linear_attention_bwd(q, k, v, decay, do, dht=dht, initial_state=h0, cu_seqlens=cu))
    want = run()
    {"q": q, "k": k, "v": v, "do": do}[what][0, 170, 1] = value
    got = run()
    for n, (a, r) in enumerate(zip(got, want)):
        a, r = ((t[0], t) if t.shape[0] == 1 else (t, t) for t in (a, r))
        a, r = a[0], r[0]
        if a.shape[0] == 3:  # states
            assert torch.equal(a[[0, 2]], r[[0, 2]])
        else:
            assert torch.equal(a[:100], r[:100]) and torch.equal(a[300:], r[300:])
    bad = got[0][0, 164:300, 1] if what in "qkv" else got[4][0, 100:164, 1]  # o, or dv
    assert not torch.isfinite(bad).all()
    assert torch.equal(got[0][0, 100:164], want[0][0, 100:164])  # chunks before are not reached


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,Hq,Hv,K,V", [(1, 1, 1, 32, 32), (5, 2, 6, 128, 64), (70, 2, 2, 64, 128)])
@pytest.mark.parametrize("pool", [False, True])
def test_attention_step(gdn, dtype, B, Hq, Hv, K, V, pool):
    announce(f"attention_step {dtype} {B} {Hq} {Hv} {K} {V} pool={pool}")
    g, dt = gen(5), DT[dtype]
    slots = B + 4 if pool else B
    q, k, v = randn(g, B, Hq, K, dt=dt), randn(g, B, Hq, K, dt=dt), randn(g, B, Hv, V, dt=dt)
    decay, st = -torch.rand(Hv, generator=g).cuda(), randn(g, slots, Hv, K, V)
    idx = torch.randperm(slots, generator=g)[:B].int().cuda() if pool else None
    live = torch.ones(B, dtype=torch.bool)
    if pool and B > 3:
        idx[1], idx[2], idx[3] = -1, slots, idx[0]  # outside, outside, named before
        live[1:4] = False
    at = idx.cpu().long()[live] if pool else torch.arange(B)
    old = st.clone()
    o = gdn.linear_attention_step(q, k, v, decay, st, state_indices=idx)
    want, new = torch.zeros(B, Hv, V, dtype=torch.float64), dbl(old)
    want[live], new[at] = ref.step(dbl(q)[live], dbl(k)[live], dbl(v)[live], dbl(decay), new[at], K ** -0.5)
    near("o", o, want, ONE[dtype])
    near("state", st, new, F32)
    rest = [i for i in range(slots) if i not in at.tolist()]
    assert torch.equal(st[rest], old[rest])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_steps_go_on_from_a_prompt(gdn, dtype):
    """A prompt's final state, moved on token by token, gives what the whole sequence gives."""
    announce(f"attention steps after a prompt {dtype}")
    q, k, v, decay, h0, *_ = attn_inputs(dtype, (2, 100, 2, 4, 64, 64, None, True, None, -0.2, -0.01), seed=8)
    o, ht = gdn.linear_attention_fwd(q[:, :90], k[:, :90], v[:, :90], decay, initial_state=h0)
    more = [gdn.linear_attention_step(q[:, t], k[:, t], v[:, t], decay, ht) for t in range(90, 100)]
    ro, rht = form(decay, None, None, 64)(dbl(q), dbl(k), dbl(v), dbl(h0))
    near("o", torch.cat([o, torch.stack(more, 1)], 1), ro, PAIRS[dtype])
    near("state", ht, rht, F32)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_behind_the_last_sequence_stay(gdn, dtype):
    """An unchecked cu_seqlens on the device whose last entry is below T: the sequences' results, and nothing
    written behind them."""
    announce(f"attention {dtype} padded")
    for Hq, Hv in ((2, 2), (1, 2)):
        case = (1, 0, Hq, Hv, 32, 64, [90, 0, 133], True, None, -0.1, -0.01)
        q, k, v, decay, h0, do, dht, cu, scale = attn_inputs(dtype, case, seed=12)
        T = q.shape[1]
        pad = lambda t: torch.cat([t, t.new_full((1, 70, *t.shape[2:]), float("nan"))], 1)  # noqa: E731
        args, ends = (pad(q), pad(k), pad(v), decay), cu.cuda()
        want_f = gdn.linear_attention_fwd(q, k, v, decay, initial_state=h0, cu_seqlens=cu)
        want_b = gdn.linear_attention_bwd(q, k, v, decay, do, dht=dht, initial_state=h0, cu_seqlens=cu)
        marks = {}
        real = torch.empty

        def marked(*shape, **kw):  # what the call allocates begins as a pattern
            t = real(*shape, **kw)
            return t.fill_(7) if t.is_floating_point() else t

        torch.empty = marked
        try:
            got_f = gdn.linear_attention_fwd(*args, initial_state=h0, cu_seqlens=ends, check_cu_seqlens=False)
            got_b = gdn.linear_attention_bwd(*args, pad(do), dht=dht, initial_state=h0, cu_seqlens=ends, check_cu_seqlens=False)
        finally:
            torch.empty = real
        del marks
        for a, r in zip((*got_f, *got_b), (*want_f, *want_b)):
            if a.shape == r.shape:
                assert torch.equal(a, r)  # states
            else:
                near("rows", a[:, :T], dbl(r), PAIRS[dtype])  # (segments of another length)
                assert bool((a[:, T:] == 7).all())


BAD = [[-5, 1, 3, 3, 6, 206, 276, 276, 100000], [0, 500, 3, 10, 400, 7, 90, 276, 100], [276] * 9, [0] * 9]


@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_bad_device_cu_seqlens_stays_in_bounds(gdn, dtype, bad):
    """Unchecked cu_seqlens that decrease or run past the batch: results are unspecified; the outputs lie between
    guards, which stay, and the library works on."""
    announce(f"attention {dtype} {bad}")
    args = attn_inputs(dtype, ATTN[7])
    q, k, v, decay, h0, do, dht, cu, scale = args
    ends = torch.tensor(bad, dtype=torch.int32).cuda()
    real, kept = torch.empty, []

    def guarded(*shape, **kw):
        n = 1
        shape = tuple(shape[0]) if len(shape) == 1 and not isinstance(shape[0], int) else shape
        for s in shape:
            n *= s
        size = 1 if kw["dtype"] == torch.uint8 else real(0, **kw).element_size()
        buf = real(8192 + (n * size + 255) // 256 * 256, device=kw["device"], dtype=torch.uint8).fill_(85)
        kept.append((buf, n * size))
        return buf[4096:4096 + n * size].view(kw["dtype"]).view(shape)

    torch.empty = guarded
    try:
        gdn.linear_attention_fwd(q, k, v, decay, initial_state=h0, cu_seqlens=ends, check_cu_seqlens=False)
        gdn.linear_attention_bwd(q, k, v, decay, do, dht=dht, initial_state=h0, cu_seqlens=ends, check_cu_seqlens=False)
    finally:
        torch.empty = real
    torch.cuda.synchronize()
    assert len(kept) >= 8
    for buf, n in kept:
        assert bool((buf[:4096] == 85).all()) and bool((buf[4096 + n:] == 85).all())
    check_attention(gdn, dtype, args)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_tensors_off_a_16_byte_boundary(gdn, dtype):
    announce(f"attention {dtype} off a boundary")
    q, k, v, decay, h0, do, dht, cu, scale = attn_inputs(dtype, ATTN[8], seed=2)
    off = lambda t: torch.cat([t.new_zeros(1), t.reshape(-1)])[1:].view(t.shape)  # noqa: E731
    want = (*gdn.linear_attention_fwd(q, k, v, decay, initial_state=h0, cu_seqlens=cu),
            *gdn.linear_attention_bwd(q, k, v, decay, do, dht=dht, initial_state=h0, cu_seqlens=cu))
    q, k, v, decay, h0, do, dht = (off(t) for t in (q, k, v, decay, h0, do, dht))
    assert q.data_ptr() % 16
    got = (*gdn.linear_attention_fwd(q, k, v, decay, initial_state=h0, cu_seqlens=cu),
           *gdn.linear_attention_bwd(q, k, v, decay, do, dht=dht, initial_state=h0, cu_seqlens=cu))
    for a, r in zip(got, want):
        assert torch.equal(a, r)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_without_tokens(gdn, dtype):
    decay, h0 = torch.full((2,), -0.1).cuda(), torch.randn(3, 2, 32, 64).cuda()
    q, v = torch.empty(3, 0, 1, 32, dtype=DT[dtype]).cuda(), torch.empty(3, 0, 2, 64, dtype=DT[dtype]).cuda()
    o, ht = gdn.linear_attention_fwd(q, q, v, decay, initial_state=h0)
    assert o.shape == v.shape and torch.equal(ht, h0)
    dq, dk, dv, dh0 = gdn.linear_attention_bwd(q, q, v, decay, v, dht=h0, initial_state=h0)
    assert dq.shape == q.shape and dv.shape == v.shape and torch.equal(dh0, h0)


# ---------------------------------------------------------------- group norm

GROUP = [
    # shape, groups, affine, gate, activation, weights in fp32
    ((1, 8), 1, False, False, None, False),
    ((5, 64), 2, True, True, None, True),
    ((37, 4, 24), 3, True, False, "silu", False),
    ((3, 1, 8192), 64, True, True, None, True),
    ((1000, 96), 3, True, True, None, True),
    ((2, 9, 7, 21), 7, True, False, "silu", True),
    ((2, 333, 77), 11, True, False, "silu", True),
    ((1, 1025, 64), 8, True, False, "silu", True),   # 8200 values a group
    ((1, 1024, 64), 8, True, False, "silu", True),   # 8192
    ((2, 2000, 40), 4, True, True, None, True),
    ((3, 700, 1000), 1, False, False, "silu", False),
    ((2, 100, 2600), 2, True, False, None, True),     # more pieces than a workgroup's
    ((1, 3000, 5), 1, True, True, None, True),
    ((1, 40, 601), 1, True, False, "silu", True),     # pieces of one channel, more than a workgroup's
    ((2, 16384), 1, True, True, None, True),          # one position, a group too wide to hold
    ((0, 5, 16), 4, True, True, None, True),
]


def group_inputs(dtype, case, seed=0, shift=0.3):
    shape, G, affine, gate, act, wf = case
    g, dt = gen(seed), DT[dtype]
    wd = torch.float32 if wf else dt
    x = (randn(g, *shape) * torch.exp(randn(g, shape[0], *[1] * (len(shape) - 1), s=0.5)) + shift).to(dt)
    w, b = (1 + randn(g, shape[-1], s=0.2)).to(wd), randn(g, shape[-1], dt=wd, s=0.2)
    return (x, G, w if affine else None, b if affine else None, randn(g, *shape, dt=dt) if gate else None, act,
            randn(g, *shape, dt=dt))


def check_group(gdn, dtype, args, eps=1e-5):
    x, G, w, b, gate, act, dy = args
    y, mean, rstd = gdn.group_norm_fwd(x, G, w, b, gate=gate, activation=act, eps=eps)
    f = lambda x, w, b, gate: ref.group_norm(x, G, w, b, gate, act, eps)  # noqa: E731
    ry, rmean, rrstd = f(dbl(x), dbl(w), dbl(b), dbl(gate))
    near("y", y, ry, ONE[dtype])
    near("mean", mean, rmean, F32)
    near("rstd", rstd, rrstd, F32)
    got = gdn.group_norm_bwd(dy, x, G, w, b, mean, rstd, gate=gate, activation=act)
    want = grads(f, [x, w, b, gate], [dy, None, None])
    for n, a, r in zip(("dx", "dw", "db", "dgate"), got, want):
        near(n, a, r, ONE[dtype])


@pytest.mark.parametrize("case", GROUP)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_group_norm(gdn, dtype, case):
    announce(f"group_norm {dtype} {case}")
    x, G, w, b, gate, act, dy = args = group_inputs(dtype, case)
    if x.shape[0]:
        check_group(gdn, dtype, args)
        return
    y, mean, rstd = gdn.group_norm_fwd(x, G, w, b, gate=gate, activation=act)
    dx, dw, db, dgate = gdn.group_norm_bwd(dy, x, G, w, b, mean, rstd, gate=gate, activation=act)
    assert y.shape == x.shape and mean.shape == (0, G) and not dw.any() and not db.any() and dx.shape == x.shape


def test_group_norm_gradient_against_differences(gdn):
    for act, gated in (("silu", False), (None, True)):
        x, G, w, b, gate, act, dy = group_inputs("f32", ((2, 30, 12), 3, True, gated, act, True), seed=5)
        _, mean, rstd = gdn.group_norm_fwd(x, G, w, b, gate=gate, activation=act)
        got = [t for t in gdn.group_norm_bwd(dy, x, G, w, b, mean, rstd, gate=gate, activation=act) if t is not None]
        args = [dbl(t) for t in (x, w, b) + ((gate,) if gated else ())]
        g = gen(1)
        dirs = [torch.randn(t.shape, generator=g, dtype=torch.float64) for t in args]
        value = lambda e: float((ref.group_norm(*[args[0] + e * dirs[0], G, *[t + e * d for t, d in zip(args[1:3], dirs[1:3])],  # noqa: E731,B023
                                                  args[3] + e * dirs[3] if gated else None, act, 1e-5])[0] * dbl(dy)).sum())
        want = (value(1e-5) - value(-1e-5)) / 2e-5
        have = sum(float((dbl(a) * d).sum()) for a, d in zip(got, dirs))
        size = sum(float((dbl(a) * d).abs().sum()) for a, d in zip(got, dirs))
        assert abs(have - want) <= 1e-6 * size


@pytest.mark.parametrize("shape,G", [((2, 64, 32), 4), ((2, 1300, 64), 4), ((3, 5000, 12), 2)])
def test_group_norm_of_values_far_from_zero(gdn, shape, G):
    """A mean of a thousand deviations, and a first position a thousand deviations from the others, cost the
    variance nothing: x itself is exact, so 1e-5 holds for rstd, and for y what a step of the mean is of a deviation."""
    announce(f"group_norm far {shape}")
    x, G, w, b, gate, act, dy = group_inputs("f32", (shape, G, True, False, None, True), seed=7, shift=1000.0)
    y, mean, rstd = gdn.group_norm_fwd(x, G, w, b)
    ry, rmean, rrstd = ref.group_norm(dbl(x), G, dbl(w), dbl(b), None, None, 1e-5)
    near("mean", mean, rmean, F32)
    near("rstd", rstd, rrstd, F32)
    far = float(rmean.abs().max() * rrstd.max())  # the mean in deviations: its half step is 2^-24 of that
    near("y", y, ry, F32 + 2 * 2.0 ** -24 * far)
    x[:, 0] -= 2000.0
    y, mean, rstd = gdn.group_norm_fwd(x, G, w, b)
    ry, rmean, rrstd = ref.group_norm(dbl(x), G, dbl(w), dbl(b), None, None, 1e-5)
    near("rstd of an outlier", rstd, rrstd, F32)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(4, 50, 32), (2, 1200, 64)])
def test_group_norm_off_a_boundary_and_strided(gdn, dtype, shape):
    announce(f"group_norm {dtype} {shape} off a boundary")
    x, G, w, b, gate, act, dy = group_inputs(dtype, (shape, 4, True, True, None, True), seed=3)
    off = lambda t: torch.cat([t.new_zeros(1), t.reshape(-1)])[1:].view(t.shape)  # noqa: E731
    check_group(gdn, dtype, (off(x), G, off(w), off(b), off(gate), act, off(dy)))
    check_group(gdn, dtype, (x.transpose(0, 1).contiguous().transpose(0, 1), G, w, b, gate, act, dy))


def test_group_norm_keeps_what_is_not_finite_in_its_group(gdn):
    for shape in ((3, 40, 32), (3, 1200, 32)):
        x, G, w, b, gate, act, dy = group_inputs("f32", (shape, 4, True, False, "silu", True), seed=9)
        want = gdn.group_norm_fwd(x, G, w, b, activation=act)
        for value in (float("nan"), float("inf")):
            z = x.clone()
            z[1, 7, 20] = value  # group 2
            got = gdn.group_norm_fwd(z, G, w, b, activation=act)
            hit = torch.zeros(3, 4, dtype=torch.bool)
            hit[1, 2] = True
            for a, r in zip(got[1:], want[1:]):
                assert torch.equal(a.cpu()[~hit], r.cpu()[~hit]) and not torch.isfinite(a.cpu()[hit]).any()
            at = lambda t: t.view(3, -1, 4, 8).permute(0, 2, 1, 3).cpu()  # noqa: E731
            assert torch.equal(at(got[0])[~hit], at(want[0])[~hit]) and torch.isnan(at(got[0])[hit]).all()


# ---------------------------------------------------------------- together


def mixer_calls(gdn, seed):
    """One mixer of this kind, prompt, backward and a token: attention over packed prompts, the gated norm over its
    heads; and a norm over positions."""
    g, bf = gen(seed), torch.bfloat16
    H, D = 4, 64
    lens = [0, 130, 1, 200, 5]
    cu, T = cu_of(lens).cuda(), sum(lens)
    x = randn(g, 1, T, 4 * H * D, dt=bf)
    q, k, v, gate = (t.unflatten(-1, (H, D)) for t in x.chunk(4, -1))
    gate = gate.reshape(T, H * D)
    decay, h0 = -torch.exp2(-torch.arange(1.0, H + 1)).cuda(), randn(g, len(lens), H, D, D)
    w, b, dy = 1 + randn(g, H * D, s=0.1), randn(g, H * D, s=0.1), randn(g, T, H * D, dt=bf)
    maps, dmaps = randn(g, 2, 1500, 48, dt=bf), randn(g, 2, 1500, 48, dt=bf)
    wm, bm = 1 + randn(g, 48, s=0.1), randn(g, 48, s=0.1)

    def run():
        o, ht = gdn.linear_attention_fwd(q, k, v, decay, initial_state=h0, cu_seqlens=cu, check_cu_seqlens=False)
        y, mean, rstd = gdn.group_norm_fwd(o.view(T, H * D), H, w, b, gate=gate)
        do, dw, db, dgate = gdn.group_norm_bwd(dy, o.view(T, H * D), H, w, b, mean, rstd, gate=gate)
        back = gdn.linear_attention_bwd(q, k, v, decay, do.view(1, T, H, D), initial_state=h0, cu_seqlens=cu, check_cu_seqlens=False)
        st = ht.clone()
        o1 = gdn.linear_attention_step(q[0, :5], k[0, :5], v[0, :5], decay, st)
        y1, m1, r1 = gdn.group_norm_fwd(o1.view(5, H * D), H, w, b, gate=gate[:5])
        ym, mm, rm = gdn.group_norm_fwd(maps, 6, wm, bm, activation="silu")
        bm_ = gdn.group_norm_bwd(dmaps, maps, 6, wm, bm, mm, rm, activation="silu")
        return [t for t in (o, ht, y, mean, rstd, do, dw, db, dgate, *back, st, o1, y1, m1, r1, ym, mm, rm, *bm_) if t is not None]

    return run, (q, k, v, gate, decay, h0, w, b, dy, cu)


def test_a_mixer_of_attention_and_norm(gdn):
    announce("attention and norm together")
    run, (q, k, v, gate, decay, h0, w, b, dy, cu) = mixer_calls(gdn, 21)
    o, ht, y, mean, rstd, do, dw, db, dgate, dq, dk, dv, dh0 = run()[:13]
    T, H = q.shape[1], 4

    def f(q, k, v, h0, w, b, gate):
        o, _ = ref.attention(q, k, v, dbl(decay), h0, cu.cpu(), 64 ** -0.5)
        return (ref.group_norm(o.reshape(T, -1), H, w, b, gate, None, 1e-5)[0],)

    args = [q, k, v, h0, w, b, gate]
    near("y", y, f(*[dbl(t) for t in args])[0], 3 * 2.0 ** -8)  # o's roundings, then y's
    want = grads(f, args, [dy])
    # o's and do's roundings and those of the passes' operands and outputs
    for n, a, r in zip(("dq", "dk", "dv", "dh0", "dw", "db", "dgate"), (dq, dk, dv, dh0, dw, db, dgate), want):
        near(n, a, r, 5 * 2.0 ** -8)


def test_graph_replays_and_other_streams(gdn):
    """Captured into graphs and replayed in turn between eager calls, and run on a stream of its own: the eager bits."""
    announce("attention and norm in graphs")
    (run, _), (other, _) = mixer_calls(gdn, 31), mixer_calls(gdn, 32)
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
