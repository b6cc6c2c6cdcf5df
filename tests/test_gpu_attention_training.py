"""Linear attention as an ordinary training step calls it: bf16, as many q-heads as
v-heads, K = V and no initial state, where dq, dk and dv are made in one launch;
and workgroups of 64 columns, which the plan takes where 32 would leave some
compute units a second round (its model of the time: for equal rows
max(1, B H (V / c) p / 256) of a row's chunks at 1.6 us with c = 64 and 1.2 with
c = 32, p = 3 passes backwards and 1 forwards).

The reference is each head by itself as one lower triangular matrix over a
sequence's tokens, in 64 bits.  Besides the bounds of test_gpu_attention an
output's error is compared with that of rounding the 64-bit result to bf16: a
kernel that rounds the pairs, or the state as an operand, once each, adds to the
output's own rounding errors of the same relative size, independent from term to
term, so that with sums of random terms its error is sqrt(2) = 1.41 times the
output's own; 1.5 leaves room for chance.  (One bf16 part of the state's weighted
operand instead of two would make it sqrt(3) where the state decides.)"""
import pytest
import torch

from tests.gpu_util import announce
from tests.mixer_ref import dbl, grads, near, spans
from tests.test_gpu_attention import F32, PAIRS, attn_inputs, form, gdn  # noqa: F401

pytestmark = pytest.mark.gpu


def matrix_form(q, k, v, decay, do, dht, cu, scale):
    """o, final state, dq, dk, dv without an initial state, Hq = Hv."""
    B, T, H, V = v.shape
    K = q.shape[-1]
    q, k, v, do = (dbl(t).reshape(B * T, H, -1).transpose(0, 1).contiguous() for t in (q, k, v, do))
    g, hts = dbl(decay)[:, None], []
    o, dq, dk, dv = torch.zeros_like(v), torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for n, a, b in spans(B, T, cu):
        t = torch.arange(b - a, dtype=torch.float64)
        M = torch.exp(torch.where(t[:, None] >= t, (t[:, None] - t) * g[:, :, None], float("-inf")))
        left = torch.exp((b - a - 1 - t) * g)[..., None]
        x, y, z, d = q[:, a:b] * scale, k[:, a:b], v[:, a:b], do[:, a:b]
        P, D = (x @ y.transpose(1, 2)) * M, (d @ z.transpose(1, 2)) * M
        o[:, a:b], dq[:, a:b] = P @ z, scale * (D @ y)
        dk[:, a:b], dv[:, a:b] = D.transpose(1, 2) @ x, P.transpose(1, 2) @ d
        hts.append((left * y).transpose(1, 2) @ z)
        if dht is not None:
            R = dbl(dht)[n]
            dk[:, a:b] += left * (z @ R.transpose(1, 2))
            dv[:, a:b] += left * (y @ R)
    back = lambda x: x.transpose(0, 1).reshape(B, T, H, -1)  # noqa: E731
    return back(o), torch.stack(hts), back(dq), back(dk), back(dv)


def near_rounding(name, got, ref, times=1.5):
    """got is off by at most `times` what rounding ref to bf16 is."""
    near(name, got, ref, PAIRS["bf16"])
    off, own = float((dbl(got) - ref).norm()), float((ref.bfloat16().double() - ref).norm())
    assert off <= times * own, f"{name}: {off / own:.3g} times the output's own rounding"


TRAIN = [
    # B, T, heads, head size, lens, log decays from .. to
    (1, 130, 2, 32, None, -0.2, -0.002),        # 32 columns
    (2, 200, 3, 64, None, -0.1, -0.01),
    (1, 257, 8, 128, None, -0.5, -0.0005),
    (1, 0, 16, 64, [130, 0, 1, 64, 65, 200], -0.3, -0.001),
    (2, 130, 32, 64, None, -0.3, -0.002),       # 64 columns
    (2, 129, 35, 64, None, -0.3, -0.002),
    (1, 193, 32, 128, None, -0.3, -0.002),
    (1, 200, 33, 128, None, -0.3, -0.002),
    (1, 0, 40, 128, [130, 0, 100, 129, 64, 70], -0.3, -0.002),
    (1, 2500, 1, 64, None, -0.004, -0.004),     # segments
    (1, 2111, 2, 128, None, -0.02, -0.0005),
    (1, 0, 1, 32, [1500, 0, 900], -0.003, -0.003),
]


@pytest.mark.parametrize("late", [False, True])
@pytest.mark.parametrize("case", TRAIN)
def test_gradients_without_an_initial_state(gdn, case, late):  # noqa: F811
    """late: with a gradient of the final state."""
    announce(f"attention training {case} late={late}")
    B, T, H, D, lens, lo, hi = case
    q, k, v, decay, _, do, _, cu, _ = attn_inputs("bf16", (B, T, H, H, D, D, lens, False, None, lo, hi), seed=T + H)
    rows = B if lens is None else len(lens)
    dht = (0.3 * torch.randn(rows, H, D, D, generator=torch.Generator().manual_seed(1))).cuda() if late else None
    want = matrix_form(q, k, v, decay, do, dht, cu, D ** -0.5)
    got = gdn.linear_attention_bwd(q, k, v, decay, do, dht=dht, cu_seqlens=cu)
    assert got[3] is None
    for n, a, r in zip(("dq", "dk", "dv"), got, want[2:]):
        near_rounding(n, a, r)


@pytest.mark.parametrize("case", [
    # B, T, q-heads, v-heads, K, V: 64 columns
    (3, 130, 32, 32, 128, 128), (6, 100, 16, 32, 128, 64), (6, 129, 32, 32, 64, 64), (3, 193, 33, 33, 128, 128),
    (3, 200, 2, 2, 128, 128),  # 32 columns
    (1, 2500, 1, 1, 128, 64),  # segments
])
@pytest.mark.parametrize("last", [False, True])
def test_forward_of_both_widths(gdn, case, last):  # noqa: F811
    """last: with the final state, which is held more exactly towards the end."""
    announce(f"attention forward {case} last={last}")
    B, T, Hq, Hv, K, V = case
    q, k, v, decay, _, do, _, cu, _ = attn_inputs("bf16", (B, T, Hq, Hv, K, V, None, False, None, -0.3, -0.002), seed=T)
    R = Hv // Hq
    ro, rht = matrix_form(q.repeat_interleave(R, 2), k.repeat_interleave(R, 2), v, decay, do, None, cu, K ** -0.5)[:2]
    o, ht = gdn.linear_attention_fwd(q, k, v, decay, output_final_state=last)
    near_rounding("o", o, ro)
    if last:
        near("ht", ht, rht, F32)


@pytest.mark.parametrize("Hq,Hv,K,V", [(1, 1, 32, 32), (1, 4, 64, 64), (2, 2, 128, 64), (3, 9, 32, 128)])
@pytest.mark.parametrize("lens", [[1], [2], [0, 1, 1, 3], [6], [17, 40], [64], [63, 1, 0, 48]])
@pytest.mark.parametrize("state", [False, True])
def test_sequences_of_one_chunk_lose_nothing(gdn, lens, state, Hq, Hv, K, V):  # noqa: F811
    """A few pairs of tokens, or a state alone, decide every output: their roundings do not average out, and those of
    v-heads that share a q-head are not small beside a sum that cancels.  They are held to 2^-17, which beside the
    output's own 2^-9 is nothing: within 5 % of rounding the output alone."""
    announce(f"attention one chunk {lens} {state} {Hq} {Hv} {K} {V}")
    q, k, v, decay, h0, do, dht, cu, scale = attn_inputs("bf16", (1, 0, Hq, Hv, K, V, lens, state, None, -1.0, -0.01), seed=sum(lens))
    f = form(decay, cu, None, K)
    o, ht = gdn.linear_attention_fwd(q, k, v, decay, initial_state=h0, cu_seqlens=cu)
    ro, rht = f(dbl(q), dbl(k), dbl(v), dbl(h0))
    near_rounding("o", o, ro, 1.05)
    near("ht", ht, rht, F32)
    got = gdn.linear_attention_bwd(q, k, v, decay, do, dht=dht, initial_state=h0, cu_seqlens=cu)
    for n, a, r in zip(("dq", "dk", "dv"), got, grads(f, [q, k, v, h0], [do, dht])):
        near_rounding(n, a, r, 1.05)


def test_infinities_of_one_chunk(gdn):  # noqa: F811
    """An infinite state or pair stays what it is: the outputs it does not meet are finite, the others are not."""
    q, k, v, decay, h0, do, dht, cu, scale = attn_inputs("bf16", (2, 5, 1, 2, 32, 64, None, True, None, -0.1, -0.01), seed=3)
    q, k = q.abs() + 0.1, k.abs() + 0.1
    h0[1, 1, 3, 7] = float("inf")
    o, ht = gdn.linear_attention_fwd(q, k, v, decay, initial_state=h0)
    hit = torch.zeros(o.shape, dtype=torch.bool)
    hit[1, :, 1, 7] = True
    assert torch.isfinite(o.cpu()[~hit]).all() and (o.cpu()[hit] == float("inf")).all()
    assert ht[1, 1, 3, 7] == float("inf") and int((~torch.isfinite(ht)).sum()) == 1


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("decay", [0.0, -1e-5])
@pytest.mark.parametrize("T,H", [(20000, 64), (50021, 2)])
def test_returned_states_of_long_sequences(gdn, dtype, decay, T, H):  # noqa: F811
    """Nothing, or next to nothing, forgotten over tens of thousands of tokens of positive mean, in one segment of
    many chunks and in many segments.  A chunk's decay, rounded to fp32, is off by 2^-25 at the most, 313 chunks of it by
    9.4e-6 for the first token and half of that for their sum; a chunk's sum is off by some 2^-24 of the state's size,
    either way."""
    announce(f"attention long states {dtype} {decay} {T} {H}")
    g = torch.Generator("cuda").manual_seed(T)
    dt, K = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype], 64
    q, k, v, do = ((torch.randn(1, T, H, K, generator=g, device="cuda") + 0.5).to(dt) for _ in range(4))
    decays = torch.full((H,), decay, device="cuda")
    h0 = torch.zeros(1, H, K, K, device="cuda")
    _, ht = gdn.linear_attention_fwd(q, k, v, decays)
    dh0 = gdn.linear_attention_bwd(q, k, v, decays, do, initial_state=h0)[3]
    t, l = torch.arange(T, device="cuda", dtype=torch.float64), float(decays[0])
    for h in range(0, H, 13):
        want = (k[0, :, h].double() * torch.exp((T - 1 - t) * l)[:, None]).T.contiguous() @ v[0, :, h].double()
        near(f"ht {h}", ht[0, h], want, F32)
        want = (q[0, :, h].double() * torch.exp((t + 1) * l)[:, None]).T.contiguous() @ do[0, :, h].double() * K ** -0.5
        near(f"dh0 {h}", dh0[0, h], want, F32)


@pytest.mark.parametrize("S,C,G", [(1, 4096, 32), (16384, 96, 8)])
def test_group_norm_sums_over_more_than_2_31_values(gdn, S, C, G):  # noqa: F811
    """dw and db over all samples of a tensor that 32-bit offsets do not reach: sums of 5 * 10^5 and 2 * 10^7 terms
    of either sign, in fp32 over a few thousand of them at a time."""
    announce(f"group norm sums {S} {C}")
    N = (1 << 31) // (S * C) + 5
    x = torch.empty(N, S, C, device="cuda", dtype=torch.bfloat16).normal_()
    dy = torch.empty(N, S, C, device="cuda", dtype=torch.bfloat16).normal_()
    w, b = torch.randn(C, device="cuda"), torch.randn(C, device="cuda")
    _, mean, rstd = gdn.group_norm_fwd(x, G, w, b, activation="silu")
    _, dw, db, _ = gdn.group_norm_bwd(dy, x, G, w, b, mean, rstd, activation="silu")
    rw, rb = torch.zeros(C, dtype=torch.float64, device="cuda"), torch.zeros(C, dtype=torch.float64, device="cuda")
    step = max(1, (1 << 25) // (S * C))
    for a in range(0, N, step):
        z = x[a:a + step].double().view(-1, S, G, C // G)
        xh = ((z - mean[a:a + step].double()[:, None, :, None]) * rstd[a:a + step].double()[:, None, :, None]).view(-1, S, C)
        z = xh * w.double() + b.double()
        s = torch.sigmoid(z)
        dz = dy[a:a + step].double() * s * (1 + z * (1 - s))
        rw += (dz * xh).sum((0, 1))
        rb += dz.sum((0, 1))
    near("dw", dw, rw, F32)
    near("db", db, rb, F32)


def test_more_than_2_31_elements(gdn):  # noqa: F811
    """One sequence whose rows of v, o and their gradients 32-bit offsets do not reach, heads in pairs; with a decay
    that forgets within some 300 tokens its two ends are those of the ends alone."""
    announce("attention of more than 2^31 elements")
    T, Hq, Hv, K, V, n = 263000, 32, 64, 32, 128, 1500
    assert T * Hv * V > 1 << 31
    mk = lambda H, D: torch.empty(1, T, H, D, device="cuda", dtype=torch.bfloat16).normal_()  # noqa: E731
    q, k, v, do = mk(Hq, K), mk(Hq, K), mk(Hv, V), mk(Hv, V)
    decay = torch.full((Hv,), -0.1, device="cuda")
    o, ht = gdn.linear_attention_fwd(q, k, v, decay)
    dq, dk, dv, _ = gdn.linear_attention_bwd(q, k, v, decay, do)
    ends = []
    for part in (slice(0, n), slice(T - n, T)):
        x = [t[:, part].contiguous() for t in (q, k, v, do)]
        ends.append((*gdn.linear_attention_fwd(*x[:3], decay), *gdn.linear_attention_bwd(*x[:3], decay, x[3])))
    # (tokens 1000 and more from the cut, e^-100; steps of bf16 where a sum falls the other way)
    for name, whole, i in (("o", o, 0), ("dq", dq, 2), ("dk", dk, 3), ("dv", dv, 4)):
        near(name + " begins", whole[:, :500], dbl(ends[0][i][:, :500]), PAIRS["bf16"])
        near(name + " ends", whole[:, -500:], dbl(ends[1][i][:, -500:]), PAIRS["bf16"])
    near("ht", ht, dbl(ends[1][1]), F32)
