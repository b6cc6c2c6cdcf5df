"""Linear attention where sequences are cut into segments and the states of their
parts summed up, and where heads share rows: against the token-by-token form in
64 bits.  (Which lengths are cut, and with how many columns a workgroup works, goes
by a model of the time: few heads and long sequences are.)"""
import ctypes

import pytest
import torch

from gated_deltanet_chunked_gdn_amd import mixer
from tests.gpu_util import announce
from tests.mixer_ref import dbl, near
from tests.test_gpu_attention import F32, PAIRS, attn_inputs, check_attention, form, gdn  # noqa: F401

pytestmark = pytest.mark.gpu

LONG = [
    # B, T, Hq, Hv, K, V, lens, state, scale, log decays from .. to
    (1, 2500, 1, 1, 32, 32, None, True, None, -0.01, -0.01),       # segments in one part each
    (1, 2500, 1, 2, 64, 128, None, True, None, -0.3, -0.0005),
    (2, 2111, 1, 1, 128, 64, None, True, None, -0.002, -0.002),
    (1, 0, 1, 1, 64, 64, [1, 2900, 0, 64, 700], True, 1.0, -0.004, -0.004),
    (1, 0, 2, 2, 32, 64, [2048, 0, 2049, 1], False, None, -0.02, -0.0001),
    (1, 2400, 1, 1, 64, 64, None, True, None, -3.0, -3.0),         # tokens of no weight behind the border
    (1, 2400, 1, 2, 64, 64, None, True, None, 0.0, 0.0),           # nothing forgotten
    (1, 2400, 1, 1, 32, 32, None, True, None, 0.002, 0.002),       # growing
]


@pytest.mark.parametrize("case", LONG)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_in_segments(gdn, dtype, case):  # noqa: F811
    announce(f"attention in segments {dtype} {case}")
    check_attention(gdn, dtype, attn_inputs(dtype, case, seed=11))


@pytest.mark.parametrize("T", [65, 300, 512, 513, 1000, 2048, 2049])
@pytest.mark.parametrize("K,V", [(32, 64), (128, 32)])
def test_attention_f32_joins_segments(gdn, T, K, V):  # noqa: F811
    """fp32 sequences of 2 to 33 segments of 64 tokens: few are joined by the passes that read them, more by
    one between; and packed, with lengths that the host does not know."""
    announce(f"attention f32 joined {T} {K} {V}")
    check_attention(gdn, "f32", attn_inputs("f32", (1, T, 1, 2, K, V, None, True, None, -0.05, -0.001), seed=T))
    q, k, v, decay, h0, do, dht, cu, scale = attn_inputs(
        "f32", (1, 0, 1, 1, K, V, [T // 2, 0, 1, T - T // 2 - 1], True, None, -0.02, -0.02), seed=T + 1)
    ro, rht = form(decay, cu, None, K)(dbl(q), dbl(k), dbl(v), dbl(h0))
    o, ht = gdn.linear_attention_fwd(q, k, v, decay, initial_state=h0, cu_seqlens=cu.cuda(), check_cu_seqlens=False)
    near("o", o, ro, PAIRS["f32"])
    near("ht", ht, rht, F32)
    want = gdn.linear_attention_bwd(q, k, v, decay, do, dht=dht, initial_state=h0, cu_seqlens=cu)
    got = gdn.linear_attention_bwd(q, k, v, decay, do, dht=dht, initial_state=h0, cu_seqlens=cu.cuda(), check_cu_seqlens=False)
    for n, x, y in zip(("dq", "dk", "dv", "dh0"), got, want):
        near(n, x, dbl(y), 2 * F32)  # both within F32 of the formula's


def test_attention_in_parts_of_segments(gdn):  # noqa: F811
    """Segments of 512 tokens and more are summed up in four parts; a decay that sees through many of them and
    one that ends inside a part."""
    T, H = 4096, 32
    for lo, hi in ((-0.2, -0.0001), (0.0, 0.0)):
        announce(f"attention in parts {lo} {hi}")
        case = (1, T, H, H, 32, 64, None, True, None, lo, hi)
        q, k, v, decay, h0, do, dht, cu, scale = attn_inputs("bf16", case, seed=2)
        p = mixer.AttnProblem(1, T, H, H, 32, 64, 1, 1, 1.0, 0, 0, 0, None, None)
        states = mixer.lib().gdn_linear_attention_fwd_workspace_size(ctypes.byref(p)) // (H * 32 * 64 * 4)
        assert states in (T // 128, T // 256), states  # parts of 128 or 256 tokens, of segments of four
        o, ht = gdn.linear_attention_fwd(q, k, v, decay, initial_state=h0)
        ro, rht = form(decay, None, None, 32)(dbl(q), dbl(k), dbl(v), dbl(h0))
        near("o", o, ro, PAIRS["bf16"])
        near("ht", ht, rht, F32)
        got = gdn.linear_attention_bwd(q, k, v, decay, do, dht=dht, initial_state=h0)
        # the gradients by their own recurrences: dq like o, the others backwards in time
        a, b, c, d = (dbl(t)[0] for t in (q, k, v, do))
        keep, s = torch.exp(dbl(decay))[:, None, None], 32 ** -0.5
        S, dq = dbl(h0)[0], []
        for t in range(T):
            S = keep * S + b[t][:, :, None] * c[t][:, None, :]
            dq.append(s * (S * d[t][:, None, :]).sum(2))
        Z, dk, dv = dbl(dht)[0], [None] * T, [None] * T
        for t in reversed(range(T)):
            Z = Z + s * a[t][:, :, None] * d[t][:, None, :]
            dk[t], dv[t] = (Z * c[t][:, None, :]).sum(2), (Z * b[t][:, :, None]).sum(1)
            Z = keep * Z
        for n, x, r in zip(("dq", "dk", "dv"), got, (dq, dk, dv)):
            near(n, x[0], torch.stack(r), PAIRS["bf16"])
        near("dh0", got[3][0], Z, F32)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_checked_and_unchecked_lengths_agree(gdn, dtype):  # noqa: F811
    """The host's lengths only choose the segments."""
    announce(f"attention lengths on the host or not {dtype}")
    case = (1, 0, 1, 2, 64, 64, [1800, 3, 0, 900, 64], True, None, -0.1, -0.003)
    q, k, v, decay, h0, do, dht, cu, scale = attn_inputs(dtype, case, seed=5)
    ro, rht = form(decay, cu, None, 64)(dbl(q), dbl(k), dbl(v), dbl(h0))
    for ends, check in ((cu, True), (cu.cuda(), True), (cu.cuda(), False), (cu.cuda().long(), False)):
        o, ht = gdn.linear_attention_fwd(q, k, v, decay, initial_state=h0, cu_seqlens=ends, check_cu_seqlens=check)
        near("o", o, ro, PAIRS[dtype])
        near("ht", ht, rht, F32)


@pytest.mark.parametrize("Hq,Hv", [(8, 8), (8, 16), (16, 16), (3, 9), (16, 64)])
def test_every_head_is_worked_on_once(gdn, Hq, Hv):  # noqa: F811
    """Heads are dealt over the chip in another order than their own."""
    announce(f"attention heads {Hq} {Hv}")
    check_attention(gdn, "bf16", attn_inputs("bf16", (1, 70, Hq, Hv, 32, 64, None, True, None, -1.0, -0.01), seed=Hq))


@pytest.mark.parametrize("T", [1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 192])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_lengths_around_a_chunk(gdn, dtype, T):  # noqa: F811
    announce(f"attention {dtype} T={T}")
    check_attention(gdn, dtype, attn_inputs(dtype, (1, T, 1, 1, 64, 64, None, True, None, -0.05, -0.05), seed=T))


def test_a_returned_state_forgets_nothing_it_can_see(gdn):  # noqa: F811
    """bf16: early tokens enter the state in two parts, the ones a returned state sees in three.  With decays
    from none to one that forgets within a chunk, and early keys 30 times the later ones, it is right to fp32."""
    announce("attention exact states")
    case = (1, 1500, 6, 6, 64, 64, None, True, None, 0, 0)
    q, k, v, decay, h0, do, dht, cu, scale = attn_inputs("bf16", case, seed=8)
    decay = torch.tensor([0.0, -1e-4, -0.003, -0.02, -0.1, -0.9]).cuda()
    k[:, :700] *= 30
    _, ht = gdn.linear_attention_fwd(q, k, v, decay, initial_state=h0)
    _, rht = form(decay, None, None, 64)(dbl(q), dbl(k), dbl(v), dbl(h0))
    for h in range(6):
        near(f"ht {h}", ht[:, h], rht[:, h], 2e-6)  # fp32 sums; two parts alone leave 2.5e-6 of the whole


def test_rows_far_apart_and_offsets_past_32_bits(gdn):  # noqa: F811
    """q, k and v inside one tensor of more than 2^31 elements."""
    announce("attention offsets past 32 bits")
    T, far = 300, 8 * (1 << 20)
    x = torch.zeros(T * far + 1024, dtype=torch.bfloat16, device="cuda")
    assert x.numel() > 1 << 31
    g = torch.Generator().manual_seed(3)
    views = []
    for off in (0, 64, 192):
        t = x.as_strided((1, T, 1, 64), (T * far, far, 64, 1), off)
        t.copy_(torch.randn(1, T, 1, 64, generator=g).bfloat16().cuda())
        views.append(t)
    decay = torch.tensor([-0.02]).cuda()
    o, ht = gdn.linear_attention_fwd(*views, decay)
    f = form(decay, None, None, 64)
    ro, rht = f(*[dbl(t) for t in views], None)
    near("o", o, ro, PAIRS["bf16"])
    near("ht", ht, rht, F32)
    del x, views


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_two_graphs_of_segments(gdn, dtype):  # noqa: F811
    """Segmented calls, forward and backward, captured twice and replayed in turn: the eager bits."""
    announce(f"attention segments in graphs {dtype}")

    def calls(seed):
        q, k, v, decay, h0, do, dht, cu, scale = attn_inputs(dtype, (1, 0, 1, 2, 64, 64, [2600, 5, 0, 800], True, None, -0.1, -0.002),
                                                             seed=seed)
        ends = cu.cuda()

        def run():
            return (*gdn.linear_attention_fwd(q, k, v, decay, initial_state=h0, cu_seqlens=ends, check_cu_seqlens=False),
                    *gdn.linear_attention_bwd(q, k, v, decay, do, dht=dht, initial_state=h0, cu_seqlens=ends, check_cu_seqlens=False))
        return run

    runs = [calls(1), calls(2)]
    wants = [r() for r in runs]
    graphs = []
    for r in runs:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs = r()
        graphs.append((gr, outs))
    for _ in range(3):
        for (gr, outs), want in zip(graphs, wants):
            for t in outs:
                t.zero_()
            gr.replay()
            runs[0]()
            torch.cuda.synchronize()
            for a, b in zip(outs, want):
                assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_broadcast_and_turned_inputs(gdn, dtype):  # noqa: F811
    """Inputs without memory of their own (one head, token or row for all, as a sum's gradient comes) and with
    other orders of dimensions give the bits of their copies, and are left as they were."""
    announce(f"attention of broadcast inputs {dtype}")
    B, T, H, D = 2, 77, 4, 64
    q, k, v, decay, h0, do, dht, cu, scale = attn_inputs(dtype, (B, T, H, H, D, D, None, True, None, -0.5, -0.01), seed=3)
    views = {
        "head": lambda x: x[:, :, :1].expand(B, T, H, D),
        "token": lambda x: x[:, :1].expand(B, T, H, D),
        "row": lambda x: x[:1].expand(B, T, H, D),
        "all": lambda x: x[:1, :1, :1, :1].expand(B, T, H, D),
        "turned": lambda x: x.transpose(1, 2).contiguous().transpose(1, 2),
        "across": lambda x: x.transpose(2, 3).contiguous().transpose(2, 3),
    }
    state = dht[:1, :1].expand(B, H, D, D)
    for name, view in views.items():
        announce(f"  {name}")
        a = [view(x) for x in (q, k, v, do)]
        c = [x.contiguous() for x in a]
        kept = [x.clone() for x in a]
        want = gdn.linear_attention_fwd(*c[:3], decay, initial_state=state.contiguous())
        got = gdn.linear_attention_fwd(*a[:3], decay, initial_state=state)
        want += gdn.linear_attention_bwd(*c[:3], decay, c[3], dht=state.contiguous(), initial_state=h0)
        got += gdn.linear_attention_bwd(*a[:3], decay, a[3], dht=state, initial_state=h0)
        s0, s1 = h0.clone(), h0.clone()
        want += (gdn.linear_attention_step(*(x[:, 0].contiguous() for x in c[:3]), decay, s0), s0)
        got += (gdn.linear_attention_step(*(x[:, 0] for x in a[:3]), decay, s1), s1)
        for x, y in zip(got, want):
            assert torch.equal(x, y), name
        assert all(torch.equal(x, y) for x, y in zip(a, kept)), name
        w, b = torch.ones(D, device="cuda"), torch.zeros(D, device="cuda")
        x, dy = a[2], a[3]
        ref = gdn.group_norm_fwd(c[2], 8, w, b)
        fwd = gdn.group_norm_fwd(x, 8, w, b)
        ref += gdn.group_norm_bwd(c[3], c[2], 8, w, b, *ref[1:])[:3]
        fwd += gdn.group_norm_bwd(dy, x, 8, w, b, *fwd[1:])[:3]
        for x, y in zip(fwd, ref):
            assert torch.equal(x, y), name


@pytest.mark.parametrize("S,C,G", [(1, 4096, 32), (16384, 96, 8)])
def test_group_norm_of_more_than_2_31_values(gdn, S, C, G):  # noqa: F811
    """The last samples of a tensor that 32-bit offsets do not reach, against a call for them alone."""
    announce(f"group norm of far samples {S} {C}")
    N = (1 << 31) // (S * C) + 5
    x = torch.empty(N, S, C, device="cuda", dtype=torch.bfloat16).normal_()
    w, b = torch.randn(C, device="cuda"), torch.randn(C, device="cuda")
    y, mean, rstd = gdn.group_norm_fwd(x, G, w, b, activation="silu")
    # the sums' order goes by the number of samples: fp32 sums, and bf16 steps where one falls the other way
    ys, ms, rs = gdn.group_norm_fwd(x[-3:], G, w, b, activation="silu")
    near("y", y[-3:], dbl(ys), 2.0 ** -8)
    near("mean", mean[-3:], dbl(ms), 1e-4 if S == 1 else 1e-3)  # (means near 0 of values near 1)
    near("rstd", rstd[-3:], dbl(rs), F32)
    del y
    dy = x.flip(0)
    dx, dw, db, _ = gdn.group_norm_bwd(dy, x, G, w, b, mean, rstd, activation="silu")
    dxs, _, _, _ = gdn.group_norm_bwd(dy[-3:], x[-3:], G, w, b, ms, rs, activation="silu")
    near("dx", dx[-3:], dbl(dxs), 2.0 ** -8)
    assert bool(torch.isfinite(dw).all()) and bool(torch.isfinite(db).all())
