"""Linear attention whose decay grows so fast that its powers pass fp32's largest
number over tokens that add nothing: places behind a sequence's end inside a
chunk, tokens of zeros, a state that is still 0.  What such tokens add is 0
however large the power, and every number of the formula is held by fp32.

Tolerances are test_gpu_attention's: a power e^80, the largest one here that
meets something, is off by its exponent's two roundings, 80 * 2 * 2^-25 = 4.8e-6
at the most."""
import pytest
import torch

from tests.gpu_util import announce
from tests.mixer_ref import dbl, grads, near
from tests.test_gpu_attention import F32, PAIRS, attn_inputs, form, gdn  # noqa: F401

pytestmark = pytest.mark.gpu


def near_parts(name, got, parts, dtype, R):
    """dq or dk against the v-heads' parts of it, R to a head.  A fast decay leaves one pair of tokens to a row, so
    that the parts are a few large vectors, which may cancel (to a tenth, here); the sum is off by no more than its
    parts, each within PAIRS of its own size."""
    parts = parts.unflatten(2, (-1, R))
    size = sum(float(parts[..., i, :].norm()) for i in range(R))
    assert torch.isfinite(got).all(), name
    off = float((dbl(got) - parts.sum(3)).norm())
    assert off <= PAIRS[dtype] * size, f"{name}: {off / size:.3g}"


def check_growing(gdn, dtype, args):  # noqa: F811
    """check_attention, but for dq and dk (near_parts)."""
    q, k, v, decay, h0, do, dht, cu, scale = args
    o, ht = gdn.linear_attention_fwd(q, k, v, decay, scale=scale, initial_state=h0, cu_seqlens=cu)
    f = form(decay, cu, scale, q.shape[-1])
    ro, rht = f(dbl(q), dbl(k), dbl(v), dbl(h0))
    near("o", o, ro, PAIRS[dtype])
    near("ht", ht, rht, F32)
    got = gdn.linear_attention_bwd(q, k, v, decay, do, dht=dht, scale=scale, initial_state=h0, cu_seqlens=cu)
    R = v.shape[2] // q.shape[2]
    want = grads(f, [q.repeat_interleave(R, 2), k.repeat_interleave(R, 2), v, h0], [do, dht])
    for n, a, r in zip(("dq", "dk"), got, want):
        near_parts(n, a, r, dtype, R)
    near("dv", got[2], want[2], PAIRS[dtype])
    near("dh0", got[3], want[3], F32)


@pytest.mark.parametrize("T,decay,scale", [(1, 9.0, None), (10, 1.5, None), (10, 3.0, 4.0), (40, 2.0, -2.0), (20, 3.0, None)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sequences_that_end_inside_a_chunk(gdn, dtype, T, decay, scale):  # noqa: F811
    """exp(63 decay) is beyond fp32, exp(T decay) is not."""
    announce(f"attention {dtype} growing {T} {decay}")
    check_growing(gdn, dtype, attn_inputs(dtype, (1, T, 1, 2, 32, 64, None, True, scale, decay, decay), seed=T))
    check_growing(gdn, dtype, attn_inputs(dtype, (1, 0, 2, 2, 64, 64, [T, 0, T // 2, 1], False, scale, decay, decay), seed=T))


@pytest.mark.parametrize("T", [94, 128, 2500])
@pytest.mark.parametrize("Hq,K,V", [(1, 64, 64), (2, 32, 128)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_tokens_of_zeros(gdn, dtype, Hq, K, V, T):  # noqa: F811
    """30 tokens at a sequence's end, zeros before them (and for the gradients that come from behind, the other
    way round): one segment, segments joined by the pass that reads them, and a carry between them."""
    announce(f"attention {dtype} zeros {T} {Hq} {K} {V}")
    q, k, v, decay, _, do, _, _, _ = attn_inputs(dtype, (1, T, Hq, 2, K, V, None, False, None, 1.5, 1.5), seed=T)
    f = form(decay, None, None, K)

    def masked(keep):
        return [torch.zeros_like(t).index_copy_(1, keep, t[:, keep]) for t in (q, k, v, do)]

    for keep, which in ((torch.arange(T - 30, T).cuda(), "end"), (torch.arange(30).cuda(), "start")):
        x = masked(keep)
        own = [t[:, keep] for t in x]  # the formula on the tokens that count
        leaves = [dbl(t.repeat_interleave(2 // t.shape[2], 2)).requires_grad_() for t in own[:3]]
        h0 = torch.zeros(1, 2, K, V, dtype=torch.float64, requires_grad=True)
        ro, rht = f(*leaves, h0)
        want = torch.autograd.grad((ro * dbl(own[3])).sum(), [*leaves, h0])
        o, ht = gdn.linear_attention_fwd(*x[:3], decay)
        dq, dk, dv, dh0 = gdn.linear_attention_bwd(*x[:3], decay, x[3], initial_state=torch.zeros(1, 2, K, V).cuda())
        if which == "end":
            near("o", o[:, keep], ro, PAIRS[dtype])
            near("ht", ht, rht, F32)
            near_parts("dq", dq[:, keep], want[0], dtype, 2 // Hq)
            assert not o[:, :T - 30].any() and not dq[:, :T - 30].any()
        else:
            near_parts("dk", dk[:, keep], want[1], dtype, 2 // Hq)
            near("dv", dv[:, keep], want[2], PAIRS[dtype])
            near("dh0", dh0, want[3], F32)
            assert not dk[:, 30:].any() and not dv[:, 30:].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_one_token_of_a_growing_head(gdn, dtype):  # noqa: F811
    """A decay beyond fp32 itself leaves a state of 0 at what the token adds, in a call and in a step."""
    announce(f"attention {dtype} one token growing")
    q, k, v, _, _, _, _, _, _ = attn_inputs(dtype, (1, 1, 1, 2, 32, 64, None, False, None, 0, 0), seed=2)
    decay = torch.tensor([100.0, float("inf")]).cuda()
    ro, rht = form(torch.zeros(2).cuda(), None, None, 32)(dbl(q), dbl(k), dbl(v), None)
    o, ht = gdn.linear_attention_fwd(q, k, v, decay)
    near("o", o, ro, PAIRS[dtype])
    near("ht", ht, rht, F32)
    st = torch.zeros(1, 2, 32, 64).cuda()
    near("o of a step", gdn.linear_attention_step(q[:, 0], k[:, 0], v[:, 0], decay, st), ro[:, 0], PAIRS[dtype])
    near("state of a step", st, rht, F32)
