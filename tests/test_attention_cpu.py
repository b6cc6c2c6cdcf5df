"""Linear attention with a decay for each head and the group norm refuse
malformed arguments before any launch: the binding's checks on CPU tensors, and
the C ABI's codes."""
import ctypes

import numpy as np
import pytest
import torch

import gated_deltanet_chunked_gdn_amd as gdn
from gated_deltanet_chunked_gdn_amd import mixer

BF, F = torch.bfloat16, torch.float32
P = ctypes.c_void_p


def z(*shape, dt=BF):
    return torch.zeros(*shape, dtype=dt)


def attn_args(**kw):
    a = dict(q=z(1, 10, 2, 32), k=z(1, 10, 2, 32), v=z(1, 10, 4, 64), log_decay=z(4, dt=F))
    a.update(kw)
    return a


def step_args(**kw):
    a = dict(q=z(3, 2, 32), k=z(3, 2, 32), v=z(3, 4, 64), log_decay=z(4, dt=F), state=z(3, 4, 32, 64, dt=F))
    a.update(kw)
    return a


def norm_args(**kw):
    a = dict(x=z(2, 5, 16), groups=4, weight=z(16), bias=z(16))
    a.update(kw)
    return a


@pytest.mark.parametrize("call", [
    lambda: gdn.linear_attention_fwd(**attn_args()),
    lambda: gdn.linear_attention_bwd(do=z(1, 10, 4, 64), **attn_args()),
    lambda: gdn.linear_attention_step(**step_args()),
    lambda: gdn.group_norm_fwd(**norm_args()),
    lambda: gdn.group_norm_fwd(z(3, 16), 16, activation="silu"),
    lambda: gdn.group_norm_fwd(z(3, 16), 1, gate=z(3, 16)),
    lambda: gdn.group_norm_bwd(z(3, 16), z(3, 16), 2, None, None, z(3, 2, dt=F), z(3, 2, dt=F)),
])
def test_valid_arguments_reach_the_device_check(call):
    with pytest.raises(ValueError, match="on the GPU"):
        call()


@pytest.mark.parametrize("kw", [
    dict(q=z(1, 10, 2, 16)), dict(k=z(1, 9, 2, 32)), dict(v=z(1, 9, 4, 64)), dict(v=z(1, 10, 4, 64, dt=F)), dict(q=z(10, 2, 32)),
    dict(log_decay=z(4)), dict(log_decay=z(2, dt=F)), dict(log_decay=None), dict(log_decay=z(1, 10, 4, dt=F)),
    dict(initial_state=z(1, 4, 64, 32, dt=F)), dict(initial_state=z(1, 4, 32, 64)), dict(cu_seqlens=torch.tensor([0, 11])),
    dict(cu_seqlens=torch.tensor([0, 7, 5, 10])), dict(cu_seqlens=torch.tensor([0.0, 10.0])),
    dict(cu_seqlens=torch.tensor([0, 4, 10]), initial_state=z(1, 4, 32, 64, dt=F)),
    dict(q=z(1, 10, 2, 32, dt=torch.float16), k=z(1, 10, 2, 32, dt=torch.float16), v=z(1, 10, 4, 64, dt=torch.float16)),
    dict(q=z(1, 10, 2, 0), k=z(1, 10, 2, 0)),
])
def test_attention_refusals(kw):
    for f, more in ((gdn.linear_attention_fwd, {}), (gdn.linear_attention_bwd, dict(do=z(1, 10, 4, 64)))):
        with pytest.raises((ValueError, TypeError)) as e:
            f(**attn_args(**kw), **more)
        assert "on the GPU" not in str(e.value)


@pytest.mark.parametrize("do", [None, z(1, 10, 4, 32), z(1, 10, 4, 64, dt=F)])
def test_attention_bwd_refuses_bad_do(do):
    with pytest.raises(ValueError, match="do must"):
        gdn.linear_attention_bwd(do=do, **attn_args())


@pytest.mark.parametrize("kw", [
    dict(q=z(3, 2, 16)), dict(v=z(2, 4, 64)), dict(log_decay=z(3, 4, dt=F)), dict(state=z(3, 4, 32, 64)),
    dict(state=z(2, 4, 32, 64, dt=F)), dict(state=z(3, 4, 64, 32, dt=F).transpose(2, 3)),
    dict(state_indices=torch.zeros(3, dtype=torch.int64)), dict(state_indices=torch.zeros(2, dtype=torch.int32)),
])
def test_step_refusals(kw):
    with pytest.raises((ValueError, TypeError)) as e:
        gdn.linear_attention_step(**step_args(**kw))
    assert "on the GPU" not in str(e.value)


@pytest.mark.parametrize("kw", [
    dict(x=z(16)), dict(x=z(2, 0, 16)), dict(x=z(2, 0)), dict(groups=0), dict(groups=3), dict(groups=-4), dict(groups=True),
    dict(groups=4.0), dict(weight=z(4)), dict(bias=z(4)), dict(bias=z(16, dt=F)), dict(gate=z(2, 5, 8)),
    dict(gate=z(2, 5, 16, dt=F)), dict(activation="relu"), dict(gate=z(2, 5, 16), activation="silu"),
    dict(x=z(2, 5, 16, dt=torch.float64)),
])
def test_group_norm_refusals(kw):
    with pytest.raises((ValueError, TypeError)) as e:
        gdn.group_norm_fwd(**norm_args(**kw))
    assert "on the GPU" not in str(e.value)
    a = norm_args(**kw)
    m = z(2, 4, dt=F)
    with pytest.raises((ValueError, TypeError)) as e:
        gdn.group_norm_bwd(z(*a["x"].shape, dt=a["x"].dtype), mean=m, rstd=m, **a)
    assert "on the GPU" not in str(e.value)


def test_group_norm_bwd_refusals():
    x, m = z(2, 5, 16), z(2, 4, dt=F)
    for dy, mean, rstd in ((z(2, 5, 8), m, m), (None, m, m), (x, None, m), (x, m, None), (x, z(2, dt=F), m), (x, m, z(2, 4))):
        with pytest.raises(ValueError) as e:
            gdn.group_norm_bwd(dy, x, 4, None, None, mean, rstd)
        assert "on the GPU" not in str(e.value)


# ---------------------------------------------------------------- C ABI


def attn(**kw):
    d = dict(B=1, T=10, Hq=2, Hv=4, K=32, V=64, N=1, dtype=1, scale=1.0, q_stride=0, k_stride=0, v_stride=0, cu_seqlens=None,
             cu_seqlens_host=None)
    d.update(kw)
    return mixer.AttnProblem(**d)


def group(**kw):
    d = dict(N=2, S=5, G=4, Dg=4, dtype=1, weight_dtype=1, silu=0, eps=1e-5)
    d.update(kw)
    return mixer.GroupProblem(**d)


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), 1), (dict(T=-1), 1), (dict(Hq=3), 2), (dict(K=16), 2), (dict(V=256), 2), (dict(V=96), 2), (dict(dtype=9), 2),
    (dict(scale=float("nan")), 1), (dict(q_stride=32), 1), (dict(v_stride=257), 3), (dict(k_stride=1 << 24), 2), (dict(N=3), 1),
    (dict(T=2 ** 31 - 1, Hv=512), 2), (dict(cu_seqlens_host=16), 1), (dict(B=2, cu_seqlens=16), 1), (dict(N=0, cu_seqlens=16), 1),
    (dict(N=2 ** 30, cu_seqlens=16), 2), (dict(Hv=2 ** 30, Hq=2 ** 30), 2),
])
def test_attention_problem_codes(kw, code):
    L, p = mixer.lib(), attn(**kw)
    r = ctypes.byref(p)
    assert L.gdn_linear_attention_fwd_workspace_size(r) == 0
    assert L.gdn_linear_attention_bwd_workspace_size(r) == 0
    assert L.gdn_linear_attention_fwd(r, *([P(16)] * 4), None, P(16), None, P(256), 1 << 60, None) == code
    assert L.gdn_linear_attention_bwd(r, *([P(16)] * 4), None, P(16), None, *([P(16)] * 3), None, P(256), 1 << 60, None) == code
    assert gdn.last_error() != ""


def test_attention_host_cu_seqlens_are_checked():
    L = mixer.lib()
    for bad in ([1, 10], [0, 7, 5, 10], [0, 5, 9]):
        a = np.array(bad, dtype=np.int32)
        p = attn(N=len(bad) - 1, cu_seqlens=16, cu_seqlens_host=a.ctypes.data)
        assert L.gdn_linear_attention_fwd_workspace_size(ctypes.byref(p)) == 0


def test_attention_pointers_alignment_and_workspaces():
    L, r = mixer.lib(), ctypes.byref(attn())
    assert L.gdn_linear_attention_fwd_workspace_size(r) > 0
    f = L.gdn_linear_attention_fwd
    assert f(r, None, P(16), P(16), P(16), None, P(16), None, P(256), 1 << 40, None) == 1
    assert f(r, P(16), P(16), P(16), None, None, P(16), None, P(256), 1 << 40, None) == 1
    assert f(r, P(16), P(16), P(24), P(16), None, P(16), None, P(256), 1 << 40, None) == 3
    assert f(r, P(16), P(16), P(16), P(18), None, P(16), None, P(256), 1 << 40, None) == 3
    assert f(r, P(16), P(16), P(16), P(16), None, P(16), P(8), P(256), 1 << 40, None) == 3
    assert f(r, P(16), P(16), P(16), P(16), None, P(16), None, P(128), 1 << 40, None) == 4
    assert f(r, P(16), P(16), P(16), P(16), None, P(16), None, None, 1 << 40, None) == 4
    b = L.gdn_linear_attention_bwd
    assert b(r, *([P(16)] * 4), None, P(16), None, *([P(16)] * 3), None, P(256), 16, None) == 4
    assert b(r, *([P(16)] * 4), None, None, None, *([P(16)] * 3), None, P(256), 1 << 40, None) == 1
    s = L.gdn_linear_attention_step
    assert s(r, *([P(16)] * 5), None, 4, P(16), None) == 1  # T = 10
    one = ctypes.byref(attn(T=1))
    assert s(one, *([P(16)] * 5), None, 0, P(16), None) == 1  # no slots
    assert s(one, *([P(16)] * 5), P(18), 4, P(16), None) == 3
    assert s(one, *([P(16)] * 4), None, None, 4, P(16), None) == 1
    far = 1 << 24  # a step takes rows at any distance
    d = ctypes.byref(attn(B=3, N=3, T=1, q_stride=far, k_stride=far, v_stride=far))
    assert s(d, None, *([P(16)] * 4), None, 3, P(16), None) == 1
    assert L.gdn_linear_attention_fwd_workspace_size(d) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(N=-1), 1), (dict(S=0), 1), (dict(G=0), 1), (dict(Dg=-2), 1), (dict(dtype=4), 2), (dict(dtype=0, weight_dtype=1), 2),
    (dict(silu=2), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(G=1 << 20, Dg=16), 2), (dict(S=1 << 31), 2),
    (dict(N=1 << 31), 2), (dict(N=1 << 20, S=1 << 14, Dg=1 << 10), 2), (dict(N=1 << 25, S=1, G=1, Dg=10000), 2),
])
def test_group_norm_problem_codes(kw, code):
    L, p = mixer.lib(), group(**kw)
    r = ctypes.byref(p)
    assert L.gdn_group_norm_fwd_workspace_size(r) == 0
    assert L.gdn_group_norm_bwd_workspace_size(r) == 0
    assert L.gdn_group_norm_fwd(r, P(16), None, None, None, P(16), P(16), P(16), P(256), 1 << 60, None) == code
    assert gdn.last_error() != ""


def test_group_norm_pointers_alignment_and_workspaces():
    L, r = mixer.lib(), ctypes.byref(group())
    f, b = L.gdn_group_norm_fwd, L.gdn_group_norm_bwd
    assert f(r, None, None, None, None, P(16), P(16), P(16), P(256), 1 << 40, None) == 1
    assert f(r, P(16), None, None, None, P(16), None, P(16), P(256), 1 << 40, None) == 1
    assert f(r, P(17), None, None, None, P(16), P(16), P(16), P(256), 1 << 40, None) == 3
    assert f(r, P(16), None, None, None, P(16), P(16), P(16), P(256), 8, None) == 4
    s = ctypes.byref(group(silu=1))
    assert f(s, P(16), None, None, P(16), P(16), P(16), P(16), P(256), 1 << 40, None) == 1  # both
    assert b(s, P(16), P(16), None, None, P(16), P(16), P(16), P(16), None, None, P(16), P(256), 1 << 40, None) == 1
    assert b(r, P(16), P(16), None, None, P(16), P(16), P(16), P(16), None, None, None, P(256), 1 << 40, None) == 1
    assert b(r, P(16), P(16), None, None, None, P(16), P(16), P(16), P(16), None, None, P(256), 1 << 40, None) == 1
    assert b(r, P(16), P(16), P(16), None, None, P(16), P(16), P(16), P(16), None, None, P(256), 8, None) == 4


def test_sizes_beyond_32_bits_are_refused():
    n = (1 << 32) + 1
    wide = lambda *shape, dt=BF: torch.empty(1, dtype=dt).expand(*shape)  # noqa: E731
    for call in (lambda: gdn.linear_attention_fwd(wide(1, n, 1, 32), wide(1, n, 1, 32), wide(1, n, 1, 32), z(1, dt=F)),
                 lambda: gdn.linear_attention_step(wide(n, 1, 32), wide(n, 1, 32), wide(n, 1, 32), z(1, dt=F), z(1, 1, 32, 32, dt=F)),
                 lambda: gdn.group_norm_fwd(wide(1, n), 1)):
        with pytest.raises(ValueError, match="32 bits"):
            call()
