"""The sequence-mixer operators refuse malformed arguments before any launch:
the binding's checks on CPU tensors (a check that let one through would stop
at the device check, whose message says so), and the C ABI's codes."""
import ctypes

import numpy as np
import pytest
import torch

import gated_deltanet_chunked_gdn_amd as gdn
from gated_deltanet_chunked_gdn_amd import mixer

BF = torch.bfloat16
P = ctypes.c_void_p


def z(*shape, dt=BF):
    return torch.zeros(*shape, dtype=dt)


def conv_args(**kw):
    a = dict(x=z(1, 10, 16), weight=z(16, 4), bias=z(16))
    a.update(kw)
    return a


def scan_args(**kw):
    a = dict(c=z(1, 10, 2, 32), b=z(1, 10, 2, 32), x=z(1, 10, 4, 64), dt=z(1, 10, 4), A=z(4, dt=torch.float32))
    a.update(kw)
    return a


def step_args(**kw):
    a = dict(q=z(3, 2, 32), k=z(3, 2, 32), v=z(3, 4, 64), g=z(3, 4, dt=torch.float32), beta=z(3, 4),
             state=z(3, 4, 32, 64, dt=torch.float32))
    a.update(kw)
    return a


@pytest.mark.parametrize("call", [
    lambda: gdn.causal_conv_fwd(**conv_args()),
    lambda: gdn.causal_conv_bwd(dy=z(1, 10, 16), **conv_args()),
    lambda: gdn.causal_conv_step(z(3, 16), z(3, 3, 16), z(16, 4)),
    lambda: gdn.selective_scan_fwd(**scan_args()),
    lambda: gdn.selective_scan_bwd(dy=z(1, 10, 4, 64), **scan_args()),
    lambda: gdn.selective_scan_step(z(3, 2, 32), z(3, 2, 32), z(3, 4, 64), z(3, 4), z(4, dt=torch.float32),
                                    z(3, 4, 32, 64, dt=torch.float32)),
    lambda: gdn.gated_delta_rule_step(**step_args()),
    lambda: gdn.layer_norm_fwd(z(3, 16)),
    lambda: gdn.layer_norm_bwd(z(3, 16), z(3, 16), None, None, z(3, dt=torch.float32), z(3, dt=torch.float32)),
])
def test_valid_arguments_reach_the_device_check(call):
    with pytest.raises(ValueError, match="on the GPU"):
        call()


@pytest.mark.parametrize("kw", [
    dict(x=z(10, 16)), dict(weight=z(8, 4)), dict(bias=z(4)), dict(weight=z(16, 4, dt=torch.float32)),
    dict(weight=z(16, 4, dt=torch.float16), bias=None), dict(x=z(1, 10, 16, dt=torch.float16)), dict(activation="relu"),
    dict(initial_state=z(1, 4, 16)), dict(initial_state=z(1, 3, 16, dt=torch.float32)),
    dict(cu_seqlens=torch.tensor([0, 5, 9])), dict(cu_seqlens=torch.tensor([0, 7, 5, 10])),
    dict(cu_seqlens=torch.tensor([1, 10])), dict(cu_seqlens=torch.tensor([0.0, 10.0])), dict(cu_seqlens=torch.tensor([10])),
    dict(cu_seqlens=torch.tensor([0, 4, 10]), initial_state=z(1, 3, 16)),
    dict(x=z(2, 10, 16), cu_seqlens=torch.tensor([0, 10])),
    dict(cu_seqlens=torch.tensor([0, 5, 9]), check_cu_seqlens=False),  # a host tensor is checked in any case
])
def test_conv_refusals(kw):
    with pytest.raises((ValueError, TypeError)) as e:
        gdn.causal_conv_fwd(**conv_args(**kw))
    assert "on the GPU" not in str(e.value)
    if "activation" in kw or "cu_seqlens" in kw or "initial_state" in kw:
        with pytest.raises((ValueError, TypeError)) as e:
            gdn.causal_conv_bwd(dy=z(*kw.get("x", z(1, 10, 16)).shape), **conv_args(**kw))
        assert "on the GPU" not in str(e.value)


@pytest.mark.parametrize("kw", [
    dict(c=z(1, 10, 2, 16)), dict(b=z(1, 9, 2, 32)), dict(x=z(1, 9, 4, 64)), dict(dt=z(1, 10, 2)),
    dict(dt=z(1, 10, 4, dt=torch.float32)), dict(A=z(4)), dict(A=z(2, dt=torch.float32)), dict(A=None),
    dict(D=z(4)), dict(dt_bias=z(3, dt=torch.float32)), dict(initial_state=z(1, 4, 64, 32, dt=torch.float32)),
    dict(initial_state=z(1, 4, 32, 64)), dict(cu_seqlens=torch.tensor([0, 11])),
])
def test_scan_refusals(kw):
    for f, more in ((gdn.selective_scan_fwd, {}), (gdn.selective_scan_bwd, dict(dy=z(1, 10, 4, 64)))):
        with pytest.raises((ValueError, TypeError)) as e:
            f(**scan_args(**kw), **more)
        assert "on the GPU" not in str(e.value)


@pytest.mark.parametrize("dy", [None, z(1, 10, 4, 32), z(1, 10, 4, 64, dt=torch.float32)])
def test_scan_bwd_refuses_bad_dy(dy):
    with pytest.raises(ValueError, match="dy must"):
        gdn.selective_scan_bwd(dy=dy, **scan_args())


@pytest.mark.parametrize("kw", [
    dict(q=z(3, 2, 16)), dict(v=z(2, 4, 64)), dict(g=z(3, 4)), dict(beta=z(3, 2)), dict(beta=z(3, 4, dt=torch.float32)),
    dict(state=z(3, 4, 32, 64)), dict(state=z(2, 4, 32, 64, dt=torch.float32)),
    dict(state=z(3, 4, 64, 32, dt=torch.float32).transpose(2, 3)), dict(state_indices=torch.zeros(3, dtype=torch.int64)),
    dict(state_indices=torch.zeros(2, dtype=torch.int32)),
])
def test_delta_step_refusals(kw):
    with pytest.raises((ValueError, TypeError)) as e:
        gdn.gated_delta_rule_step(**step_args(**kw))
    assert "on the GPU" not in str(e.value)


@pytest.mark.parametrize("args,kw", [
    ((z(3, 0),), {}), ((z(3, 16), z(8)), {}), ((z(3, 16), z(16), z(16, dt=torch.float32)), {}),
    ((z(3, 16),), dict(gate=z(3, 8))), ((z(3, 16),), dict(gate=z(3, 16, dt=torch.float32))),
    ((z(3, 16, dt=torch.float64),), {}),
])
def test_norm_refusals(args, kw):
    with pytest.raises((ValueError, TypeError)) as e:
        gdn.layer_norm_fwd(*args, **kw)
    assert "on the GPU" not in str(e.value)


def test_norm_bwd_refusals():
    x, m = z(3, 16), z(3, dt=torch.float32)
    for dy, mean, rstd in ((z(3, 8), m, m), (x, None, m), (x, m, None), (x, z(2, dt=torch.float32), m), (x, m, z(3))):
        with pytest.raises(ValueError) as e:
            gdn.layer_norm_bwd(dy, x, None, None, mean, rstd)
        assert "on the GPU" not in str(e.value)


# ---------------------------------------------------------------- C ABI


def conv(**kw):
    d = dict(B=1, T=10, D=16, W=4, N=1, dtype=1, weight_dtype=1, silu=1, x_stride=0, cu_seqlens=None, cu_seqlens_host=None)
    d.update(kw)
    return mixer.ConvProblem(**d)


def scan(**kw):
    d = dict(B=1, T=10, Hq=2, Hv=4, K=32, V=64, N=1, dtype=1, dt_softplus=1, c_stride=0, b_stride=0, x_stride=0,
             cu_seqlens=None, cu_seqlens_host=None)
    d.update(kw)
    return mixer.ScanProblem(**d)


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), 1), (dict(T=-1), 1), (dict(D=0), 1), (dict(W=5), 2), (dict(W=1), 2), (dict(dtype=3), 2),
    (dict(dtype=0, weight_dtype=1), 2), (dict(silu=2), 1), (dict(x_stride=8), 1), (dict(N=2), 1),
    (dict(cu_seqlens_host=16), 1), (dict(B=2, cu_seqlens=16), 1), (dict(N=0, cu_seqlens=16), 1),
    (dict(T=2 ** 31 - 1, B=2, N=2), 2),
])
def test_conv_problem_codes(kw, code):
    L, p = mixer.lib(), conv(**kw)
    assert L.gdn_causal_conv_bwd_workspace_size(ctypes.byref(p)) == 0
    assert L.gdn_causal_conv_fwd(ctypes.byref(p), P(16), P(16), P(16), None, P(16), None, None) == code
    assert gdn.last_error() != ""


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), 1), (dict(Hq=3), 2), (dict(K=16), 2), (dict(V=256), 2), (dict(dtype=0, K=128), 2), (dict(dtype=9), 2),
    (dict(dt_softplus=2), 1), (dict(c_stride=32), 1), (dict(x_stride=257), 3), (dict(N=3), 1),
    (dict(T=2 ** 31 - 1, Hv=512), 2),
])
def test_scan_problem_codes(kw, code):
    L, p = mixer.lib(), scan(**kw)
    assert L.gdn_selective_scan_fwd_workspace_size(ctypes.byref(p)) == 0
    assert L.gdn_selective_scan_bwd_workspace_size(ctypes.byref(p)) == 0
    rc = L.gdn_selective_scan_fwd(ctypes.byref(p), *([P(16)] * 5), None, None, None, P(16), None, P(256), 1 << 40, None)
    assert rc == code and gdn.last_error() != ""


def test_host_cu_seqlens_are_checked():
    L = mixer.lib()
    for bad in ([1, 10], [0, 7, 5, 10], [0, 5, 9]):
        a = np.array(bad, dtype=np.int32)
        p = conv(N=len(bad) - 1, cu_seqlens=16, cu_seqlens_host=a.ctypes.data)
        assert L.gdn_causal_conv_fwd(ctypes.byref(p), P(16), P(16), P(16), None, P(16), None, None) == 1
        p = scan(N=len(bad) - 1, cu_seqlens=16, cu_seqlens_host=a.ctypes.data)
        assert L.gdn_selective_scan_bwd_workspace_size(ctypes.byref(p)) == 0


def test_pointers_alignment_and_workspaces():
    L, p, s = mixer.lib(), conv(), scan()
    c, r = ctypes.byref(p), ctypes.byref(s)
    assert L.gdn_causal_conv_fwd(c, None, P(16), P(16), None, P(16), None, None) == 1
    assert L.gdn_causal_conv_fwd(c, P(17), P(16), P(16), None, P(16), None, None) == 3
    assert L.gdn_causal_conv_bwd(c, *([P(16)] * 4), None, None, P(16), P(16), None, None, P(256), 8, None) == 4
    assert L.gdn_causal_conv_bwd(c, P(16), P(16), None, P(16), None, None, P(16), P(16), P(16), None, P(256), 1 << 30, None) == 1
    assert L.gdn_causal_conv_step(c, P(16), P(16), P(16), None, None, 4, P(16), None) == 1  # T = 10
    one = ctypes.byref(conv(T=1))
    assert L.gdn_causal_conv_step(one, P(16), P(16), P(16), None, None, 0, P(16), None) == 1  # no slots
    assert L.gdn_selective_scan_fwd(r, *([P(16)] * 5), None, None, None, P(24), None, P(256), 1 << 40, None) == 3
    assert L.gdn_selective_scan_fwd(r, *([P(16)] * 4), None, None, None, None, P(16), None, P(256), 1 << 40, None) == 1
    assert L.gdn_selective_scan_fwd(r, *([P(16)] * 5), None, None, None, P(16), None, P(128), 1 << 40, None) == 4
    assert L.gdn_selective_scan_bwd(r, *([P(16)] * 18), P(256), 16, None) == 4
    n = ctypes.byref(mixer.NormProblem(rows=4, D=16, dtype=1, weight_dtype=1, rms=0, eps=1e-5))
    assert L.gdn_layer_norm_fwd(n, None, None, None, None, P(16), None, None, None) == 1
    assert L.gdn_layer_norm_fwd(n, P(17), None, None, None, P(16), None, None, None) == 3
    assert L.gdn_layer_norm_bwd(n, P(16), P(16), None, None, None, None, P(16), P(16), None, None, None, P(256), 1 << 30, None) == 1
    assert L.gdn_layer_norm_bwd(n, P(16), P(16), None, None, None, P(16), P(16), P(16), P(16), None, None, P(256), 1 << 30, None) == 1
    for bad in (dict(rows=-1), dict(D=0), dict(rms=3), dict(eps=-1.0), dict(dtype=5), dict(weight_dtype=7)):
        d = dict(rows=4, D=16, dtype=1, weight_dtype=1, rms=0, eps=1e-5)
        d.update(bad)
        q = mixer.NormProblem(**d)
        assert L.gdn_layer_norm_bwd_workspace_size(ctypes.byref(q)) == 0
    d = gdn.GdnProblem(3, 1, 2, 4, 32, 64, 3, gdn.GDN_BF16, float("nan"), None, None, -1, 0)
    assert L.gdn_delta_rule_step(ctypes.byref(d), *([P(16)] * 5), 0, 0, 0, P(16), None, 3, P(16), None) == 1


def test_strided_rows_are_taken_as_they_are():
    wide = z(2, 5, 64)
    t, s = mixer._rows(wide[..., 8:24], 2)
    assert s == 64 and t.data_ptr() == wide.data_ptr() + 16
    t, s = mixer._rows(wide[..., 3:24], 2)  # not in 16-byte pieces
    assert s == 21 and t.is_contiguous()
    t, s = mixer._rows(wide[:, :3, :16], 2)  # rows of two batches at two distances
    assert s == 16 and t.is_contiguous()
    t, s = mixer._rows(z(1, 1, 16).expand(2, 5, 16), 2)
    assert s == 16 and t.is_contiguous()
    t, s = mixer._rows(z(2, 5, 4, 64)[..., :32], 2)
    assert s == 128 and t.is_contiguous()


def test_sizes_beyond_32_bits_are_refused():
    """They would be cut in the descriptors (2^32 + 1 tokens to one)."""
    n = (1 << 32) + 1
    wide = lambda *shape, dt=BF: torch.empty(1, dtype=dt).expand(*shape)  # noqa: E731
    for call in (
            lambda: gdn.causal_conv_fwd(wide(1, n, 1), z(1, 2)),
            lambda: gdn.causal_conv_step(wide(n, 1), z(3, 1, 1), z(1, 2)),
            lambda: gdn.selective_scan_fwd(wide(1, n, 1, 32), wide(1, n, 1, 32), wide(1, n, 1, 32), wide(1, n, 1),
                                           z(1, dt=torch.float32)),
            lambda: gdn.layer_norm_fwd(wide(1, n))):
        with pytest.raises(ValueError, match="32 bits"):
            call()


def test_channels_whose_workgroups_end_past_32_bits_are_refused():
    """A channel's index is 32-bit: the last workgroup's, up to 1023 past D, has to fit as well (it would come out
    negative, in front of every buffer)."""
    L = mixer.lib()
    for D in (2 ** 31 - 1, 2 ** 31 - 1023):
        p = ctypes.byref(conv(D=D, T=1))
        assert L.gdn_causal_conv_bwd_workspace_size(p) == 0
        assert L.gdn_causal_conv_fwd(p, P(16), P(16), P(16), None, P(16), None, None) == 2
        assert L.gdn_causal_conv_bwd(p, *([P(16)] * 4), None, None, *([P(16)] * 3), None, P(256), 1 << 62, None) == 2
        assert L.gdn_causal_conv_step(p, P(16), P(16), P(16), None, None, 1, P(16), None) == 2
    assert L.gdn_causal_conv_bwd_workspace_size(ctypes.byref(conv(D=(2 ** 31 - 1) // 8, T=1))) == 0  # its sums' launch
    assert L.gdn_causal_conv_bwd_workspace_size(ctypes.byref(conv(D=50_000_000, T=1))) > 0


def test_a_step_takes_rows_at_any_distance():
    """x[:, t] of a long [B, T, ...]: the limit of 2^24 elements is the scan's, whose rows are 32-bit byte offsets
    apart.  (Both calls stop at a missing pointer, past the sizes' checks.)"""
    L = mixer.lib()
    far = 1 << 24
    s = scan(B=3, T=1, N=3, c_stride=far, b_stride=far, x_stride=far)
    assert L.gdn_selective_scan_step(ctypes.byref(s), None, *([P(16)] * 4), None, None, P(16), None, 3, P(16), None) == 1
    d = gdn.GdnProblem(3, 1, 2, 4, 32, 64, 3, gdn.GDN_BF16, 1.0, None, None, -1, 0)
    assert L.gdn_delta_rule_step(ctypes.byref(d), None, *([P(16)] * 4), far, far, far, P(16), None, 3, P(16), None) == 1
    assert L.gdn_selective_scan_fwd_workspace_size(ctypes.byref(s)) == 0


def test_rows_that_the_kernels_do_not_take_are_copied():
    """A contiguous tensor off a 16-byte boundary like a strided one there, and tokens too far apart for the scan."""
    off = torch.arange(2 * 5 * 16 + 1, dtype=torch.float32)[1:].view(2, 5, 16)
    assert off.is_contiguous() and off.data_ptr() % 16
    t, s = mixer._rows(off, 2, aligned=True)
    assert s == 16 and t.data_ptr() % 16 == 0 and torch.equal(t, off)
    t, s = mixer._rows(off, 2)  # the convolution takes any
    assert s == 16 and t.data_ptr() == off.data_ptr()
    far = torch.empty((1 << 24) + 32, dtype=BF)[:1].as_strided((1, 2, 1, 32), (1 << 25, 1 << 24, 32, 1))
    far[:] = 1
    t, s = mixer._rows(far, 2, most=(1 << 24) - 1)
    assert s == 32 and t.is_contiguous()
    t, s = mixer._rows(far, 2)
    assert s == 1 << 24 and t.data_ptr() == far.data_ptr()
    assert mixer._aligned(None) is None and mixer._aligned(off).data_ptr() % 16 == 0
    even = z(3, 16)
    assert mixer._aligned(even) is even
