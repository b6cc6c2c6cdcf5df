"""Problems whose launches would have 2^32 threads or more are refused before
anything is launched."""
import ctypes

import pytest

import gated_deltanet_chunked_gdn_amd as gdn
from gated_deltanet_chunked_gdn_amd import GdnProblem, mixer
from tests.test_attention_cpu import P, attn, group


@pytest.mark.parametrize("N,S,G,Dg,fits", [
    (1, 256, 9000001, 1, False),    # a workgroup of 512 a group and one for 32 sums: 1.14 * 2^32 threads
    (1, 512, 7895160, 1, False),    # 2^23 workgroups
    (1, 512, 7895159, 1, True),     # one fewer
    (5000, 1000, 2000, 16, False),  # groups of many samples
])
def test_group_norm_backward_of_too_many_groups(N, S, G, Dg, fits):
    L, r = mixer.lib(), ctypes.byref(group(N=N, S=S, G=G, Dg=Dg))
    assert (N * G + (2 * G * Dg + 31) // 32 < 1 << 23) == fits
    assert L.gdn_group_norm_fwd_workspace_size(r) > 0  # a workgroup of 256 a group
    assert (L.gdn_group_norm_bwd_workspace_size(r) > 0) == fits
    code = L.gdn_group_norm_bwd(r, *([P(16)] * 2), None, None, None, *([P(16)] * 3), None, None, None, P(256), 8, None)
    assert code == (4 if fits else 2) and gdn.last_error() != ""  # (a workspace of 8 bytes)


@pytest.mark.parametrize("B,Hv,V,fits", [(1 << 21, 32, 32, False), (1 << 19, 32, 128, False), (1 << 26, 1, 32, False),
                                         ((1 << 26) - 3, 1, 32, False), ((1 << 26) - 4, 1, 32, True), ((1 << 20) - 1, 32, 64, True)])
def test_steps_of_too_many_rows(B, Hv, V, fits):
    """A wave for 32 columns of a row's head, in workgroups of four."""
    L, x = mixer.lib(), P(16)
    assert ((B * Hv * V // 32 + 3) // 4 * 256 < 1 << 32) == fits
    a = attn(B=B, N=B, T=1, Hq=1, Hv=Hv, V=V)
    s = mixer.ScanProblem(B, 1, 1, Hv, 32, V, B, 1, 0, 0, 0, 0, None, None)
    d = GdnProblem(B, 1, 1, Hv, 32, V, B, 1, 1.0, None, None, 0, 0)
    # (where the sizes are taken, the state's missing slots are what is refused)
    for code in (L.gdn_linear_attention_step(ctypes.byref(a), x, x, x, x, x, None, 0, x, None),
                 L.gdn_selective_scan_step(ctypes.byref(s), *[x] * 7, x, None, 0, x, None),
                 L.gdn_delta_rule_step(ctypes.byref(d), *[x] * 5, 0, 0, 0, x, None, 0, x, None)):
        assert code == (1 if fits else 2), gdn.last_error()
