"""Problems whose launches would have 2^32 threads or more are refused before
anything is launched."""
import ctypes

import pytest

import gated_deltanet_chunked_gdn_amd as gdn
from gated_deltanet_chunked_gdn_amd import mixer
from tests.test_attention_cpu import P, group


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
