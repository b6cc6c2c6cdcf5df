"""How linear attention cuts sequences, as its workspace shows it (one state for
each part of a segment and head)."""
import ctypes

import numpy as np
import pytest

from gated_deltanet_chunked_gdn_amd import mixer
from tests.test_attention_cpu import attn


def parts(T, lens, known, Hv, K, V, dtype, bwd=False):
    """States of a head that the workspace holds, but for the N that a packed batch has over."""
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    p = attn(T=T, Hq=Hv, Hv=Hv, K=K, V=V, N=len(lens), dtype=dtype, cu_seqlens=16, cu_seqlens_host=cu.ctypes.data if known else None)
    L = mixer.lib()
    n = (L.gdn_linear_attention_bwd_workspace_size if bwd else L.gdn_linear_attention_fwd_workspace_size)(ctypes.byref(p))
    n //= Hv * K * V * 4 * (2 if bwd else 1)
    return n - len(lens) if n else 0


@pytest.mark.parametrize("bwd", [False, True])
@pytest.mark.parametrize("dtype,K,V", [(1, 128, 128), (1, 64, 64), (0, 64, 64)])
@pytest.mark.parametrize("Hv", [1, 4, 16])
def test_known_lengths_are_taken_as_they_are(Hv, dtype, K, V, bwd):
    """One sequence of all tokens among empty ones is cut as one that leaves a token to another is: its length is
    known, and is not guessed from the mean."""
    T = 8192
    whole = parts(T, [0] * 15 + [T], True, Hv, K, V, dtype, bwd)
    almost = parts(T, [0] * 14 + [1, T - 1], True, Hv, K, V, dtype, bwd)
    assert whole == almost
    if Hv == 1:  # alone, it leaves nearly all of the chip idle: cut
        assert whole > 1
