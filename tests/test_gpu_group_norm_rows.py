"""Group norm over many positions, in fp32, where rows of a channel lie far from
the others: rstd is right to what test_gpu_attention asks of every one (F32).

Each thread joins the means and squares of its rows, eight at a time, in fp32:
sums of positive terms, one for eight rows.  A term is off by 9 * 2^-24 of itself
at the most (its sums are about one of the eight), and the sum of 125 of them,
1000 rows, by a random walk near sqrt(125) 2^-24: together 1.2e-6 of the variance."""
import pytest
import torch

from tests.gpu_util import announce
from tests.test_gpu_attention import F32, gdn  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("where", ["first", "middle", "last"])
@pytest.mark.parametrize("off", [0.0, 20.0, 2000.0])
@pytest.mark.parametrize("N,S,C,G", [(1600, 1000, 256, 4), (1600, 61, 1024, 2), (3, 5000, 12, 2), (40, 3001, 100, 4)])
def test_a_row_far_from_the_others(gdn, N, S, C, G, off, where):  # noqa: F811
    """One position of every channel `off` deviations away: as many samples as fill the chip (a block has all rows
    of a sample) and few; and a mean of a thousand deviations besides."""
    announce(f"group_norm row {N} {S} {C} {G} off={off} {where}")
    g = torch.Generator("cuda").manual_seed(S)
    for shift in (0.0, 1000.0):
        x = torch.randn(N, S, C, generator=g, device="cuda") + shift
        x[:, {"first": 0, "middle": S // 2, "last": S - 1}[where]] -= off
        _, mean, rstd = gdn.group_norm_fwd(x, G)
        for a in range(0, N, 400):
            z = x[a:a + 400].double().view(-1, S, G, C // G)
            rmean = z.mean((1, 3))
            var = ((z - rmean[:, None, :, None]) ** 2).mean((1, 3))
            off_rstd = (rstd[a:a + 400].double() * (var + 1e-5).sqrt() - 1).abs().max()
            off_mean = ((mean[a:a + 400].double() - rmean).abs() / (rmean.abs() + var.sqrt())).max()
            assert float(off_rstd) <= F32 and float(off_mean) <= F32, (float(off_rstd), float(off_mean))
