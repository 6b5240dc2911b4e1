"""A row of the attention does not depend on the rows beside it, to the last bit."""
import pytest
import torch

from means_clustering_amd import kvcache

from .test_gpu_kvcache import BF, FP, Case
from .test_gpu_kvcache_forms import FormCase

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n,hq", [(1, 4), (4, 4), (90, 4), (40, 8)])
@pytest.mark.parametrize("eight,window", [(False, 0), (False, 50), (True, 0)])
def test_rows_beside_rows_of_huge_scores(eight, window, n, hq, D, dt):
    """Scores of 2^24 and more, whose terms are made another way, in one head and one token: all other rows keep their
    bits."""
    lens = [(150, n), (100, n)]
    c = FormCase(lens, hq, 2, D, dt, window=window, eight=True) if eight else Case(lens, hq, 2, D, dt, window=window)
    c.scale = 64.0
    c.q = (c.q.float() * 2e-3).to(dt)
    out, lse = kvcache.attend(**c.device(), lse=True)
    c.q[:, 1] = c.q[:, 1].sign() * 6e4
    c.q[n // 2] = c.q[n // 2].sign() * 6e4
    out2, lse2 = kvcache.attend(**c.device(), lse=True)
    assert float(lse2[:, 1].abs().min()) > 0 and float(lse2[:, 1].abs().max()) >= 2.0 ** 24
    keep = torch.ones(2 * n, hq, dtype=torch.bool, device=out.device)
    keep[:, 1] = keep[n // 2] = False
    assert torch.equal(out[keep].view(torch.int16), out2[keep].view(torch.int16))
    assert torch.equal(lse[keep].view(torch.int32), lse2[keep].view(torch.int32))
