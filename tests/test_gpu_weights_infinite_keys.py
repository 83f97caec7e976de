"""Gathered weights over keys that hold infinities: a score of -inf is a weight of 0,
whatever the row tiles' unused rows would make of such a key."""
import math

import pytest
import torch

from tests.serve_ref import Paged
from tests.test_gpu_weights import run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("hq,hkv,d,ps", [(3, 1, 64, 16), (6, 2, 128, 32), (5, 1, 160, 16), (48, 1, 96, 64),
                                         (100, 1, 128, 16), (66, 1, 64, 32), (8, 2, 128, 16)])
@pytest.mark.parametrize("causal", [True, False])
def test_scores_of_minus_infinity(hq, hkv, d, ps, causal):
    """Row tiles of 128 rows that head groups fill in part and in full."""
    p = Paged([150, 3], [700, 300], hq, hkv, d, ps, seed=11)
    p.q[:, :, 0] = -p.q[:, :, 0].abs() - 1.0
    for i, pos in ((0, 10), (0, 300), (1, 7)):
        page, row = p.places(i, torch.tensor([pos], device=p.q.device))
        p.keys[i][pos, :, 0] = math.inf
        p.k_pages[page, :, row] = p.keys[i][pos]
    batch, lse, old, out = run(p, decay=0.5, causal=causal)
    assert torch.isfinite(lse).all()
    for i, pos in ((0, 10), (0, 300), (1, 7)):
        assert torch.equal(out[i, :, pos], old[i, :, pos] * 0.5)
    assert int(p.status.item()) == 0
