"""Dropout, residual add and layer norm called by several host threads at once with rows
of different lengths that one kernel serves."""
import pytest
import torch

import attention_core_gb300 as ac
from tests.test_gpu_host_threads import at_once

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


class Boundary:
    """Rows at a residual boundary: forward, then backward from its results."""

    def __init__(self, hidden, seed, n=4):
        gen = torch.Generator(device=DEV).manual_seed(seed)

        def randn(*shape):
            return torch.randn(shape, generator=gen, device=DEV)
        self.x, self.r, self.dy = (randn(n, hidden).to(torch.bfloat16) for _ in range(3))
        self.gamma, self.beta = randn(hidden), randn(hidden)
        self.p = ac.DalParams(n_rows=n, hidden=hidden, p_drop=0.1, eps=1e-5, seed=seed, offset=0)
        self.z, self.y, self.dx, self.dres = (torch.zeros_like(self.x) for _ in range(4))
        self.mean, self.rstd = torch.zeros(n, device=DEV), torch.zeros(n, device=DEV)
        self.dgamma, self.dbeta = torch.zeros_like(self.gamma), torch.zeros_like(self.gamma)
        self.ws = torch.zeros(ac.attn_core_dropout_add_ln_bwd_workspace_bytes(self.p), dtype=torch.uint8, device=DEV)
        at = [t.data_ptr() for t in (self.x, self.r, self.gamma, self.beta, self.z, self.y, self.mean, self.rstd)]
        self.forward = lambda stream=0: ac.attn_core_dropout_add_ln_fwd(self.p, *at, stream)
        back = [self.dy.data_ptr(), 0] + [t.data_ptr() for t in (self.z, self.mean, self.rstd, self.gamma, self.dx, self.dres,
                                                                 self.dgamma, self.dbeta, self.ws)]
        self.backward = lambda stream=0: ac.attn_core_dropout_add_ln_bwd(self.p, *back, self.ws.numel(), stream)

    def outputs(self):
        return [t.clone() for t in (self.z, self.y, self.mean, self.rstd, self.dx, self.dres, self.dgamma, self.dbeta)]


@pytest.mark.parametrize("which", ["forward", "backward"])
@pytest.mark.parametrize("long,short", [(12288, 8200), (28672, 24584), (2048, 64)])
def test_rows_of_different_lengths(long, short, which):
    rows = [Boundary(h, i) for i, h in enumerate([long, short] * 4)]
    want = []
    for b in rows:
        assert b.forward() == ac.OK and b.backward() == ac.OK
        want.append(b.outputs())
    assert at_once([getattr(b, which) for b in rows], 3000) == []
    for b, w in zip(rows, want):
        assert all(torch.equal(x, y) for x, y in zip(b.outputs(), w))
