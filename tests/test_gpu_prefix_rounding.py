"""Single tokens over shared keys: probabilities go in as two bf16 terms, as
``paged_fwd`` has them for such batches, so that O is off by its own rounding."""
import pytest
import torch

import attention_core_gb300 as ac
from tests.serve_ref import attend, check_attention
from tests.test_gpu_prefix import shared

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("n,pages,hq,hkv,d,ps,causal", [(64, 40, 8, 1, 128, 16, True), (40, 20, 16, 16, 160, 32, True),
                                                       (24, 64, 16, 2, 64, 64, True), (48, 30, 8, 2, 96, 16, False)])
def test_only_the_result_is_rounded(n, pages, hq, hkv, d, ps, causal):
    """With R the 2-norm of what rounding the 64-bit O to bf16 changes: two terms leave
    2^-17 of each probability, far below R, and an error of R again within a few
    percent (elements at a tie may go the other way); one term's own 2^-9 of each
    probability, as random as R's, would make it 1.4 R."""
    p = shared([(n, pages)], [1] * n, [1 + i % 5 for i in range(n)], hq, hkv, d, ps, seed=n)
    for groups in (dict(group_starts=p.starts, prefix_pages=p.pages), None):
        batch = p.batch(causal=causal, **(groups or {}))
        call = ac.paged_prefix_fwd if groups else ac.paged_fwd
        o, lse = call(batch, p.q, p.k_pages, p.v_pages)
        want = attend(p, causal=causal)
        check_attention(o, lse, want, p)
        exact = want[0]
        rounding = (exact.to(torch.bfloat16).double() - exact).norm()
        assert (o.double() - exact).norm() <= 1.1 * rounding
    assert int(p.status.item()) == 0
