"""Eviction within the sequences' own pages again and again from the same state: what
its blocks wait for one another for (flags, loads before stores) must come out the
same every time, alone and beside other work."""
import pytest
import torch

import attention_core_gb300 as ac
from tests.test_gpu_evict import bits, check, make

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


# many times more chunks of 64 rows than blocks at once; few lines over clusters; lines
# beyond shared memory; chunks over several small pages
CASES = [([20000] * 8 + [333, 0, 64], 4, 64, 16, 15000), ([100000, 33000], 1, 128, 64, 60000),
         ([50000, 47000, 100], 32, 64, 256, 40000), ([1500, 700, 65, 1], 3, 160, 16, 640), ([9000] * 5, 8, 96, 128, 8999)]


@pytest.mark.parametrize("beside", [False, True])
@pytest.mark.parametrize("nk,hkv,d,ps,keep", CASES)
def test_the_same_every_time(nk, hkv, d, ps, keep, beside):
    p, w = make(nk, hkv, d, ps, seed=4, kind="ties")
    batch = p.batch()
    k0, v0, w0 = p.k_pages.clone(), p.v_pages.clone(), w.clone()
    check(p, batch, w, [keep] * len(nk), 4, 200)                 # the first is the definition's
    want = [bits(x).clone() for x in (p.k_pages, p.v_pages, w)]
    keep_dev = torch.tensor([keep] * len(nk), dtype=torch.int32, device=DEV)
    kept = torch.zeros(w.shape, dtype=torch.int32, device=DEV)
    first = None
    side, work = torch.cuda.Stream(), torch.randn(2048, 2048, device=DEV)
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(40):
        for a, b in ((p.k_pages, k0), (p.v_pages, v0), (w, w0)):
            a.copy_(b)
        kept.zero_()
        if beside:
            with torch.cuda.stream(side):
                torch.mm(work, work)
        ac.paged_evict(batch, w, keep_dev, p.k_pages, p.v_pages, first=4, recent=200, kept=kept)
        for a, b in zip((p.k_pages, p.v_pages, w), want):
            assert torch.equal(bits(a), b)
        first = kept.clone() if first is None else first
        assert torch.equal(kept, first)
    torch.cuda.synchronize()
    assert int(p.status.item()) == 0


def test_a_wait_that_runs_out_leaves_both_caches():
    """... the rows of V like those of K."""
    p, w = make([4000, 700], 2, 128, 16)
    k0, v0 = p.k_pages.clone(), p.v_pages.clone()
    batch = p.batch(flags=ac.FLAG_TEST_WAIT_TIMEOUT, wait_timeout_ms=5)
    ac.paged_evict(batch, w, torch.tensor([1000, 600], dtype=torch.int32, device=DEV), p.k_pages, p.v_pages)
    torch.cuda.synchronize()
    assert int(p.status.item()) & 0xff == ac.ERR_DEVICE_TIMEOUT
    assert torch.equal(bits(p.k_pages), bits(k0)) and torch.equal(bits(p.v_pages), bits(v0))
