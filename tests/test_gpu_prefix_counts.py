"""Counts of shared pages that are smaller than what sequences share, and counts that
follow the page table under a captured graph while a pool forks, copies and evicts."""
import pytest
import torch

import attention_core_gb300 as ac
from attention_core_gb300.pagepool import PagePool
from tests.serve_ref import attend, check_attention
from tests.test_gpu_prefix import shared

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("hq,hkv", [(2, 2), (16, 2)])
@pytest.mark.parametrize("counts", [[0, 0], [1, 0], [7, 5], [12, 9]])
def test_smaller_counts(hq, hkv, counts):
    p = shared([(6, 12), (5, 9)], [1] * 11, [3 * i + 1 for i in range(11)], hq, hkv, 128, 16)
    p.pages.copy_(torch.tensor(counts, dtype=torch.int32))
    batch = p.batch(group_starts=p.starts, prefix_pages=p.pages)
    o, lse = ac.paged_prefix_fwd(batch, p.q, p.k_pages, p.v_pages)
    check_attention(o, lse, attend(p), p)
    assert int(p.status.item()) == 0


class Pooled:
    """Sequences of a pool as the batch that the plain attention takes."""

    def __init__(self, n, h_q, h_kv, d, ps, cols, n_pages):
        gen = torch.Generator(device=DEV).manual_seed(5)
        self.h_q, self.h_kv, self.d, self.ps, self.n_tokens = h_q, h_kv, d, ps, n
        self.nq, self.cu_host = [1] * n, list(range(n + 1))

        def randn(*shape):
            return torch.randn(shape, generator=gen, device=DEV).to(torch.bfloat16)
        self.q = randn(n, h_q, d)
        self.k_pages, self.v_pages = randn(n_pages, h_kv, ps, d), randn(n_pages, h_kv, ps, d)
        self.cu = torch.arange(n + 1, dtype=torch.int32, device=DEV)
        self.kv_lens = torch.zeros(n, dtype=torch.int32, device=DEV)
        self.table = torch.zeros((n, cols), dtype=torch.int32, device=DEV)
        self.starts = torch.zeros(n + 1, dtype=torch.int32, device=DEV)
        self.counts = torch.zeros(n, dtype=torch.int32, device=DEV)
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)

    def follow(self, pool, seqs):
        table, lens = pool.tables(seqs, self.table.shape[1])
        starts, counts = pool.groups(seqs)
        n, groups = len(seqs), len(counts)
        full = [int(x) for x in starts] + [n] * (n - groups)               # empty groups behind
        for a, b in ((self.table, table), (self.kv_lens, lens), (self.starts, full),
                     (self.counts, [int(x) for x in counts] + [0] * (n - groups))):
            a.copy_(torch.as_tensor(b, dtype=torch.int32))
        self.nk = [int(x) for x in lens]
        self.keys, self.values = [], []
        for i, m in enumerate(self.nk):
            at = torch.arange(m, device=DEV)
            page, row = self.table[i].long()[at // self.ps], at % self.ps
            self.keys.append(self.k_pages[page, :, row])
            self.values.append(self.v_pages[page, :, row])


def test_counts_follow_a_pool_under_a_captured_graph():
    n, ps = 12, 16
    pool = PagePool(400, ps)
    seqs = [pool.add()]
    pool.extend(seqs[0], 200)
    seqs += [pool.fork(seqs[0]) for _ in range(n - 1)]
    p = Pooled(n, 8, 1, 64, ps, 30, 400)
    batch = ac.PagedBatch(p.cu, p.kv_lens, p.table, n_tokens=n, h_q=8, h_kv=1, d=64, page_size=ps, n_pages=400,
                          dev_status=p.status.data_ptr(), group_starts=p.starts, prefix_pages=p.counts)
    out, lse = torch.empty_like(p.q), torch.empty((8, n), device=DEV)

    def call():
        ac.paged_prefix_fwd(batch, p.q, p.k_pages, p.v_pages, out=out, lse=lse)

    def check():
        p.follow(pool, seqs)
        graph.replay()
        torch.cuda.synchronize()
        check_attention(out, lse, attend(p), p)
    p.follow(pool, seqs)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    check()
    for step in range(3):
        for i, s in enumerate(seqs):
            pairs = pool.extend(s, 1 + (i + step) % 5)
            if pairs:
                ac.page_copy(p.k_pages, pairs)
                ac.page_copy(p.v_pages, pairs)
        check()
    for some, keep in ((seqs[2:5], 50), (seqs[:1], 33), (seqs[6:], 64)):
        pool_table = pool.shrink(some, [keep] * len(some), 30)
        assert (pool_table[:, :-(-keep // ps)] >= 0).all()
        check()
    assert int(p.status.item()) == 0
