"""Calls made by several host threads at once through the C entries (which run without
the interpreter's lock), each with its own stream, batch and workspace: the sizes of
one thread's calls are no business of another's."""
import threading

import pytest
import torch

import attention_core_gb300 as ac
from tests.test_gpu_evict import bits, make

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def at_once(calls, times):
    """Each of `calls` that often by a thread and on a stream of its own, which it is
    given; what went wrong."""
    torch.cuda.synchronize()
    ready, wrong = threading.Barrier(len(calls)), []

    def work(call):
        stream = torch.cuda.Stream(DEV)
        ready.wait(60)
        try:
            for _ in range(times):
                rc = call(stream.cuda_stream)
                assert rc == ac.OK, rc
        except Exception as e:              # noqa: BLE001 (reported below)
            wrong.append(repr(e))
        stream.synchronize()
    threads = [threading.Thread(target=work, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    return wrong


class Eviction:
    """Lines that move to pages of their own, so that a call can be repeated."""

    def __init__(self, nk, h_kv, width, seed, ps=16):
        self.p, self.w = make(nk, h_kv, 64, ps, seed=seed, spare=sum(-(-(n // 2) // ps) for n in nk), cols=-(-width // ps))
        used = set(self.p.host_table[self.p.host_table >= 0].tolist())
        fresh = [x for x in range(self.p.n_pages) if x not in used]
        out = torch.full(self.p.table.shape, -1, dtype=torch.int32)
        for i, n in enumerate(nk):
            for c in range(-(-(n // 2) // ps)):
                out[i, c] = fresh.pop()
        self.out_table = out.to(DEV)
        self.keep = torch.tensor([n // 2 for n in nk], dtype=torch.int32, device=DEV)
        self.left, self.kept = torch.zeros_like(self.w), torch.zeros(self.w.shape, dtype=torch.int32, device=DEV)
        self.batch = self.p.batch()

        ws = self.batch.workspace
        self.args = (self.batch.params, self.keep.data_ptr(), 4, 20, self.out_table.data_ptr(), self.p.k_pages.data_ptr(),
                     self.p.v_pages.data_ptr(), self.w.data_ptr(), self.left.data_ptr(), self.kept.data_ptr(),
                     ws.data_ptr(), ws.numel())

    def __call__(self, stream=0):
        return ac.attn_core_paged_evict(*self.args, stream)

    def results(self):
        return [bits(x).clone() for x in (self.left, self.kept, self.p.k_pages, self.p.v_pages)]


@pytest.mark.parametrize("n_seq,h_kv,wide,narrow", [(10, 8, 16384, 600),       # a block for each line
                                                    (1, 1, 200000, 5000)])      # clusters
def test_evictions_from_tables_of_different_width(n_seq, h_kv, wide, narrow):
    """What a line takes of shared memory goes by the table's width: here 64 KB, more than
    a kernel may have unasked, beside 8.  Short lines, so that the threads spend their
    time launching."""
    calls = [Eviction([300] * n_seq, h_kv, width, i) for i, width in enumerate([wide, narrow] * 4)]
    want = []
    for c in calls:
        assert c() == ac.OK
        want.append(c.results())
    for c in calls:
        c.left.zero_()
        c.kept.zero_()
    assert at_once(calls, 3000) == []
    for c, w in zip(calls, want):
        assert all(torch.equal(a, b) for a, b in zip(c.results(), w))
        assert int(c.p.status.item()) == 0
