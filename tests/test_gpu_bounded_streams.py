"""The operators of the bounded cache as programs run them: a whole step captured in
one graph and replayed, two batches at once on two streams, batches dropped while
their calls run, runs repeated bit by bit."""
import pytest
import torch

import attention_core_gb300 as ac
from tests.test_gpu_evict import bits
from tests.test_gpu_prefix import shared

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def problem(seed, n=12, pages=40, d=128, ps=16):
    """Samples of a prompt, two of them with several new tokens, and what bounds them."""
    nq = [1] * n
    nq[1], nq[2] = 3, 40
    own = [max(a, 1 + (37 * i + seed) % 300) for i, a in enumerate(nq)]
    p = shared([(n, pages)], nq, own, 8, 2, d, ps, seed=seed)
    shape = (n, 2, p.table.shape[1] * ps)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    p.weights = torch.rand(shape, generator=gen, device=DEV)
    p.keep = torch.tensor([pages * ps // 2 + 5 * i for i in range(n)], dtype=torch.int32, device=DEV)
    # each sequence moves to pages of its own
    cols = [-(-int(k) // ps) for k in p.keep]
    total = sum(cols)
    for name in ("k_pages", "v_pages"):
        old = getattr(p, name)
        setattr(p, name, torch.cat((old, torch.zeros((total,) + old.shape[1:], dtype=old.dtype, device=DEV))))
    out, at = torch.full(p.table.shape, -1, dtype=torch.int32), p.n_pages
    for i, c in enumerate(cols):
        out[i, :c] = torch.arange(at, at + c)
        at += c
    p.n_pages, p.out_table = at, out.to(DEV)
    return p


class Step:
    def __init__(self, p):
        self.p = p
        self.batch = p.batch(group_starts=p.starts, prefix_pages=p.pages)
        self.o = torch.empty_like(p.q)
        self.lse = torch.empty((p.h_q, p.n_tokens), dtype=torch.float32, device=DEV)
        self.gathered = torch.zeros_like(p.weights)
        self.left = torch.zeros_like(p.weights)
        self.kept = torch.zeros(p.weights.shape, dtype=torch.int32, device=DEV)

    def run(self):
        p = self.p
        ac.paged_prefix_fwd(self.batch, p.q, p.k_pages, p.v_pages, out=self.o, lse=self.lse)
        ac.paged_weights(self.batch, p.q, self.lse, p.k_pages, p.weights, decay=0.9, out=self.gathered)
        ac.paged_evict(self.batch, self.gathered, p.keep, p.k_pages, p.v_pages, first=4, recent=20,
                       out_table=p.out_table, out_weights=self.left, kept=self.kept)

    def results(self):
        return [bits(x).clone() for x in (self.o, self.lse, self.gathered, self.left, self.kept, self.p.k_pages,
                                          self.p.v_pages)]

    def clear(self):
        for x in (self.o, self.lse, self.gathered, self.left):
            x.zero_()
        self.kept.zero_()


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_a_step_in_one_graph():
    s = Step(problem(1))
    s.run()
    torch.cuda.synchronize()
    want = s.results()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    for _ in range(3):
        s.clear()
        s.batch.workspace.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert same(want, s.results())
    assert int(s.p.status.item()) == 0


def test_two_streams_at_once():
    """Two batches, with a workspace each, whose calls overlap: each as by itself."""
    steps = [Step(problem(2)), Step(problem(3, n=5, pages=200, d=96))]
    wants = []
    for s in steps:
        s.run()
        torch.cuda.synchronize()
        wants.append(s.results())
        s.clear()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(20):
        for s, stream in zip(steps, streams):
            with torch.cuda.stream(stream):
                s.run()
    torch.cuda.synchronize()
    for s, want in zip(steps, wants):
        assert same(want, s.results())
        assert int(s.p.status.item()) == 0


def test_a_batch_dropped_while_its_calls_run():
    """On another stream than its memory's: nothing that is allocated afterwards may
    take its tables' or its workspace's place before the calls are done."""
    p = problem(4)
    s = Step(p)
    s.run()
    torch.cuda.synchronize()
    want = s.results()
    s.clear()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    junk = []
    for _ in range(10):
        tables = [x.clone() for x in (p.cu, p.kv_lens, p.table, p.starts, p.pages)]
        batch = ac.PagedBatch(*tables[:3], n_tokens=p.n_tokens, h_q=p.h_q, h_kv=p.h_kv, d=p.d, page_size=p.ps,
                              n_pages=p.n_pages, group_starts=tables[3], prefix_pages=tables[4])
        del tables
        s.batch = batch
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(200000)
            s.run()
        size = batch.workspace.numel()
        del batch
        s.batch = None
        junk = [torch.full((size,), 255, dtype=torch.uint8, device=DEV)] + \
               [torch.full((n,), 1 << 29, dtype=torch.int32, device=DEV) for n in (13, 12, 12 * 64, 2, 1)]
    torch.cuda.synchronize()
    assert same(want, s.results()) and len(junk) == 6


def test_other_splits_of_the_sms_do_not_matter_for_the_bits():
    """The same call again and again among other work on the card."""
    s = Step(problem(5, n=30, pages=100))
    s.run()
    torch.cuda.synchronize()
    want = s.results()
    other, busy = torch.cuda.Stream(), torch.randn(2048, 2048, device=DEV)
    for _ in range(10):
        with torch.cuda.stream(other):
            busy = (busy @ busy).clamp(-1, 1)
        s.run()
        torch.cuda.synchronize()
        assert same(want, s.results())
