"""Attention over shared prefixes where one kernel plans and another, beside it, takes
the plan over: calls of different lengths in one workspace, each of which finds the
other's plan there, on their own and replayed from graphs."""
import pytest
import torch

import attention_core_gb300 as ac
from tests.serve_ref import attend, check_attention
from tests.test_gpu_evict import bits
from tests.test_gpu_prefix import shared

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def of_lengths(groups, each, pages, own, seed):
    """Groups whose rows are many together and few each."""
    n = groups * each
    return shared([(each, max(1, pages - 3 * g)) for g in range(groups)], [1] * n,
                  [1 + (own * (i + 1) + 7 * seed) % 211 for i in range(n)], 16, 2, 128, 16, seed=seed, cols=pages + 14)


@pytest.mark.parametrize("groups,each", [(2, 12), (5, 25)])          # planned by the block, by a kernel
def test_a_plan_is_the_calls_own(groups, each):
    p = [of_lengths(groups, each, pages, own, s) for s, (pages, own) in enumerate([(40, 37), (22, 101)])]
    batch = [x.batch(group_starts=x.starts, prefix_pages=x.pages) for x in p]
    batch[1].workspace = batch[0].workspace
    out = [(torch.empty_like(x.q), torch.empty((x.h_q, x.n_tokens), device=DEV)) for x in p]

    def call(i):
        ac.paged_prefix_fwd(batch[i], p[i].q, p[i].k_pages, p[i].v_pages, out=out[i][0], lse=out[i][1])
    want = []
    for i in range(2):
        call(i)
        check_attention(*out[i], attend(p[i]), p[i])
        want.append([bits(x).clone() for x in out[i]])
    graphs = []
    for i in range(2):
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call(i)
    wrong = torch.zeros((), dtype=torch.int64, device=DEV)
    for turn in range(300):
        i = turn % 2 if turn % 7 else 0
        for x in out[i]:
            x.zero_()
        call(i) if turn % 3 else graphs[i].replay()
        wrong += sum((bits(x) != w).sum() for x, w in zip(out[i], want[i]))
    assert int(wrong) == 0
    assert all(int(x.status.item()) == 0 for x in p)


def test_lengths_that_change_between_calls_of_one_graph():
    """Two calls of one batch in a graph, its lengths changed between them: the second
    finds the first's plan and stamps where it puts its own."""
    p = of_lengths(2, 12, 40, 37, 3)
    full = p.kv_lens.clone()
    # the first call's lengths end inside the shared pages for one group's sequences
    short = torch.where(torch.arange(24, device=DEV) % 12 < 5, full, full - (full % 16)).to(torch.int32)
    batch = p.batch(group_starts=p.starts, prefix_pages=p.pages)
    out = [(torch.empty_like(p.q), torch.empty((p.h_q, p.n_tokens), device=DEV)) for _ in range(2)]

    def both():
        for lens, (o, lse) in zip((short, full), out):
            p.kv_lens.copy_(lens)
            ac.paged_prefix_fwd(batch, p.q, p.k_pages, p.v_pages, out=o, lse=lse)
    both()
    whole = p.keys, p.values, p.nk
    for lens, x in zip((short, full), out):
        p.nk = lens.tolist()
        p.keys, p.values = ([k[:n] for k, n in zip(y, p.nk)] for y in whole[:2])
        check_attention(*x, attend(p), p)
    want = [[bits(x).clone() for x in y] for y in out]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    wrong = torch.zeros((), dtype=torch.int64, device=DEV)
    for _ in range(100):
        for y in out:
            for x in y:
                x.zero_()
        graph.replay()
        wrong += sum((bits(x) != w).sum() for y, v in zip(out, want) for x, w in zip(y, v))
    assert int(wrong) == 0 and int(p.status.item()) == 0


def test_few_tokens_among_many_sequences():
    """More sequences than a block plans for, nearly all without new tokens."""
    nq = [1 if i % 9 == 0 else 0 for i in range(180)]
    p = shared([(90, 4), (60, 7), (30, 2)], nq, [1 + 3 * i for i in range(180)], 1, 1, 64, 16, seed=7)
    batch = p.batch(group_starts=p.starts, prefix_pages=p.pages)
    for _ in range(2):
        o, lse = ac.paged_prefix_fwd(batch, p.q, p.k_pages, p.v_pages)
        check_attention(o, lse, attend(p), p)
        batch.workspace.fill_(255)
    assert int(p.status.item()) == 0
