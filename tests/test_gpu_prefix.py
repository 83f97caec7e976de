"""Attention of sequences that share their first pages against the plain 64-bit
attention of each sequence over all its keys: groups of every shape, rows that
begin inside the shared pages, empty sequences and groups, cut tiles, and tables
that change under a captured graph."""
import math

import pytest
import torch

import attention_core_gb300 as ac
from tests.serve_ref import Paged, attend, check_attention

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def shared(groups, nq, own, h_q, h_kv, d, ps, seed=0, outside=(), **kw):
    """A paged cache whose sequences share pages: `groups` = [(sequences, shared
    pages)], then the sequences `outside` = [(new tokens, keys)] of no group.  A
    member's own copies of the shared pages hold NaN."""
    prefix = [p * ps for n, p in groups for _ in range(n)]
    nk = [a + b for a, b in zip(prefix, own)] + [k for _, k in outside]
    p = Paged(list(nq) + [n for n, _ in outside], nk, h_q, h_kv, d, ps, seed=seed, **kw)
    first = 0
    for n, pages in groups:
        for i in range(first + 1, first + n):
            for x in (p.k_pages, p.v_pages):
                x[p.table[i, :pages].long()] = math.nan
            p.table[i, :pages] = p.table[first, :pages]
            for x in (p.keys, p.values):
                x[i][: pages * ps] = x[first][: pages * ps]
        first += n
    starts = [0]
    for n, _ in groups:
        starts.append(starts[-1] + n)
    p.starts = torch.tensor(starts, dtype=torch.int32, device=DEV)
    p.pages = torch.tensor([n for _, n in groups], dtype=torch.int32, device=DEV)
    return p


def run(p, **kw):
    batch = p.batch(group_starts=p.starts, prefix_pages=p.pages, **kw)
    out = torch.full(p.q.shape, 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((p.h_q, p.n_tokens), 7.0, dtype=torch.float32, device=DEV)
    ac.paged_prefix_fwd(batch, p.q, p.k_pages, p.v_pages, out=out, lse=lse)
    return out, lse


def rest_untouched(p, o, lse):
    used = p.cu_host[-1]
    assert (o[used:] == 7).all() and (lse[:, used:] == 7).all()


@pytest.mark.parametrize("d,ps", [(64, 16), (96, 32), (128, 64), (160, 128), (128, 256)])
@pytest.mark.parametrize("hq,hkv", [(8, 2), (3, 3), (6, 2), (16, 1)])
def test_single_tokens(hq, hkv, d, ps):
    """Samples of three prompts, a group of one and a sequence outside."""
    own = [1, 5, 130, 2, 77, 1, 300, 9, 40]
    p = shared([(4, 3), (3, 1), (2, 5)], [1] * 9, own, hq, hkv, d, ps, outside=[(1, 40), (1, 1)], n_tokens=13)
    o, lse = run(p)
    check_attention(o, lse, attend(p), p)
    rest_untouched(p, o, lse)
    assert int(p.status.item()) == 0


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("hq,hkv,d,ps", [(4, 4, 160, 32), (8, 1, 128, 16), (12, 4, 96, 64), (5, 1, 64, 16)])
def test_several_new_tokens(hq, hkv, d, ps, causal):
    """Drafts and chunks over shared pages: row tiles of the group that span
    sequences, and own parts of several tiles."""
    nq = [3, 200, 1, 17, 64, 129, 0, 8]
    own = [5, 240, 1, 30, 64, 300, 20, 11]
    p = shared([(5, 20), (3, 7)], nq, own, hq, hkv, d, ps, seed=1)
    o, lse = run(p, causal=causal)
    check_attention(o, lse, attend(p, causal=causal), p)
    assert int(p.status.item()) == 0


def test_new_tokens_begin_inside_the_shared_pages():
    """A sequence whose new tokens' own keys lie in pages named as shared: only the
    pages that all hold before their first new token are taken together."""
    p = shared([(4, 8)], [1, 40, 2, 1], [1, 3, 90, 60], 8, 2, 128, 16)
    o, lse = run(p)                                    # sequence 1 has 131 keys, 91 of them old
    check_attention(o, lse, attend(p), p)
    # fewer keys than new tokens: its first rows see none, and nothing is shared
    p = shared([(3, 2)], [1, 50, 1], [4, 2, 9], 4, 2, 64, 16)
    assert p.nk[1] < p.nq[1]
    o, lse = run(p)
    check_attention(o, lse, attend(p), p)
    assert int(p.status.item()) == 0


@pytest.mark.parametrize("hq,hkv,d,ps,n,pages,own", [(64, 8, 128, 64, 20, 60, 500), (8, 8, 96, 16, 33, 300, 1000),
                                                     (16, 16, 160, 32, 9, 100, 70), (128, 1, 64, 128, 2, 150, 1)])
def test_cut_tiles(hq, hkv, d, ps, n, pages, own):
    """Long shared and own parts, whose tiles are cut and joined; the same bits
    again, on another stream, with what the workspace held before left in it."""
    gen = torch.Generator().manual_seed(n)
    mine = [int(x) for x in torch.randint(1, own + 1, (n,), generator=gen)]
    p = shared([(n, pages)], [1] * n, mine, hq, hkv, d, ps)
    o, lse = run(p)
    check_attention(o, lse, attend(p), p)
    batch = p.batch(group_starts=p.starts, prefix_pages=p.pages)
    batch.workspace.fill_(255)                          # NaN rows, records of every kind
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = [ac.paged_prefix_fwd(batch, p.q, p.k_pages, p.v_pages) for _ in range(2)]
    torch.cuda.synchronize()
    for a, b in again:
        assert torch.equal(a.view(torch.int16), o.view(torch.int16)) and torch.equal(b, lse)
    assert int(p.status.item()) == 0


@pytest.mark.parametrize("n", [62, 63, 64, 150, 1100])
def test_many_sequences(n):
    """On both sides of what a block plans for itself (128 sequences and groups)."""
    gen = torch.Generator().manual_seed(n)
    groups = [(2, 1 + i % 5) for i in range(n // 2)] + [(n % 2, 3)]
    own = [int(x) for x in torch.randint(1, 60, (n,), generator=gen)]
    nq = [1 + (i % 7 == 3) * 2 for i in range(n)]
    own = [max(a, b) for a, b in zip(own, nq)]
    p = shared(groups, nq, own, 4, 2, 64, 16, outside=[(1, 30), (40, 50)])
    o, lse = run(p)
    check_attention(o, lse, attend(p), p)
    assert int(p.status.item()) == 0
    # one group of all: more rows than a tile
    p = shared([(n, 9)], nq, own, 4, 2, 64, 16, seed=1)
    o, lse = run(p)
    check_attention(o, lse, attend(p), p)
    assert int(p.status.item()) == 0


def test_empty_groups_and_sequences():
    p = shared([(2, 3), (0, 5), (3, 2)], [1, 0, 0, 2, 0], [4, 6, 1, 9, 0], 8, 2, 128, 16, n_tokens=5)
    o, lse = run(p)
    check_attention(o, lse, attend(p), p)
    rest_untouched(p, o, lse)
    p = shared([(2, 3)], [0, 0], [4, 6], 8, 2, 128, 16, n_tokens=3)
    o, lse = run(p)
    rest_untouched(p, o, lse)
    assert int(p.status.item()) == 0


@pytest.mark.parametrize("starts,pages", [([0, 5, 3, 6], [2, 2, 2]), ([0, 4, 9, 9], [2, 2, 2]), ([-1, 2, 4, 6], [1, 1, 1]),
                                          ([0, 2, 4, 6], [2, -1, 2])])
def test_groups_that_do_not_fit_are_reported(starts, pages):
    """... and share nothing: the results are right."""
    p = shared([(6, 4)], [1] * 6, [3, 9, 1, 20, 40, 5], 8, 2, 128, 16)
    p.starts = torch.tensor(starts, dtype=torch.int32, device=DEV)
    p.pages = torch.tensor(pages, dtype=torch.int32, device=DEV)
    o, lse = run(p)
    check_attention(o, lse, attend(p), p)
    assert int(p.status.item()) == ac.ERR_DEVICE_TABLE


def test_tokens_without_a_key():
    """New tokens of sequences that hold nothing, in a group and outside."""
    p = shared([(3, 0)], [1, 2, 1], [0, 0, 5], 8, 2, 128, 16, outside=[(1, 0), (40, 0), (1, 3)])
    o, lse = run(p)
    check_attention(o, lse, attend(p), p)
    assert (lse[:, :3] == -math.inf).all() and (o[4:45] == 0).all()
    assert int(p.status.item()) == 0


def test_more_pages_than_the_sequences_hold():
    p = shared([(2, 4)], [1, 1], [1, 1], 8, 2, 128, 16)
    p.pages.fill_(1 << 30)
    o, lse = run(p)
    check_attention(o, lse, attend(p), p)
    assert int(p.status.item()) == 0


def test_a_captured_graph_follows_the_tables():
    p = shared([(3, 6), (3, 2)], [1] * 6, [200, 9, 1, 20, 40, 5], 16, 2, 128, 16, n_tokens=8)
    batch = p.batch(group_starts=p.starts, prefix_pages=p.pages)
    out, lse = torch.empty_like(p.q), torch.empty((p.h_q, p.n_tokens), dtype=torch.float32, device=DEV)

    def call():
        ac.paged_prefix_fwd(batch, p.q, p.k_pages, p.v_pages, out=out, lse=lse)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for starts, pages in (([0, 3, 6], [6, 2]), ([0, 2, 3], [6, 6]), ([3, 3, 6], [1, 2]), ([0, 0, 0], [6, 6])):
        p.starts.copy_(torch.tensor(starts, dtype=torch.int32))
        p.pages.copy_(torch.tensor(pages, dtype=torch.int32))
        out.fill_(7.0)
        lse.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        check_attention(out, lse, attend(p), p)
        rest_untouched(p, out, lse)
    # other lengths: two sequences fewer new tokens, shorter contexts
    p.cu.copy_(torch.tensor([0, 1, 2, 3, 3, 4, 4], dtype=torch.int32))
    p.nq, p.cu_host = [1, 1, 1, 0, 1, 0], [0, 1, 2, 3, 3, 4, 4]
    p.nk = [100, 100, 97, 33, 40, 30]
    p.kv_lens.copy_(torch.tensor(p.nk, dtype=torch.int32))
    p.keys, p.values = [k[:n] for k, n in zip(p.keys, p.nk)], [v[:n] for v, n in zip(p.values, p.nk)]
    p.starts.copy_(torch.tensor([0, 3, 6], dtype=torch.int32))
    p.pages.copy_(torch.tensor([6, 2], dtype=torch.int32))
    out.fill_(7.0)
    lse.fill_(7.0)
    graph.replay()
    torch.cuda.synchronize()
    check_attention(out, lse, attend(p), p)
    rest_untouched(p, out, lse)
    assert int(p.status.item()) == 0


def test_special_values():
    """NaN and infinite scores as paged_fwd has them, in shared and in own keys."""
    p = shared([(3, 4)], [1, 1, 1], [70, 1, 9], 4, 2, 64, 16)
    page = int(p.table[0, 1])
    p.k_pages[page, 0, 3] = math.nan                    # a shared key: every row of KV head 0
    p.k_pages[int(p.table[0, 5]), 1, 0] = math.inf      # an own key of sequence 0, KV head 1
    batch = p.batch(group_starts=p.starts, prefix_pages=p.pages)
    o, lse = ac.paged_prefix_fwd(batch, p.q, p.k_pages, p.v_pages)
    want_o, want_lse = ac.paged_fwd(batch, p.q, p.k_pages, p.v_pages)
    assert torch.isnan(lse[:2]).all() and torch.isnan(o[:, :2]).all()
    assert torch.equal(torch.isnan(lse), torch.isnan(want_lse))
    assert torch.equal(torch.isnan(o.float()), torch.isnan(want_o.float()))
    fine = torch.isfinite(want_lse)
    assert ((lse - want_lse)[fine].abs() <= 2.0 ** -12).all()


def test_a_wait_that_runs_out_is_reported():
    p = shared([(3, 4)], [1, 1, 1], [70, 1, 9], 4, 2, 64, 16)
    run(p, flags=ac.FLAG_TEST_WAIT_TIMEOUT, wait_timeout_ms=5)
    torch.cuda.synchronize()
    assert int(p.status.item()) & 0xff == ac.ERR_DEVICE_TIMEOUT
    p.status.zero_()
    o, lse = run(p)
    check_attention(o, lse, attend(p), p)
