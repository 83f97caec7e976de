"""The two ways in which attention over the paged cache shares out its work, on the
GPU: that whole tiles really are handed out (the counter in the workspace says
so), that a captured call moves between the two, and that the results are the
definition's either way."""
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


def _counter(b):
    """The next tile to hand out, the last 256 bytes' first word of the workspace."""
    need = ac.attn_core_paged_workspace_bytes(b.params)
    return int(b.workspace[need - 256:need - 252].view(torch.int32).item()) & 0xffffffff


def _tiles(p):
    return sum(-(-n // (128 // (p.h_q // p.h_kv))) for n in p.nq) * p.h_kv


UNTOUCHED = 0xffffffff

# (new tokens, keys, h_q, h_kv, d, page_size, causal)
HANDED_OUT = [
    ([700, 700], [4000, 1500], 32, 4, 128, 128, False),                       # 8 heads a KV head, every key seen
    ([64, 50, 57, 60], [3000, 90, 2000, 128], 128, 16, 128, 64, True),        # fewer keys than a tile among them
    ([500] * 4, [2500, 500, 1300, 512], 16, 16, 128, 64, True),
    ([210, 200, 170], [1500, 1400, 1300], 48, 16, 128, 16, True),             # 3 heads a KV head: 126 rows a tile
    ([700] * 3, [9000, 700, 4000], 16, 16, 128, 64, True),
    ([1600, 1600], [9000, 7000], 16, 16, 128, 64, True),                      # over 2.5 a block: the keys do not fit L2
    ([400] * 5, [3000] * 5, 16, 4, 160, 256, False),
]


@pytest.mark.parametrize("case", HANDED_OUT, ids=lambda c: "n{}_h{}-{}_d{}_{}".format(sum(c[0]), *c[2:5], "c" if c[6] else "n"))
def test_whole_tiles_come_from_the_counter(case):
    nq, nk, hq, hkv, d, ps, causal = case
    p = Paged(nq, nk, hq, hkv, d, ps, seed=50, n_tokens=sum(nq) + 9)
    b = p.batch(causal=causal)
    o, lse = torch.full_like(p.q, 7.0), torch.full((hq, p.n_tokens), 7.0, device=DEV)
    for _ in range(3):
        b.workspace.fill_(0xFF)
        ac.paged_fwd(b, p.q, p.k_pages, p.v_pages, out=o, lse=lse)
        torch.cuda.synchronize()
        # every tile was asked for, and every block asked once too often
        assert _tiles(p) < _counter(b) <= _tiles(p) + 160
    assert int(p.status.item()) == 0
    check_attention(o, lse, attend(p, causal), p)
    assert (o[sum(nq):] == 7).all() and (lse[:, sum(nq):] == 7).all()
    again, lse_again = ac.paged_fwd(b, p.q, p.k_pages, p.v_pages)
    assert torch.equal(again[:sum(nq)], o[:sum(nq)]) and torch.equal(lse_again[:, :sum(nq)], lse[:, :sum(nq)])


@pytest.mark.parametrize("hq,hkv,d", [(16, 16, 64), (16, 16, 160), (40, 20, 128)])
def test_replays_on_both_sides_of_the_rule(hq, hkv, d):
    """One capture: whole tiles from the counter where the lengths give enough of
    them, equal shares of cut tiles where they do not."""
    n = 500 if hq == hkv else 250
    p = Paged([n] * 5, [2000] * 5, hq, hkv, d, 64, seed=51)
    b = p.batch()
    o, lse = torch.empty_like(p.q), torch.empty(hq, p.n_tokens, device=DEV)
    ac.paged_fwd(b, p.q, p.k_pages, p.v_pages, out=o, lse=lse)
    torch.cuda.synchronize()
    assert _counter(b) > _tiles(p)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ac.paged_fwd(b, p.q, p.k_pages, p.v_pages, out=o, lse=lse)
    splits = []
    for lens in ([n] * 5, [100, 3, 2, 1, 0], [n] * 5, [1, 1, 1, 1, n], [n - 1, n, n - 90, n, n]):
        cu = [0]
        for x in lens:
            cu.append(cu[-1] + x)
        p.cu.copy_(torch.tensor(cu, dtype=torch.int32, device=DEV))
        sub = Paged.__new__(Paged)
        sub.__dict__.update(p.__dict__)
        sub.nq, sub.cu_host = lens, cu
        for _ in range(2):
            b.workspace.fill_(0xFF)
            g.replay()
            torch.cuda.synchronize()
            count = _counter(b)
            assert count == 0 or _tiles(sub) < count <= _tiles(sub) + 160
            splits.append(count > 0)
            check_attention(o, lse, attend(sub), sub)
        assert int(p.status.item()) == 0
    assert splits == [True, True, False, False, True, True, False, False, True, True]


def test_shares_where_the_counter_cannot_help():
    """Single tokens, a long context, short ones, too few tiles: no counter is set."""
    for nq, nk, hq, hkv, ps in (([1] * 64, [500] * 64, 8, 2, 64), ([1], [30000], 8, 8, 64),
                                ([300] * 3, [300] * 3, 16, 16, 64), ([90, 100, 1], [1500, 1400, 1300], 48, 16, 16)):
        p = Paged(nq, nk, hq, hkv, 128, ps, seed=52)
        b = p.batch()
        b.workspace.fill_(0xFF)
        o, lse = ac.paged_fwd(b, p.q, p.k_pages, p.v_pages)
        torch.cuda.synchronize()
        assert _counter(b) == UNTOUCHED
        check_attention(o, lse, attend(p), p)
