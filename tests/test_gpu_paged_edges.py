"""The paged cache's operators at their edges: results that depend on nothing but
their inputs, lengths and pages; tables that are out of order; NaN among the
keys; who owns the workspace, and for how long."""
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


# (new tokens a sequence, sequences, h_q, h_kv, d): head groups that leave rows of a
# tile unused (3: 126 rows of 128, 5: 125, 6: 126, 7: 126, 100: 100)
LEFT_OVER = [(42, 20, 24, 8, 128), (25, 40, 20, 4, 96), (21, 20, 48, 8, 160), (18, 40, 28, 4, 64), (8, 20, 100, 1, 128)]


@pytest.mark.parametrize("case", LEFT_OVER, ids=lambda c: "g{}_d{}".format(c[2] // c[3], c[4]))
def test_bits_do_not_depend_on_what_ran_before(case):
    """Rows of a tile that no head uses hold what an earlier kernel left in shared
    memory: a launch whose tiles are full, of large values or of zeros, changes no
    bit of the next launch's results."""
    n, n_seq, hq, hkv, d = case
    p = Paged([n] * n_seq, [1024] * n_seq, hq, hkv, d, 64, seed=40 + d)
    full = Paged([128] * 20, [256] * 20, 8, 8, d, 64, seed=41)       # one head a KV head: every row of a tile
    b, before = p.batch(), full.batch()
    results = []
    for scale in (0.0, 30.0, 0.0, 200.0):
        q = (full.q.float() * scale).to(torch.bfloat16)
        ac.paged_fwd(before, q, full.k_pages, full.v_pages)
        results.append(ac.paged_fwd(b, p.q, p.k_pages, p.v_pages))
    torch.cuda.synchronize()
    assert int(p.status.item()) == 0
    check_attention(*results[0], attend(p), p)
    for o, lse in results[1:]:
        assert torch.equal(o, results[0][0]) and torch.equal(lse, results[0][1])


@pytest.mark.parametrize("n,hq,hkv,d", [(1, 8, 1, 128), (5, 8, 1, 128), (1, 4, 2, 160), (9, 3, 1, 64), (1, 1, 1, 96)])
def test_bits_do_not_depend_on_the_neighbours_queries(n, hq, hkv, d):
    """Rows of a tile behind a sequence's last new token hold the next sequences'
    queries: other queries there change no bit of this one's results."""
    n_seq = 160 // hkv
    p = Paged([n] * n_seq, [1024] * n_seq, hq, hkv, d, 64, seed=42 + d)
    b = p.batch()
    o, lse = ac.paged_fwd(b, p.q, p.k_pages, p.v_pages)
    q = p.q.view(n_seq, n, hq, d).clone()
    q[1::2] = (q[1::2].float() * 30).to(torch.bfloat16)
    o2, lse2 = ac.paged_fwd(b, q.view_as(p.q), p.k_pages, p.v_pages)
    torch.cuda.synchronize()
    check_attention(o, lse, attend(p), p)
    assert torch.equal(o2.view_as(q)[::2], o.view_as(q)[::2])
    assert torch.equal(lse2.view(hq, n_seq, n)[:, ::2], lse.view(hq, n_seq, n)[:, ::2])


@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 64), (8, 1, 128), (3, 1, 96), (2, 2, 160)])
@pytest.mark.parametrize("nq,nk,at", [([1, 1], [300, 30], 7), ([1, 1], [30011, 40], 17000), ([9, 2], [500, 20], 494),
                                      ([200, 3], [2000, 50], 1900), ([1, 1], [1, 5], 0)])
def test_rows_that_see_a_nan_key_say_so(nq, nk, at, hq, hkv, d):
    """One key of the first sequence is NaN: O and LSE of the rows that see it are
    NaN (an LSE of -inf would say that they see no key), and those of the other
    rows, which the mask keeps from it, are the definition's."""
    p = Paged(nq, nk, hq, hkv, d, 32, seed=43 + d)
    page, row = p.places(0, torch.tensor([at], device=DEV))
    p.k_pages[page, :, row] = math.nan
    o, lse = ac.paged_fwd(p.batch(), p.q, p.k_pages, p.v_pages)
    torch.cuda.synchronize()
    assert int(p.status.item()) == 0
    sees = torch.zeros(p.n_tokens, dtype=torch.bool, device=DEV)
    sees[:nq[0]] = nk[0] - nq[0] + torch.arange(nq[0], device=DEV) >= at
    assert sees.any()
    assert torch.isnan(o[sees]).all() and torch.isnan(lse[:, sees]).all()
    ro, rlse, size = attend(p)             # of the keys as they were
    rest = ~sees
    assert ((o[rest].double() - ro[rest]).abs() <= 2.0 ** -8 * (ro[rest].abs() + size[rest]) + 2.0 ** -12 * size[rest]).all()
    assert ((lse[:, rest].double() - rlse[:, rest]).abs() <= 2.0 ** -12).all()


def _append_status(p, **kw):
    k0, v0 = p.k_pages.clone(), p.v_pages.clone()
    ac.paged_append(p.batch(**kw), p.q, p.k_new, p.v_new, p.k_pages, p.v_pages, table=ac.rope_table(p.d))
    torch.cuda.synchronize()
    code = int(p.status.item()) & 0xff
    p.status.zero_()
    same = torch.equal(k0.view(torch.int16), p.k_pages.view(torch.int16)) and \
        torch.equal(v0.view(torch.int16), p.v_pages.view(torch.int16))
    p.k_pages.copy_(k0), p.v_pages.copy_(v0)
    return code, same


def test_append_reports_starts_out_of_order():
    """Starts that decrease leave no sequence that owns the tokens between: nothing
    is written, and the status word says so."""
    for cu in ([0, 5, 3, 9], [0, 3, 9, 5], [4, 0, 6, 9], [0, 9, 0, 9], [0, -3, 4, 9]):
        p = Paged([5, 1, 3], [40, 33, 60], 4, 2, 64, 16, seed=44)
        assert _append_status(p) == (0, False)
        p.cu.copy_(torch.tensor(cu, dtype=torch.int32, device=DEV))
        assert _append_status(p) == (ac.ERR_DEVICE_TABLE, True), cu
    many = 700                                        # more starts than a block has threads
    p = Paged([1] * many, [20] * many, 2, 1, 64, 16, seed=45)
    assert _append_status(p) == (0, False)
    p.cu[600] = 400
    assert _append_status(p) == (ac.ERR_DEVICE_TABLE, True)


def test_append_reports_every_bad_table():
    def fresh():
        return Paged([2, 3], [40, 60], 4, 2, 64, 16, seed=46)
    p = fresh()
    p.table[0, 38 // 16] = p.n_pages
    assert _append_status(p)[0] == ac.ERR_DEVICE_TABLE
    p = fresh()
    p.table[0, 38 // 16] = -1
    assert _append_status(p)[0] == ac.ERR_DEVICE_TABLE
    for kv in (p.table.shape[1] * p.ps + 1, -5, 1):   # the last: a token before the sequence's start
        p = fresh()
        p.kv_lens[0] = kv
        assert _append_status(p)[0] == ac.ERR_DEVICE_TABLE, kv
    for cu in ([0, 2, 55], [0, 5, 55], [-2, 2, 5], [0, 6, 6]):
        p = fresh()
        p.cu.copy_(torch.tensor(cu, dtype=torch.int32, device=DEV))
        assert _append_status(p)[0] == ac.ERR_DEVICE_TABLE, cu


def test_append_writes_the_sequences_beside_a_bad_one():
    p = Paged([2, 3], [40, 60], 4, 2, 64, 16, seed=47)
    p.kv_lens[0] = -5
    ac.paged_append(p.batch(), p.q, p.k_new, p.v_new, p.k_pages, p.v_pages)
    torch.cuda.synchronize()
    assert int(p.status.item()) & 0xff == ac.ERR_DEVICE_TABLE
    page, row = p.places(1, torch.arange(57, 60, device=DEV))
    assert torch.equal(p.k_pages[page, :, row], p.k_new[2:]) and torch.equal(p.v_pages[page, :, row], p.v_new[2:])


def test_batch_dropped_while_its_call_runs():
    """The workspace and the tables that only the batch holds are not handed out
    again before a call on another stream has run."""
    p = Paged([1, 1], [9000, 300], 8, 1, 128, 64, seed=48)
    want = attend(p)
    side = torch.cuda.Stream()
    b = ac.PagedBatch(p.cu.clone(), p.kv_lens.clone(), p.table.clone(), n_tokens=2, h_q=8, h_kv=1, d=128, page_size=64,
                      n_pages=p.n_pages)
    mine = [b.workspace.data_ptr()] + [t.data_ptr() for t in b.tables]
    sizes = [b.workspace.numel()] + [t.numel() for t in b.tables]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(1 << 28)                    # about 0.15 s ahead of the call
        o, lse = ac.paged_fwd(b, p.q, p.k_pages, p.v_pages)
    del b
    taken = [torch.empty(sizes[0], dtype=torch.uint8, device=DEV)]
    taken += [torch.empty(n, dtype=torch.int32, device=DEV) for n in sizes[1:]]
    assert not side.query()                           # the call is still ahead
    assert not {t.data_ptr() for t in taken} & set(mine)
    torch.cuda.synchronize()
    check_attention(o, lse, want, p)
    # once the stream is done, its memory is there again
    del taken
    again = ac.PagedBatch(p.cu, p.kv_lens, p.table, n_tokens=2, h_q=8, h_kv=1, d=128, page_size=64, n_pages=p.n_pages)
    check_attention(*ac.paged_fwd(again, p.q, p.k_pages, p.v_pages), want, p)


def test_workspace_replaced():
    """The workspace in use is the one that the batch shows."""
    p = Paged([1, 2], [9000, 300], 8, 1, 128, 64, seed=49)
    b = p.batch()
    first, other = b.workspace, torch.zeros_like(b.workspace)
    b.workspace = other
    first.fill_(7)
    o, lse = ac.paged_fwd(b, p.q, p.k_pages, p.v_pages)
    torch.cuda.synchronize()
    assert (first == 7).all() and (other != 0).any()
    check_attention(o, lse, attend(p), p)
    for bad in (torch.empty(first.numel(), dtype=torch.uint8), None):
        with pytest.raises(ValueError):
            b.workspace = bad
    assert b.workspace is other


def test_workspace_smaller_than_its_elements_say():
    """An expanded tensor counts more elements than it has memory."""
    p = Paged([1], [20], 2, 1, 64, 16)
    need = p.batch().workspace.numel()
    with pytest.raises(ValueError):
        p.batch(workspace=torch.empty(1, dtype=torch.uint8, device=DEV).expand(need))
    with pytest.raises(ValueError):
        p.batch(workspace=torch.empty(2 * need, dtype=torch.uint8, device=DEV)[::2])


def test_more_tokens_than_32_bits():
    """Sizes that the argument structure cannot hold are refused, not cut."""
    x = torch.randn(1, 1, 64, device=DEV).to(torch.bfloat16)
    y = torch.zeros(1, 1, 64, device=DEV, dtype=torch.bfloat16)
    n = 2 ** 32 + 1
    with pytest.raises(ValueError):
        ac.rope_fwd(x.expand(n, 1, 64), None, ac.rope_table(64), out_q=y.expand(n, 1, 64))
    with pytest.raises(ValueError):
        ac.rope_fwd(x.expand(1, n, 64), None, ac.rope_table(64), out_q=y.expand(1, n, 64))
    p = Paged([1], [20], 2, 1, 64, 16)
    for kw in (dict(n_tokens=n), dict(h_q=2 ** 32 + 2), dict(n_pages=2 ** 32 + p.n_pages), dict(wait_timeout_ms=2 ** 32),
               dict(page_size=2 ** 32 + 16), dict(flags=2 ** 32)):
        with pytest.raises(ValueError):
            p.batch(**kw)
