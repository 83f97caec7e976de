"""Eviction from the paged cache against a plain selection on the host: exact
choices with ties, infinities and NaN, rows moved within their pages and to others,
everything else left as it was."""
import math

import numpy as np
import pytest
import torch

import attention_core_gb300 as ac
from tests.serve_ref import Paged

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def choose(w, n, keep, first, recent):
    """The keys that stay, in order: w fp32 [n] on the host."""
    m = min(keep, n)
    r = min(recent, m)
    f = min(first, m - r)
    middle = np.arange(f, n - r)
    x = w[f:n - r].astype(np.float64)
    nan = np.isnan(x)
    best = middle[np.lexsort((middle, -np.where(nan, 0, x), nan))][: m - f - r]
    return np.concatenate([np.arange(f), np.sort(best), np.arange(n - r, n)]).astype(np.int64)


def bits(x):
    return x.view(torch.int16 if x.element_size() == 2 else torch.int32)


def check(p, batch, w, keep, first, recent, out_table=None, in_place=True):
    """One call against the definition, and again with a clean cache: the same bits."""
    k0, v0, w0 = p.k_pages.clone(), p.v_pages.clone(), w.clone()
    length = w.shape[-1]
    kept = torch.full(w.shape, -5, dtype=torch.int32, device=DEV)
    out = w if in_place else torch.full_like(w, 7.0)
    keep_dev = torch.tensor(keep, dtype=torch.int32, device=DEV)
    want_k, want_v, want_w, want_kept = k0.clone(), v0.clone(), out.clone(), kept.clone()
    host = w0.cpu().numpy()
    src_table = p.table.long()
    dst_table = src_table if out_table is None else out_table.long()
    for i, n in enumerate(p.nk):
        for h in range(p.h_kv):
            src = torch.from_numpy(choose(host[i, h, :n], n, keep[i], first, recent)).to(DEV)
            j = torch.arange(len(src), device=DEV)
            want_kept[i, h, :len(src)] = src.to(torch.int32)
            want_w[i, h, :len(src)] = w0[i, h, src]
            a, b = src_table[i][src // p.ps], dst_table[i][j // p.ps]
            want_k[b, h, j % p.ps] = k0[a, h, src % p.ps]
            want_v[b, h, j % p.ps] = v0[a, h, src % p.ps]
    got = ac.paged_evict(batch, w, keep_dev, p.k_pages, p.v_pages, first=first, recent=recent, out_table=out_table,
                         out_weights=None if in_place else out, kept=kept)
    assert got is kept and length == kept.shape[-1]
    assert torch.equal(kept, want_kept)
    assert torch.equal(bits(out), bits(want_w))
    assert torch.equal(bits(p.k_pages), bits(want_k)) and torch.equal(bits(p.v_pages), bits(want_v))
    if not in_place:
        assert torch.equal(bits(w), bits(w0))


def make(nk, h_kv, d, ps, seed=0, kind="spread", **kw):
    p = Paged([0] * len(nk), nk, h_kv, h_kv, d, ps, seed=seed, **kw)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    shape = (len(nk), h_kv, p.table.shape[1] * ps)
    w = torch.rand(shape, generator=gen, device=DEV)
    if kind == "ties":
        w = torch.floor(w * 4)
    elif kind == "same":
        w.fill_(0.25)
    elif kind == "special":
        w = torch.randn(shape, generator=gen, device=DEV)
        pick = torch.randint(0, 12, shape, generator=gen, device=DEV)
        for i, x in enumerate((math.nan, math.inf, -math.inf, 0.0, -0.0, -math.nan, 1e-42)):
            w[pick == i] = x
    return p, w


@pytest.mark.parametrize("kind", ["spread", "ties", "same", "special"])
@pytest.mark.parametrize("d,ps,hkv", [(64, 16, 3), (96, 32, 2), (128, 64, 1), (160, 128, 2), (128, 256, 2)])
def test_within_the_pages(d, ps, hkv, kind):
    nk = [1, 2, 63, 64, 65, 130, 700, 1500, 0, 999]
    p, w = make(nk, hkv, d, ps, kind=kind)
    batch = p.batch()
    check(p, batch, w, [1, 1, 40, 64, 64, 0, 300, 1499, 5, 64], 4, 20)
    assert int(p.status.item()) == 0


@pytest.mark.parametrize("first,recent", [(0, 0), (0, 1000), (1000, 0), (3, 128), (200, 200), (100, 250)])
def test_the_keys_that_always_stay(first, recent):
    """... count backwards from what stays: the recent ones before the first ones."""
    p, w = make([500, 310, 300, 299, 1], 2, 64, 16)
    check(p, p.batch(), w, [300] * 5, first, recent, in_place=False)


@pytest.mark.parametrize("kind", ["spread", "ties", "special"])
def test_long_lines(kind):
    """Lines that the blocks of a cluster share, of more and less than their shares."""
    p, w = make([100000, 33000, 5], 1, 64, 64, kind=kind)
    check(p, p.batch(), w, [25000, 32999, 3], 16, 1024)
    p, w = make([40000], 4, 128, 128, kind=kind, seed=1)
    check(p, p.batch(), w, [10000], 0, 0, in_place=False)
    assert int(p.status.item()) == 0


@pytest.mark.parametrize("nk,hkv", [([400000], 1), ([47000, 100, 46000], 40)])
@pytest.mark.parametrize("in_place", [True, False])
def test_lines_beyond_shared_memory(nk, hkv, in_place):
    p, w = make(nk, hkv, 64, 256, kind="ties")
    check(p, p.batch(), w, [n // 2 for n in nk], 5, 300, in_place=in_place)
    assert int(p.status.item()) == 0


@pytest.mark.parametrize("shared", [0, 1, 3, 100])
def test_to_other_pages(shared):
    """The first `shared` pages of each sequence move to fresh ones, the others stay
    (what a pool does where forks share pages); then all of them."""
    nk, keep = [1000, 400, 90], [500, 390, 90]
    p, w = make(nk, 2, 128, 16, spare=100)
    fresh = [x for x in range(p.n_pages) if x not in set(p.host_table[p.host_table >= 0].tolist())]
    out = p.host_table.copy()
    for i, m in enumerate(keep):
        for c in range(min(shared, -(-m // 16))):
            out[i, c] = fresh.pop()
    check(p, p.batch(), w, keep, 4, 50, out_table=torch.from_numpy(out).to(DEV))
    assert int(p.status.item()) == 0


def test_two_sequences_leave_their_common_pages():
    """A fork and its parent, both evicted: each reads the common pages and writes its
    own."""
    p, w = make([640, 640], 2, 64, 32, spare=60)
    p.host_table[1, :20] = p.host_table[0, :20]
    p.table.copy_(torch.from_numpy(p.host_table))
    used = set(p.host_table[p.host_table >= 0].tolist())
    fresh = [x for x in range(p.n_pages) if x not in used]
    out = p.host_table.copy()
    out[0, :10], out[1, :10] = fresh[:10], fresh[10:20]
    check(p, p.batch(), w, [320, 300], 0, 64, out_table=torch.from_numpy(out).to(DEV))


def test_repeated_and_captured():
    """Step by step in a captured graph whose lengths and budgets change, as a long
    answer is bounded."""
    p, w = make([2000, 1100], 2, 128, 64)
    batch = p.batch()
    keep = torch.tensor([1500, 1100], dtype=torch.int32, device=DEV)
    kept = torch.zeros(w.shape, dtype=torch.int32, device=DEV)
    graph = torch.cuda.CUDAGraph()
    k0, v0, w0 = p.k_pages.clone(), p.v_pages.clone(), w.clone()
    ac.paged_evict(batch, w, keep, p.k_pages, p.v_pages, first=2, recent=100, kept=kept)
    torch.cuda.synchronize()
    for a, b in ((p.k_pages, k0), (p.v_pages, v0), (w, w0)):
        a.copy_(b)
    with torch.cuda.graph(graph):
        ac.paged_evict(batch, w, keep, p.k_pages, p.v_pages, first=2, recent=100, kept=kept)
    for want in ([1500, 1100], [700, 1000], [700, 64], [3, 1], [0, 1]):
        host = w.cpu().numpy()
        keep.copy_(torch.tensor(want, dtype=torch.int32))
        k0, v0, w0 = p.k_pages.clone(), p.v_pages.clone(), w.clone()
        graph.replay()
        torch.cuda.synchronize()
        for i, n in enumerate(p.nk):
            for h in range(2):
                src = torch.from_numpy(choose(host[i, h, :n], n, want[i], 2, 100)).to(DEV)
                j = torch.arange(len(src), device=DEV)
                assert torch.equal(kept[i, h, :len(src)].long(), src)
                assert torch.equal(w[i, h, :len(src)], w0[i, h, src])
                t = p.table[i].long()
                assert torch.equal(bits(p.k_pages[t[j // 64], h, j % 64]), bits(k0[t[src // 64], h, src % 64]))
                assert torch.equal(bits(p.v_pages[t[j // 64], h, j % 64]), bits(v0[t[src // 64], h, src % 64]))
        p.nk = [min(a, b) for a, b in zip(want, p.nk)]
        p.kv_lens.copy_(torch.tensor(p.nk, dtype=torch.int32))
    assert int(p.status.item()) == 0


def test_bad_tables_are_reported():
    p, w = make([300, 100, 200], 2, 64, 16)
    batch = p.batch()
    k0 = p.k_pages.clone()
    for change in ("keep", "length", "page"):
        keep = torch.tensor([100, 50, 60], dtype=torch.int32, device=DEV)
        p.kv_lens.copy_(torch.tensor(p.nk, dtype=torch.int32))
        p.table.copy_(torch.from_numpy(p.host_table))
        if change == "keep":
            keep[0] = -1
        elif change == "length":
            p.kv_lens[0] = 1 << 30
        else:
            p.table[0] = p.n_pages
        p.k_pages.copy_(k0)
        p.status.zero_()
        kept = ac.paged_evict(batch, w, keep, p.k_pages, p.v_pages, out_weights=torch.empty_like(w))
        assert int(p.status.item()) == ac.ERR_DEVICE_TABLE, change
        for i in (1, 2):
            for h in range(2):
                want = choose(w[i, h].cpu().numpy()[:p.nk[i]], p.nk[i], int(keep[i]), 0, 0)
                assert kept[i, h, :len(want)].tolist() == want.tolist()


def test_a_wait_that_runs_out_is_reported():
    """... and nothing is written over rows that may still be wanted."""
    p, w = make([3000], 2, 64, 16)
    k0 = p.k_pages.clone()
    batch = p.batch(flags=ac.FLAG_TEST_WAIT_TIMEOUT, wait_timeout_ms=5)
    ac.paged_evict(batch, w, torch.tensor([1000], dtype=torch.int32, device=DEV), p.k_pages, p.v_pages)
    torch.cuda.synchronize()
    assert int(p.status.item()) & 0xff == ac.ERR_DEVICE_TIMEOUT
    assert torch.equal(bits(p.k_pages), bits(k0))


def test_empty_rows_of_the_batch():
    p, w = make([0, 0], 2, 64, 16, cols=2)
    check(p, p.batch(), w, [5, 0], 1, 1)
    assert int(p.status.item()) == 0
