"""Gathered attention weights against a plain 64-bit sum: masks, rows that see
nothing, fresh keys in place of old values, cut items, special values."""
import math

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


def gathered(p, lse, old, decay, out, causal=True):
    """(the weights in 64 bits over `out`'s other entries, what the call added)."""
    want, gain = out.double().clone(), torch.zeros_like(out, dtype=torch.float64)
    g = p.h_q // p.h_kv
    scale = 1.0 / math.sqrt(p.d)
    for i, (n, m) in enumerate(zip(p.nq, p.nk)):
        if n == 0:
            continue
        k = p.keys[i].double()
        for h in range(p.h_kv):
            total = torch.zeros(m, dtype=torch.float64, device=DEV)
            for t in range(0, n, 512):
                rows = slice(p.cu_host[i] + t, p.cu_host[i] + min(t + 512, n))
                q = p.q[rows, h * g:(h + 1) * g].double()
                x = torch.einsum("qgd,kd->gqk", q, k[:, h]) * scale
                z = lse[h * g:(h + 1) * g, rows].double()
                w = torch.exp(x - z[..., None])
                sees = (z != -math.inf)[..., None].expand(w.shape)
                if causal:
                    pos = m - n + t + torch.arange(q.shape[0], device=DEV)
                    sees = sees & (torch.arange(m, device=DEV)[None] <= pos[:, None])
                total += torch.where(sees, w, torch.zeros_like(w)).sum((0, 1))
            before = max(m - n, 0)
            gain[i, h, :m] = total
            want[i, h, :m] = total
            want[i, h, :before] += old[i, h, :before].double() * decay
    return want, gain


def check(got, want, gain):
    """A score of d <= 160 products is off by less than 2^-13 after the scale (see
    check_attention), its exponent's own roundings and ex2.approx by less, and all
    terms are positive: 2^-12 of what was added.  Sums of up to 128 terms in four
    chains, then one per tile, stay below 2^-17 of it for the tiles here; the old
    value's product and sum round once each (2^-24)."""
    assert torch.isfinite(got).all()
    tol = 2.0 ** -12 * gain + 2.0 ** -23 * want.abs() + 1e-37
    err = (got.double() - want).abs()
    assert (err <= tol).all(), float((err - tol).max())


def run(p, decay=1.0, seed=0, in_place=False, **kw):
    batch = p.batch(**kw)
    o, lse = ac.paged_fwd(batch, p.q, p.k_pages, p.v_pages)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    shape = (len(p.nq), p.h_kv, p.table.shape[1] * p.ps)
    old = torch.rand(shape, generator=gen, device=DEV) * 3
    for i, (n, m) in enumerate(zip(p.nq, p.nk)):
        old[i, :, max(m - n, 0):] = math.nan            # fresh keys' places hold anything
    out = old.clone() if in_place else torch.full(shape, 7.0, device=DEV)
    left = out.clone()
    got = ac.paged_weights(batch, p.q, lse, p.k_pages, out if in_place else old, decay=decay, out=None if in_place else out)
    assert got is out
    want, gain = gathered(p, lse, old, decay, left, causal=kw.get("causal", True))
    used = torch.zeros(shape, dtype=torch.bool, device=DEV)
    for i, (n, m) in enumerate(zip(p.nq, p.nk)):
        used[i, :, :m if n else 0] = True
    assert torch.equal(got[~used].view(torch.int32), left[~used].view(torch.int32))
    check(torch.where(used, got, torch.zeros_like(got)), torch.where(used, want, torch.zeros_like(want)), gain)
    return batch, lse, old, out


@pytest.mark.parametrize("d,ps", [(64, 16), (96, 32), (128, 64), (160, 128), (128, 256)])
@pytest.mark.parametrize("hq,hkv", [(8, 2), (3, 3), (6, 2), (16, 1)])
def test_single_tokens(hq, hkv, d, ps):
    p = Paged([1] * 9, [1, 2, 127, 128, 129, 255, 256, 257, 700], hq, hkv, d, ps, n_tokens=11)
    run(p)
    assert int(p.status.item()) == 0


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("hq,hkv,d,ps", [(4, 4, 160, 32), (8, 1, 128, 16), (12, 4, 96, 64), (5, 1, 64, 16), (128, 1, 64, 16)])
def test_chunks(hq, hkv, d, ps, causal):
    """Chunks of every length over shorter and longer contexts; rows that see no key
    (fewer keys than new tokens), no keys at all, sequences without new tokens."""
    nq = [3, 200, 1, 17, 64, 129, 0, 8, 50, 4, 128]
    nk = [3, 240, 1, 530, 64, 1300, 20, 259, 20, 0, 384]
    p = Paged(nq, nk, hq, hkv, d, ps, seed=1)
    run(p, decay=0.75, causal=causal, in_place=causal)
    assert int(p.status.item()) == 0


@pytest.mark.parametrize("hq,hkv,d,ps,nq", [(48, 1, 64, 16, 30), (56, 1, 128, 32, 40), (100, 1, 96, 64, 12), (48, 1, 128, 16, 300),
                                            (34, 2, 64, 16, 200), (6, 2, 128, 64, 1400), (33, 1, 160, 16, 90)])
def test_head_groups_that_leave_much_of_a_tile(hq, hkv, d, ps, nq):
    """Row tiles with rows that no token has, after scores of NaN in the same columns
    (what the tensor memory held before must not count)."""
    bad = Paged([nq], [nq + 300], hq, hkv, d, ps, seed=9)
    lse = torch.zeros(hq, nq, device=DEV)
    bad.q.fill_(math.nan)
    w = torch.zeros((1, hkv, bad.table.shape[1] * ps), device=DEV)
    ac.paged_weights(bad.batch(), bad.q, lse, bad.k_pages, w)
    full = Paged([128], [500], 1, 1, d, ps, seed=9)
    full.q.fill_(math.nan)
    for n in (128, 32):
        ac.paged_weights(full.batch(), full.q, torch.zeros(1, 128, device=DEV), full.k_pages,
                         torch.zeros((1, 1, full.table.shape[1] * ps), device=DEV))
    p = Paged([nq, 3], [nq + 300, 40], hq, hkv, d, ps, seed=9)
    run(p)
    assert int(p.status.item()) == 0


@pytest.mark.parametrize("hq,hkv,d,nq,nk", [(16, 2, 128, 1500, 2100), (8, 8, 96, 900, 900), (5, 1, 64, 1025, 5000),
                                            (4, 2, 160, 2000, 2300), (64, 1, 128, 70, 900), (1, 1, 64, 5000, 5000),
                                            (2, 1, 96, 1100, 400)])
def test_cut_items(hq, hkv, d, nq, nk):
    """Many row tiles over few keys: items are cut and their parts joined; the same
    bits again, on another stream, with anything in the workspace."""
    p = Paged([nq, 1], [nk, 300], hq, hkv, d, 64, seed=2)
    batch, lse, old, out = run(p, decay=0.5)
    batch.workspace.fill_(255)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = [ac.paged_weights(batch, p.q, lse, p.k_pages, old, decay=0.5, out=torch.full_like(old, 7.0)) for _ in range(2)]
    torch.cuda.synchronize()
    for x in again:
        assert torch.equal(x.view(torch.int32), out.view(torch.int32))
    assert int(p.status.item()) == 0


@pytest.mark.parametrize("hq,hkv,d,ps", [(8, 1, 128, 16), (6, 2, 96, 32), (32, 1, 64, 64), (3, 3, 160, 16)])
def test_one_chunk_among_single_tokens(hq, hkv, d, ps):
    """Batches of single tokens on average, which have row tiles of 32 rows, with one
    sequence of many such tiles, whose items are cut."""
    nq = [1] * 60 + [200] + [1] * 200
    nk = [1 + (37 * i) % 400 for i in range(261)]
    nk[60] = 700
    p = Paged(nq, nk, hq, hkv, d, ps, seed=8)
    run(p, decay=0.5, in_place=True)
    assert int(p.status.item()) == 0


def test_long_context():
    p = Paged([1, 1], [70000, 33000], 8, 1, 64, 128, seed=3)
    run(p)
    total = run(p, seed=1)[3]
    assert int(p.status.item()) == 0 and total.shape[-1] >= 70000


def test_weights_of_a_row_add_up():
    """What a row pays adds up to one: all keys of a head gain the number of rows."""
    p = Paged([40, 1], [300, 900], 6, 2, 128, 32, seed=4)
    batch = p.batch()
    o, lse = ac.paged_fwd(batch, p.q, p.k_pages, p.v_pages)
    w = ac.paged_weights(batch, p.q, lse, p.k_pages, torch.zeros(batch._weights_shape, device=DEV))
    for i, (n, m) in enumerate(zip(p.nq, p.nk)):
        # the rows' exponentials are those of the softmax up to 2^-12 of each (check)
        assert ((w[i, :, :m].double().sum(-1) - 3 * n).abs() <= 2.0 ** -11 * 3 * n).all()


def test_special_values():
    p = Paged([3, 1], [300, 140], 4, 2, 64, 16, seed=5)
    batch = p.batch()
    o, lse = ac.paged_fwd(batch, p.q, p.k_pages, p.v_pages)
    clean = ac.paged_weights(batch, p.q, lse, p.k_pages, torch.zeros(batch._weights_shape, device=DEV))
    # a NaN LSE reaches the keys that its row sees, and no others
    lse2 = lse.clone()
    lse2[0, 1] = math.nan                               # head 0, token 1 of sequence 0: sees 299 keys
    w = ac.paged_weights(batch, p.q, lse2, p.k_pages, torch.zeros_like(clean))
    assert torch.isnan(w[0, 0, :299]).all() and torch.equal(w[0, 0, 299], clean[0, 0, 299])
    assert torch.equal(w[0, 1], clean[0, 1]) and torch.equal(w[1], clean[1])
    # rows of LSE -inf add nothing, whatever their scores are
    lse2 = lse.clone()
    lse2[:, 3] = -math.inf
    q = p.q.clone()
    q[3] = math.nan
    w = ac.paged_weights(batch, q, lse2, p.k_pages, torch.zeros_like(clean))
    assert (w[1, :, :140] == 0).all() and torch.equal(w[0], clean[0])
    # an infinite LSE takes all of the row
    lse2[:, 3] = math.inf
    w = ac.paged_weights(batch, p.q, lse2, p.k_pages, torch.zeros_like(clean))
    assert (w[1, :, :140] == 0).all()
    # the next sequence's rows, which lie behind the last tile's, have no say
    q = p.q.clone()
    q[3] = math.inf
    w = ac.paged_weights(batch, q, lse, p.k_pages, torch.zeros_like(clean))
    assert torch.equal(w[0], clean[0])
    # a key that is NaN concerns itself alone
    p.k_pages[int(p.table[0, 2]), :, 5] = math.nan      # key 37 of sequence 0
    w = ac.paged_weights(batch, p.q, lse, p.k_pages, torch.zeros_like(clean))
    assert torch.isnan(w[0, :, 37]).all()
    w[0, :, 37] = clean[0, :, 37]
    assert torch.equal(w, clean)
    assert int(p.status.item()) == 0


def test_a_captured_graph_follows_the_tables():
    p = Paged([1, 40, 1], [300, 500, 64], 8, 2, 128, 16, seed=6, cols=40, n_tokens=42)
    batch = p.batch()
    w = torch.zeros(batch._weights_shape, device=DEV)
    lse = ac.paged_fwd(batch, p.q, p.k_pages, p.v_pages)[1]
    ac.paged_weights(batch, p.q, lse, p.k_pages, w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ac.paged_weights(batch, p.q, lse, p.k_pages, w, decay=0.5)
    for cu, nk in (([0, 1, 41, 42], [300, 500, 64]), ([0, 20, 20, 21], [100, 500, 1]), ([0, 0, 42, 42], [1, 45, 1])):
        p.cu.copy_(torch.tensor(cu, dtype=torch.int32))
        p.kv_lens.copy_(torch.tensor(nk, dtype=torch.int32))
        p.cu_host, p.nq = cu, [b - a for a, b in zip(cu, cu[1:])]
        full, p.nk = (p.keys, p.nk), nk
        p.keys = [k[:n] for k, n in zip(p.keys, nk)]
        lse.copy_(ac.paged_fwd(batch, p.q, p.k_pages, p.v_pages)[1])
        w.copy_(torch.rand(w.shape, device=DEV))
        before = w.clone()
        graph.replay()
        torch.cuda.synchronize()
        want, gain = gathered(p, lse, before, 0.5, before)
        check(w, want, gain)
        p.keys, p.nk = full
    assert int(p.status.item()) == 0


def test_bad_tables_are_reported():
    p = Paged([1, 1], [300, 100], 4, 2, 64, 16)
    batch = p.batch()
    lse = ac.paged_fwd(batch, p.q, p.k_pages, p.v_pages)[1]
    w = torch.zeros(batch._weights_shape, device=DEV)
    good = ac.paged_weights(batch, p.q, lse, p.k_pages, w, out=torch.zeros_like(w))
    p.table[0, 3] = p.n_pages
    out = ac.paged_weights(batch, p.q, lse, p.k_pages, w, out=torch.zeros_like(w))
    assert int(p.status.item()) == ac.ERR_DEVICE_TABLE and torch.equal(out[1], good[1])
    p.status.zero_()
    p.kv_lens[0] = 1 << 30
    out = ac.paged_weights(batch, p.q, lse, p.k_pages, w, out=torch.zeros_like(w))
    assert int(p.status.item()) == ac.ERR_DEVICE_TABLE
    assert torch.equal(out[1], good[1]) and (out[0] == 0).all()


def test_a_wait_that_runs_out_is_reported():
    p = Paged([1, 1], [300, 100], 4, 2, 64, 16)
    batch = p.batch(flags=ac.FLAG_TEST_WAIT_TIMEOUT, wait_timeout_ms=5)
    w = torch.zeros(batch._weights_shape, device=DEV)
    ac.paged_weights(batch, p.q, torch.zeros(4, 2, device=DEV), p.k_pages, w)
    torch.cuda.synchronize()
    assert int(p.status.item()) & 0xff == ac.ERR_DEVICE_TIMEOUT
