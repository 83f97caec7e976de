"""The paged key/value cache on the GPU: appending new tokens and attending
over the cache, against 64-bit definitions; pages past a sequence's end hold
NaN throughout."""
import math

import pytest
import torch

import attention_core_gb300 as ac
from tests.serve_ref import BF16, ORIGINAL, Paged, attend, check_attention, rope_tolerance, rotate

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def _run(p, **kw):
    o, lse = ac.paged_fwd(p.batch(**kw), p.q, p.k_pages, p.v_pages)
    torch.cuda.synchronize()
    assert int(p.status.item()) == 0
    return o, lse


# (new tokens, keys, h_q, h_kv, d, page_size, causal)
CASES = [
    ([1], [1], 1, 1, 64, 16, True),
    ([1], [500], 8, 1, 128, 16, True),
    ([1], [127], 2, 2, 96, 16, True),
    ([1], [128], 2, 2, 160, 32, True),
    ([1], [129], 4, 1, 160, 64, True),
    ([1] * 7, [1, 64, 65, 333, 16, 17, 1024], 8, 2, 128, 32, True),
    ([1] * 5, [5000, 3, 700, 0, 4097], 8, 2, 64, 64, True),           # one sequence has no keys
    ([4, 0, 1, 9], [4, 0, 300, 260], 6, 2, 128, 128, True),            # an empty sequence; 3 heads share a KV head
    ([130], [130], 2, 1, 64, 16, True),                               # a prompt from its start
    ([300, 5, 1], [300, 700, 40], 4, 4, 96, 64, True),
    ([200], [1200], 16, 2, 128, 256, True),
    ([257, 64], [257, 2000], 5, 1, 128, 32, True),                     # 5 heads: tiles of 125 rows
    ([40, 3], [10, 1], 4, 2, 64, 16, True),                            # more new tokens than keys: rows that see nothing
    ([140], [3], 1, 1, 160, 16, True),
    ([65, 1, 30], [200, 128, 1], 8, 4, 128, 64, False),
    ([3, 2], [0, 100], 2, 2, 160, 16, False),
    ([3], [200], 128, 1, 64, 16, True),                                # 128 heads share one KV head
    ([17], [400], 100, 1, 96, 32, True),
    ([500, 1, 77], [900, 4001, 77], 16, 16, 160, 32, True),
    ([700], [3000], 8, 1, 128, 16, True),
]


def _id(c):
    return "q{}_k{}_h{}-{}_d{}_p{}_{}".format("-".join(map(str, c[0])), "-".join(map(str, c[1])), *c[2:6],
                                              "c" if c[6] else "n")


@pytest.mark.parametrize("case", CASES, ids=_id)
def test_attention_matches_definition(case):
    nq, nk, hq, hkv, d, ps, causal = case
    p = Paged(nq, nk, hq, hkv, d, ps, seed=len(nq) + d)
    o, lse = _run(p, causal=causal)
    check_attention(o, lse, attend(p, causal), p)


def _with_rounded_probabilities(p):
    """O in 64 bits but for the probabilities, rounded to bf16 relative to their row's largest."""
    o = torch.zeros(p.q.shape, dtype=torch.float64, device=p.q.device)
    for i, m in enumerate(p.nk):
        rows = slice(p.cu_host[i], p.cu_host[i + 1])
        k, v = (x[i].double().repeat_interleave(p.h_q // p.h_kv, 1) for x in (p.keys, p.values))
        x = torch.einsum("qhd,khd->hqk", p.q[rows].double(), k) / math.sqrt(p.d)
        w = torch.exp(x - x.amax(-1, keepdim=True))
        o[rows] = torch.einsum("hqk,khd->qhd", w.to(torch.bfloat16).double(), v) / w.sum(-1).t()[..., None]
    return o


@pytest.mark.parametrize("d,hq,hkv", [(64, 32, 1), (96, 6, 2), (128, 8, 1), (160, 4, 4)])
def test_single_tokens_round_only_the_result(d, hq, hkv):
    """Batches of single tokens: the probabilities keep two bf16 terms, so what the
    second rounding leaves is 2^-16 of each (2^-15 here, a probability's fp32
    exponential included) and only O's own rounding remains.  Few keys, so that
    rounded probabilities' errors do not average out; those would be seen."""
    nk = [3 + i % 9 for i in range(40)]
    p = Paged([1] * len(nk), nk, hq, hkv, d, 16, seed=d)
    ro, _, size = attend(p)
    tol = BF16 * ro.abs() + (2.0 ** -12 + 2.0 ** -15) * size
    assert ((_with_rounded_probabilities(p) - ro).abs() > 2 * tol).any()
    o, _ = _run(p)
    err = (o.double() - ro).abs()
    assert (err <= tol).all(), float((err - tol).max())


@pytest.mark.parametrize("d,hkv", [(64, 2), (96, 1), (128, 8), (160, 2)])
def test_prompts_among_single_tokens(d, hkv):
    """Few rows a sequence on average, but whole tiles of prompts among them: both
    kinds follow one another in a block.  The single tokens' rows round only the
    result, a hundred runs agree in every bit."""
    nq = [1] * 40 + [200] + [1] * 30 + [33]
    nk = [3 + i % 9 for i in range(40)] + [700] + [129 + 40 * i for i in range(30)] + [33]
    p = Paged(nq, nk, 4 * hkv, hkv, d, 32, seed=d + 1)
    assert sum(nq) * 4 <= 32 * len(nq)
    o, lse = _run(p)
    want = attend(p)
    check_attention(o, lse, want, p)
    ro, size = want[0][:40], want[2][:40]
    assert ((o[:40].double() - ro).abs() <= BF16 * ro.abs() + (2.0 ** -12 + 2.0 ** -15) * size).all()
    for _ in range(100):
        again, lse_again = _run(p)
        assert torch.equal(again, o) and torch.equal(lse_again, lse)


@pytest.mark.parametrize("d", [64, 96, 128, 160])
def test_every_length_around_the_block_borders(d):
    """Sequences of 1..3 new tokens and lengths around multiples of the page and
    of 128 keys, all in one batch."""
    nk = [n + e for n in (16, 112, 128, 256, 384) for e in (-2, -1, 0, 1, 2)]
    nq = [1 + i % 3 for i in range(len(nk))]
    p = Paged(nq, nk, 4, 2, d, 16, seed=d)
    o, lse = _run(p)
    check_attention(o, lse, attend(p), p)


@pytest.mark.parametrize("d,hq,hkv", [(128, 8, 1), (64, 2, 2), (160, 4, 2), (96, 1, 1)])
def test_long_context_is_shared_out(d, hq, hkv):
    """A context of tens of thousands of keys beside short ones: its keys are
    split over many blocks and the parts joined."""
    p = Paged([1, 2, 1], [30011, 50, 129], hq, hkv, d, 64, seed=9)
    o, lse = _run(p)
    check_attention(o, lse, attend(p), p)


def test_more_sequences_than_threads():
    """A thousand single tokens: every thread of a block looks after several
    sequences when it finds its share."""
    nk = [1 + (37 * i) % 300 for i in range(1000)]
    nq = [0 if i % 11 == 0 else 1 for i in range(1000)]
    p = Paged(nq, nk, 2, 1, 64, 16, seed=15)
    o, lse = _run(p)
    check_attention(o, lse, attend(p), p)


# batches whose tiles are handed out whole: at least 1.4 per CTA, several per KV head
HANDED_OUT = [
    ([500] * 5, [700, 2500, 500, 1300, 512], 16, 16, 160, 32, True),
    ([300, 1, 0, 450, 64, 200, 129], [300, 9, 40, 0, 1000, 150, 4000], 24, 24, 64, 16, True),   # no keys; fewer keys than tokens
    ([130 + 3 * i for i in range(40)], [200 + 31 * i for i in range(40)], 4, 4, 96, 64, True),   # more than 32 sequences
    ([700, 900], [4000, 900], 32, 4, 128, 128, False),
    ([100, 90, 77, 128], [3000, 90, 2000, 128], 128, 16, 128, 64, True),
]


@pytest.mark.parametrize("case", HANDED_OUT, ids=lambda c: f"n{len(c[0])}_h{c[2]}-{c[3]}_d{c[4]}")
def test_whole_tiles_handed_out(case):
    nq, nk, hq, hkv, d, ps, causal = case
    p = Paged(nq, nk, hq, hkv, d, ps, seed=16, n_tokens=sum(nq) + 9)
    tiles = sum(-(-n // (128 // (hq // hkv))) for n in nq) * hkv
    assert tiles >= 1.4 * 152
    o, lse = torch.full_like(p.q, 7.0), torch.full((hq, p.n_tokens), 7.0, device=DEV)
    b = p.batch(causal=causal)
    for _ in range(3):
        b.workspace.fill_(0xFF)
        ac.paged_fwd(b, p.q, p.k_pages, p.v_pages, out=o, lse=lse)
    torch.cuda.synchronize()
    assert int(p.status.item()) == 0
    check_attention(o, lse, attend(p, causal), p)
    assert (o[sum(nq):] == 7).all() and (lse[:, sum(nq):] == 7).all()
    # one bad sequence: reported, the others' rows unchanged
    good = o.clone()
    p.kv_lens[0] = -1
    ac.paged_fwd(b, p.q, p.k_pages, p.v_pages, out=o, lse=lse)
    torch.cuda.synchronize()
    assert int(p.status.item()) & 0xff == ac.ERR_DEVICE_TABLE
    rest = slice(nq[0], sum(nq))
    assert ((o[rest].double() - good[rest].double()).abs() <= 2.0 ** -7 * (1 + good[rest].double().abs())).all()


def test_graph_moves_between_the_splits():
    """A captured call whose lengths change: tiles handed out whole at one replay,
    equal shares of cut tiles at the next."""
    n = [500] * 6
    p = Paged(n, [2000] * 6, 16, 16, 64, 64, seed=17)
    b = p.batch()
    o, lse = torch.empty_like(p.q), torch.empty(16, p.n_tokens, device=DEV)
    ac.paged_fwd(b, p.q, p.k_pages, p.v_pages, out=o, lse=lse)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ac.paged_fwd(b, p.q, p.k_pages, p.v_pages, out=o, lse=lse)
    for lens in ([500] * 6, [100, 3, 2, 1, 0, 50], [1, 1, 1, 1, 1, 500], [500, 500, 0, 0, 500, 500]):
        cu = [0]
        for x in lens:
            cu.append(cu[-1] + x)
        p.cu.copy_(torch.tensor(cu, dtype=torch.int32, device=DEV))
        for _ in range(2):
            g.replay()
        torch.cuda.synchronize()
        sub = Paged.__new__(Paged)
        sub.__dict__.update(p.__dict__)
        sub.nq, sub.cu_host = lens, cu
        check_attention(o, lse, attend(sub), sub)
        assert int(p.status.item()) == 0


def test_chunk_over_long_context():
    p = Paged([33, 128], [9000, 20000], 8, 2, 128, 128, seed=4)
    o, lse = _run(p)
    check_attention(o, lse, attend(p), p)


def test_scores_that_grow_and_fall_along_the_keys():
    """The running maximum moves late, or never after the first block: keys
    scaled up and down along the context."""
    p = Paged([2, 130], [700, 900], 4, 2, 128, 32, seed=5)
    for i in range(2):
        n = p.nk[i]
        ramp = torch.linspace(0.1, 6.0, n, device=DEV) if i == 0 else torch.linspace(6.0, 0.1, n, device=DEV)
        p.keys[i] = (p.keys[i].float() * ramp[:, None, None]).to(torch.bfloat16)
        page, row = p.places(i, torch.arange(n, device=DEV))
        p.k_pages[page, :, row] = p.keys[i]
    # scores are up to 6 times larger than with normal inputs, so their fp32 error
    # is too: 2^-13 * 6 < 2^-10 against the 2^-12 of check_attention
    o, lse = _run(p)
    ro, rlse, size = attend(p)
    tol = 2.0 ** -8 * (ro.abs() + size) + 2.0 ** -9 * size
    assert ((o.double() - ro).abs() <= tol).all()
    assert ((lse.double() - rlse).abs() <= 2.0 ** -10).all()


def test_scale_is_taken():
    p = Paged([5], [77], 2, 1, 64, 16, seed=6)
    o, lse = _run(p, scale=0.02)
    check_attention(o, lse, attend(p, scale=float(torch.tensor(0.02).float())), p)


def test_rows_behind_the_last_sequence_stay():
    p = Paged([3, 140], [50, 300], 4, 2, 128, 16, seed=7, n_tokens=200)
    o = torch.full_like(p.q, 7.0)
    lse = torch.full((4, 200), 7.0, device=DEV)
    ac.paged_fwd(p.batch(), p.q, p.k_pages, p.v_pages, out=o, lse=lse)
    torch.cuda.synchronize()
    assert (o[143:] == 7).all() and (lse[:, 143:] == 7).all()
    check_attention(o, lse, attend(p), p)
    qo = torch.full_like(p.q, 5.0)
    ac.paged_append(p.batch(), p.q, p.k_new, p.v_new, p.k_pages, p.v_pages, out_q=qo)
    torch.cuda.synchronize()
    assert (qo[143:] == 5).all() and torch.equal(qo[:143], p.q[:143])
    assert int(p.status.item()) == 0


def test_no_tokens():
    p = Paged([0, 0], [5, 0], 2, 1, 64, 16)
    o, lse = _run(p)
    assert o.shape == (0, 2, 64) and lse.shape == (2, 0)
    ac.paged_append(p.batch(), p.q, p.k_new, p.v_new, p.k_pages, p.v_pages)


def test_same_inputs_same_bits():
    p = Paged([1, 60], [9000, 5000], 8, 1, 128, 64, seed=8)
    b = p.batch()
    first = ac.paged_fwd(b, p.q, p.k_pages, p.v_pages)
    for _ in range(3):
        again = ac.paged_fwd(b, p.q, p.k_pages, p.v_pages)
        assert all(torch.equal(x, y) for x, y in zip(first, again))


@pytest.mark.parametrize("d,hq,hkv,ps", [(128, 8, 8, 64), (128, 16, 2, 64), (160, 16, 4, 16), (64, 4, 4, 32)])
def test_a_hundred_runs_agree(d, hq, hkv, ps):
    """Memory-bound batches whose tiles are cut, over and over without a pause and
    with a workspace that starts as NaN each time: the first result is the
    definition's and every other one is the same bits."""
    nk = [300 + (977 * i) % 3700 for i in range(24)]
    p = Paged([1 + (5 * i) % 40 for i in range(24)], nk, hq, hkv, d, ps, seed=d + hq)
    b = p.batch()
    o, lse = _run(p)
    check_attention(o, lse, attend(p), p)
    differ = torch.zeros(1, dtype=torch.int64, device=DEV)
    for _ in range(100):
        b.workspace.fill_(0xFF)
        o2, lse2 = ac.paged_fwd(b, p.q, p.k_pages, p.v_pages)
        differ += (o2 != o).any() | (lse2 != lse).any()
    assert int(differ.item()) == 0


def test_large_offsets():
    """Pages whose elements lie past 2^31 (and bytes past 2^32) of the cache."""
    d, ps, hkv = 128, 128, 8
    n_pages = (1 << 31) // (hkv * ps * d) + 40
    p = Paged([1, 70], [300, 1000], 16, hkv, d, ps, seed=10)
    shift = n_pages - p.n_pages
    k_big = torch.full((n_pages, hkv, ps, d), math.nan, dtype=torch.bfloat16, device=DEV)
    v_big = k_big.clone()
    k_big[shift:], v_big[shift:] = p.k_pages, p.v_pages
    p.table += shift
    b = p.batch(n_pages=n_pages)
    o, lse = ac.paged_fwd(b, p.q, k_big, v_big)
    torch.cuda.synchronize()
    assert int(p.status.item()) == 0
    check_attention(o, lse, attend(p), p)
    ac.paged_append(b, p.q, p.k_new, p.v_new, k_big, v_big)
    torch.cuda.synchronize()
    page, row = p.places(1, torch.arange(930, 1000, device=DEV))
    assert torch.equal(k_big[page, :, row], p.k_new[1:]) and torch.equal(v_big[page, :, row], p.v_new[1:])


# (new tokens, keys, h_q, h_kv, d, page_size, rot, interleaved, scaling, factor)
APPENDS = [
    ([1], [1], 2, 1, 64, 16, 64, False, "none", 1.0),
    ([1] * 9, [5, 16, 17, 100, 1, 33, 32, 4096, 900], 8, 2, 128, 16, 128, False, "bands", 8.0),
    ([30, 0, 7], [30, 0, 500], 6, 3, 96, 64, 24, False, "linear", 2.0),
    ([300, 1, 2, 150], [1000, 77, 2, 150], 4, 4, 160, 128, 80, True, "yarn", 4.0),
    ([3000], [3100], 8, 8, 96, 32, 96, False, "none", 1.0),
    ([5], [9], 3, 1, 128, 256, 0, False, "none", 1.0),                 # no rotation
]


@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("case", APPENDS, ids=lambda c: f"q{len(c[0])}-{sum(c[0])}_d{c[4]}_p{c[5]}_r{c[6]}")
def test_append_matches_definition(case, fused):
    nq, nk, hq, hkv, d, ps, rot, inter, scaling, factor = case
    p = Paged(nq, nk, hq, hkv, d, ps, seed=sum(nq))
    t = ac.rope_table(d, rot_dim=rot, interleaved=inter, scaling=scaling, factor=factor, original_len=ORIGINAL) if rot else None
    if fused:                                        # slices of one projection
        qkv = torch.cat((p.q, p.k_new, p.v_new), 1)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    else:
        q, k, v = p.q, p.k_new, p.v_new
    p.v_new[0, 0, 0] = math.inf                      # a value that no rotation may touch
    if fused:
        v[0, 0, 0] = math.inf
    k0, v0 = p.k_pages.clone(), p.v_pages.clone()
    got = ac.paged_append(p.batch(), q, k, v, p.k_pages, p.v_pages, table=t)
    torch.cuda.synchronize()
    assert int(p.status.item()) == 0
    for i, (n, m) in enumerate(zip(nq, nk)):
        rows = slice(p.cu_host[i], p.cu_host[i] + n)
        pos = torch.arange(m - n, m, device=DEV)
        page, row = p.places(i, pos)
        for x, y in ((p.q[rows], got[rows]), (p.k_new[rows], p.k_pages[page, :, row])):
            if not rot:
                assert torch.equal(x, y)
                continue
            want, size = rotate(x, pos[:, None], rot, interleaved=inter, scaling=scaling, factor=factor)
            assert ((y.double() - want).abs() <= rope_tolerance(want, size, rot)).all()
        assert torch.equal(p.v_pages[page, :, row], p.v_new[rows])
        k0[page, :, row], v0[page, :, row] = p.k_pages[page, :, row], p.v_pages[page, :, row]
    # nothing else moved (NaN where no key lies, so bits are compared)
    assert torch.equal(k0.view(torch.int16), p.k_pages.view(torch.int16))
    assert torch.equal(v0.view(torch.int16), p.v_pages.view(torch.int16))


def test_append_without_q_and_in_place():
    p = Paged([4, 1], [20, 7], 4, 2, 64, 16, seed=1)
    t = ac.rope_table(64)
    want = ac.paged_append(p.batch(), p.q, p.k_new, p.v_new, p.k_pages, p.v_pages, table=t)
    k1 = p.k_pages.clone()
    p.k_pages.fill_(math.nan)
    assert ac.paged_append(p.batch(), None, p.k_new, p.v_new, p.k_pages, p.v_pages, table=t) is None
    page, row = p.places(0, torch.arange(16, 20, device=DEV))
    assert torch.equal(p.k_pages[page, :, row], k1[page, :, row])
    q = p.q.clone()
    ac.paged_append(p.batch(), q, p.k_new, p.v_new, p.k_pages, p.v_pages, table=t, out_q=q)
    assert torch.equal(q, want)


def _bad(p, what):
    if what == "page":
        p.table[0, 0] = p.n_pages
    elif what == "negative page":
        p.table[0, 0] = -1
    elif what == "too many keys":
        p.kv_lens[0] = p.table.shape[1] * p.ps + 1
    elif what == "negative keys":
        p.kv_lens[0] = -5
    elif what == "decreasing":
        p.cu[1] = -3
    elif what == "past the tokens":
        p.cu[2] = p.n_tokens + 50


@pytest.mark.parametrize("what", ["page", "negative page", "too many keys", "negative keys", "decreasing", "past the tokens"])
def test_bad_tables_are_reported(what):
    """Entries out of range: the status word says so, the other sequences'
    results and everything outside the tensors stay right."""
    p = Paged([2, 3], [40, 60], 4, 2, 64, 16, seed=2)
    want = attend(p)
    _bad(p, what)
    o, lse = ac.paged_fwd(p.batch(), p.q, p.k_pages, p.v_pages)
    torch.cuda.synchronize()
    assert int(p.status.item()) & 0xff == ac.ERR_DEVICE_TABLE
    if what in ("page", "negative page", "too many keys", "negative keys"):
        used = slice(2, 5)
        assert ((o[used].double() - want[0][used]).abs() <= 2.0 ** -6).all()
    if what in ("page", "negative page", "negative keys"):
        p.status.zero_()
        if what != "negative keys":                  # the first page is the first two tokens' only in a short sequence
            p.kv_lens[0] = 2
        ac.paged_append(p.batch(), p.q, p.k_new, p.v_new, p.k_pages, p.v_pages)
        torch.cuda.synchronize()
        assert int(p.status.item()) & 0xff == ac.ERR_DEVICE_TABLE


def test_captured_graph_follows_the_tables():
    """One capture, replayed as the sequences grow: append and attention follow
    the lengths and pages in the tables."""
    d, ps, hq, hkv = 128, 16, 8, 2
    p = Paged([1, 1], [400, 90], hq, hkv, d, ps, seed=3)
    t = ac.rope_table(d)
    b = p.batch()
    full = p.kv_lens.clone()
    o, lse, qo = torch.empty_like(p.q), torch.empty(hq, 2, device=DEV), torch.empty_like(p.q)

    def step():
        ac.paged_append(b, p.q, p.k_new, p.v_new, p.k_pages, p.v_pages, table=t, out_q=qo)
        ac.paged_fwd(b, qo, p.k_pages, p.v_pages, out=o, lse=lse)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    gen = torch.Generator(device=DEV).manual_seed(11)
    for lens in ([5, 90], [130, 1], [400, 33]):
        p.kv_lens.copy_(torch.tensor(lens, dtype=torch.int32, device=DEV))
        for x in (p.q, p.k_new, p.v_new):
            x.copy_(torch.randn(x.shape, generator=gen, device=DEV))
        g.replay()
        torch.cuda.synchronize()
        assert int(p.status.item()) == 0
        sub = Paged.__new__(Paged)
        sub.__dict__.update(p.__dict__)
        sub.nk, sub.q = lens, qo
        sub.keys, sub.values = [], []
        for i, n in enumerate(lens):
            page, row = p.places(i, torch.arange(n, device=DEV))
            sub.keys.append(p.k_pages[page, :, row])
            sub.values.append(p.v_pages[page, :, row])
        check_attention(o, lse, attend(sub), sub)
    p.kv_lens.copy_(full)


def test_wait_that_runs_out_is_reported():
    """The test hook: every thread waits on a barrier that nothing completes,
    gives up after the limit and leaves; the next call is sound."""
    p = Paged([1, 3], [500, 40], 4, 2, 128, 16, seed=13)
    ac.paged_fwd(p.batch(flags=ac.FLAG_TEST_WAIT_TIMEOUT, wait_timeout_ms=20), p.q, p.k_pages, p.v_pages)
    torch.cuda.synchronize()
    assert int(p.status.item()) & 0xff == ac.ERR_DEVICE_TIMEOUT
    p.status.zero_()
    o, lse = _run(p)
    check_attention(o, lse, attend(p), p)


def test_captured_graphs_with_cut_tiles():
    """Two graphs, each with a batch of its own, replayed on two streams at once
    while their contexts change length: the tiles are cut elsewhere each time."""
    ps = [Paged([1, 3], [9000, 700], 8, 2, 128, 64, seed=s) for s in (30, 31)]
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in ps]
    for p in ps:
        b, o, lse = p.batch(), torch.empty_like(p.q), torch.empty(8, 4, device=DEV)
        ac.paged_fwd(b, p.q, p.k_pages, p.v_pages, out=o, lse=lse)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ac.paged_fwd(b, p.q, p.k_pages, p.v_pages, out=o, lse=lse)
        graphs.append((g, b))
        outs.append((o, lse))
    for lens in ([9000, 700], [4000, 3], [8191, 650]):
        for p in ps:
            p.kv_lens.copy_(torch.tensor(lens, dtype=torch.int32, device=DEV))
        torch.cuda.synchronize()
        for _ in range(3):
            for (g, _), s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        for p, (o, lse) in zip(ps, outs):
            sub = Paged.__new__(Paged)
            sub.__dict__.update(p.__dict__)
            sub.nk = lens
            sub.keys = [k[:n] for k, n in zip(p.keys, lens)]
            sub.values = [v[:n] for v, n in zip(p.values, lens)]
            check_attention(o, lse, attend(sub), sub)
            assert int(p.status.item()) == 0


def test_two_streams_with_a_batch_each():
    ps = [Paged([1, 40], [6000, 300], 8, 2, 128, 64, seed=s) for s in (20, 21)]
    streams = [torch.cuda.Stream() for _ in ps]
    batches = [p.batch() for p in ps]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(4):
        for i, (p, s) in enumerate(zip(ps, streams)):
            with torch.cuda.stream(s):
                outs[i].append(ac.paged_fwd(batches[i], p.q, p.k_pages, p.v_pages))
    torch.cuda.synchronize()
    for i, p in enumerate(ps):
        want = attend(p)
        for o, lse in outs[i]:
            check_attention(o, lse, want, p)


def test_prompt_equals_the_cores_forward():
    """A prompt from its start, its keys in pages, against the core's packed
    forward: the same function, so within the roundings of both."""
    n, hq, hkv, d = 300, 4, 2, 128
    p = Paged([n], [n], hq, hkv, d, 64, seed=12)
    o, lse = _run(p)
    o2, lse2 = ac.fwd_varlen(p.q, p.keys[0], p.values[0], [0, n])
    size = attend(p)[2]
    assert ((o.double() - o2.double()).abs() <= 2.0 ** -6 * size + 2.0 ** -11 * size).all()
    assert ((lse - lse2).abs() <= 2.0 ** -11).all()


def test_python_refusals():
    p = Paged([1], [20], 2, 1, 64, 16)
    b = p.batch()
    with pytest.raises(ValueError):
        ac.paged_fwd(b, p.q.float(), p.k_pages, p.v_pages)
    with pytest.raises(ValueError):
        ac.paged_fwd(b, p.q, p.k_pages[:1], p.v_pages)
    with pytest.raises(ValueError):
        ac.paged_fwd(b, p.q, p.k_pages, p.v_pages.cpu())
    with pytest.raises(ValueError):
        ac.paged_append(b, p.q, p.q, p.v_new, p.k_pages, p.v_pages)
    with pytest.raises(ValueError):
        ac.paged_append(b, None, p.k_new, p.v_new, p.k_pages, p.v_pages, out_q=p.q)
    with pytest.raises(ac.AttnCoreError):
        ac.paged_append(b, p.q, p.k_new, p.v_new, p.k_pages, p.v_pages, table=ac.rope_table(128))
    with pytest.raises(ac.AttnCoreError) as e:
        p.batch(page_size=24)
    assert e.value.code == ac.ERR_UNSUPPORTED
    with pytest.raises(ac.AttnCoreError):
        p.batch(h_q=3, h_kv=2)
    with pytest.raises(ValueError):
        p.batch(workspace=torch.empty(64, dtype=torch.uint8))
    with pytest.raises(ac.AttnCoreError):
        ac.paged_fwd(b, p.q, p.k_pages, p.v_pages, out=p.q)
    small = p.batch(workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
    if ac.attn_core_paged_workspace_bytes(b.params) > 64:
        with pytest.raises(ac.AttnCoreError) as e:
            ac.paged_fwd(small, p.q, p.k_pages, p.v_pages)
        assert e.value.code == ac.ERR_WORKSPACE_TOO_SMALL
