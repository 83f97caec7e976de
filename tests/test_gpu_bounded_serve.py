"""Many continuations of a prompt in a bounded cache, with the operators as they are
used together: a prompt, its forks, steps of attention over the shared pages, the
weights that the keys gather, and the eviction that bounds each sequence, on two
layers, every step's outputs against a plain 64-bit attention over the keys that each
head still has."""
import math

import numpy as np
import pytest
import torch

import attention_core_gb300 as ac
from attention_core_gb300.pagepool import PagePool
from tests.serve_ref import BF16, rope_tolerance, rotate
from tests.test_gpu_evict import choose

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("hq,hkv,d,ps", [(8, 2, 128, 16), (4, 4, 96, 32), (6, 2, 160, 64)])
def test_bounded_answers(hq, hkv, d, ps):
    layers, max_pages, g = 2, 512 // ps, hq // hkv
    pool = PagePool(2400 // ps, ps)
    pages = torch.full((2 * layers, pool.n_pages, hkv, ps, d), math.nan, dtype=torch.bfloat16, device=DEV)
    table = ac.rope_table(d)
    gen = torch.Generator(device=DEV).manual_seed(d)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    kept = {}          # per sequence and layer: keys, values [n, hkv, d] as stored; gathered weights fp64 [hkv, n]
    weights = {}       # per sequence and layer: the library's weights [hkv, max_pages ps]
    position = {}      # of a sequence's next token

    def dev(x):
        return torch.as_tensor(np.asarray(x), dtype=torch.int32, device=DEV)

    def batch_of(seqs, counts):
        host, lens = pool.tables(seqs, max_pages)
        cu = np.concatenate([[0], np.cumsum(counts)])
        starts, shared = pool.groups(seqs)
        return ac.PagedBatch(dev(cu), dev(lens), dev(host), n_tokens=int(cu[-1]), h_q=hq, h_kv=hkv, d=d, page_size=ps,
                             n_pages=pool.n_pages, dev_status=status.data_ptr(), group_starts=dev(starts),
                             prefix_pages=dev(shared)), cu, lens, shared

    def step(new):
        seqs = [s for s, _ in new]
        ac.page_copy(pages, [c for s, n in new for c in pool.extend(s, n)])
        batch, cu, lens, shared = batch_of(seqs, [n for _, n in new])
        pos = torch.cat([torch.arange(position[s], position[s] + n) for s, n in new])
        for layer in range(layers):
            qkv = torch.randn(int(cu[-1]), hq + 2 * hkv, d, generator=gen, device=DEV).to(torch.bfloat16)
            q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
            kp, vp = pages[2 * layer], pages[2 * layer + 1]
            want_k, size = rotate(k, pos.to(DEV)[:, None], d)
            # places in the cache are not positions any more: rotated by positions, appended as they are
            qr, kr = ac.rope_fwd(q, k, table, positions=dev(pos))
            # (against the unrounded value: two rounded ones may lie a whole step, 2^-7, apart)
            assert ((kr.double() - want_k).abs() <= rope_tolerance(want_k, size, d)).all()
            ac.paged_append(batch, None, kr, v, kp, vp)
            o, lse = ac.paged_prefix_fwd(batch, qr, kp, vp)
            both = torch.stack([weights[s][layer] for s in seqs])
            ac.paged_weights(batch, qr, lse, kp, both, decay=0.9)
            for i, (s, n) in enumerate(new):
                rows = slice(int(cu[i]), int(cu[i]) + n)
                weights[s][layer] = both[i]
                keys, values, gained = kept[s][layer]
                keys, values = torch.cat((keys, kr[rows])), torch.cat((values, v[rows]))
                m = len(keys)
                assert m == lens[i]
                x = torch.einsum("qhd,khd->hqk", qr[rows].double(), keys.double().repeat_interleave(g, 1)) / math.sqrt(d)
                last = m - n + torch.arange(n, device=DEV)
                x = x.masked_fill(torch.arange(m, device=DEV)[None] > last[:, None], -math.inf)
                w = torch.softmax(x, -1)
                ref = torch.einsum("hqk,khd->qhd", w, values.double().repeat_interleave(g, 1))
                mag = torch.einsum("hqk,khd->qhd", w, values.double().abs().repeat_interleave(g, 1))
                # P and O are rounded once each (2^-8), scores are off by less than 2^-12
                assert ((o[rows].double() - ref).abs() <= BF16 * (ref.abs() + mag) + 2.0 ** -12 * mag).all()
                z = torch.logsumexp(x, -1)
                assert ((lse[:, rows].double() - z).abs() <= 2.0 ** -12).all()
                added = w.view(hkv, g, n, m).sum((1, 2))
                now = torch.cat((gained * 0.9, torch.zeros(hkv, n, dtype=torch.float64, device=DEV)), 1) + added
                got = both[i, :, :m].double()
                # each term is off by less than 2^-12 (the scores) and 2^-12 (the LSE), and every
                # step's value is taken on from the library's own
                assert ((got - now).abs() <= 2.0 ** -11 * added + 2.0 ** -22 * now).all()
                kept[s][layer] = (keys, values, got)
        for s, n in new:
            position[s] += n
        return shared

    def bound(seqs, most, first, recent):
        batch, _, lens, _ = batch_of(seqs, [0] * len(seqs))
        keep = [min(most, int(n)) for n in lens]
        out = dev(pool.shrink(seqs, keep, max_pages))
        for layer in range(layers):
            both = torch.stack([weights[s][layer] for s in seqs])
            host = both.cpu().numpy()
            got = ac.paged_evict(batch, both, dev(keep), pages[2 * layer], pages[2 * layer + 1], first=first,
                                 recent=recent, out_table=out)
            for i, s in enumerate(seqs):
                keys, values, gained = kept[s][layer]
                src = torch.stack([torch.from_numpy(choose(host[i, h, :int(lens[i])], int(lens[i]), keep[i], first, recent))
                                   for h in range(hkv)]).to(DEV)
                assert torch.equal(got[i, :, :keep[i]].long(), src)
                pick = src.t()[..., None].expand(-1, -1, d)
                kept[s][layer] = (keys.gather(0, pick), values.gather(0, pick), gained.gather(1, src))
                weights[s][layer] = both[i]

    def add():
        s = pool.add()
        none = torch.zeros(0, hkv, d, dtype=torch.bfloat16, device=DEV)
        kept[s] = [(none, none, torch.zeros(hkv, 0, dtype=torch.float64, device=DEV))] * layers
        weights[s] = [torch.full((hkv, max_pages * ps), math.nan, device=DEV) for _ in range(layers)]
        position[s] = 0
        return s

    def fork(s):
        t = pool.fork(s)
        kept[t], weights[t], position[t] = list(kept[s]), [w.clone() for w in weights[s]], position[s]
        return t

    a, other = add(), add()
    step([(a, 260), (other, 70)])                     # two prompts
    answers = [a] + [fork(a) for _ in range(4)]
    for _ in range(3):                                 # the forks' first tokens: their prompt is visited once
        shared = step([(s, 1) for s in answers] + [(other, 1)])
        assert shared.max() == 260 // ps
    step([(s, 1 + i) for i, s in enumerate(answers)])  # drafts of several lengths
    bound(answers[:2], 200, 4, 32)                     # two answers drop keys: they leave the shared pages
    shared = step([(s, 1) for s in answers])
    assert shared.max() == 260 // ps                   # the others still share theirs
    b = fork(answers[0])                               # a fork of a shortened answer
    shared = step([(answers[0], 1), (b, 2), (answers[3], 1), (answers[4], 1)])
    assert len(shared) == 2 and shared.min() >= 200 // ps
    bound([answers[0], b, answers[3], answers[4], other], 128, 2, 40)
    for s in answers[1:3]:
        pool.free(s)
    step([(s, 3) for s in (answers[0], b, answers[3], other)])
    bound([answers[0], b], 64, 0, 64)
    ac.page_copy(pages, pool.compact())
    step([(answers[0], 40), (b, 1), (answers[4], 1)])
    assert int(status.item()) == 0
