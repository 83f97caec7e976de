"""A small serving loop over the paged cache, as the operators are used together:
prompts in chunks, single tokens, a fork, a freed sequence and a compaction, on
two layers, with every step's outputs against a plain 64-bit attention over the
tokens that each sequence has seen; and training-side use, the rotation around
the core's forward and backward."""
import math

import pytest
import torch

import attention_core_gb300 as ac
from attention_core_gb300.pagepool import PagePool
from tests.serve_ref import BF16, rotate

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("hq,hkv,d,ps", [(8, 2, 128, 16), (4, 4, 96, 32), (6, 2, 160, 64)])
def test_serving_loop(hq, hkv, d, ps):
    layers, max_pages = 2, 40
    pool = PagePool(60, ps)
    pages = torch.full((2 * layers, pool.n_pages, hkv, ps, d), math.nan, dtype=torch.bfloat16, device=DEV)
    table = ac.rope_table(d, scaling="yarn", factor=4.0, original_len=4096)
    kw = dict(scaling="yarn", factor=4.0)
    gen = torch.Generator(device=DEV).manual_seed(d)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    seen = {}                                         # per sequence and layer: (rotated keys as stored, values)

    def step(new):
        """One forward pass: `new` = [(sequence, new tokens)]."""
        copies = [c for s, n in new for c in pool.extend(s, n)]
        ac.page_copy(pages, copies)
        host, lens = pool.tables([s for s, _ in new], max_pages)
        cu = [0]
        for _, n in new:
            cu.append(cu[-1] + n)
        dev = lambda x: torch.as_tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
        batch = ac.PagedBatch(dev(cu), dev(lens), dev(host), n_tokens=cu[-1], h_q=hq, h_kv=hkv, d=d, page_size=ps,
                              n_pages=pool.n_pages, dev_status=status.data_ptr())
        for layer in range(layers):
            qkv = torch.randn(cu[-1], hq + 2 * hkv, d, generator=gen, device=DEV).to(torch.bfloat16)
            q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
            kp, vp = pages[2 * layer], pages[2 * layer + 1]
            qr = ac.paged_append(batch, q, k, v, kp, vp, table=table)
            o, lse = ac.paged_fwd(batch, qr, kp, vp)
            for i, (s, n) in enumerate(new):
                rows = slice(cu[i], cu[i] + n)
                pos = torch.arange(int(lens[i]) - n, int(lens[i]), device=DEV)
                keys, values = seen.setdefault(s, [(None, None)] * layers)[layer]
                want_k, size = rotate(k[rows], pos[:, None], d, **kw)
                # the stored keys are the rotation rounded once; what follows is computed from them
                stored = want_k.to(torch.bfloat16)
                keys = stored if keys is None else torch.cat((keys, stored))
                values = v[rows] if values is None else torch.cat((values, v[rows]))
                seen[s][layer] = (keys, values)
                want_q = rotate(q[rows], pos[:, None], d, **kw)[0].to(torch.bfloat16).double()
                g = hq // hkv
                x = torch.einsum("qhd,khd->hqk", want_q, keys.double().repeat_interleave(g, 1)) / math.sqrt(d)
                x = x.masked_fill(torch.arange(len(keys), device=DEV)[None] > pos[:, None], -math.inf)
                w = torch.softmax(x, -1)
                ref = torch.einsum("hqk,khd->qhd", w, values.double().repeat_interleave(g, 1))
                mag = torch.einsum("hqk,khd->qhd", w, values.double().abs().repeat_interleave(g, 1))
                # P and O are rounded once each (2^-8), and the library's rotated q and k
                # may round the other way where the 64-bit value lies near a border: one
                # step (2^-7) of a few elements, a score change far below 2^-8
                assert ((o[rows].double() - ref).abs() <= BF16 * (ref.abs() + 2 * mag)).all()
                assert ((lse[:, rows].t().double() - torch.logsumexp(x, -1).t()).abs() <= 2.0 ** -7).all()

    def fork(s):
        new = pool.fork(s)
        seen[new] = list(seen[s])
        return new

    a, b = pool.add(), pool.add()
    step([(a, 37), (b, 5)])                           # prompts
    step([(a, 90), (b, 1)])                           # the next chunk, and a single token
    c = fork(a)
    step([(a, 1), (b, 1), (c, 1)])                    # the fork writes into a shared page
    step([(c, 3), (a, 2)])
    pool.free(b)
    del seen[b]
    e = pool.add()
    step([(e, 150), (a, 1)])
    pool.free(c)
    del seen[c]
    ac.page_copy(pages, pool.compact())
    step([(a, 1), (e, 1)])
    f = fork(e)
    ac.page_copy(pages, pool.compact())
    step([(f, 20), (e, 1), (a, 130)])
    assert int(status.item()) == 0


def test_rotation_around_the_core():
    """Training: q and k rotated, the core's forward and recompute-backward, and
    the rotation's backward, against autograd through a 64-bit attention of the
    same rounded q and k."""
    b, hq, hkv, s, d = 2, 4, 2, 200, 128
    gen = torch.Generator(device=DEV).manual_seed(1)
    q, k, v, g = (torch.randn(b, h, s, d, generator=gen, device=DEV).to(torch.bfloat16) for h in (hq, hkv, hkv, hq))
    t = ac.rope_table(d, scaling="linear", factor=2.0)
    qr, kr = ac.rope_fwd(q, k, t)
    o, lse = ac.fwd(qr, kr, v, causal=True)
    dqr, dkr, dv = ac.bwd_recompute(qr, kr, v, o, lse, g, causal=True)
    dq, dk = ac.rope_bwd(dqr, dkr, t)
    xq, xk, xv = (x.double().requires_grad_() for x in (qr, kr, v))
    x = xq @ xk.repeat_interleave(hq // hkv, 1).transpose(-1, -2) / math.sqrt(d)
    x = x.masked_fill(torch.triu(torch.ones(s, s, dtype=torch.bool, device=DEV), 1), -math.inf)
    y = torch.softmax(x, -1) @ xv.repeat_interleave(hq // hkv, 1)
    gq, gk, gv = torch.autograd.grad((y * g.double()).sum(), (xq, xk, xv))
    pos = torch.arange(s, device=DEV)
    for got, grad in ((dq, gq), (dk, gk)):
        want, size = rotate(grad, pos, d, backward=True, scaling="linear", factor=2.0)
        # the core's gradients are within 1e-2 of each row's largest value; the turn
        # back mixes pairs of a row (a factor of at most sqrt 2) and rounds once
        row = want.abs().amax(-1, keepdim=True)
        assert ((got.double() - want).abs() <= (1.5e-2 + BF16) * row + 1e-3).all()
    assert ((dv.double() - gv).abs() <= 1e-2 * gv.abs().amax(-1, keepdim=True) + 1e-3).all()
