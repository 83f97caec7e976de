"""Plain 64-bit implementations of rotary positions and of attention over a
paged cache, and the paged batches the tests run them on."""
from __future__ import annotations

import math

import numpy as np
import torch

ORIGINAL = 4096.0

# A rounding to bf16 is off by at most half a step: 2^-8 of the value.
BF16 = 2.0 ** -8


def frequencies(rot, base=10000.0, scaling="none", factor=1.0, original_len=ORIGINAL):
    """(radians per position of each pair, factor on the values)."""
    f = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    m = 1.0
    if scaling == "linear":
        f = [x / factor for x in f]
    elif scaling == "bands":
        out = []
        for x in f:
            n = original_len * x / (2 * math.pi)
            k = min(1.0, max(0.0, (n - 1.0) / 3.0))
            out.append(k * x + (1 - k) * x / factor)
        f = out
    elif scaling == "yarn":
        def pair(turns):
            return rot * math.log(original_len / (2 * math.pi * turns)) / (2 * math.log(base))
        lo, hi = max(math.floor(pair(32.0)), 0), min(math.ceil(pair(1.0)), rot - 1)
        f = [x * (1 - k) + x / factor * k
             for x, k in ((x, min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))) for i, x in enumerate(f))]
        m = 0.1 * math.log(factor) + 1.0
    return f, m


def rotate(x, pos, rot, interleaved=False, backward=False, **scaling):
    """x [..., d] in 64 bits, pos broadcast against x[..., 0].  Returns the
    rotated values and, per element, the sum of the magnitudes it is formed
    from (what a rounding of the factors scales with)."""
    f, m = frequencies(rot, **scaling)
    x = x.double()
    y, size = x.clone(), x.abs().clone()
    for i, w in enumerate(f):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        ang = pos.double() * w * (-1.0 if backward else 1.0)
        c, s = torch.cos(ang) * m, torch.sin(ang) * m
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
        size[..., a] = size[..., b] = m * (x[..., a].abs() + x[..., b].abs())
    return y, size


def rope_tolerance(y, size, rot):
    """One rounding to bf16, and for the rotated part the fp32 arithmetic: the
    angle's fraction in 24 bits (pi 2^-25 rad), sincospi (2 ulp), the factor m
    and two products and a sum (4 x 2^-24), together below 2^-21 of the sum of
    magnitudes.  The part that is copied has to be equal."""
    tol = BF16 * y.abs() + 2.0 ** -21 * size
    tol[..., rot:] = 0
    return tol


class Paged:
    """A paged cache on the GPU with sequences of the given new tokens and keys
    in randomly ordered pages, filled with NaN wherever no key lies."""

    def __init__(self, nq, nk, h_q, h_kv, d, page_size, seed=0, spare=3, n_tokens=None, dev="cuda:0", cols=None):
        gen = torch.Generator(device=dev).manual_seed(seed)
        self.nq, self.nk, self.h_q, self.h_kv, self.d, self.ps = list(nq), list(nk), h_q, h_kv, d, page_size
        need = [-(-n // page_size) for n in nk]
        self.n_pages = sum(need) + spare
        cols = cols or max(1, max(need))
        order = np.random.RandomState(seed).permutation(self.n_pages).astype(np.int32)
        table = np.full((len(nq), cols), -7, dtype=np.int32)
        at = 0
        for i, n in enumerate(need):
            table[i, :n] = order[at:at + n]
            at += n
        self.host_table = table
        self.cu_host = [0] + [int(x) for x in np.cumsum(nq)]
        self.n_tokens = n_tokens if n_tokens is not None else self.cu_host[-1]
        dev_i = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
        self.cu, self.kv_lens, self.table = dev_i(self.cu_host), dev_i(list(nk)), torch.from_numpy(table).to(dev)

        def randn(*shape):
            return torch.randn(shape, generator=gen, device=dev).to(torch.bfloat16)
        self.q = randn(self.n_tokens, h_q, d)
        self.k_new, self.v_new = randn(self.n_tokens, h_kv, d), randn(self.n_tokens, h_kv, d)
        self.k_pages = torch.full((self.n_pages, h_kv, page_size, d), math.nan, dtype=torch.bfloat16, device=dev)
        self.v_pages = self.k_pages.clone()
        self.keys = [randn(n, h_kv, d) for n in nk]
        self.values = [randn(n, h_kv, d) for n in nk]
        for i, n in enumerate(nk):
            page, row = self.places(i, torch.arange(n, device=dev))
            self.k_pages[page, :, row] = self.keys[i]
            self.v_pages[page, :, row] = self.values[i]
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)

    def places(self, i, pos):
        return self.table[i].long()[pos // self.ps], pos % self.ps

    def batch(self, **kw):
        import attention_core_gb300 as ac
        kw = {"n_tokens": self.n_tokens, "h_q": self.h_q, "h_kv": self.h_kv, "d": self.d, "page_size": self.ps,
              "n_pages": self.n_pages, "dev_status": self.status.data_ptr(), **kw}
        return ac.PagedBatch(self.cu, self.kv_lens, self.table, **kw)


def attend(p: Paged, causal=True, scale=None):
    """(O, LSE, sum of P |V| per element) of every sequence's new tokens in 64
    bits; rows of no sequence are NaN."""
    scale = scale or float(np.float32(1.0) / np.sqrt(np.float32(p.d)))
    o = torch.full(p.q.shape, math.nan, dtype=torch.float64, device=p.q.device)
    size = o.clone()
    lse = torch.full((p.h_q, p.n_tokens), math.nan, dtype=torch.float64, device=p.q.device)
    g = p.h_q // p.h_kv
    for i, (n, m) in enumerate(zip(p.nq, p.nk)):
        rows = slice(p.cu_host[i], p.cu_host[i] + n)
        k, v = p.keys[i].double(), p.values[i].double()
        for t in range(0, n, 512):                       # in slices of rows: the scores are written out
            part = slice(rows.start + t, min(rows.start + t + 512, rows.stop))
            q = p.q[part].double()
            x = torch.einsum("qhd,khd->hqk", q, k.repeat_interleave(g, 1)) * scale
            if causal:
                pos = m - n + t + torch.arange(q.shape[0], device=x.device)
                x = x.masked_fill(torch.arange(m, device=x.device)[None, :] > pos[:, None], -math.inf)
            z = torch.logsumexp(x, -1) if m else torch.full(x.shape[:2], -math.inf, dtype=x.dtype, device=x.device)
            w = torch.exp(x - torch.where(z == -math.inf, torch.zeros_like(z), z)[..., None])
            o[part] = torch.einsum("hqk,khd->qhd", w, v.repeat_interleave(g, 1))
            size[part] = torch.einsum("hqk,khd->qhd", w, v.abs().repeat_interleave(g, 1))
            lse[:, part] = z
    return o, lse, size


def check_attention(o, lse, want, p: Paged):
    """O within one rounding of each probability and one of the result (2^-8
    each) and 2^-12 of sum P |V| for the fp32 scores: a score of d products is
    off by at most d 2^-24 times the sum of their magnitudes, times the scale
    -- below 2^-13 for d <= 160 and normal inputs -- which moves P by that
    much, and its row sum likewise.  LSE within the same 2^-13, and 2^-12
    overall with the logarithm's rounding."""
    ro, rlse, size = want
    used = p.cu_host[-1]
    err = (o[:used].double() - ro[:used]).abs()
    tol = BF16 * (ro[:used].abs() + size[:used]) + 2.0 ** -12 * size[:used]
    assert torch.isfinite(o[:used].float()).all()
    assert (err <= tol).all(), float((err - tol).max())
    a, b = lse[:, :used].double(), rlse[:, :used]
    empty = b == -math.inf
    assert torch.equal(a == -math.inf, empty)
    assert not (o[:used].double().permute(1, 0, 2)[empty] != 0).any()
    assert ((a - b)[~empty].abs() <= 2.0 ** -12).all(), float((a - b)[~empty].abs().max())
