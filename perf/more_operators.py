"""Operators measured for many continuations of one prompt in a bounded cache:
attention of sequences that share the first pages of a paged key/value cache,
the attention weight that each cached key has gathered, and the eviction of the
keys that gathered least.

``run`` computes one pass of a case.  With ``own`` false it is the plain form:
elementary torch operations in 32 bits, rounded once at the end.  With ``own``
true it makes the library's calls.  ``exact`` gives the same outputs from the
definitions in 64 bits.

Layouts (bf16 but for the weights, which are fp32):
  q        [tokens, h_q, d]; sequence i owns the tokens cu[i] .. cu[i + 1] - 1
  pages    k, v [n_pages, h_kv, page_size, d]; position j of sequence i is row
           j % page_size of page page_table[i, j // page_size]
  groups   the sequences starts[g] .. starts[g + 1] - 1 name the same pages in
           their first prefix_pages[g] columns
  weights  [n_seq, h_kv, max_pages * page_size]; of key j of sequence i
New token t of a sequence with n new tokens and kv keys (the new ones among
them) sees the keys 0 .. kv - n + t.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases ---

def _prefix(name, n_groups, per_group, prefix, suffix, max_q, h_q, h_kv, d, page_size, **kw):
    c = dict(op="prefix", n_groups=n_groups, per_group=per_group, prefix=prefix, suffix=suffix, max_q=max_q, h_q=h_q,
             h_kv=h_kv, d=d, page_size=page_size, ragged=True)
    c.update(kw)
    return dict(c, name=name) if name else c


def _weights(name, n_seq, max_q, max_kv, h_q, h_kv, d, page_size, **kw):
    c = dict(op="weights", n_seq=n_seq, max_q=max_q, max_kv=max_kv, h_q=h_q, h_kv=h_kv, d=d, page_size=page_size,
             decay=1.0, ragged=True)
    c.update(kw)
    return dict(c, name=name) if name else c


def _evict(name, n_seq, max_kv, keep, first, recent, h_kv, d, page_size, **kw):
    c = dict(op="evict", n_seq=n_seq, max_kv=max_kv, keep=keep, first=first, recent=recent, h_kv=h_kv, d=d,
             page_size=page_size, ragged=True)
    c.update(kw)
    return dict(c, name=name) if name else c


def listed():
    return [
        # four answers to one short question, early on: latency
        _prefix("prefix four short", 1, 4, 512, 40, 1, 64, 8, 128, 16),
        # one decoding step of 64 samples of one long prompt
        _prefix("prefix 64 samples", 1, 64, 8192, 500, 1, 64, 8, 128, 64),
        # six prompts with eight samples each, of unequal lengths, the 22B-shaped shard's heads (d = 96)
        _prefix("prefix six prompts", 6, 8, 4000, 700, 1, 8, 8, 96, 16),
        # sixteen questions about one very long document
        _prefix("prefix long document", 1, 16, 131072, 300, 1, 64, 8, 128, 128),
        # several drafted tokens of each sequence are verified at once, the 530B-shaped shard's heads (d = 160)
        _prefix("prefix drafts", 2, 16, 2000, 100, 8, 16, 16, 160, 32),
        # one user's next token over a short context: latency
        _weights("weights one short", 1, 1, 500, 64, 8, 128, 16),
        # one decoding step of 64 users with contexts of all lengths up to 8192 tokens
        _weights("weights decode batch", 64, 1, 8192, 64, 8, 128, 64),
        # a chunk of a long prompt over what the cache already holds, after which keys are dropped
        _weights("weights chunk", 1, 2048, 8192, 64, 8, 128, 64, ragged=False),
        # chunks and single tokens in one batch, earlier weights fading
        _weights("weights mixed", 8, 500, 4001, 16, 16, 160, 32, decay=0.9),
        # a short context drops what does not fit any more: latency
        _evict("evict one short", 1, 600, 512, 4, 64, 2, 64, 16),
        # 64 users' contexts are cut to a quarter of the longest
        _evict("evict batch", 64, 8192, 2048, 4, 256, 8, 128, 64),
        # one very long prompt is cut to a quarter before it is answered
        _evict("evict one long", 1, 131072, 32768, 16, 1024, 8, 128, 128, ragged=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.4)))))


def draw(rng):
    op = rng.choice(["prefix", "prefix", "weights", "evict"])
    d = rng.choice([64, 96, 128, 160])
    h_kv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 1, 2, 3, 4, 8])
    ps = rng.choice([16, 32, 64, 128])
    if op == "prefix":
        n_groups = _log(rng, 1, 6)
        per_group = _log(rng, 1, max(1, 64 // n_groups))
        n_seq = n_groups * per_group
        max_q = rng.choice([1, 1, _log(rng, 1, max(1, 256 // n_seq))])
        prefix = _log(rng, ps, max(ps, min(131072, 500000 // n_seq)))
        return _prefix(None, n_groups, per_group, prefix, max_q + _log(rng, 1, 500), max_q, h_kv * group, h_kv, d, ps)
    if op == "weights":
        n_seq = _log(rng, 1, 64)
        max_q = rng.choice([1, _log(rng, 1, max(1, 2048 // n_seq))])
        room = (1 << 30) // (n_seq * max_q * h_kv * group)          # scores that the plain form holds
        max_kv = max(1, min(max_q + _log(rng, 1, max(2, 262144 // n_seq)), room, 131072))
        return _weights(None, n_seq, max_q, max_kv, h_kv * group, h_kv, d, ps, decay=rng.choice([1.0, 0.98]))
    n_seq = _log(rng, 1, 64)
    max_kv = _log(rng, 16, min(131072, 524288 // n_seq))
    keep = _log(rng, 1, max_kv)
    return _evict(None, n_seq, max_kv, keep, rng.choice([0, 4, 16]), rng.randint(0, max(1, keep // 4)), h_kv, d, ps)


def _lens(c):
    """(new tokens, keys) of each sequence: unequal ones where the case is ragged."""
    rng = random.Random("%d %d %d" % (c["n_seq"], c.get("max_q", 0), c["max_kv"]))
    nq, nk = [], []
    for i in range(c["n_seq"]):
        q, k = c.get("max_q", 0), c["max_kv"]
        if c["ragged"] and not (i == 0 and c["n_seq"] > 1):
            q = rng.randint(max(1, q // 8), q) if q else 0
            k = rng.randint(max(1, k // 8), k)
            if i % 4 == 1 and q:
                q = 1
        nq.append(q)
        nk.append(max(k, q))
    return nq, nk


def _groups(c):
    """Prefix pages of each group, and (new tokens, own keys) of each sequence."""
    rng = random.Random("%d %d %d %d" % (c["n_groups"], c["per_group"], c["prefix"], c["suffix"]))
    pages, nq, own_keys = [], [], []
    for g in range(c["n_groups"]):
        keys = c["prefix"] if g == 0 else rng.randint(max(1, c["prefix"] // 4), c["prefix"])
        pages.append(max(1, keys // c["page_size"]))       # what is shared are whole pages
        for i in range(c["per_group"]):
            q = rng.randint(1, c["max_q"])
            nq.append(q)
            own_keys.append(rng.randint(q, max(q, c["suffix"])))
    return pages, nq, own_keys


def work(case):
    c = case
    d, h_kv = c["d"], c["h_kv"]
    if c["op"] == "evict":
        kept = sum(min(c["keep"], n) for n in _lens(c)[1])
        return {"bytes": h_kv * (4 * sum(_lens(c)[1]) + kept * (8 + 8 * d)), "flops": 0}
    h_q = c["h_q"]
    if c["op"] == "prefix":
        pages, nq, mine = _groups(c)
        shared = [p * c["page_size"] for p in pages for _ in range(c["per_group"])]
        keys = sum(pages) * c["page_size"] + sum(mine)
        pairs = sum(sum(s + m - q + t + 1 for t in range(q)) for s, m, q in zip(shared, mine, nq))
        return {"bytes": 4 * sum(nq) * h_q * d + 4 * keys * h_kv * d + 4 * sum(nq) * h_q, "flops": 4 * pairs * h_q * d}
    nq, nk = _lens(c)
    pairs = sum(sum(k - q + t + 1 for t in range(q)) for q, k in zip(nq, nk))
    # old keys' weights are read, all keys' are written
    return {"bytes": 2 * sum(nq) * h_q * d + 4 * sum(nq) * h_q + h_kv * (2 * sum(nk) * d + 8 * sum(nk) - 4 * sum(nq)),
            "flops": 2 * pairs * h_q * d}


# ----------------------------------------------------------------- inputs ---

def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).to(torch.bfloat16)


def _dev(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV).manual_seed(int(seed) & (2**62 - 1))
    mix = np.random.RandomState(int(seed) % (2**32))
    s = {"case": c}
    h_kv, d, ps = c["h_kv"], c["d"], c["page_size"]
    if c["op"] == "prefix":
        shared, nq, mine = _groups(c)
        nk = [shared[i // c["per_group"]] * ps + m for i, m in enumerate(mine)]
    else:
        nq, nk = _lens(c)
    need = [-(-k // ps) for k in nk]
    cols = max(need)
    n_seq, total = len(nk), sum(nq)
    out_pages = sum(-(-min(c["keep"], k) // ps) for k in nk) if c["op"] == "evict" else 0
    n_pages = sum(need) + out_pages + 3
    order = mix.permutation(n_pages)
    table, at = np.full((n_seq, cols), -1, dtype=np.int32), 0       # entries past a sequence's pages are never read
    for i, n in enumerate(need):
        have = 0
        if c["op"] == "prefix" and i % c["per_group"]:
            have = shared[i // c["per_group"]]
            table[i, :have] = table[i - 1, :have]
        table[i, have:n] = order[at:at + n - have]
        at += n - have
    s["cu"], s["kv_lens"], s["page_table"] = _dev([0] + [int(x) for x in np.cumsum(nq)]), _dev(nk), torch.from_numpy(table).to(DEV)
    s["nq"], s["nk"] = nq, nk
    s["k_pages"], s["v_pages"] = _randn(gen, n_pages, h_kv, ps, d), None
    if c["op"] != "weights":
        s["v_pages"] = _randn(gen, n_pages, h_kv, ps, d)
    if c["op"] != "evict":
        s["q"] = _randn(gen, total, c["h_q"], d)
    if c["op"] == "prefix":
        s["starts"] = _dev([g * c["per_group"] for g in range(c["n_groups"] + 1)])
        s["prefix_pages"] = _dev(shared)
    else:
        # what keys gather: nearly all little, a few a lot
        s["weights"] = torch.rand((n_seq, h_kv, cols * ps), generator=gen, device=DEV).clamp_(min=1e-7).pow_(-0.4).sub_(1.0)
        s["new_weights"] = torch.zeros_like(s["weights"])
    if c["op"] == "weights":
        s["lse"] = _logsumexp(s)
    if c["op"] == "evict":
        s["keep"] = _dev([c["keep"]] * n_seq)
        to = np.full((n_seq, cols), -1, dtype=np.int32)              # pages that the kept keys move to
        for i, n in enumerate(nk):
            n = -(-min(c["keep"], n) // ps)
            to[i, :n] = order[at:at + n]
            at += n
        s["out_table"] = torch.from_numpy(to).to(DEV)
        s["kept"] = torch.full((n_seq, h_kv, cols * ps), -1, dtype=torch.int32, device=DEV)
    if own:
        import attention_core_gb300 as ac
        s["batch"] = ac.PagedBatch(s["cu"], s["kv_lens"], s["page_table"], n_tokens=total, h_q=c.get("h_q", h_kv),
                                   h_kv=h_kv, d=d, page_size=ps, n_pages=n_pages, group_starts=s.get("starts"),
                                   prefix_pages=s.get("prefix_pages"))
    return s


# ------------------------------------------------------------- plain form ---

def _scores(s):
    """Scaled scores [n_seq, h_kv, group, new tokens (padded), keys], -inf where
    unseen, and the padded rows' tokens."""
    c = s["case"]
    h_kv, d, ps, n = c["h_kv"], c["d"], c["page_size"], s["q"].shape[0]
    g, mq, n_seq = c["h_q"] // h_kv, max(s["nq"]), len(s["nk"])
    cu, kv = s["cu"].long(), s["kv_lens"].long()
    nq = cu[1:] - cu[:-1]
    local = torch.arange(mq, device=DEV)
    tok = (cu[:-1, None] + local).clamp(max=n - 1)
    q = s["q"].float()[tok].view(n_seq, mq, h_kv, g, d).permute(0, 2, 3, 1, 4).reshape(n_seq, h_kv, g * mq, d)
    pages = s["page_table"].long().clamp(min=0)
    at = torch.arange(pages.shape[1] * ps, device=DEV)
    k = s["k_pages"][pages].float().transpose(1, 2).reshape(n_seq, h_kv, -1, d)
    x = torch.matmul(q, k.transpose(-1, -2)).mul_(1.0 / math.sqrt(d)).view(n_seq, h_kv, g, mq, -1)
    del k
    sees = at <= (kv - nq)[:, None, None] + local[:, None]                 # [n_seq, mq, keys]
    sees &= (local < nq[:, None])[:, :, None]                              # padding
    return x.masked_fill_(~sees[:, None, None], -math.inf), pages


def _rows(s):
    """(sequence, index within its new tokens) of each new token."""
    tok = torch.arange(s["q"].shape[0], device=DEV)
    cu = s["cu"].long()
    seq = torch.searchsorted(cu, tok, right=True) - 1
    return seq, tok - cu[seq]


def _logsumexp(s):
    x, _ = _scores(s)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    lse = (top + torch.log(x.sub_(top).exp_().sum(-1, keepdim=True)))[..., 0]
    seq, t = _rows(s)
    return lse[seq, :, :, t].reshape(len(seq), -1).t().contiguous()


def _plain_prefix(s):
    c = s["case"]
    h_q, h_kv, d, n = c["h_q"], c["h_kv"], c["d"], s["q"].shape[0]
    x, pages = _scores(s)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)        # padded rows
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    v = s["v_pages"][pages].float().transpose(1, 2).reshape(len(s["nk"]), h_kv, -1, d)
    o = torch.matmul(p.flatten(2, 3), v).view(*p.shape[:4], d)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (top + torch.log(total))[..., 0]
    seq, t = _rows(s)
    return {"o": o[seq, :, :, t].reshape(n, h_q, d).to(torch.bfloat16), "lse": lse[seq, :, :, t].reshape(n, h_q).t().contiguous()}


def _plain_weights(s):
    c = s["case"]
    h_kv, g = c["h_kv"], c["h_q"] // c["h_kv"]
    x, _ = _scores(s)
    n_seq, mq = x.shape[0], x.shape[3]
    cu, kv = s["cu"].long(), s["kv_lens"].long()
    nq = cu[1:] - cu[:-1]
    local = torch.arange(mq, device=DEV)
    tok = (cu[:-1, None] + local).clamp(max=s["q"].shape[0] - 1)
    lse = s["lse"].view(h_kv, g, -1)[:, :, tok].permute(2, 0, 1, 3)        # [n_seq, h_kv, g, mq]
    gained = x.sub_(lse[..., None]).exp_().sum((2, 3))                     # unseen pairs give exp(-inf)
    at = torch.arange(gained.shape[-1], device=DEV)
    old = (at < (kv - nq)[:, None])[:, None]
    new = torch.where(old, s["weights"] * c["decay"], torch.zeros_like(gained)) + gained
    out = s["new_weights"]
    out.copy_(torch.where((at < kv[:, None])[:, None], new, out))
    return out


def _plain_evict(s):
    c = s["case"]
    ps, keep = c["page_size"], c["keep"]
    w, kv = s["weights"], s["kv_lens"].long()
    length = w.shape[-1]
    at = torch.arange(length, device=DEV)
    n = torch.minimum(kv, s["keep"].long())                                # keys that stay
    recent = n.clamp(max=c["recent"])
    first = (n - recent).clamp(max=c["first"])
    sure = (at >= (kv - recent)[:, None]) | (at < first[:, None])
    rank = torch.where(sure[:, None], torch.full_like(w, math.inf), w)
    rank = torch.where((at < kv[:, None])[:, None], rank, torch.full_like(w, -math.inf))
    best = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., : min(keep, length)]
    best = torch.where((at[: best.shape[-1]] < n[:, None])[:, None], best, torch.full_like(best, length))
    best = best.sort(-1).values                                            # in order; past n the places are `length`
    here = best < length
    seq, head, j = here.nonzero(as_tuple=True)
    src = best[seq, head, j]
    s["kept"][seq, head, j] = src.to(torch.int32)
    s["new_weights"][seq, head, j] = w[seq, head, src]
    old, new = s["page_table"].long()[seq, src // ps], s["out_table"].long()[seq, j // ps]
    for x in (s["k_pages"], s["v_pages"]):
        x[new, head, j % ps] = x[old, head, src % ps]
    return {"kept": s["kept"], "weights": s["new_weights"], "k": s["k_pages"], "v": s["v_pages"]}


# ---------------------------------------------------------------- library ---

def _own(s):
    import attention_core_gb300 as ac
    c = s["case"]
    if c["op"] == "prefix":
        o, lse = ac.paged_prefix_fwd(s["batch"], s["q"], s["k_pages"], s["v_pages"])
        return {"o": o, "lse": lse}
    if c["op"] == "weights":
        return ac.paged_weights(s["batch"], s["q"], s["lse"], s["k_pages"], s["weights"], decay=c["decay"], out=s["new_weights"])
    kept = ac.paged_evict(s["batch"], s["weights"], s["keep"], s["k_pages"], s["v_pages"], first=c["first"],
                          recent=c["recent"], out_table=s["out_table"], out_weights=s["new_weights"], kept=s["kept"])
    return {"kept": kept, "weights": s["new_weights"], "k": s["k_pages"], "v": s["v_pages"]}


def run(state):
    if own:
        return _own(state)
    return {"prefix": _plain_prefix, "weights": _plain_weights, "evict": _plain_evict}[state["case"]["op"]](state)


# ------------------------------------------------------------------ exact ---

def exact(case, seed):
    c = case
    s = prepare(c, seed)
    h_kv, d, ps = c["h_kv"], c["d"], c["page_size"]
    table, nq, nk = s["page_table"].tolist(), s["nq"], s["nk"]
    if c["op"] == "evict":
        k, v = s["k_pages"].double(), s["v_pages"].double()
        kept, weights = s["kept"].clone(), s["new_weights"].double()
        w, to = s["weights"].cpu().numpy(), s["out_table"].tolist()
        for i, n in enumerate(nk):
            m = min(c["keep"], n)
            recent = min(c["recent"], m)
            first = min(c["first"], m - recent)
            old, new = (torch.tensor(x[i], device=DEV) for x in (table, to))
            for h in range(h_kv):
                middle = np.arange(first, n - recent)
                # by falling weight, then by rising index
                best = middle[np.lexsort((middle, -w[i, h, first:n - recent].astype(np.float64)))][: m - first - recent]
                src = np.concatenate([np.arange(first), np.sort(best), np.arange(n - recent, n)])
                src = torch.from_numpy(src).to(DEV)
                j = torch.arange(m, device=DEV)
                kept[i, h, :m] = src.to(torch.int32)
                weights[i, h, :m] = s["weights"][i, h, src].double()
                a, b = old[src.div(ps, rounding_mode="floor")], new[j.div(ps, rounding_mode="floor")]
                k[b, h, j.remainder(ps)] = s["k_pages"][a, h, src.remainder(ps)].double()
                v[b, h, j.remainder(ps)] = s["v_pages"][a, h, src.remainder(ps)].double()
        return {"kept": kept, "weights": weights, "k": k, "v": v}
    h_q, start = c["h_q"], 0
    g = h_q // h_kv
    if c["op"] == "prefix":
        o = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
        lse = torch.zeros((h_q, s["q"].shape[0]), dtype=torch.float64, device=DEV)
    else:
        gained = s["new_weights"].double()
    for i, (q, n) in enumerate(zip(nq, nk)):
        page = torch.tensor(table[i][: -(-n // ps)], device=DEV)
        hidden = torch.arange(n, device=DEV)[None, :] > torch.arange(n - q, n, device=DEV)[:, None]
        for h in range(h_kv):
            k = s["k_pages"][page, h].double().reshape(-1, d)[:n]
            heads = range(h * g, (h + 1) * g)
            if c["op"] == "prefix":
                v = s["v_pages"][page, h].double().reshape(-1, d)[:n]
                for e in heads:
                    x = (s["q"][start:start + q, e].double() @ k.t() / math.sqrt(d)).masked_fill(hidden, -math.inf)
                    z = torch.logsumexp(x, -1)
                    o[start:start + q, e] = torch.exp(x - z[:, None]) @ v
                    lse[e, start:start + q] = z
            else:
                total = torch.zeros(n, dtype=torch.float64, device=DEV)
                total[: n - q] = s["weights"][i, h, : n - q].double() * c["decay"]
                for e in heads:
                    x = (s["q"][start:start + q, e].double() @ k.t() / math.sqrt(d)).masked_fill(hidden, -math.inf)
                    total += torch.exp(x - s["lse"][e, start:start + q].double()[:, None]).sum(0)
                gained[i, h, :n] = total
        start += q
    return {"o": o, "lse": lse} if c["op"] == "prefix" else gained
