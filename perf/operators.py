"""Operators measured beside the attention core: rotary positions (forward and
backward), rotary positions fused with the append to a paged key/value cache,
attention of new tokens over such a cache, and the cache's page copies.

``run`` computes one pass of a case.  With ``own`` false it is the plain form:
elementary torch operations in 32 bits (angles in 64), rounded once at the end.
With ``own`` true it makes the library's calls.  ``exact`` gives the same
outputs from the definitions in 64 bits.

Layouts (bf16 throughout, as everywhere in the library):
  padded   q [b, h_q, s, d], k [b, h_kv, s, d]
  packed   q [tokens, h_q, d], k, v [tokens, h_kv, d]; sequence i owns the
           tokens cu[i] .. cu[i + 1] - 1
  pages    k, v [n_pages, h_kv, page_size, d]; position j of sequence i is row
           j % page_size of page page_table[i, j // page_size]
Position of new token t of a sequence with n new tokens and kv_len keys (the
new ones among them): kv_len - n + t; under the causal mask it sees the keys
0 .. kv_len - n + t.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases ---

def _rope(name, b, h_q, h_kv, s, d, rot, **kw):
    c = dict(op="rope", b=b, h_q=h_q, h_kv=h_kv, s=s, d=d, rot=rot, interleaved=False, scaling="none", factor=1.0,
             packed=False, backward=False, far=0)
    c.update(kw)
    return dict(c, name=name) if name else c


def _append(name, n_seq, max_q, max_kv, h_q, h_kv, d, page_size, **kw):
    c = dict(op="append", n_seq=n_seq, max_q=max_q, max_kv=max_kv, h_q=h_q, h_kv=h_kv, d=d, page_size=page_size,
             rot=d, interleaved=False, scaling="none", factor=1.0, ragged=True)
    c.update(kw)
    return dict(c, name=name) if name else c


def _attend(name, n_seq, max_q, max_kv, h_q, h_kv, d, page_size, **kw):
    c = dict(op="attend", n_seq=n_seq, max_q=max_q, max_kv=max_kv, h_q=h_q, h_kv=h_kv, d=d, page_size=page_size,
             causal=True, ragged=True)
    c.update(kw)
    return dict(c, name=name) if name else c


def _copy(name, planes, n_pages, n_pairs, h_kv, page_size, d, **kw):
    c = dict(op="copy", planes=planes, n_pages=n_pages, n_pairs=n_pairs, h_kv=h_kv, page_size=page_size, d=d)
    c.update(kw)
    return dict(c, name=name) if name else c


def listed():
    return [
        # the smallest training shape of this repository: launch cost is what counts
        _rope("rope tiny", 1, 2, 2, 128, 64, 64),
        # the Llama-3-70B-shaped layer (64 query heads, 8 KV heads, 8192 tokens), frequencies scaled by bands
        _rope("rope llama layer", 1, 64, 8, 8192, 128, 128, scaling="bands", factor=8.0),
        # the 175B-shaped shard's backward, interleaved pairs, half of each head rotated, positions far out
        _rope("rope 175b backward", 2, 12, 12, 2048, 128, 64, interleaved=True, backward=True, far=500000),
        # one decoding step of a serving batch: one new token of each of 64 sequences joins the cache
        _append("append decode 64", 64, 1, 4096, 64, 8, 128, 16, scaling="yarn", factor=4.0),
        # chunks of prompts of unequal lengths, the 22B-shaped shard's heads (d = 96)
        _append("append chunks", 6, 2048, 6000, 8, 8, 96, 64),
        # one user's next token over a short context: latency
        _attend("decode one short", 1, 1, 500, 64, 8, 128, 16),
        # one decoding step of 64 users with contexts of all lengths up to 8192 tokens
        _attend("decode batch", 64, 1, 8192, 64, 8, 128, 64),
        # one user's next token over a very long context: the keys have to be shared out
        _attend("decode one long", 1, 1, 131072, 64, 8, 128, 128, ragged=False),
        # a chunk of a long prompt over what the cache already holds
        _attend("chunk llama layer", 1, 2048, 8192, 64, 8, 128, 64, ragged=False),
        # chunks and single tokens in one batch, the 530B-shaped shard's heads (d = 160, no sharing)
        _attend("mixed batch", 8, 500, 4001, 16, 16, 160, 32),
        # a fork: the last, partly filled page of a sequence is copied in every layer
        _copy("fork one page", 16, 64, 1, 8, 16, 128),
        # compaction of a cache that emptied out: hundreds of pages move in every layer
        _copy("compact", 16, 1200, 400, 8, 64, 128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.4)))))


def draw(rng):
    op = rng.choice(["rope", "append", "attend", "attend", "copy"])
    d = rng.choice([64, 96, 128, 160])
    h_kv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 1, 2, 3, 4, 8])
    ps = rng.choice([16, 32, 64, 128])
    scaling = rng.choice(["none", "linear", "bands", "yarn"])
    rope = dict(interleaved=rng.random() < 0.5, scaling=scaling, factor=1.0 if scaling == "none" else float(rng.choice([2, 4, 8])))
    rot = rng.choice([d, d // 2, 16])
    if op == "rope":
        s = _log(rng, 1, 8192)
        b = _log(rng, 1, max(1, min(8, 8192 // s)))
        return _rope(None, b, h_kv * group, h_kv, s, d, rot, packed=rng.random() < 0.5, backward=rng.random() < 0.5,
                     far=rng.choice([0, _log(rng, 1, 1000000)]), **rope)
    if op == "append":
        n_seq = _log(rng, 1, 64)
        max_q = rng.choice([1, _log(rng, 1, max(1, 8192 // n_seq))])
        max_kv = max_q + _log(rng, 1, max(2, min(16384, 131072 // n_seq)))
        return _append(None, n_seq, max_q, max_kv, h_kv * group, h_kv, d, ps, rot=rot, **rope)
    if op == "attend":
        n_seq = _log(rng, 1, 64)
        max_q = rng.choice([1, _log(rng, 1, max(1, 2048 // n_seq))])
        room = (1 << 30) // (n_seq * max_q * h_kv * group)          # scores that the plain form holds
        max_kv = max(1, min(max_q + _log(rng, 1, max(2, 262144 // n_seq)), room, 131072))
        return _attend(None, n_seq, max_q, max_kv, h_kv * group, h_kv, d, ps, causal=rng.random() < 0.8)
    n_pages = _log(rng, 8, 1000)
    return _copy(None, rng.choice([2, 8, 16]), n_pages, _log(rng, 1, n_pages // 2), h_kv, ps, d)


def _lens(c):
    """(new tokens, keys) of each sequence: unequal ones where the case is ragged."""
    rng = random.Random("%d %d %d" % (c["n_seq"], c["max_q"], c["max_kv"]))
    nq, nk = [], []
    for i in range(c["n_seq"]):
        if not c["ragged"] or (i == 0 and c["n_seq"] > 1):
            q, k = c["max_q"], c["max_kv"]
        else:
            q = rng.randint(max(1, c["max_q"] // 8), c["max_q"])
            k = rng.randint(max(1, c["max_kv"] // 8), c["max_kv"])
            if i % 4 == 1:
                q = 1
        if c["op"] == "append":
            k = max(k, q)
        nq.append(q)
        nk.append(k)
    return nq, nk


def work(case):
    c = case
    if c["op"] == "rope":
        n = c["b"] * c["s"] * (c["h_q"] + c["h_kv"])
        return {"bytes": 4 * n * c["d"], "flops": 3 * n * c["rot"]}
    if c["op"] == "copy":
        return {"bytes": 4 * c["planes"] * c["n_pairs"] * c["h_kv"] * c["page_size"] * c["d"], "flops": 0}
    nq, nk = _lens(c)
    d, h_q, h_kv = c["d"], c["h_q"], c["h_kv"]
    if c["op"] == "append":
        return {"bytes": 4 * sum(nq) * (h_q + 2 * h_kv) * d, "flops": 3 * sum(nq) * (h_q + h_kv) * c["rot"]}
    # a sequence's keys are read once if any of its rows sees them
    keys = sum(k for q, k in zip(nq, nk) if q)
    if c["causal"]:
        pairs = sum(sum(max(0, k - q + t + 1) for t in range(q)) for q, k in zip(nq, nk))
    else:
        pairs = sum(q * k for q, k in zip(nq, nk))
    return {"bytes": 4 * sum(nq) * h_q * d + 4 * keys * h_kv * d + 4 * sum(nq) * h_q, "flops": 4 * pairs * h_q * d}


# ----------------------------------------------------------------- inputs ---

ORIGINAL = 4096       # context length before scaling
BASE = 10000.0


def _frequencies(c):
    """(radians per position of each rotated pair, factor on the rotated values), float64."""
    r = c["rot"]
    i = np.arange(r // 2, dtype=np.float64)
    f = BASE ** (-2.0 * i / r)
    m = 1.0
    if c["scaling"] == "linear":
        f = f / c["factor"]
    elif c["scaling"] == "bands":       # long waves slowed by the factor, short ones kept, a ramp in between
        turns = ORIGINAL * f / (2 * math.pi)
        keep = np.clip((turns - 1.0) / (4.0 - 1.0), 0.0, 1.0)
        f = f / c["factor"] * (1 - keep) + f * keep
    elif c["scaling"] == "yarn":        # a ramp over the pairs' index, and a factor on the values
        at = lambda turns: r * math.log(ORIGINAL / (turns * 2 * math.pi)) / (2 * math.log(BASE))  # noqa: E731
        lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), r - 1)
        slow = np.clip((i - lo) / max(hi - lo, 0.001), 0.0, 1.0)
        f = f / c["factor"] * slow + f * (1 - slow)
        m = 0.1 * math.log(c["factor"]) + 1.0
    return f, m


def _table(c):
    import attention_core_gb300 as ac
    return ac.rope_table(c["d"], rot_dim=c["rot"], base=BASE, interleaved=c["interleaved"], scaling=c["scaling"],
                         factor=c["factor"], original_len=ORIGINAL)


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).to(torch.bfloat16)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV).manual_seed(int(seed) & (2**62 - 1))
    s = {"case": dict(c)}
    if c["op"] == "copy":
        n, p = c["n_pairs"], c["n_pages"]
        s["pages"] = _randn(gen, c["planes"], p, c["h_kv"], c["page_size"], c["d"])
        order = np.random.RandomState(int(seed) % (2**32)).permutation(p)[: 2 * n].astype(np.int32)
        s["pairs"] = np.ascontiguousarray(order.reshape(n, 2))             # the allocator's list of (from, to), on the host
        s["pairs_dev"] = torch.from_numpy(s["pairs"].astype(np.int64)).to(DEV)
        return s
    h_q, h_kv, d = c["h_q"], c["h_kv"], c["d"]
    if c["op"] != "attend":
        f, m = _frequencies(c)
        s["freq"], s["mscale"] = torch.from_numpy(f).to(DEV), m
        if own:
            s["table"] = _table(c)
    if c["op"] == "rope":
        b, n = c["b"], c["s"]
        lead = (b * n,) if c["packed"] else (b,)
        s["q"] = _randn(gen, *lead, h_q, d) if c["packed"] else _randn(gen, b, h_q, n, d)
        s["k"] = _randn(gen, *lead, h_kv, d) if c["packed"] else _randn(gen, b, h_kv, n, d)
        pos = torch.arange(n, device=DEV, dtype=torch.int32)
        pos = pos + torch.randint(0, c["far"] + 1, (b, 1), generator=gen, device=DEV, dtype=torch.int32)
        s["pos"] = pos.reshape(-1).contiguous() if c["packed"] else pos.contiguous()
        return s
    nq, nk = _lens(c)
    ps, total = c["page_size"], sum(nq)
    need = [-(-k // ps) for k in nk]
    cols = -(-c["max_kv"] // ps)
    n_pages = sum(need) + 3
    order = np.random.RandomState(int(seed) % (2**32)).permutation(n_pages)
    table = np.full((len(nq), cols), -1, dtype=np.int32)                   # entries past a sequence's pages are never read
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    s["cu"], s["kv_lens"], s["page_table"] = dev([0] + list(np.cumsum(nq))), dev(nk), torch.from_numpy(table).to(DEV)
    s["max_q"], s["max_kv"] = max(nq), max(nk)
    s["k_pages"] = _randn(gen, n_pages, h_kv, ps, d)
    s["v_pages"] = _randn(gen, n_pages, h_kv, ps, d)
    if c["op"] == "append":
        # the projection's output: q, k and v of a token side by side
        qkv = _randn(gen, total, h_q + 2 * h_kv, d)
        s["q"], s["k"], s["v"] = qkv[:, :h_q], qkv[:, h_q:h_q + h_kv], qkv[:, h_q + h_kv:]
    else:
        s["q"] = _randn(gen, total, h_q, d)
    if own:
        import attention_core_gb300 as ac
        s["batch"] = ac.PagedBatch(s["cu"], s["kv_lens"], s["page_table"], n_tokens=total, h_q=h_q, h_kv=h_kv, d=d,
                                   page_size=ps, n_pages=n_pages, causal=c.get("causal", True))
    return s


# ------------------------------------------------------------- plain form ---

def _rotate(x, cos, sin, c, sign):
    """x [..., d] in 32 bits, cos / sin [..., rot / 2] that fit it."""
    r = c["rot"]
    x = x.float()
    if c["interleaved"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
    else:
        a, b = x[..., : r // 2], x[..., r // 2:r]
    u, v = a * cos - sign * (b * sin), b * cos + sign * (a * sin)
    y = torch.stack((u, v), -1).flatten(-2) if c["interleaved"] else torch.cat((u, v), -1)
    return torch.cat((y, x[..., r:]), -1).to(torch.bfloat16)


def _cos_sin(s, pos):
    ang = pos.double()[..., None] * s["freq"]
    return (torch.cos(ang) * s["mscale"]).float(), (torch.sin(ang) * s["mscale"]).float()


def _plain_rope(s):
    c = s["case"]
    cos, sin = _cos_sin(s, s["pos"])
    cos, sin = (x[:, None] for x in (cos, sin))       # over the heads of [b, h, s, d] or [tokens, h, d]
    sign = -1.0 if c["backward"] else 1.0
    return {"q": _rotate(s["q"], cos, sin, c, sign), "k": _rotate(s["k"], cos, sin, c, sign)}


def _places(s, n):
    """(sequence, index within its new tokens, position) of each new token."""
    tok = torch.arange(n, device=DEV)
    cu = s["cu"].long()
    seq = torch.searchsorted(cu, tok, right=True) - 1
    t = tok - cu[seq]
    return seq, t, s["kv_lens"].long()[seq] - (cu[seq + 1] - cu[seq]) + t


def _plain_append(s):
    c = s["case"]
    seq, t, pos = _places(s, s["q"].shape[0])
    cos, sin = (x[:, None] for x in _cos_sin(s, pos))
    ps = c["page_size"]
    page = s["page_table"].long()[seq, pos // ps]
    s["k_pages"][page, :, pos % ps] = _rotate(s["k"], cos, sin, c, 1.0)
    s["v_pages"][page, :, pos % ps] = s["v"]
    return {"q": _rotate(s["q"], cos, sin, c, 1.0), "k": s["k_pages"], "v": s["v_pages"]}


def _plain_attend(s):
    c = s["case"]
    h_q, h_kv, d, ps, n = c["h_q"], c["h_kv"], c["d"], c["page_size"], s["q"].shape[0]
    g, mq, n_seq = h_q // h_kv, s["max_q"], c["n_seq"]
    cu, kv = s["cu"].long(), s["kv_lens"].long()
    nq = cu[1:] - cu[:-1]
    local = torch.arange(mq, device=DEV)
    tok = (cu[:-1, None] + local).clamp(max=n - 1)                         # [n_seq, mq], padded
    q = s["q"].float()[tok].view(n_seq, mq, h_kv, g, d).permute(0, 2, 3, 1, 4).reshape(n_seq, h_kv, g * mq, d)
    pages = s["page_table"].long().clamp(min=0)
    at = torch.arange(pages.shape[1] * ps, device=DEV)
    here = at < kv[:, None]                                                # [n_seq, keys]
    k = s["k_pages"][pages].float().transpose(1, 2).reshape(n_seq, h_kv, -1, d)
    x = torch.matmul(q, k.transpose(-1, -2)).mul_(1.0 / math.sqrt(d)).view(n_seq, h_kv, g, mq, -1)
    del k
    last = kv[:, None] - nq[:, None] + local if c["causal"] else (kv[:, None] - 1).expand(n_seq, mq)
    sees = here[:, None, :] & (at <= last[:, :, None])                     # [n_seq, mq, keys]
    x = x.masked_fill_(~sees[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)        # rows that see no key
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    v = s["v_pages"][pages].float().transpose(1, 2).reshape(n_seq, h_kv, -1, d)
    v = torch.where(here[:, None, :, None], v, torch.zeros_like(v))
    o = torch.matmul(p.view(n_seq, h_kv, g * mq, -1), v).view(n_seq, h_kv, g, mq, d)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (top + torch.log(total))[..., 0]
    seq, t, _ = _places(s, n)
    return {"o": o[seq, :, :, t].reshape(n, h_q, d).to(torch.bfloat16), "lse": lse[seq, :, :, t].reshape(n, h_q).t().contiguous()}


def _plain_copy(s):
    s["pages"][:, s["pairs_dev"][:, 1]] = s["pages"][:, s["pairs_dev"][:, 0]]
    return s["pages"]


# ---------------------------------------------------------------- library ---

def _own(s):
    import attention_core_gb300 as ac
    c = s["case"]
    if c["op"] == "rope":
        f = ac.rope_bwd if c["backward"] else ac.rope_fwd
        q, k = f(s["q"], s["k"], s["table"], positions=s["pos"])
        return {"q": q, "k": k}
    if c["op"] == "append":
        q = ac.paged_append(s["batch"], s["q"], s["k"], s["v"], s["k_pages"], s["v_pages"], table=s["table"])
        return {"q": q, "k": s["k_pages"], "v": s["v_pages"]}
    if c["op"] == "attend":
        o, lse = ac.paged_fwd(s["batch"], s["q"], s["k_pages"], s["v_pages"])
        return {"o": o, "lse": lse}
    ac.page_copy(s["pages"], s["pairs"])
    return s["pages"]


def run(state):
    if own:
        return _own(state)
    return {"rope": _plain_rope, "append": _plain_append, "attend": _plain_attend, "copy": _plain_copy}[state["case"]["op"]](state)


# ------------------------------------------------------------------ exact ---

def _turn(x, pos, s, backward):
    """The definition, pair by pair, in 64 bits: x [..., d] with pos of the same leading shape (or broadcast to it)."""
    c = s["case"]
    y = x.double().clone()
    for i in range(c["rot"] // 2):
        a, b = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + c["rot"] // 2)
        w = pos.double() * s["freq"][i]
        if backward:
            w = -w
        z = torch.complex(x[..., a].double(), x[..., b].double()) * torch.polar(torch.full_like(w, s["mscale"]), w)
        y[..., a], y[..., b] = z.real, z.imag
    return y


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    if c["op"] == "copy":
        pages = s["pages"].double()
        for a, b in s["pairs"].tolist():
            pages[:, b] = s["pages"][:, a].double()
        return pages
    if c["op"] == "rope":
        pos = s["pos"][:, None]
        return {"q": _turn(s["q"], pos, s, c["backward"]), "k": _turn(s["k"], pos, s, c["backward"])}
    nq, nk = _lens(c)
    ps, start, table = c["page_size"], 0, s["page_table"].tolist()
    if c["op"] == "append":
        out = {"q": torch.empty(s["q"].shape, dtype=torch.float64, device=DEV), "k": s["k_pages"].double(), "v": s["v_pages"].double()}
        for i, (q, n) in enumerate(zip(nq, nk)):
            rows = slice(start, start + q)
            pos = torch.arange(n - q, n, device=DEV)
            out["q"][rows] = _turn(s["q"][rows], pos[:, None], s, False)
            page = torch.tensor(table[i], device=DEV)[pos.div(ps, rounding_mode="floor")]
            out["k"][page, :, pos.remainder(ps)] = _turn(s["k"][rows], pos[:, None], s, False)
            out["v"][page, :, pos.remainder(ps)] = s["v"][rows].double()
            start += q
        return out
    h_q, h_kv, d = c["h_q"], c["h_kv"], c["d"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros((h_q, s["q"].shape[0]), dtype=torch.float64, device=DEV)
    for i, (q, n) in enumerate(zip(nq, nk)):
        page = torch.tensor(table[i][: -(-n // ps)], device=DEV)
        k, v = (x[page].double().permute(1, 0, 2, 3).reshape(h_kv, -1, d)[:, :n] for x in (s["k_pages"], s["v_pages"]))
        hidden = None
        if c["causal"]:
            hidden = torch.arange(n, device=DEV)[None, :] > torch.arange(n - q, n, device=DEV)[:, None]
        for h in range(h_q):
            x = s["q"][start:start + q, h].double() @ k[h // (h_q // h_kv)].t() / math.sqrt(d)
            if hidden is not None:
                x = x.masked_fill(hidden, -math.inf)
            z = torch.logsumexp(x, -1)
            w = torch.exp(x - torch.where(torch.isfinite(z), z, torch.zeros_like(z))[:, None])
            o[start:start + q, h] = w @ v[h // (h_q // h_kv)]
            lse[h, start:start + q] = z
        start += q
    return {"o": o, "lse": lse}
