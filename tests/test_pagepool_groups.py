"""Which sequences share their first pages, and the pages of sequences that drop
keys (host side, no GPU)."""
import random

import numpy as np
import pytest

from attention_core_gb300.pagepool import OutOfPages, PagePool


def consistent(pool):
    """Every page is free or held by as many sequences as it says."""
    count = [0] * pool.n_pages
    for p in pool._pages.values():
        for x in p:
            count[x] += 1
    assert count == pool._users
    assert sorted(pool._free) == [i for i, c in enumerate(count) if c == 0]


def tree(pool, lengths):
    a = pool.add()
    pool.extend(a, lengths[0])
    return a


def test_groups():
    pool = PagePool(400, 16)
    a = tree(pool, [160])                       # ten pages
    b, c = pool.fork(a), pool.fork(a)
    for s in (a, b, c):
        pool.extend(s, 5)
    x = tree(pool, [64])
    y = pool.fork(x)
    lone = tree(pool, [40])
    starts, pages = pool.groups([a, b, c, lone, x, y])
    assert starts.tolist() == [0, 3, 4, 6] and pages.tolist() == [10, 0, 4]
    assert starts.dtype == pages.dtype == np.int32
    assert [v.tolist() for v in pool.groups([lone])] == [[0, 1], [0]]
    assert [v.tolist() for v in pool.groups([a, x, b])] == [[0, 1, 2, 3], [0, 0, 0]]      # neighbours only
    with pytest.raises(ValueError):
        pool.groups([])


def test_nested_groups_take_what_saves_more():
    pool = PagePool(4000, 16)
    system = tree(pool, [32])                   # two pages that everyone shares
    doc = pool.fork(system)
    pool.extend(doc, 1600)                      # and a hundred that some do
    readers = [pool.fork(doc) for _ in range(3)]
    others = [pool.fork(system) for _ in range(4)]
    for s in readers + others:
        pool.extend(s, 3)
    starts, pages = pool.groups(others + readers)
    assert starts.tolist() == [0, 4, 7] and pages.tolist() == [2, 102]
    # a short document among many users of the system prompt: one group
    pool2 = PagePool(4000, 16)
    system = tree(pool2, [160])
    doc = pool2.fork(system)
    pool2.extend(doc, 16)
    batch = [pool2.fork(doc), pool2.fork(doc)] + [pool2.fork(system) for _ in range(8)]
    starts, pages = pool2.groups(batch)
    assert starts.tolist() == [0, 10] and pages.tolist() == [10]


def test_groups_cover_and_agree():
    rng = random.Random(3)
    for _ in range(200):
        pool = PagePool(3000, 16)
        seqs = [tree(pool, [rng.randint(0, 100)])]
        for _ in range(rng.randint(0, 30)):
            s = pool.fork(rng.choice(seqs)) if rng.random() < 0.8 else pool.add()
            pool.extend(s, rng.randint(0, 60))
            seqs.append(s)
        rng.shuffle(seqs)
        starts, pages = pool.groups(seqs)
        assert starts[0] == 0 and starts[-1] == len(seqs) and (np.diff(starts) > 0).all()
        for g, n in enumerate(pages):
            rows = {tuple(pool.pages(s)[:n]) for s in seqs[starts[g]:starts[g + 1]]}
            assert len(rows) == 1 and len(rows.pop()) == n


def test_many_forks_of_one_prompt():
    pool = PagePool(5000, 16)
    a = tree(pool, [320])
    seqs = [a] + [pool.fork(a) for _ in range(3000)]
    starts, pages = pool.groups(seqs)
    assert starts.tolist() == [0, 3001] and pages.tolist() == [20]


def test_shrink_within_own_pages():
    pool = PagePool(20, 16)
    a, b = tree(pool, [100]), tree(pool, [30])
    before, free = pool.pages(a), pool.free_pages
    out = pool.shrink([a, b], [40, 30], 8)
    assert out.dtype == np.int32 and out[0].tolist() == before[:3] + [-1] * 5
    assert pool.pages(a) == before[:3] and pool.length(a) == 40 and pool.length(b) == 30
    assert pool.free_pages == free + 4
    consistent(pool)
    pool.shrink([a], [0], 1)
    assert pool.pages(a) == [] and pool.length(a) == 0
    consistent(pool)


def test_shrink_leaves_shared_pages():
    pool = PagePool(40, 16)
    a = tree(pool, [160])
    b = pool.fork(a)
    pool.extend(b, 32)                          # two pages of its own
    old_a, old_b = pool.pages(a), pool.pages(b)
    # both at once: neither writes into a page that the other reads
    out = pool.shrink([a, b], [64, 170], 12)
    named = set(old_a) | set(old_b)
    assert not named & set(out[0, :4].tolist())
    assert not named & set(out[1, :10].tolist()) and out[1, 10] == old_b[10]
    assert len(set(out[out >= 0].tolist())) == 4 + 11
    consistent(pool)
    assert pool.free_pages == 40 - 15
    # one alone: the other keeps its pages
    c = pool.fork(b)
    keep = pool.pages(c)
    out = pool.shrink([b], [20], 12)
    assert pool.pages(c) == keep and not set(out[0, :2].tolist()) & set(keep)
    consistent(pool)


def test_shrink_refusals_change_nothing():
    pool = PagePool(12, 16)
    a = tree(pool, [160])
    b = pool.fork(a)
    state = (pool.pages(a), pool.pages(b), pool.free_pages)
    with pytest.raises(OutOfPages):
        pool.shrink([a, b], [160, 160], 10)     # twenty pages wanted
    with pytest.raises(OutOfPages):
        pool.shrink([a], [33], 10)              # three of two
    for args in (([a, a], [1, 1], 10), ([a], [1, 2], 10), ([a], [161], 11), ([a], [-1], 10), ([a], [160], 9)):
        with pytest.raises(ValueError):
            pool.shrink(*args)
    assert state == (pool.pages(a), pool.pages(b), pool.free_pages)
    pool.shrink([a], [32], 10)
    consistent(pool)
