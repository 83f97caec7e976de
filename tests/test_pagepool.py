"""The page pool on the host: pages are handed out once, shared by forks, copied
before a shared page is written, given back, and moved together, checked against
a cache of plain lists that holds every sequence's tokens."""
import random

import numpy as np
import pytest

from attention_core_gb300.pagepool import OutOfPages, PagePool


class Model:
    """A cache of plain values that follows the pool: what page p holds at row r."""

    def __init__(self, n_pages, page_size):
        self.pool = PagePool(n_pages, page_size)
        self.cells = [[None] * page_size for _ in range(n_pages)]
        self.want = {}

    def copy(self, pairs):
        targets = [b for _, b in pairs]
        assert len(set(targets)) == len(targets) and not set(targets) & {a for a, _ in pairs}
        old = [list(c) for c in self.cells]
        for a, b in pairs:
            self.cells[b] = list(old[a])

    def write(self, seq, values):
        at = self.pool.length(seq)
        self.copy(self.pool.extend(seq, len(values)))
        pages, ps = self.pool.pages(seq), self.pool.page_size
        for i, v in enumerate(values):
            self.cells[pages[(at + i) // ps]][(at + i) % ps] = v
        self.want[seq] = self.want.get(seq, []) + list(values)

    def check(self):
        pool, ps = self.pool, self.pool.page_size
        held = set()
        for seq, want in self.want.items():
            pages = pool.pages(seq)
            assert len(pages) == -(-len(want) // ps) and pool.length(seq) == len(want)
            assert [self.cells[pages[i // ps]][i % ps] for i in range(len(want))] == want
            held |= set(pages)
        assert pool.free_pages == pool.n_pages - len(held)
        seqs = list(self.want)
        if seqs:
            table, lens = pool.tables(seqs, pool.n_pages)
            assert table.dtype == lens.dtype == np.int32
            for i, s in enumerate(seqs):
                n = len(pool.pages(s))
                assert table[i, :n].tolist() == pool.pages(s) and (table[i, n:] == -1).all() and lens[i] == len(self.want[s])


@pytest.mark.parametrize("seed", range(6))
def test_random_life(seed):
    rng = random.Random(seed)
    m = Model(40, rng.choice([1, 3, 16]))
    for step in range(400):
        op, seqs = rng.random(), list(m.want)
        if not seqs or op < 0.1:
            m.want[m.pool.add()] = []
        elif op < 0.55:
            s = rng.choice(seqs)
            before = (m.pool.pages(s), m.pool.length(s), m.pool.free_pages)
            try:
                m.write(s, [(step, i) for i in range(rng.randint(0, 3 * m.pool.page_size))])
            except OutOfPages:
                assert before == (m.pool.pages(s), m.pool.length(s), m.pool.free_pages)
        elif op < 0.7:
            s = rng.choice(seqs)
            m.want[m.pool.fork(s)] = list(m.want[s])
        elif op < 0.8:
            s = rng.choice(seqs)
            m.pool.free(s)
            del m.want[s]
        elif op < 0.9:
            s = rng.choice(seqs)
            n = rng.randint(0, len(m.want[s]))
            m.pool.truncate(s, n)
            m.want[s] = m.want[s][:n]
        else:
            m.copy(m.pool.compact())
            used = m.pool.n_pages - m.pool.free_pages
            assert all(p < used for s in m.want for p in m.pool.pages(s))
        m.check()


def test_fork_shares_and_copies_on_write():
    m = Model(8, 4)
    a = m.pool.add()
    m.write(a, list("abcdef"))
    b = m.pool.fork(a)
    m.want[b] = list("abcdef")
    assert m.pool.free_pages == 6
    assert m.pool.extend(b, 0) == []                  # nothing is written: nothing is copied
    m.write(b, ["x"])
    assert m.pool.pages(a)[0] == m.pool.pages(b)[0] and m.pool.pages(a)[1] != m.pool.pages(b)[1]
    m.write(a, ["y"])                                 # the parent's page is its own again
    assert m.pool.free_pages == 5
    m.check()
    c = m.pool.fork(a)                                # full pages only: a new page, no copy
    m.want[c] = list(m.want[a])
    m.write(c, ["z", "w"])
    m.check()


def test_refusals():
    pool = PagePool(2, 4)
    s = pool.add()
    with pytest.raises(OutOfPages):
        pool.extend(s, 9)
    assert pool.extend(s, 8) == [] and pool.free_pages == 0
    t = pool.fork(s)
    with pytest.raises(OutOfPages):
        pool.extend(t, 1)
    with pytest.raises(ValueError):
        pool.extend(s, -1)
    with pytest.raises(ValueError):
        pool.truncate(s, 9)
    with pytest.raises(ValueError):
        pool.tables([s], 1)
    with pytest.raises(KeyError):
        pool.free(99)
    with pytest.raises(ValueError):
        PagePool(0, 4)
    pool.truncate(t, 7)                               # partly filled, shared, no page free for the copy
    with pytest.raises(OutOfPages):
        pool.extend(t, 1)
    pool.free(s)
    assert pool.extend(t, 1) == []                    # its own now


def test_a_fork_of_nothing_leaves_nothing():
    """Forking a sequence that is not there raises and adds no sequence."""
    pool = PagePool(4, 4)
    s = pool.add()
    pool.extend(s, 6)
    pool.free(s)
    with pytest.raises(KeyError):
        pool.fork(s)
    with pytest.raises(KeyError):
        pool.fork(99)
    for seq in range(s, s + 3):
        with pytest.raises(KeyError):
            pool.length(seq)
    assert pool.free_pages == 4 and pool.add() == s + 1
