"""How long what ``PagePool.groups`` found holds: tokens that are added change nothing,
and a fork's copied page, a truncation or a shrink takes columns away."""
import random

import numpy as np
import pytest

from attention_core_gb300.pagepool import OutOfPages, PagePool


def agree(pool, seqs, starts, shared):
    """No count reaches into columns where the group's rows differ."""
    for g, n in enumerate(shared):
        rows = [pool.pages(s) for s in seqs[starts[g]:starts[g + 1]]]
        for r in rows[1:]:
            m = min(len(r), len(rows[0]), int(n))
            if r[:m] != rows[0][:m]:
                return False
    return True


@pytest.mark.parametrize("seed", range(20))
def test_added_tokens_change_nothing(seed):
    rng = random.Random(seed)
    pool = PagePool(400, 4)
    seqs = [pool.add()]
    pool.extend(seqs[0], rng.randint(1, 40))
    for _ in range(rng.randint(2, 9)):
        seqs.append(pool.fork(rng.choice(seqs)))
        pool.extend(rng.choice(seqs), rng.randint(0, 9))
    rng.shuffle(seqs)
    found = pool.groups(seqs)
    asked = 1
    for _ in range(60):
        try:
            copies = pool.extend(rng.choice(seqs), rng.randint(0, 5))
        except OutOfPages:
            break
        if copies:
            found, asked = pool.groups(seqs), asked + 1
        again = pool.groups(seqs)
        assert all(np.array_equal(a, b) for a, b in zip(found, again))
        assert agree(pool, seqs, *found)
    assert asked < 20


def test_what_takes_columns_away():
    pool = PagePool(60, 4)
    a = pool.add()
    pool.extend(a, 18)                                    # four whole pages and half of a fifth
    b = pool.fork(a)
    seqs = [a, b]
    found = pool.groups(seqs)
    assert found[1].tolist() == [5]
    assert pool.extend(b, 1)                              # writes into the fifth: copied
    assert not agree(pool, seqs, *found) and pool.groups(seqs)[1].tolist() == [4]
    found = pool.groups(seqs)
    pool.shrink([b], [9], 10)                             # every page that b keeps is its own now
    assert not agree(pool, seqs, *found) and pool.groups(seqs)[1].tolist() == [0, 0]
    c = pool.fork(a)
    seqs = [a, c]
    found = pool.groups(seqs)
    pool.truncate(c, 6)
    pool.extend(c, 20)
    assert not agree(pool, seqs, *found) and pool.groups(seqs)[1].tolist() == [1]
