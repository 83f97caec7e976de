"""Page copies inside a cache on the GPU: exact, in every plane, nothing else."""
import numpy as np
import pytest
import torch

import attention_core_gb300 as ac

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def _pages(planes, n, h, ps, d, seed=0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randint(-2**15, 2**15, (planes, n, h, ps, d), generator=gen, device=DEV, dtype=torch.int16).view(torch.bfloat16)


# (planes, pages, h_kv, page_size, d, copies): one unit of 16 bytes up to thousands of copies
@pytest.mark.parametrize("case", [(1, 2, 1, 1, 8, 1), (3, 40, 2, 16, 96, 17), (2, 9, 8, 64, 128, 4),
                                  (4, 5000, 1, 16, 64, 2400), (1, 70, 3, 32, 160, 33), (2, 4, 8, 256, 160, 2)])
def test_copies_are_exact(case):
    planes, n, h, ps, d, m = case
    x = _pages(planes, n, h, ps, d)
    order = np.random.RandomState(m).permutation(n)
    pairs = np.stack((order[:m], order[m:2 * m]), 1)
    want = x.clone()
    want[:, torch.from_numpy(pairs[:, 1]).to(DEV)] = x[:, torch.from_numpy(pairs[:, 0]).to(DEV)]
    ac.page_copy(x, pairs)
    assert torch.equal(x.view(torch.int16), want.view(torch.int16))


def test_one_source_to_many_and_single_plane():
    x = _pages(1, 50, 2, 16, 64)[0]
    want = x.clone()
    want[10:45] = x[3]
    ac.page_copy(x, [(3, i) for i in range(10, 45)])
    assert torch.equal(x.view(torch.int16), want.view(torch.int16))


def test_empty_list():
    x = _pages(1, 4, 1, 16, 64)
    before = x.clone()
    ac.page_copy(x, [])
    ac.page_copy(x, np.zeros((0, 2), np.int32))
    assert torch.equal(x.view(torch.int16), before.view(torch.int16))


def test_far_pages():
    """Bytes past 2^32 of a plane."""
    x = torch.zeros(1, (1 << 32) // (16 * 128 * 2 * 8) + 10, 8, 16, 128, dtype=torch.bfloat16, device=DEV)
    n = x.shape[1]
    x[0, n - 1] = 3.0
    ac.page_copy(x, [(n - 1, n - 2), (n - 1, 5)])
    assert (x[0, n - 2] == 3).all() and (x[0, 5] == 3).all() and (x[0, n - 3] == 0).all() and (x[0, 6] == 0).all()


def test_refusals():
    x = _pages(2, 8, 1, 16, 64)
    before = x.clone()
    for pairs in ([(0, 8)], [(-1, 2)], [(0, 0)], [(0, 1), (2, 1)], [(0, 1), (1, 2)]):
        with pytest.raises(ac.AttnCoreError) as e:
            ac.page_copy(x, pairs)
        assert e.value.code == ac.ERR_INVALID_ARG
    with pytest.raises(ValueError):
        ac.page_copy(x, [(0, 1 << 40)])
    with pytest.raises(ValueError):
        ac.page_copy(x, [0, 1])
    with pytest.raises(ValueError):
        ac.page_copy(x, [(0.5, 1.0)])
    with pytest.raises(ValueError):
        ac.page_copy(x, torch.zeros(1, 2, dtype=torch.int32, device=DEV))
    with pytest.raises(ValueError):
        ac.page_copy(x.transpose(0, 1), [(0, 1)])
    assert torch.equal(x.view(torch.int16), before.view(torch.int16))
