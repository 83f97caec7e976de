"""Host-side checks of the shared-prefix, gathered-weight and eviction entry points
(no GPU): arguments are refused before the device is touched."""
import ctypes
import math

import pytest

import attention_core_gb300 as ac
from attention_core_gb300 import build as lib_build
from tests.test_serve_abi import FAKE, PAGED_INVALID, PAGED_UNSUPPORTED, _paged


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lib_build.build()
    return ac.load_library()


BIG = 1 << 40
Q, KP, VP, O, LSE, WS, W, W2, KEPT = (FAKE + i * (1 << 24) for i in range(1, 10))


def _prefix(p, groups=1, starts=FAKE + 256, pages=FAKE + 512, ptr=(Q, KP, VP, O, LSE, WS), n=BIG):
    return ac.attn_core_paged_prefix_fwd(p, groups, starts, pages, *ptr, n, 0)


def _weights(p, ptr=(Q, KP, LSE), decay=1.0, w=(W, W2), ws=WS, n=BIG):
    return ac.attn_core_paged_weights(p, *ptr, decay, *w, ws, n, 0)


def _evict(p, keep=FAKE + 1024, first=0, recent=0, out=0, pages=(KP, VP), w=(W, W2, KEPT), ws=WS, n=BIG):
    return ac.attn_core_paged_evict(p, keep, first, recent, out, *pages, *w, ws, n, 0)


@pytest.mark.parametrize("f", [_prefix, _weights, _evict])
def test_sizes(f):
    for kw in PAGED_INVALID:
        assert f(_paged(**kw)) == ac.ERR_INVALID_ARG, kw
    for kw in PAGED_UNSUPPORTED:
        assert f(_paged(**kw)) == ac.ERR_UNSUPPORTED, kw
    assert f(_paged(kv_lens=FAKE + 2)) == ac.ERR_MISALIGNED
    assert f(None) == ac.ERR_INVALID_ARG


def test_prefix():
    assert _prefix(_paged(n_tokens=0)) == ac.OK
    for groups in (0, -1, 3):                          # of two sequences
        assert _prefix(_paged(), groups) == ac.ERR_INVALID_ARG
        assert ac.attn_core_paged_prefix_workspace_bytes(_paged(), groups) == 0
    assert _prefix(_paged(), starts=0) == ac.ERR_INVALID_ARG
    assert _prefix(_paged(), pages=0) == ac.ERR_INVALID_ARG
    assert _prefix(_paged(), starts=FAKE + 2) == ac.ERR_MISALIGNED
    assert _prefix(_paged(), pages=FAKE + 1) == ac.ERR_MISALIGNED
    for i in range(6):
        ptr = [Q, KP, VP, O, LSE, WS]
        ptr[i] = 0
        assert _prefix(_paged(), ptr=ptr) == ac.ERR_INVALID_ARG
        ptr[i] = FAKE + 8
        assert _prefix(_paged(), ptr=ptr) == ac.ERR_MISALIGNED
    assert _prefix(_paged(), ptr=(Q, KP, VP, Q, LSE, WS)) == ac.ERR_INVALID_ARG
    need = ac.attn_core_paged_prefix_workspace_bytes(_paged(), 2)
    plain = ac.attn_core_paged_workspace_bytes(_paged())
    assert need > plain and _prefix(_paged(), 2, n=need - 1) == ac.ERR_WORKSPACE_TOO_SMALL
    # two fp32 rows of d values, their LSEs and records for each new token and head
    more = ac.attn_core_paged_prefix_workspace_bytes(_paged(n_tokens=1005), 2)
    assert abs(more - need - 1000 * 4 * 2 * (64 * 4 + 4 + 8)) <= 4 * 256
    assert _prefix(_paged(n_seq=2**31 - 1), 2**31 - 1) == ac.ERR_UNSUPPORTED


def test_weights():
    assert _weights(_paged(n_tokens=0)) == ac.OK
    for decay in (math.nan, math.inf, -0.5):
        assert _weights(_paged(), decay=decay) == ac.ERR_INVALID_ARG
    for i in range(3):
        ptr = [Q, KP, LSE]
        ptr[i] = 0
        assert _weights(_paged(), ptr) == ac.ERR_INVALID_ARG
        ptr[i] = FAKE + 8
        assert _weights(_paged(), ptr) == ac.ERR_MISALIGNED
    for w in ((0, W), (W, 0), (W, Q), (W, KP), (W, LSE)):
        assert _weights(_paged(), w=w) == ac.ERR_INVALID_ARG
    assert _weights(_paged(), w=(W + 4, W)) == ac.ERR_MISALIGNED
    assert _weights(_paged(), w=(W, W + 8)) == ac.ERR_MISALIGNED
    assert _weights(_paged(), ws=0) == ac.ERR_INVALID_ARG
    assert _weights(_paged(), ws=FAKE + 64) == ac.ERR_MISALIGNED
    need = ac.attn_core_paged_weights_workspace_bytes(_paged())
    assert 0 < need <= ac.attn_core_paged_workspace_bytes(_paged())      # the attention's serves
    assert _weights(_paged(), n=need - 1) == ac.ERR_WORKSPACE_TOO_SMALL


def test_evict():
    for kw in (dict(first=-1), dict(recent=-1), dict(keep=0), dict(pages=(0, VP)), dict(pages=(KP, 0)),
               dict(pages=(KP, KP)), dict(w=(0, W2, KEPT)), dict(w=(W, 0, KEPT)), dict(w=(W, W2, 0)),
               dict(w=(W, W2, W)), dict(w=(W, W2, W2)), dict(ws=0)):
        assert _evict(_paged(), **kw) == ac.ERR_INVALID_ARG, kw
    for kw in (dict(keep=FAKE + 2), dict(out=FAKE + 1), dict(pages=(KP + 8, VP)), dict(w=(W + 4, W2, KEPT)),
               dict(w=(W, W2, KEPT + 4)), dict(ws=FAKE + 128)):
        assert _evict(_paged(), **kw) == ac.ERR_MISALIGNED, kw
    need = ac.attn_core_paged_evict_workspace_bytes(_paged())
    assert need > 0 and _evict(_paged(), n=need - 1) == ac.ERR_WORKSPACE_TOO_SMALL
    # more keys or lines than it counts in 32 bits
    for kw in (dict(max_pages=(1 << 26) + 1), dict(n_seq=1 << 20, max_pages=1 << 16), dict(n_seq=1 << 28)):
        assert _evict(_paged(**kw)) == ac.ERR_UNSUPPORTED, kw
        assert ac.attn_core_paged_evict_workspace_bytes(_paged(**kw)) == 0


def test_the_binding_refuses_what_is_not_on_the_gpu():
    import torch
    cu, lens, table = (torch.zeros(n, dtype=torch.int32) for n in (2, 1, 4))
    with pytest.raises(ValueError):
        ac.PagedBatch(cu, lens, table.view(1, 4), n_tokens=1, h_q=2, h_kv=1, d=64, page_size=16, n_pages=4)


def test_structures_have_not_changed():
    """The batch's structure is the attention's: what is new comes as arguments."""
    assert ctypes.sizeof(ac._CPagedParams) == 40 + 4 * 8 + 8
