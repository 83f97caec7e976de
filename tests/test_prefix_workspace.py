"""What include/attn_core.h says of the shared-prefix workspace's size, beside
attn_core_paged_fwd's."""
import ctypes

import pytest

import attention_core_gb300 as ac


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("d", [64, 96, 128, 160])
@pytest.mark.parametrize("n_tokens,h_q,h_kv,n_seq,n_groups", [(0, 8, 8, 1, 1), (4, 64, 8, 4, 1), (64, 64, 8, 64, 3),
                                                             (5000, 16, 2, 300, 40)])
def test_the_size_that_is_stated(d, n_tokens, h_q, h_kv, n_seq, n_groups):
    dummy = (ctypes.c_int32 * 8)()
    at = ctypes.addressof(dummy)
    p = ac._CPagedParams(n_seq, n_tokens, h_q, h_kv, d, 16, 1000, 64, 1, 0.0, at, at, at, None, 0, 0)
    plain, prefix = ac.attn_core_paged_workspace_bytes(p), ac.attn_core_paged_prefix_workspace_bytes(p, n_groups)
    stated = 123000 * d + 8 * n_tokens * h_q * (d + 3) + 32 * (n_seq + n_groups)
    assert 0.97 * stated - 2048 <= prefix - plain <= 1.03 * stated + 2048
