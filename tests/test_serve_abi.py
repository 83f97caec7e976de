"""Host-side checks of the rotary, paged-cache and page-copy entry points (no
GPU): arguments are refused before the device is touched, and the frequency
table is the definition's."""
import ctypes
import math

import numpy as np
import pytest

import attention_core_gb300 as ac
from attention_core_gb300 import build as lib_build
from tests.serve_ref import ORIGINAL, frequencies

FAKE = 0x7f0000000000   # 16-byte aligned, never dereferenced: validation fails first


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lib_build.build()
    return ac.load_library()


@pytest.mark.parametrize("rot", [8, 24, 40, 64, 128, 256])
@pytest.mark.parametrize("scaling,factor", [("none", 1.0), ("linear", 4.0), ("bands", 8.0), ("yarn", 4.0), ("yarn", 32.0)])
def test_table_holds_the_definition(rot, scaling, factor):
    """A frequency is an fp64 value (a few 2^-53 off the definition's: pow, a
    product and a quotient, 2^-51 together) cut to a 64-bit fraction of a turn:
    an absolute 2^-64 turns more, which is what is left of the slow pairs' (the
    slowest here turns 2^-26 times per position, so 2^-38 of it)."""
    t = ac.rope_table(256, rot_dim=rot, scaling=scaling, factor=factor, original_len=ORIGINAL)
    f, m = frequencies(rot, scaling=scaling, factor=factor)
    got = np.array([t.turns[i] / 2.0 ** 64 * 2 * math.pi for i in range(rot // 2)])
    assert np.all(np.abs(got - np.array(f)) <= 2.0 ** -46 * np.array(f) + 2 * math.pi * 2.0 ** -64)
    assert abs(t.mscale - m) <= 2.0 ** -24 * m
    assert (t.d, t.rot_dim, t.interleaved) == (256, rot, 0)


def test_table_defaults_and_whole_turns():
    t = ac.rope_table(512)
    assert t.rot_dim == 256
    t = ac.rope_table(64, interleaved=True, mscale=0.5)
    assert (t.rot_dim, t.interleaved, t.mscale) == (64, 1, 0.5)
    # a factor below 1 speeds up: the first pair turns 10 rad per position, taken modulo a turn
    t = ac.rope_table(64, scaling="linear", factor=0.1)
    assert abs(t.turns[0] / 2.0 ** 64 - (10 / (2 * math.pi)) % 1) < 2.0 ** -40


@pytest.mark.parametrize("kw", [dict(d=0), dict(d=12), dict(d=520), dict(d=64, rot_dim=72), dict(d=64, rot_dim=12),
                                dict(d=64, rot_dim=-8), dict(d=512, rot_dim=264), dict(d=64, base=1.0),
                                dict(d=64, base=-5.0), dict(d=64, base=math.nan), dict(d=64, factor=-1.0),
                                dict(d=64, factor=math.inf), dict(d=64, scaling="bands"),
                                dict(d=64, scaling="yarn", original_len=math.nan),
                                dict(d=64, scaling="bands", original_len=10, low_freq=4, high_freq=4),
                                dict(d=64, scaling="yarn", original_len=10, beta_fast=1, beta_slow=2),
                                dict(d=64, mscale=-1.0), dict(d=64, mscale=math.nan)])
def test_table_refusals(kw):
    with pytest.raises(ac.AttnCoreError) as e:
        ac.rope_table(**kw)
    assert e.value.code == ac.ERR_INVALID_ARG


def test_unknown_scaling():
    with pytest.raises(ValueError):
        ac.rope_table(64, scaling="quadratic")


def _rope(**kw):
    d = dict(b=2, s=10, h_q=4, h_kv=2, q_stride=(4 * 640, 640, 64), k_stride=(2 * 640, 640, 64),
             yq_stride=(4 * 640, 640, 64), yk_stride=(2 * 640, 640, 64), pos0=0, positions=None)
    d.update(kw)
    p = ac._CRopeParams()
    for n, v in d.items():
        if n.endswith("stride"):
            getattr(p, n)[:] = v
        else:
            setattr(p, n, v)
    return p


@pytest.mark.parametrize("fn", ["attn_core_rope_fwd", "attn_core_rope_bwd"])
def test_rope_refusals(fn):
    f, t = getattr(ac, fn), ac.rope_table(64)
    q, k, yq, yk = (FAKE + i * (1 << 20) for i in range(4))

    def rc(p, ptr=(q, k, yq, yk), table=t):
        return f(p, table, *ptr, 0)
    for kw in (dict(b=0), dict(s=-1), dict(h_q=-1), dict(h_q=0, h_kv=0), dict(b=1 << 16, s=1 << 16),
               dict(q_stride=(-8, 640, 64)), dict(yq_stride=(4 * 640, 640, 0)), dict(yk_stride=(0, 640, 64)),
               dict(yq_stride=(640, 640, 64)), dict(yq_stride=(4 * 640, 632, 64)), dict(yq_stride=(1 << 43, 640, 64))):
        assert rc(_rope(**kw)) == ac.ERR_INVALID_ARG, kw
    assert rc(_rope(h_q=40000, h_kv=30000)) == ac.ERR_UNSUPPORTED
    for kw in (dict(q_stride=(4 * 640, 641, 64)), dict(yk_stride=(2 * 640, 640, 68)), dict(positions=FAKE + 2)):
        assert rc(_rope(**kw)) == ac.ERR_MISALIGNED, kw
    assert rc(_rope(), (q + 2, k, yq, yk)) == ac.ERR_MISALIGNED
    assert rc(_rope(), (q, k, yq, yk + 8)) == ac.ERR_MISALIGNED
    assert rc(_rope(), (0, k, yq, yk)) == ac.ERR_INVALID_ARG
    assert rc(_rope(), (q, k, yq, 0)) == ac.ERR_INVALID_ARG
    assert rc(_rope(q_stride=(4 * 640, 0, 64)), (q, k, q, yk)) == ac.ERR_INVALID_ARG       # in place elsewhere
    for ptr in ((q, k, yq, yq), (q, k, k, yk), (q, k, yq, q), (q, k, k, q)):               # one tensor in two roles
        assert rc(_rope(), ptr) == ac.ERR_INVALID_ARG
    assert rc(_rope(), table=None) == ac.ERR_INVALID_ARG
    assert rc(None) == ac.ERR_INVALID_ARG
    bad = ac.rope_table(64)
    bad.rot_dim = 72
    assert rc(_rope(), table=bad) == ac.ERR_INVALID_ARG
    assert rc(_rope(s=0)) == ac.OK                                                         # nothing to do
    assert rc(_rope(s=0, h_q=0), (0, k, 0, yk)) == ac.OK


def _paged(**kw):
    d = dict(n_seq=2, n_tokens=5, h_q=4, h_kv=2, d=64, page_size=16, n_pages=10, max_pages=4, causal=1, scale=0.0,
             cu_seqlens_q=FAKE, kv_lens=FAKE + 64, page_table=FAKE + 128, dev_status=None, flags=0, wait_timeout_ms=0)
    d.update(kw)
    return ac._CPagedParams(**d)


PAGED_INVALID = [dict(n_seq=0), dict(n_tokens=-1), dict(h_q=0), dict(h_q=3), dict(h_kv=0), dict(d=0), dict(n_pages=0),
                 dict(max_pages=0), dict(causal=2), dict(scale=math.nan), dict(scale=math.inf), dict(cu_seqlens_q=None),
                 dict(kv_lens=None), dict(page_table=None), dict(n_pages=1 << 30, h_kv=4),
                 dict(max_pages=1 << 28), dict(n_tokens=1 << 30), dict(flags=1)]
PAGED_UNSUPPORTED = [dict(d=72), dict(max_pages=1 << 20, n_tokens=1 << 29, h_q=1, h_kv=1, page_size=256), dict(page_size=8), dict(page_size=48), dict(page_size=512), dict(h_q=258, h_kv=2),
                     dict(h_q=30000, h_kv=30000)]


def test_paged_refusals():
    q, kp, vp, o, lse, ws = (FAKE + i * (1 << 24) for i in range(1, 7))
    big = 1 << 40

    def fwd(p, ptr=(q, kp, vp, o, lse, ws), n=big):
        return ac.attn_core_paged_fwd(p, *ptr, n, 0)

    def app(p, ptr=(q, kp, vp), st=None, out=(o, kp, vp), t=None):
        return ac.attn_core_paged_append(p, t, *ptr, st, *out, 0)
    for f in (fwd, app):
        for kw in PAGED_INVALID:
            assert f(_paged(**kw)) == ac.ERR_INVALID_ARG, kw
        for kw in PAGED_UNSUPPORTED:
            assert f(_paged(**kw)) == ac.ERR_UNSUPPORTED, kw
        assert f(_paged(kv_lens=FAKE + 2)) == ac.ERR_MISALIGNED
        assert f(None) == ac.ERR_INVALID_ARG
        assert f(_paged(n_tokens=0)) == ac.OK
    for i in range(6):
        ptr = [q, kp, vp, o, lse, ws]
        ptr[i] = 0
        assert fwd(_paged(), tuple(ptr)) == ac.ERR_INVALID_ARG
        ptr[i] = FAKE + 8
        assert fwd(_paged(), tuple(ptr)) == ac.ERR_MISALIGNED
    need = ac.attn_core_paged_workspace_bytes(_paged())
    assert need > 0
    assert fwd(_paged(), n=need - 1) == ac.ERR_WORKSPACE_TOO_SMALL
    for kw in PAGED_INVALID + PAGED_UNSUPPORTED:
        assert ac.attn_core_paged_workspace_bytes(_paged(**kw)) == 0
    assert app(_paged(), (0, kp, vp)) == ac.ERR_INVALID_ARG            # q_out without q
    assert app(_paged(), (q, 0, vp)) == ac.ERR_INVALID_ARG
    assert app(_paged(), out=(o, 0, vp)) == ac.ERR_INVALID_ARG
    assert app(_paged(), (q + 4, kp, vp)) == ac.ERR_MISALIGNED
    assert app(_paged(), st=(256, 130, 128)) == ac.ERR_MISALIGNED
    assert app(_paged(), st=(256, -128, 128)) == ac.ERR_INVALID_ARG
    assert app(_paged(), st=(512, 128, 128), out=(q, kp, vp)) == ac.ERR_INVALID_ARG    # in place, not packed
    assert app(_paged(), out=(o, kp, kp)) == ac.ERR_INVALID_ARG
    assert app(_paged(), (q, o, vp)) == ac.ERR_INVALID_ARG              # q_out over the new keys
    assert fwd(_paged(), (q, kp, vp, q, lse, ws)) == ac.ERR_INVALID_ARG
    assert app(_paged(), t=ac.rope_table(96)) == ac.ERR_INVALID_ARG
    assert app(_paged(flags=ac.FLAG_TEST_WAIT_TIMEOUT)) == ac.ERR_INVALID_ARG


def _copy(pairs, planes=2, stride=1 << 20, n_pages=100, page=256, base=FAKE):
    a = np.array(pairs, dtype=np.int32).reshape(-1, 2)
    return ac.attn_core_page_copy(base, planes, stride, n_pages, page, a.ctypes.data if a.size else 0, len(a), 0)


def test_page_copy_refusals():
    many = [(i, 50 + i) for i in range(40)]
    for pairs in ([(0, 100)], [(100, 0)], [(-1, 0)], [(3, 3)], [(1, 2), (3, 2)], [(1, 2), (2, 3)],
                  many + [(0, 50)], many + [(55, 99)], [(0, 1)] * 101):
        assert _copy(pairs) == ac.ERR_INVALID_ARG, pairs[-2:]
    assert _copy([(0, 1)], planes=0) == ac.ERR_INVALID_ARG
    assert _copy([(0, 1)], n_pages=0) == ac.ERR_INVALID_ARG
    assert _copy([(0, 1)], page=0) == ac.ERR_INVALID_ARG
    assert _copy([(0, 1)], stride=256 * 99) == ac.ERR_INVALID_ARG
    assert _copy([(0, 1)], base=0) == ac.ERR_INVALID_ARG
    assert _copy([(0, 1)], page=264) == ac.ERR_MISALIGNED
    assert _copy([(0, 1)], base=FAKE + 8) == ac.ERR_MISALIGNED
    assert _copy([(0, 1)], stride=(1 << 20) + 8) == ac.ERR_MISALIGNED
    assert _copy([(0, 1)], planes=1 << 17) == ac.ERR_UNSUPPORTED
    assert ac.attn_core_page_copy(FAKE, 1, 1 << 20, 4, 256, 0, 3, 0) == ac.ERR_INVALID_ARG
    assert _copy([]) == ac.OK


def test_status_text():
    assert "table" in ac.attn_core_strerror(ac.ERR_DEVICE_TABLE)


def test_structures_match_the_header():
    """The binding's structures have the C ones' layout (fields and paddings as
    the header's types give them)."""
    assert ctypes.sizeof(ac.RopeTable) == 16 + 128 * 8
    assert ctypes.sizeof(ac._CRopeConfig) == 16 + 8 * 8
    assert ctypes.sizeof(ac._CRopeParams) == 16 + 4 * 24 + 8 + 8
    assert ctypes.sizeof(ac._CPagedParams) == 40 + 4 * 8 + 8


def test_sizes_past_32_bits_are_refused():
    """The binding cuts no size or position to the structures' 32 bits."""
    import torch
    for kw in (dict(d=2 ** 32 + 64), dict(d=64, rot_dim=2 ** 32 + 8), dict(d=-2 ** 32 + 64)):
        with pytest.raises(ValueError, match="32 bits"):
            ac.rope_table(**kw)
    t = ac.rope_table(64)
    for pos0 in (2 ** 31, -2 ** 31 - 1, 2 ** 32):
        for f in (ac.rope_fwd, ac.rope_bwd):
            with pytest.raises(ValueError, match="pos0"):
                f(torch.zeros(2, 1, 64, dtype=torch.bfloat16), None, t, pos0=pos0)
    cu, lens, table = (torch.zeros(n, dtype=torch.int32) for n in (2, 1, 4))
    sizes = dict(n_tokens=1, h_q=2, h_kv=1, d=64, page_size=16, n_pages=4)
    for name in ("n_tokens", "h_q", "h_kv", "d", "page_size", "n_pages", "flags", "wait_timeout_ms"):
        with pytest.raises(ValueError, match=name):
            ac.PagedBatch(cu, lens, table.view(1, 4), **{**sizes, name: 2 ** 32 + sizes.get(name, 0)})


def test_an_output_without_its_input_is_refused():
    """out_q or out_k beside a missing q or k would come back as it was."""
    import torch
    t, x = ac.rope_table(64), torch.zeros(2, 1, 64, dtype=torch.bfloat16)
    for f in (ac.rope_fwd, ac.rope_bwd):
        with pytest.raises(ValueError, match="out_q without q"):
            f(None, x, t, out_q=x.clone())
        with pytest.raises(ValueError, match="out_k without k"):
            f(x, None, t, out_k=x.clone())
