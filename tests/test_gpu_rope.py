"""Rotary positions on the GPU against the 64-bit definition: layouts, strides,
part of the head, scalings, far positions, the backward pass, in place."""
import math

import pytest
import torch

import attention_core_gb300 as ac
from tests.serve_ref import BF16, ORIGINAL, frequencies, rope_tolerance, rotate

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def _randn(*shape, seed=0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(shape, generator=gen, device=DEV).to(torch.bfloat16)


def _near(got, x, pos, rot, **kw):
    y, size = rotate(x, pos, rot, **kw)
    err, tol = (got.double() - y).abs(), rope_tolerance(y, size, rot)
    assert (err <= tol).all(), float((err - tol).max())


# (b, h_q, h_kv, s, d, rot, interleaved, scaling, factor)
CASES = [
    (1, 2, 2, 128, 64, 64, False, "none", 1.0),
    (2, 3, 1, 1, 96, 96, False, "linear", 2.0),
    (1, 8, 2, 77, 128, 64, True, "bands", 8.0),
    (2, 5, 5, 33, 160, 40, False, "yarn", 4.0),      # a quarter of the head: 4-pair units
    (1, 1, 1, 1000, 96, 24, False, "none", 1.0),
    (3, 2, 1, 19, 160, 8, True, "linear", 4.0),
    (1, 16, 16, 517, 512, 256, False, "bands", 4.0),
    (1, 64, 8, 2500, 128, 128, True, "yarn", 8.0),
    (1, 1, 1, 1, 8, 8, True, "none", 1.0),           # the smallest head, one token
    (3, 1, 2, 70, 16, 16, False, "none", 1.0),
    (1, 300, 1, 2, 32, 8, False, "linear", 2.0),     # more heads than tokens
]


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_rope_matches_definition(case, backward, packed):
    b, hq, hkv, s, d, rot, inter, scaling, factor = case
    t = ac.rope_table(d, rot_dim=rot, interleaved=inter, scaling=scaling, factor=factor, original_len=ORIGINAL)
    gen = torch.Generator(device=DEV).manual_seed(s)
    pos = torch.randint(-50, 1 << 20, (b, s), generator=gen, device=DEV, dtype=torch.int32)
    if packed:
        q, k, lead = _randn(b * s, hq, d, seed=1), _randn(b * s, hkv, d, seed=2), pos.reshape(-1, 1)
    else:
        q, k, lead = _randn(b, hq, s, d, seed=1), _randn(b, hkv, s, d, seed=2), pos[:, None]
    f = ac.rope_bwd if backward else ac.rope_fwd
    yq, yk = f(q, k, t, positions=pos)
    kw = dict(interleaved=inter, backward=backward, scaling=scaling, factor=factor)
    _near(yq, q, lead, rot, **kw)
    _near(yk, k, lead, rot, **kw)


def test_default_positions_in_place_and_strides():
    """Slices of one fused projection, rotated in place; token t is at pos0 + t."""
    n, hq, hkv, d = 300, 6, 2, 128
    qkv = _randn(n, (hq + 2 * hkv) * d)
    before = qkv.clone()
    q = qkv[:, :hq * d].view(n, hq, d)
    k = qkv[:, hq * d:(hq + hkv) * d].view(n, hkv, d)
    t = ac.rope_table(d)
    ac.rope_fwd(q, k, t, pos0=5, out_q=q, out_k=k)
    pos = 5 + torch.arange(n, device=DEV)[:, None]
    _near(q, before[:, :hq * d].view(n, hq, d), pos, d)
    _near(k, before[:, hq * d:(hq + hkv) * d].view(n, hkv, d), pos, d)
    assert torch.equal(qkv[:, (hq + hkv) * d:], before[:, (hq + hkv) * d:])


def test_broadcast_input_transposed_output_and_q_alone():
    x = _randn(1, 1, 40, 64).expand(2, 3, 40, 64)
    out = torch.zeros(2, 40, 3, 64, dtype=torch.bfloat16, device=DEV).transpose(1, 2)
    t = ac.rope_table(64)
    y, none = ac.rope_fwd(x, None, t, out_q=out)
    assert none is None and y is out
    _near(out, x, torch.arange(40, device=DEV), 64)


def test_zero_tokens():
    t = ac.rope_table(64)
    q, k = ac.rope_fwd(_randn(0, 2, 64), _randn(0, 2, 64), t)
    assert q.shape == (0, 2, 64) and k.shape == (0, 2, 64)


def test_far_positions_turn_back_exactly():
    """The angle of any 32-bit position is reduced exactly: positions a whole
    number of turns of the slowest pair apart agree, and a forward turn at
    position x and its backward turn give the input back to two roundings."""
    d = 128
    x = _randn(64, 4, d)
    gen = torch.Generator(device=DEV).manual_seed(3)
    pos = torch.randint(-(2**31), 2**31 - 1, (64,), generator=gen, device=DEV, dtype=torch.int64).to(torch.int32)
    t = ac.rope_table(d)
    y, _ = ac.rope_fwd(x, None, t, positions=pos)
    z, _ = ac.rope_bwd(y, None, t, positions=pos)
    a, b = x[..., : d // 2].double(), x[..., d // 2:].double()
    size = (a.abs() + b.abs()).repeat(1, 1, 2)
    # |y| <= |a| + |b|, rounded once (2^-8); the turn back rounds once more
    assert ((z.double() - x.double()).abs() <= 2 * BF16 * size + BF16 * x.double().abs() + 2.0 ** -20 * size).all()
    assert (y.double().square().sum() / x.double().square().sum() - 1).abs() < 1e-2


def test_backward_is_the_gradient():
    """The formula's gradient by autograd in 64 bits, and central differences of
    the 64-bit definition along random directions."""
    n, h, d, rot = 29, 3, 96, 48
    x, g = _randn(n, h, d, seed=4), _randn(n, h, d, seed=5)
    pos = torch.arange(100, 100 + n, device=DEV, dtype=torch.int32)
    t = ac.rope_table(d, rot_dim=rot, scaling="yarn", factor=4.0, original_len=ORIGINAL)
    dx, _ = ac.rope_bwd(g, None, t, positions=pos)
    f, m = frequencies(rot, scaling="yarn", factor=4.0)
    xd = x.double().requires_grad_()
    ang = pos.double()[:, None, None] * torch.tensor(f, dtype=torch.float64, device=DEV)
    c, s = torch.cos(ang) * m, torch.sin(ang) * m
    a, b = xd[..., : rot // 2], xd[..., rot // 2:rot]
    y = torch.cat((a * c - b * s, b * c + a * s, xd[..., rot:]), -1)
    (want,) = torch.autograd.grad((y * g.double()).sum(), xd)
    size = rotate(g, pos[:, None], rot, backward=True, scaling="yarn", factor=4.0)[1]
    assert ((dx.double() - want).abs() <= rope_tolerance(want, size, rot)).all()
    u = torch.randn(x.shape, generator=torch.Generator(device=DEV).manual_seed(6), device=DEV).double()
    kw = dict(scaling="yarn", factor=4.0)
    h_ = 1e-4
    lo, hi = (rotate(x.double() + e * h_ * u, pos[:, None], rot, **kw)[0] for e in (-1, 1))
    num = float(((hi - lo) / (2 * h_) * g.double()).sum())
    # each element of dx is off by its tolerance at most
    bound = float((rope_tolerance(want, size, rot) * u.abs()).sum())
    assert abs(float((dx.double() * u).sum()) - num) <= bound + 1e-6 * abs(num)


def test_scores_depend_on_the_distance_alone():
    """q at p + n against k at p gives the same score for every p, up to the
    roundings of q and k."""
    d, n = 128, 17
    q, k = _randn(1, 1, d, seed=7).expand(4, 1, d), _randn(1, 1, d, seed=8).expand(4, 1, d)
    t = ac.rope_table(d, scaling="bands", factor=8.0, original_len=ORIGINAL)
    p = torch.tensor([0, 1000, 70000, 1 << 24], device=DEV, dtype=torch.int32)
    yq, _ = ac.rope_fwd(q, None, t, positions=p + n)
    yk, _ = ac.rope_fwd(k, None, t, positions=p)
    s = (yq.double() * yk.double()).sum(-1)[:, 0]
    a, b = (x[0, 0].double() for x in (q, k))
    size = sum(float((a[i].abs() + a[i + 64].abs()) * (b[i].abs() + b[i + 64].abs())) for i in range(64))
    assert float((s - s[0]).abs().max()) <= 2 * 2 * (2 * BF16 + BF16**2) * size


def test_captured_graph_follows_its_inputs():
    x = _randn(2, 4, 50, 64)
    pos = torch.zeros(2, 50, dtype=torch.int32, device=DEV)
    t = ac.rope_table(64)
    y = torch.empty_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ac.rope_fwd(x, None, t, positions=pos, out_q=y)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ac.rope_fwd(x, None, t, positions=pos, out_q=y)
    pos.copy_(torch.arange(100, device=DEV, dtype=torch.int32).view(2, 50))
    g.replay()
    torch.cuda.synchronize()
    _near(y, x, pos[:, None], 64)
    assert not math.isnan(float(y.float().sum()))


def test_outputs_without_the_short_allocation_path(monkeypatch):
    x = _randn(2, 3, 10, 64)
    t = ac.rope_table(64)
    want = ac.rope_fwd(x, None, t)[0]
    monkeypatch.setattr(ac, "_HOST", [])
    monkeypatch.delattr(torch._C._dynamo.guards, "_empty_strided_cuda", raising=False)
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    got = ac.rope_fwd(x.transpose(1, 2).contiguous().transpose(1, 2), None, t)[0]
    assert got.is_contiguous() and torch.equal(got, want)


def test_python_refusals():
    t = ac.rope_table(64)
    q = _randn(4, 2, 64)
    with pytest.raises(ValueError):
        ac.rope_fwd(q.float(), None, t)
    with pytest.raises(ValueError):
        ac.rope_fwd(_randn(4, 2, 96), None, t)
    with pytest.raises(ValueError):
        ac.rope_fwd(q, _randn(5, 2, 64), t)
    with pytest.raises(ValueError):
        ac.rope_fwd(None, None, t)
    with pytest.raises(ValueError):
        ac.rope_fwd(q, None, t, positions=torch.zeros(3, dtype=torch.int32, device=DEV))
    with pytest.raises(ValueError):
        ac.rope_fwd(q, None, t, positions=torch.zeros(4, dtype=torch.int64, device=DEV))
    with pytest.raises(ValueError):
        ac.rope_fwd(q, None, t, positions=torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError):
        ac.rope_fwd(q.transpose(1, 2).contiguous().transpose(1, 2), None, t)
    with pytest.raises(ac.AttnCoreError) as e:      # rows not on 16-byte boundaries
        ac.rope_fwd(_randn(4, 2 * 64 + 4)[:, :128].view(4, 2, 64), None, t)
    assert e.value.code == ac.ERR_MISALIGNED
    with pytest.raises(ac.AttnCoreError) as e:      # an output whose rows coincide
        ac.rope_fwd(q, None, t, out_q=torch.empty(4, 1, 64, dtype=torch.bfloat16, device=DEV).expand(4, 2, 64))
    assert e.value.code == ac.ERR_INVALID_ARG
