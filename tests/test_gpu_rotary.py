"""GPU tests of H2ORotary against its formulas in 64 bits.

Tolerances: the norm's sum of squares is an fp32 sum of d terms (d 2^-24 relative, halved by the root), the reciprocal
root is within 2 units (2^-23 each), and the mean, the products with it and the weight round once each (2^-24): e_n =
(d / 2 + 8) 2^-24 of the normed value.  A turn is the nearest of 2^32 (2^-33 turns), taken to 24 bits (of at most half a turn:
2^-25 of it in turns) and through sincospif (2 units of a result of at most 1): e_a = 2 pi (2^-33 + 2^-26) + 2^-22.  A rotated
element adds two products and their sum, 3 roundings.  All relative to |a| + |b| of the pair; then one half step of
the output's type."""
from __future__ import annotations

import math

import pytest
import torch

from h2o_heavy_hitter_decode_gb300 import H2OError, H2ORotary

pytestmark = pytest.mark.gpu

DEV = "cuda"
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # relative to the value


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def rows(g, B, heads, n, d, dtype, layout="dense"):
    """Dense, a view of token-first rows, or heads of a wider token-first row."""
    if layout == "tokens":
        return torch.randn(B, n, heads, d, generator=g, device=DEV).to(dtype).transpose(1, 2)
    if layout == "slice":
        return torch.randn(B, n, heads + 3, d + 16, generator=g, device=DEV).to(dtype)[:, :, 2:-1, 8:-8].transpose(1, 2)
    return torch.randn(B, heads, n, d, generator=g, device=DEV).to(dtype)


def reference(x, position, frequency, axis, interleaved, eps, weight):
    """The rows in 64 bits, and how far the kernel may be off: [B, heads, n, d] both.  position [axes, B, n]."""
    x = x.detach().cpu().double()
    d, pairs = x.shape[-1], len(frequency)
    tol = torch.zeros_like(x)
    if eps is not None:
        x = x / (x.pow(2).mean(-1, keepdim=True) + eps).sqrt() * (1.0 if weight is None else weight.cpu().double())
        tol += (d / 2 + 8) * 2.0 ** -24 * x.abs()
    y = x.clone()
    e_a = 2 * math.pi * (2.0 ** -33 + 2.0 ** -26) + 2.0 ** -22
    where = position.cpu().double()
    for i in range(pairs):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)
        t = (where[axis[i]] * frequency[i])[:, None]
        c, s = t.cos(), t.sin()
        y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
        size = x[..., a].abs() + x[..., b].abs()
        # an angle in 64 bits is off by a half step of it itself
        e = (e_a + 3 * 2.0 ** -24 + t.abs() * 2.0 ** -52) * size + tol[..., a] + tol[..., b]
        tol[..., a], tol[..., b] = e, e
    return y, tol


def check(got, want, tol):
    half = HALF_STEP[got.dtype]
    got = got.detach().cpu().double()
    bad = ~((got - want).abs() <= tol + half * (want.abs() + tol) + 1e-37)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4], got[bad][:4], want[bad][:4], tol[bad][:4])


def theta(pairs, base=10000.0):
    return [base ** (-i / pairs) for i in range(pairs)]


CASES = [  # B, query heads, key heads, n, d, dims, dtype, axes, interleaved, norm, layout, far
    (1, 1, 1, 1, 64, 64, torch.bfloat16, 1, False, False, "dense", 1),
    (1, 32, 32, 1, 128, 128, torch.bfloat16, 1, False, True, "tokens", 8192),
    (3, 5, 1, 7, 128, 128, torch.bfloat16, 1, True, True, "slice", 4194304),
    (2, 8, 2, 33, 64, 16, torch.bfloat16, 1, False, True, "tokens", 2 ** 31 - 64),
    (2, 3, 3, 5, 128, 96, torch.float32, 1, False, True, "slice", 2 ** 31 - 64),
    (2, 7, 7, 65, 64, 32, torch.float32, 3, True, False, "dense", 300),
    (1, 2, 4, 9, 128, 112, torch.float32, 4, False, False, "tokens", 100000),
    (5, 71, 1, 3, 64, 48, torch.bfloat16, 2, True, True, "dense", 77),
    (2, 4, 4, 4, 128, 0, torch.bfloat16, 1, False, True, "dense", 9),
    (700, 6, 3, 1, 64, 64, torch.bfloat16, 1, False, False, "dense", 5000),
    (1, 3, 2, 2257, 128, 128, torch.bfloat16, 3, False, True, "tokens", 64),
    (7, 2, 1, 33, 64, 64, torch.bfloat16, 1, False, True, "tokens", 999),      # fewer heads than a warp takes at a time
    (3, 1, 1, 5, 128, 64, torch.float32, 2, True, False, "slice", 40),
    (9, 2, 2, 1, 128, 128, torch.bfloat16, 1, True, True, "dense", 100000),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x).replace("torch.", "") for x in c))
def test_against_formulas(case):
    B, hq, hk, n, d, dims, dtype, axes, interleaved, norm, layout, far = case
    g = torch.Generator(DEV).manual_seed(5)
    q, k = rows(g, B, hq, n, d, dtype, layout), rows(g, B, hk, n, d, dtype, layout)
    axis = [i * axes // max(1, dims // 2) for i in range(dims // 2)]
    wq, wk = torch.randn(d, generator=g, device=DEV).bfloat16(), torch.randn(d, generator=g, device=DEV)
    r = H2ORotary(d, dims=dims, axis=axis, interleaved=interleaved,
                  **(dict(eps=1e-5, q_weight=wq, k_weight=wk) if norm else {}))
    if axes == 1:
        position = torch.randint(0, far, (B,), generator=g, device=DEV, dtype=torch.int32)
        where = (position[:, None].long() + torch.arange(n, device=DEV))[None]
    else:
        where = position = torch.randint(-far, far, (axes, B, n), generator=g, device=DEV, dtype=torch.int32)
    a, b = q.clone(), k.clone()
    oq, ok = r.apply(q, k, position)
    assert torch.equal(q, a) and torch.equal(k, b)
    for x, y, w in ((q, oq, wq), (k, ok, wk)):
        assert y.shape == x.shape and y.dtype == dtype
        check(y, *reference(x, where, theta(dims // 2) if dims else [], axis, interleaved, 1e-5 if norm else None, w))
    # the same bits in place, and for one of the two alone
    only, none = r.apply(None, k, position)[1], r.apply(q, None, position)
    assert torch.equal(only, ok) and torch.equal(none[0], oq) and none[1] is None
    r.apply(q, k, position, q_out=q, k_out=k)
    assert torch.equal(q, oq) and torch.equal(k, ok)


def test_frequencies_of_the_caller():
    """Scaled and negative frequencies, and some of many turns a position."""
    g = torch.Generator(DEV).manual_seed(6)
    frequency = torch.tensor([0.25, -1.0, 3.0, 100.0, 1e-8, 0.0, -7.5, 2.0 ** 20], dtype=torch.float64)
    r = H2ORotary(64, frequency=frequency)
    k = rows(g, 2, 3, 50, 64, torch.float32)
    where = ints([0, 1 << 20])
    y = r.apply(None, k, where)[1]
    at = (where[:, None].long() + torch.arange(50, device=DEV))[None]
    check(y, *reference(k, at, frequency.tolist(), [0] * 8, False, None, None))


def test_far_positions_agree_with_near_ones():
    """A frequency of a whole number of turns over 2^20 positions: positions 2^20 apart give the same bits."""
    g = torch.Generator(DEV).manual_seed(7)
    r = H2ORotary(64, frequency=[2 * math.pi * m / 2 ** 20 for m in (1, 3, 5, 7, 1023, 4097, 65537, 524287)])
    k = rows(g, 1, 2, 16, 64, torch.float32)
    near, far = r.apply(None, k, ints([12345]))[1], r.apply(None, k, ints([12345 + 1024 * 2 ** 20]))[1]
    # the frequencies are numbers of 53 bits: 2^-53 of m 2^30 / 2^20 turns and more
    assert float((near - far).abs().max()) <= 2 * math.pi * 524287 * 1024 * 2.0 ** -53 * 8 + 2.0 ** -20


@pytest.mark.parametrize("hq,hk", [(3, 2), (1, 1), (2, 1), (9, 20)])
def test_padded_batch(hq, hk):
    """Rows behind the counts are neither read nor written; counts out of range are the nearest that is not."""
    g = torch.Generator(DEV).manual_seed(8)
    q, k = rows(g, 5, hq, 4, 128, torch.bfloat16, "tokens"), rows(g, 5, hk, 4, 128, torch.bfloat16)
    r = H2ORotary(128, eps=0.0)
    counts, real = ints([0, 1, 4, -3, 9]), [0, 1, 4, 0, 4]
    position = ints([3, 0, 9, 1, 2])
    full = r.apply(q, k, position)
    oq, ok = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    for b, c in enumerate(real):
        q[b, :, c:] = math.nan
        k[b, :, c:] = math.inf
    r.apply(q, k, position, counts, q_out=oq, k_out=ok)
    zq, zk = r.apply(q, k, position, counts)
    for b, c in enumerate(real):
        for got, zero, want in ((oq, zq, full[0]), (ok, zk, full[1])):
            assert torch.equal(got[b, :, :c], want[b, :, :c]) and bool((got[b, :, c:] == 7).all())
            assert torch.equal(zero[b, :, :c], want[b, :, :c]) and bool((zero[b, :, c:] == 0).all())


def test_rows_that_hold_nothing_or_no_numbers():
    """A row of zeros with eps 0 (0 / 0: NaN), with eps; one NaN stays in its row; infinities."""
    k = torch.ones(1, 4, 3, 64, device=DEV, dtype=torch.bfloat16)
    k[0, 0, 1] = 0
    k[0, 1, 1, 5] = math.nan
    k[0, 2, 1, 40] = math.inf
    for eps in (None, 1e-6):
        y = H2ORotary(64, eps=eps).apply(None, k, ints([3]))[1]
        assert bool((y[0, 0, 1] == 0).all())
        assert bool(y[0, 1, 1, 5].isnan()) and bool(y[0, 1, 1, 37].isnan())
        assert bool(torch.isfinite(y[0, :, [0, 2]]).all())
        if eps is None:
            assert int((~torch.isfinite(y)).sum()) == 4  # the pairs (5, 37) and (8, 40)


def test_streams_graphs_and_lifetime():
    g = torch.Generator(DEV).manual_seed(9)
    q, k = rows(g, 2, 8, 3, 128, torch.bfloat16), rows(g, 2, 2, 3, 128, torch.bfloat16)
    position = ints([5, 6])
    r = H2ORotary(128, eps=1e-6)
    want = [r.apply(q, k, position + i) for i in range(3)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = r.apply(q, k, position)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[0], want[0][0]) and torch.equal(got[1], want[0][1])
    oq, ok = torch.empty_like(q), torch.empty_like(k)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r.apply(q, k, position, q_out=oq, k_out=ok)
    for i in range(3):  # reads the positions of its replay
        graph.replay()
        assert torch.equal(oq, want[i][0]) and torch.equal(ok, want[i][1])
        position += 1


def test_refusals():
    for bad in (dict(d=96), dict(d=64, dims=24), dict(d=64, dims=80), dict(d=64, dims=-16), dict(d=64, theta=0.0),
                dict(d=64, frequency=[1.0] * 12), dict(d=64, frequency=[math.inf] * 8), dict(d=64, frequency=[1.0] * 8, dims=32),
                dict(d=64, axis=[0] * 31), dict(d=64, axis=[256] * 32), dict(d=64, eps=-1.0), dict(d=64, eps=math.nan),
                dict(d=64, q_weight=torch.ones(64, device=DEV)), dict(d=64, eps=0.0, k_weight=torch.ones(63, device=DEV)),
                dict(d=64, device="cpu")):
        with pytest.raises(ValueError):
            H2ORotary(**bad)
    r = H2ORotary(64)
    k, p = torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16, device=DEV), ints([0, 0])
    odd = torch.zeros(2, 3, 4, 72, dtype=torch.bfloat16, device=DEV)
    for args, more in [((None, None, p), {}), ((None, k[0], p), {}), ((None, k.half(), p), {}), ((k.float(), k, p), {}),
                       ((None, odd, p), {}), ((None, k.cpu(), p), {}), ((None, k, p.long()), {}), ((None, k, ints([0])), {}),
                       ((None, k, ints([0, 0, 0, 0])[::2]), {}), ((None, k, p.cpu()), {}),
                       ((None, k, ints([[[0] * 4]])), {}), ((None, k, p, ints([1])), {}), ((None, k, p), dict(q_out=k)),
                       ((None, k, p), dict(k_out=k.float())), ((None, k, p), dict(k_out=k[:1])),
                       ((k, k[:, :, :2], p), {}), ((None, odd[..., 4:68], p), {}), ((None, k.transpose(2, 3), p), {})]:
        with pytest.raises((ValueError, TypeError)):
            r.apply(*args, **more)
    with pytest.raises(H2OError):  # two rows of an output in one place
        r.apply(None, k, p, k_out=k[:, :1].expand(2, 3, 4, 64))
    with pytest.raises(H2OError):
        r.apply(None, k[:, :, :0], p)
