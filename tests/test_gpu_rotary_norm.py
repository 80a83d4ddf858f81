"""GPU tests of H2ORotary's norm at the ends of fp32's range: rows whose squares are lost in it, with an eps of 0 or a tiny
one, rows of zeros, rows whose squares pass it, rows that hold no numbers; each beside ordinary rows, whose bits stay."""
from __future__ import annotations

import math

import pytest
import torch

from h2o_heavy_hitter_decode_gb300 import H2ORotary
from test_gpu_rotary import check, ints, reference, theta

pytestmark = pytest.mark.gpu

DEV = "cuda"
ODD = 2  # of the rows below, each third is not an ordinary one


def with_odd_rows(g, dtype, d, size, heads=5, n=7):
    """[2, heads, n, d], rows of `size` among those of size 1."""
    x = torch.randn(2, heads, n, d, generator=g, device=DEV)
    odd = (torch.arange(2 * heads * n, device=DEV) % 3 == ODD).view(2, heads, n)
    x = torch.where(odd[..., None], (x.double() * size).float(), x).to(dtype)
    return x, odd


@pytest.mark.parametrize("eps", [0.0, 2.0 ** -149, 2.0 ** -100, 2.0 ** -97])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,dims,heads", [(64, 64, 5), (128, 32, 5), (128, 0, 5), (64, 32, 1), (128, 128, 40)])
def test_rows_of_tiny_elements(eps, dtype, d, dims, heads):
    """x / sqrt(mean x^2 + eps) is an ordinary row where eps is 0, however small x is.  The tolerances are those of the
    norm anywhere: a power of two costs nothing."""
    g = torch.Generator(DEV).manual_seed(4)
    r = H2ORotary(d, dims=dims, eps=eps, k_weight=torch.randn(d, generator=g, device=DEV))
    position = ints([3, 77])
    where = (position[:, None].long() + torch.arange(7, device=DEV))[None]
    for e in (-40, -46, -50, -60, -63, -70, -75, -100, -120, -126, -130):
        k, odd = with_odd_rows(g, dtype, d, 2.0 ** e, heads)
        k[0, 0, 2] = 2.0 ** e  # all the same
        y = r.apply(None, k, position)[1]
        check(y, *reference(k, where, theta(dims // 2) if dims else [], [0] * (dims // 2), False, eps, r._weights[1]))
        if eps == 0.0:
            assert bool(torch.isfinite(y).all()) and float(y[odd].float().abs().amax()) > 1


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_the_least_numbers(dtype):
    """One least number of the type among zeros, and rows full of it, with eps 0."""
    least = torch.tensor(2.0 ** (-133 if dtype == torch.bfloat16 else -149), device=DEV).to(dtype)
    k = torch.zeros(1, 3, 2, 64, dtype=dtype, device=DEV)
    k[0, 0, 0, 5], k[0, 1, 1], k[0, 2] = least, -least, 1.0
    k[0, 0, 1, 63], k[0, 1, 0, 0], k[0, 1, 0, 1] = least, 3 * least.float(), 4 * least.float()
    y = H2ORotary(64, dims=0, eps=0.0).apply(None, k, None)[1]
    check(y, *reference(k, torch.zeros(1, 1, 2), [], [], False, 0.0, None))
    assert float(y[0, 0, 0, 5].float()) == 8.0 and bool((y[0, 1, 1].float() == -1.0).all())


@pytest.mark.parametrize("dims", [0, 64])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_odd_rows_stay_among_themselves(dtype, dims):
    """Zeros with eps 0 are 0 / 0; squares past fp32's range give 0; a NaN makes its row NaN.  What lies beside them keeps
    the bits that it has beside ordinary rows."""
    g = torch.Generator(DEV).manual_seed(5)
    for size, eps, want in ((0.0, 0.0, math.nan), (0.0, 1e-6, 0.0), (0.0, 2.0 ** -149, 0.0), (2.0 ** -70, 0.0, None),
                            (1e25, 0.0, 0.0), (1e25, 1e-6, 0.0), (math.nan, 0.0, math.nan), (math.nan, 1e-6, math.nan)):
        r = H2ORotary(64, dims=dims, eps=eps)
        for heads in (1, 5, 40):
            k, odd = with_odd_rows(g, dtype, 64, 1.0, heads)
            plain = r.apply(None, k.clone().masked_fill_(odd[..., None], 1.0), ints([3, 77]))[1]
            k[odd] = size
            y = r.apply(None, k, ints([3, 77]))[1]
            assert torch.equal(y[~odd], plain[~odd])
            if want is None:
                assert bool(torch.isfinite(y).all())
            else:
                assert bool(y[odd].isnan().all() if math.isnan(want) else (y[odd] == want).all())


def test_one_nan_makes_its_row_nan():
    k = torch.ones(1, 4, 3, 64, device=DEV, dtype=torch.bfloat16)
    k[0, 1, 1, 5] = math.nan
    k[0, 2, 1, 40] = math.inf  # the mean square is infinite: all but the pair (8, 40) become 0
    for eps in (0.0, 1e-6):
        y = H2ORotary(64, eps=eps).apply(None, k, ints([3]))[1]
        assert bool(y[0, 1, 1].isnan().all()) and bool(torch.isfinite(y[0, [0, 3]]).all())
        assert int((~torch.isfinite(y[0, 2])).sum()) == 2 and bool((y[0, 2, 1, :8] == 0).all())
        assert bool(torch.isfinite(y[0, :, [0, 2]]).all())
