"""GPU test of how exact H2ORotary's angles are: pairs (1, 0) become the cosine and the sine themselves, in fp32."""
from __future__ import annotations

import pytest
import torch

from h2o_heavy_hitter_decode_gb300 import H2ORotary

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,dims", [(64, 64), (128, 128), (128, 48)])
def test_sines_and_cosines(d, dims, interleaved):
    """sincospif is off by one unit at most, 2^-24 below 1; turning it on by the rest of the angle rounds once, 2^-25; a
    turn is the nearest of 2^32, 2 pi 2^-33 < 2^-30; the products with 1 and 0 are exact.  The reference's angles of up
    to 2^20 in 64 bits are off by 2^-33 at most."""
    n, pairs = 4096, dims // 2
    k = torch.zeros(3, 1, n, d, device=DEV)
    first = range(0, dims, 2) if interleaved else range(pairs)
    other = range(1, dims, 2) if interleaved else range(pairs, dims)
    k[..., list(first)] = 1.0
    position = torch.tensor([0, 123456, (1 << 20) - n], dtype=torch.int32, device=DEV)
    frequency = 10000.0 ** (-torch.arange(pairs, dtype=torch.float64) / pairs)
    y = H2ORotary(d, frequency=frequency, interleaved=interleaved).apply(None, k, position)[1].double()
    at = (position[:, None].double() + torch.arange(n, device=DEV))[..., None] * frequency.to(DEV)
    for where, want in ((first, at.cos()), (other, at.sin())):
        off = float((y[:, 0][..., list(where)] - want).abs().max())
        assert off <= 2.0 ** -24 + 2.0 ** -25 + 2.0 ** -30 + 2.0 ** -33, off
