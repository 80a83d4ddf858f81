"""GPU test of sparse attention where one CTA's logits are 2^31 and more: every block of a cache of 2^27 entries, 256 query
heads to its one cached head.  Takes 155 GB of the GPU's memory and a second or two."""
from __future__ import annotations

import math

import pytest
import torch

from h2o_heavy_hitter_decode_gb300 import H2OBlockCache

pytestmark = pytest.mark.gpu

DEV = "cuda"


def test_logits_past_31_bits():
    """Equal keys: every weight is 2^-27, sums and products of powers of two.  ex2 and log2 are off by 2^-21 at most, the
    join by a few 2^-23, the sum of 256 weights by 256 2^-24 at most."""
    cap, G, d = 1 << 27, 256, 64
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 170 * 10 ** 9:
        pytest.skip("needs 170 GB")
    c = H2OBlockCache(1, 1, d, cap, group=G, kv="int8", bounds=True)
    value = (torch.arange(d, device=DEV) % 15 - 7).to(torch.int8)
    c.V.copy_(value)
    c.K_scale.fill_(1.0)
    c.V_scale.fill_(1.0)
    g = torch.Generator(DEV).manual_seed(1)
    q = torch.randn(1, G, 1, d, generator=g, device=DEV).bfloat16()
    lens, lse = torch.tensor([cap], dtype=torch.int32, device=DEV), torch.zeros(1, G, 1, device=DEV)
    out = c.attend_sparse(q, lens, cap // 32, lse=lse)
    assert c.error_bits() == 0
    off = 2.0 ** -21 * 2 + 32 * 2.0 ** -23
    assert bool(((out.double() - value.double()).abs() <= (2.0 ** -8 + off) * value.double().abs()).all())
    assert bool(((lse.double() - 27 * math.log(2)).abs() <= 2.0 ** -21 * 27).all())
    low, high = (float(x) for x in c.score.aminmax())
    off += 256 * 2.0 ** -24
    assert 2.0 ** -19 * (1 - off) <= low <= high <= 2.0 ** -19 * (1 + off), (low, high)
    del c
    torch.cuda.empty_cache()
