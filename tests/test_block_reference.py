"""The 64-bit block-cache reference against torch's own conversions, brute
force and softmax (CPU)."""
from __future__ import annotations

import math

import pytest
import torch

from block_reference import BLOCK, LIMIT, RefCache, pow2_scale, round_code


def test_e4m3_rounding_is_torchs():
    x = torch.cat([torch.arange(-448, 448, 0.37), torch.logspace(-12, 8.8, 4001, base=2), torch.zeros(1)]).double()
    x = torch.cat([x, -x]).clamp(-448, 448)
    want = x.float().to(torch.float8_e4m3fn).double()
    assert torch.equal(round_code(x.float().double(), "e4m3"), want)


def test_int8_rounding_ties_to_even():
    assert round_code(torch.tensor([0.5, 1.5, 2.5, -0.5, 126.5, 300.0], dtype=torch.float64), "int8").tolist() == \
        [0, 2, 2, 0, 126, 127]


@pytest.mark.parametrize("kv", ["e4m3", "int8"])
def test_scale_is_the_least_power_of_two(kv):
    for amax in [1e-38, 2.0 ** -92, 0.3, 1.0, LIMIT[kv], LIMIT[kv] + 1e-9, 448.5, 3.3e38]:
        s = pow2_scale(amax, kv)
        assert math.frexp(s)[0] == 0.5 and amax <= LIMIT[kv] * s
        assert s == 2.0 ** -100 or amax > LIMIT[kv] * s / 2
    assert pow2_scale(0.0, kv) == 2.0 ** -100


@pytest.mark.parametrize("kv", ["e4m3", "int8"])
def test_append_in_pieces_errs_by_less_than_a_step(kv):
    """Rows appended one at a time, some making the block's scale grow: each value stays within one final step
    (int8), or within two half steps of e4m3's spacing at it (a re-scaling rounds subnormals only)."""
    g = torch.Generator().manual_seed(3)
    x = torch.randn(1, 1, 70, 64, generator=g) * torch.logspace(-3, 3, 70)[None, None, :, None]
    r = RefCache(1, 1, 64, 96, 1, kv)
    for t in range(70):
        r.append(x[:, :, t : t + 1], x[:, :, t : t + 1], [t])
    got = r.values("K", 0, 0, 70)
    s = r.K_scale[0, 0].repeat_interleave(BLOCK)[:70, None]
    step = s if kv == "int8" else s * torch.exp2((torch.frexp((x[0, 0].double() / s))[1].double() - 1).clamp(min=-6) - 3)
    assert ((got - x[0, 0].double()).abs() <= step).all()


def test_attend_is_softmax_attention():
    g = torch.Generator().manual_seed(5)
    r = RefCache(1, 2, 64, 64, 3, "int8")
    k, v = torch.randn(1, 2, 40, 64, generator=g), torch.randn(1, 2, 40, 64, generator=g)
    r.append(k, v, [0])
    q = torch.randn(1, 6, 4, 64, generator=g).double()
    out, lse, _, _ = r.attend(q, [40])
    kf = torch.stack([r.values("K", 0, h // 3, 40) for h in range(6)])[None]
    vf = torch.stack([r.values("V", 0, h // 3, 40) for h in range(6)])[None]
    mask = torch.ones(4, 40, dtype=torch.bool).tril(36)
    want = torch.nn.functional.scaled_dot_product_attention(q, kf, vf, attn_mask=mask)
    assert torch.allclose(out, want, atol=1e-12)
    assert abs(float(r.score[0].sum()) - 24) < 1e-9  # every query spends a weight of one


def test_no_entry_visible():
    r = RefCache(1, 1, 64, 32, 1, "int8")
    out, lse, _, _ = r.attend(torch.randn(1, 1, 2, 64), [1])
    assert (out[0, 0, 0] == 0).all() and lse[0, 0, 0] == -math.inf and math.isfinite(lse[0, 0, 1])


def test_evict_ties_go_to_the_lowest_index():
    r = RefCache(1, 1, 64, 32, 1, "int8")
    r.append(torch.randn(1, 1, 8, 64), torch.randn(1, 1, 8, 64), [0], score=torch.tensor([[[1., 1, 2, 1, 1, 0, 9, 9]]]))
    assert r.evict([8], 3, 2) == [5]
    assert r.pos[0, 0, :5].tolist() == [2, 3, 4, 6, 7]
