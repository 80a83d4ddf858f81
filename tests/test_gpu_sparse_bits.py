"""GPU tests of how many bits the sparse attention keeps of its weights: outputs that cancel show what a weight's rounding
leaves, where outputs near sum w |v| hide it behind their own."""
from __future__ import annotations

import math

import pytest
import torch

from h2o_heavy_hitter_decode_gb300 import H2OBlockCache

pytestmark = pytest.mark.gpu

DEV = "cuda"


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kv", ["e4m3", "int8"])
@pytest.mark.parametrize("B,H,G,n", [(1, 1, 1, 1), (2, 3, 8, 1), (3, 2, 5, 3), (1, 2, 12, 1), (48, 4, 2, 1), (60, 8, 4, 1), (40, 8, 3, 2), (40, 8, 9, 1)])
def test_weights_whose_values_cancel(kv, d, B, H, G, n):
    """Entries in pairs whose weights differ by a few thousandths and whose values are opposite: what is left of a weight's
    rounding to 11 bits would be as large as the outputs.

    Keys and queries have one element that is not 0, so a logit s is one product, exact but for its factors (4 half steps
    of 2^-24 and |s| log2 e 2^-24 in base 2): e_s = 2^-23 4 |s|.  A weight: 2 e_s + 2^-21 (|s - top| + 8), as in the
    reference; its two parts 2^-22; the sums of blocks of 32 entries, of up to 4 blocks and of the parts that meet, in
    fp32, some of them truncated: 64 2^-23.  All of sum w |v|; then a half step of bf16."""
    g = torch.Generator(DEV).manual_seed(3)
    cap, end = 256, 250
    c = H2OBlockCache(B, H, d, cap, group=G, max_queries=n, kv=kv, bounds=True)
    even = torch.randint(4, 60, (B, H, cap // 2), generator=g, device=DEV) * 2 if kv == "int8" else \
        torch.randint(8, 15, (B, H, cap // 2), generator=g, device=DEV)
    codes = torch.stack([even, even + 1], -1).flatten(2).float()
    K = torch.zeros(B, H, cap, d, device=DEV)
    K[..., 3] = codes
    sign = torch.randint(0, 2, (B, H, cap // 2, d), generator=g, device=DEV).float() * 2 - 1
    V = torch.stack([sign, -sign], 3).flatten(2, 3) * 96
    for to, x in ((c.K, K), (c.V, V)):
        to.copy_(x.to(to.dtype))
        assert torch.equal(to.float(), x if kv == "int8" else x.to(torch.float8_e4m3fn).float())
    c.K_scale.fill_(2.0 ** -3)
    c.V_scale.fill_(2.0 ** -6)
    c.bound(ints([end] * B))
    q = torch.zeros(B, H * G, n, d, dtype=torch.bfloat16, device=DEV)
    q[..., 3] = torch.rand(B, H * G, n, generator=g, device=DEV).add_(0.5).mul_(0.25 if kv == "int8" else 2 ** -0.5).bfloat16()
    blocks = torch.zeros(B, H, n, 4, dtype=torch.int32, device=DEV)
    out = c.attend_sparse(q, ints([end] * B), 4, accumulate=False, causal=False, blocks=blocks)
    at = (blocks[..., None].long() * 32 + torch.arange(32, device=DEV)).flatten(-2)             # [B, H, n, 128]
    k = codes.double()[:, :, None].expand(-1, -1, n, -1).gather(-1, at) * 2.0 ** -3
    v = (V.double() * 2.0 ** -6)[:, :, None].expand(-1, -1, n, -1, -1).gather(3, at[..., None].expand(*at.shape, d))
    s = q[..., 3].double().unflatten(1, (H, G)).permute(0, 1, 3, 2)[..., None] * k[:, :, :, None] / math.sqrt(d)  # [B, H, n, G, 128]
    s.masked_fill_((at >= end)[:, :, :, None], -math.inf)
    w = torch.softmax(s, -1)
    want, mass = (w @ v).permute(0, 1, 3, 2, 4).flatten(1, 2), (w @ v.abs()).permute(0, 1, 3, 2, 4).flatten(1, 2)
    fine = torch.where(s.isinf(), 0.0, s)
    off = fine.amax(-1, keepdim=True) - fine
    e_w = 2 * 2.0 ** -21 * fine.abs().amax() + 2.0 ** -21 * (off.amax() + 8) + 2.0 ** -22 + 64 * 2.0 ** -23
    tol = 2.0 ** -8 * want.abs() + e_w * mass * (1 + 2.0 ** -7)
    assert float((e_w * mass).max()) < 2.0 ** -14 * float(mass.max())  # half of 11 bits' own
    got = out.double()
    bad = (got - want).abs() > tol
    assert not bad.any(), (int(bad.sum()), got[bad][:4], want[bad][:4], tol[bad][:4])
    assert c.error_bits() == 0
