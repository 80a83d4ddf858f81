"""GPU tests of H2OBlockCache (append, attend, step, evict) against the plain
64-bit reference of block_reference.py: codes, scales, positions and kept
entries exactly, outputs, log-sum-exps and scores within the reference's
derived tolerances."""
from __future__ import annotations

import math

import pytest
import torch

from block_reference import BLOCK, RefCache, close, load, same_state
from h2o_heavy_hitter_decode_gb300 import H2OBlockCache, H2OError

pytestmark = pytest.mark.gpu

DEV = "cuda"


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def rows(g, B, heads, n, d, layout="dense", scale=1.0):
    """bf16 [B, heads, n, d]: dense, a view of token-first rows, a slice of a wider row, or one head broadcast."""
    if layout == "tokens":
        return (torch.randn(B, n, heads, d, generator=g, device=DEV) * scale).bfloat16().transpose(1, 2)
    if layout == "slice":
        return (torch.randn(B, n, heads + 3, d + 16, generator=g, device=DEV) * scale).bfloat16()[:, :, 2:-1, 8:-8].transpose(1, 2)
    if layout == "broadcast":
        return (torch.randn(B, 1, n, d, generator=g, device=DEV) * scale).bfloat16().expand(B, heads, n, d)
    return (torch.randn(B, heads, n, d, generator=g, device=DEV) * scale).bfloat16()


def filled(seed, B, H, d, cap, lens, group=1, max_queries=1, kv="e4m3", scale=1.0, junk=True):
    """A cache and its reference with lens entries per sequence; places behind them hold other sequences' rows,
    e4m3 NaN codes and infinite scales among them."""
    g = torch.Generator(DEV).manual_seed(seed)
    c = H2OBlockCache(B, H, d, cap, group=group, max_queries=max_queries, kv=kv)
    full = rows(g, B, H, cap, d, scale=scale)
    c.append(full, rows(g, B, H, cap, d, scale=scale), ints([0] * B), score=torch.rand(B, H, cap, generator=g, device=DEV) * 9)
    if junk:
        for b, n in enumerate(lens):
            if kv == "e4m3":
                c.K.view(torch.uint8)[b, :, n:] = 0x7F
                c.V.view(torch.uint8)[b, :, n:] = 0xFF
            first = (n + BLOCK - 1) // BLOCK
            c.K_scale[b, :, first:] = math.inf
            c.V_scale[b, :, first:] = math.nan
            c.score[b, :, n:] = math.nan
    r = RefCache(B, H, d, cap, group, kv)
    load(r, c)
    return c, r, g


# ------------------------------------------------------------------- append

@pytest.mark.parametrize("layout", ["dense", "tokens", "slice", "broadcast"])
@pytest.mark.parametrize("kv,d", [("e4m3", 128), ("e4m3", 64), ("int8", 128), ("int8", 64)])
def test_append_ragged(kv, d, layout):
    lens = [0, 1, 31, 32, 33, 95, 60]
    counts = [70, 0, 1, 33, 31, 5, 64]
    c, r, g = filled(11, 7, 3, d, 160, lens, kv=kv)
    k, v = rows(g, 7, 3, 70, d, layout), rows(g, 7, 3, 70, d, layout, scale=3.0)
    score = torch.rand(7, 3, 70, generator=g, device=DEV)
    where = [1000 * b for b in range(7)]
    c.append(k, v, ints(lens), ints(counts), position=ints(where), score=score)
    r.append(k, v, lens, counts, where, score)
    same_state(c, r)
    assert c.error_bits() == 0


@pytest.mark.parametrize("kv", ["e4m3", "int8"])
def test_append_one_at_a_time_scale_grows(kv):
    g = torch.Generator(DEV).manual_seed(2)
    c = H2OBlockCache(2, 2, 64, 96, kv=kv)
    r = RefCache(2, 2, 64, 96, 1, kv)
    for t in range(75):
        k = rows(g, 2, 2, 1, 64, scale=2.0 ** ((t * 5) % 13 - 6))
        v = rows(g, 2, 2, 1, 64, scale=1.1 ** t)
        c.append(k, v, ints([t, t + 3]))
        r.append(k, v, [t, t + 3])
    same_state(c, r)


@pytest.mark.parametrize("kv", ["e4m3", "int8"])
def test_append_extreme_values(kv):
    """Zeros, bf16's least and largest numbers, the borders of the code range, infinities and NaN."""
    x = torch.zeros(1, 4, 40, 64)
    x[0, 0, 0, :4] = torch.tensor([448.0, -448.0, 127.0, 0.5])
    x[0, 0, 33, :2] = torch.tensor([450.0, 127.5])
    x[0, 1, 5, :3] = torch.tensor([1e-40, -9e-41, 1.2e-38])
    x[0, 1, 35, 0] = 2.0 ** -101
    x[0, 2, 7, :3] = torch.tensor([3.0e38, -1.0e38, 1.0])
    x[0, 3, 9, :4] = torch.tensor([math.inf, -math.inf, math.nan, 2.5])
    x[0, 3, 39, 0] = math.nan
    k = x.bfloat16().to(DEV)
    c = H2OBlockCache(1, 4, 64, 64, kv=kv)
    r = RefCache(1, 4, 64, 64, 1, kv)
    c.append(k, -k, ints([0]))
    r.append(k, -k, [0])
    same_state(c, r)
    assert c.error_bits() == 2
    with pytest.raises(H2OError):
        c.check_device_error()


@pytest.mark.parametrize("kv", ["e4m3", "int8"])
@pytest.mark.parametrize("n", [1, 8, 40])
def test_append_infinity_next_to_the_largest_number(kv, n):
    """An infinity takes the largest code also where largest code * scale is beyond fp32."""
    x = torch.zeros(1, 1, n, 64)
    x[0, 0, n - 1, :3] = torch.tensor([3.38e38, math.inf, -math.inf])
    k = x.bfloat16().to(DEV)
    c, r = H2OBlockCache(1, 1, 64, 64, kv=kv), RefCache(1, 1, 64, 64, 1, kv)
    c.append(k, -k, ints([0]))
    r.append(k, -k, [0])
    same_state(c, r)


# ------------------------------------------------------------------- attend

ATTEND = [  # B, H, G, n, d, kv, cap, lens, counts, causal
    (1, 1, 1, 1, 128, "e4m3", 32, [1], None, True),
    (1, 1, 1, 1, 64, "int8", 32, [32], None, True),
    (3, 2, 1, 1, 128, "int8", 96, [33, 0, 96], None, True),
    (9, 3, 2, 1, 64, "e4m3", 128, [1, 2, 31, 32, 33, 64, 65, 127, 128], None, True),
    (2, 2, 4, 1, 128, "e4m3", 1024, [1000, 517], None, False),
    (3, 2, 8, 2, 128, "int8", 512, [500, 2, 77], [2, 1, 0], True),
    (2, 1, 5, 7, 64, "int8", 256, [256, 3], None, True),        # 35 rows, fewer entries than queries
    (2, 2, 1, 16, 128, "e4m3", 160, [150, 9], [16, 13], True),
    (2, 2, 3, 16, 64, "e4m3", 160, [150, 9], [16, 3], False),   # 48 rows
    (1, 2, 16, 4, 128, "e4m3", 96, [90], None, True),           # 64 rows
    (2, 1, 71, 1, 64, "int8", 96, [90, 31], None, True),        # one cached head for 71
    (1, 1, 16, 16, 128, "int8", 96, [70], [11], True),          # 256 rows
    (40, 2, 1, 1, 64, "e4m3", 64, [(7 * b) % 65 for b in range(40)], None, True),
    (1, 2, 2, 1, 128, "e4m3", 8192, [8191], None, True),
    # shapes at the border of what one CTA takes whole: capacity, rows, heads
    (9, 3, 2, 1, 64, "e4m3", 544, [1, 2, 31, 32, 33, 64, 65, 127, 544], None, True),
    (3, 2, 4, 2, 128, "int8", 544, [500, 2, 77], [2, 1, 0], True),
    (3, 2, 4, 2, 128, "e4m3", 512, [512, 2, 77], [2, 1, 0], True),
    (4, 2, 3, 3, 64, "int8", 512, [512, 0, 77, 300], None, False),
    (70, 3, 1, 2, 128, "int8", 96, [(13 * b) % 97 for b in range(70)], None, True),
    (103, 3, 1, 1, 64, "e4m3", 64, [(13 * b) % 65 for b in range(103)], None, True),
    # 17 to 64 rows: two to four warps a worker, some without a row of the sequence
    (3, 2, 8, 4, 128, "e4m3", 320, [300, 31, 129], [4, 1, 3], True),
    (3, 2, 4, 6, 64, "int8", 320, [300, 31, 129], [6, 2, 0], False),
    (3, 2, 3, 11, 128, "int8", 320, [300, 31, 129], [11, 1, 5], True),
    (3, 2, 5, 12, 128, "e4m3", 320, [300, 31, 129], [12, 3, 7], True),
]


@pytest.mark.parametrize("case", ATTEND, ids=lambda c: "-".join(str(x) for x in c[:7]))
@pytest.mark.parametrize("layout", ["dense", "slice"])
def test_attend(case, layout):
    B, H, G, n, d, kv, cap, lens, counts, causal = case
    c, r, g = filled(21, B, H, d, cap, lens, G, n, kv)
    q = rows(g, B, H * G, n, d, layout, scale=2.0)
    out = rows(g, B, H * G, n, d, layout)
    lse = torch.full((B, H * G, n), 7.0, device=DEV)
    before = out.clone()
    res = c.attend(q, ints(lens), None if counts is None else ints(counts), causal=causal, out=out, lse=lse)
    assert res is out
    want, want_lse, tol, lse_tol = r.attend(q, lens, counts, causal)
    close(out, want, tol, "out")
    close(lse, want_lse, lse_tol, "lse")
    idle = want_lse.isnan()  # rows behind the counts
    assert torch.equal(out.cpu()[idle], before.cpu()[idle]) and (lse.cpu()[idle] == 7.0).all()
    same_state(c, r)
    assert c.error_bits() == 0
    # again, without touching the scores
    out2 = c.attend(q, ints(lens), None if counts is None else ints(counts), causal=causal, accumulate=False)
    live = ~idle
    assert torch.equal(out2.cpu()[live], out.cpu()[live])
    same_state(c, r)


@pytest.mark.parametrize("kv", ["e4m3", "int8"])
def test_attend_scales_of_very_different_size(kv):
    """Blocks whose V scales lie 2^40 apart, a block of zeros, and a block that takes all the weight."""
    lens = [192, 160]
    c, r, g = filled(31, 2, 2, 128, 192, lens, 4, 1, kv)
    for j, e in enumerate([-30, 10, -3, 0, -30, 7]):
        c.V_scale[:, :, j] = 2.0 ** e
    c.V.view(torch.uint8)[:, 0, 32:64] = 0
    c.V_scale[:, 0, 1] = 2.0 ** -100
    load(r, c)
    q = rows(g, 2, 8, 1, 128, scale=1.0)
    key = (c.K[0, 1, 70].float() * c.K_scale[0, 1, 2]).bfloat16()
    q[0, 5, 0] = key * 3
    lse = torch.zeros(2, 8, 1, device=DEV)
    out = c.attend(q, ints(lens), lse=lse)
    want, want_lse, tol, lse_tol = r.attend(q, lens)
    close(out, want, tol, "out")
    close(lse, want_lse, lse_tol, "lse")
    same_state(c, r)


@pytest.mark.parametrize("size", [2.0 ** -20, 2.0 ** 14, 2.0 ** 60])
def test_attend_query_sizes(size):
    """Queries far outside f16's range; with the large ones one entry takes all the weight."""
    lens = [100]
    c, r, g = filled(37, 1, 2, 64, 128, lens, 2, 2, "e4m3")
    q = rows(g, 1, 4, 2, 64, scale=size)
    lse = torch.zeros(1, 4, 2, device=DEV)
    out = c.attend(q, ints(lens), lse=lse)
    want, want_lse, tol, lse_tol = r.attend(q, lens)
    top = (want_lse.abs().amax() * 2.0 ** -18).item()
    if size < 2.0 ** 13:
        close(out, want, tol, "out")
        same_state(c, r)
    assert torch.isfinite(out).all()
    assert ((lse.cpu().double() - want_lse).abs() <= lse_tol + top).all()
    assert abs(float((c.score[:, :, :100].double().cpu().sum() - r.score[:, :, :100].sum()))) <= 1e-3


@pytest.mark.parametrize("kv", ["e4m3", "int8"])
@pytest.mark.parametrize("cap", [96, 1024])
def test_attend_huge_query_and_key(kv, cap):
    """A query of 2^70 and one key of -2^90 along it, the others across: its logit is below fp32's range and its weight 0,
    those of the entries beside it in its block are 0 and their weights equal."""
    d = 128
    c = H2OBlockCache(1, 1, d, cap, kv=kv)
    k, v = torch.zeros(1, 1, cap, d), torch.ones(1, 1, cap, d)
    k[0, 0, 40, 0], v[0, 0, 40] = -2.0 ** 90, 64.0
    c.append(k.bfloat16().to(DEV), v.bfloat16().to(DEV), ints([0]))
    q = torch.zeros(1, 1, 1, d, dtype=torch.bfloat16, device=DEV)
    q[..., 0] = 2.0 ** 70
    lse = torch.zeros(1, 1, 1, device=DEV)
    out = c.attend(q, ints([cap]), lse=lse)
    # all weights but one equal and of value 1: f16 and fp32 roundings of them (2^-11) and of the output (2^-8)
    assert ((out.float() - 1).abs() <= 2.0 ** -8 + 2.0 ** -11).all()
    # 2^-20: the logarithm's and its factors' roundings, at most 2^-22 each of log2(1023) < 10
    assert abs(float(lse) - math.log(cap - 1)) <= 2.0 ** -20 * 10
    score = c.score[0, 0].double()
    assert score[40] == 0
    score[40] = 1 / (cap - 1)
    assert ((score * (cap - 1) - 1).abs() <= 2.0 ** -18).all()


@pytest.mark.parametrize("B,H,G,n,cap,kv", [(2, 2, 2, 3, 256, "e4m3"), (1, 2, 4, 2, 704, "int8"), (20, 8, 1, 2, 640, "e4m3"),
                                            (1, 20, 1, 2, 65536, "e4m3"), (1, 48, 8, 2, 28672, "int8"), (1, 10, 8, 5, 5120, "e4m3")])
def test_nan_query_leaves_what_it_does_not_see(B, H, G, n, cap, kv):
    """A NaN in the first of several query tokens makes its output and the scores of the entries that it sees NaN.  The
    tokens behind it and the scores of the entries behind those are within the reference's tolerances (the rows of a
    head share the moves of their weights' reference), other heads have the bits of a run with a zero in its place."""
    d, total = 64, cap - 3
    a, _, g = filled(167, B, H, d, cap, [total] * B, G, n, kv, junk=False)
    z, r = H2OBlockCache(B, H, d, cap, group=G, max_queries=n, kv=kv), RefCache(1, 1, d, cap, G, kv)
    for name in ("K", "V", "K_scale", "V_scale", "pos", "score"):
        getattr(z, name).copy_(getattr(a, name))
        getattr(r, name).copy_(getattr(a, name)[:1, :1].cpu())
    q = rows(g, B, H * G, n, d)
    q[0, 0, 0, 5] = math.nan
    out = a.attend(q, ints([total] * B))
    want, _, tol, _ = r.attend(q[:1, :G], [total])
    assert out[0, 0, 0].isnan().all() and not out[0, :G].flatten(0, 1)[1:].isnan().any()
    close(out[:1, :G], want, tol, "out")
    seen = total - n + 1
    assert a.score[0, 0, :seen].isnan().all() and not a.score[0, 0, seen:].isnan().any()
    close(a.score[:1, :1, seen:], r.score[:, :, seen:], r.score_tol[:, :, seen:], "score")
    q[0, 0, 0, 5] = 0.0
    want = z.attend(q, ints([total] * B))
    out[0, :G] = want[0, :G] = a.score[0, 0] = z.score[0, 0] = 0.0
    assert torch.equal(out, want) and torch.equal(a.score, z.score) and a.error_bits() == 0


LARGE = [  # B, H, G, n, d, kv, cap, longest: a CTA a head, parts of heads joined, whole heads, many rows
    (1, 2, 1, 1, 128, "e4m3", 64, 50),
    (2, 2, 4, 2, 64, "int8", 512, 512),
    (3, 2, 2, 1, 128, "int8", 1024, 1000),
    (40, 8, 1, 1, 64, "e4m3", 544, 540),
    (8, 4, 2, 8, 128, "e4m3", 544, 540),
    (700, 4, 1, 1, 64, "e4m3", 64, 64),
    (3, 2, 8, 4, 128, "e4m3", 320, 300),
    (1, 1, 16, 16, 128, "int8", 96, 70),
    (1, 1, 1, 1, 64, "int8", 65536, 65500),
]


@pytest.mark.parametrize("case", LARGE, ids=str)
def test_attend_large_values(case):
    """Values up to 2^126, all of one sign: the sums before the division by the weights' sum lie beyond fp32, the
    outputs do not."""
    B, H, G, n, d, kv, cap, longest = case
    lens = [max(1, longest - 37 * b % longest) for b in range(B)]
    c, r, g = filled(139, B, H, d, cap, lens, G, n, kv, junk=False)
    if kv == "e4m3":
        c.V.view(torch.uint8).bitwise_and_(0x7F)
    else:
        c.V.abs_()
    c.V_scale.mul_(2.0 ** 123)
    load(r, c)
    q = rows(g, B, H * G, n, d)
    lse = torch.zeros(B, H * G, n, device=DEV)
    out = c.attend(q, ints(lens), lse=lse)
    assert torch.isfinite(out).all()
    want, want_lse, tol, lse_tol = r.attend(q, lens)
    close(out, want, tol, "out")
    close(lse, want_lse, lse_tol, "lse")
    same_state(c, r)
    out2 = c.attend(-q, ints(lens), accumulate=False)
    want, _, tol, _ = r.attend(-q, lens, accumulate=False)
    close(out2, want, tol, "out")


@pytest.mark.parametrize("kv", ["e4m3", "int8"])
@pytest.mark.parametrize("cap,d", [(256, 64), (8192, 128)])
@pytest.mark.parametrize("low,high", [(2.0 ** -100, 2.0 ** 60), (2.0 ** -60, 2.0 ** 117), (2.0 ** -3, 2.0 ** 117)])
def test_attend_large_values_without_weight(kv, cap, d, low, high):
    """Blocks of values up to 2^177 times larger, before and after the one whose first entry takes all the weight: the
    others' weights are below 2^-280, so that 2^13 entries of at most 2^126 add less than 2^-140 to its row."""
    g = torch.Generator(DEV).manual_seed(149)
    c = H2OBlockCache(1, 2, d, cap, kv=kv)
    K = torch.zeros(1, 2, cap, d, device=DEV)
    at = cap // 2
    K[:, :, at, 0] = 64.0
    c.append(K.bfloat16(), rows(g, 1, 2, cap, d), ints([0]))
    c.V_scale.fill_(high)
    c.V_scale[:, :, at // BLOCK] = low
    q = torch.zeros(1, 2, 1, d, dtype=torch.bfloat16, device=DEV)
    q[..., 0] = 200 * math.log(2) * d ** 0.5 / 64 * 1.5
    out = c.attend(q, ints([cap])).double()
    want = c.V[:, :, at].double()[:, :, None] * low
    # the entry's weight is one: half a step of f16 for it, of bf16 for the output
    assert ((out - want).abs() <= (2.0 ** -11 + 2.0 ** -8) * want.abs() * (1 + 2.0 ** -7) + 2.0 ** -140).all()


def test_attend_many_splits_long():
    """One head long enough that every worker of the device holds a part of it."""
    n = 70000
    cap = (n + 31) // 32 * 32
    c, r, g = filled(41, 1, 1, 64, cap, [n], 3, 2, "int8", junk=True)
    q = rows(g, 1, 3, 2, 64, scale=4.0)
    lse = torch.zeros(1, 3, 2, device=DEV)
    out = c.attend(q, ints([n]), lse=lse)
    want, want_lse, tol, lse_tol = r.attend(q, [n])
    close(out, want, tol, "out")
    close(lse, want_lse, lse_tol, "lse")
    same_state(c, r)


def test_attend_small_weights_next_to_a_large_one():
    """One entry holds nearly all the weight and 60,000 others 2^-25 of it each, with equal values: their share of the
    output (0.2 %) is not lost to the weights' rounding."""
    n = 60000
    c = H2OBlockCache(1, 1, 64, 60000 // 32 * 32 + 32, kv="int8")
    k = torch.zeros(1, 1, n, 64, device=DEV)
    k[0, 0, 77, 0] = 64.0
    v = torch.full((1, 1, n, 64), 100.0, device=DEV)
    v[0, 0, 77] = 1.0
    c.append(k.bfloat16(), v.bfloat16(), ints([0]))
    q = torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16, device=DEV)
    q[..., 0] = 25 * math.log(2) * 8 / 64
    out = c.attend(q, ints([n]))
    w = math.exp(-float(q[0, 0, 0, 0]) * 64 / 8)
    want = (1 + (n - 1) * w * 100) / (1 + (n - 1) * w)
    # the tail's weights: f16 half steps 2^-11 (2^-12 for a power of two's neighbours) of their share; bf16 2^-8 of the sum
    assert abs(float(out[0, 0, 0, 5]) - want) <= 2.0 ** -8 * want + 2.0 ** -11 * want


@pytest.mark.parametrize("H,G,n,cap,kv", [(20, 1, 1, 65536, "e4m3"), (48, 8, 2, 28672, "int8"), (10, 8, 5, 5120, "e4m3")])
def test_attend_forms_of_the_finishing_launch(H, G, n, cap, kv):
    """Few heads in many runs each, many rows over many entries, and many rows over few: some heads against the
    reference."""
    d, lens = 64, [cap - 77]
    g = torch.Generator(DEV).manual_seed(45)
    c = H2OBlockCache(1, H, d, cap, group=G, max_queries=n, kv=kv)
    c.append(rows(g, 1, H, cap, d), rows(g, 1, H, cap, d), ints([0]), score=torch.rand(1, H, cap, generator=g, device=DEV))
    refs = {}
    for h in (0, H // 3, H - 1):
        r = refs[h] = RefCache(1, 1, d, cap, G, kv)
        for name in ("K", "V", "K_scale", "V_scale", "score"):
            getattr(r, name).copy_(getattr(c, name)[:, h : h + 1].cpu().double())
    q = rows(g, 1, H * G, n, d, scale=2.0)
    lse = torch.zeros(1, H * G, n, device=DEV)
    out = c.attend(q, ints(lens), lse=lse)
    for h, r in refs.items():
        want, want_lse, tol, lse_tol = r.attend(q[:, h * G : h * G + G], lens)
        close(out[:, h * G : h * G + G], want, tol, f"out {h}")
        close(lse[:, h * G : h * G + G], want_lse, lse_tol, f"lse {h}")
        close(c.score[:, h : h + 1], r.score, r.score_tol, f"score {h}")
    assert c.error_bits() == 0


# ---------------------------------------------------------- scores over time

@pytest.mark.parametrize("B,H,G,n,cap,kv", [(1, 2, 1, 1, 256, "e4m3"), (1, 2, 4, 2, 704, "int8"), (20, 8, 1, 1, 640, "e4m3"),
                                            (1, 20, 1, 1, 65536, "e4m3"), (1, 48, 8, 2, 28672, "int8"), (1, 10, 8, 5, 5120, "e4m3")])
def test_scores_of_many_small_weights(B, H, G, n, cap, kv):
    """500 calls whose weights are each below a quarter of the half step of an entry's score add up: the score is off by
    a step of its own at most, and the weights by 2^-18 of them (2^-21 for each of the exponential, its argument's
    difference and the sum), not by a step a call."""
    calls, d, total = 500, 64, cap - 5
    g = torch.Generator(DEV).manual_seed(157)
    c = H2OBlockCache(B, H, d, cap, group=G, max_queries=n, kv=kv)
    w = G * n / total  # equal keys
    start = 2.0 ** (math.floor(math.log2(w)) + 27)  # half a step: 4 to 8 times w
    x = torch.ones(B, H, cap, d, dtype=torch.bfloat16, device=DEV)
    c.append(x, x, ints([0] * B), score=torch.full((B, H, cap), start, device=DEV))
    q, L = rows(g, B, H * G, n, d), ints([total] * B)
    out = torch.empty_like(q)
    for _ in range(calls):
        c.attend(q, L, causal=False, out=out)
    want = start + calls * w
    got = c.score[:, :, :total].double()
    assert ((got - want).abs() <= start * 2.0 ** -23 + calls * w * 2.0 ** -18).all()
    assert (c.score[:, :, total:] == start).all()
    # a score that the caller writes counts as written
    fresh = H2OBlockCache(B, H, d, cap, group=G, max_queries=n, kv=kv)
    fresh.append(x, x, ints([0] * B))
    c.score.zero_()
    for cache in (c, fresh):
        cache.attend(q, L, causal=False, out=out)
    assert torch.equal(c.score[:, :, :total], fresh.score[:, :, :total])
    assert c.error_bits() == 0


@pytest.mark.parametrize("B,H,cap,every", [(1, 2, 256, 2), (1, 2, 704, 5), (1, 400, 704, 5), (3, 24, 2048, 9)])
def test_small_weights_across_evictions(B, H, cap, every):
    """The same with an eviction of one entry after every few calls, fewer than their weights take to reach half a step:
    what the sums lost moves with the entries.  Every second entry takes all the weight, the others' is below 2^-57."""
    d, evictions = 64, 150
    c = H2OBlockCache(B, H, d, cap, kv="int8")
    k = torch.zeros(B, H, cap, d, device=DEV)
    k[:, :, ::2, 0], k[:, :, 1::2, 0] = -8.0, 8.0
    start = 2.0 ** 20 + 64.0 * torch.arange(cap, device=DEV)  # entry 0 goes first
    c.append(k.bfloat16(), k.bfloat16(), ints([0] * B), score=start.expand(B, H, cap).contiguous())
    q = torch.zeros(B, H, 1, d, dtype=torch.bfloat16, device=DEV)
    q[..., 0] = 20.0
    n, want = cap, start.double()
    for _ in range(evictions):
        odd = torch.arange(cap - n, cap, device=DEV) % 2 == 1
        assert every / int(odd.sum()) < 2.0 ** -4  # half a step of 2^20
        for _ in range(every):
            c.attend(q, ints([n] * B))
        want[cap - n :] += odd * (every / int(odd.sum()))
        c.evict(ints([n] * B), n - 1, 0)
        n -= 1
    got = c.score[:, :, :n].double()
    moved = want[cap - n :]
    assert float((moved - start[cap - n :]).max()) > 1  # eight steps of 2^-3 at least
    assert ((got - moved).abs() <= 2.0 ** -3 + (moved - start[cap - n :]) * 2.0 ** -18).all()
    assert torch.equal(c.pos[0, 0, :n].long(), torch.arange(cap - n, cap, device=DEV))


def test_attend_many_sequences():
    """More sequences than a warp looks over at once, most of them short, some empty."""
    B = 700
    lens = [(17 * b) % 33 for b in range(B)]
    c, r, g = filled(43, B, 1, 64, 32, lens, 2, 1, "int8")
    q = rows(g, B, 2, 1, 64)
    lse = torch.zeros(B, 2, 1, device=DEV)
    out = c.attend(q, ints(lens), lse=lse)
    want, want_lse, tol, lse_tol = r.attend(q, lens)
    close(out, want, tol, "out")
    close(lse, want_lse, lse_tol, "lse")
    same_state(c, r)


@pytest.mark.parametrize("kv", ["e4m3", "int8"])
def test_offsets_past_32_bits(kv):
    """4.6 GB of codes for K alone: the last head's append, attention, scores and eviction against those of a cache of
    that head's own."""
    H, cap, d, n = 512, 70016, 128, 69990
    g = torch.Generator(DEV).manual_seed(47)
    big, one = H2OBlockCache(1, H, d, cap, group=2, kv=kv), H2OBlockCache(1, 1, d, cap, group=2, kv=kv)
    for j in range(0, n, 23330):
        k, v = rows(g, 1, 1, 23330, d), rows(g, 1, 1, 23330, d)
        one.append(k, v, ints([j]))
        big.append(k.expand(1, H, 23330, d), v.expand(1, H, 23330, d), ints([j]))
    q = rows(g, 1, 2, 1, d, scale=2.0)
    a = big.attend(q.repeat(1, H, 1, 1), ints([n]))
    z = one.attend(q, ints([n]))
    for h in (0, 1, 300, H - 1):
        # the heads' blocks are shared out to workers differently: sums in another order
        assert torch.allclose(a[:, 2 * h : 2 * h + 2].float(), z.float(), atol=2e-3, rtol=2.0 ** -7), h
        assert torch.allclose(big.score[:, h, :n], one.score[:, 0, :n], rtol=1e-4, atol=1e-9), h
        assert torch.equal(big.K[:, h].view(torch.uint8), one.K[:, 0].view(torch.uint8))
    big.score.copy_(one.score.expand(1, H, cap))
    assert big.evict(ints([n]), 5000, 1000).tolist() == one.evict(ints([n]), 5000, 1000).tolist() == [6000]
    for name in ("K", "V", "K_scale", "V_scale", "pos", "score"):
        x, y = getattr(big, name), getattr(one, name)
        for h in (0, 257, H - 1):
            assert torch.equal(x[:, h].contiguous().view(torch.uint8), y[:, 0].contiguous().view(torch.uint8)), (name, h)
    assert big.error_bits() == one.error_bits() == 0


# --------------------------------------------------------------------- step

@pytest.mark.parametrize("kv,d,G,n", [("e4m3", 128, 1, 1), ("int8", 64, 4, 1), ("e4m3", 64, 3, 5), ("int8", 128, 8, 3), ("int8", 128, 1, 8)])
@pytest.mark.parametrize("layout", ["dense", "tokens"])
@pytest.mark.parametrize("cap", [224, 544])
def test_step_is_append_then_attend(kv, d, G, n, layout, cap):
    lens = [0, 1, 30, 32, 63, 200]
    counts = [n, max(n - 1, 0), n, 0, n, 1]
    a, r, g = filled(51, 6, 2, d, cap, lens, G, n, kv)
    z = H2OBlockCache(6, 2, d, cap, group=G, max_queries=n, kv=kv)
    for name in ("K", "V", "K_scale", "V_scale", "pos", "score"):
        getattr(z, name).copy_(getattr(a, name))
    q, k, v = rows(g, 6, 2 * G, n, d, layout), rows(g, 6, 2, n, d, layout), rows(g, 6, 2, n, d, layout)
    where = ints([x + 5 for x in lens])
    lse = torch.zeros(6, 2 * G, n, device=DEV)
    out = a.step(q, k, v, ints(lens), ints(counts), position=where, lse=lse)
    want, want_lse, tol, lse_tol = r.step(q, k, v, lens, counts, [x + 5 for x in lens])
    close(out, want, tol, "out")
    close(lse, want_lse, lse_tol, "lse")
    same_state(a, r)
    z.append(k, v, ints(lens), ints(counts), position=where)
    out2 = z.attend(q, ints([x + y for x, y in zip(lens, counts)]), ints(counts))
    assert torch.equal(out, out2)
    for name in ("K", "V", "K_scale", "V_scale", "pos", "score"):
        x, y = getattr(a, name), getattr(z, name)
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8)), name


# -------------------------------------------------------------------- evict

EVICT = [  # lens, k_heavy, k_local, n_sink, mode
    ([0, 1, 39, 40, 41, 64, 200, 173], 20, 20, 0, 0),
    ([0, 1, 39, 40, 41, 64, 200, 173], 40, 0, 3, 1),
    ([0, 1, 39, 40, 41, 64, 200, 173], 0, 40, 0, 0),
    ([224, 224, 1, 2, 3, 100, 50, 33], 1, 0, 1, 0),
    ([224, 223, 33, 32, 160, 161, 159, 96], 32, 1, 32, 1),
    ([224, 223, 33, 32, 160, 161, 159, 96], 7, 190, 0, 1),
]


@pytest.mark.parametrize("kv,d", [("e4m3", 128), ("int8", 64), ("e4m3", 64), ("int8", 128)])
@pytest.mark.parametrize("case", EVICT, ids=str)
def test_evict(case, kv, d):
    lens, kh, kl, sink, mode = case
    c, r, g = filled(61, 8, 3, d, 224, lens, kv=kv)
    gaps = torch.randint(1, 4, (8, 3, 224), generator=g, device=DEV)
    c.pos.copy_(gaps.cumsum(-1) - gaps[..., :1])
    r.pos.copy_(c.pos.cpu())
    where = [900 + b for b in range(8)]
    new = c.evict(ints(lens), kh, kl, n_sink=sink, score_mode=mode, position=ints(where))
    assert new.tolist() == r.evict(lens, kh, kl, sink, mode, where)
    same_state(c, r)
    assert c.error_bits() == 0


@pytest.mark.parametrize("kv", ["e4m3", "int8"])
def test_evict_ties_and_odd_scores(kv):
    """Equal scores, zeros of both signs, negative ones, infinities, NaN, and positions that repeat below n_sink."""
    lens = [300, 300, 300, 290]
    c, r, g = filled(67, 4, 2, 64, 320, lens, kv=kv, junk=False)
    c.score[0] = 1.0
    c.score[1] = torch.randint(-2, 3, (2, 320), generator=g, device=DEV).float() * 0.5
    c.score[1][c.score[1] == 0] = torch.tensor(-0.0, device=DEV)
    c.score[1, :, ::7] = 0.0
    c.score[2, :, ::3] = math.inf
    c.score[2, :, 1::5] = -math.inf
    c.score[2, :, 2::11] = math.nan
    c.score[3] = math.nan
    c.pos[3, :, 100:260] = 1
    load(r, c)
    new = c.evict(ints(lens), 90, 37, n_sink=5)
    assert new.tolist() == r.evict(lens, 90, 37, 5)
    same_state(c, r)


@pytest.mark.parametrize("kv", ["e4m3", "int8"])
def test_evict_rows_of_zeros_and_far_scales(kv):
    lens = [128]
    c, r, g = filled(71, 1, 2, 64, 128, lens, kv=kv, junk=False)
    for j, e in enumerate([100, -90, 3, -100]):
        c.K_scale[:, :, j] = 2.0 ** e
        c.V_scale[:, :, j] = 2.0 ** -e if e > -100 else 2.0 ** 60
    c.K.view(torch.uint8)[:, :, :32] = 0  # zeros under a scale of 2^100
    load(r, c)
    assert c.evict(ints(lens), 30, 30).tolist() == r.evict(lens, 30, 30)
    same_state(c, r)


def test_evict_mean_weight_without_positions():
    """score_mode 1 without positions: the lengths are the next positions."""
    lens = [200, 130]
    c, r, g = filled(77, 2, 2, 64, 224, lens, kv="int8")
    assert c.evict(ints(lens), 50, 40, score_mode=1).tolist() == r.evict(lens, 50, 40, 0, 1)
    same_state(c, r)


def test_evict_long():
    n, k = 60000, 9001
    c, r, g = filled(73, 1, 2, 64, 60000, [n], kv="e4m3", junk=False)
    new = c.evict(ints([n]), k - 4000, 4000)
    assert new.tolist() == r.evict([n], k - 4000, 4000)
    same_state(c, r)


@pytest.mark.parametrize("B,H,cap,lens,kv", [(2, 10, 8192, [8192, 5001], "e4m3"), (6, 10, 4096, [4001, 4096, 600, 599, 3333, 2048], "int8"),
                                             (12, 10, 2048, [2048 - 31 * b for b in range(12)], "e4m3"),
                                             (1, 240, 30016, [30011], "int8")], ids=str)
@pytest.mark.parametrize("mode", [0, 1])
def test_evict_shared_heads(B, H, cap, lens, kv, mode):
    """Heads taken by clusters of 8, 4 and 2 CTAs, and by one CTA with more candidates than it keeps in shared memory;
    the positions of all heads by a stable sort, the whole state of some."""
    d, kh, kl = 64, 401, 198
    g = torch.Generator(DEV).manual_seed(79)
    c = H2OBlockCache(B, H, d, cap, kv=kv)
    c.append(rows(g, B, H, cap, d), rows(g, B, H, cap, d), ints([0] * B), score=torch.rand(B, H, cap, generator=g, device=DEV).mul_(200).round_())
    refs = {}
    for b, h in [(0, 0), (B - 1, H - 1), (B // 2, H // 3)]:
        r = refs[b, h] = RefCache(1, 1, d, cap, 1, kv)
        for n in ("K", "V", "K_scale", "V_scale", "score"):
            getattr(r, n).copy_(getattr(c, n)[b : b + 1, h : h + 1].cpu().double())
        r.pos.copy_(c.pos[b : b + 1, h : h + 1].cpu().long())
    i = torch.arange(cap, device=DEV)
    n = ints(lens)[:, None, None].long()
    key = c.score / (cap - c.pos).clamp(min=1).float() if mode else c.score
    key = torch.where((i >= n - kl) | (c.pos < 3), math.inf, key)
    gone = torch.zeros_like(key, dtype=torch.bool).scatter_(2, key.sort(dim=-1, stable=True).indices, (i < n - (kh + kl)).expand(B, H, cap))
    kept = ~gone & (i < n)
    new = c.evict(ints(lens), kh, kl, n_sink=3, score_mode=mode, position=ints([cap] * B))
    assert new.tolist() == [min(x, kh + kl) for x in lens]
    for b in range(B):
        want = i.expand(H, cap)[kept[b]].view(H, -1)
        assert torch.equal(c.pos[b, :, : want.shape[1]].long(), want), b
    for (b, h), r in refs.items():
        r.evict([lens[b]], kh, kl, 3, mode, [cap])
        for name in ("K", "V", "K_scale", "V_scale", "score", "pos"):
            assert torch.equal(getattr(c, name)[b, h].cpu().double(), getattr(r, name)[0, 0].double()), (name, b, h)
    assert c.error_bits() == 0


@pytest.mark.parametrize("H,cap", [(80, 49152), (40, 98304), (16, 229376), (3, 425984)])
@pytest.mark.parametrize("mode", [0, 1])
def test_evict_more_candidates_than_a_cluster_holds(H, cap, mode):
    """Clusters of 2, 4, 8 and 16 CTAs whose share of the candidates is more than they keep in shared memory."""
    d, n, kh, kl = 64, cap - 13, cap // 9, 1001
    g = torch.Generator(DEV).manual_seed(163)
    c = H2OBlockCache(1, H, d, cap, kv="int8")
    for j in range(0, cap, cap // 8):
        c.append(rows(g, 1, H, cap // 8, d), rows(g, 1, H, cap // 8, d), ints([j]))
    c.score.copy_(torch.rand(1, H, cap, generator=g, device=DEV).mul_(500).round_())  # many equal ones
    score = c.score.clone()
    i = torch.arange(cap, device=DEV)
    key = score / (cap - i).clamp(min=1).float() if mode else score
    key = torch.where((i >= n - kl) | (i < 4), math.inf, key)
    order = key[..., :n].sort(dim=-1, stable=True).indices
    gone = torch.zeros(1, H, n, dtype=torch.bool, device=DEV).scatter_(2, order, (i[:n] < n - (kh + kl)).expand(1, H, n))
    want = i[:n].expand(1, H, n)[~gone].view(1, H, -1)
    rows_of = {}
    for name in ("K", "V"):
        scales = getattr(c, name + "_scale").double().repeat_interleave(BLOCK, 2)
        rows_of[name] = (getattr(c, name)[:, -1].double() * scales[:, -1, :, None])[0][want[0, -1]]
    assert c.evict(ints([n]), kh, kl, n_sink=4, score_mode=mode, position=ints([cap])).tolist() == [kh + kl]
    assert torch.equal(c.pos[:, :, : kh + kl].long(), want)
    assert torch.equal(c.score[:, :, : kh + kl], score.gather(2, want))
    r = RefCache(1, 1, d, cap, 1, "int8")
    for name in ("K", "V"):  # the last head's rows, quantised anew
        r._quantise(getattr(r, name)[0, 0], getattr(r, name + "_scale")[0, 0], rows_of[name].cpu(), 0, kh + kl)
        assert torch.equal(getattr(c, name)[0, -1, : kh + kl].cpu().double(), getattr(r, name)[0, 0, : kh + kl])
        used = (kh + kl + BLOCK - 1) // BLOCK
        assert torch.equal(getattr(c, name + "_scale")[0, -1, :used].cpu().double(), getattr(r, name + "_scale")[0, 0, :used])
    assert c.error_bits() == 0


@pytest.mark.parametrize("H,cap", [(3, 20480), (240, 4096)])
@pytest.mark.parametrize("every", [8, 16, 20, 40, 80])
def test_evict_scores_with_a_period(H, cap, every):
    """Scores whose largest (or least) values lie at regular distances, so that a regular sample of them misleads."""
    g = torch.Generator(DEV).manual_seed(113)
    c = H2OBlockCache(1, H, 64, cap, kv="int8")
    c.append(rows(g, 1, H, cap, 64), rows(g, 1, H, cap, 64), ints([0]))
    c.score.copy_(torch.rand(1, H, cap, generator=g, device=DEV))
    c.score[:, ::2, ::every] += 100
    c.score[:, 1::2, ::every] -= 100
    for kh in (cap // 7, 1, cap - 200):
        i = torch.arange(cap, device=DEV)
        score, pos = c.score.clone(), c.pos.clone()
        K, V, Ks, Vs = c.K.clone(), c.V.clone(), c.K_scale.clone(), c.V_scale.clone()
        key = torch.where(i >= cap - 100, math.inf, score)
        gone = torch.zeros_like(key, dtype=torch.bool).scatter_(2, key.sort(dim=-1, stable=True).indices, (i < cap - kh - 100).expand(1, H, cap))
        c.evict(ints([cap]), kh, 100)
        want = i.expand(1, H, cap)[~gone].view(1, H, -1)
        assert torch.equal(c.pos[:, :, : kh + 100].long(), want)
        assert torch.equal(c.score[:, :, : kh + 100], score.gather(2, want))
        for name, x in dict(score=score, pos=pos, K=K, V=V, K_scale=Ks, V_scale=Vs).items():
            getattr(c, name).copy_(x)


# -------------------------------------------------- used together, and where

def test_serving_run():
    """Prompts of different lengths, decode steps, an eviction, draft tokens of which some are taken back, another
    eviction: every output and the whole state against the reference throughout."""
    B, H, G, d, cap, kv = 4, 2, 4, 64, 192, "e4m3"
    g = torch.Generator(DEV).manual_seed(83)
    c, r = H2OBlockCache(B, H, d, cap, group=G, max_queries=4, kv=kv), RefCache(B, H, d, cap, G, kv)
    lens, pos = [0] * B, [0] * B

    def grow(by):
        for b in range(B):
            lens[b] += by[b]
            pos[b] += by[b]

    prompt = [100, 7, 64, 33]
    k, v, s = rows(g, B, H, 100, d), rows(g, B, H, 100, d), torch.rand(B, H, 100, generator=g, device=DEV)
    c.append(k, v, ints(lens), ints(prompt), score=s)
    r.append(k, v, lens, prompt, score=s)
    grow(prompt)
    for step in range(24):
        n = 4 if step % 5 == 4 else 1
        counts = [n - (b + step) % n for b in range(B)]
        q, k, v = rows(g, B, H * G, n, d, scale=3.0), rows(g, B, H, n, d), rows(g, B, H, n, d)
        out = c.step(q, k, v, ints(lens), ints(counts), position=ints(pos))
        want, _, tol, _ = r.step(q, k, v, lens, counts, pos)
        close(out, want, tol, f"step {step}")
        grow([max(1, m - step % 3) if m else 0 for m in counts])  # the last draft tokens taken back
        if step in (9, 17):
            load(r, c)  # the scores' roundings must not pick other entries than the kernel's
            new = c.evict(ints(lens), 24, 16, n_sink=2, score_mode=step % 2, position=ints(pos))
            lens = r.evict(lens, 24, 16, 2, step % 2, pos)
            assert new.tolist() == lens
        same_state(c, r)
    assert c.error_bits() == 0


@pytest.mark.parametrize("mode", [0, 1])
def test_positions_count_on_behind_evictions(mode):
    """Prompts, steps and evictions with lengths and positions kept apart: the positions of a head's entries increase
    throughout, end with the last token's, and rank by mean weight as the reference does."""
    B, H, G, d, cap = 3, 2, 2, 64, 96
    g = torch.Generator(DEV).manual_seed(173)
    c, r = H2OBlockCache(B, H, d, cap, group=G, kv="int8"), RefCache(B, H, d, cap, G, "int8")
    prompts, lengths = ints([40, 7, 61]), ints([0] * B)
    k, v = rows(g, B, H, 61, d), rows(g, B, H, 61, d)
    c.append(k, v, lengths, counts=prompts)
    r.append(k, v, [0] * B, [40, 7, 61])
    lengths = lengths + prompts
    position = lengths.clone()
    for t in range(60):
        q, k, v = rows(g, B, H * G, 1, d, scale=2.0), rows(g, B, H, 1, d), rows(g, B, H, 1, d)
        out = c.step(q, k, v, lengths, position=position)
        want, _, tol, _ = r.step(q, k, v, lengths.tolist(), position=position.tolist())
        close(out, want, tol, f"step {t}")
        lengths += 1
        position += 1
        if t % 20 == 19:
            load(r, c)
            new = c.evict(lengths, 20, 12, score_mode=mode, position=position)
            assert new.tolist() == r.evict(lengths.tolist(), 20, 12, 0, mode, position.tolist())
            lengths = new
        for b, n in enumerate(lengths.tolist()):
            assert (c.pos[b, :, 1:n] > c.pos[b, :, : n - 1]).all() and (c.pos[b, :, n - 1] == position[b] - 1).all()
        same_state(c, r)


def test_prefill_then_block_cache():
    """The prompt through H2OCache.prefill (its column sums are the scores), then the block cache."""
    from h2o_heavy_hitter_decode_gb300 import H2OCache
    B, H, d, L = 2, 3, 128, 200
    g = torch.Generator(DEV).manual_seed(89)
    Q, K, V = (rows(g, B, H, L, d) for _ in range(3))
    _, _, colsum = H2OCache(B, H, d, 16, 16).prefill(Q, K, V)
    c, r = H2OBlockCache(B, H, d, 256), RefCache(B, H, d, 256, 1, "e4m3")
    c.append(K, V, ints([0, 0]), score=colsum)
    r.append(K, V, [0, 0], score=colsum)
    assert c.evict(ints([L, L]), 40, 24).tolist() == r.evict([L, L], 40, 24) == [64, 64]
    q, k, v = (rows(g, B, H, 1, d) for _ in range(3))
    out = c.step(q, k, v, ints([64, 64]), position=ints([L, L]))
    want, _, tol, _ = r.step(q, k, v, [64, 64], position=[L, L])
    close(out, want, tol, "out")
    same_state(c, r)


@pytest.mark.parametrize("cap", [128, 640])
def test_captured_step_reads_current_lengths(cap):
    B, H, G, d = 3, 2, 2, 64
    lens = [10, 40, 63]
    c, r, g = filled(97, B, H, d, cap, lens, G, 1, "int8")
    z, _, _ = filled(97, B, H, d, cap, lens, G, 1, "int8")
    L = ints(lens)
    q, k, v = rows(g, B, H * G, 1, d), rows(g, B, H, 1, d), rows(g, B, H, 1, d)
    out = torch.zeros(B, H * G, 1, d, dtype=torch.bfloat16, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.step(q, k, v, L, out=out)  # warm-up outside of the capture, at the same lengths
    torch.cuda.current_stream().wait_stream(side)
    for name in ("K", "V", "K_scale", "V_scale", "pos", "score"):
        getattr(c, name).copy_(getattr(z, name))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.step(q, k, v, L, out=out)
        new = c.evict(L + 1, 30, 20)
    load(r, z)
    cur = lens
    for i in range(3):
        L.copy_(ints(cur))
        for x in (q, k, v):
            x.copy_(rows(g, *x.shape))
        graph.replay()
        want, _, tol, _ = r.step(q, k, v, cur)
        close(out, want, tol, f"replay {i}")
        cur = r.evict([x + 1 for x in cur], 30, 20)
        assert new.tolist() == cur
        same_state(c, r)


@pytest.mark.parametrize("cap", [512, 1024])
def test_other_stream(cap):
    lens = [500, 77]
    c, r, g = filled(101, 2, 2, 128, cap, lens, 2, 1, "e4m3")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    q, k, v = rows(g, 2, 4, 1, 128), rows(g, 2, 2, 1, 128), rows(g, 2, 2, 1, 128)
    L = ints(lens)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        out = c.step(q, k, v, L)
    s.synchronize()
    want, _, tol, _ = r.step(q, k, v, lens)
    close(out, want, tol, "out")
    same_state(c, r)


def test_dropped_while_another_stream_runs_its_call():
    """The workspace of a cache that is dropped with a call still to run on another stream is not given out again."""
    cap = 65536
    c, r, g = filled(151, 1, 2, 64, cap, [500], 2, 1, "int8", junk=False)
    q, k, v = rows(g, 1, 4, 1, 64), rows(g, 1, 2, 1, 64), rows(g, 1, 2, 1, 64)
    L, s = ints([500]), torch.cuda.Stream()
    other_cache = filled(151, 1, 2, 64, cap, [500], 2, 1, "int8", junk=False)[0]
    torch.cuda._sleep(1)
    other_cache.step(q, k, v, L)  # the kernels are loaded: a first launch may wait for the device
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(1_000_000_000)  # about half a second
        out = c.step(q, k, v, L)
    at, size = c.workspace.data_ptr(), c.workspace.numel()
    del c
    other = torch.empty(size, dtype=torch.uint8, device=DEV)
    assert not s.query() and not at <= other.data_ptr() < at + size
    other.fill_(0x7F)
    s.synchronize()
    want, _, tol, _ = r.step(q, k, v, [500])
    close(out, want, tol, "out")


def test_two_caches_on_two_streams():
    """Calls of different caches may overlap on the GPU: steps, attention with many rows and evictions of two caches on
    two streams at once give the bits that they give one after the other."""
    def script(c, g, lens, q1, k, v, q8, outs):
        L = ints(lens)
        for i in range(6):
            outs.append(c.step(q1, k, v, L).clone())
            L = L + 1
            outs.append(c.attend(q8, L).clone())
            L = c.evict(L, 700 - 40 * i, 300)
        outs += [L] + [getattr(c, n).clone() for n in ("K", "V", "K_scale", "V_scale", "pos", "score")]

    def setup(seed, kv):
        lens = [2000, 1500, 900, 33]
        c, _, g = filled(seed, 4, 6, 128, 2048, lens, 4, 8, kv, junk=False)
        return c, g, lens, rows(g, 4, 24, 1, 128), rows(g, 4, 6, 1, 128), rows(g, 4, 6, 1, 128), rows(g, 4, 24, 8, 128)

    want = []
    for seed, kv in ((131, "e4m3"), (137, "int8")):
        want.append([])
        script(*setup(seed, kv), want[-1])
    got, streams = [[], []], [torch.cuda.Stream(), torch.cuda.Stream()]
    both = [setup(131, "e4m3"), setup(137, "int8")]
    torch.cuda.synchronize()
    for s, args, outs in zip(streams, both, got):
        with torch.cuda.stream(s):
            script(*args, outs)
    torch.cuda.synchronize()
    for w, o in zip(want, got):
        assert len(w) == len(o)
        for x, y in zip(w, o):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_two_host_threads_with_caches_of_their_own():
    """Caches of other capacities, so of other amounts of shared memory, from two host threads on streams of their own:
    the same bits as one after the other."""
    import threading

    def work(seed, cap, outs):
        c, _, g = filled(seed, 2, 3, 64, cap, [cap - 40, 9], 4, 2, "int8", junk=False)
        q, k, v = rows(g, 2, 12, 2, 64), rows(g, 2, 3, 2, 64), rows(g, 2, 3, 2, 64)
        L = ints([cap - 40, 9])
        for i in range(12):
            outs.append(c.step(q, k, v, L).clone())
            L = c.evict(L + 2, cap // 2 - i, 10)
        outs += [L] + [getattr(c, n).clone() for n in ("K", "V", "K_scale", "V_scale", "pos", "score")]
        assert c.error_bits() == 0

    shapes = [(179, 512), (181, 96), (191, 20480), (193, 6144)]
    want = [[] for _ in shapes]
    for (seed, cap), outs in zip(shapes, want):
        work(seed, cap, outs)
    got, errors = [[] for _ in shapes], []

    def in_thread(seed, cap, outs):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                work(seed, cap, outs)
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001  (reported below)
            errors.append(e)

    threads = [threading.Thread(target=in_thread, args=(*s, o)) for s, o in zip(shapes, got)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for w, o in zip(want, got):
        assert len(w) == len(o)
        for x, y in zip(w, o):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_same_call_twice_gives_the_same_bits():
    lens = [3000, 1234, 17]
    outs = []
    for _ in range(2):
        c, _, g = filled(103, 3, 4, 128, 3008, lens, 4, 2, "e4m3")
        q = rows(g, 3, 16, 2, 128)
        lse = torch.zeros(3, 16, 2, device=DEV)
        out = c.attend(q, ints(lens), lse=lse)
        outs.append((out, lse, c.score[0, :, :3000].clone(), c.score[1, :, :1234].clone()))
    for x, y in zip(*outs):
        assert torch.equal(x, y)


# ------------------------------------------------------------------ refusals

def test_ranges_out_of_bounds_leave_the_sequence_alone():
    lens = [64, 64, 64, 64, 64]
    c, r, g = filled(107, 5, 2, 64, 96, lens, 2, 2, "int8")
    q, k, v = rows(g, 5, 4, 2, 64), rows(g, 5, 2, 2, 64), rows(g, 5, 2, 2, 64)
    out = torch.full((5, 4, 2, 64), 9.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((5, 4, 2), 9.0, device=DEV)
    bad_lens, bad_counts = [64, -1, 95, 64, 64], [2, 1, 2, 3, -1]
    c.step(q, k, v, ints(bad_lens), ints(bad_counts), out=out, lse=lse)
    assert c.error_bits() == 1
    assert (out[1:] == 9).all() and (lse[1:] == 9).all()
    want, _, tol, _ = r.step(q, k, v, bad_lens[:1] + [0] * 4, bad_counts[:1] + [0] * 4)
    close(out, want, tol, "out")
    same_state(c, r)
    c2, r2, _ = filled(109, 3, 2, 64, 96, [96] * 3)
    assert c2.evict(ints([97, -5, 96]), 10, 10).tolist() == [97, -5, 20]
    assert c2.error_bits() == 1
    r2.evict([0, 0, 96], 10, 10)
    same_state(c2, r2)


def test_arguments_rejected():
    c = H2OBlockCache(2, 2, 64, 64, group=2, max_queries=2, kv="int8")
    q, k = torch.zeros(2, 4, 1, 64, dtype=torch.bfloat16, device=DEV), torch.zeros(2, 2, 1, 64, dtype=torch.bfloat16, device=DEV)
    L, P = ints([0, 0]), ints([5, 5])
    c.step(q, k, k, L)
    bad = [
        lambda: c.step(q.float(), k, k, L), lambda: c.step(q, k.half(), k, L), lambda: c.step(q.cpu(), k, k, L),
        lambda: c.step(q[:1], k, k, L), lambda: c.step(q, k, k[:, :1], L), lambda: c.step(q, k, k, L.long()),
        lambda: c.step(q, k, k, ints([0])), lambda: c.step(q, k, k, L.cpu()), lambda: c.step(q, k, k, L, counts=L.float()),
        lambda: c.step(q[..., 0], k, k, L), lambda: c.step(None, k, k, L), lambda: c.step(q, k, k, None),
        lambda: c.step(q, k, k, L, lse=torch.zeros(2, 4, 2, device=DEV)),
        lambda: c.step(q, k, k, L, out=torch.zeros(2, 4, 1, 64, device=DEV)),
        lambda: c.step(q, k, k, L, out=torch.zeros(2, 1, 1, 64, device=DEV, dtype=torch.bfloat16).expand(2, 4, 1, 64)),
        lambda: c.step(q.transpose(1, 3).contiguous().transpose(1, 3), k, k, L),
        lambda: c.append(torch.zeros(2 * 2 * 65 + 1, dtype=torch.bfloat16, device=DEV)[1:261].view(2, 2, 65)[..., :64].unsqueeze(2), k, L),
        lambda: c.append(torch.zeros(2, 2, 65, 64, dtype=torch.bfloat16, device=DEV), torch.zeros(2, 2, 65, 64, dtype=torch.bfloat16, device=DEV), L),
        lambda: c.append(k, k, L, score=torch.zeros(2, 2, device=DEV)),
        lambda: c.attend(torch.zeros(2, 4, 3, 64, dtype=torch.bfloat16, device=DEV), L),
        lambda: c.evict(L, 0, 0), lambda: c.evict(L, -1, 4), lambda: c.evict(L, 4, -1), lambda: c.evict(L, 4, 4, n_sink=5),
        lambda: c.evict(L, 4, 4, score_mode=2), lambda: c.evict(L, 4, 4, new_lengths=L), lambda: c.evict(L, 4, 4, position=P, new_lengths=P), lambda: c.evict(L.float(), 4, 4),
        lambda: H2OBlockCache(2, 2, 96, 64), lambda: H2OBlockCache(2, 2, 64, 40), lambda: H2OBlockCache(2, 2, 64, 64, group=32, max_queries=9),
    ]
    for i, call in enumerate(bad):
        with pytest.raises((TypeError, ValueError, H2OError)):
            call()
            print("not refused:", i)
    assert c.error_bits() == 0


def test_new_cache_is_empty():
    c = H2OBlockCache(1, 2, 128, 64)
    assert (c.pos == -1).all() and (c.score == 0).all() and (c.K.float() == 0).all() and (c.V_scale == 0).all()
    q = torch.ones(1, 2, 1, 128, dtype=torch.bfloat16, device=DEV)
    assert (c.attend(q, ints([0])) == 0).all()
