"""GPU tests of H2OBlockCache's sparse attention (bounds, attend_sparse, step_sparse) against the 64-bit reference:
bounds, chosen blocks, codes and positions exactly, outputs, log-sum-exps and scores within its tolerances."""
from __future__ import annotations

import math

import pytest
import torch

from block_reference import BLOCK, close, load, same_state
from h2o_heavy_hitter_decode_gb300 import H2OBlockCache, H2OError
from sparse_reference import SparseRef

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


def filled(seed, B, H, d, cap, lens, group=1, max_queries=1, kv="e4m3", scale=1.0):
    """A cache with bounds and its reference with lens entries per sequence, keys of different sizes from block to block;
    places behind them hold other rows, e4m3 NaN codes, and scales and bounds that nothing may read."""
    g = torch.Generator(DEV).manual_seed(seed)
    c = H2OBlockCache(B, H, d, cap, group=group, max_queries=max_queries, kv=kv, bounds=True)
    k = rows(g, B, H, cap, d, scale=scale)
    k *= torch.exp2(torch.randint(-2, 3, (B, H, cap // BLOCK, 1, 1), generator=g, device=DEV).float()).expand(
        -1, -1, -1, BLOCK, -1).flatten(2, 3).bfloat16()
    c.append(k, rows(g, B, H, cap, d, scale=scale), ints([0] * B), counts=ints([min(cap, max(0, n)) for n in lens]),
             score=torch.rand(B, H, cap, generator=g, device=DEV) * 9)
    for b, n in enumerate(lens):
        n = min(cap, max(0, n))
        if kv == "e4m3":
            c.K.view(torch.uint8)[b, :, n:] = 0x7F
            c.V.view(torch.uint8)[b, :, n:] = 0xFF
        else:
            c.K[b, :, n:] = 99
        first = (n + BLOCK - 1) // BLOCK
        c.K_scale[b, :, first:] = math.inf
        c.V_scale[b, :, first:] = math.nan
        c.bounds[b, :, first:] = 101
        c.score[b, :, n:] = math.nan
    r = SparseRef(B, H, d, cap, group, kv)
    load(r, c)
    return c, r, g


def same_bounds(c, r, lens):
    for b, n in enumerate(lens):
        for h in range(c.H):
            want = r.bounds_of(b, h, n)
            assert torch.equal(c.bounds[b, h, : len(want)].cpu().long(), want), (b, h)


def same_lists(blocks, lists, n_blocks):
    got = blocks.cpu()
    for (b, h, t), mine in lists.items():
        assert got[b, h, t].tolist() == mine + [-1] * (n_blocks - len(mine)), (b, h, t)


def compare(c, r, out, lse, blocks, want, n_blocks):
    o, L, o_tol, L_tol, lists = want
    same_lists(blocks, lists, n_blocks)
    odd = L == math.inf  # rows that hold a NaN or an infinity
    nan_o, nan_L = out.cpu().double().isnan(), lse.cpu().double().isnan()
    assert bool(nan_o[odd].all()) and bool(nan_L[odd].all())
    o, L = o.clone(), L.clone()
    o[odd], L[odd] = math.nan, math.nan
    close(out, o, o_tol, "out")
    close(lse, L, L_tol, "lse")
    same_state(c, r)


# ------------------------------------------------------------------ bounds

@pytest.mark.parametrize("kv,d", [("e4m3", 128), ("e4m3", 64), ("int8", 128), ("int8", 64)])
def test_bounds_follow_every_call(kv, d):
    lens = [0, 1, 31, 32, 33, 95, 120]
    c, r, g = filled(3, 7, 2, d, 192, lens, kv=kv)
    same_bounds(c, r, lens)
    for n, counts in ((40, [40, 0, 1, 33, 31, 5, 64 - 24]), (1, None), (3, [3, 2, 1, 0, 3, 3, 3])):
        k, v = rows(g, 7, 2, n, d, "tokens", 2.0), rows(g, 7, 2, n, d)
        c.append(k, v, ints(lens), None if counts is None else ints(counts))
        r.append(k, v, lens, counts)
        lens = [a + (n if counts is None else z) for a, z in zip(lens, counts or [0] * 7)]
        same_bounds(c, r, lens)
    q, k, v = rows(g, 7, 2, 1, d), rows(g, 7, 2, 1, d, scale=8.0), rows(g, 7, 2, 1, d)
    c.step(q, k, v, ints(lens))
    r.step(q, k, v, lens)
    lens = [a + 1 for a in lens]
    same_bounds(c, r, lens)
    load(r, c)  # the scores
    new = c.evict(ints(lens), 20, 21).cpu().tolist()
    assert new == r.evict(lens, 20, 21)
    same_bounds(c, r, new)
    # what the caller writes
    c.K.view(torch.uint8).copy_(torch.where(c.K.view(torch.uint8) == 127, 0, c.K.view(torch.uint8)).flip(2))
    load(r, c)
    c.bounds.fill_(77)
    c.bound(ints(new))
    same_bounds(c, r, new)
    for b, n in enumerate(new):
        assert bool((c.bounds[b, :, (n + BLOCK - 1) // BLOCK :] == 77).all())
    assert c.error_bits() == 0
    c.bound(ints([-1, 193] + new[2:]))
    assert c.error_bits() == 1


def test_bounds_of_extreme_codes():
    """Every e4m3 number and every int8 code as the least and as the largest of a block."""
    for kv, codes in (("e4m3", [x for x in range(256) if x & 127 != 127]), ("int8", list(range(256)))):
        c = H2OBlockCache(1, len(codes), 64, 32, kv=kv, bounds=True)
        c.K.view(torch.uint8).copy_(torch.tensor(codes, dtype=torch.uint8, device=DEV)[None, :, None, None].expand(1, -1, 32, 64))
        c.K.view(torch.uint8)[:, :, 5:9, 3:] = 0
        c.K_scale.fill_(1.0)
        r = SparseRef(1, len(codes), 64, 32, 1, kv)
        load(r, c)
        for n in (1, 7, 32):
            c.bound(ints([n]))
            same_bounds(c, r, [n])


# ------------------------------------------------------------------ attend

ATTEND = [  # B, H, G, n, d, kv, cap, lens, counts, causal, (n_blocks, n_first, n_last)
    (1, 1, 1, 1, 128, "e4m3", 32, [1], None, True, (1, 0, 1)),
    (2, 1, 1, 1, 64, "int8", 96, [96, 0], None, True, (1, 0, 1)),
    (3, 2, 1, 1, 128, "int8", 512, [500, 0, 512], None, True, (4, 1, 2)),
    (9, 3, 2, 1, 64, "e4m3", 288, [1, 32, 33, 64, 65, 127, 160, 161, 288], None, True, (4, 1, 1)),
    (2, 2, 4, 1, 128, "e4m3", 2048, [2048, 1030], None, False, (9, 0, 1)),
    (3, 2, 8, 2, 128, "int8", 1024, [1000, 2, 577], [2, 1, 0], True, (7, 2, 2)),
    (2, 1, 5, 7, 64, "int8", 512, [512, 3], None, True, (6, 1, 1)),
    (2, 2, 1, 16, 128, "e4m3", 640, [630, 9], [16, 13], True, (5, 0, 3)),
    (2, 2, 3, 16, 64, "e4m3", 640, [630, 109], [16, 3], False, (3, 1, 2)),      # nothing left to choose
    (1, 2, 12, 3, 128, "e4m3", 1024, [1010], None, True, (8, 1, 2)),            # 12 rows a token
    (2, 1, 71, 1, 64, "int8", 512, [490, 31], None, True, (5, 1, 2)),           # one cached head for 71
    (1, 1, 128, 2, 128, "int8", 512, [470], [1], True, (5, 1, 2)),
    (1, 1, 256, 1, 128, "e4m3", 320, [320], None, True, (4, 0, 1)),
    (40, 8, 1, 1, 64, "e4m3", 256, [(37 * b) % 257 for b in range(40)], None, True, (3, 1, 1)),  # a CTA each
    (1, 2, 2, 1, 128, "e4m3", 8192, [8191], None, True, (17, 1, 2)),
    (1, 1, 1, 1, 64, "int8", 16384, [16384], None, True, (300, 3, 5)),
    (1, 2, 8, 1, 64, "e4m3", 16384, [16001], None, True, (509, 0, 1)),          # nearly all
    (1, 2, 8, 1, 64, "e4m3", 16384, [16001], None, True, (501, 0, 1)),          # all
    (1, 1, 2, 1, 64, "int8", 64, [64], None, True, (1000, 400, 500)),           # more than there are
    (3, 1, 1, 5, 64, "e4m3", 96, [2, 5, 40], None, True, (1, 0, 1)),            # fewer entries than queries
    (70, 8, 2, 1, 128, "int8", 160, [(53 * b) % 161 for b in range(70)], None, True, (3, 1, 1)),   # more heads than CTAs fit at once
    (60, 4, 3, 3, 64, "e4m3", 128, [(29 * b) % 129 for b in range(60)], [b % 4 for b in range(60)], True, (2, 0, 1)),
    (40, 4, 10, 1, 64, "int8", 128, [(31 * b) % 129 for b in range(40)], None, False, (2, 0, 1)),  # 10 rows a token
]


# every layout of the smaller ones
EACH = [(c, x) for c in ATTEND for x in ("dense", "tokens", "slice", "broadcast") if x == "dense" or c[1] * c[2] * c[3] * max(c[7]) <= 40000]


@pytest.mark.parametrize("case,layout", EACH, ids=lambda c: c if isinstance(c, str) else "-".join(
    str(x) for x in c[:7]) + f"-{c[9]}-{c[10]}".replace(" ", ""))
def test_attend(case, layout):
    B, H, G, n, d, kv, cap, lens, counts, causal, choice = case
    c, r, g = filled(21, B, H, d, cap, lens, G, n, kv)
    q = rows(g, B, H * G, n, d, layout, 1.5)
    out = torch.full((B, H * G, n, d), 5.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((B, H * G, n), 5.0, device=DEV)
    blocks = torch.full((B, H, n, choice[0]), -7, dtype=torch.int32, device=DEV)
    cnt = None if counts is None else ints(counts)
    for accumulate in (True, False):
        c.attend_sparse(q, ints(lens), *choice, counts=cnt, causal=causal, accumulate=accumulate, out=out, lse=lse, blocks=blocks)
        compare(c, r, out, lse, blocks, r.attend_sparse(q, lens, *choice, counts, causal, accumulate), choice[0])
    for b in range(B):
        z = n if counts is None else counts[b]
        assert bool((out[b, :, z:] == 5).all()) and bool((lse[b, :, z:] == 5).all()) and bool((blocks[b, :, z:] == -7).all())
    assert c.error_bits() == 0


def test_all_blocks_is_attend():
    """Where nothing is left out the sparse form is the dense one: the same entries, tolerances of both."""
    lens = [700, 33, 1024]
    c, r, g = filled(4, 3, 2, 128, 1024, lens, 4, 2)
    q = rows(g, 3, 8, 2, 128)
    a = c.attend(q, ints(lens), accumulate=False)
    z = c.attend_sparse(q, ints(lens), 32, accumulate=False)
    _, _, tol, _ = r.attend(q, lens, accumulate=False)
    assert bool(((a.cpu().double() - z.cpu().double()).abs() <= 2 * tol).all())


def test_equal_keys_go_to_the_lowest_index():
    """Blocks with the same codes and scales, and queries of zeros: all keys equal."""
    for q_scale in (0.0, 1.0):
        c, r, g = filled(5, 1, 2, 64, 1024, [1024], 2, 1, "int8")
        one = rows(g, 1, 2, 32, 64).repeat(1, 1, 32, 1)
        c.append(one, one, ints([0]))
        load(r, c)
        q = rows(g, 1, 4, 1, 64, scale=q_scale)
        blocks = torch.zeros(1, 2, 1, 9, dtype=torch.int32, device=DEV)
        lse = torch.zeros(1, 4, 1, device=DEV)
        out = c.attend_sparse(q, ints([1000]), 9, 2, 3, lse=lse, blocks=blocks)
        assert blocks[0, 0, 0].tolist() == [0, 1, 2, 3, 4, 5, 29, 30, 31]
        compare(c, r, out, lse, blocks, r.attend_sparse(q, [1000], 9, 2, 3), 9)


@pytest.mark.parametrize("kv", ["e4m3", "int8"])
def test_scales_and_queries_from_end_to_end_of_bf16(kv):
    """Blocks of 2^-100 to 2^120 and rows of 2^-120 to 2^120: the choice stays exact."""
    g = torch.Generator(DEV).manual_seed(6)
    c = H2OBlockCache(4, 1, 64, 1024, group=3, kv=kv, bounds=True)
    size = torch.exp2(torch.linspace(-110, 118, 32, device=DEV).round())[torch.randperm(32, generator=g, device=DEV)]
    k = (torch.randn(4, 1, 1024, 64, generator=g, device=DEV) * size.repeat_interleave(32)[:, None]).bfloat16()
    c.append(k, rows(g, 4, 1, 1024, 64), ints([0] * 4))
    r = SparseRef(4, 1, 64, 1024, 3, kv)
    load(r, c)
    q = rows(g, 4, 3, 1, 64)
    for b, e in enumerate((-120, 0, 100, 120)):
        q[b] *= 2.0 ** e
    q[1, 1] *= 2.0 ** -30  # the group's rows share a scale
    blocks = torch.zeros(4, 1, 1, 7, dtype=torch.int32, device=DEV)
    c.attend_sparse(q, ints([1024] * 4), 7, 1, 1, accumulate=False, blocks=blocks)
    for b in range(4):
        mine = r.choose(q[b, :, 0].cpu().double(), b, 0, 1024, 7, 1, 1, r.bounds_of(b, 0, 1024))
        assert blocks[b, 0, 0].tolist() == mine


def test_queries_that_are_no_numbers():
    """A NaN counts 0 in the choice and an infinity the largest code; the row's output is NaN, the others' are not."""
    c, r, g = filled(7, 2, 2, 128, 1024, [1000, 900], 3, 2, "int8")
    q = rows(g, 2, 6, 2, 128)
    q[0, 1, 0, 17] = math.nan
    q[0, 4, 1, 3] = math.inf
    q[0, 5, 1, 90] = -math.inf
    q[1, 3, :, :] = math.nan
    lse = torch.zeros(2, 6, 2, device=DEV)
    blocks = torch.zeros(2, 2, 2, 6, dtype=torch.int32, device=DEV)
    out = c.attend_sparse(q, ints([1000, 900]), 6, lse=lse, blocks=blocks)
    compare(c, r, out, lse, blocks, r.attend_sparse(q, [1000, 900], 6, 1, 2), 6)


def test_scores_of_tokens_that_chose_the_same_blocks():
    """Eight tokens with nearly the same query: their weights meet in one order, call after call the same bits."""
    got = []
    for _ in range(2):
        c, r, g = filled(8, 2, 2, 64, 2048, [2000, 2048], 2, 8)
        q = (rows(g, 2, 4, 1, 64).float() * 2 + rows(g, 2, 4, 8, 64).float() * 0.05).bfloat16()
        lse, blocks = torch.zeros(2, 4, 8, device=DEV), torch.zeros(2, 2, 8, 10, dtype=torch.int32, device=DEV)
        out = c.attend_sparse(q, ints([2000, 2048]), 10, lse=lse, blocks=blocks)
        compare(c, r, out, lse, blocks, r.attend_sparse(q, [2000, 2048], 10, 1, 2), 10)
        got.append((out.clone(), lse.clone(), c.score.clone()))
    assert all(torch.equal(a.nan_to_num(3.5), z.nan_to_num(3.5)) for a, z in zip(*got))


def test_more_keys_than_shared_memory_holds():
    """65,536 blocks of one head, places past 2^27 bytes of codes."""
    cap = 1 << 21
    g = torch.Generator(DEV).manual_seed(10)
    c = H2OBlockCache(1, 1, 64, cap, group=2, max_queries=2, kv="int8", bounds=True)
    c.K.copy_(torch.randint(-90, 91, (1, 1, cap, 64), generator=g, device=DEV, dtype=torch.int8))
    c.V.copy_(torch.randint(-127, 128, (1, 1, cap, 64), generator=g, device=DEV, dtype=torch.int8))
    c.K_scale.fill_(2.0 ** -6)
    c.V_scale.fill_(2.0 ** -6)
    c.K_scale[0, 0, torch.randperm(cap // 32, generator=g, device=DEV)[:600]] = 2.0 ** -5
    n = cap - 45
    c.bound(ints([n]))
    q = rows(g, 1, 2, 2, 64)
    blocks = torch.zeros(1, 1, 2, 700, dtype=torch.int32, device=DEV)
    out = c.attend_sparse(q, ints([n]), 700, 4, 4, blocks=blocks)
    # the choice and the outputs in 64 bits on the device
    K = c.K[0, 0].view(-1, 32, 64)
    lo, hi = K.amin(1).double(), K.amax(1).double()
    lo[-2], hi[-2] = K[-2, :19].amin(0).double(), K[-2, :19].amax(0).double()
    for t in range(2):
        rows_t = q[0, :, t].double()
        e = math.ceil(math.log2(float(rows_t.abs().max()) / 127))
        x = torch.round(rows_t / 2.0 ** e)
        m = (x.clamp(min=0) @ hi.T + x.clamp(max=0) @ lo.T).amax(0) * c.K_scale[0, 0].double()
        end = n - 1 + t
        nb = -(-end // 32)
        best = (-m[4 : nb - 4]).sort(stable=True).indices[:692] + 4
        mine = torch.cat([torch.arange(4, device=DEV), best, torch.arange(nb - 4, nb, device=DEV)]).sort().values
        assert torch.equal(blocks[0, 0, t].long(), mine)
        at = (mine[:, None] * 32 + torch.arange(32, device=DEV)).flatten()
        at = at[at < end]
        k, v = c.K[0, 0, at].double() * c.K_scale[0, 0, at // 32, None].double(), c.V[0, 0, at].double() * 2.0 ** -6
        s = rows_t @ k.T / 8
        w = torch.softmax(s, -1)
        # 2^-23 (64 terms + 4) sum|q k| / 8 in logits of up to 22, 2^-11 of each weight, a half step of bf16
        e_w = 2 * 2.0 ** -23 * 68 * float((rows_t.abs() @ k.abs().T).max()) / 8 + 2.0 ** -21 * 98
        tol = 2.0 ** -8 * (w @ v).abs() + (e_w + 2.0 ** -11) * (w @ v.abs()) * (1 + 2.0 ** -7) + 1e-6
        assert bool(((out[0, :, t].double() - w @ v).abs() <= tol).all())
    assert c.error_bits() == 0


# -------------------------------------------------------------------- step

STEP = [  # B, H, G, n, d, kv, cap, lens, counts, (n_blocks, n_first, n_last)
    (1, 4, 1, 1, 128, "e4m3", 1024, [255], None, (4, 1, 1)),
    (1, 2, 1, 1, 64, "int8", 96, [0], None, (1, 0, 1)),
    (5, 2, 4, 1, 128, "int8", 512, [31, 32, 33, 480, 511], None, (5, 1, 2)),
    (3, 2, 8, 5, 64, "e4m3", 512, [500, 29, 0], [5, 4, 0], (6, 1, 1)),
    (2, 1, 3, 40, 64, "int8", 640, [60, 300], [40, 37], (4, 1, 1)),   # blocks fill within the call
    (2, 1, 1, 100, 128, "e4m3", 640, [31, 500], None, (3, 0, 1)),
]


@pytest.mark.parametrize("layout", ["dense", "tokens", "slice"])
@pytest.mark.parametrize("case", STEP, ids=lambda c: "-".join(str(x) for x in c[:7]).replace(" ", ""))
def test_steps(case, layout):
    B, H, G, n, d, kv, cap, lens, counts, choice = case
    c, r, g = filled(31, B, H, d, cap, lens, G, n, kv)
    cnt = None if counts is None else ints(counts)
    for i in range(4):
        if max(a + (n if counts is None else z) for a, z in zip(lens, counts or [0] * B)) > cap:
            break
        q, k, v = rows(g, B, H * G, n, d, layout), rows(g, B, H, n, d, layout, 1.0 + i), rows(g, B, H, n, d, layout)
        where = [900 * b + 7 * i for b in range(B)]
        lse, blocks = torch.zeros(B, H * G, n, device=DEV), torch.zeros(B, H, n, choice[0], dtype=torch.int32, device=DEV)
        out = c.step_sparse(q, k, v, ints(lens), *choice, counts=cnt, position=ints(where), lse=lse, blocks=blocks)
        compare(c, r, out, lse, blocks, r.step_sparse(q, k, v, lens, *choice, counts, where), choice[0])
        lens = [a + (n if counts is None else z) for a, z in zip(lens, counts or [0] * B)]
        same_bounds(c, r, lens)
    assert c.error_bits() == 0


@pytest.mark.parametrize("B,H,cap,length", [(1, 8, 131072, 130000), (2, 8, 32768, 32000), (8, 8, 8192, 8000), (16, 8, 40000 // 32 * 32, 39000),
                                            (16, 8, 4096, 4000), (40, 12, 2048, 2000), (3, 1, 64, 33)])
@pytest.mark.parametrize("kv", ["e4m3", "int8"])
def test_one_launch_is_append_and_attend(B, H, cap, length, kv):
    """A step of one token in every size of cluster, few and many candidates: the bits of the two calls."""
    twins = []
    for i in range(2):
        g = torch.Generator(DEV).manual_seed(16)
        c = H2OBlockCache(B, H, 64, cap, group=2, kv=kv, bounds=True)
        k, v = rows(g, B, H, cap, 64), rows(g, B, H, cap, 64)
        lens = ints([max(0, length - 31 * b) for b in range(B)])
        c.append(k, v, ints([0] * B), counts=lens)
        q, k, v = rows(g, B, 2 * H, 1, 64), rows(g, B, H, 1, 64, "tokens", 3.0), rows(g, B, H, 1, 64)
        out, lse = torch.zeros_like(q), torch.zeros(B, 2 * H, 1, device=DEV)
        blocks = torch.zeros(B, H, 1, 20, dtype=torch.int32, device=DEV)
        where = lens + 5
        for _ in range(2):
            if i == 0:
                c.step_sparse(q, k, v, lens, 20, position=where, out=out, lse=lse, blocks=blocks)
            else:
                c.append(k, v, lens, position=where)
                c.attend_sparse(q, lens + 1, 20, out=out, lse=lse, blocks=blocks)
            lens, where = lens + 1, where + 1
        assert c.error_bits() == 0
        twins.append([x.view(torch.uint8) for x in (out, lse, blocks, c.K, c.V, c.K_scale, c.V_scale, c.pos, c.score, c.bounds)])
    for a, z in zip(*twins):
        assert torch.equal(a, z)


def test_rejected_draft_tokens():
    """The smaller length takes tokens back, across the end of a block too; the next step's choice is the reference's."""
    c, r, g = filled(9, 2, 2, 64, 512, [300, 318], 2, 6)
    lens = [300, 318]
    for n, kept in ((6, 2), (6, 6), (6, 1), (3, 0), (6, 4)):
        q, k, v = rows(g, 2, 4, n, 64), rows(g, 2, 2, n, 64, scale=4.0), rows(g, 2, 2, n, 64)
        lse, blocks = torch.zeros(2, 4, n, device=DEV), torch.zeros(2, 2, n, 5, dtype=torch.int32, device=DEV)
        out = c.step_sparse(q, k, v, ints(lens), 5, 1, 1, lse=lse, blocks=blocks)
        compare(c, r, out, lse, blocks, r.step_sparse(q, k, v, lens, 5, 1, 1), 5)
        lens = [a + kept for a in lens]
        q = rows(g, 2, 4, 1, 64)
        lse, blocks = torch.zeros(2, 4, 1, device=DEV), torch.zeros(2, 2, 1, 5, dtype=torch.int32, device=DEV)
        out = c.attend_sparse(q, ints(lens), 5, 1, 1, lse=lse, blocks=blocks)
        compare(c, r, out, lse, blocks, r.attend_sparse(q, lens, 5, 1, 1), 5)


def test_lengths_out_of_range():
    c, r, g = filled(12, 4, 2, 64, 256, [200, 100, 250, 60], 2, 3)
    before = (c.K.clone(), c.score.clone(), c.bounds.clone())
    out = torch.full((4, 4, 3, 64), 5.0, dtype=torch.bfloat16, device=DEV)
    blocks = torch.full((4, 2, 3, 4), -7, dtype=torch.int32, device=DEV)
    q, k = rows(g, 4, 4, 3, 64), rows(g, 4, 2, 3, 64)
    c.step_sparse(q, k, k, ints([200, -1, 254, 60]), 4, 1, 2, counts=ints([4, 1, 3, -1]), out=out, blocks=blocks)
    assert bool((out == 5).all()) and bool((blocks == -7).all())
    for a, z in zip(before, (c.K, c.score, c.bounds)):
        assert torch.equal(a.view(torch.uint8), z.view(torch.uint8))
    assert c.error_bits() == 1


def test_graph_reads_the_lengths_of_its_replay():
    c, r, g = filled(13, 2, 2, 128, 1024, [700, 31], 4)
    q, k, v = (torch.empty(2, h, 1, 128, dtype=torch.bfloat16, device=DEV) for h in (8, 2, 2))
    lens, lse = ints([700, 31]), torch.zeros(2, 8, 1, device=DEV)
    out, blocks = torch.zeros_like(q), torch.zeros(2, 2, 1, 6, dtype=torch.int32, device=DEV)
    for t, h in ((q, 8), (k, 2), (v, 2)):
        t.copy_(rows(g, 2, h, 1, 128))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # the graph's first call is a plain one
        c.step_sparse(q, k, v, lens, 6, out=out, lse=lse, blocks=blocks)
    torch.cuda.current_stream().wait_stream(side)
    compare(c, r, out, lse, blocks, r.step_sparse(q, k, v, [700, 31], 6, 1, 2), 6)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.step_sparse(q, k, v, lens, 6, out=out, lse=lse, blocks=blocks)
    for i in range(3):
        lens += 1
        for t, h in ((q, 8), (k, 2), (v, 2)):
            t.copy_(rows(g, 2, h, 1, 128))
        graph.replay()
        compare(c, r, out, lse, blocks, r.step_sparse(q, k, v, [701 + i, 32 + i], 6, 1, 2), 6)


def test_two_caches_on_two_streams():
    made = [filled(40 + i, 2, 2, 64, 512, [500, 77], 2) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in made]
    lens, q = [500, 77], [rows(g, 2, 4, 1, 64) for _, _, g in made]
    outs = [(torch.zeros_like(x), torch.zeros(2, 4, 1, device=DEV), torch.zeros(2, 2, 1, 4, dtype=torch.int32, device=DEV)) for x in q]
    where = ints(lens)
    torch.cuda.synchronize()
    for _ in range(20):
        for (c, _, _), st, x, (o, L, bl) in zip(made, streams, q, outs):
            with torch.cuda.stream(st):
                c.attend_sparse(x, where, 4, 1, 1, out=o, lse=L, blocks=bl)
    torch.cuda.synchronize()
    for (c, r, _), x, (o, L, bl) in zip(made, q, outs):
        for _ in range(20):
            want = r.attend_sparse(x, lens, 4, 1, 1)
        compare(c, r, o, L, bl, want, 4)


def test_refusals():
    c = H2OBlockCache(2, 2, 64, 64, group=2, max_queries=2, bounds=True)
    plain = H2OBlockCache(2, 2, 64, 64, group=2, max_queries=2)
    q, k, lens = (torch.zeros(2, h, 1, 64, dtype=torch.bfloat16, device=DEV) for h in (4, 2, 2)), None, ints([0, 0])
    q, k, _ = q
    for choice in ((0, 0, 0), (3, 1, 0), (3, -1, 2), (3, 2, 2), (-1, 0, 1), (2, 2 ** 31 - 1, 2 ** 31 - 1)):
        with pytest.raises((H2OError, ValueError)):
            c.attend_sparse(q, lens, *choice)
        with pytest.raises((H2OError, ValueError)):
            c.step_sparse(q, k, k, lens, *choice)
    with pytest.raises(H2OError) as e:  # 2^26 + 1 places a token
        H2OBlockCache(1, 1, 64, 32, bounds=True).attend_sparse(q[:1, :1], lens[:1], 2 ** 26 + 1)
    assert e.value.status == 1
    for choice in ((2 ** 31, 0, 1), (3, 2 ** 40, 1)):
        with pytest.raises(ValueError):
            c.attend_sparse(q, lens, *choice)
    for x in (plain.attend_sparse, lambda *a: plain.step_sparse(q, k, k, *a[1:])):
        with pytest.raises(H2OError) as e:
            x(q, lens, 3)
        assert e.value.status == 2
    with pytest.raises(H2OError) as e:
        plain.bound(lens)
    assert e.value.status == 2
    wrong = torch.zeros(2, 2, 1, 4, dtype=torch.int32, device=DEV)
    for blocks in (wrong, wrong[..., :3], wrong[..., :3].long(), wrong[..., :3].contiguous().cpu()):
        with pytest.raises(ValueError):
            c.attend_sparse(q, lens, 3, blocks=blocks)
    with pytest.raises(ValueError):
        c.attend_sparse(q, lens.long(), 3)
    with pytest.raises(H2OError):
        c.attend_sparse(torch.zeros(2, 4, 3, 64, dtype=torch.bfloat16, device=DEV), lens, 3)
    assert c.bounds.shape == (2, 2, 2, 2, 64) and plain.bounds is None


@pytest.mark.parametrize("cap", [2048, 32768])
def test_keys_one_apart(cap):
    """Sums next to 2^21 that differ by 1, in an order of their own: few candidates, and more than a CTA takes."""
    g = torch.Generator(DEV).manual_seed(14)
    n = cap // 32
    c = H2OBlockCache(1, 1, 128, cap, kv="int8", bounds=True)
    c.K.fill_(127)
    step = torch.randperm(n, generator=g, device=DEV)
    low = (step % 128).to(torch.int8)          # times a query code of 1
    high = (step // 128).to(torch.int8)        # times a query code of 127, with 127 - low beside it
    c.K[0, 0, :, 126] = low.repeat_interleave(32)
    c.K[0, 0, :, 127] = high.repeat_interleave(32)
    c.K_scale.fill_(1.0)
    c.V_scale.fill_(1.0)
    c.bound(ints([cap]))
    q = torch.full((1, 1, 1, 128), 127.0, device=DEV).bfloat16()
    q[..., 126] = 1.0
    blocks = torch.zeros(1, 1, 1, 40, dtype=torch.int32, device=DEV)
    c.attend_sparse(q, ints([cap]), 40, 0, 1, accumulate=False, blocks=blocks)
    m = low.long() + 127 * high.long()
    best = (-m[: n - 1]).sort(stable=True).indices[:39].sort().values
    assert blocks[0, 0, 0, :39].tolist() == best.tolist()


@pytest.mark.parametrize("B,H,n,cap,len_", [(1, 8, 1, 131072, 130001), (1, 1, 1, 65536, 65536), (2, 4, 2, 65536, 65001),
                                            (40, 4, 1, 20000 // 32 * 32, 19900), (16, 2, 1, 32768, 32768)])
def test_forms_of_many_candidates(B, H, n, cap, len_):
    """Clusters of 16, 8, 4, 2 and one CTA, each with more candidates than a CTA takes: the choice on the device."""
    g = torch.Generator(DEV).manual_seed(15)
    c = H2OBlockCache(B, H, 64, cap, group=3, max_queries=n, kv="int8", bounds=True)
    c.K.copy_(torch.randint(-30, 31, c.K.shape, generator=g, device=DEV, dtype=torch.int8))
    c.V.copy_(torch.randint(-127, 128, c.V.shape, generator=g, device=DEV, dtype=torch.int8))
    c.K_scale.fill_(2.0 ** -5)
    c.V_scale.fill_(2.0 ** -6)
    lens = [len_ - 977 * b for b in range(B)]
    c.bound(ints(lens))
    q = rows(g, B, 3 * H, n, 64)
    blocks = torch.zeros(B, H, n, 30, dtype=torch.int32, device=DEV)
    lse = torch.zeros(B, 3 * H, n, device=DEV)
    out = c.attend_sparse(q, ints(lens), 30, 1, 2, lse=lse, blocks=blocks)
    for b in range(B):
        if lens[b] < 0:  # refused
            continue
        K = c.K[b].view(H, -1, 32, 64)
        lo, hi = K.amin(2).double(), K.amax(2).double()
        for t in range(n):
            end = lens[b] - n + t + 1
            nb = -(-end // 32)
            qt = q[b, :, t].double().view(H, 3, 64)
            e = torch.ceil(torch.log2(qt.abs().amax((1, 2)) / 127))
            x = torch.round(qt / torch.exp2(e)[:, None, None])
            m = (x.clamp(min=0) @ hi.transpose(1, 2) + x.clamp(max=0) @ lo.transpose(1, 2)).amax(1)[:, :nb]
            if nb > 30:
                best = (-m[:, 1 : nb - 2]).sort(dim=-1, stable=True).indices[:, :27] + 1
                ends = torch.tensor([0, nb - 2, nb - 1], device=DEV).expand(H, -1)
                mine = torch.cat([best, ends], 1).sort(-1).values
            else:  # all of them
                mine = torch.arange(nb, device=DEV).expand(H, -1)
            assert torch.equal(blocks[b, :, t, : mine.shape[1]].long(), mine), b
            assert bool((blocks[b, :, t, mine.shape[1] :] == -1).all())
            if nb == 0:
                assert bool((out[b, :, t] == 0).all()) and bool((lse[b, :, t] == -math.inf).all())
                continue
            at = (mine[:, :, None] * 32 + torch.arange(32, device=DEV)).flatten(1)
            h = torch.arange(H, device=DEV)[:, None]
            k, v = c.K[b][h, at].double() * 2.0 ** -5, c.V[b][h, at].double() * 2.0 ** -6
            s = (qt @ k.transpose(1, 2) / 8).masked_fill((at >= end)[:, None], -math.inf)
            w = torch.softmax(s, -1)
            e_w = 2 * 2.0 ** -23 * 68 * float((qt.abs() @ k.abs().transpose(1, 2)).max()) / 8 + 2.0 ** -21 * 98
            want, mass = (w @ v).flatten(0, 1), (w @ v.abs()).flatten(0, 1)
            tol = 2.0 ** -8 * want.abs() + (e_w + 2.0 ** -11) * mass * (1 + 2.0 ** -7) + 1e-6
            assert bool(((out[b, :, t].double() - want).abs() <= tol).all())
            L = torch.logsumexp(s, -1).flatten()
            assert bool(((lse[b, :, t].double() - L).abs() <= e_w + 2.0 ** -21 * (1 + L.abs())).all())
    # every row's weights add up to 1, within e_w and the fp32 sums of scores
    seen = sum(a - n + t + 1 > 0 for a in lens for t in range(n)) * H * 3
    assert abs(float(c.score.double().sum()) - seen) <= seen * (e_w + 2.0 ** -20)
    assert c.error_bits() == (1 if min(lens) < 0 else 0)


def test_offsets_past_32_bits():
    """A second sequence whose codes lie behind 2^31 bytes of the first's: attention to its end, and a copy of it."""
    cap = 1 << 24
    g = torch.Generator(DEV).manual_seed(17)
    c = H2OBlockCache(2, 1, 128, cap, group=2, kv="int8", bounds=True)
    c.K.random_(-30, 31, generator=g)
    c.V.random_(-127, 128, generator=g)
    c.K_scale.fill_(2.0 ** -5)
    c.V_scale.fill_(2.0 ** -6)
    lens = [1000, cap - 7]
    c.K_scale[1, 0, -5000:] = 2.0 ** -4  # the choice lies behind
    q, k = rows(g, 2, 2, 1, 128), rows(g, 2, 1, 1, 128)
    c.bound(ints(lens))
    blocks, lse = torch.zeros(2, 1, 1, 70, dtype=torch.int32, device=DEV), torch.zeros(2, 2, 1, device=DEV)
    out = c.step_sparse(q, k, k, ints(lens), 70, 2, 3, lse=lse, blocks=blocks)
    K = c.K[1, 0].view(-1, 32, 128)
    x = q[1, :, 0].double()
    x = torch.round(x / 2.0 ** math.ceil(math.log2(float(x.abs().max()) / 127)))
    m = torch.zeros(cap // 32, dtype=torch.float64, device=DEV)
    for a in range(0, cap // 32, 1 << 16):
        lo, hi = K[a : a + (1 << 16)].amin(1).double(), K[a : a + (1 << 16)].amax(1).double()
        m[a : a + (1 << 16)] = (x.clamp(min=0) @ hi.T + x.clamp(max=0) @ lo.T).amax(0)
    m *= c.K_scale[1, 0].double()
    nb = cap // 32
    best = (-m[2 : nb - 3]).sort(stable=True).indices[:65] + 2
    ends = torch.tensor([0, 1, nb - 3, nb - 2, nb - 1], device=DEV)
    mine = torch.cat([best, ends]).sort().values
    assert torch.equal(blocks[1, 0, 0].long(), mine) and int(mine[2]) >= nb - 5000
    at = (mine[:, None] * 32 + torch.arange(32, device=DEV)).flatten()
    at = at[at < lens[1] + 1]
    key = c.K[1, 0, at].double() * c.K_scale[1, 0, at // 32, None].double()
    v = c.V[1, 0, at].double() * c.V_scale[1, 0, at // 32, None].double()
    s = q[1, :, 0].double() @ key.T / math.sqrt(128)
    w = torch.softmax(s, -1)
    size = float((q[1, :, 0].double().abs() @ key.abs().T).max()) / math.sqrt(128)
    e_s = 2.0 ** -23 * (128 * size + 4 * float(s.abs().max()))
    e_w = 2 * e_s + 2.0 ** -21 * 98
    want, mass = w @ v, w @ v.abs()
    assert bool(((out[1, :, 0].double() - want).abs() <= 2.0 ** -8 * want.abs() + (e_w + 2.0 ** -11) * mass * (1 + 2.0 ** -7) + 1e-6).all())
    L = torch.logsumexp(s, -1)
    assert bool(((lse[1, :, 0].double() - L).abs() <= e_s + 2.0 ** -21 * (1 + L.abs())).all())
    assert bool(((c.score[1, 0, at].double() - w.sum(0)).abs() <= 2 * e_w * w.sum(0) + 2.0 ** -23).all())
    got = c.copy(ints([1, -1]), ints([1001, cap - 6]))
    assert got.tolist() == [cap - 6, cap - 6]
    for n in ("K", "V", "K_scale", "V_scale", "pos", "score", "bounds"):
        x = getattr(c, n)
        assert torch.equal(x[0], x[1]), n
    assert c.error_bits() == 0


def test_batches_of_nothing():
    """No real row, no entry, every sequence refused: the calls behind find what the ones before left."""
    c, r, g = filled(18, 3, 2, 64, 128, [100, 5, 64], 2, 3)
    q, k = rows(g, 3, 4, 3, 64), rows(g, 3, 2, 3, 64)
    before = [getattr(c, n).clone().view(torch.uint8) for n in ("K", "score", "bounds", "pos")]
    out = torch.full((3, 4, 3, 64), 5.0, dtype=torch.bfloat16, device=DEV)
    blocks = torch.full((3, 2, 3, 3), -7, dtype=torch.int32, device=DEV)
    c.step_sparse(q, k, k, ints([100, 5, 64]), 3, counts=ints([0, 0, 0]), out=out, blocks=blocks)
    c.attend_sparse(q, ints([100, 5, 64]), 3, counts=ints([0, 0, 0]), out=out, blocks=blocks)
    assert c.error_bits() == 0
    c.step_sparse(q, k, k, ints([-1, 129, 126]), 3, out=out, blocks=blocks)
    assert c.error_bits() == 1
    assert bool((out == 5).all()) and bool((blocks == -7).all())
    for a, n in zip(before, ("K", "score", "bounds", "pos")):
        assert torch.equal(a, getattr(c, n).view(torch.uint8))
    lse = torch.zeros(3, 4, 3, device=DEV)
    for causal in (True, False):  # nothing to see
        out = c.attend_sparse(q, ints([0, 0, 0]), 3, causal=causal, lse=lse, blocks=blocks)
        assert bool((out == 0).all()) and bool((lse == -math.inf).all()) and bool((blocks == -1).all())
    for a, n in zip(before, ("K", "score", "bounds", "pos")):
        assert torch.equal(a, getattr(c, n).view(torch.uint8))
    out = c.step_sparse(q, k, k, ints([100, 5, 64]), 3, 0, 1, lse=lse, blocks=blocks)
    compare(c, r, out, lse, blocks, r.step_sparse(q, k, k, [100, 5, 64], 3, 0, 1), 3)


def test_two_graphs_of_one_cache():
    """A step of one token and one of three, captured apart and replayed in turn: they share the cache and its scratch."""
    c, r, g = filled(19, 2, 2, 128, 1024, [600, 40], 3, 3)
    lens = ints([600, 40])
    made = []
    for n in (1, 3):
        q, k, v = rows(g, 2, 6, n, 128), rows(g, 2, 2, n, 128), rows(g, 2, 2, n, 128)
        out, lse = torch.zeros_like(q), torch.zeros(2, 6, n, device=DEV)
        blocks = torch.zeros(2, 2, n, 5, dtype=torch.int32, device=DEV)
        side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            c.step_sparse(q, k, v, lens, 5, out=out, lse=lse, blocks=blocks)
        torch.cuda.current_stream().wait_stream(side)
        r.step_sparse(q, k, v, lens.tolist(), 5, 1, 2)
        with torch.cuda.graph(graph):
            c.step_sparse(q, k, v, lens, 5, out=out, lse=lse, blocks=blocks)
        made.append((n, q, k, v, out, lse, blocks, graph))
    for i in range(4):
        n, q, k, v, out, lse, blocks, graph = made[i % 2]
        q.copy_(rows(g, 2, 6, n, 128)), k.copy_(rows(g, 2, 2, n, 128)), v.copy_(rows(g, 2, 2, n, 128))
        graph.replay()
        compare(c, r, out, lse, blocks, r.step_sparse(q, k, v, lens.tolist(), 5, 1, 2), 5)
        lens += n
    assert c.error_bits() == 0
