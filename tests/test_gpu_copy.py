"""GPU tests of H2OBlockCache.copy: every byte of the blocks that move, and of those that stay, against indexing."""
from __future__ import annotations

import pytest
import torch

from h2o_heavy_hitter_decode_gb300 import H2OBlockCache, H2OError

pytestmark = pytest.mark.gpu

DEV = "cuda"
ENTRIES, BLOCKS = ("K", "V", "pos", "score"), ("K_scale", "V_scale", "bounds")


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def low_of(c):
    """What the scores' sums have lost: behind the scores, whose place the workspace pads to 256 bytes."""
    at = c.score.data_ptr() - c.workspace.data_ptr() + c.score.nbytes
    at = (at + 255) // 256 * 256
    return c.workspace[at : at + c.score.nbytes].view(torch.float32).view(c.score.shape)


def arrays(c):
    got = {n: getattr(c, n) for n in ENTRIES + BLOCKS if getattr(c, n) is not None}
    got["low"] = low_of(c)
    return {n: x.view(torch.uint8).reshape(*x.shape[:3], -1) for n, x in got.items()}


def noise(seed, B, H, d, cap, kv="e4m3", bounds=True, **more):
    """A cache whose arrays are random bytes."""
    g = torch.Generator(DEV).manual_seed(seed)
    c = H2OBlockCache(B, H, d, cap, kv=kv, bounds=bounds, **more)
    for x in arrays(c).values():
        x.copy_(torch.randint(0, 256, x.shape, generator=g, device=DEV, dtype=torch.uint8))
    return c


def expected(to, lens, parent, source=None, source_lens=None):
    """The arrays and lengths after a copy."""
    old = {n: x.clone() for n, x in arrays(source or to).items()}
    want, new = {n: x.clone() for n, x in arrays(to).items()}, list(lens)
    rows, cap = (source or to).B, (source or to).capacity
    lengths = lens if source is None else source_lens
    for b, p in enumerate(parent):
        if not 0 <= p < rows or not 0 <= lengths[p] <= min(cap, to.capacity):
            continue
        new[b], m = lengths[p], -(-lengths[p] // 32)
        for n in want:
            if n in old:
                e = m * 32 if n in ENTRIES + ("low",) else m
                want[n][b, :, :e] = old[n][p, :, :e]
    return want, new


def same(c, want):
    for n, x in arrays(c).items():
        assert torch.equal(x, want[n]), n


MAPS = [
    ("stay", 5, lambda b, B: b),
    ("cycle", 6, lambda b, B: (b + 1) % B),
    ("reverse", 7, lambda b, B: B - 1 - b),
    ("one to all", 9, lambda b, B: 4),
    ("beams", 12, lambda b, B: b - b % 4 + (0, 0, 3, 1)[b % 4]),
    ("some stay", 8, lambda b, B: -1 if b % 3 else (b + 3) % B),
    ("none", 4, lambda b, B: -1),
    ("many", 300, lambda b, B: (7 * b + 3) % B),
    ("chain", 70, lambda b, B: max(0, b - 1)),
]


@pytest.mark.parametrize("kv,d,cap,bounds", [("e4m3", 128, 128, True), ("int8", 64, 160, False), ("e4m3", 64, 32, True)])
@pytest.mark.parametrize("name,B,of", MAPS, ids=[m[0] for m in MAPS])
def test_in_place(name, B, of, kv, d, cap, bounds):
    c = noise(1, B, 3, d, cap, kv, bounds)
    lens = [(37 * b + 5) % (cap + 1) for b in range(B)]
    lens[0], lens[-1] = 0, cap
    parent = [of(b, B) for b in range(B)]
    want, new = expected(c, lens, parent)
    got = c.copy(ints(parent), ints(lens))
    assert got.tolist() == new
    same(c, want)
    assert c.error_bits() == 0


@pytest.mark.parametrize("B,rows", [(1, 1), (4, 1), (9, 2), (2, 70), (130, 5), (3, 4096), (4096, 1), (300, 4000)])
def test_from_another_cache(B, rows):
    """Other batch sizes, capacities, groups and numbers of queries."""
    to, source = noise(2, B, 2, 64, 256, "int8", group=4, max_queries=3), noise(3, rows, 2, 64, 96, "int8", max_queries=2)
    lens, source_lens = [(11 * b) % 257 for b in range(B)], [(29 * p + 96) % 97 for p in range(rows)]
    parent = [-1 if b % 5 == 4 else (3 * b) % rows for b in range(B)]
    want, new = expected(to, lens, parent, source, source_lens)
    before = {n: x.clone() for n, x in arrays(source).items()}
    got = to.copy(ints(parent), ints(lens), source, ints(source_lens))
    assert got.tolist() == new
    same(to, want)
    same(source, before)


def test_bounds_where_only_one_has_them():
    g = torch.Generator(DEV).manual_seed(4)
    lens, rows = [70, 33], torch.randn(2, 3, 96, 64, generator=g, device=DEV).bfloat16()
    for mine in (True, False):
        to, source = H2OBlockCache(3, 3, 64, 96, bounds=mine), H2OBlockCache(2, 3, 64, 96, bounds=not mine)
        source.append(rows, rows, ints([0, 0]), counts=ints(lens))
        got = to.copy(ints([1, 0, -1]), ints([0, 0, 0]), source, ints(lens))
        assert got.tolist() == [33, 70, 0] and (to.bounds is None) == (not mine)
        if mine:
            full = H2OBlockCache(2, 3, 64, 96, bounds=True)
            full.append(rows, rows, ints([0, 0]), counts=ints(lens))
            assert torch.equal(to.bounds[0, :, :2], full.bounds[1, :, :2])
            assert torch.equal(to.bounds[1, :, :3], full.bounds[0, :, :3])
        assert torch.equal(to.K[1, :, :70].view(torch.uint8), source.K[0, :, :70].view(torch.uint8))
        assert to.error_bits() == 0


def test_rows_out_of_range_stay():
    c = noise(5, 6, 2, 64, 96)
    lens, parent = [10, 97, -1, 60, 96, 5], [6, 2, 1, -2, 3, 4]
    want, new = expected(c, lens, parent)
    assert new == [10, 97, -1, 60, 60, 96]
    got = c.copy(ints(parent), ints(lens))
    assert got.tolist() == new
    same(c, want)
    assert c.error_bits() == 1
    # a source longer than the cache
    to, source = noise(6, 2, 2, 64, 64), noise(7, 2, 2, 64, 128)
    want, new = expected(to, [1, 2], [0, 1], source, [65, 64])
    assert to.copy(ints([0, 1]), ints([1, 2]), source, ints([65, 64])).tolist() == new == [1, 64]
    same(to, want)
    assert to.error_bits() == 1 and source.error_bits() == 0


def test_largest_batch():
    """4,096 rows, each read and written: pieces of 16 bytes."""
    c = noise(8, 4096, 1, 64, 32)
    lens = [b % 33 for b in range(4096)]
    parent = [(b * 1021 + 17) % 4096 for b in range(4096)]
    want, new = expected(c, lens, parent)
    assert c.copy(ints(parent), ints(lens)).tolist() == new
    same(c, want)
    with pytest.raises(H2OError) as e:
        H2OBlockCache(4097, 1, 64, 32).copy(ints([0] * 4097), ints([0] * 4097))
    assert e.value.status == 6


def test_many_heads_and_long_rows():
    c = noise(9, 5, 41, 128, 4096, "int8")
    lens, parent = [4096, 3999, 1, 2048, 3000], [1, 0, 4, 2, 2]
    want, new = expected(c, lens, parent)
    assert c.copy(ints(parent), ints(lens)).tolist() == new
    same(c, want)


def test_graph_and_streams():
    """A captured copy reads the map and lengths of its replay; a source on its own stream is waited for by the caller."""
    c = noise(10, 4, 3, 64, 96)
    parent, lens, new = ints([1, 2, 3, 0]), ints([96, 1, 40, 77]), ints([0] * 4)
    graph = torch.cuda.CUDAGraph()
    c.copy(ints([-1] * 4), lens)  # the first call raises the kernel's limit of shared memory
    with torch.cuda.graph(graph):
        c.copy(parent, lens, new_lengths=new)
    for p in ([1, 2, 3, 0], [0, 0, 0, 0], [3, 3, -1, 1]):
        parent.copy_(ints(p))
        want, after = expected(c, lens.tolist(), p)
        graph.replay()
        assert new.tolist() == after
        same(c, want)
        lens.copy_(new)
    side = torch.cuda.Stream()
    to = noise(11, 2, 3, 64, 96)
    want, after = expected(to, [0, 0], [3, 1], c, lens.tolist())
    zero, par = ints([0, 0]), ints([3, 1])
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = to.copy(par, zero, c, lens)
    torch.cuda.current_stream().wait_stream(side)
    assert got.tolist() == after
    same(to, want)


def test_refusals():
    c, lens = H2OBlockCache(2, 2, 64, 64), ints([0, 0])
    for args, more in [((None, lens), {}), ((lens[:1], lens), {}), ((lens.long(), lens), {}), ((lens, None), {}),
                       ((lens, lens), dict(source_lengths=lens)), ((lens, lens), dict(source=3)),
                       ((lens, lens, H2OBlockCache(3, 2, 64, 64), lens), {}), ((lens, lens, H2OBlockCache(2, 2, 64, 64)), {}),
                       ((lens.cpu(), lens), {})]:
        with pytest.raises((TypeError, ValueError)):
            c.copy(*args, **more)
    for other in (H2OBlockCache(2, 3, 64, 64), H2OBlockCache(2, 2, 128, 64), H2OBlockCache(2, 2, 64, 64, kv="int8")):
        with pytest.raises(H2OError):
            c.copy(lens, lens.clone(), other, lens.clone())
    both = ints([0, 0, 0])
    for new in (lens, both[1:]):
        with pytest.raises(H2OError):
            c.copy(ints([0, 1]), both[:2] if new is not lens else lens, new_lengths=new)
    with pytest.raises(H2OError):
        c.copy(lens, ints([0, 0]), new_lengths=lens)
    other = H2OBlockCache(2, 2, 64, 64)
    with pytest.raises(H2OError):
        c.copy(ints([0, 1]), ints([0, 0]), other, lens, new_lengths=lens)
