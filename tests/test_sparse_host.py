"""H2OBlockCache's sparse calls on the host: the memory that a call uses without being given it lives until the call is
enqueued (CPU, with a stand-in for the library)."""
from __future__ import annotations

import gc
import weakref

import pytest
import torch

from h2o_heavy_hitter_decode_gb300 import HEADER_PATH, H2OBlockCache
from test_block_cache_threads import B, D, H, N, Library, cache_on_the_host


class Sparse(Library):
    """Calls that note their arguments, and whether every tensor in `made` is there meanwhile."""

    def __init__(self):
        super().__init__()
        self.inside.abort()
        self.made, self.calls = [], []

    def note(self, kind, n, n_blocks, n_first, n_last, blocks):
        gc.collect()
        alive = [t() for t in self.made]
        assert all(t is not None for t in alive), "memory of a call was given back before the call"
        assert blocks is None or any(t.data_ptr() == blocks and t.numel() == B * H * n * n_blocks for t in alive)
        self.calls.append((kind, n, n_blocks, n_first, n_last, blocks))
        return 0

    def h2o_bcache_attend_sparse(self, handle, n, q, lengths, counts, causal, accumulate, n_blocks, n_first, n_last, out,
                                 lse, blocks):
        return self.note("attend", n, n_blocks, n_first, n_last, blocks)

    def h2o_bcache_step_sparse(self, handle, n, q, k, v, lengths, counts, position, accumulate, n_blocks, n_first, n_last,
                               out, lse, blocks):
        return self.note("step", n, n_blocks, n_first, n_last, blocks)


def sparse_on_the_host(monkeypatch):
    c, _, here = cache_on_the_host(monkeypatch)
    c._lib = lib = Sparse()
    here.stream = 1
    empty = torch.empty

    def noted(*args, **kwargs):
        t = empty(*args, **kwargs)
        if t.dtype == torch.int32:
            lib.made.append(weakref.ref(t))
        return t

    monkeypatch.setattr(torch, "empty", noted)
    return c, lib


def call(c, kind, *choice, **more):
    q, k, v = (torch.zeros(B, H, N, D, dtype=torch.bfloat16) for _ in range(3))
    L = torch.zeros(B, dtype=torch.int32)
    return c.attend_sparse(q, L, *choice, **more) if kind == "attend" else c.step_sparse(q, k, v, L, *choice, **more)


@pytest.mark.parametrize("kind", ["attend", "step"])
def test_the_list_of_blocks_lives_until_the_call(monkeypatch, kind):
    c, lib = sparse_on_the_host(monkeypatch)
    call(c, kind, 1, 0, 1)
    assert len(lib.made) == len(lib.calls) == 1 and lib.calls[0][:5] == (kind, N, 1, 0, 1)
    mine = torch.zeros(B, H, N, 1, dtype=torch.int32)
    lib.made.append(weakref.ref(mine))
    lib.made.pop(0)
    call(c, kind, 1, 0, 1, blocks=mine)
    assert len(lib.made) == 1 and lib.calls[1][5] == mine.data_ptr()


@pytest.mark.parametrize("kind", ["attend", "step"])
def test_a_list_is_no_longer_than_the_cache(monkeypatch, kind):
    """More blocks than the cache has are all of them (here one): a list of 2^26 for each token and head would not fit a
    GPU.  A choice that is refused gets no memory at all, and reaches the library as it was given."""
    c, lib = sparse_on_the_host(monkeypatch)
    for choice in ((2, 1, 1), (1 << 26, 5, 1 << 25), (1 << 26, 0, 1), (1000, 0, 1000)):
        call(c, kind, *choice)
        assert lib.calls.pop()[:5] == (kind, N, 1, 0, 1)
        assert lib.made.pop()() is None  # one word a token and head was enough (note), and is gone with the call
    for bad in ((0, 0, 1), (-1, 0, 1), (1, 0, 0), (1, 1, 1), (1, -1, 2), (2 ** 26 + 1, 1, 1), (2 ** 31 - 1, 2 ** 31 - 1, 1),
                (1 << 26, 1 << 26, 1)):
        call(c, kind, *bad)
        assert lib.calls.pop() == (kind, N, *bad, None) and not lib.made
    with pytest.raises(ValueError):
        call(c, kind, 2 ** 31, 0, 1)
    # the caller's own list is as long as the caller says
    mine = torch.zeros(B, H, N, 7, dtype=torch.int32)
    lib.made.append(weakref.ref(mine))
    call(c, kind, 7, 2, 3, blocks=mine)
    assert lib.calls.pop() == (kind, N, 7, 2, 3, mine.data_ptr())


def test_the_largest_list_is_the_library_s():
    text = open(HEADER_PATH).read()
    assert "#define H2O_SPARSE_MAX_BLOCKS (1 << 26)" in text and H2OBlockCache._most_blocks == 1 << 26
