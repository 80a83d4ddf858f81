"""H2OBlockCache shared by host threads, and used on several streams: each
call passes its own rows and stream, the workspace's allocation knows of
every stream, and numbers arrive whole (CPU, with a stand-in for the
library)."""
from __future__ import annotations

import ctypes as C
import threading

import pytest
import torch

from h2o_heavy_hitter_decode_gb300 import H2OBlockCache
from h2o_heavy_hitter_decode_gb300 import block_cache

B, H, D, N = 1, 1, 64, 2


class Library:
    """Calls that look at their arguments only once the other thread had the time to begin its own."""

    def __init__(self):
        self.stream, self.seen, self.inside = None, [], threading.Barrier(2)

    def h2o_bcache_set_stream(self, handle, stream):
        self.stream = stream.value
        return 0

    def _call(self, kind, *rows):
        try:
            self.inside.wait(0.3)
        except threading.BrokenBarrierError:
            pass
        self.seen.append((kind, self.stream) + tuple((C.c_int64 * 4).from_address(r)[0] for r in rows))
        return 0

    def h2o_bcache_append(self, handle, n, k, v, lengths, counts, position, score):
        return self._call("append", k, v)

    def h2o_bcache_attend(self, handle, n, q, lengths, counts, causal, accumulate, out, lse):
        return self._call("attend", q, out)

    def h2o_bcache_step(self, handle, n, q, k, v, lengths, counts, position, accumulate, out, lse):
        return self._call("step", q, k, v, out)

    def h2o_bcache_evict(self, handle, *args):
        return self._call("evict")


def cache_on_the_host(monkeypatch):
    """A cache object without a device: its tensors are CPU tensors (device index -1)."""
    lib = Library()
    monkeypatch.setattr(block_cache, "lib", lambda: lib)
    c = H2OBlockCache.__new__(H2OBlockCache)
    c._lib, c._h, c._set_stream, c._index, c.device = lib, None, None, -1, torch.device("cpu")
    c.B, c.H, c.d, c.capacity, c.group, c.max_queries = B, H, D, 32, 1, N
    c._heads, c._per_seq, c._recorded = H, (B,), {1, 2}
    c._lock = threading.Lock()
    c._slots = [(C.c_int64 * 4)() for _ in range(4)]
    c._slot_at = [C.addressof(s) for s in c._slots]
    here = threading.local()
    c._stream = lambda: here.stream
    return c, lib, here


@pytest.mark.parametrize("call", ["append", "attend", "step", "evict"])
def test_two_threads_pass_their_own_rows_and_streams(monkeypatch, call):
    c, lib, here = cache_on_the_host(monkeypatch)
    want, errors = [], []

    def work(stream):
        try:
            here.stream = stream
            q, k, v, out = (torch.zeros(B, H, N, D, dtype=torch.bfloat16) for _ in range(4))
            L = torch.zeros(B, dtype=torch.int32)
            args = {"append": (k, v), "attend": (q, out), "step": (q, k, v, out), "evict": ()}[call]
            want.append((call, stream) + tuple(t.data_ptr() for t in args))
            if call == "append":
                c.append(k, v, L)
            elif call == "attend":
                c.attend(q, L, out=out)
            elif call == "step":
                c.step(q, k, v, L, out=out)
            else:
                c.evict(L, 4, 4)
        except Exception as e:  # noqa: BLE001  (reported by the test)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(s,)) for s in (1, 2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    assert sorted(lib.seen) == sorted(want)


def test_the_workspace_knows_its_streams(monkeypatch):
    """Each stream but the one that the workspace was allocated on is recorded with it, before the first call there."""
    c, lib, here = cache_on_the_host(monkeypatch)
    seen = []

    class Workspace:
        def record_stream(self, stream):
            assert lib.stream != stream
            seen.append(stream)

    c.workspace, c._recorded, c._set_stream = Workspace(), {1}, 1
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: here.stream)
    lib.inside.abort()
    L = torch.zeros(B, dtype=torch.int32)
    for s in (1, 2, 1, 3, 2, 3):
        here.stream = s
        c.evict(L, 4, 4)
    assert seen == [2, 3]
    assert [x[1] for x in lib.seen] == [None, 2, 1, 3, 2, 3]


@pytest.mark.parametrize("name", ["k_heavy", "k_local", "n_sink", "score_mode"])
@pytest.mark.parametrize("value", [2 ** 31, 2 ** 32, 2 ** 32 + 4, 2 ** 64 + 4, -2 ** 32 + 4])
def test_numbers_beyond_32_bits_are_refused(monkeypatch, name, value):
    """2^32 + 4 is not 4."""
    c, lib, here = cache_on_the_host(monkeypatch)
    lib.inside.abort()
    here.stream = 1
    with pytest.raises(ValueError):
        c.evict(torch.zeros(B, dtype=torch.int32), **{"k_heavy": 4, "k_local": 4, name: value})
    assert not lib.seen


@pytest.mark.parametrize("at", range(6))
def test_shapes_beyond_the_types_are_refused(at):
    shape = [1, 1, 64, 32, 1, 1]
    shape[at] += 2 ** 64 if at == 3 else 2 ** 32
    with pytest.raises(ValueError):
        H2OBlockCache(*shape[:4], group=shape[4], max_queries=shape[5], device="cuda:0")
