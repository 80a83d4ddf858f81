"""H2ORotary shared by host threads and used on several streams, and a block cache's copy out of another cache: each call
passes its own rows and stream, and memory that a stream reads is known to it (CPU, with a stand-in for the library)."""
from __future__ import annotations

import ctypes as C
import threading

import pytest
import torch

from h2o_heavy_hitter_decode_gb300 import H2OBlockCache, H2ORotary


class Library:
    """Calls that look at their arguments only once the other thread had the time to begin its own."""

    def __init__(self):
        self.seen, self.inside = [], threading.Barrier(2)

    def h2o_rotate(self, desc, dtype, B, n, hq, hk, q, k, position, per_token, counts, q_out, k_out, stream):
        try:
            self.inside.wait(0.3)
        except threading.BrokenBarrierError:
            pass
        self.seen.append((stream, B, n, hq, hk) + tuple((C.c_int64 * 4).from_address(r)[0] for r in (q, k, q_out, k_out)))
        return 0

    def h2o_bcache_copy(self, *args):
        self.seen.append(args)
        return 0

    def h2o_bcache_set_stream(self, handle, stream):
        return 0


def rotary_on_the_host():
    """A rotary object without a device: its tensors are CPU tensors (device index -1)."""
    lib, here = Library(), threading.local()
    r = H2ORotary.__new__(H2ORotary)
    r._lib, r.d, r.dims, r.axes, r.device, r._index = lib, 64, 64, 1, torch.device("cpu"), -1
    r._raw_stream, r._known, r._tables = (lambda index: here.stream), {1, 2}, []
    r._lock, r._slots, r._desc_at = threading.Lock(), (C.c_int64 * 16)(), 256
    r._slots_at = C.addressof(r._slots)
    r._current_device = lambda: -1
    return r, lib, here


def test_two_threads_pass_their_own_rows_and_streams():
    r, lib, here = rotary_on_the_host()
    want, errors = [], []

    def work(stream):
        try:
            here.stream = stream
            rows = [torch.zeros(2, 3 + stream, 4, 64, dtype=torch.bfloat16) for _ in range(4)]
            want.append((stream, 2, 4, 3 + stream, 3 + stream) + tuple(t.data_ptr() for t in rows))
            r.apply(rows[0], rows[1], torch.zeros(2, dtype=torch.int32), None, rows[2], rows[3])
        except Exception as e:  # noqa: BLE001  (reported by the test)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(s,)) for s in (1, 2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors and sorted(lib.seen) == sorted(want)


class Memory:
    """Stands for a tensor whose allocation learns of streams."""

    def __init__(self):
        self.streams = []

    def record_stream(self, stream):
        self.streams.append(stream)


def test_tables_know_their_streams(monkeypatch):
    r, lib, here = rotary_on_the_host()
    lib.inside.abort()
    r._known, r._tables = {1}, [Memory(), Memory()]
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: here.stream)
    q, k = (torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16) for _ in range(2))
    for here.stream in (1, 3, 1, 2, 3):
        r.apply(q, k, torch.zeros(1, dtype=torch.int32), None, q, k)
    assert [t.streams for t in r._tables] == [[3, 2], [3, 2]]
    assert [x[0] for x in lib.seen] == [1, 3, 1, 2, 3]


def test_a_copied_cache_knows_the_stream_that_reads_it(monkeypatch):
    lib, made = Library(), []
    for stream in (1, 2):
        c = H2OBlockCache.__new__(H2OBlockCache)
        c._lib, c._h, c._set_stream, c._index, c.device, c.B, c._per_seq = lib, None, stream, -1, torch.device("cpu"), 1, (1,)
        c._recorded, c._lock, c.workspace, c.bounds = {stream}, threading.Lock(), Memory(), Memory()
        made.append(c)
    to, source = made
    to._stream = lambda: 1
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: 1)
    one, other = torch.zeros(1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    for _ in range(2):
        to.copy(one, one, source, other)
    assert source.workspace.streams == source.bounds.streams == [1] and to.workspace.streams == []
    assert len(lib.seen) == 2 and lib.seen[0][3] == other.data_ptr()
    for bad in (dict(source=source), dict(source_lengths=other), dict(source=to, source_lengths=other)):
        with pytest.raises((ValueError, TypeError)):
            to.copy(one, one, **bad)
