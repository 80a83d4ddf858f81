"""Block-scaled 8-bit K/V caches with grouped queries and bulk eviction
(``h2o_bcache_*`` of the C ABI): argument checks and marshalling only."""
from __future__ import annotations

import ctypes as C
import struct
import threading

import torch

from . import H2OError, _check, _ptr, lib

__all__ = ["H2OBlockCache"]

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
PACK = struct.Struct("4q").pack_into  # an h2o_rows
KV = {"e4m3": (0, torch.float8_e4m3fn), "int8": (1, torch.int8)}


def _whole(x, name, bits=31):
    """x as an integer that the library's type holds (ctypes would drop the bits above)."""
    n = int(x)
    if not -(1 << bits) <= n < 1 << bits:
        raise ValueError(f"{name} is out of range: {n}")
    return n


class H2OBlockCache:
    """Per (sequence, cached head) up to ``capacity`` entries in the order of
    their positions; ``group`` query heads share a cached head, and a call
    takes up to ``max_queries`` query tokens per sequence.

    The entries a sequence holds are the caller's to count: every call takes
    ``lengths``, an int32 [B] tensor on the device, so one tensor serves the
    caches of all layers and captured graphs read its current values.
    ``counts`` (int32 [B], optional) are the real rows of a padded batch.

    Draft tokens are taken back by passing the smaller length; the scales that
    they made grow, and what their queries added to scores, stay.

    K, V [B, H, capacity, d] are the codes (torch.float8_e4m3fn or torch.int8),
    K_scale, V_scale [B, H, capacity / 32] the scales of blocks of 32 entries
    (powers of two; an entry is code * scale), pos and score [B, H, capacity]
    the entries' positions and accumulated attention weights: views of the
    workspace, one torch uint8 tensor owned by this object.  With ``bounds`` the
    cache keeps, for ``step_sparse`` and ``attend_sparse``, bounds [B, H,
    capacity / 32, 2, d] (torch.int8): the least and largest code of each
    dimension of a block's keys (in units of 4 for e4m3).  Calls enqueue on
    torch's current CUDA stream of the cache's device; calls of one cache must
    not overlap on the GPU (host threads may share a cache: each call passes
    its own arguments and its own stream, one thread at a time).  A cache may
    be dropped with calls still running on any stream; one that a captured
    graph uses is kept for as long as the graph is replayed."""

    BLOCK = 32
    _most_blocks = 1 << 26  # H2O_SPARSE_MAX_BLOCKS
    bounds = None

    def __init__(self, B: int, H: int, d: int, capacity: int, group: int = 1, max_queries: int = 1, kv: str = "e4m3",
                 device=None, bounds: bool = False):
        L = self._lib = lib()
        if kv not in KV:
            raise ValueError(f"kv must be one of {sorted(KV)}, got {kv!r}")
        code, store = KV[kv]
        B, H, d, group, max_queries = (_whole(x, n) for x, n in ((B, "B"), (H, "H"), (d, "d"), (group, "group"),
                                                                 (max_queries, "max_queries")))
        capacity = _whole(capacity, "capacity", 63)
        self.B, self.H, self.d, self.capacity, self.group, self.max_queries = B, H, d, capacity, group, max_queries
        self.kv = kv
        self.device = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
        if self.device.type != "cuda":
            raise ValueError("H2OBlockCache lives on a CUDA device")
        if self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self._index = self.device.index
        # torch.cuda.current_stream(device).cuda_stream without its objects; a torch without CUDA has no such function
        self._raw_stream = torch._C._cuda_getCurrentRawStream
        shape = (B, H, d, capacity, group, max_queries, code)
        with torch.cuda.device(self.device):
            nbytes = L.h2o_bcache_workspace_bytes(*shape)
            if nbytes == 0:
                raise H2OError(1, f"h2o_bcache_workspace_bytes{shape}")
            self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
            h = C.c_void_p()
            stream = self._stream()
            _check(L.h2o_bcache_create(*shape, _ptr(self.workspace), C.c_void_p(stream), C.byref(h)),
                   "h2o_bcache_create")
        self._h, self._set_stream = h, stream
        self._recorded = {stream}  # streams that the workspace's allocation knows of
        self._heads, self._per_seq = H * group, (B,)
        # h2o_rows of q, k, v and out, filled in by each call; the lock covers them and the handle's stream until the call
        # is enqueued
        self._lock = threading.Lock()
        self._slots = [(C.c_int64 * 4)() for _ in range(4)]
        self._slot_at = [C.addressof(s) for s in self._slots]
        at = [C.c_void_p() for _ in range(6)]
        _check(L.h2o_bcache_arrays(h, *[C.byref(p) for p in at]), "h2o_bcache_arrays")
        rows, blocks = (B, H, capacity), (B, H, capacity // self.BLOCK)
        self.K, self.V = self._view(at[0], store, rows + (d,)), self._view(at[1], store, rows + (d,))
        self.K_scale, self.V_scale = self._view(at[2], torch.float32, blocks), self._view(at[3], torch.float32, blocks)
        self.pos, self.score = self._view(at[4], torch.int32, rows), self._view(at[5], torch.float32, rows)
        if bounds:
            with torch.cuda.device(self.device):
                self.bounds = torch.zeros(blocks + (2, d), dtype=torch.int8, device=self.device)
            assert self.bounds.nbytes == L.h2o_bcache_bounds_bytes(h)
            _check(L.h2o_bcache_set_bounds(h, _ptr(self.bounds)), "h2o_bcache_set_bounds")

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None:
            self._lib.h2o_bcache_destroy(h)
            self._h = None

    # -------------------------------------------------------------- helpers
    def _view(self, p, dtype, shape):
        at = p.value - self.workspace.data_ptr()
        n = dtype.itemsize
        for s in shape:
            n *= s
        return self.workspace[at : at + n].view(dtype).view(shape)

    def _stream(self) -> int:
        return self._raw_stream(self._index)

    def _use_stream(self):
        s = self._stream()
        if s != self._set_stream:
            self._record(s)
            _check(self._lib.h2o_bcache_set_stream(self._h, C.c_void_p(s)), "h2o_bcache_set_stream")
            self._set_stream = s

    def _record(self, s):
        """The current stream, s, runs kernels on this cache's memory: a cache that is dropped meanwhile keeps it until
        they are done."""
        if s not in self._recorded:
            for t in (self.workspace, self.bounds):
                if t is not None:
                    t.record_stream(torch.cuda.current_stream(self.device))
            self._recorded.add(s)

    def _dense(self, t, dtype, shape, name):
        """Address of a contiguous tensor, None for None."""
        if t is None:
            return None
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a tensor")
        if t.dtype is not dtype or t.shape != shape or t.get_device() != self._index or not t.is_contiguous():
            raise ValueError(f"{name}: expected contiguous {dtype} {shape} on {self.device}, got {t.dtype} "
                             f"{tuple(t.shape)} on {t.device} (contiguous={t.is_contiguous()})")
        return t.data_ptr()

    def _lengths(self, t, name):
        if t is None:
            raise TypeError(f"{name} must be a tensor")
        return self._dense(t, I32, self._per_seq, name)

    def _rows(self, slot, t, shape, name):
        """Address of the h2o_rows of a bf16 tensor [B, heads, n, d] whose rows are contiguous."""
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a tensor")
        if t.dtype is not BF16 or t.shape != shape or t.get_device() != self._index:
            raise ValueError(f"{name}: expected torch.bfloat16 {shape} on {self.device}, got {t.dtype} "
                             f"{tuple(t.shape)} on {t.device}")
        sb, sh, st, one = t.stride()
        p = t.data_ptr()
        if one != 1 or (sb | sh | st) & 7 or p & 15:
            # a dimension of size 1 is never stepped over: its stride may be anything
            sb, sh, st = (s if n > 1 else 0 for s, n in zip((sb, sh, st), shape))
            if one != 1 or (sb | sh | st) & 7 or p & 15:
                raise ValueError(f"{name}: rows must be contiguous and start at 16-byte boundaries, got strides "
                                 f"{t.stride()} at address {p:#x}")
        PACK(self._slots[slot], 0, p, sb, sh, st)
        return self._slot_at[slot]

    @staticmethod
    def _tokens(t, name):
        if not isinstance(t, torch.Tensor) or t.dim() != 4:
            raise ValueError(f"{name}: expected a [B, heads, n, d] tensor")
        return t.shape[2]

    def _shape(self, heads, n):
        return (self.B, heads, n, self.d)

    # ---------------------------------------------------------------- calls
    def append(self, k, v, lengths, counts=None, position=None, score=None, rotary=None):
        """Quantise rows k, v [B, H, n, d] (bf16) into entries ``lengths[b]``
        .. of each sequence, with positions from ``position`` (int32 [B],
        default ``lengths``) and scores ``score`` (fp32 [B, H, n], for example
        a prompt's column sums; default 0).  With an H2ORotary ``rotary`` the
        keys are normed and rotated by those positions first.  See
        h2o_bcache_append."""
        n = self._tokens(k, "k")
        shape = self._shape(self.H, n)
        if rotary is not None:
            k = self._turned(rotary, None, k, lengths, counts, position)[1]
        with self._lock:
            args = (self._rows(1, k, shape, "k"), self._rows(2, v, shape, "v"), self._lengths(lengths, "lengths"),
                    self._dense(counts, I32, self._per_seq, "counts"),
                    self._dense(position, I32, self._per_seq, "position"),
                    self._dense(score, F32, shape[:3], "score"))
            self._use_stream()
            _check(self._lib.h2o_bcache_append(self._h, n, *args), "h2o_bcache_append")

    def attend(self, q, lengths, counts=None, causal=True, accumulate=True, out=None, lse=None):
        """Attention of q [B, H * group, n, d] over the ``lengths[b]`` entries
        each sequence holds; returns out (shaped like q).  ``causal``: the last
        entries are the queries' own tokens; ``accumulate``: the weights are
        added to the entries' scores; ``lse`` (fp32 [B, H * group, n]) receives
        the log-sum-exps.  Rows of a sequence whose length or count is out of
        range are not written (error_bits).  See h2o_bcache_attend."""
        n = self._tokens(q, "q")
        shape = self._shape(self._heads, n)
        with self._lock:
            qr, lens = self._rows(0, q, shape, "q"), self._lengths(lengths, "lengths")
            cnt = self._dense(counts, I32, self._per_seq, "counts")
            if out is None:
                out = self._new_out(shape, counts)
            args = (qr, lens, cnt, 1 if causal else 0, 1 if accumulate else 0, self._rows(3, out, shape, "out"),
                    self._dense(lse, F32, shape[:3], "lse"))
            self._use_stream()
            _check(self._lib.h2o_bcache_attend(self._h, n, *args), "h2o_bcache_attend")
        return out

    def step(self, q, k, v, lengths, counts=None, position=None, accumulate=True, out=None, lse=None, rotary=None):
        """Append k, v [B, H, n, d] behind ``lengths[b]`` entries, then attend
        causally with q [B, H * group, n, d]; returns out.  The caller adds the
        counts (or n) to ``lengths`` afterwards, and to ``position``, which is
        needed from the first eviction on (the default are the lengths).  With
        an H2ORotary ``rotary``, q and k are normed and rotated by those
        positions first (q and k themselves stay as they are).  See
        h2o_bcache_step."""
        n = self._tokens(q, "q")
        shape, kv_shape = self._shape(self._heads, n), self._shape(self.H, n)
        if rotary is not None:
            q, k = self._turned(rotary, q, k, lengths, counts, position)
        with self._lock:
            rows = (self._rows(0, q, shape, "q"), self._rows(1, k, kv_shape, "k"), self._rows(2, v, kv_shape, "v"))
            lens, cnt = self._lengths(lengths, "lengths"), self._dense(counts, I32, self._per_seq, "counts")
            if out is None:
                out = self._new_out(shape, counts)
            args = rows + (lens, cnt, self._dense(position, I32, self._per_seq, "position"), 1 if accumulate else 0,
                           self._rows(3, out, shape, "out"), self._dense(lse, F32, shape[:3], "lse"))
            self._use_stream()
            _check(self._lib.h2o_bcache_step(self._h, n, *args), "h2o_bcache_step")
        return out

    def attend_sparse(self, q, lengths, n_blocks: int, n_first: int = 1, n_last: int = 2, counts=None, causal=True,
                      accumulate=True, out=None, lse=None, blocks=None):
        """``attend`` over ``n_blocks`` blocks of 32 entries for each query
        token and cached head: the first ``n_first``, the last ``n_last`` and
        those with the highest bound on the group's logits between them (all,
        where there are no more).  ``blocks`` (int32 [B, H, n, n_blocks])
        receives their indices, -1 behind them.  Needs a cache with ``bounds``.
        See h2o_bcache_attend_sparse."""
        n = self._tokens(q, "q")
        shape, choice = self._shape(self._heads, n), self._choice(n_blocks, n_first, n_last)
        if blocks is None:
            choice, blocks = self._new_blocks(n, *choice)
        with self._lock:
            qr, lens = self._rows(0, q, shape, "q"), self._lengths(lengths, "lengths")
            cnt = self._dense(counts, I32, self._per_seq, "counts")
            if out is None:
                out = self._new_out(shape, counts)
            args = (qr, lens, cnt, 1 if causal else 0, 1 if accumulate else 0, *choice, self._rows(3, out, shape, "out"),
                    self._dense(lse, F32, shape[:3], "lse"), self._blocks(blocks, n, choice[0]))
            self._use_stream()
            _check(self._lib.h2o_bcache_attend_sparse(self._h, n, *args), "h2o_bcache_attend_sparse")
        return out

    def step_sparse(self, q, k, v, lengths, n_blocks: int, n_first: int = 1, n_last: int = 2, counts=None, position=None,
                    accumulate=True, out=None, lse=None, blocks=None, rotary=None):
        """``step`` whose queries attend to ``n_blocks`` chosen blocks each
        (``attend_sparse``).  See h2o_bcache_step_sparse."""
        n = self._tokens(q, "q")
        shape, kv_shape = self._shape(self._heads, n), self._shape(self.H, n)
        if rotary is not None:
            q, k = self._turned(rotary, q, k, lengths, counts, position)
        choice = self._choice(n_blocks, n_first, n_last)
        if blocks is None:
            choice, blocks = self._new_blocks(n, *choice)
        with self._lock:
            rows = (self._rows(0, q, shape, "q"), self._rows(1, k, kv_shape, "k"), self._rows(2, v, kv_shape, "v"))
            lens, cnt = self._lengths(lengths, "lengths"), self._dense(counts, I32, self._per_seq, "counts")
            if out is None:
                out = self._new_out(shape, counts)
            args = rows + (lens, cnt, self._dense(position, I32, self._per_seq, "position"), 1 if accumulate else 0,
                           *choice, self._rows(3, out, shape, "out"), self._dense(lse, F32, shape[:3], "lse"),
                           self._blocks(blocks, n, choice[0]))
            self._use_stream()
            _check(self._lib.h2o_bcache_step_sparse(self._h, n, *args), "h2o_bcache_step_sparse")
        return out

    def bound(self, lengths):
        """Make ``bounds`` anew for ``lengths`` entries a sequence: after K or
        K_scale have been written other than by this object's calls."""
        lens = self._lengths(lengths, "lengths")
        with self._lock:
            self._use_stream()
            _check(self._lib.h2o_bcache_bound(self._h, lens), "h2o_bcache_bound")

    @staticmethod
    def _choice(n_blocks, n_first, n_last):
        if type(n_blocks) is type(n_first) is type(n_last) is int and 0 <= n_first <= n_blocks < 1 << 31 > n_last >= 0:
            return n_blocks, n_first, n_last
        return _whole(n_blocks, "n_blocks"), _whole(n_first, "n_first"), _whole(n_last, "n_last")

    def _new_blocks(self, n, n_blocks, n_first, n_last):
        """A choice as the call makes it, and room for its list of blocks, which the kernels hand on through memory.  The
        caller holds that until its call is enqueued: only work enqueued behind it may be given the memory anew."""
        if not (n_first >= 0 and 1 <= n_last and n_first + n_last <= n_blocks <= self._most_blocks):
            return (n_blocks, n_first, n_last), None  # the library refuses it
        most = self.capacity // self.BLOCK
        if n_blocks > most:  # every block, however they are named: no list longer than that
            n_blocks, n_first, n_last = most, 0, 1
        return (n_blocks, n_first, n_last), torch.empty((self.B, self.H, n, n_blocks), dtype=I32, device=self.device)

    def _blocks(self, t, n, n_blocks):
        return self._dense(t, I32, (self.B, self.H, n, n_blocks), "blocks")

    def _turned(self, rotary, q, k, lengths, counts, position):
        """q and k normed and rotated by their positions, in rows of their own (those behind a count hold anything: no
        call reads them)."""
        outs = [None if t is None else torch.empty(t.shape, dtype=t.dtype, device=self.device) for t in (q, k)]
        return rotary.apply(q, k, lengths if position is None else position, counts, *outs)

    def _new_out(self, shape, counts):
        # rows behind a sequence's count are not written
        make = torch.empty if counts is None else torch.zeros
        return make(shape, dtype=torch.bfloat16, device=self.device)

    def evict(self, lengths, k_heavy: int, k_local: int, n_sink: int = 0, score_mode: int = 0, position=None,
              new_lengths=None):
        """Cut every sequence down to ``k_heavy + k_local`` entries: its last
        ``k_local`` and the ``k_heavy`` others that rank highest (by score, or
        with ``score_mode`` 1 by score / (position - pos)); entries at positions
        below ``n_sink`` rank first.  Returns the new lengths (int32 [B]).  See
        h2o_bcache_evict."""
        lens = self._lengths(lengths, "lengths")
        if new_lengths is None:
            new_lengths = torch.empty_like(lengths)
        args = (lens, _whole(k_heavy, "k_heavy"), _whole(k_local, "k_local"), _whole(n_sink, "n_sink"),
                _whole(score_mode, "score_mode"),
                self._dense(position, I32, self._per_seq, "position"), self._lengths(new_lengths, "new_lengths"))
        with self._lock:
            self._use_stream()
            _check(self._lib.h2o_bcache_evict(self._h, *args), "h2o_bcache_evict")
        return new_lengths

    def copy(self, parent, lengths, source=None, source_lengths=None, new_lengths=None):
        """Row b receives the sequence of row ``parent[b]`` (int32 [B]; -1: it
        stays), in place with any map, or out of the H2OBlockCache ``source``
        that holds ``source_lengths``: beams reordered, prompts forked,
        sequences moved up or taken into a running batch.  Returns the new
        lengths (int32 [B]); what else the caller keeps for a row (positions)
        is the caller's to reorder.  See h2o_bcache_copy."""
        par, lens = self._dense(parent, I32, self._per_seq, "parent"), self._lengths(lengths, "lengths")
        if par is None:
            raise TypeError("parent must be a tensor")
        if source is self:
            source = None
        if source is None:
            if source_lengths is not None:
                raise ValueError("source_lengths belong to another cache: pass it as source")
            other, src = None, None
        else:
            if not isinstance(source, H2OBlockCache):
                raise TypeError("source must be an H2OBlockCache")
            other, src = source._h, source._lengths(source_lengths, "source_lengths")
        if new_lengths is None:
            new_lengths = torch.empty_like(lengths)
        args = (other, par, src, lens, self._lengths(new_lengths, "new_lengths"))
        with self._lock:
            self._use_stream()
            if source is not None:
                source._record(self._set_stream)
            _check(self._lib.h2o_bcache_copy(self._h, *args), "h2o_bcache_copy")
        return new_lengths

    def error_bits(self) -> int:
        """The sticky error flag (H2O_BERR_* bits; 0 = none); synchronises."""
        bits = C.c_int32()
        with self._lock:
            self._use_stream()
            rc = self._lib.h2o_bcache_get_error(self._h, C.byref(bits))
        if rc not in (0, 5):
            _check(rc, "h2o_bcache_get_error")
        return bits.value

    def check_device_error(self):
        bits = self.error_bits()
        if bits:
            raise H2OError(5, f"h2o_bcache_get_error (bits {bits})")
