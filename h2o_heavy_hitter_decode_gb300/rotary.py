"""Norm and rotation of queries and keys (``h2o_rotate`` of the C ABI):
argument checks and marshalling only."""
from __future__ import annotations

import ctypes as C
import math
import struct
import threading
from fractions import Fraction

import torch

from . import H2O_BF16, H2O_F32, _check, lib

__all__ = ["H2ORotary"]

BF16, I32 = torch.bfloat16, torch.int32
TYPES = {BF16: H2O_BF16, torch.float32: H2O_F32}
PACK = struct.Struct("4q").pack_into  # an h2o_rows
# 2 pi to 50 digits: a frequency's fraction of a turn is taken to 64 bits
TWO_PI = Fraction("6.2831853071795864769252867665590057683943387987502")


class _Rotary(C.Structure):
    """h2o_rotary"""
    _fields_ = [("d", C.c_int), ("pairs", C.c_int), ("interleaved", C.c_int), ("axes", C.c_int), ("norm", C.c_int),
                ("eps", C.c_float), ("turns", C.c_void_p), ("axis", C.c_void_p), ("q_weight", C.c_void_p),
                ("k_weight", C.c_void_p)]


class H2ORotary:
    """What a model's layers do to queries and keys before they meet a cache:
    an RMS norm of each head where ``eps`` is given (times ``q_weight`` and
    ``k_weight`` [d], default ones), then the rotation of the first ``dims``
    dimensions (a multiple of 16; default all ``d``) by the token's position.

    Pair i of them (i and i + dims / 2, or 2 i and 2 i + 1 with
    ``interleaved``) turns by position * ``frequency[i]`` radians; default
    frequencies are theta ** (-2 i / dims).  Other tables (scaled, or per axis)
    are passed as ``frequency`` [dims / 2]; they are taken as 64-bit fractions
    of a turn, so far positions lose nothing.  ``axis`` [dims / 2] says which
    of several axes (time, height, width) a pair's position is on.  ``dims=0``
    norms only.

    The object owns small tables on its device and nothing else: layers that
    agree in them share it, on any streams and host threads.  The weights are
    copied into them, as fp32: a weight that is changed afterwards takes a new
    object.  One that a captured graph uses is kept for as long as the graph is
    replayed."""

    def __init__(self, d: int, dims: int | None = None, theta: float = 10000.0, frequency=None, axis=None,
                 interleaved: bool = False, eps: float | None = None, q_weight=None, k_weight=None, device=None):
        self._lib = lib()
        if d not in (64, 128):
            raise ValueError(f"d must be 64 or 128, got {d}")
        if frequency is not None:
            frequency = [float(f) for f in (frequency.tolist() if isinstance(frequency, torch.Tensor) else frequency)]
            if dims is not None and dims != 2 * len(frequency):
                raise ValueError(f"{len(frequency)} frequencies for {dims} dimensions")
            dims = 2 * len(frequency)
        dims = d if dims is None else int(dims)
        if dims < 0 or dims > d or dims % 16:
            raise ValueError(f"rotated dimensions: a multiple of 16 up to {d}, got {dims}")
        pairs = dims // 2
        if frequency is None:
            if not (theta > 0 and math.isfinite(theta)):
                raise ValueError(f"theta must be a positive number, got {theta}")
            frequency = [theta ** (-i / pairs) for i in range(pairs)]
        if not all(math.isfinite(f) for f in frequency):
            raise ValueError("frequencies must be finite")
        axis = [0] * pairs if axis is None else [int(a) for a in (axis.tolist() if isinstance(axis, torch.Tensor) else axis)]
        if len(axis) != pairs or any(not 0 <= a < 256 for a in axis):
            raise ValueError(f"axis: expected {pairs} numbers from 0 to 255, got {axis}")
        if eps is None:
            if q_weight is not None or k_weight is not None:
                raise ValueError("weights belong to a norm: pass its eps")
        elif not (eps >= 0 and math.isfinite(eps)):
            raise ValueError(f"eps must be a number of at least 0, got {eps}")
        self.d, self.dims, self.interleaved, self.eps = d, dims, bool(interleaved), eps
        self.axes = max(axis, default=0) + 1
        self.device = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
        if self.device.type != "cuda":
            raise ValueError("H2ORotary lives on a CUDA device")
        if self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self._index = self.device.index
        # torch.cuda.current_stream(device).cuda_stream and current_device() without their objects and checks
        self._raw_stream, self._current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
        turns = [round(Fraction(f) / TWO_PI * 2 ** 64) % 2 ** 64 for f in frequency]
        turns = [t - 2 ** 64 if t >= 2 ** 63 else t for t in turns]  # the same bits in an int64

        def weight(w, name):
            if w is None:
                return None
            if not isinstance(w, torch.Tensor) or w.shape != (d,):
                raise ValueError(f"{name}: expected a [{d}] tensor")
            return w.detach().to(device=self.device, dtype=torch.float32, copy=True).contiguous()

        self._turns = torch.tensor(turns, dtype=torch.int64, device=self.device)
        self._axis = torch.tensor(axis, dtype=torch.uint8, device=self.device)
        self._weights = weight(q_weight, "q_weight"), weight(k_weight, "k_weight")
        self._tables = [t for t in (self._turns, self._axis, *self._weights) if t is not None]
        at = [t.data_ptr() if t is not None and t.numel() else None for t in (self._turns, self._axis, *self._weights)]
        torch.cuda.current_stream(self.device).synchronize()  # the tables are there for every stream
        self._known = {self._raw_stream(self._index)}  # streams that the tables' allocations know of
        self._lock = threading.Lock()
        self._slots = (C.c_int64 * 16)()  # h2o_rows of q, k, q_out and k_out
        self._slots_at = C.addressof(self._slots)
        self._desc = _Rotary(d, pairs, int(self.interleaved), self.axes, int(eps is not None),
                             0.0 if eps is None else eps, *at)
        self._desc_at = C.addressof(self._desc)

    def _rows(self, slot, t, shape, dtype, name):
        """Address of the h2o_rows of a tensor of that shape and type whose rows are contiguous."""
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a tensor")
        if t.dtype is not dtype or t.shape != shape or t.get_device() != self._index:
            raise ValueError(f"{name}: expected {dtype} {tuple(shape)} on {self.device}, got {t.dtype} {tuple(t.shape)} "
                             f"on {t.device}")
        step = 7 if dtype is BF16 else 3
        sb, sh, st, one = t.stride()
        p = t.data_ptr()
        if one != 1 or (sb | sh | st) & step or p & 15:
            # a dimension of size 1 is never stepped over: its stride may be anything
            sb, sh, st = (s if n > 1 else 0 for s, n in zip((sb, sh, st), shape))
            if one != 1 or (sb | sh | st) & step or p & 15:
                raise ValueError(f"{name}: rows must be contiguous and start at 16-byte boundaries, got strides "
                                 f"{t.stride()} at address {p:#x}")
        PACK(self._slots, slot, p, sb, sh, st)
        return self._slots_at + slot

    def _ints(self, t, shape, name):
        if not isinstance(t, torch.Tensor) or t.dtype is not I32 or t.shape != shape or \
                t.get_device() != self._index or not t.is_contiguous():
            raise ValueError(f"{name}: expected contiguous {I32} {shape} on {self.device}")
        return t.data_ptr()

    def apply(self, q, k, position, counts=None, q_out=None, k_out=None):
        """Norm and rotate q [B, query heads, n, d] and k [B, key heads, n, d]
        (bf16 or fp32; either may be None) in one launch on the current stream;
        returns (q_out, k_out), which may be q and k themselves.

        ``position``: int32 [B], token t of sequence b being at position[b] + t
        on every axis, or int32 [axes, B, n].  ``counts`` (int32 [B]): rows
        behind a sequence's count are not read, and left as they were in the
        outputs.  See h2o_rotate."""
        ref = k if q is None else q
        if not isinstance(ref, torch.Tensor) or ref.dim() != 4:
            raise ValueError("q, k: expected [B, heads, n, d] tensors, one of them at least")
        B, _, n, d = ref.shape
        dtype = ref.dtype
        if d != self.d or dtype not in TYPES:
            raise ValueError(f"q, k: expected rows of {self.d} torch.bfloat16 or torch.float32, got {d} {dtype}")
        cnt = None if counts is None else self._ints(counts, (B,), "counts")
        if position is None and self.dims == 0:
            where, per_token = None, 0
        elif isinstance(position, torch.Tensor) and position.dim() == 3:
            where, per_token = self._ints(position, (max(self.axes, position.shape[0]), B, n), "position"), 1
        else:
            where, per_token = self._ints(position, (B,), "position"), 0
        with self._lock:  # its rows' descriptors
            hq = hk = 0
            qi = ki = qo = ko = None
            if q is not None:
                hq = ref.shape[1]
                shape = (B, hq, n, d)
                qi = self._rows(0, q, shape, dtype, "q")
                if q_out is None:
                    q_out = self._new(shape, dtype, counts)
                qo = self._rows(64, q_out, shape, dtype, "q_out")
            elif q_out is not None:
                raise ValueError("q_out without q")
            if k is not None:
                if not isinstance(k, torch.Tensor) or k.dim() != 4:
                    raise ValueError("k: expected a [B, heads, n, d] tensor")
                hk = k.shape[1]
                shape = (B, hk, n, d)
                ki = self._rows(32, k, shape, dtype, "k")
                if k_out is None:
                    k_out = self._new(shape, dtype, counts)
                ko = self._rows(96, k_out, shape, dtype, "k_out")
            elif k_out is not None:
                raise ValueError("k_out without k")
            stream = self._raw_stream(self._index)
            if stream not in self._known:
                # tables that are dropped while this stream still runs keep their memory until it is done
                for t in self._tables:
                    t.record_stream(torch.cuda.current_stream(self.device))
                self._known.add(stream)
            args = (self._desc_at, TYPES[dtype], B, n, hq, hk, qi, ki, where, per_token, cnt, qo, ko, stream)
            if self._current_device() == self._index:
                rc = self._lib.h2o_rotate(*args)
            else:
                with torch.cuda.device(self._index):
                    rc = self._lib.h2o_rotate(*args)
        if rc:
            _check(rc, "h2o_rotate")
        return q_out, k_out

    def _new(self, shape, dtype, counts):
        # rows behind a sequence's count are not written
        return (torch.empty if counts is None else torch.zeros)(shape, dtype=dtype, device=self.device)
