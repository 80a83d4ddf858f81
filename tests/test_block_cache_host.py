"""Refusals of the block-cache C ABI that reach no device (CPU)."""
from __future__ import annotations

import ctypes as C
import subprocess
import sys

import pytest

import h2o_heavy_hitter_decode_gb300 as h2o
from h2o_heavy_hitter_decode_gb300 import build as hbuild

GOOD = (2, 3, 64, 64, 2, 4, 0)


@pytest.fixture(scope="module")
def L():
    hbuild.build()
    return h2o.lib()


BAD = [(0, 3, 64, 64, 2, 4, 0), (2, 0, 64, 64, 2, 4, 0), (2, 3, 0, 64, 2, 4, 0), (2, 3, 64, 0, 2, 4, 0),
       (2, 3, 64, 63, 2, 4, 0), (2, 3, 64, 2 ** 40, 2, 4, 0), (1, 1, 64, 2 ** 30 + 32, 1, 1, 0), (2, 3, 64, 64, 0, 4, 0), (2, 3, 64, 64, 2, 0, 0),
       (2, 3, 64, 64, 32, 9, 0), (2, 3, 64, 64, 257, 1, 0), (2, 3, 64, 64, 2, 4, 2), (2, 3, 64, 64, 2, 4, -1),
       (1 << 13, 1 << 12, 64, 64, 1, 1, 0), (1 << 12, 1 << 12, 64, 128, 1, 1, 0)]


@pytest.mark.parametrize("shape", BAD, ids=str)
def test_bad_shapes(L, shape):
    h = C.c_void_p()
    assert L.h2o_bcache_workspace_bytes(*shape) == 0
    assert L.h2o_bcache_create(*shape, C.c_void_p(256), None, C.byref(h)) == 1
    assert not h.value


def test_unsupported_head_size(L):
    h = C.c_void_p()
    shape = (2, 3, 96, 64, 2, 4, 0)
    assert L.h2o_bcache_workspace_bytes(*shape) == 0
    assert L.h2o_bcache_create(*shape, C.c_void_p(256), None, C.byref(h)) == 6


def test_workspace_pointer(L):
    h = C.c_void_p()
    assert L.h2o_bcache_create(*GOOD, None, None, C.byref(h)) == 1
    assert L.h2o_bcache_create(*GOOD, C.c_void_p(128), None, C.byref(h)) == 1
    assert L.h2o_bcache_create(*GOOD, C.c_void_p(256), None, None) == 1


def test_null_handle(L):
    r = C.byref(h2o.Rows(256, 64, 64, 64))
    p = C.c_void_p(256)
    assert L.h2o_bcache_append(None, 1, r, r, p, None, None, None) == 1
    assert L.h2o_bcache_attend(None, 1, r, p, None, 1, 1, r, None) == 1
    assert L.h2o_bcache_step(None, 1, r, r, r, p, None, None, 1, r, None) == 1
    assert L.h2o_bcache_evict(None, p, 1, 1, 0, 0, None, C.c_void_p(512)) == 1
    assert L.h2o_bcache_arrays(None, None, None, None, None, None, None) == 1
    assert L.h2o_bcache_set_stream(None, None) == 1
    assert L.h2o_bcache_get_error(None, None) == 1
    assert L.h2o_bcache_destroy(None) == 0


def test_binding_refuses_before_the_device():
    with pytest.raises(ValueError):
        h2o.H2OBlockCache(1, 1, 64, 32, kv="fp4", device="cuda:0")
    with pytest.raises(ValueError):
        h2o.H2OBlockCache(1, 1, 64, 32, device="cpu")


def test_import_with_a_torch_without_cuda():
    """The package, its header's functions and its refusals are there on a host whose torch has no CUDA functions."""
    code = ("import torch\n"
            "for n in [n for n in dir(torch._C) if n.startswith('_cuda_getCurrent')]: delattr(torch._C, n)\n"
            "import h2o_heavy_hitter_decode_gb300 as h2o\n"
            "assert 'h2o_bcache_step' in h2o.declared_functions()\n")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300, cwd=hbuild.ROOT)
    assert r.returncode == 0, r.stderr
