"""csa_cache_copy: what the host refuses, and the test model itself (no GPU needed)."""
import ctypes

import numpy as np
import pytest
import torch

import fp4_kv_cache_csa_b200 as csa
from fp4_kv_cache_csa_b200 import build as csa_build
from copy_model import copy_slots

OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_CUDA = range(7)


@pytest.fixture(scope="module")
def lib():
    csa_build.build()
    return csa.load_library()


def fake(at=0x10000000, **kw):
    # host addresses, a gigabyte apart per cache, that are never dereferenced
    d = dict(batch=2, dim=512, block=4, capacity=1024, fp4=at, scale=at + 0x8000000, idx_key=at + 0x10000000,
             idx_dim=128, idx_dtype=1, n_blocks=at + 0x20000000, status=None, scale_fmt=0, idx_key_scale=None)
    d.update(kw)
    return csa._CCache(*(d[f[0]] for f in csa._CCache._fields_))


def call(lib, src=None, dst=None, n=2, s=0x1000, d=0x2000, keep=None, cols=0, lim=None, ws=0x100, wsb=1 << 40):
    src = fake() if src is None else src
    dst = fake(0x50000000) if dst is None else dst
    return lib.csa_cache_copy(ctypes.byref(src), ctypes.byref(dst), n, s, d, keep, cols, lim, ws, wsb, None)


def test_refusals(lib):
    assert lib.csa_cache_copy(None, ctypes.byref(fake()), 1, 4, 4, None, 0, None, 256, 1 << 20, None) == ERR_NULL
    assert lib.csa_cache_copy(ctypes.byref(fake()), None, 1, 4, 4, None, 0, None, 256, 1 << 20, None) == ERR_NULL
    assert call(lib, n=-1) == ERR_SHAPE
    assert call(lib, cols=5) == ERR_SHAPE
    assert call(lib, keep=0x3000) == ERR_SHAPE
    assert call(lib, keep=0x3000, cols=-1) == ERR_SHAPE
    for kw in (dict(dim=128), dict(block=8), dict(scale_fmt=1), dict(idx_key=None), dict(idx_dim=64), dict(idx_dtype=0)):
        assert call(lib, dst=fake(0x50000000, **kw)) == ERR_SHAPE, kw
    assert call(lib, n=65536) == ERR_UNSUPPORTED
    assert call(lib, keep=0x3000, cols=(1 << 19) + 1) == ERR_UNSUPPORTED
    assert call(lib, src=fake(dim=544), dst=fake(0x50000000, dim=544)) == ERR_UNSUPPORTED
    assert call(lib, s=None) == ERR_NULL
    assert call(lib, d=None) == ERR_NULL
    assert call(lib, s=0x1002) == ERR_ALIGN
    assert call(lib, d=0x2002) == ERR_ALIGN
    assert call(lib, keep=0x3002, cols=4) == ERR_ALIGN
    assert call(lib, lim=0x3002) == ERR_ALIGN
    assert call(lib, ws=None) == ERR_WORKSPACE
    assert call(lib, wsb=lib.csa_cache_copy_workspace(ctypes.byref(fake()), 2, 0) - 1) == ERR_WORKSPACE
    assert call(lib, ws=0x180) == ERR_ALIGN
    assert call(lib, n=0, s=None, d=None, ws=None, wsb=0) == OK


def test_caches_that_share_memory(lib):
    assert call(lib, dst=fake(0x50000000, fp4=0x10000000 + 1024)) == ERR_SHAPE
    assert call(lib, dst=fake(0x50000000, n_blocks=0x30000004)) == ERR_SHAPE
    assert call(lib, dst=fake(capacity=512)) == ERR_SHAPE        # one memory read with two capacities
    assert call(lib, dst=fake(scale=0x70000000)) == ERR_SHAPE
    if not torch.cuda.is_available():  # passing calls end at the device query on a machine without a GPU
        assert call(lib) == ERR_CUDA
        assert call(lib, dst=fake()) == ERR_CUDA
        assert call(lib, dst=fake(0x50000000, capacity=7, batch=9), keep=0x3000, cols=4, lim=0x4000) == ERR_CUDA


def test_workspace_sizes(lib):
    def ws(n, cols, **kw):
        return lib.csa_cache_copy_workspace(ctypes.byref(fake(**kw)), n, cols)

    assert ws(-1, 0) == 0 and ws(1, -1) == 0 and ws(65536, 0) == 0 and ws(1, (1 << 19) + 1) == 0
    assert ws(0, 0) > 0
    assert ws(32, 131072) >= 32 * 4 * (131072 // 64)     # a flag per tile of a list
    assert ws(1, 0, batch=100000) >= 12 * 100000         # the slot tables of a large batch


def test_binding_refusals(lib):
    c = csa.Cache.allocate(2, 8, 128, 4, device="cpu")
    s = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(csa.CsaError, match="src_slot"):
        csa.csa_cache_copy(c, c, s.long(), s)
    with pytest.raises(csa.CsaError, match="dst_slot"):
        csa.csa_cache_copy(c, c, s, s[:1])
    with pytest.raises(csa.CsaError, match="keep"):
        csa.csa_cache_copy(c, c, s, s, keep=s)
    with pytest.raises(csa.CsaError, match="keep"):
        csa.csa_cache_copy(c, c, s, s, keep=torch.zeros(2, 0, dtype=torch.int32))
    with pytest.raises(csa.CsaError, match="max_blocks"):
        csa.csa_cache_copy(c, c, s, s, max_blocks=s[:1])
    with pytest.raises(csa.CsaError, match="CUDA device"):
        csa.csa_cache_copy(c, c, s, s)


def test_model_by_hand():
    a = np.arange(12, dtype=np.uint8).reshape(2, 3, 2)
    out, n, st = copy_slots([a], [3, 2], [a], [3, 2], [0], [1], same=True)
    assert st == 0 and list(n) == [3, 3] and (out[0][1] == a[0]).all()
    out, n, st = copy_slots([a], [3, 2], [a], [3, 2], [0], [0], keep=[[0, 2, -1]], same=True)
    assert st == 0 and list(n) == [2, 2] and (out[0][0] == a[0][[0, 2, 2]]).all()
    out, n, st = copy_slots([a], [3, 2], [a], [3, 2], [0, 1], [1, 0], same=True)   # a swap reads what it writes
    assert st == 4 and list(n) == [3, 2]
    out, n, st = copy_slots([a], [3, 2], [a], [3, 2], [-1, 0, 0], [1, 1, 5], max_blocks=[9, 1, 1], same=True)
    assert st == 4 and list(n) == [3, 0]
