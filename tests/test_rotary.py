"""csa_rotary / csa_rotary_frequencies: what the host refuses and computes (no GPU needed)."""
import ctypes
import math

import numpy as np
import pytest
import torch

import fp4_kv_cache_csa_b200 as csa
from fp4_kv_cache_csa_b200 import build as csa_build

OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_UNSUPPORTED, ERR_CUDA = 0, 1, 2, 3, 4, 6


@pytest.fixture(scope="module")
def lib():
    csa_build.build()
    return csa.load_library()


def call(lib, rows=4, heads=2, dim=64, x=(0x10000, 0, 128, 64), out=(0x20000, 0, 128, 64), freq=0x30000, begin=0,
         rot=64, layout=0, pos=0x40000, inverse=0):
    # host addresses that are never dereferenced: every call here fails its checks or has no rows
    cx = csa._CVectors(*x) if x is not None else None
    co = csa._CVectors(*out) if out is not None else None
    rope = csa._CRope(freq, begin, rot, layout, 1.0)
    return lib.csa_rotary(ctypes.byref(cx) if cx is not None else None, ctypes.byref(co) if co is not None else None,
                          rows, heads, dim, ctypes.byref(rope), pos, inverse, None)


def test_refusals(lib):
    assert call(lib, x=None) == ERR_NULL
    assert call(lib, out=None) == ERR_NULL
    assert call(lib, x=(None, 0, 128, 64)) == ERR_NULL
    assert call(lib, freq=None) == ERR_NULL
    assert call(lib, pos=None) == ERR_NULL
    assert call(lib, rows=-1) == ERR_SHAPE
    assert call(lib, heads=0) == ERR_SHAPE
    assert call(lib, dim=1, rot=2) == ERR_SHAPE
    assert call(lib, rot=0) == ERR_SHAPE
    assert call(lib, rot=31) == ERR_SHAPE
    assert call(lib, rot=66) == ERR_SHAPE
    assert call(lib, begin=2) == ERR_SHAPE
    assert call(lib, begin=-2, rot=32) == ERR_SHAPE
    assert call(lib, begin=2**31 - 1, rot=32) == ERR_SHAPE
    assert call(lib, layout=2) == ERR_SHAPE
    assert call(lib, x=(0x10000, 2, 128, 64)) == ERR_SHAPE
    assert call(lib, out=(0x20000, -1, 128, 64)) == ERR_SHAPE
    assert call(lib, x=(0x10001, 0, 128, 64)) == ERR_ALIGN
    assert call(lib, out=(0x20002, 1, 128, 64)) == ERR_ALIGN
    assert call(lib, freq=0x30002) == ERR_ALIGN
    assert call(lib, pos=0x40002) == ERR_ALIGN
    assert call(lib, dim=8194, rot=8194) == ERR_UNSUPPORTED
    assert call(lib, x=(0x10000, 0, -128, 64)) == ERR_SHAPE
    assert call(lib, x=(0x10000, 0, 1 << 62, 64)) == ERR_SHAPE


def test_overlaps(lib):
    # outputs that overlap one another, and outputs that run into the input
    assert call(lib, out=(0x20000, 0, 64, 64)) == ERR_SHAPE           # row 1 is head 1 of row 0
    assert call(lib, out=(0x20000, 0, 0, 64)) == ERR_SHAPE
    assert call(lib, out=(0x20000, 0, 128, 32)) == ERR_SHAPE
    assert call(lib, out=(0x10000 + 8, 0, 128, 64)) == ERR_SHAPE      # x shifted by four channels
    assert call(lib, out=(0x10000 + 128, 0, 128, 64)) == ERR_SHAPE    # head 0 of out is head 1 of x
    assert call(lib, out=(0x10000, 1, 128, 64)) == ERR_SHAPE          # in place in another type
    assert call(lib, x=(0x10000, 0, 0, 64), out=(0x10000, 0, 128, 64)) == ERR_SHAPE
    assert call(lib, x=(0x10000, 0, 64, 256), out=(0x10000 + 2, 0, 64, 256), heads=2) == ERR_SHAPE
    if torch.cuda.is_available():
        return  # the calls below would launch on these addresses
    # passing calls end at the launch on a machine without a GPU
    assert call(lib) == ERR_CUDA
    assert call(lib, out=(0x10000, 0, 128, 64)) == ERR_CUDA                                  # in place
    assert call(lib, x=(0x10000, 0, 256, 128), out=(0x10000 + 128, 0, 256, 128)) == ERR_CUDA  # other channels of the rows
    assert call(lib, out=(0x20000, 0, 64, 256)) == ERR_CUDA                                  # head-major
    assert call(lib, x=(0x10000, 0, 0, 0)) == ERR_CUDA                                       # broadcast
    assert call(lib, rows=1, out=(0x20000, 0, 0, 64)) == ERR_CUDA                            # stride of one row unused


def test_no_rows_is_no_work(lib):
    assert call(lib, rows=0, x=(None, 0, 128, 64), out=(None, 0, 128, 64), freq=None, pos=None) == OK


def test_binding_refusals(lib):
    x = torch.zeros(3, 2, 8)
    pos, inv = torch.zeros(3, dtype=torch.int32), torch.ones(4)
    with pytest.raises(csa.CsaError, match="float16"):
        csa.csa_rotary(x.half(), pos, inv)
    with pytest.raises(csa.CsaError, match="adjacent"):
        csa.csa_rotary(x.transpose(1, 2), pos, inv)
    with pytest.raises(csa.CsaError, match="pos"):
        csa.csa_rotary(x, pos.long(), inv)
    with pytest.raises(csa.CsaError, match="pos"):
        csa.csa_rotary(x, pos[:2], inv)
    with pytest.raises(csa.CsaError, match="inv_freq"):
        csa.csa_rotary(x, pos, inv.double())
    with pytest.raises(csa.CsaError, match="out"):
        csa.csa_rotary(x, pos, inv, out=x[:2])
    with pytest.raises(csa.CsaError, match="out"):
        csa.csa_rotary(x, pos, inv, out=x, out_dtype=torch.bfloat16)
    with pytest.raises(csa.CsaError, match="CUDA device"):
        csa.csa_rotary(x, pos, inv)


@pytest.mark.parametrize("rot", [2, 4, 64, 128])
def test_frequencies(lib, rot):
    p = np.arange(rot // 2)
    plain = 10000.0 ** (-2.0 * p / rot)

    def got(**kw):
        inv, m = csa.csa_rotary_frequencies(rot, **kw)
        return inv.numpy(), m

    # float32 rounding of a float64 power: half a step, and one step where the powers themselves differ in their last bit
    def close(a, b):
        return np.all(np.abs(a.astype(np.float64) - b) <= np.finfo(np.float32).eps * b)

    inv, m = got()
    assert close(inv, plain) and m == 1.0
    inv, m = got(scaling=csa.CSA_ROPE_SCALE_LINEAR, factor=4.0)
    assert close(inv, plain / 4) and m == 1.0
    if rot > 2:
        inv, m = got(scaling=csa.CSA_ROPE_SCALE_BASE, factor=8.0)
        assert close(inv, (10000.0 * 8.0 ** (rot / (rot - 2))) ** (-2.0 * p / rot)) and m == 1.0
    inv, m = got(scaling=csa.CSA_ROPE_SCALE_PARTS, factor=40.0, original_len=4096)
    turns = 4096 * plain / (2 * math.pi)
    assert abs(m - (0.1 * math.log(40.0) + 1)) < 1e-6
    assert inv[0] == 1.0                                              # the fastest pair turns 652 times: kept
    assert close(inv[turns < 0.5], plain[turns < 0.5] / 40)  # half a turn: at least a whole pair behind beta_slow
    assert np.all(inv <= plain * (1 + 1e-6)) and np.all(inv >= plain / 40 * (1 - 1e-6))
    assert np.all(np.diff(inv) < 0)
    if rot == 128:  # the ramp by hand: pairs 20 (32 turns: 20.95) to 46 (one turn: 45.03)
        ramp = np.clip((p - 20) / 26, 0, 1)
        assert close(inv, plain / 40 * ramp + plain * (1 - ramp))


def test_frequency_refusals(lib):
    out = (ctypes.c_float * 64)()

    def f(rot=128, base=1e4, scaling=0, factor=1.0, length=4096, fast=32.0, slow=1.0, to=out):
        return lib.csa_rotary_frequencies(rot, base, scaling, factor, length, fast, slow, to, None)

    assert f() == OK
    assert f(to=None) == ERR_NULL
    for bad in (dict(rot=0), dict(rot=3), dict(rot=8194), dict(base=1.0), dict(base=math.nan), dict(base=math.inf),
                dict(scaling=4), dict(scaling=-1), dict(scaling=1, factor=0.5), dict(scaling=1, factor=math.nan),
                dict(scaling=2, factor=2.0, rot=2), dict(scaling=3, factor=2.0, length=0),
                dict(scaling=3, factor=2.0, slow=0.0), dict(scaling=3, factor=2.0, fast=0.5)):
        assert f(**bad) == ERR_SHAPE, bad
