"""Failure detection without a GPU fault: bounded waits of csa_cache_copy and hca_shared_attend run out.

As in test_gpu_timeout.py, a variant of the library is built into the test's temporary directory, in which
one arrival that others wait for never happens (`-DCSA_TEST_LOST_ARRIVALS`) and the limit is about half a
millisecond: an in-place compaction's first tile never says that it has loaded, and one warp never says
that a group's queries are there. The calls flag CSA_DEV_TIMEOUT and return, and the shipped library then
works in the same context."""
import ctypes

import numpy as np
import pytest

from fp4_kv_cache_csa_b200 import datagen
from gpu_util import dev
from test_gpu_shared_attend import check, random_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def short(tmp_path_factory):
    import fp4_kv_cache_csa_b200 as csa
    from fp4_kv_cache_csa_b200 import build as csa_build

    at = tmp_path_factory.mktemp("lost")
    path = csa_build.build(force=True, defines=["CSA_WAIT_CYCLES=1000000", "CSA_TEST_LOST_ARRIVALS"],
                           lib_path=str(at / "libcsa_lost.so"), build_dir=str(at / "build"))
    return csa.declare(ctypes.CDLL(path))


def status_of(lib, cache, call):
    import fp4_kv_cache_csa_b200 as csa

    shipped = csa.load_library()
    csa._lib = lib
    try:
        call()
        return csa.csa_read_device_status(cache)
    finally:
        csa._lib = shipped


@pytest.mark.parametrize("D,fmt", [(512, 0), (512, 1), (128, 0)])
def test_shared_attend(short, D, fmt):
    import torch

    import fp4_kv_cache_csa_b200 as csa

    c = random_cache(2, 1500, D, fmt, n=[1500, 700])
    q = dev(datagen.normal_bf16((7, 64, D), 3, 1))
    offs = [0, 5, 7]
    lse = torch.empty(7, 64, device="cuda")
    args = (c, q, dev(np.asarray(offs, np.int32)))
    assert status_of(short, c, lambda: csa.hca_shared_attend(*args, softmax_scale=0.1)) & csa.CSA_DEV_TIMEOUT
    c.status.zero_()
    out = csa.hca_shared_attend(*args, softmax_scale=0.1, lse=lse)
    assert csa.csa_read_device_status(c) == 0
    check(out, lse, c, q, offs, None, 0.1)


def test_cache_copy_in_place(short):
    import torch

    import fp4_kv_cache_csa_b200 as csa

    c = random_cache(1, 900, 512)
    before = c.fp4.clone()
    slot, keep = dev(np.zeros(1, np.int32)), dev(np.arange(0, 800, 2, dtype=np.int32)[None])
    assert status_of(short, c, lambda: csa.csa_cache_copy(c, c, slot, slot, keep=keep)) & csa.CSA_DEV_TIMEOUT
    # the first tile needs no other and is written; the one that waits for it is not
    assert torch.equal(c.fp4[0, :64], before[0, 0:128:2])
    assert torch.equal(c.fp4[0, 64:128], before[0, 64:128])
    c.fp4.copy_(before)
    c.n_blocks.fill_(900)
    c.status.zero_()
    csa.csa_cache_copy(c, c, slot, slot, keep=keep)
    assert csa.csa_read_device_status(c) == 0
    assert torch.equal(c.fp4[0, :400], before[0, 0:800:2])
