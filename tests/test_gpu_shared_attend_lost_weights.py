"""hca_shared_attend whose O^T never gets its last tile's weights: every thread that waits for that product gives up,
while S^T was issued to its end. The call flags CSA_DEV_TIMEOUT and returns with nothing of its own still running,
and the shipped library works in the same context (a test build, as in test_gpu_lost_arrivals.py)."""
import ctypes

import numpy as np
import pytest

from fp4_kv_cache_csa_b200 import datagen
from gpu_util import dev
from test_gpu_lost_arrivals import status_of
from test_gpu_shared_attend import check, random_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lost(tmp_path_factory):
    import fp4_kv_cache_csa_b200 as csa
    from fp4_kv_cache_csa_b200 import build as csa_build

    at = tmp_path_factory.mktemp("weights")
    path = csa_build.build(force=True, defines=["CSA_WAIT_CYCLES=1000000", "CSA_TEST_LOST_WEIGHTS"],
                           lib_path=str(at / "libcsa_weights.so"), build_dir=str(at / "build"))
    return csa.declare(ctypes.CDLL(path))


@pytest.mark.parametrize("D,fmt,n,queries", [(512, 0, 1500, 7), (512, 1, 300, 400), (128, 0, 2000, 7), (128, 1, 90, 400)])
def test_last_weights_lost(lost, D, fmt, n, queries):
    import torch

    import fp4_kv_cache_csa_b200 as csa

    c = random_cache(2, n, D, fmt, n=[n, n // 2])
    q = dev(datagen.normal_bf16((queries, 64, D), 3, 1))
    offs = [0, queries // 2, queries]
    args = (c, q, dev(np.asarray(offs, np.int32)))
    for _ in range(3):
        assert status_of(lost, c, lambda: csa.hca_shared_attend(*args, softmax_scale=0.1)) & csa.CSA_DEV_TIMEOUT
    lse = torch.empty(queries, 64, device="cuda")
    out = csa.hca_shared_attend(*args, softmax_scale=0.1, lse=lse)
    assert csa.csa_read_device_status(c) == 0
    check(out, lse, c, q, offs, None, 0.1)
