"""csa_cache_copy in place whose bounded waits run out: n_blocks ends before the first block that was not written, so
that no block of the old contents counts as a compacted one (see test_gpu_lost_arrivals.py for the test build)."""
import numpy as np
import pytest

from gpu_util import dev
from test_gpu_lost_arrivals import short, status_of  # noqa: F401 (short: fixture)
from test_gpu_shared_attend import random_cache

pytestmark = pytest.mark.gpu


def test_count_ends_at_the_first_block_not_written(short):  # noqa: F811
    import torch

    import fp4_kv_cache_csa_b200 as csa

    c = random_cache(3, 900, 512)
    before = c.fp4.clone()
    # slot 0: the second tile waits in vain for the first, which has sources among the second's places; slot 1: the
    # third tile does, and later ones are written; slot 2: one tile, which waits for none
    keep = np.full((3, 800), -1, np.int32)
    keep[0, :400] = np.arange(0, 800, 2)
    keep[1, :32] = np.arange(32)
    keep[1, 32:400] = np.arange(132, 500)
    keep[2, :30] = np.arange(100, 130)
    slots = dev(np.arange(3, dtype=np.int32))
    keep_d = dev(keep)
    for status in (c.status, None):                    # with a status word and without one
        c.fp4.copy_(before)
        c.n_blocks.fill_(900)
        seen = csa.Cache(fp4=c.fp4, scale=c.scale, n_blocks=c.n_blocks, block=4, status=status)
        bits = status_of(short, c, lambda: csa.csa_cache_copy(seen, seen, slots, slots, keep=keep_d))
        assert bits == (0 if status is None else csa.CSA_DEV_TIMEOUT)
        n = c.n_blocks.tolist()
        assert n == [64, 128, 30]
        for s in range(3):
            assert torch.equal(c.fp4[s, :n[s]], before[s][dev(keep[s, :n[s]]).long()])
