"""csa_cache_copy with lists around the limits of what its plan kernel reads by itself: 4096 columns, and 32768
entries in all."""
import pytest

from test_gpu_cache_copy import E4M3, lists, make, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("jobs,cols", [(8, 4096), (7, 4097), (1, 8192), (9, 4096), (33, 1000), (1, 4096), (1, 4097)])
def test_lists_around_the_limits(jobs, cols):
    src = make(jobs, 8200, 64, 0, E4M3, 64, seed=jobs, n=[8200 - 5 * i for i in range(jobs)])
    dst = make(jobs, 8200, 64, 0, E4M3, 64, seed=cols)
    slots = list(range(jobs))
    keep = lists(src[2], slots, cols, cols, 0.6)
    assert run(src, dst, slots, slots[::-1], keep=keep) == 0
    assert run(src, None, slots, slots, keep=keep) == 0
    # the last entry of a full list, right or beyond the slot's end
    keep[0] = range(cols)
    keep[0, cols - 1] = 8199
    for n, status in ((8200, 0), (8199, 0x4)):
        src = make(1, 8200, 64, 0, E4M3, 64, seed=jobs, n=[n])
        dst = make(2, 8200, 64, 0, E4M3, 64, seed=cols)
        assert run(src, dst, [0], [1], keep=keep[:1]) == status
