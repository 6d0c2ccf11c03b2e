"""csa_cache_copy from several host threads at once, each with a stream, a workspace and a cache layout of its own."""
import ctypes
import threading

import numpy as np
import pytest

from gpu_util import dev
from test_gpu_cache_copy import BF16, make, planes_of

pytestmark = pytest.mark.gpu


def test_layouts_side_by_side():
    import torch

    import fp4_kv_cache_csa_b200 as csa

    # tiles of 50 KB (more shared memory than a kernel has without asking) and of 4 KB
    layouts = [(512, 1, BF16, 256), (64, 0, None, 0), (512, 0, BF16, 256), (128, 0, None, 0)]
    lib, slots, work, seen = csa.load_library(), dev(np.array([0, 1], np.int32)), [], set()
    for k, (dim, fmt, key, dI) in enumerate(layouts):
        src, dst = (make(2, 130, dim, fmt, key, dI, seed=2 * k + j, n=[130, 77])[0] for j in (0, 1))
        ws = torch.empty(csa.csa_cache_copy_workspace(dst, 2), dtype=torch.uint8, device="cuda")
        work.append((src, dst, ws, torch.cuda.Stream()))
    torch.cuda.synchronize()
    begin = threading.Barrier(len(work))

    def loop(src, dst, ws, stream):
        # the library's call alone (a thread holds no Python lock in it), so that calls overlap as often as they can
        cs, cd = src.c_struct(), dst.c_struct()
        args = (ctypes.byref(cs), ctypes.byref(cd), 2, slots.data_ptr(), slots.data_ptr(), None, 0, None, ws.data_ptr(),
                ws.nbytes, stream.cuda_stream)
        begin.wait()
        for _ in range(30):
            seen.update([lib.csa_cache_copy(*args) for _ in range(500)])
            stream.synchronize()

    threads = [threading.Thread(target=loop, args=w) for w in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert seen == {0}, seen
    for src, dst, _, _ in work:
        assert csa.csa_read_device_status(dst) == 0
        for a, b in zip(planes_of(src), planes_of(dst)):
            assert np.array_equal(a[0], b[0]) and np.array_equal(a[1, :77], b[1, :77])
