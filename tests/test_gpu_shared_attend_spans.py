"""hca_shared_attend: slots whose first blocks are smaller than the others by up to fp4's whole range of scales,
at the tolerance that tests/shared_model.py derives."""
import numpy as np
import pytest

from gpu_util import dev
from shared_model import attend, entries
from test_gpu_shared_attend import random_cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,H", [(128, 16), (512, 64)])
@pytest.mark.parametrize("first,others", [((1, 1), (127, 130)), ((1, 6), (118, 122)), ((1, 20), (126, 128)),
                                          ((30, 40), (125, 130)), ((2, 3), (100, 160)), ((1, 1), (1, 1)),
                                          ((127, 128), (1, 3)), ((150, 152), (1, 127)), ((0, 0), (50, 60)),
                                          ((1, 1), (175, 180)), ((1, 9), (1, 180))])
def test_first_blocks_of_another_scale(D, H, first, others):
    import torch

    import fp4_kv_cache_csa_b200 as csa

    c = random_cache(1, 700, D, seed=3)
    g = torch.Generator("cuda").manual_seed(4)
    for rows, (lo, hi) in ((slice(0, 256), first), (slice(256, None), others)):
        s = c.scale[0, rows]
        s.copy_(torch.randint(lo, hi + 1, s.shape, generator=g, device="cuda", dtype=torch.uint8))
    c.scale[0, 5::50] = 0                             # rows of zeros among them
    c.fp4[0, c.scale[0].amax(1) == 0] = 0
    q = torch.randn(10240 // H, H, D, generator=g, device="cuda").to(torch.bfloat16)
    e = entries(c.fp4[0], c.scale[0])
    scale = 8.0 / float((q[0].double() @ e.T).std())  # logits of a few bits
    scale = min(scale, 2.0 ** 100)
    lse = torch.empty(q.shape[:2], device="cuda")
    got = csa.hca_shared_attend(c, q, dev(np.array([0, q.shape[0]], np.int32)), softmax_scale=scale, lse=lse)
    out, ref, tol, dl = attend(e, q, scale)
    assert csa.csa_read_device_status(c) == 0
    d = (lse.double() - ref).abs()
    assert (d <= dl).all(), float((d / dl).max())
    # bf16 keeps no output below 2^-133
    err = (got.double() - out).abs()
    assert (err <= tol + 2.0 ** -133).all(), float((err / (tol + 2.0 ** -133)).max())
