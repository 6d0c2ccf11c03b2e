"""hca_shared_attend: blocks of small weight that count together, and long slots, at the tolerance that
tests/shared_model.py derives."""
import math

import numpy as np
import pytest

from gpu_util import dev, make_cache
from shared_model import attend, entries

pytestmark = pytest.mark.gpu


def run(c, q, scale, seen=None, pos=None):
    import torch

    import fp4_kv_cache_csa_b200 as csa

    lse = torch.empty(q.shape[:2], device="cuda")
    got = csa.hca_shared_attend(c, q, dev(np.array([0, q.shape[0]], np.int32)), pos, softmax_scale=scale, lse=lse)
    assert csa.csa_read_device_status(c) == 0
    e = entries(c.fp4[0, :int(c.n_blocks[0])], c.scale[0, :int(c.n_blocks[0])], bool(c.scale_fmt))
    out, ref, tol, dl = attend(e, q, scale, seen)
    err = (got.double() - out).abs()
    assert (err <= tol).all(), (float(err.max()), float((err / tol.clamp(min=1e-300)).max()))
    d = (lse.double() - ref).abs()
    assert (d <= dl).all(), float((d / dl).max())


@pytest.mark.parametrize("D,H,n", [(128, 64, 40000), (128, 16, 9000), (512, 64, 20000)])
@pytest.mark.parametrize("bits", [13.5, 25.05, 25.9, 31.0])
def test_many_small_weights_count(D, H, n, bits):
    # one block leads by `bits` bits and the others, alone in half of the channels, have next to no weight
    # each but n of it together; there are enough queries for one thread block to see a slot from end to end
    import torch

    fp4 = np.zeros((1, n, D // 2), np.uint8)
    fp4[0, 0, :D // 4] = 0x77
    fp4[0, 1:, D // 4:] = 0x22
    c = make_cache(fp4, np.full((1, n, D // 32), 127, np.uint8), [n], 4)
    q = torch.zeros(400 * H // 64, H, D, device="cuda")
    spread = 1 + 0.002 * torch.rand(q.shape[:2], generator=torch.Generator("cuda").manual_seed(1), device="cuda")
    q[..., :D // 2] = (bits * math.log(2) / (6 * D // 2) * spread)[..., None]
    run(c, q.to(torch.bfloat16), 1.0)


def test_small_weights_count_beside_a_raised_reference():
    # the lead comes tiles after the others: what they left is kept when the reference rises
    import torch

    D, n = 128, 9000
    fp4 = np.zeros((1, n, D // 2), np.uint8)
    fp4[0, :, D // 4:] = 0x22
    fp4[0, 5000] = 0
    fp4[0, 5000, :D // 4] = 0x77
    c = make_cache(fp4, np.full((1, n, D // 32), 127, np.uint8), [n], 4)
    q = torch.zeros(300, 64, D, device="cuda")
    q[..., :D // 2] = (torch.linspace(1, 60, 64, device="cuda") * math.log(2) / (6 * D // 2))[None, :, None]
    run(c, q.to(torch.bfloat16), 1.0)


@pytest.mark.parametrize("D,H,Q,n,fmt", [(512, 64, 1, 16385, 0), (512, 64, 40, 4101, 1), (128, 40, 320, 16385, 0),
                                         (512, 16, 20, 30011, 0)])
def test_long_slots(D, H, Q, n, fmt):
    import torch

    from test_gpu_shared_attend import random_cache

    c = random_cache(1, n, D, fmt, seed=n)
    q = torch.randn(Q, H, D, generator=torch.Generator("cuda").manual_seed(5), device="cuda").to(torch.bfloat16)
    run(c, q, D ** -0.5)
    pos = torch.randint(-1, 4 * n, (Q,), generator=torch.Generator("cuda").manual_seed(6), device="cuda", dtype=torch.int32)
    seen = [(int(p) + 1) // 4 for p in pos]
    run(c, q, 2 * D ** -0.5, seen, pos)
