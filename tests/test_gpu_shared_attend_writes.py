"""hca_shared_attend: tensors passed as out and lse count as written."""
import numpy as np
import pytest

from gpu_util import dev
from test_gpu_shared_attend import random_cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", ["out", "lse"])
def test_kept_results_are_found_changed(name):
    import torch

    import fp4_kv_cache_csa_b200 as csa

    c = random_cache(1, 100, 128)
    q = torch.randn(3, 16, 128, device="cuda").to(torch.bfloat16)
    out, lse = torch.zeros_like(q), torch.zeros(3, 16, device="cuda")
    kept = out if name == "out" else lse
    w = torch.ones_like(kept, requires_grad=True)
    y = (w * kept).float().sum()                       # keeps it for its backward pass
    csa.hca_shared_attend(c, q, dev(np.array([0, 3], np.int32)), out=out, lse=lse)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
