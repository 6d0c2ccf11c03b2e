"""csa_cache_copy without jobs launches nothing and is no error, with a list's columns too (no GPU needed)."""
import torch

import fp4_kv_cache_csa_b200 as csa
from test_cache_copy import ERR_SHAPE, OK, call, lib  # noqa: F401 (lib: fixture)


def test_no_jobs(lib):  # noqa: F811
    assert call(lib, n=0, s=None, d=None, ws=None, wsb=0) == OK
    assert call(lib, n=0, s=None, d=None, cols=512, ws=None, wsb=0) == OK         # an empty [0, 512] has no address
    assert call(lib, n=0, s=None, d=None, keep=0x3000, cols=512, ws=None, wsb=0) == OK
    assert call(lib, n=0, cols=-1) == ERR_SHAPE
    assert call(lib, n=1, cols=512) == ERR_SHAPE


def test_no_jobs_through_the_binding(lib, monkeypatch):  # noqa: F811
    monkeypatch.setattr(csa, "_on", lambda device, stream, launch: launch(None))
    c = csa.Cache.allocate(2, 8, 128, 4, device="cpu")
    none = torch.zeros(0, dtype=torch.int32)
    csa.csa_cache_copy(c, c, none, none)
    csa.csa_cache_copy(c, c, none, none, keep=torch.zeros(0, 512, dtype=torch.int32), max_blocks=none)
