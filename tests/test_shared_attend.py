"""hca_shared_attend: what the host refuses (no GPU needed)."""
import ctypes

import pytest
import torch

import fp4_kv_cache_csa_b200 as csa
from fp4_kv_cache_csa_b200 import build as csa_build

OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_CUDA = range(7)


@pytest.fixture(scope="module")
def lib():
    csa_build.build()
    return csa.load_library()


def fake(**kw):
    # host addresses that are never dereferenced
    d = dict(batch=2, dim=512, block=4, capacity=1024, fp4=0x10000, scale=0x20000, idx_key=None, idx_dim=0,
             idx_dtype=0, n_blocks=0x40000, status=None, scale_fmt=0, idx_key_scale=None)
    d.update(kw)
    return csa._CCache(*(d[f[0]] for f in csa._CCache._fields_))


def call(lib, c=None, q=0x10000000, n=4, heads=64, offs=0x1000, pos=None, jo=None, jl=None, out=0x20000000,
         lse=None, ws=None, wsb=0):
    c = fake() if c is None else c
    return lib.hca_shared_attend(ctypes.byref(c), q, n, heads, offs, pos, jo, jl, 0.1, out, lse, ws, wsb, None)


def test_refusals(lib):
    assert lib.hca_shared_attend(None, 16, 1, 1, 4, None, None, None, 0.1, 4096, None, None, 0, None) == ERR_NULL
    assert call(lib, c=fake(fp4=None)) == ERR_NULL
    assert call(lib, q=None) == ERR_NULL
    assert call(lib, offs=None) == ERR_NULL
    assert call(lib, out=None) == ERR_NULL
    assert call(lib, jo=0x30000000) == ERR_NULL       # the joined part is all or nothing
    assert call(lib, jl=0x30000000) == ERR_NULL
    assert call(lib, n=0) == ERR_SHAPE
    assert call(lib, heads=0) == ERR_SHAPE
    assert call(lib, heads=65) == ERR_UNSUPPORTED
    assert call(lib, c=fake(dim=256)) == ERR_UNSUPPORTED
    assert call(lib, q=0x10000008) == ERR_ALIGN
    assert call(lib, out=0x20000008) == ERR_ALIGN
    assert call(lib, jo=0x30000004, jl=0x40000000) == ERR_ALIGN
    assert call(lib, offs=0x1002) == ERR_ALIGN
    assert call(lib, pos=0x1002) == ERR_ALIGN
    assert call(lib, lse=0x50000002) == ERR_ALIGN
    size = 4 * 64 * 512
    assert call(lib, out=0x10000000) == ERR_SHAPE                                    # over q
    assert call(lib, out=0x10000000 + 2 * size - 16) == ERR_SHAPE
    assert call(lib, jo=0x20000000, jl=0x40000000) == ERR_SHAPE                      # over join_out
    assert call(lib, jo=0x30000000, jl=0x40000000, lse=0x40000000) == ERR_SHAPE      # over join_lse
    assert call(lib, jo=0x30000000, jl=0x40000000, lse=0x30000000 + 4 * size - 4) == ERR_SHAPE
    assert call(lib, lse=0x20000000) == ERR_SHAPE
    if not torch.cuda.is_available():
        # the workspace's size depends on the device: without one the query says 0 and a call ends there
        assert lib.hca_shared_attend_workspace(ctypes.byref(fake()), 4, 64) == 0
        assert call(lib) == ERR_CUDA
    for bad in ((0, 64), (4, 0), (4, 65)):
        assert lib.hca_shared_attend_workspace(ctypes.byref(fake()), *bad) == 0
    assert lib.hca_shared_attend_workspace(ctypes.byref(fake(dim=256)), 4, 64) == 0
    assert lib.hca_shared_attend_workspace(None, 4, 64) == 0


def test_binding_refusals(lib):
    c = csa.Cache.allocate(2, 8, 128, 4, device="cpu")
    q, offs = torch.zeros(3, 4, 128, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    f = torch.zeros(3, 4, 128)
    for kw, name in ((dict(q=q.float()), "q"), (dict(q=q[..., :64]), "q"), (dict(q=q.transpose(0, 1)), "q"),
                     (dict(q_offsets=offs.long()), "q_offsets"), (dict(q_offsets=offs[:2]), "q_offsets"),
                     (dict(q_pos=offs[:2]), "q_pos"), (dict(join_out=f.half()), "join_out"),
                     (dict(join_lse=f), "join_lse"), (dict(out=f), "out"), (dict(lse=f), "lse")):
        with pytest.raises(csa.CsaError, match=name):
            csa.hca_shared_attend(**dict(dict(cache=c, q=q, q_offsets=offs), **kw))
    with pytest.raises(csa.CsaError, match="CUDA device"):
        csa.hca_shared_attend(c, q, offs)


def test_other_streams_and_workspaces_are_refused():
    class Stream:
        device = torch.device("cuda:1")

    with pytest.raises(csa.CsaError, match="stream is of cuda:1"):
        csa._on(torch.device("cuda:0"), Stream(), lambda s: None)
    with pytest.raises(csa.CsaError, match="workspace"):
        csa._expect_workspace("hca_shared_attend", torch.empty(4096, dtype=torch.uint8), torch.device("cuda:0"))
    with pytest.raises(csa.CsaError, match="workspace"):
        csa._expect_workspace("hca_shared_attend", torch.empty(64, 64, dtype=torch.uint8).t()[:9], torch.device("cpu"))
