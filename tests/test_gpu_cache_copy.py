"""csa_cache_copy on the GPU against the numpy model: every byte of every plane, n_blocks and status."""
import numpy as np
import pytest

from copy_model import copy_slots
from gpu_util import dev, host

pytestmark = pytest.mark.gpu

BF16, E4M3, MXFP4 = 0, 1, 2


def make(batch, cap, dim=512, fmt=0, key=None, dI=128, seed=0, n=None, at=0):
    """A cache of random bytes; `at`: bytes that its planes lie behind their allocation's start (16's multiple)."""
    import torch

    import fp4_kv_cache_csa_b200 as csa

    rng = np.random.default_rng(seed)
    rows = [dim // 2, dim // (16 if fmt else 32)]
    if key is not None:
        rows.append({BF16: 2 * dI, E4M3: dI, MXFP4: dI // 2}[key])
        if key == MXFP4:
            rows.append(dI // 32)
    planes = [rng.integers(0, 256, (batch, cap, r), dtype=np.uint8) for r in rows]
    n = np.asarray(rng.integers(0, cap + 1, batch) if n is None else n, np.int32)
    t = []
    for p in planes:
        buf = torch.zeros(p.size + at, dtype=torch.uint8, device="cuda")[at:]
        buf.copy_(torch.from_numpy(p.reshape(-1)))
        t.append(buf.view(p.shape))
    ik = None
    if key is not None:
        ik = t[2].view(torch.bfloat16) if key == BF16 else t[2]
    c = csa.Cache(fp4=t[0], scale=t[1], n_blocks=dev(n), block=4, idx_key=ik, idx_dtype=key or 0,
                  status=torch.zeros(1, dtype=torch.int32, device="cuda"), scale_fmt=fmt,
                  idx_key_scale=t[3] if key == MXFP4 else None)
    return c, planes, n


def planes_of(c):
    import torch

    t = [c.fp4, c.scale] + ([c.idx_key] if c.idx_key is not None else [])
    t += [c.idx_key_scale] if c.idx_key_scale is not None else []
    return [host(x.view(torch.uint8)) for x in t]


def i32(v):
    return None if v is None else dev(np.asarray(v, np.int32))


def run(src, dst, src_slot, dst_slot, keep=None, max_blocks=None):
    """src, dst: results of make(); dst None: within src."""
    import fp4_kv_cache_csa_b200 as csa

    same = dst is None
    dst = src if same else dst
    want, want_n, want_st = copy_slots(src[1], src[2], dst[1], dst[2], src_slot, dst_slot, keep, max_blocks, same)
    csa.csa_cache_copy(src[0], dst[0], i32(src_slot), i32(dst_slot), i32(keep), i32(max_blocks))
    status = csa.csa_read_device_status(dst[0])
    assert list(host(dst[0].n_blocks)) == list(want_n)
    for g, w in zip(planes_of(dst[0]), want):
        assert np.array_equal(g, w), np.argwhere(g != w)[:4]
    assert status == want_st
    if not same:  # the source keeps its bytes
        for g, w in zip(planes_of(src[0]), src[1]):
            assert np.array_equal(g, w)
    return status


def lists(src_n, src_slot, cols, seed, frac=0.5):
    rng = np.random.default_rng(seed)
    keep = np.full((len(src_slot), cols), -1, np.int32)
    for i, s in enumerate(src_slot):
        n = src_n[s] if 0 <= s < len(src_n) else 0
        pick = np.flatnonzero(rng.random(n) < frac)[:cols]
        keep[i, :len(pick)] = pick
    return keep


FORMATS = [(512, 0, None, 0), (512, 0, BF16, 256), (512, 1, MXFP4, 128), (128, 0, E4M3, 64), (64, 0, MXFP4, 64),
           (96, 0, E4M3, 128), (128, 1, BF16, 64)]  # dim 96: scale rows of 3 bytes


@pytest.mark.parametrize("cap", [1, 64, 65, 333])
@pytest.mark.parametrize("dim,fmt,key,dI", FORMATS)
def test_fork_between_caches(dim, fmt, key, dI, cap):
    src = make(3, cap, dim, fmt, key, dI, seed=cap, n=[cap, 0, max(1, cap - 1)])
    dst = make(9, cap + 6, dim, fmt, key, dI, seed=7, at=16)
    assert run(src, dst, [0, 0, 0, 0, 0, 2, 1, 0], [8, 1, 2, 3, 4, 0, 6, 5]) == 0


@pytest.mark.parametrize("dim,fmt,key,dI", FORMATS)
def test_fork_within_a_cache(dim, fmt, key, dI):
    src = make(7, 201, dim, fmt, key, dI, seed=11, n=[200, 131, 5, 0, 201, 77, 1])
    assert run(src, None, [0, 0, 1, 5], [2, 3, 4, 6], max_blocks=[1000, 70, 64, 0]) == 0


def test_cut_free_and_out_of_range():
    src = make(6, 90, seed=12, n=[90, 80, 70, 60, 50, 40])
    # cut slot 0 (which slot 1 is forked from, with its old length), free slot 2, bad slots, a slot written twice
    st = run(src, None, [0, 0, -1, 9, 3, 3, -5], [0, 1, 2, 4, 6, -1, 1], max_blocks=[33, 99, 9, 9, 9, 9, 9])
    assert st == 0x4


def test_jobs_that_would_overwrite_a_source_are_skipped():
    src = make(5, 70, seed=13, n=[70, 60, 50, 40, 30])
    assert run(src, None, [0, 1, 2], [1, 2, 3]) == 0x4           # only 2 -> 3 can go
    src = make(5, 70, seed=13, n=[70, 60, 50, 40, 30])
    keep = lists(src[2], [0, 0], 70, 5)
    assert run(src, None, [0, 0], [0, 1], keep=keep) == 0x4      # compacting slot 0 while slot 1 is made from it


def test_capacity_and_odd_counts():
    src = make(3, 100, seed=14, n=[100, 150, -3])                # counts beyond the capacity or below zero are clamped
    dst = make(3, 99, seed=15)
    assert run(src, dst, [0, 1, 2], [0, 1, 2]) == 0x2
    dst = make(3, 99, seed=15)
    assert run(src, dst, [0, 1, 2], [0, 1, 2], max_blocks=[99, -1, 4]) == 0


@pytest.mark.parametrize("dim,fmt,key,dI", FORMATS)
@pytest.mark.parametrize("cols", [1, 63, 400])
def test_compact_between_caches(dim, fmt, key, dI, cols):
    src = make(4, 391, dim, fmt, key, dI, seed=16, n=[391, 7, 200, 0])
    dst = make(6, 400, dim, fmt, key, dI, seed=17)
    slots = [0, 1, 2, 3, 0, -1]
    assert run(src, dst, slots, [5, 4, 3, 2, 1, 0], keep=lists(src[2], slots, cols, cols)) == 0


@pytest.mark.parametrize("frac", [0.02, 0.5, 0.98, 1.0])
@pytest.mark.parametrize("dim,fmt,key,dI", FORMATS[:4])
def test_compact_in_place(dim, fmt, key, dI, frac):
    src = make(5, 6007, dim, fmt, key, dI, seed=18, n=[6007, 6000, 1, 0, 4097])
    slots = [4, 0, 1, 2, 3]
    assert run(src, None, slots, slots, keep=lists(src[2], slots, 6007, 3, frac)) == 0


def test_compact_in_place_extremes():
    # the last blocks only (every source lies beyond every destination), one gap at the front
    # (every tile waits for its neighbour), identity, one far block
    n = 20000
    src = make(4, n, 128, 0, E4M3, 64, seed=19, n=[n] * 4)
    keep = np.full((4, n), -1, np.int32)
    keep[0, :5000] = np.arange(n - 5000, n)
    keep[1, :n - 1] = np.arange(1, n)
    keep[2] = np.arange(n)
    keep[3, 0] = n - 1
    assert run(src, None, [0, 1, 2, 3], [0, 1, 2, 3], keep=keep) == 0


def test_lists_end_where_they_stop_making_sense():
    src = make(5, 9000, 128, seed=20, n=[9000, 100, 9000, 9000, 9000])
    keep = np.full((5, 9000), -1, np.int32)
    keep[0, :3] = [5, 5, 6]               # not ascending
    keep[1, :4] = [0, 50, 100, 101]       # at the source's end
    keep[2] = np.arange(9000)
    keep[2, 5000] = 17                    # out of order behind the first check block
    keep[2, 200 + 5000:] = -1
    keep[3, :6] = [1, 2, -1, 3, 2, 9000]  # nothing behind the padding counts
    keep[4, :2] = [-7, 3]
    dst = make(5, 9000, 128, seed=21)
    assert run(src, dst, [0, 1, 2, 3, 4], [0, 1, 2, 3, 4], keep=keep) == 0x4
    ok = make(5, 9000, 128, seed=21)
    assert run(src, ok, [3, 4], [0, 1], keep=keep[3:]) == 0
    assert run(src, None, [2, 0], [2, 0], keep=keep[[2, 0]], max_blocks=[4999, 1]) == 0x4


def test_many_jobs_and_a_large_batch():
    rng = np.random.default_rng(22)
    src = make(40, 70, 128, 0, MXFP4, 64, seed=22)
    dst = make(1500, 70, 128, 0, MXFP4, 64, seed=23)   # slot tables in the workspace
    jobs = 1400
    assert run(src, dst, rng.integers(0, 40, jobs), rng.permutation(1500)[:jobs]) == 0


def test_offsets_beyond_32_bits():
    import torch

    import fp4_kv_cache_csa_b200 as csa

    cap, batch = 1 << 19, 34               # 34 x 2^19 x 256 bytes: the last slots lie beyond 2^32
    c = csa.Cache.allocate(batch, cap, 512, 4)
    n = 1000
    c.fp4[batch - 1, cap - n:] = torch.randint(0, 256, (n, 256), dtype=torch.uint8, device="cuda")
    c.scale[batch - 1, cap - n:] = torch.randint(0, 256, (n, 16), dtype=torch.uint8, device="cuda")
    want = c.fp4[batch - 1, cap - n:].clone(), c.scale[batch - 1, cap - n:].clone()
    c.n_blocks[batch - 1] = cap
    keep = torch.arange(cap - n, cap, dtype=torch.int32, device="cuda")[None]
    csa.csa_cache_copy(c, c, i32([batch - 1]), i32([batch - 2]), keep=keep)
    assert csa.csa_read_device_status(c) == 0
    assert torch.equal(c.fp4[batch - 2, :n], want[0]) and torch.equal(c.scale[batch - 2, :n], want[1])
    assert int(c.n_blocks[batch - 2]) == n and int(c.fp4[batch - 2, n:].sum()) == 0


def test_graph_stream_and_shared_workspace():
    import torch

    import fp4_kv_cache_csa_b200 as csa

    src, a, b = make(2, 300, seed=24, n=[300, 200]), make(2, 300, seed=25), make(2, 300, seed=26)
    keep = i32(lists(src[2], [0, 1], 300, 9))
    slots = i32([0, 1])
    ws = torch.empty(csa.csa_cache_copy_workspace(a[0], 2, 300), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    for c in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            csa.csa_cache_copy(src[0], c[0], slots, slots, keep=keep, workspace=ws)
        graphs.append(g)
    for g in graphs * 3:                   # two graphs over one workspace, in turn on one stream
        with torch.cuda.stream(side):
            g.replay()
    side.synchronize()
    for c in (a, b):
        want = copy_slots(src[1], src[2], c[1], c[2], [0, 1], [0, 1], host(keep))
        assert all(np.array_equal(g, w) for g, w in zip(planes_of(c[0]), want[0]))
        assert list(host(c[0].n_blocks)) == list(want[1])
    other = make(2, 300, seed=27)
    csa.csa_cache_copy(src[0], other[0], slots, slots, stream=side)
    side.synchronize()
    assert list(host(other[0].n_blocks)) == [300, 200]


def test_compacted_selection_attends_like_the_selection():
    """The indexer's blocks moved to a cache of their own: dense attention over it is the sparse attention."""
    import torch

    import fp4_kv_cache_csa_b200 as csa
    from fp4_kv_cache_csa_b200 import datagen

    B, n, k, H, D = 3, 2048, 192, 64, 512
    fp4, sc = datagen.random_cache_bytes(B * n, D, 5, 40, scale_lo=123, scale_hi=126)
    keys = datagen.normal_bf16((B, n, 128), 5, 7)
    src = csa.Cache(fp4=dev(fp4.reshape(B, n, D // 2)), scale=dev(sc.reshape(B, n, D // 32)), n_blocks=i32([n] * B),
                    block=4, idx_key=dev(keys), idx_dtype=BF16, status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    q, qo, pos = dev(datagen.normal_bf16((B, H, D), 5, 8)), i32([0, 1, 2, 3]), i32([4 * n - 1] * B)
    sel = csa.csa_index_topk(src, dev(datagen.normal_bf16((B, 4, 128), 5, 9)), dev(datagen.normal_f32((B, 4), 5, 10)),
                             qo, pos, k)
    want = csa.csa_decode_attend(src, q, qo, sel)
    dst = csa.Cache.allocate(B, k, D, 4, 128)
    csa.csa_cache_copy(src, dst, i32([0, 1, 2]), i32([0, 1, 2]), keep=sel)
    got = csa.hca_decode_attend(dst, q, qo, pos)
    assert csa.csa_read_device_status(dst) == 0
    assert torch.equal(got, want)          # the same entries in the same order through the same kernel
