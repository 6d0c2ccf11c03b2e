"""The tolerance of tests/shared_model.py: the arithmetic it stands for passes, a tile left out of the output or put
in another order does not, at lengths where each tile weighs little (no GPU needed; faults are in the copy made here)."""
import pytest
import torch

from fp4_kv_cache_csa_b200 import datagen
from shared_model import attend, entries


def by_hand(e, q, scale, start=7.0, fault=None):
    """Output and lse of one query with weights as fp16 numbers that start at 2^start, sums in float64, output in bf16."""
    u = scale * (q.double() @ e.T) / torch.log(torch.tensor(2.0, dtype=torch.float64))
    rho = u.amax(-1, keepdim=True) - start
    p = torch.exp2(u - rho)
    total = p.sum(-1)
    p = p.half().double()
    x = e.clone()
    t = slice(e.shape[0] // 2 // 128 * 128, e.shape[0] // 2 // 128 * 128 + 128)
    if fault == "tile left out":
        x[t] = 0
    if fault == "tile reversed":
        x[t] = x[t].flip(0)
    if fault == "tile twice":
        x[t] *= 2
    return (p @ x / total[:, None]).to(torch.bfloat16), (torch.log2(total) + rho[:, 0]) * 0.6931471805599453


def cache(n, D, seed):
    fp4, sc = datagen.random_cache_bytes(n, D, seed, 40, scale_lo=123, scale_hi=126)
    return entries(torch.from_numpy(fp4.reshape(n, D // 2)), torch.from_numpy(sc.reshape(n, D // 32)))


@pytest.mark.parametrize("D,n", [(512, 16385), (512, 4101), (128, 30011)])
@pytest.mark.parametrize("sharp", [1.0, 3.0])
def test_faults_of_one_tile_do_not_pass(D, n, sharp):
    e = cache(n, D, n)
    q = torch.randn(1, 64, D, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    scale = sharp * D ** -0.5
    out, lse, tol, dl = attend(e, q, scale)
    got, got_lse = by_hand(e, q[0], scale)
    assert ((got.double() - out[0]).abs() <= tol[0]).all() and ((got_lse - lse[0]).abs() <= dl[0]).all()
    for fault in ("tile left out", "tile reversed", "tile twice"):
        got, _ = by_hand(e, q[0], scale, fault=fault)
        assert ((got.double() - out[0]).abs() > 1.5 * tol[0]).any(), fault


def test_small_weights_left_out_do_not_pass():
    D, n = 128, 40000
    codes = torch.zeros(n, D // 2, dtype=torch.uint8)
    codes[0, :D // 4] = 0x77
    codes[1:, D // 4:] = 0x22
    e = entries(codes, torch.full((n, D // 32), 127, dtype=torch.uint8))
    q = torch.zeros(1, 2, D)
    q[0, :, :D // 2] = 25.3 * 0.6931471805599453 / (6 * D // 2)
    q = q.to(torch.bfloat16)
    out, _, tol, _ = attend(e, q, 1.0)
    assert ((by_hand(e, q[0], 1.0)[0].double() - out[0]).abs() <= tol[0]).all()
    assert ((by_hand(e, q[0], 1.0, start=0.0)[0].double() - out[0]).abs() > 2 * tol[0]).any()
