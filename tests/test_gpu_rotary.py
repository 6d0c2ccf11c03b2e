"""GPU parity of csa_rotary with the definition in 64 bits.

Tolerance per element, from the arithmetic (u = 2^-24): the reduced angle, as a multiple of pi in
[-1, 1], is rounded once (pi u in the angle); sine and cosine are good to 2 ulp (2 u) and scaled by
mscale (u); the two products and their sum round by at most u each on |a| and |b|. Together
(pi + 2 + 1 + 1 + 1) u < 9 u on mscale (|a| + |b|). The output's own rounding adds half a step of
its type (bf16: 2^-8, float32: 2^-24, relative)."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def dtype(name):
    import torch

    return torch.bfloat16 if name == "bf16" else torch.float32


def make(shape, name, seed):
    import torch

    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype(name))


def positions(rows, seed, top=1 << 20):
    import torch

    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1000)
    return torch.randint(0, top, (rows,), generator=g, device="cuda", dtype=torch.int32)


def frequencies(rot, scaled=1.0):
    import fp4_kv_cache_csa_b200 as csa

    return csa.csa_rotary_frequencies(rot, scaling=csa.CSA_ROPE_SCALE_LINEAR, factor=scaled)[0].cuda()


def reference(x, pos, inv, begin, half, inverse, mscale):
    """float64 numpy: (y, bound without the output's rounding)."""
    x = x.detach().double().cpu().numpy()
    x3 = x.reshape(x.shape[0], -1, x.shape[-1])
    f = inv.cpu().numpy().astype(np.float64)
    t = pos.cpu().numpy().astype(np.float64)[:, None] * f[None]
    c, s = np.cos(t)[:, None] * mscale, np.sin(t)[:, None] * mscale * (-1 if inverse else 1)
    r = len(f)
    ia = begin + (np.arange(r) if half else 2 * np.arange(r))
    ib = ia + (r if half else 1)
    y, tol = x3.copy(), np.zeros_like(x3)
    a, b = x3[..., ia], x3[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
    tol[..., ia] = tol[..., ib] = 9 * 2.0 ** -24 * abs(mscale) * (np.abs(a) + np.abs(b))
    return y.reshape(x.shape), tol.reshape(x.shape)


def check(got, x, pos, inv, begin, half, inverse, mscale, out):
    y, tol = reference(x, pos, inv, begin, half, inverse, mscale)
    err = np.abs(got.double().cpu().numpy() - y)
    bad = err > tol + HALF_STEP[out] * (np.abs(y) + tol)
    assert not bad.any(), (bad.sum(), err.max())


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("kinds", [("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("rows,heads,dim,begin,rot", [
    (1, 1, 64, 0, 64), (5, 64, 512, 448, 64), (1, 64, 512, 448, 64), (300, 1, 128, 0, 128), (33, 3, 128, 32, 64),
    (7, 2, 192, 64, 64),             # channels copied on both sides
    (3, 5, 30, 4, 22), (2, 1, 2, 0, 2), (9, 2, 40, 8, 24),  # not in chunks of 16 bytes (half layout: 24 / 2 = 12)
    (2, 3, 1030, 6, 1024), (1, 2, 8192, 0, 8192),  # a vector over several thread blocks
    (257, 1, 64, 56, 8), (1025, 2, 16, 0, 16)])
def test_parity(rows, heads, dim, begin, rot, kinds, inverse, half):
    import fp4_kv_cache_csa_b200 as csa

    x, pos, inv = make((rows, heads, dim), kinds[0], dim + rows), positions(rows, rows), frequencies(rot, 2.0)
    before = x.clone()
    got = csa.csa_rotary(x, pos, inv, rot_begin=begin, layout=int(half), inverse=inverse, mscale=1.25,
                         out_dtype=dtype(kinds[1]))
    check(got, x, pos, inv, begin, half, inverse, 1.25, kinds[1])
    assert (x == before).all()


@pytest.mark.parametrize("half", [False, True])
def test_far_and_negative_positions(half):
    import fp4_kv_cache_csa_b200 as csa
    import torch

    pos = torch.tensor([0, 1, -1, 2**31 - 1, -2**31, 2**24 + 1, 1048575, -77777], dtype=torch.int32, device="cuda")
    x, inv = make((8, 4, 64), "f32", 3), frequencies(64)
    got = csa.csa_rotary(x, pos, inv, layout=int(half))
    check(got, x, pos, inv, 0, half, False, 1.0, "f32")
    assert (got[0] == x[0]).all()  # position 0 is the identity, bit for bit


@pytest.mark.parametrize("name", ["bf16", "f32"])
@pytest.mark.parametrize("half", [False, True])
def test_in_place_touches_the_rotated_channels_only(name, half):
    import fp4_kv_cache_csa_b200 as csa
    import torch

    buf = make((40, 8, 160), name, 7)
    buf[:, :, 130:] = float("nan")
    buf[::3, :, 0] = float("inf")
    x = buf[:, 1:7, 16:144]                      # a view: heads and channels around it belong to others
    want = buf.clone()
    pos, inv = positions(40, 5), frequencies(64)
    clean = torch.nan_to_num(x.clone(), posinf=0.0)
    y = csa.csa_rotary(x, pos, inv, out=x, rot_begin=32, layout=int(half))
    assert y is x
    check(x[..., 32:96], clean[..., 32:96], pos, inv, 0, half, False, 1.0, name)
    want[:, 1:7, 48:112] = buf[:, 1:7, 48:112]
    assert torch.equal(torch.nan_to_num(want, nan=7.0), torch.nan_to_num(buf, nan=7.0))


def test_strides_broadcast_and_offsets():
    import fp4_kv_cache_csa_b200 as csa
    import torch

    pos, inv = positions(12, 8), frequencies(32)
    x = make((12, 6, 64), "bf16", 11)
    want = csa.csa_rotary(x, pos, inv)
    # head-major input and output, an offset of one element (one channel at a time), a broadcast row
    xt = x.transpose(0, 1).contiguous().transpose(0, 1)
    ot = torch.empty(6, 12, 64, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    assert torch.equal(csa.csa_rotary(xt, pos, inv, out=ot), want)
    odd = torch.zeros(12 * 6 * 64 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(12, 6, 64)
    odd.copy_(x)
    assert torch.equal(csa.csa_rotary(odd, pos, inv), want)
    one = x[:1].expand(12, 6, 64)
    assert torch.equal(csa.csa_rotary(one, pos, inv), csa.csa_rotary(one.contiguous(), pos, inv))
    # input and output as other channels of the same rows
    both = torch.cat((x, torch.zeros_like(x)), -1)
    csa.csa_rotary(both[..., :64], pos, inv, out=both[..., 64:])
    assert torch.equal(both[..., 64:], want) and torch.equal(both[..., :64], x)
    # [rows, dim] without heads
    assert torch.equal(csa.csa_rotary(x[:, 2], pos, inv), want[:, 2])


def test_no_rows():
    import fp4_kv_cache_csa_b200 as csa

    x = make((0, 4, 64), "bf16", 1)
    assert csa.csa_rotary(x, positions(0, 1), frequencies(64)).shape == x.shape


@pytest.mark.parametrize("half", [False, True])
def test_gradient(half):
    """The inverse is the gradient: against the formula's transpose (float64 autograd) and against
    central differences of a float64 loss through the forward call."""
    import fp4_kv_cache_csa_b200 as csa
    import torch

    rows, heads, dim, rot = 6, 3, 48, 32
    x, dy = make((rows, heads, dim), "f32", 21), make((rows, heads, dim), "f32", 22)
    pos, inv, m = positions(rows, 23), frequencies(rot), 1.1
    dx = csa.csa_rotary(dy, pos, inv, layout=int(half), inverse=True, mscale=m)
    # copied channels carry no mscale, so theirs is dy itself
    check(dx, dy, pos, inv, dim - rot, half, True, m, "f32")
    xr = x.double().cpu().requires_grad_()
    t = pos.double().cpu()[:, None, None] * inv.double().cpu()
    c, s = torch.cos(t) * m, torch.sin(t) * m
    lead, z = xr[..., :dim - rot], xr[..., dim - rot:]
    a, b = (z[..., :rot // 2], z[..., rot // 2:]) if half else (z[..., 0::2], z[..., 1::2])
    ya, yb = a * c - b * s, a * s + b * c
    y = torch.cat((lead, torch.cat((ya, yb), -1) if half else torch.stack((ya, yb), -1).flatten(-2)), -1)
    y.backward(dy.double().cpu())
    # |a| + |b| of dy is at most 10 here: 9 u * 1.1 * 10, and u of the result
    assert float((dx.double().cpu() - xr.grad).abs().max()) <= 2.0 ** -24 * (9 * 1.1 * 10 + 10)
    # the map is linear, so a central difference has no truncation error: steps of 1 leave the
    # rounding of y, two values of at most (9 + 1) u * 1.1 * (|a| + |b|) <= 130 u, summed over a pair with |dy| <= 5
    for r, h, k in ((0, 0, 0), (1, 2, 16), (5, 1, 47), (3, 0, 33)):
        lo, hi = x.clone(), x.clone()
        lo[r, h, k] -= 1
        hi[r, h, k] += 1
        step = float(hi[r, h, k].double() - lo[r, h, k].double())

        def loss(v):
            return float((csa.csa_rotary(v, pos, inv, layout=int(half), mscale=m).double() * dy.double()).sum())

        diff = (loss(hi) - loss(lo)) / step
        assert abs(diff - float(dx[r, h, k])) <= 2 * 2 * 5 * 130 * 2.0 ** -24


def test_streams_and_graphs():
    import fp4_kv_cache_csa_b200 as csa
    import torch

    x, pos, inv = make((64, 8, 128), "bf16", 31), positions(64, 31), frequencies(64)
    want = csa.csa_rotary(x, pos, inv)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = torch.empty_like(want)
    csa.csa_rotary(x, pos, inv, out=got, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    out = torch.zeros_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        csa.csa_rotary(x, pos, inv, out=out)
    for seed in (1, 2):
        x.copy_(make((64, 8, 128), "bf16", seed))
        pos.copy_(positions(64, seed))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, csa.csa_rotary(x, pos, inv))
