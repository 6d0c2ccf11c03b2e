"""csa_rotary in a training step: wrapped in an autograd function of the caller's, with the inverse as its backward
pass, and in place on tensors that other operators have kept."""
import pytest

pytestmark = pytest.mark.gpu


def test_inverse_as_a_backward_pass():
    import torch

    import fp4_kv_cache_csa_b200 as csa

    class Rotary(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, pos, inv):
            ctx.save_for_backward(pos, inv)
            return csa.csa_rotary(x, pos, inv)

        @staticmethod
        def backward(ctx, dy):
            pos, inv = ctx.saved_tensors
            return csa.csa_rotary(dy.contiguous(), pos, inv, inverse=True), None, None

    x = torch.randn(5, 3, 64, device="cuda", requires_grad=True)
    pos, inv = torch.arange(5, dtype=torch.int32, device="cuda") * 999, torch.rand(16, device="cuda")
    dy = torch.randn_like(x)
    (Rotary.apply(x, pos, inv) * dy).sum().backward()
    t = pos.double()[:, None, None] * inv.double()
    z = torch.complex(dy[..., 32::2].double(), dy[..., 33::2].double()) * torch.polar(torch.ones_like(t), -t)
    # 9 steps of 2^-24 on |a| + |b| (at most 10 here), and the result's own rounding
    want = torch.cat((dy[..., :32].double(), torch.stack((z.real, z.imag), -1).flatten(-2)), -1)
    assert float((x.grad.double() - want).abs().max()) <= 2.0 ** -24 * (9 * 10 + 10)


def test_a_call_in_place_counts_as_a_write():
    import torch

    import fp4_kv_cache_csa_b200 as csa

    w = torch.ones(4, 2, 64, device="cuda", requires_grad=True)
    x = torch.randn(4, 2, 64, device="cuda")
    pos, inv = torch.ones(4, dtype=torch.int32, device="cuda"), torch.ones(32, device="cuda")
    y = w * x                                          # keeps x for its backward pass
    csa.csa_rotary(x, pos, inv, out=x)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    buf = torch.randn(4, 2, 64, device="cuda")
    y = w * buf
    csa.csa_rotary(x, pos, inv, out=buf)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    with torch.inference_mode():
        z = torch.randn(4, 2, 64, device="cuda")
        assert csa.csa_rotary(z, pos, inv, out=z) is z
