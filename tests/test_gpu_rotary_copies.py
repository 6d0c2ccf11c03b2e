"""csa_rotary: channels outside the rotated range keep every bit, NaN payloads and signs among them, where the
output has the input's type."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim,begin,rot,at", [(128, 64, 32, 0), (128, 32, 64, 1), (30, 4, 22, 0), (512, 448, 64, 0)])
@pytest.mark.parametrize("name", ["bfloat16", "float32"])
def test_copied_channels_keep_their_bits(name, dim, begin, rot, at):
    import torch

    import fp4_kv_cache_csa_b200 as csa

    t = getattr(torch, name)
    word = torch.int16 if t == torch.bfloat16 else torch.int32
    rows, heads = 41, 3
    top = torch.iinfo(word)
    g = torch.Generator("cuda").manual_seed(dim + begin)
    bits = torch.randint(top.min, top.max + 1, (rows * heads * dim + at,), generator=g, device="cuda", dtype=word)
    bits[at:].view(rows, heads, dim)[::2] |= 0x7F80 if t == torch.bfloat16 else 0x7F800000  # Inf and NaNs of all kinds
    x = bits.view(t)[at:].view(rows, heads, dim)
    y = csa.csa_rotary(x, torch.arange(rows, dtype=torch.int32, device="cuda"), torch.ones(rot // 2, device="cuda"),
                       rot_begin=begin)
    for part in (slice(0, begin), slice(begin + rot, dim)):
        assert torch.equal(y.view(word)[..., part], x.view(word)[..., part])
