"""csa_rotary and tensors that autograd follows (no GPU needed): the call records no gradient, so it refuses inputs
that ask for one instead of returning a detached result."""
import pytest
import torch

import fp4_kv_cache_csa_b200 as csa


@pytest.fixture(autouse=True)
def no_launch(monkeypatch):
    from fp4_kv_cache_csa_b200 import build as csa_build

    csa_build.build()
    # a passing call ends where it would take the device's stream
    monkeypatch.setattr(csa, "_on", lambda device, stream, call: "launched")


def test_inputs_that_require_a_gradient_are_refused():
    x, pos, inv = torch.zeros(3, 2, 8), torch.zeros(3, dtype=torch.int32), torch.ones(4)
    asks = x.clone().requires_grad_()
    for a, f, kw in ((asks, inv, {}), (asks * 2, inv, {}), (x, inv.clone().requires_grad_(), {}),
                     (x, inv, dict(out=asks * 2)), (asks.bfloat16(), inv, {})):
        with pytest.raises(csa.CsaError, match="inverse"):
            csa.csa_rotary(a, pos, f, **kw)
    y = asks * 2
    with pytest.raises(csa.CsaError, match="inverse"):
        csa.csa_rotary(y, pos, inv, out=y)
    with torch.no_grad():
        assert csa.csa_rotary(asks, pos, inv) == "launched"
    assert csa.csa_rotary(asks.detach(), pos, inv) == "launched"
    assert csa.csa_rotary(x, pos, inv) == "launched"
