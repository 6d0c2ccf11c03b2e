"""Caches that csa_cache_copy and hca_shared_attend refuse: planes that the kernels would not find where the sizes say,
and counts of another type or device (no GPU needed)."""
import dataclasses

import pytest
import torch

import fp4_kv_cache_csa_b200 as csa


def cache(**kw):
    return dataclasses.replace(csa.Cache.allocate(2, 8, 128, 4, 64, csa.CSA_IDX_E4M3, device="cpu"), **kw)


BAD = {
    "counts of 64 bits": dict(n_blocks=torch.zeros(2, dtype=torch.int64)),
    "too few counts": dict(n_blocks=torch.zeros(1, dtype=torch.int32)),
    "every other count": dict(n_blocks=torch.zeros(4, dtype=torch.int32)[::2]),
    "a slice of larger planes": dict(fp4=torch.zeros(2, 16, 64, dtype=torch.uint8)[:, :8]),
    "scales of a slice": dict(scale=torch.zeros(2, 16, 4, dtype=torch.uint8)[:, :8]),
    "keys of a slice": dict(idx_key=torch.zeros(2, 16, 64, dtype=torch.uint8)[:, :8]),
    "scales of another format": dict(scale_fmt=csa.CSA_SCALE_E4M3_16),
    "scales for fewer blocks": dict(scale=torch.zeros(2, 7, 4, dtype=torch.uint8)),
}


@pytest.mark.parametrize("name", list(BAD))
def test_refusals(name):
    good, bad = cache(), cache(**BAD[name])
    slots = torch.zeros(1, dtype=torch.int32)
    q, offs = torch.zeros(3, 4, 128, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    for call in (lambda: csa.csa_cache_copy(bad, good, slots, slots), lambda: csa.csa_cache_copy(good, bad, slots, slots),
                 lambda: csa.csa_cache_copy(bad, bad, slots, slots), lambda: csa.hca_shared_attend(bad, q, offs)):
        with pytest.raises(csa.CsaError, match="planes"):
            call()


def test_counts_on_another_device():
    # a stand-in for a tensor of a GPU: only its device's number is asked for before the refusal
    class Elsewhere:
        def get_device(self):
            return 0

    with pytest.raises(csa.CsaError, match="planes"):
        csa.csa_cache_copy(cache(n_blocks=Elsewhere()), cache(), torch.zeros(1, dtype=torch.int32),
                           torch.zeros(1, dtype=torch.int32))


def test_others_pass_these_checks():
    slots = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(csa.CsaError, match="CUDA device"):
        csa.csa_cache_copy(cache(), cache(status=None), slots, slots)
    with pytest.raises(csa.CsaError, match="CUDA device"):  # the counts' first ones of a longer tensor
        csa.csa_cache_copy(cache(n_blocks=torch.zeros(5, dtype=torch.int32)), cache(), slots, slots)
