"""Codes that weight_quant allocates are the same bytes on every run, padding and all."""
from __future__ import annotations

import pytest

from tests._gpu import announce

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("k", [1, 33, 500, 1000, 1023, 1024])
def test_padding_of_new_codes_is_zero(k):
    import torch
    import dense_linear_algebra_potrf_amd as bl
    announce("weight_quant padding", k)
    W = torch.randn(200, k, generator=torch.Generator().manual_seed(k)).cuda()
    held = []
    for fill in (0x00, 0xFF):
        garbage = [torch.full((1 << e,), fill, dtype=torch.uint8, device="cuda") for e in range(6, 22) for _ in range(8)]
        torch.cuda.synchronize()
        del garbage
        held.append(bl.weight_quant(W, group=32)[0])
    assert torch.equal(held[0], held[1])
    assert held[0].shape[1] % 16 == 0 and not held[0][:, (k + 1) // 2:].any()
