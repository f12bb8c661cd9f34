"""Outputs of the norms around a block that are one and the same array are refused: each would be lost in the other."""
from __future__ import annotations

import pytest

import dense_linear_algebra_potrf_amd as bl
from tests.test_integer_abi import GRAD, NORM, P, call, lib  # noqa: F401


def test_one_array_for_two_outputs(lib):  # noqa: F811
    st, text = call(lib, "block_norm", NORM, dict(h=2 * P, v=2 * P))
    assert st == 1 and "h and v must be different" in text
    st, text = call(lib, "block_norm_grad", GRAD, dict(dy=2 * P, dx=2 * P))
    assert st == 1 and "dy and dx must be different" in text


@pytest.mark.gpu
def test_binding_refuses_one_tensor_for_two_outputs():
    import torch
    from tests._gpu import announce
    announce("block_norm: one tensor for two outputs")
    x, w = torch.randn(4, 64, device="cuda"), torch.ones(64, device="cuda")
    out = torch.empty_like(x)
    with pytest.raises(bl.BatchlasError, match="h and v"):
        bl.block_norm(x, x, w, out=out, residual_out=out)
    for both in (out, x):
        with pytest.raises(bl.BatchlasError, match="dy and dx"):
            bl.block_norm_grad(x, x, x, w, dy=both, dx=both)
    assert bl.block_norm(x[:0], x[:0], w, out=out[:0], residual_out=out[:0])[0].shape == (0, 64)
