"""int8_quant's values are a float of x (and of given scales): their gradient or tangent is not lost silently."""
from __future__ import annotations

import pytest
import torch
from torch.autograd import forward_ad

import dense_linear_algebra_potrf_amd as bl


def args():
    return dict(x=torch.zeros(2, 32), given=torch.ones(2))


@pytest.mark.parametrize("name", ["x", "given"])
@pytest.mark.parametrize("values", [True, torch.zeros(2, 32)])
def test_values_refuse_to_lose_a_gradient(name, values):
    a = args()
    a[name].requires_grad_(True)
    with pytest.raises(ValueError, match="gradient would be lost"):
        bl.int8_quant(**a, values=values)
    with torch.no_grad(), pytest.raises(ValueError, match="GPU"):      # accepted as far as that goes
        bl.int8_quant(**a, values=values)
    with pytest.raises(ValueError, match="GPU"):
        bl.int8_quant(**{k: v.detach() for k, v in a.items()}, values=values)


@pytest.mark.parametrize("name", ["x", "given"])
def test_values_refuse_to_lose_a_tangent(name):
    a = args()
    with forward_ad.dual_level():
        a[name] = forward_ad.make_dual(a[name], torch.ones_like(a[name]))
        with pytest.raises(ValueError, match="tangent would be lost"):
            bl.int8_quant(**a, values=True)


def test_codes_alone_have_none():
    with pytest.raises(ValueError, match="GPU"):
        bl.int8_quant(torch.nn.Parameter(torch.zeros(2, 32)))


@pytest.mark.gpu
def test_channels_of_a_parameter_are_calibrated():
    from tests._gpu import announce
    announce("calibrate channels of a parameter")
    W = torch.randn(12, 128, generator=torch.Generator().manual_seed(0)).cuda()
    H = bl.second_moments(torch.randn(400, 128, generator=torch.Generator().manual_seed(1)).cuda(), 64)
    want = bl.calibrate_channels(W, H, group=32)
    got = bl.calibrate_channels(torch.nn.Parameter(W), H, group=32)
    assert all(torch.equal(a, b) and not b.requires_grad for a, b in zip(want, got))
