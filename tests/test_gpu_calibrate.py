"""The calibrated low-bit layer from end to end: the sweep over groups against
the same sweep in 64 bits, less output error than plain rounding, and the
products with the calibrated weights."""
from __future__ import annotations

import numpy as np
import pytest

from tests import _layer_ref as ref
from tests._gpu import announce

pytestmark = pytest.mark.gpu


def test_one_step_leaves_the_least_error():
    """After the first group is rounded, the compensated columns are where the
    64-bit least-squares solution puts them: within 1e-4 of their change, the
    parity tolerance of the fp32 solve."""
    import torch
    import dense_linear_algebra_potrf_amd as bl
    announce("calibrate one step")
    n, block, group = 24, 64, 32
    g = torch.Generator().manual_seed(0)
    X = torch.randn(500, 2 * block, generator=g) @ (torch.eye(2 * block) + 0.3 * torch.randn(2 * block, 2 * block, generator=g) / 8)
    W = torch.randn(n, 2 * block, generator=g)
    H = bl.second_moments(X.cuda(), block)
    values = bl.calibrate_weights(W.cuda(), H, group=group)[3]
    H64, W64 = ref.f64(H), ref.f64(W)
    first = ref.quant(W.view(n, 2, block)[:, :, :group].reshape(2 * n, group).numpy(), "int4", group, False)[3].reshape(n, 2, group)
    got = ref.f64(values).reshape(n, 2, block)
    assert np.array_equal(got[:, :, :group], first)
    for b in range(2):
        E = W64.reshape(n, 2, block)[:, b, :group] - first[:, b]
        move = E @ np.linalg.solve(H64[b][group:, group:], H64[b][group:, :group]).T
        target = W64.reshape(n, 2, block)[:, b, group:] + move
        scale = np.abs(target).reshape(n, 1, group).max(2) / 7        # the second group's steps
        # half a step of the rounding (of scales that bf16 holds within 2^-9), and the solve's error
        assert (np.abs(got[:, b, group:] - target) <= 0.5 * scale * (1 + 2.0 ** -8) + 7 * 2.0 ** -8 * scale + 1e-4 * np.abs(move).max()).all()


@pytest.mark.parametrize("format,group,zeros", [("int4", 32, True), ("int4", 64, False), ("fp4", 32, False)])
def test_calibration_lowers_the_output_error(format, group, zeros):
    import torch
    import dense_linear_algebra_potrf_amd as bl
    from dense_linear_algebra_potrf_amd.calibrate import output_error
    announce("calibrate", format, group, zeros)
    g = torch.Generator().manual_seed(1)
    k, n = 512, 96
    X = (torch.randn(2000, k, generator=g) @ (torch.eye(k) * 0.5 + torch.randn(k, k, generator=g) / k ** 0.5)).cuda()
    W = torch.randn(n, k, generator=g).cuda()
    plain = bl.weight_quant(W, format=format, group=group, zeros=zeros, values=True)
    tuned = bl.calibrate_weights(W, bl.second_moments(X, 256), format=format, group=group, zeros=zeros)
    assert output_error(W, tuned[3], X) < 0.95 * output_error(W, plain[3], X)
    # the codes stand for the values, and the products use them
    x = X[:3].bfloat16()
    y = bl.weight_matvec(x, *tuned[:3], format=format, group=group, out_dtype=torch.float32)
    want = ref.f64(x) @ ref.f64(tuned[3]).T
    assert np.abs(ref.f64(y) - want).max() <= 2.0 ** -13 * np.abs(ref.f64(x)).sum(1).max() * float(tuned[1].float().max())


def test_refuses_what_is_not_positive_definite():
    import torch
    import dense_linear_algebra_potrf_amd as bl
    announce("calibrate refusals")
    W = torch.randn(8, 128, device="cuda")
    H = torch.eye(64, device="cuda").repeat(2, 1, 1)
    H[1, 40, 40] = -1
    with pytest.raises(ValueError, match="positive definite"):
        bl.calibrate_weights(W, H, group=32)
    with pytest.raises(ValueError, match="multiple of the group"):
        bl.calibrate_weights(W, torch.eye(32, device="cuda").repeat(4, 1, 1), group=64)
    with pytest.raises(ValueError, match="multiple of block"):
        bl.second_moments(W, 96)


def test_demo_runs():
    from dense_linear_algebra_potrf_amd.calibrate import demo
    announce("calibrate demo")
    out = demo(n=128, k=512, samples=1024)
    for format in ("int4", "fp4"):
        o = out[format]
        assert o["calibrated"] < o["rounded"]
        # the tokens' outputs are as far from the unrounded ones as the calibrated weights make them
        far = float((o["y"].float() - o["want"]).norm() / o["want"].norm())
        assert far < 2 * o["calibrated"] + 2.0 ** -7
    assert bool(out["dw"].isfinite().all()) and bool(out["dx"].float().isfinite().all())
