"""8-bit weights calibrated channel by channel: the sweep over groups against the
same sweep in 64 bits, less output error than plain rounding, the products with
the calibrated weights, and the layer from end to end."""
from __future__ import annotations

import numpy as np
import pytest

from tests import _integer_ref as ref
from tests._gpu import announce

pytestmark = pytest.mark.gpu


def f64(t):
    return t.detach().double().cpu().numpy()


def state(seed, n, k, samples=2000):
    """Inputs whose columns are correlated, and weights."""
    import torch
    g = torch.Generator().manual_seed(seed)
    X = torch.randn(samples, k, generator=g) @ (torch.eye(k) * 0.5 + torch.randn(k, k, generator=g) / k ** 0.5)
    return X.cuda(), torch.randn(n, k, generator=g).cuda()


def test_one_step_leaves_the_least_error():
    """After the first group is rounded, the compensated columns are where the 64-bit least-squares solution puts
    them: within 1e-4 of their change, the parity tolerance of the fp32 solve, and half a step of their own rounding."""
    import dense_linear_algebra_potrf_amd as bl
    announce("calibrate channels one step")
    n, block, group = 24, 64, 32
    X, W = state(0, n, 2 * block)
    H = bl.second_moments(X, block)
    q, scales, values = bl.calibrate_channels(W, H, group=group)
    W64, H64 = f64(W), f64(H)
    step = np.abs(W64).max(1) / 127
    assert (np.abs(f64(scales) - step) <= 2.0 ** -23 * step).all()
    got = f64(values).reshape(n, 2, block)
    first = np.rint(W64.reshape(n, 2, block)[:, :, :group] / f64(scales)[:, None, None])
    assert np.array_equal(f64(q).reshape(n, 2, block)[:, :, :group], first)
    s = f64(scales)[:, None]
    for b in range(2):
        E = W64.reshape(n, 2, block)[:, b, :group] - got[:, b, :group]
        move = E @ np.linalg.solve(H64[b][group:, group:], H64[b][group:, :group]).T
        # a target beyond the channel's largest code saturates there
        target = np.clip(W64.reshape(n, 2, block)[:, b, group:] + move, -127 * s, 127 * s)
        assert (np.abs(got[:, b, group:] - target) <= 0.5 * s * (1 + 2.0 ** -16) + 1e-4 * np.abs(move).max()).all()


@pytest.mark.parametrize("n,k,block,group", [(96, 512, 256, 64), (33, 520, 260, 20), (5, 128, 128, 128), (200, 512, 512, 32)])
@pytest.mark.parametrize("t", ["float32", "bfloat16"])
def test_calibration_lowers_the_output_error(n, k, block, group, t):
    import torch
    import dense_linear_algebra_potrf_amd as bl
    from dense_linear_algebra_potrf_amd.calibrate import output_error
    announce("calibrate channels", n, k, block, group, t)
    X, W = state(1, n, k)
    W = W.to(getattr(torch, t))
    plain = bl.int8_quant(W.float(), values=True)
    tuned = bl.calibrate_channels(W, bl.second_moments(X, block), group=group)
    assert torch.equal(tuned[1], plain[1]) and tuned[0].shape == W.shape
    if block > group:
        assert output_error(W, tuned[2], X) < 0.97 * output_error(W, plain[2], X)
    else:                                                     # nothing is left to take the change up
        assert torch.equal(tuned[0], plain[0])
    # the codes stand for the values, and the products use them
    assert torch.equal(tuned[2], tuned[0].float() * tuned[1][:, None])
    q, s, _ = bl.int8_quant(X[:3].bfloat16())
    y = bl.int8_matmul(q, tuned[0], s, tuned[1], out_dtype=torch.float32)
    want = (f64(q) @ f64(tuned[0]).T) * f64(s)[:, None] * f64(tuned[1])
    assert (np.abs(f64(y) - want) <= 3 * ref.U * np.abs(want)).all()


def test_refuses_what_is_not_positive_definite():
    import torch
    import dense_linear_algebra_potrf_amd as bl
    announce("calibrate channels refusals")
    W = torch.randn(8, 128, device="cuda")
    H = torch.eye(64, device="cuda").repeat(2, 1, 1)
    H[1, 40, 40] = -1
    with pytest.raises(ValueError, match="positive definite"):
        bl.calibrate_channels(W, H, group=32)
    with pytest.raises(ValueError, match="multiple of the group"):
        bl.calibrate_channels(W, torch.eye(32, device="cuda").repeat(4, 1, 1), group=64)


def test_demo_runs_the_integer_layer():
    from dense_linear_algebra_potrf_amd.calibrate import demo
    announce("calibrate demo, integers")
    out = demo(n=128, k=512, samples=1024)
    o = out["int8"]
    assert o["calibrated"] < o["rounded"]
    far = float((o["y"].float() - o["want"]).norm() / o["want"].norm())
    assert far < 2 * o["calibrated"] + 2.0 ** -7
    for name, g in out["block_norm"].items():
        assert bool(g.float().isfinite().all()) and bool(g.any()), name
