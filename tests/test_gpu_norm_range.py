"""The norms and their gradients where a row and eps, or the two rows of a block's norms, are of
very different magnitude: against the definitions in 64 bits, within the bounds that
tests/_integer_ref.py derives."""
from __future__ import annotations

import numpy as np
import pytest

from tests import _integer_ref as ref
from tests._gpu import announce
from tests.test_gpu_integer import NAMES, close, dtype, f64s, grad_inputs, norm_inputs, rand

pytestmark = pytest.mark.gpu

WIDTHS = [60, 700, 1500, 5000, 16000]        # every way in which the gradient holds a row


def check_rows(got, inputs, eps):
    """Every output against the definition; dweight, dpost_weight and dgate are sums over the rows."""
    with np.errstate(all="ignore"):
        want = ref.block_norm_grad(*f64s(*inputs), 1.0, eps)
    for name, t in zip(NAMES, got):
        assert (t is None) == (name not in want)
        if t is not None:
            assert np.isfinite(want[name][0]).all(), f"{name}: the case itself is not finite"
            close(t, *want[name], name)


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("n", WIDTHS)
@pytest.mark.parametrize("post", [True, False])
def test_gradient_of_a_small_row_beside_a_large_one(t, n, post):
    """eps = 1e-6, and of the two rows that a token's gradient reads one is zero, tiny or ordinary and the other
    ordinary or so large that its products with the gradients are taken of a scaled row."""
    import dense_linear_algebra_potrf_amd as bl
    announce("block_norm_grad, rows apart", t, n, post)
    of_h = [1e8, 0.0, 1.0, 1e-30, 1e8, 1e-30, 1e9, 0.0]
    of_y = [0.0, 1e8, 1e-30, 1.0, 1e-30, 1e8, 1.0, 1.0]
    dv, y, h, w, p, g, dh = grad_inputs(21, dtype(t), len(of_h), n, post, 2, True)
    for row, (a, b) in enumerate(zip(of_h, of_y)):
        h[row] *= a
        y[row] *= b
    for part in (dh, None):
        inputs = (dv, y, h, w, p, g, part)
        check_rows(bl.block_norm_grad(*inputs, eps=1e-6), inputs, 1e-6)


@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n", WIDTHS)
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("eps", [1e-16, 1e-20])
def test_gradient_of_rows_of_zeros_under_a_small_eps(t, n, post, eps):
    """Rows of zeros, or smaller than sqrt(eps) or about it, whose inverse root is that of eps."""
    import dense_linear_algebra_potrf_amd as bl
    announce("block_norm_grad, small eps", t, n, post, eps)
    # 1 / sqrt(eps) is 1e8 or 1e10: in half precision the gradients are small, so that dx and dy stay in range
    small = 1e-6 if t == "f16" else 1.0
    of_h = [0.0, 0.0, 1.0, 1e-30, 1.0, 1e-9]
    of_y = [0.0, 1.0, 0.0, 1.0, 1e-30, 1e-9]
    dv, y, h, w, p, g, dh = grad_inputs(22, dtype(t), len(of_h), n, post, 2, True)
    for row, (a, b) in enumerate(zip(of_h, of_y)):
        h[row] *= a
        y[row] *= b
    if not post:
        y *= small                                     # dgate sums a y, and a is about 1 / sqrt(eps)
    inputs = (dv * small, y, h, w, p, g * small if post else g, dh * small)
    check_rows(bl.block_norm_grad(*inputs, eps=eps), inputs, eps)


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("n", [60, 700, 5000, 16000])
def test_eps_beyond_the_range_of_squares(t, n):
    """eps = 1e30: ordinary, tiny and empty rows are divided by its root."""
    import torch
    import dense_linear_algebra_potrf_amd as bl
    announce("norms, large eps", t, n)
    eps = 1e30
    y, x, w, p, g = norm_inputs(23, dtype(t), 6, n, True, 2)
    x[1] *= 1e-5
    x[2] = 0
    y[3] = 0
    y[4] = x[4] = 0
    for post in (p, None):
        v, _, h = bl.block_norm(y, x, w, post, g, eps=eps)
        wh, wv, eh, ev = ref.block_norm(*f64s(y, x, w, post, g), 1.0, eps)
        close(h, wh, eh, "h")
        close(v, wv, ev, "v")
        assert bool(v[[0, 1, 3]].any(1).all()) and not v[4].any()
    # the norm to 8 bits: its row scales are those of v = w x / sqrt(mean(x^2) + eps)
    s = bl.rmsnorm_quant(x, w, scale="row", eps=eps)[1]
    top = np.abs(ref.block_norm(*f64s(torch.zeros_like(x), x, w), None, None, 1.0, eps)[1]).max(1)
    assert (np.abs(ref.f64(s) - np.maximum(top / 448, 2.0 ** -126)) <= 32 * ref.U * ref.f64(s)).all()
    # gradients, scaled so that what is left of them after the division is an ordinary number
    dv = (rand(24, 6, n) * 1e15).to(dtype(t)).cuda()
    for post in (p, None):
        inputs = (dv, y, x, w, post, g, None)
        check_rows(bl.block_norm_grad(*inputs, eps=eps), inputs, eps)
    dx, dw = bl.rmsnorm_grad(dv, x, w, eps=eps)
    want = ref.block_norm_grad(*f64s(dv, y, x, w), None, None, None, 1.0, eps)
    close(dx, *want["dx"], "dx")
    close(dw, *want["dweight"], "dweight")


@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n", [60, 700, 5000, 16000])
def test_a_row_of_zeros_without_eps_has_no_root(t, n):
    """eps = 0: a row of zeros is 0 / 0, as in the definition, and stays in its row (and in the sums over rows)."""
    import torch
    import dense_linear_algebra_potrf_amd as bl
    announce("norms, rows of zeros without eps", t, n)
    y, x, w, p, g = norm_inputs(25, dtype(t), 4, n, True, 0)
    x[1] = y[1] = 0                                # both norms of it
    y[2] = 0                                       # the first alone, where there is one
    for post in (p, None):
        lost = [1, 2] if post is not None else [1]
        kept = [i for i in range(4) if i not in lost]
        v, _, h = bl.block_norm(y, x, w, post, eps=0.0)
        q, s, h8 = bl.block_norm(y, x, w, post, eps=0.0, int8=True)
        assert torch.equal(torch.nan_to_num(h), torch.nan_to_num(h8))
        assert bool(v[lost].isnan().all()) and bool(s[lost].isnan().all()) and not q[lost].any()
        assert bool(h[1].isnan().all()) if post is not None else not h[1].any()
        assert bool(v[kept].isfinite().all()) and bool(s[kept].isfinite().all()) and bool(h[kept].isfinite().all())
        dy, dx, _, dw, dp = bl.block_norm_grad(x, y, x, w, post, eps=0.0)
        assert bool(dx[1].isnan().all()) and bool(dw.isnan().all()) and bool(dx[[0, 2, 3]].isfinite().all())
        assert bool(dy[lost].isnan().all()) and bool(dy[kept].isfinite().all())
        assert dp is None or bool(dp.isnan().all())


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("n", WIDTHS)
def test_gradient_where_means_cancel(t, n):
    """Without a residual h is g p y t itself, so that the gradient that comes through its norm has no part along
    y, and the sums from which that mean is put together cancel; and dv along h, of which the norm leaves nothing."""
    import torch
    import dense_linear_algebra_potrf_amd as bl
    announce("block_norm_grad, means that cancel", t, n)
    dv, y, x, w, p, g, _ = grad_inputs(26, dtype(t), 6, n, True, 2, False)
    y[3:] = y[3:].abs() + 1                            # sums that do not average out either
    h = bl.block_norm(y, x, w, p, g, residual_scale=0.0)[2]
    along = (h.float() / w.float()).to(dtype(t))
    for grad in (dv, along, along * 100):
        for part in (None, 1e-3 * grad):
            inputs = (grad, y, h, w, p, g, part)
            with np.errstate(all="ignore"):
                want = ref.block_norm_grad(*f64s(*inputs), 0.0, 1e-6)
            got = bl.block_norm_grad(*inputs, residual_scale=0.0)
            for name, out in zip(NAMES, got):
                close(out, *want[name], name)
            assert not got[1].any()


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("n", WIDTHS)
def test_large_gradients_of_rows_that_go_together(t, n):
    """Rows of 1e7, just within the range that is summed as it is, whose sums do not average out, under gradients of
    1e25: each sum of products stays in 32 bits, and so do the results."""
    import dense_linear_algebra_potrf_amd as bl
    announce("block_norm_grad, large gradients", t, n)
    dv, y, h, w, p, g, dh = grad_inputs(27, dtype(t), 6, n, True, 2, True)
    dv, y, h, dh = (dv.abs() + 0.5) * 1e25, (y.abs() + 0.5) * 5e6, (h.abs() + 0.5) * 3e6, dh * 1e18
    inputs = (dv, y, h, w.abs(), p.abs(), g.abs(), dh)
    check_rows(bl.block_norm_grad(*inputs, eps=1e-6), inputs, 1e-6)
