"""Sums over rows whose terms are small integers, so that they are exact in 32 bits in any order and a row
that is left out or counted twice shows; and outputs beyond the largest value of their type."""
from __future__ import annotations

import numpy as np
import pytest

from tests import _integer_ref as ref
from tests._gpu import announce
from tests.test_gpu_integer import TYPES, close, dtype, f64s, grad_inputs, norm_inputs

pytestmark = pytest.mark.gpu


def integers(seed, low, high, *shape):
    import torch
    return torch.randint(low, high + 1, shape, generator=torch.Generator().manual_seed(seed)).float()


def signs(seed, *shape):
    return 2 * integers(seed, 0, 1, *shape) - 1


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("rows,n,gates", [(40000, 24, 8), (40000, 24, 0), (40000, 24, 40000), (9000, 40, 2), (9000, 40, 1),
                                          (9000, 40, 500), (1700, 65, 425), (6000, 130, 4), (2100, 300, 7), (2100, 600, 3),
                                          (2100, 1100, 700), (513, 2000, 1), (600, 2000, 2), (2060, 4100, 2), (2060, 4100, 1030),
                                          (1100, 9000, 2), (1100, 9000, 0), (777, 9000, 777)])
@pytest.mark.parametrize("post", [True, False])
def test_sums_over_rows_are_exact(t, rows, n, gates, post):
    """Rows of ones and minus ones have a root of one under eps = 0.  dv h sums to zero over each row, so that with
    w = 1 the norm's gradient is a = dv + dh, at most 16; with the gate's and post's at most 2, every sum is an
    integer of at most 40000 * 64, below 2^24."""
    import torch
    import dense_linear_algebra_potrf_amd as bl
    announce("block_norm_grad exact sums", t, rows, n, gates, post)
    T, half = dtype(t), n // 2
    h, y = signs(1, rows, n), signs(2, rows, n)
    dv = integers(3, -8, 8, rows, n)
    dv[:, half:2 * half] = -(dv * h)[:, :half] * h[:, half:2 * half]
    dv[:, 2 * half:] = 0
    dh = integers(4, -8, 8, rows, n)
    p = integers(5, 1, 2, n) if post else None
    g = signs(6, gates, n) * integers(7, 1, 2, gates, n) if gates else None
    put = lambda x: None if x is None else x.to(T).cuda()  # noqa: E731
    out = torch.full((gates, n), 7.0, device="cuda") if gates else None
    _, dx, dgate, dweight, dpost = bl.block_norm_grad(put(dv), put(y), put(h), put(torch.ones(n)), put(p), put(g), put(dh), eps=0.0,
                                                      dgate=out)
    a, unit = (dv + dh).double(), y.double()
    assert torch.equal(dx.double().cpu(), a)
    assert torch.equal(dweight.double().cpu(), (dv * h).double().sum(0))
    each = 1.0 if g is None else g.double().repeat_interleave(rows // gates, 0)
    if post:
        assert torch.equal(dpost.double().cpu(), (a * each * unit).sum(0))
    if gates:
        d = a * unit if p is None else a * unit * p.double()
        assert torch.equal(dgate.double().cpu(), d.view(gates, -1, n).sum(1))


def beyond(got, want, off, what):
    """Infinite with the definition's sign where that is past the type's largest value by more than the error allowed."""
    import torch
    top = torch.finfo(got.dtype).max
    g = ref.f64(got)
    with np.errstate(invalid="ignore"):
        over = np.abs(want) * (1 - 2 * ref.half_step(got.dtype)) - off > top
    assert over.any(), f"{what}: nothing to see"
    assert (g[over] == np.sign(want[over]) * np.inf).all(), what
    close(got, want, off, what)


@pytest.mark.parametrize("n", [60, 700, 5000, 16000])
@pytest.mark.parametrize("post", [True, False])
def test_half_precision_overflows_to_infinity(n, post):
    import torch
    import dense_linear_algebra_potrf_amd as bl
    announce("norms beyond half precision", n, post)
    y, x, w, p, g = norm_inputs(31, torch.float16, 6, n, post, 3)
    x[1] = x[1].clamp(-4, 4) * 15000
    w[::3] *= 40000
    with np.errstate(all="ignore"):
        wh, wv, eh, ev = ref.block_norm(*f64s(y, x, w, p, g), 2.0, 1e-6)
    v, _, h = bl.block_norm(y, x, w, p, g, residual_scale=2.0)
    beyond(h, wh, eh, "h")
    beyond(v, wv, ev, "v")
    q, s, h8 = bl.block_norm(y, x, w, p, g, residual_scale=2.0, int8=True)      # codes: v in 32 bits
    assert torch.equal(h, h8)
    if bool(w.isfinite().all()):
        assert bool(s.isfinite().all()) and bool((q.abs().amax(1) == 127).all())
    else:                                                                       # of many weights some are infinite themselves
        assert bool(s.isnan().all()) and not q.any()
    dv, y, h, w, p, g, dh = inputs = grad_inputs(32, torch.float16, 6, n, post, 3, True)
    h[1] *= 2.0 ** -8
    dv[1] *= 1000
    y[1] *= 100
    want = ref.block_norm_grad(*f64s(*inputs), 1.0, 1e-6)
    dy, dx, dgate, dweight, dpost = bl.block_norm_grad(*inputs)
    beyond(dx, *want["dx"], "dx")
    if not post:                                                                # a y; with post y's root takes its size back
        beyond(dgate, *want["dgate"], "dgate")
    close(dweight, *want["dweight"], "dweight")
    close(dy, *want["dy"], "dy")


@pytest.mark.parametrize("m", [3, 70, 300])
@pytest.mark.parametrize("t", TYPES)
def test_products_overflow_to_infinity(t, m):
    import torch
    import dense_linear_algebra_potrf_amd as bl
    announce("int8_matmul beyond the type", t, m)
    k, n = 500, 90
    x, w = (integers(i, -127, 127, r, 512).to(torch.int8).cuda()[:, :k] for i, r in ((41, m), (42, n)))
    xs, ws = torch.full((m,), 1.0, device="cuda"), torch.full((n,), float(torch.finfo(dtype(t)).max) / 3e5, device="cuda")
    y = bl.int8_matmul(x, w, xs, ws, out_dtype=dtype(t))
    want = ref.product(x.cpu().numpy(), w.cpu().numpy()) * ref.f64(ws)
    beyond(y, want, 3.001 * ref.U * np.abs(want), "y")
