"""The 8-bit-integer layer at the widths where its kernels change shape, one column less and one more: every output
against its definition, in a wider array whose other elements stay as they were, and a workspace of no more than is asked for."""
from __future__ import annotations

import numpy as np
import pytest

from tests import _integer_ref as ref
from tests._gpu import announce
from tests.test_gpu_integer import TYPES, check_grad, check_norm, codes, dtype, grad_inputs, norm_inputs, rand

pytestmark = pytest.mark.gpu

WIDTHS = sorted({e + d for e in (8, 128, 256, 512, 1024, 2048, 4096, 6144, 8192, 12288, 16384) for d in (-1, 0, 1)} - {16385})


class Within:
    """A rows x n array of one value inside a larger one, at an odd offset, its rows further apart."""

    def __init__(self, rows, n, t, fill=7.0, step=1, ahead=3):
        import torch
        self.ld = -(-(n + 5) // step) * step
        self.buffer = torch.full((ahead * step + rows * self.ld + 64,), fill, dtype=t, device="cuda")
        self.view = self.buffer[ahead * step:ahead * step + rows * self.ld].view(rows, self.ld)[:, :n]
        self.fill, self.shape, self.at = fill, (rows, n), ahead * step

    def rest_untouched(self):
        import torch
        seen = torch.ones_like(self.buffer, dtype=torch.bool)
        rows, n = self.shape
        seen[self.at:self.at + rows * self.ld].view(rows, self.ld)[:, :n] = False
        return bool((self.buffer[seen] == self.fill).all())


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("n", WIDTHS)
def test_norms_at_the_widths_where_shapes_change(t, n):
    import torch
    import dense_linear_algebra_potrf_amd as bl
    announce("integer layer: widths", t, n)
    T, rows = dtype(t), 5 if n > 300 else 37
    for post, gates in ((True, rows), (False, 1)):
        y, x, w, p, g = norm_inputs(n, T, rows, n, post, gates)
        for int8 in (False, True):
            h, v = Within(rows, n, T), Within(rows, n, torch.int8, 0x55, 16) if int8 else Within(rows, n, T)
            s = Within(1, rows, torch.float32)
            _, scales, _ = bl.block_norm(y, x, w, p, g, eps=1e-5, int8=int8, out=v.view, residual_out=h.view,
                                         scales=s.view[0] if int8 else None)
            check_norm(y, x, w, p, g, 1.0, 1e-5, int8, h.view, v.view, scales)
            assert h.rest_untouched() and v.rest_untouched() and s.rest_untouched()
        inputs = grad_inputs(n, T, rows, n, post, gates, post)
        outs = {"dy": Within(rows, n, T), "dx": Within(rows, n, T), "dgate": Within(gates, n, T if post else torch.float32)}
        sums = {name: Within(1, n, torch.float32) for name in ("dweight", "dpost_weight")[:2 if post else 1]}
        need = bl.block_norm_grad_workspace(T, rows, n, gates)
        work = Within(1, need, torch.uint8, 0x55, 16)
        got = bl.block_norm_grad(*inputs, eps=1e-5, workspace=work.view[0], **{k: o.view for k, o in outs.items()},
                                 **{k: o.view[0] for k, o in sums.items()})
        check_grad(inputs, 1.0, 1e-5, got)
        assert all(o.rest_untouched() for o in (*outs.values(), *sums.values(), work))


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("n", WIDTHS + [32767, 32768, 32769])
def test_rounding_at_the_widths_where_shapes_change(t, n):
    import torch
    import dense_linear_algebra_potrf_amd as bl
    announce("int8_quant: widths", t, n)
    T, rows = dtype(t), 5 if n > 300 else 37
    x = rand(n, rows, n).to(T)
    wide = Within(rows, n, T, float("nan"))               # what is beside a row is not read as part of it
    wide.view.copy_(x)
    own = None
    for given in (False, True):
        q, s, v = Within(rows, n, torch.int8, 0x55, 16), Within(1, rows, torch.float32), Within(rows, n, T)
        bl.int8_quant(wide.view, out=q.view, values=v.view, **({"given": own} if given else {"scales": s.view[0]}))
        wq, ws = ref.quant(x.float().numpy())
        if not given:
            own = s.view[0].clone()
            assert np.array_equal(own.cpu().numpy(), ws)
        assert np.array_equal(q.view.cpu().numpy(), wq)
        assert torch.equal(v.view.cpu(), torch.from_numpy(wq.astype(np.float32) * ws[:, None]).to(T))
        assert q.rest_untouched() and s.rest_untouched() and v.rest_untouched()


@pytest.mark.parametrize("t", TYPES)
def test_products_beside_other_elements(t):
    import torch
    import dense_linear_algebra_potrf_amd as bl
    announce("int8_matmul within larger arrays", t)
    T = dtype(t)
    for m, n, k in ((1, 17, 129), (16, 33, 128), (17, 65, 127), (64, 31, 384), (65, 129, 500), (129, 257, 64), (257, 513, 1000),
                    (513, 255, 130), (1025, 1030, 70), (3000, 3100, 40)):
        x, w = codes(m, m, k), codes(n + 1, n, k)
        xs, ws = 0.01 * torch.exp(rand(m, m)).cuda(), 0.01 * torch.exp(rand(n, n)).cuda()
        y = Within(m, n, T)
        bl.int8_matmul(x, w, xs, ws, out=y.view)
        want = ref.product(x.cpu().numpy(), w.cpu().numpy()) * ref.f64(xs)[:, None] * ref.f64(ws)
        off = (3.001 * ref.U + ref.half_step(T) * 1.001) * np.abs(want) + ref.smallest(T)
        assert (np.abs(ref.f64(y.view) - want) <= off).all(), (m, n, k)
        assert y.rest_untouched(), (m, n, k)
