"""An empty batch whose gate has a row for each of its rows, without a GPU: nothing to do, and no error."""
from __future__ import annotations

import pytest

import dense_linear_algebra_potrf_amd as bl
from tests.test_integer_abi import GRAD, NORM, P, call, lib  # noqa: F401


@pytest.mark.parametrize("gate", [None, P])
def test_no_rows_and_no_gates(lib, gate):  # noqa: F811
    assert call(lib, "block_norm", NORM, dict(rows=0, gates=0, gate=gate))[0] == 0
    none = dict(rows=0, gates=0, gate=gate, dgate=None, dw=None, dpost=None, workspace=None, bytes=0)
    assert call(lib, "block_norm_grad", GRAD, none)[0] == 0


def test_rows_without_gates_are_refused(lib):  # noqa: F811
    for over in (dict(gates=0), dict(rows=0, gates=-1)):
        st, text = call(lib, "block_norm", NORM, over)
        assert st == 1 and "gates must be >=" in text


def test_binding_takes_an_empty_gate():
    import torch
    from dense_linear_algebra_potrf_amd.integer import _gate
    gate = torch.zeros(4, 8)
    assert _gate(gate[:0], 0, 8, torch.float32)[1] == 0
    assert _gate(torch.zeros(0, 1, 8), 0, 8, torch.float32)[1] == 0
    assert _gate(gate[:2], 0, 8, torch.float32)[1] == 2
    for rows, n in ((4, 8), (0, 9)):
        with pytest.raises(ValueError, match="gate must have"):
            _gate(gate[:0], rows, n, torch.float32)


@pytest.mark.gpu
@pytest.mark.parametrize("t", ["float32", "float16", "bfloat16"])
def test_empty_batches_with_a_gate_for_each_row(t):
    import torch
    from tests._gpu import announce
    announce("integer layer: empty batch with token gates", t)
    n = 100
    x = torch.randn(4, n, device="cuda", dtype=getattr(torch, t))
    w = torch.ones(n, device="cuda", dtype=x.dtype)
    for e in (x[:0], x.view(4, 1, n)[:0]):
        v, s, h = bl.block_norm(e, e, w, w, e)
        assert v.shape == h.shape == e.shape and s is None
        v, s, h = bl.block_norm(e, e, w, w, e, int8=True)
        assert v.shape == e.shape and s.shape == (0,)
        dy, dx, dgate, dw, dp = bl.block_norm_grad(e, e, e, w, w, e)
        assert dy.shape == dx.shape == dgate.shape == e.shape
        assert dw.shape == dp.shape == (n,) and not dw.any() and not dp.any()
        assert bl.block_norm_grad(e, e, e, w, w, e, dgate=torch.empty_like(e, dtype=torch.float32))[2].shape == e.shape
