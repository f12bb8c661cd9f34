"""The 8-bit-integer layer operators without a GPU: refusals in the documented
order before anything touches the GPU, the empty calls, the workspace query, the
binding's own checks, and the 64-bit formulas that the GPU tests compare against
(the gradient against differences)."""
from __future__ import annotations

import ctypes
import os

import numpy as np
import pytest

import dense_linear_algebra_potrf_amd as bl
from dense_linear_algebra_potrf_amd import build as blbuild
from tests import _integer_ref as ref


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(bl.LIB_PATH):
        blbuild.build(incremental=True, verbose=False)
    return bl.load_library()


P = 0x1000     # never dereferenced: validation fails first


def call(lib, name, defaults, over):
    a = dict(defaults, **over)
    st = getattr(lib, "batchlas_" + name)(*a.values())
    return st, lib.batchlas_last_error().decode()


QUANT = dict(type=2, rows=4, n=60, x=P, ldx=60, given=None, q=P, ldq=64, scales=P, values=P, ldv=60, stream=None)


@pytest.mark.parametrize("over,status,msg", [
    (dict(type=3), 1, "type must be"), (dict(rows=-1), 1, "rows must be"), (dict(n=0), 1, "n must be"),
    (dict(rows=1 << 31), 1, "out of range"), (dict(ldx=59), 1, "ldx must be"), (dict(ldq=48), 1, "ldq must be >="),
    (dict(ldq=72), 1, "multiple of 16"), (dict(ldv=59), 1, "ldv must be"), (dict(ldx=1 << 60), 1, "overflows"),
    (dict(given=P), 1, "either given or computed"), (dict(x=None), 2, "x is NULL"), (dict(q=None), 2, "q is NULL"),
    (dict(scales=None), 2, "scales is NULL"), (dict(q=P + 8), 1, "aligned to 16"), (dict(x=P + 1), 1, "not aligned"),
    (dict(scales=P + 2), 1, "not aligned"), (dict(type=9, n=0, x=None), 1, "type must be"),
    (dict(rows=0, x=None, q=None, scales=None, values=None), 0, ""),
])
def test_integer_quant_refusals(lib, over, status, msg):
    st, text = call(lib, "integer_quant", QUANT, over)
    assert st == status
    assert msg in text


MATMUL = dict(ytype=2, m=3, n=5, k=100, x=P, ldx=112, xs=P, w=P, ldw=112, ws=P, y=P, ldy=5, stream=None)


@pytest.mark.parametrize("over,status,msg", [
    (dict(ytype=3), 1, "ytype must be"), (dict(m=-1), 1, "m must be"), (dict(n=0), 1, "n must be"),
    (dict(k=0), 1, "k must be"), (dict(n=1 << 31), 1, "out of range"), (dict(ldx=96), 1, "ldx must be >="),
    (dict(ldw=96), 1, "ldw must be >="), (dict(ldx=104), 1, "multiples of 16"), (dict(ldw=104), 1, "multiples of 16"),
    (dict(ldy=4), 1, "ldy must be"), (dict(ldy=1 << 60), 1, "overflows"), (dict(x=None), 2, "x is NULL"),
    (dict(xs=None), 2, "xscales is NULL"), (dict(w=None), 2, "w is NULL"), (dict(ws=None), 2, "wscales is NULL"),
    (dict(y=None), 2, "y is NULL"), (dict(x=P + 8), 1, "aligned to 16"), (dict(w=P + 4), 1, "aligned to 16"),
    (dict(y=P + 1), 1, "not aligned"), (dict(ws=P + 2), 1, "not aligned"),
    (dict(k=1 << 17, ldx=1 << 17, ldw=1 << 17), 3, "2^17"), (dict(n=(1 << 24) + 1, ldy=1 << 25), 3, "beyond 2^24"),
    (dict(m=1 << 20, n=1 << 17, ldy=1 << 17), 3, "beyond 2^36"), (dict(ldw=(1 << 22) + 16), 3, "beyond 2^22"),
    (dict(m=0, x=None, xs=None, w=None, ws=None, y=None), 0, ""),
])
def test_integer_matmul_refusals(lib, over, status, msg):
    st, text = call(lib, "integer_matmul", MATMUL, over)
    assert st == status
    assert msg in text


NORM = dict(type=1, scale=1, rows=6, n=60, y=P, ldy=60, x=P, ldx=60, w=P, post=P, gate=P, gates=2, ldg=60, c=1.0,
            eps=1e-6, h=P, ldh=60, v=P, ldv=64, scales=P, stream=None)


@pytest.mark.parametrize("over,status,msg", [
    (dict(type=3), 1, "type must be"), (dict(scale=2), 1, "scale must be"), (dict(rows=-6), 1, "rows must be"),
    (dict(n=0), 1, "n must be"), (dict(gates=0), 1, "gates must be >="), (dict(gates=4), 1, "gates must divide"),
    (dict(eps=-1.0), 1, "eps must be"), (dict(eps=float("nan")), 1, "eps must be"), (dict(eps=1e39), 1, "eps must be"),
    (dict(c=float("inf")), 1, "residual_scale must be"), (dict(c=1e39), 1, "residual_scale must be"),
    (dict(ldy=59), 1, "ldy must be"), (dict(ldx=59), 1, "ldx must be"), (dict(ldg=59), 1, "ldg must be"),
    (dict(ldh=59), 1, "ldh must be"), (dict(ldv=48), 1, "ldv must be >="), (dict(ldv=60), 1, "multiple of 16"),
    (dict(ldh=1 << 60), 1, "overflows"), (dict(scale=0, ldv=60), 1, "scales are for codes"), (dict(y=None), 2, "y is NULL"),
    (dict(x=None), 2, "x is NULL"), (dict(w=None), 2, "w is NULL"), (dict(h=None), 2, "h is NULL"),
    (dict(v=None), 2, "v is NULL"), (dict(scales=None), 2, "scales is NULL"), (dict(v=P + 8), 1, "aligned to 16"),
    (dict(gate=P + 1), 1, "not aligned"), (dict(post=P + 1), 1, "not aligned"),
    (dict(n=32769, ldy=32769, ldx=32769, ldg=32769, ldh=32769, ldv=32784), 3, "at most"),
    (dict(rows=0, y=None, x=None, w=None, h=None, v=None, scales=None), 0, ""),
])
def test_block_norm_refusals(lib, over, status, msg):
    st, text = call(lib, "block_norm", NORM, over)
    assert st == status
    assert msg in text


GRAD = dict(type=1, rows=600, n=60, dv=P, lddv=60, y=P, ldy=60, h=P, ldh=60, w=P, post=P, gate=P, gates=2, ldg=60, dh=P,
            lddh=60, c=1.0, eps=1e-6, dy=P, lddy=60, dx=P, lddx=60, dgtype=0, dgate=P, lddg=60, dw=P, dpost=P, workspace=P,
            bytes=1 << 30, stream=None)


@pytest.mark.parametrize("over,status,msg", [
    (dict(type=3), 1, "type must be"), (dict(dgtype=2), 1, "dgtype must be"), (dict(rows=-2), 1, "rows must be"),
    (dict(n=0), 1, "n must be"), (dict(gates=-1), 1, "gates must be >="), (dict(gates=7), 1, "gates must divide"),
    (dict(eps=-1.0), 1, "eps must be"), (dict(c=float("nan")), 1, "residual_scale must be"),
    (dict(lddv=59), 1, "lddv must be"), (dict(ldy=59), 1, "ldy must be"), (dict(ldh=59), 1, "ldh must be"),
    (dict(ldg=59), 1, "ldg must be"), (dict(lddh=59), 1, "lddh must be"), (dict(lddy=59), 1, "lddy must be"),
    (dict(lddx=59), 1, "lddx must be"), (dict(lddg=59), 1, "lddg must be"), (dict(lddx=1 << 60), 1, "overflows"),
    (dict(post=None), 1, "dpost needs post"), (dict(gate=None), 1, "dgate needs a gate"), (dict(dv=None), 2, "dv is NULL"),
    (dict(y=None), 2, "y is NULL"), (dict(h=None), 2, "h is NULL"), (dict(w=None), 2, "w is NULL"),
    (dict(dy=None), 2, "dy is NULL"), (dict(dx=None), 2, "dx is NULL"), (dict(dgate=P + 2), 1, "not aligned"),
    (dict(dw=P + 2), 1, "not aligned"), (dict(dv=P + 1), 1, "not aligned"), (dict(workspace=None), 2, "workspace is NULL"),
    (dict(bytes=64), 1, "workspace_bytes"),
    (dict(n=16385, lddv=16385, ldy=16385, ldh=16385, ldg=16385, lddh=16385, lddy=16385, lddx=16385, lddg=16385), 3, "at most"),
    (dict(rows=0, dv=None, y=None, h=None, w=None, dy=None, dx=None, dgate=None, dw=None, dpost=None), 0, ""),
])
def test_block_norm_grad_refusals(lib, over, status, msg):
    st, text = call(lib, "block_norm_grad", GRAD, over)
    assert st == status
    assert msg in text


def test_block_norm_grad_workspace(lib):
    size = ctypes.c_int64(-1)
    ask = lambda *a: lib.batchlas_block_norm_grad_workspace(*a, ctypes.byref(size))  # noqa: E731
    assert ask(2, 0, 100, 0) == 0 and size.value == 0
    assert ask(2, 0, 100, 3) == 0 and size.value == 0
    for rows, n, gates in ((2, 1, 1), (517, 1537, 0), (1 << 20, 4096, 8), (1 << 20, 64, 1 << 20), (3, 16384, 3), (900, 33, 9)):
        assert ask(1, rows, n, gates) == 0
        # whole rows of floats; the sums of a run of rows at most
        assert size.value % (4 * n) == 0 and 0 < size.value <= 2 * 4 * n * max(1, rows)
    assert ask(1, 4, 16385, 0) == 3
    assert ask(3, 4, 64, 0) == 1
    assert ask(1, 4, 64, 3) == 1
    assert lib.batchlas_block_norm_grad_workspace(1, 4, 64, 0, None) == 2


# ---------------------------------------------------------------- the binding, on CPU tensors

def test_binding_refusals():
    import torch
    x, v = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(64, dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="x must be"):
        bl.int8_quant(torch.zeros(4, 64, dtype=torch.int8))
    with pytest.raises(ValueError, match="on the GPU"):
        bl.int8_quant(x)
    with pytest.raises(ValueError, match="on the GPU"):
        bl.int8_matmul(torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4), torch.zeros(4))
    with pytest.raises(ValueError, match="on the GPU"):
        bl.block_norm(x, x, v)
    with pytest.raises(ValueError, match="on the GPU"):
        bl.block_norm_grad(x, x, x, v)


def test_lost_gradients_and_tangents_are_refused():
    import torch
    from torch.autograd import forward_ad
    x, v = torch.zeros(4, 64), torch.zeros(64)
    grad = lambda t: t.clone().requires_grad_()  # noqa: E731
    codes, s = torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4)
    for call in (lambda: bl.block_norm(grad(x), x, v), lambda: bl.block_norm(x, grad(x), v),
                 lambda: bl.block_norm(x, x, grad(v)), lambda: bl.block_norm(x, x, v, grad(v)),
                 lambda: bl.block_norm(x, x, v, v, grad(v)), lambda: bl.int8_matmul(codes, codes, grad(s), s),
                 lambda: bl.int8_matmul(codes, codes, s, grad(s))):
        with pytest.raises(ValueError, match="gradient would be lost"):
            call()
        with torch.no_grad(), pytest.raises(ValueError, match="on the GPU"):
            call()
    with forward_ad.dual_level():
        with pytest.raises(ValueError, match="tangent would be lost"):
            bl.block_norm(x, x, v, gate=forward_ad.make_dual(v, v))
        with pytest.raises(ValueError, match="tangent would be lost"):
            bl.int8_matmul(codes, codes, forward_ad.make_dual(s, s), s)


def test_code_rows_are_whole_16_bytes():
    import torch
    from dense_linear_algebra_potrf_amd.integer import _codes
    held = torch.zeros(6, 48, dtype=torch.int8)
    assert _codes(held[:, :41], "x") == (6, 41, 48)
    assert _codes(held.view(2, 3, 48)[..., :41], "x") == (6, 41, 48)
    assert _codes(held[2, :], "x") == (1, 48, 48)
    assert _codes(held[::2], "x") == (3, 48, 96)
    with pytest.raises(TypeError, match="int8"):
        _codes(held.view(torch.uint8), "x")
    with pytest.raises(ValueError, match="multiples of 16"):
        _codes(torch.zeros(6, 41, dtype=torch.int8), "x")
    with pytest.raises(ValueError, match="multiples of 16"):
        _codes(held[:, 1:33], "x")
    with pytest.raises(ValueError, match="contiguous rows"):
        _codes(held.t(), "x")
    with pytest.raises(ValueError, match="whole 16 bytes"):
        _codes(torch.zeros(5 * 48 + 41, dtype=torch.int8).as_strided((6, 41), (48, 1)), "x")
    with pytest.raises(ValueError, match="one row stride"):
        _codes(torch.zeros(2, 4, 48, dtype=torch.int8)[:, :3, :41], "x")


# ---------------------------------------------------------------- the formulas

def test_quant_reference_takes_even_codes_on_a_half():
    x = np.array([[127, 0.5, 1.5, 2.5, -0.5, -1.5, 126.5, -126.5]], np.float32)
    q, s = ref.quant(x)
    assert s[0] == 1 and q[0].tolist() == [127, 0, 2, 2, 0, -2, 126, -126]


@pytest.mark.parametrize("post,gates,dh", [(True, 1, True), (True, 2, False), (True, 6, True), (False, 3, True),
                                           (False, 0, False), (True, 0, True)])
def test_gradient_reference_against_differences(post, gates, dh):
    """d of sum(dv v + dh h) by central differences: they are off by the third derivative times
    step^2 / 6 and by the rounding of 64 bits over the step, both below 1e-8 of the largest gradient here."""
    rng = np.random.default_rng(3)
    rows, n, eps, c = 6, 10, 1e-3, 0.8
    y, x, dv = (rng.standard_normal((rows, n)) for _ in range(3))
    w, p = 1 + 0.2 * rng.standard_normal(n), 1 + 0.2 * rng.standard_normal(n)
    e = rng.standard_normal((rows, n)) if dh else None
    gate = rng.standard_normal((gates, n)) if gates else None
    inputs = {"dy": y, "dx": x, "dweight": w}
    if post:
        inputs["dpost_weight"] = p
    if gates:
        inputs["dgate"] = gate

    def loss():
        h, v, _, _ = ref.block_norm(y, x, w, p if post else None, gate, c, eps)
        return (dv * v).sum() + (0 if e is None else (e * h).sum())

    h = ref.block_norm(y, x, w, p if post else None, gate, c, eps)[0]
    got = ref.block_norm_grad(dv, y, h, w, p if post else None, gate, e, c, eps)
    assert set(got) == set(inputs)
    for name, t in inputs.items():
        want = np.zeros_like(t)
        for i in np.ndindex(t.shape):
            keep = t[i]
            t[i] = keep + 1e-5
            up = loss()
            t[i] = keep - 1e-5
            want[i] = (up - loss()) / 2e-5
            t[i] = keep
        assert np.abs(got[name][0] - want).max() <= 1e-8 * max(1, np.abs(want).max())
