"""The low-bit layer operators on the GPU against their definitions in 64 bits
(tests/_layer_ref.py): every type, odd and unaligned sizes, strided rows,
non-finite and empty inputs, in-place buffers, other streams, graph replay, and
two runs bit for bit.

Tolerances, from the arithmetic (u = 2^-24):
  sums of n squares: each thread adds at most 64 terms in a row, the joins at
    most 14 more, so the sum is within 78 u and 1/sqrt within 40 u plus an ulp or
    two for the root: below NORM = 2^-18 (64 u);
  e4m3: half a step, 2^-4 of the value or half the subnormal step 2^-10, of the
    scale, and NORM for the value that is rounded;
  dx: NORM of the two terms' magnitudes, twice, and half an ulp of the type;
  dw: a sum of `rows` terms in some order: (rows + 64) u of the magnitudes' sum;
  products: sums of k terms.  With integers and bf16 x the codes may be carried
    with an offset of up to 136 + 15, in partial sums of at most 128 terms with
    at most 8 roundings each: 8 * 151 u < PRODUCT = 2^-13 of sum |x| scale; any
    other form stays below it.  The exact tests below allow no error at all.
"""
from __future__ import annotations

import numpy as np
import pytest

from tests import _layer_ref as ref
from tests._gpu import announce

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
NORM, PRODUCT = 2.0 ** -18, 2.0 ** -13
HALF_ULP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
SUBNORMAL = {"f32": 2.0 ** -149, "f16": 2.0 ** -24, "bf16": 2.0 ** -133}


def dtypes():
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def rand(seed, *shape):
    import torch
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed))


def strided(t, pad, offset=0):
    """A GPU copy of t [rows, n] inside a larger buffer of NaN bytes: row stride n + pad, starting at `offset`.
    Returns (view, buffer)."""
    import torch
    rows, n = t.shape
    ld = n + pad
    buf = torch.full(((rows * ld + offset + 64) * t.element_size(),), 0xFF, dtype=torch.uint8, device="cuda").view(t.dtype)
    v = buf[offset:offset + rows * ld].view(rows, ld)[:, :n]
    v.copy_(t)
    return v, buf


def untouched(view, buf) -> bool:
    """Whether the buffer around the view still holds its 0xFF bytes."""
    import torch
    view.fill_(0)
    es = view.element_size()
    raw = buf.view(torch.uint8)
    return int((raw != 0xFF).sum()) == view.numel() * es


# ---------------------------------------------------------------- rmsnorm_quant

def check_norm(x, r, w, eps, scale, q, s, h, dt):
    """x, r, w: CPU tensors of the type; q, s, h: GPU results."""
    import torch
    n = x.shape[1]
    h64 = ref.f64(x) + (0 if r is None else ref.f64(r))
    if r is not None:
        want = (x.float() + r.float()).to(x.dtype)
        assert torch.equal(h.cpu().float().nan_to_num(7e30), want.float().nan_to_num(7e30)), "h"
    v = ref.norm(h64, ref.f64(w), eps)
    qv = ref.f64(q.float())
    sc = ref.f64(s.float())
    if scale == "block":
        top = np.abs(ref.groups(v, 32)).max(2)
        bad = ~np.isfinite(ref.groups(v, 32)).all(2)
        lo, hi = (ref.least_exponent(np.where(bad, 0, top) * f, 448.0) for f in (1 - NORM, 1 + NORM))
        e = np.where(bad, 0, np.log2(np.where(bad, 1, sc)))
        assert ((e >= lo) & (e <= hi))[~bad].all(), "block scales"
        wide = np.repeat(sc, 32, 1)[:, :n]
    else:
        top = np.abs(v).max(1)
        bad = ~np.isfinite(v).all(1)
        want = np.maximum(top / 448, 2.0 ** -126)
        assert (np.abs(sc - want)[~bad] <= (NORM * want)[~bad]).all(), "row scales"
        wide = np.broadcast_to(sc[:, None], v.shape)
    assert np.isnan(sc[bad]).all()
    broken = np.isnan(wide)
    assert np.isnan(qv[broken]).all()
    got = qv * wide
    bound = np.maximum(np.abs(v) * 2.0 ** -4, wide * 2.0 ** -10) + 2 * NORM * np.abs(v)
    off = np.abs(got - v)
    assert (off[~broken] <= bound[~broken]).all(), float(np.nanmax((off / bound)[~broken]))


NORM_SIZES = [(1, 1), (1, 4096), (2, 31), (3, 32), (5, 33), (4, 512), (9, 513), (7, 1024), (6, 1031), (3, 2048), (5, 2049),
              (2, 4103), (3, 8192), (2, 9001), (2, 16384), (1, 16391), (2, 32768)]


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("scale", ["block", "row"])
def test_norm_sizes(dt, scale):
    import torch
    import dense_linear_algebra_potrf_amd as bl
    for i, (rows, n) in enumerate(NORM_SIZES):
        announce("rmsnorm_quant", dt, scale, rows, n)
        ty = dtypes()[dt]
        x, r, w = rand(i, rows, n).to(ty), (3 * rand(i + 50, rows, n)).to(ty), (1 + 0.2 * rand(i + 99, 1, n)[0]).to(ty)
        if rows > 2:
            x[1], r[1] = 0, 0                      # an empty row
        with_r = i % 2 == 0
        q, s, h = bl.rmsnorm_quant(x.cuda(), w.cuda(), r.cuda() if with_r else None, scale=scale)
        assert (h is None) == (not with_r)
        check_norm(x, r if with_r else None, w, 1e-6, scale, q, s, h, dt)
        if rows > 2:
            assert not q[1].float().any()


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("scale", ["block", "row"])
@pytest.mark.parametrize("rows,n,pad,offset", [(5, 200, 3, 1), (3, 1000, 1, 3), (2, 2500, 5, 7), (130, 96, 0, 5)])
def test_norm_strided_rows_and_padding(dt, scale, rows, n, pad, offset):
    import torch
    import dense_linear_algebra_potrf_amd as bl
    announce("rmsnorm_quant strided", dt, scale, rows, n, pad, offset)
    ty = dtypes()[dt]
    x, r, w = rand(1, rows, n).to(ty), rand(2, rows, n).to(ty), rand(3, 1, n)[0].to(ty)
    xv, _ = strided(x, pad, offset)
    rv, _ = strided(r, pad + 2, offset)
    wbuf = torch.full((n + 3,), float("nan"), dtype=ty, device="cuda")
    wbuf[1:n + 1] = w.cuda()
    hv, hb = strided(torch.zeros(rows, n, dtype=ty), pad + 1, offset + 1)
    qv, qb = strided(torch.zeros(rows, n, dtype=torch.uint8), pad + 4, offset)
    qv, qb = qv.view(torch.float8_e4m3fn), qb
    out_s = sb = None
    if scale == "block":
        sv, sb = strided(torch.zeros(rows, -(-n // 32), dtype=torch.uint8), 3, 1)
        out_s = sv.view(torch.float8_e8m0fnu)
    q, s, h = bl.rmsnorm_quant(xv, wbuf[1:n + 1], rv, scale=scale, out=qv, scales=out_s, residual_out=hv)
    assert q is qv and h is hv
    check_norm(x, r, w, 1e-6, scale, q, s, h, dt)
    assert untouched(hv, hb) and untouched(qv.view(torch.uint8), qb)
    assert scale == "row" or untouched(out_s.view(torch.uint8), sb)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("into", ["x", "residual"])
def test_norm_in_place(dt, into):
    import dense_linear_algebra_potrf_amd as bl
    for rows, n in ((3, 4096), (4, 333), (2, 20000)):
        announce("rmsnorm_quant in place", dt, into, rows, n)
        ty = dtypes()[dt]
        x, r, w = rand(4, rows, n).to(ty), rand(5, rows, n).to(ty), rand(6, 1, n)[0].to(ty)
        xc, rc = x.cuda(), r.cuda()
        q, s, h = bl.rmsnorm_quant(xc, w.cuda(), rc, residual_out=xc if into == "x" else rc)
        check_norm(x, r, w, 1e-6, "block", q, s, h, dt)


@pytest.mark.parametrize("scale", ["block", "row"])
def test_norm_values_that_are_not_finite_and_extremes(scale):
    import dense_linear_algebra_potrf_amd as bl
    announce("rmsnorm_quant extremes", scale)
    ty = dtypes()["f32"]
    x = rand(7, 10, 100)
    x[0, 5] = float("nan")
    x[1, 40] = float("inf")
    x[2] = 0
    x[3] = 1e-30
    x[4] *= 1e15
    x[5, 3] = 3e9
    x[6] *= 1e-19
    w = rand(8, 1, 100)[0]
    w[99] = 1e38                     # a large and a tiny weight in the last, short block
    w[98] = 1e-38
    q, s, _ = bl.rmsnorm_quant(x.cuda(), w.cuda(), scale=scale)
    check_norm(x, None, w, 1e-6, scale, q, s, None, "f32")
    # eps = 0: an empty row is 0 / 0
    q, s, _ = bl.rmsnorm_quant(x.cuda(), w.cuda(), scale=scale, eps=0.0)
    check_norm(x, None, w, 0.0, scale, q, s, None, "f32")
    # weights that are not finite break their own block (row) in every row
    w = rand(9, 1, 100)[0]
    w[33] = float("inf")
    w[70] = float("nan")
    x = rand(10, 3, 100)
    q, s, _ = bl.rmsnorm_quant(x.cuda(), w.cuda(), scale=scale)
    check_norm(x, None, w, 1e-6, scale, q, s, None, "f32")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("scale", ["block", "row"])
@pytest.mark.parametrize("n", [8, 120, 128, 129, 200, 256, 257])
def test_norm_short_rows_share_a_wavefront(dt, scale, n):
    """Several rows to a wavefront, the last one of the launch not full; rows of
    zeros, NaN and magnitudes that take the rescaled sum beside ordinary ones."""
    import dense_linear_algebra_potrf_amd as bl
    announce("rmsnorm_quant short rows", dt, scale, n)
    ty = dtypes()[dt]
    for rows in (1, 3, 37, 1030):
        x, r, w = rand(rows, rows, n).to(ty), rand(rows + 1, rows, n).to(ty), (1 + 0.2 * rand(3, 1, n)[0]).to(ty)
        r[:, 0] = 0
        if rows > 3:
            x[2], r[2] = 0, 0
            x[5, n // 2] = float("nan")
            x[9], r[9] = x[9] * 1e-25, 0
            x[10], r[10] = x[10] * 1e20, 0
            x[35], r[35] = x[35] * 1e25, 0
        q, s, h = bl.rmsnorm_quant(x.cuda(), w.cuda(), r.cuda(), scale=scale, eps=1e-38)
        check_norm(x, r, w, 1e-38, scale, q, s, h, dt)


# ---------------------------------------------------------------- rmsnorm_grad

def check_grad(dy, h, w, dh, eps, dx, dw, dt):
    g64, h64, w64 = ref.f64(dy), ref.f64(h), ref.f64(w)
    e64 = None if dh is None else ref.f64(dh)
    want, want_w = ref.norm_grad(g64, h64, w64, e64, eps)
    s = 1 / np.sqrt((h64 * h64).mean(1, keepdims=True) + eps)
    parts = s * (np.abs(g64 * w64) + np.abs(h64) * s * s * np.abs(g64 * w64 * h64).mean(1, keepdims=True))
    bound = 2 * NORM * parts + (HALF_ULP[dt] + 2 * U) * np.abs(want) + SUBNORMAL[dt]
    if dh is not None:
        bound += U * np.abs(e64)
    off = np.abs(ref.f64(dx) - want)
    assert (off <= bound).all(), f"dx {float((off / bound).max())}"
    if dw is not None:
        bound = (NORM + (h.shape[0] + 64) * U) * (np.abs(g64 * h64) * s).sum(0) + SUBNORMAL["f32"]
        off = np.abs(ref.f64(dw) - want_w)
        assert (off <= bound).all(), f"dw {float((off / bound).max())}"


GRAD_SIZES = [(1, 1), (1, 700), (1, 4096), (2, 33), (3, 512), (5, 513), (9, 1024), (517, 1537), (6, 2049), (3, 4103),
              (4, 8192), (2, 9001), (2, 16384), (2051, 64), (1100, 300), (3000, 128), (129, 127), (65, 256), (1, 100), (33, 250),
              (33000, 16)]


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_grad_sizes(dt):
    import dense_linear_algebra_potrf_amd as bl
    for i, (rows, n) in enumerate(GRAD_SIZES):
        announce("rmsnorm_grad", dt, rows, n)
        ty = dtypes()[dt]
        h, dy, dh = (rand(i + k, rows, n).to(ty) for k in (0, 100, 200))
        w = (1 + 0.2 * rand(i + 300, 1, n)[0]).to(ty)
        dh = dh if i % 2 else None
        dx, dw = bl.rmsnorm_grad(dy.cuda(), h.cuda(), w.cuda(), None if dh is None else dh.cuda())
        check_grad(dy, h, w, dh, 1e-6, dx, dw, dt)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("into", ["dy", "h", "dh"])
def test_grad_strided_in_place_and_without_dw(dt, into):
    import torch
    import dense_linear_algebra_potrf_amd as bl
    announce("rmsnorm_grad strided", dt, into)
    ty = dtypes()[dt]
    rows, n = 70, 1001
    h, dy, dh, w = rand(1, rows, n).to(ty), rand(2, rows, n).to(ty), rand(3, rows, n).to(ty), rand(4, 1, n)[0].to(ty)
    (hv, _), (yv, _), (ev, _) = strided(h, 3, 1), strided(dy, 5, 3), strided(dh, 1, 5)
    dx, buf = strided(torch.zeros(rows, n, dtype=ty), 7, 3)
    got, dw = bl.rmsnorm_grad(yv, hv, w.cuda(), ev, dx=dx)
    check_grad(dy, h, w, dh, 1e-6, got, dw, dt)
    again, none = bl.rmsnorm_grad(yv, hv, w.cuda(), ev, dweight=False)
    assert none is None and torch.equal(again, got)
    target = {"dy": yv, "h": hv, "dh": ev}[into]
    inplace, dw2 = bl.rmsnorm_grad(yv, hv, w.cuda(), ev, dx=target)
    assert inplace is target and torch.equal(inplace, again) and torch.equal(dw2, dw)
    assert untouched(dx, buf)


def test_grad_against_differences_of_the_forward():
    """The kernel's gradient against central differences of the 64-bit forward
    (step 1e-5: truncation and rounding near 1e-9), f32: NORM of O(1) terms."""
    import dense_linear_algebra_potrf_amd as bl
    announce("rmsnorm_grad differences")
    rows, n = 2, 9
    h, dy, dh, w = rand(1, rows, n), rand(2, rows, n), rand(3, rows, n), rand(4, 1, n)[0]
    dx, dw = bl.rmsnorm_grad(dy.cuda(), h.cuda(), w.cuda(), dh.cuda())
    h64, g64, e64, w64 = (ref.f64(t) for t in (h, dy, dh, w))
    loss = lambda a, b: (g64 * ref.norm(a, b, 1e-6)).sum() + (e64 * a).sum()  # noqa: E731
    step = 1e-5
    for i in range(rows):
        for c in range(n):
            d = np.zeros_like(h64)
            d[i, c] = step
            want = (loss(h64 + d, w64) - loss(h64 - d, w64)) / (2 * step)
            assert abs(want - float(dx[i, c])) <= 1e-4 * max(1, abs(want))
    for c in range(n):
        d = np.zeros(n)
        d[c] = step
        want = (loss(h64, w64 + d) - loss(h64, w64 - d)) / (2 * step)
        assert abs(want - float(dw[c])) <= 1e-4 * max(1, abs(want))


@pytest.mark.parametrize("n", [100, 200, 700, 3000])
def test_rows_of_zeros_with_an_eps_below_the_normal_range(n):
    """1 / sqrt(eps) is an ordinary number, so the rows are zeros and their gradient dy w / sqrt(eps)."""
    import torch
    import dense_linear_algebra_potrf_amd as bl
    for eps in (1e-38, 3e-44, 1e-30):
        announce("rows of zeros", n, eps)
        eps = float(np.float32(eps))
        h, w, dy = torch.zeros(3, n), 1 + 0.2 * rand(1, 1, n)[0], rand(2, 3, n)
        h[1] = 1e-22
        for scale in ("block", "row"):
            q, s, _ = bl.rmsnorm_quant(h.cuda(), w.cuda(), scale=scale, eps=eps)
            check_norm(h, None, w, eps, scale, q, s, None, "f32")
            assert not q[0].float().any()
        dx, dw = bl.rmsnorm_grad(dy.cuda(), h.cuda(), w.cuda(), eps=eps)
        check_grad(dy, h, w, None, eps, dx, dw, "f32")


def test_grad_without_rows():
    import torch
    import dense_linear_algebra_potrf_amd as bl
    announce("rmsnorm_grad no rows")
    e = torch.empty(0, 77, device="cuda")
    dw = torch.full((77,), 5.0, device="cuda")
    dx, out = bl.rmsnorm_grad(e, e, torch.ones(77, device="cuda"), dweight=dw)
    assert dx.shape == (0, 77) and out is dw and not dw.any()
    q, s, h = bl.rmsnorm_quant(e, torch.ones(77, device="cuda"), e)
    assert q.shape == (0, 77) and s.shape == (0, 3) and h.shape == (0, 77)


# ---------------------------------------------------------------- weight_quant

FORMS = [("int4", 32, False), ("int4", 64, False), ("int4", 128, False), ("int4", 32, True), ("int4", 64, True),
         ("int4", 128, True), ("fp4", 32, False)]


def check_quant(W, fmt, group, zeros, codes, scales, z, values):
    import torch
    n, k = W.shape
    want_u, want_s, want_z, want_v = ref.quant(W.float().numpy(), fmt, group, zeros)
    got_u = ref.unpack(codes.cpu().numpy(), k)
    assert np.array_equal(got_u, want_u), f"codes differ at {np.argwhere(got_u != want_u)[:5]}"
    got_s = ref.f64(scales.float())
    assert np.array_equal(got_s, want_s.astype(np.float64), equal_nan=True), "scales"
    if zeros:
        assert np.array_equal(ref.f64(z), want_z), "zeros"
    if values is not None:
        v = torch.from_numpy(want_v.astype(np.float32)).to(W.dtype)
        assert np.array_equal(ref.f64(values), ref.f64(v), equal_nan=True), "values"


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("fmt,group,zeros", FORMS)
def test_quant_sizes(dt, fmt, group, zeros):
    import dense_linear_algebra_potrf_amd as bl
    for i, (n, k) in enumerate([(1, 1), (3, 2), (5, 7), (2, 31), (4, 33), (3, 127), (2, 129), (7, 500), (64, 512), (33, 1037)]):
        announce("weight_quant", dt, fmt, group, zeros, n, k)
        W = (0.02 * rand(i, n, k) + 0.003).to(dtypes()[dt])
        if n > 2:
            W[1] = 0
            W[2] = W[2].abs()                      # one sign: the zero point at an end
        out = bl.weight_quant(W.cuda(), format=fmt, group=group, zeros=zeros, values=True)
        check_quant(W, fmt, group, zeros, *out)


@pytest.mark.parametrize("fmt,group,zeros", FORMS)
def test_quant_ties_extremes_and_broken_groups(fmt, group, zeros):
    import torch
    import dense_linear_algebra_potrf_amd as bl
    announce("weight_quant extremes", fmt, group, zeros)
    k = 4 * group + 5
    W = torch.randint(-28, 29, (12, k), generator=torch.Generator().manual_seed(3)).float() / 4    # quarters: many ties
    W[0, :2] = torch.tensor([7.0, -7.0])
    W[1] *= 2.0 ** -130                              # subnormal magnitudes
    W[2] *= 1e37
    W[3, 1] = float("nan")
    W[4, group + 1] = float("inf")
    W[5, -1] = -float("inf")
    W[6, 0], W[6, 1] = 3.4e38, -3.4e38               # finite, but the span is not
    W[7] = 3.0e-39
    W[8] = -1.0
    W[9] = 6.0
    W[10] = 6.0000005
    W[11] = -0.0
    out = bl.weight_quant(W.cuda(), format=fmt, group=group, zeros=zeros, values=True)
    check_quant(W, fmt, group, zeros, *out)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("fmt,group,zeros", [("int4", 64, True), ("fp4", 32, False)])
def test_quant_strided(dt, fmt, group, zeros):
    import torch
    import dense_linear_algebra_potrf_amd as bl
    announce("weight_quant strided", dt, fmt)
    n, k = 37, 333
    W = rand(5, n, k).to(dtypes()[dt])
    Wv, _ = strided(W, 3, 1)
    vals, vb = strided(torch.zeros_like(W), 5, 3)
    buf = torch.full((n, 256), 0xFF, dtype=torch.uint8, device="cuda")
    st = dtypes()["bf16"] if fmt == "int4" else torch.float8_e8m0fnu
    sv, sb = strided(torch.zeros(n, -(-k // group), dtype=st if fmt == "int4" else torch.uint8), 3, 1)
    out = bl.weight_quant(Wv, format=fmt, group=group, zeros=zeros, values=vals, codes=buf, scales=sv.view(st))
    check_quant(W, fmt, group, zeros, *out)
    assert int((buf[:, (k + 1) // 2:] != 0xFF).sum()) == 0, "wrote past a row's codes"
    assert untouched(vals, vb) and untouched(sv, sb)
    codes, _, _, none = bl.weight_quant(Wv, format=fmt, group=group, zeros=zeros)
    assert none is None and torch.equal(codes[:, :k // 2], buf[:, :k // 2])


# ---------------------------------------------------------------- weight_matvec

def make_weights(seed, n, k, fmt, group, zeros, exact=False):
    """(codes [n, k], scales, zeros, GPU tensors) of random 4-bit weights; exact: small power-of-two scales."""
    import torch
    rng = np.random.default_rng(seed)
    codes = rng.integers(0, 16, (n, k))
    shape = (n, -(-k // group))
    z = rng.integers(0, 16, shape).astype(np.uint8) if zeros else None
    if fmt == "fp4":
        b = rng.integers(125, 129, shape).astype(np.uint8)
        scales, st = 2.0 ** (b.astype(np.float64) - 127), torch.from_numpy(b).view(torch.float8_e8m0fnu)
    else:
        f = 2.0 ** rng.integers(-2, 2, shape).astype(np.float64) if exact else 0.01 * np.exp(0.4 * rng.standard_normal(shape))
        st = torch.from_numpy(f).to(torch.bfloat16)
        scales = ref.f64(st)
    cuda = (torch.from_numpy(ref.pack(codes)).cuda(), st.cuda(), None if z is None else torch.from_numpy(z).cuda())
    return codes, scales, z, cuda


def make_x(seed, m, k, kind, exact=False):
    """(x as 64-bit values, GPU x, GPU x_scales)."""
    import torch
    g = torch.Generator().manual_seed(seed)
    x = torch.randint(-8, 9, (m, k), generator=g).float() if exact else torch.randn(m, k, generator=g)
    if kind in ("bf16", "f16"):
        x = x.to(dtypes()[kind])
        return ref.f64(x), x.cuda(), None
    q = (x if exact else 40 * x).to(torch.float8_e4m3fn)
    if kind == "f8block":
        b = torch.randint(125, 129, (m, -(-k // 32)), generator=g, dtype=torch.uint8)
        wide = np.repeat(2.0 ** (b.double().numpy() - 127), 32, 1)[:, :k]
        return ref.f64(q.float()) * wide, q.cuda(), b.view(torch.float8_e8m0fnu).cuda()
    s = 2.0 ** torch.randint(-2, 3, (m,), generator=g).float() if exact else 0.5 + torch.rand(m, generator=g)
    return ref.f64(q.float()) * ref.f64(s)[:, None], q.cuda(), s.cuda()


MV_SIZES = [(1, 1, 1), (1, 16, 32), (2, 17, 31), (3, 5, 65), (1, 40, 128), (5, 33, 129), (16, 64, 256), (17, 31, 333),
            (4, 100, 1000), (1, 130, 4096), (33, 47, 640), (64, 48, 512), (65, 20, 200), (130, 16, 96), (7, 24, 5001)]


@pytest.mark.parametrize("kind", ["bf16", "f16", "f8block", "f8row"])
@pytest.mark.parametrize("fmt,group,zeros", FORMS)
def test_matvec_exact_integers(kind, fmt, group, zeros):
    """Small integers times small powers of two: every sum is exact in 32 bits,
    so y must be exact too."""
    import torch
    import dense_linear_algebra_potrf_amd as bl
    for i, (m, n, k) in enumerate(MV_SIZES):
        announce("weight_matvec exact", kind, fmt, group, zeros, m, n, k)
        codes, sc, z, cuda = make_weights(i, n, k, fmt, group, zeros, exact=True)
        x64, x, xs = make_x(i + 40, m, k, kind, exact=True)
        want = x64 @ ref.held(codes, sc, z, fmt, group, k).T
        y = bl.weight_matvec(x, *cuda, format=fmt, group=group, x_scales=xs, out_dtype=torch.float32)
        got = ref.f64(y)
        assert np.array_equal(got, want), f"{int((got != want).sum())} of {want.size} differ"


@pytest.mark.parametrize("kind", ["bf16", "f16", "f8block", "f8row"])
@pytest.mark.parametrize("fmt,group,zeros", FORMS)
def test_matvec_many_columns_and_long_rows(kind, fmt, group, zeros):
    """Exact, as above: n where a workgroup takes 32 rows of W (with a last one that
    is not full), 16 rows and 8 or 16 wavefronts, at every number of rows of x that
    has its own kernel; and k where a row has more groups than are held at a time."""
    import torch
    import dense_linear_algebra_potrf_amd as bl
    long = 256 * group                              # columns of the groups held at a time
    sizes = [(1, 8200, 300), (4, 8193, 129), (8, 8223, 257), (16, 8192, 130), (20, 8201, 200), (40, 8195, 290),
             (2, 4100, 257), (19, 4097, 140), (1, 33, long + 17), (5, 20, 2 * long + 300), (16, 17, long + 1),
             (21, 18, long + 33), (64, 33, long + 129)]
    if fmt == "int4" and group > 32:
        sizes = sizes[:2] + sizes[5:6] + sizes[8:]
    for i, (m, n, k) in enumerate(sizes):
        announce("weight_matvec wide", kind, fmt, group, zeros, m, n, k)
        codes, sc, z, cuda = make_weights(i, n, k, fmt, group, zeros, exact=True)
        x64, x, xs = make_x(i + 40, m, k, kind, exact=True)
        want = x64 @ ref.held(codes, sc, z, fmt, group, k).T
        y = bl.weight_matvec(x, *cuda, format=fmt, group=group, x_scales=xs, out_dtype=torch.float32)
        got = ref.f64(y)
        assert np.array_equal(got, want), f"{int((got != want).sum())} of {want.size} differ"


@pytest.mark.parametrize("kind", ["bf16", "f16", "f8block", "f8row"])
@pytest.mark.parametrize("fmt,group,zeros", [("int4", 32, False), ("int4", 128, True), ("fp4", 32, False)])
def test_matvec_many_rows_that_are_not_finite(kind, fmt, group, zeros):
    """More than 16 rows, each with its own range: infinities, NaN, rows of zeros,
    rows of one value near the type's largest, rows down to its smallest ones."""
    import torch
    import dense_linear_algebra_potrf_amd as bl
    announce("weight_matvec many rows not finite", kind, fmt, group, zeros)
    m, n, k = 37, 50, 300
    codes, sc, z, (cc, cs, cz) = make_weights(3, n, k, fmt, group, zeros, exact=True)
    x64, x, xs = make_x(4, m, k, kind, exact=True)
    eight = kind.startswith("f8")
    big = {"bf16": 3e38, "f16": 6e4}.get(kind, 448.0)
    v = x.float()
    if not eight:
        v[1, 7] = float("inf")
        v[2, 299] = -float("inf")
        v[17, 200], v[17, 3] = float("inf"), float("inf")
    v[3, 100] = float("nan")
    v[4] = 0
    v[18] = 0
    v[18, 33] = big
    v[19] *= 2.0 ** (-126 if kind == "bf16" else -20 if kind == "f16" else -6)
    v[20, 5] *= 2.0 ** (30 if kind == "bf16" else 8 if kind == "f16" else 3)      # one that dwarfs its row
    x = v.to(x.dtype)
    s2 = cs.float()
    s2[5, 1], sc[5, 1] = float("nan"), np.nan
    if fmt == "int4":
        s2[11, 0], sc[11, 0] = float("inf"), np.inf
    if kind == "f8block":
        raw_scales = xs.view(torch.uint8)
        raw_scales[30, 2], raw_scales[31, 1], raw_scales[32], raw_scales[33, 0] = 255, 200, 0, 20
        b = raw_scales.cpu().numpy()
        xw = np.repeat(np.where(b == 255, np.nan, 2.0 ** (b.astype(np.float64) - 127)), 32, 1)[:, :k]
    elif kind == "f8row":
        xs[30], xs[31], xs[32] = float("nan"), float("inf"), 2.0 ** -126
        xw = ref.f64(xs)[:, None]
    else:
        xw = 1.0
    with np.errstate(all="ignore"):
        x64 = ref.f64(x.float()) * xw
        W = ref.held(codes, sc, z, fmt, group, k)
        want = np.stack([(ref.f64(x.float())[i] * (xw if np.isscalar(xw) else xw[i]) * W).sum(1) for i in range(m)])
        want32 = want.astype(np.float32)
        size = (np.abs(np.where(np.isfinite(x64), x64, 0)) @
                np.repeat(np.where(np.isfinite(sc), sc, 0), group, 1)[:, :k].T)
    y = bl.weight_matvec(x, cc, s2.to(cs.dtype), cz, format=fmt, group=group, x_scales=xs, out_dtype=torch.float32)
    got = y.cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(want32)), np.argwhere(np.isnan(got) != np.isnan(want32))[:8]
    inf = np.isinf(want32)
    assert np.array_equal(got[inf], want32[inf])
    ok = np.isfinite(want32)
    off = np.abs(got - want)
    bound = PRODUCT * size + 4 * U * np.abs(want) + SUBNORMAL["f32"]
    assert (off <= bound)[ok].all(), np.argwhere(ok & ~(off <= bound))[:8]


@pytest.mark.parametrize("kind", ["bf16", "f16", "f8block", "f8row"])
@pytest.mark.parametrize("fmt,group,zeros", FORMS)
def test_matvec_error(kind, fmt, group, zeros):
    import torch
    import dense_linear_algebra_potrf_amd as bl
    for i, (m, n, k, out) in enumerate([(1, 300, 4096, "bf16"), (3, 77, 2500, "f16"), (16, 128, 1024, "f32"), (64, 96, 2048, "bf16")]):
        announce("weight_matvec error", kind, fmt, group, zeros, m, n, k, out)
        codes, sc, z, cuda = make_weights(i + 7, n, k, fmt, group, zeros)
        x64, x, xs = make_x(i + 70, m, k, kind)
        W = ref.held(codes, sc, z, fmt, group, k)
        want = x64 @ W.T
        y = bl.weight_matvec(x, *cuda, format=fmt, group=group, x_scales=xs, out_dtype=dtypes()[out])
        size = np.repeat(sc, group, 1)[:, :k]
        bound = PRODUCT * (np.abs(x64) @ size.T) + (HALF_ULP[out] + 4 * U) * np.abs(want) + SUBNORMAL[out]
        off = np.abs(ref.f64(y) - want)
        assert (off <= bound).all(), float((off / bound).max())


@pytest.mark.parametrize("kind", ["bf16", "f16", "f8block", "f8row"])
@pytest.mark.parametrize("fmt,group,zeros", [("int4", 64, True), ("int4", 128, False), ("fp4", 32, False)])
def test_matvec_strided_rows_and_outputs(kind, fmt, group, zeros):
    import torch
    import dense_linear_algebra_potrf_amd as bl
    for i, (m, n, k) in enumerate([(3, 37, 333), (18, 65, 1000)]):
        announce("weight_matvec strided", kind, fmt, m, n, k)
        codes, sc, z, (cc, cs, cz) = make_weights(i, n, k, fmt, group, zeros, exact=True)
        x64, x, xs = make_x(i + 40, m, k, kind, exact=True)
        wide = torch.full((n, cc.shape[1] + 48), 0xEE, dtype=torch.uint8, device="cuda")
        wide[:, :cc.shape[1]] = cc
        raw = x.view(torch.uint8) if kind.startswith("f8") else x
        xv, _ = strided(raw, 5, 3)
        xv = xv.view(x.dtype)
        sv, _ = strided(cs if fmt == "int4" else cs.view(torch.uint8), 3, 1)
        sv = sv.view(cs.dtype)
        zv = None if cz is None else strided(cz, 5, 1)[0]
        if kind == "f8block":
            xs = strided(xs.view(torch.uint8), 3, 1)[0].view(xs.dtype)
        y, yb = strided(torch.zeros(m, n, dtype=torch.float32), 5, 3)
        got = bl.weight_matvec(xv, wide[:, :cc.shape[1]], sv, zv, format=fmt, group=group, x_scales=xs, out=y)
        assert got is y and np.array_equal(ref.f64(y), x64 @ ref.held(codes, sc, z, fmt, group, k).T)
        assert untouched(y, yb)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("fmt,group,zeros", FORMS)
def test_matvec_values_that_are_not_finite(kind, fmt, group, zeros):
    """Infinities and NaN in x and in scales reach exactly the results that the
    definition gives them, and no others; very large x does not overflow early."""
    import torch
    import dense_linear_algebra_potrf_amd as bl
    announce("weight_matvec not finite", kind, fmt, group, zeros)
    m, n, k = 6, 50, 300
    codes, sc, z, (cc, cs, cz) = make_weights(3, n, k, fmt, group, zeros, exact=True)
    x64, x, _ = make_x(4, m, k, kind, exact=True)
    big = 3e38 if kind == "bf16" else 6e4
    x[1, 7] = float("inf")
    x[2, 299] = -float("inf")
    x[3, 100] = float("nan")
    x[4] = 0
    x[4, 33] = big                                  # times a weight of a small scale it is still finite
    sc, s2 = sc.copy(), cs.float()
    s2[5, 1], s2[9, 0] = float("nan"), 2.0 ** -20
    sc[5, 1], sc[9, 0] = np.nan, 2.0 ** -20
    if fmt == "int4":
        s2[11, 1], sc[11, 1] = float("inf"), np.inf
    x64 = ref.f64(x)
    with np.errstate(all="ignore"):
        want = np.stack([(x64[i] * ref.held(codes, sc, z, fmt, group, k)).sum(1) for i in range(m)])
        want32 = want.astype(np.float32)
    y = bl.weight_matvec(x, cc, s2.to(cs.dtype), cz, format=fmt, group=group, out_dtype=torch.float32)
    got = y.cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(want32)), np.argwhere(np.isnan(got) != np.isnan(want32))[:8]
    inf = np.isinf(want32)
    assert np.array_equal(got[inf], want32[inf])
    ok = np.isfinite(want32)
    bound = 2 * PRODUCT * np.abs(np.where(np.isfinite(x64), x64, 0)).sum(1)[:, None] * 16 + 1e-30
    assert (np.abs(got - want)[ok] <= np.broadcast_to(bound, got.shape)[ok]).all()


@pytest.mark.parametrize("m", [1, 20])
def test_matvec_extreme_powers(m):
    """Scale bytes at both ends of the range: 2^-127 times a large x, 2^126 times a small one."""
    import torch
    import dense_linear_algebra_potrf_amd as bl
    announce("weight_matvec extreme powers", m)
    n, k = 20, 64
    codes = np.random.default_rng(0).integers(0, 16, (n, k))
    for byte, mag in ((0, 2.0 ** 120), (1, 2.0 ** 100), (2, 2.0 ** 100), (253, 2.0 ** -120)):
        b = np.full((n, 2), byte, np.uint8)
        x = (torch.randint(-4, 5, (m, k), generator=torch.Generator().manual_seed(1)).double() * mag).to(torch.bfloat16)
        want = ref.f64(x) @ ref.held(codes, 2.0 ** (b.astype(np.float64) - 127), None, "fp4", 32, k).T
        y = bl.weight_matvec(x.cuda(), torch.from_numpy(ref.pack(codes)).cuda(), torch.from_numpy(b).view(torch.float8_e8m0fnu).cuda(),
                             format="fp4", out_dtype=torch.float32)
        assert np.array_equal(ref.f64(y), want), byte


def test_matvec_without_rows_and_refusals():
    import torch
    import dense_linear_algebra_potrf_amd as bl
    announce("weight_matvec refusals")
    _, _, _, (cc, cs, cz) = make_weights(0, 8, 64, "int4", 32, True)
    x = torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda")
    assert bl.weight_matvec(x, cc, cs, cz, group=32).shape == (0, 8)
    x = torch.zeros(2, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="scales must be"):
        bl.weight_matvec(x, cc, cs, cz, group=64)
    with pytest.raises(ValueError, match="contiguous rows"):
        bl.weight_matvec(x.t().contiguous().t(), cc, cs, cz, group=32)
    with pytest.raises(ValueError, match="codes must be rows"):
        bl.weight_matvec(x, cc[:, :16], cs, cz, group=32)
    with pytest.raises(TypeError, match="codes must be"):
        bl.weight_matvec(x, cc.view(torch.int8), cs, cz, group=32)
    with pytest.raises(TypeError, match="scales must be"):
        bl.weight_matvec(x, cc, cs.float(), cz, group=32)
    with pytest.raises(ValueError, match="x_scales"):
        bl.weight_matvec(x, cc, cs, cz, group=32, x_scales=torch.ones(2, device="cuda"))
    with pytest.raises(ValueError, match="needs x_scales"):
        bl.weight_matvec(x.to(torch.float8_e4m3fn), cc, cs, cz, group=32)
    with pytest.raises(ValueError, match="GPU"):
        bl.weight_matvec(x, cc.cpu(), cs, cz, group=32)
    with pytest.raises(bl.BatchlasError, match="group must be"):
        bl.weight_matvec(x, cc, cs[:, :1].expand(8, 1), None, group=256)
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="needs a residual"):
        bl.rmsnorm_quant(x, w, residual_out=x)
    with pytest.raises(ValueError, match="weight must be"):
        bl.rmsnorm_quant(x, w[:32])
    with pytest.raises(bl.BatchlasError, match="at most"):
        big = torch.zeros(1, 40000, device="cuda")
        bl.rmsnorm_quant(big, big[0])
    with pytest.raises(bl.BatchlasError, match="workspace_bytes"):
        tall = x.repeat(100, 1)                       # more than one workgroup's rows
        bl.rmsnorm_grad(tall, tall, w, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


# ---------------------------------------------------------------- together

def layer_step(bl, s, stream=None):
    """Norm, product and gradient as one layer's step; `s` holds the inputs and outputs."""
    bl.rmsnorm_quant(s["x"], s["w"], s["r"], out=s["q"], scales=s["qs"], residual_out=s["h"], stream=stream)
    bl.weight_quant(s["W"], format="int4", group=64, zeros=True, codes=s["codes"], scales=s["ws"], zeros_out=s["wz"], values=s["wv"],
                    stream=stream)
    bl.weight_matvec(s["q"], s["codes"], s["ws"], s["wz"], group=64, x_scales=s["qs"], out=s["y"], stream=stream)
    bl.rmsnorm_grad(s["dy"], s["h"], s["w"], s["r"], dx=s["dx"], dweight=s["dw"], workspace=s["ws_grad"], stream=stream)
    return [s[k] for k in ("q", "qs", "h", "codes", "ws", "wz", "wv", "y", "dx", "dw")]


def layer_state(seed, m=37, n=200, k=1000):
    import torch
    import dense_linear_algebra_potrf_amd as bl
    b = torch.bfloat16
    dev = dict(device="cuda")
    s = {key: rand(seed + i, m, k).to(b).cuda() for i, key in enumerate(("x", "r", "dy"))}
    s["w"], s["W"] = rand(seed + 8, 1, k)[0].to(b).cuda(), rand(seed + 9, n, k).to(b).cuda()
    s["q"] = torch.zeros(m, k, dtype=torch.float8_e4m3fn, **dev)
    s["qs"] = torch.zeros(m, -(-k // 32), dtype=torch.uint8, **dev).view(torch.float8_e8m0fnu)
    s["h"], s["dx"], s["wv"] = torch.zeros(m, k, dtype=b, **dev), torch.zeros(m, k, dtype=b, **dev), torch.zeros(n, k, dtype=b, **dev)
    s["codes"] = torch.zeros(n, -(-k // 32) * 16, dtype=torch.uint8, **dev)
    g = -(-k // 64)
    s["ws"], s["wz"] = torch.zeros(n, g, dtype=b, **dev), torch.zeros(n, g, dtype=torch.uint8, **dev)
    s["y"], s["dw"] = torch.zeros(m, n, dtype=b, **dev), torch.zeros(k, **dev)
    s["ws_grad"] = torch.zeros(bl.rmsnorm_grad_workspace(b, m, k), dtype=torch.uint8, **dev)
    return s


def raw(ts):
    import torch
    return [t.contiguous().view(torch.uint8).clone() for t in ts]


def test_runs_alike_on_another_stream_and_in_a_graph():
    """Two runs, a run on another stream and every replay of a graph (with eager
    work between the replays) give the same bits."""
    import torch
    import dense_linear_algebra_potrf_amd as bl
    announce("layer step: streams and graph")
    s = layer_state(0)
    want = raw(layer_step(bl, s))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, raw(layer_step(bl, s))))
    side = torch.cuda.Stream()
    late = torch.zeros(1 << 22, device="cuda")
    other = layer_state(0)
    for t in (other["x"], other["r"]):
        t.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):                   # inputs written on the side stream, after a delay
        for _ in range(20):
            late.add_(1)
        other["x"].copy_(s["x"])
        other["r"].copy_(s["r"])
    got = layer_step(bl, other, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, raw(got)))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = layer_step(bl, other)
    for rep in range(4):
        fresh = layer_state(10 * rep)
        for key in ("x", "r", "dy", "w", "W"):
            other[key].copy_(fresh[key])
        for t in out:
            t.view(torch.uint8).zero_()
        torch.cuda.synchronize()
        eager = raw(layer_step(bl, fresh))
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, raw(out))), f"replay {rep}"


def test_what_a_call_on_a_stream_allocates_belongs_to_it():
    """Workspaces and outputs of calls that wait on a side stream are not handed out
    again to work that runs meanwhile on the current one."""
    import torch
    import dense_linear_algebra_potrf_amd as bl
    announce("allocations on a side stream")
    s = layer_state(5)
    kw = dict(group=64, x_scales=s["qs"])
    layer_step(bl, s)
    want = [bl.weight_matvec(s["q"], s["codes"], s["ws"], s["wz"], **kw), *bl.rmsnorm_grad(s["dy"], s["h"], s["w"], s["r"]),
            *bl.rmsnorm_quant(s["x"], s["w"], s["r"]), *bl.weight_quant(s["W"], group=64, zeros=True, values=True)]
    want = raw(want)
    late, side = torch.zeros(1 << 24, device="cuda"), torch.cuda.Stream()
    sizes = sorted({t.numel() for t in want} | {bl.weight_matvec_workspace(37, 1000), s["ws_grad"].numel()})
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(100):
            late.add_(1)
    got = [bl.weight_matvec(s["q"], s["codes"], s["ws"], s["wz"], stream=side, **kw),
           *bl.rmsnorm_grad(s["dy"], s["h"], s["w"], s["r"], stream=side), *bl.rmsnorm_quant(s["x"], s["w"], s["r"], stream=side),
           *bl.weight_quant(s["W"], group=64, zeros=True, values=True, stream=side)]
    keep = [torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda") for size in sizes for _ in range(8)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, raw(got)))
    assert all(bool((t == 0xFF).all()) for t in keep)


def test_offsets_beyond_32_bits():
    """Arrays past 4 GiB: the last rows of a tall norm, of wide codes and of their products."""
    import torch
    import dense_linear_algebra_potrf_amd as bl
    announce("layer operators beyond 2^32 bytes")
    n, rows = 16384, (1 << 17) + 5                   # 2^31 elements and some
    x = torch.zeros(rows, n, dtype=torch.bfloat16, device="cuda")
    tail = rand(1, 5, n).to(torch.bfloat16)
    x[-5:] = tail.cuda()
    w = torch.ones(n, dtype=torch.bfloat16)
    q, s, _ = bl.rmsnorm_quant(x, w.cuda())
    check_norm(tail, None, w, 1e-6, "block", q[-5:], s[-5:], None, "bf16")
    assert not q[:-5].view(torch.int32).any()
    # W of the same size: rounded, and multiplied
    codes, sc, z, values = bl.weight_quant(x, format="int4", group=128, values=True)
    check_quant(tail, "int4", 128, False, codes[-5:], sc[-5:], None, values[-5:])
    del values, q
    wide = torch.zeros((1 << 16) + 3, 1 << 16, dtype=torch.uint8, device="cuda")      # codes past 2^32 bytes
    wide[-3:, :n // 2] = codes[-3:]
    scales = torch.ones(wide.shape[0], 128, dtype=torch.bfloat16, device="cuda")
    act = torch.randint(-8, 9, (2, n), generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    y = bl.weight_matvec(act.cuda(), wide[:, :n // 2], scales, out_dtype=torch.float32)
    u = ref.unpack(codes[-3:].cpu().numpy(), n)
    assert np.array_equal(ref.f64(y[:, -3:]), ref.f64(act) @ (u - 8.0).T)
    assert torch.equal(y[:, 0].cpu(), -8 * act.float().sum(1))
