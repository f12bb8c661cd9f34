"""Products with 4-bit weights on x of a wide range, against the definition in 64
bits and with a bound that follows |x| |w| (not |x| times the codes).

The bound, from the arithmetic (u = 2^-24): codes less their zero point and x are
exact in 16 bits, so their products are exact in 32.  A product of the matrix
cores adds 32 of them to a sum with at most 32 roundings of 2 u each (should it
cut off); up to 4 of them make a group, whose sum takes one rounding with its
scale; a wavefront adds its groups in turn, at most 16 wavefronts are joined, and
4 roundings are left for the scale of x's row and the output:
    (4 * 32 * 2 + groups + 16 + 4) u  of  sum |x| |w|.
"""
from __future__ import annotations

import numpy as np
import pytest

from tests import _layer_ref as ref
from tests._gpu import announce
from tests.test_gpu_layer import FORMS, SUBNORMAL, U, dtypes, make_weights

pytestmark = pytest.mark.gpu


def bound(x64, W, groups: int) -> np.ndarray:
    return (4 * 32 * 2 + groups + 20) * U * (np.abs(x64) @ np.abs(W).T) + (groups + 20) * SUBNORMAL["f32"]


def wide_x(kind, m, k, column, seed):
    """(x in 64 bits, GPU x, GPU x_scales): ordinary values, and one column that dwarfs them by 2^14 and more."""
    import torch
    g = torch.Generator().manual_seed(seed)
    v = torch.randn(m, k, generator=g)
    if kind in ("bf16", "f16"):
        if kind == "bf16":
            v[:, column] = 2.0 ** torch.tensor([14, 22, 31, 40, 60, 100])[torch.arange(m) % 6].float()
        else:
            v *= 2.0 ** -8
            v[:, column] = torch.tensor([1e3, 6e4])[torch.arange(m) % 2]
        x = v.to(dtypes()[kind])
        return ref.f64(x), x.cuda(), None
    v = (v * 2.0 ** -6).clamp(-1, 1)
    v[:, column] = 448.0
    if kind == "f8row":
        q, s = v.to(torch.float8_e4m3fn), 0.5 + torch.rand(m, generator=g)
        return ref.f64(q.float()) * ref.f64(s)[:, None], q.cuda(), s.cuda()
    at = column // 32
    own = v[:, column].clone()
    v[:, 32 * at:32 * at + 32] = 0                  # the large column is alone in its block of scales
    v[:, column] = own
    q = v.to(torch.float8_e4m3fn)
    b = torch.randint(125, 129, (m, -(-k // 32)), generator=g, dtype=torch.uint8)
    b[:, at] = torch.tensor([127, 140, 160, 200])[torch.arange(m) % 4].to(torch.uint8)
    wide = np.repeat(2.0 ** (b.double().numpy() - 127), 32, 1)[:, :k]
    return ref.f64(q.float()) * wide, q.cuda(), b.view(torch.float8_e8m0fnu).cuda()


def check_large_column(kind, fmt, group, zeros, rows):
    import torch
    import dense_linear_algebra_potrf_amd as bl
    n, k = 33, 300
    for i, m in enumerate(rows):
        for column in (5, 131, 299):
            announce("weight_matvec large column", kind, fmt, group, zeros, m, column)
            codes, sc, z, (_, cs, cz) = make_weights(i, n, k, fmt, group, zeros)
            codes[:30, column] = 0 if fmt == "fp4" else 8 if z is None else z[:30, column // group]
            x64, x, xs = wide_x(kind, m, k, column, i)
            W = ref.held(codes, sc, z, fmt, group, k)
            assert not W[:30, column].any()
            y = bl.weight_matvec(x, torch.from_numpy(ref.pack(codes)).cuda(), cs, cz, format=fmt, group=group, x_scales=xs,
                                 out_dtype=torch.float32)
            off, most = np.abs(ref.f64(y) - x64 @ W.T), bound(x64, W, -(-k // group))
            assert (off <= most).all(), float((off / most).max())


KINDS = ["bf16", "f16", "f8block", "f8row"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("fmt,group,zeros", FORMS)
def test_a_large_column_without_weight_leaves_the_others(kind, fmt, group, zeros):
    """Up to 16 rows of x: a column whose weights are zero adds nothing, however large it is."""
    check_large_column(kind, fmt, group, zeros, (1, 4, 7, 16))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("fmt,group,zeros", FORMS)
def test_a_large_column_without_weight_among_many_rows(kind, fmt, group, zeros):
    """As above from 17 rows of x on."""
    check_large_column(kind, fmt, group, zeros, (17, 33, 65))


def check_scale_bytes(rows):
    """Every kind of scale byte of 8-bit x against 4-bit float weights of every kind of scale: exact where the result
    is a normal number, infinite or NaN where it is."""
    import torch
    import dense_linear_algebra_potrf_amd as bl
    xb = np.array([0, 1, 2, 3, 4, 5, 60, 120, 127, 200, 243, 244, 246, 247, 251, 252, 253, 254, 255], np.uint8)
    wb = np.array([0, 1, 2, 60, 127, 131, 200, 240, 252, 253, 254], np.uint8)
    rng = np.random.default_rng(0)
    small = np.concatenate([np.arange(0, 0x39), np.arange(0x80, 0xb9)])         # e4m3 values up to 1, subnormal ones among them
    for m in rows:
        for k in (20, 100, 300):
            blocks = -(-k // 32)
            x = torch.from_numpy(rng.choice(small, (m, k)).astype(np.uint8)).view(torch.float8_e4m3fn)
            if m > 1:
                x[0] = 0                                                        # an empty row, whatever its scales are
            codes = rng.integers(0, 16, (len(wb), k))
            b = np.broadcast_to(wb[:, None], (len(wb), blocks)).copy()
            held = ref.held(codes, 2.0 ** (b.astype(np.float64) - 127), None, "fp4", 32, k)
            cc, cs = torch.from_numpy(ref.pack(codes)).cuda(), torch.from_numpy(b).view(torch.float8_e8m0fnu).cuda()
            for shift in range(0, len(xb), m):
                announce("weight_matvec scale bytes", m, k, shift)
                s = np.broadcast_to(xb[(np.arange(m) + shift) % len(xb)][:, None], (m, blocks)).copy()
                with np.errstate(all="ignore"):
                    one = np.where(s[:, 0] == 255, np.nan, 2.0 ** (s[:, 0].astype(np.float64) - 127))
                    want = ((ref.f64(x.float()) * one[:, None]) @ held.T).astype(np.float32)
                y = bl.weight_matvec(x.cuda(), cc, cs, format="fp4", x_scales=torch.from_numpy(s).view(torch.float8_e8m0fnu).cuda(),
                                     out_dtype=torch.float32).cpu().numpy()
                assert np.array_equal(np.isnan(y), np.isnan(want))
                inf = np.isinf(want)
                assert np.array_equal(y[inf], want[inf])
                with np.errstate(all="ignore"):
                    # subnormal results: each group rounds to a step
                    ok = np.abs(y - want) <= np.where(np.abs(want) < 2.0 ** -126, (blocks + 1) * SUBNORMAL["f32"], 0)
                ok |= ~np.isfinite(want)
                assert ok.all(), [(int(s[i, 0]), int(wb[j]), float(y[i, j]), float(want[i, j])) for i, j in np.argwhere(~ok)[:6]]


@pytest.mark.parametrize("m", [1, 4, 7, 16])
def test_scale_bytes_of_a_few_rows(m):
    check_scale_bytes((m,))


@pytest.mark.parametrize("m", [17, 40])
def test_scale_bytes_of_many_rows(m):
    check_scale_bytes((m,))


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("m", [1, 4, 16, 17, 33])
def test_subnormal_x(kind, m):
    """The smallest numbers of x's type, times large weights: exact."""
    import torch
    import dense_linear_algebra_potrf_amd as bl
    announce("weight_matvec subnormal x", kind, m)
    n, k = 20, 200
    step = 2.0 ** (-133 if kind == "bf16" else -24)
    x = (torch.randint(-8, 9, (m, k), generator=torch.Generator().manual_seed(m)).double() * step).to(dtypes()[kind])
    assert np.array_equal(ref.f64(x) / step, np.rint(ref.f64(x) / step)) and x.bool().any()
    codes = np.random.default_rng(m).integers(0, 16, (n, k))
    packed = torch.from_numpy(ref.pack(codes)).cuda()
    b = np.full((n, 7), 220, np.uint8)
    want = ref.f64(x) @ ref.held(codes, 2.0 ** (b.astype(np.float64) - 127), None, "fp4", 32, k).T
    y = bl.weight_matvec(x.cuda(), packed, torch.from_numpy(b).view(torch.float8_e8m0fnu).cuda(), format="fp4", out_dtype=torch.float32)
    assert np.array_equal(ref.f64(y), want)
    s = torch.full((n, 2), 2.0 ** 90, dtype=torch.bfloat16)
    want = ref.f64(x) @ ref.held(codes, ref.f64(s), None, "int4", 128, k).T
    y = bl.weight_matvec(x.cuda(), packed, s.cuda(), out_dtype=torch.float32)
    assert np.array_equal(ref.f64(y), want)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("fmt,group,zeros", FORMS)
def test_many_rows_on_a_wide_weight(kind, fmt, group, zeros):
    """More than 32 rows of x on 16384 rows of W and more, which has workgroups of its own: exact, as small integers
    times small powers of two are; rows shorter than, as long as and longer than one round of the wavefronts."""
    import torch
    import dense_linear_algebra_potrf_amd as bl
    from tests.test_gpu_layer import make_x
    for i, (m, n, k) in enumerate([(33, 16384, 300), (64, 16401, 512), (65, 16385, 129), (40, 16400, 1500)]):
        announce("weight_matvec wide and many", kind, fmt, group, zeros, m, n, k)
        codes, sc, z, cuda = make_weights(i, n, k, fmt, group, zeros, exact=True)
        x64, x, xs = make_x(i + 40, m, k, kind, exact=True)
        if kind in ("bf16", "f16") and i == 0:
            x[7, 3], x[32, 299] = float("inf"), float("nan")
        with np.errstate(all="ignore"):
            W = ref.held(codes, sc, z, fmt, group, k)
            want = x64 @ W.T
            if kind in ("bf16", "f16") and i == 0:
                want[7] = (ref.f64(x[7]) * W).sum(1)
                want[32] = np.nan
        got = ref.f64(bl.weight_matvec(x, *cuda, format=fmt, group=group, x_scales=xs, out_dtype=torch.float32))
        assert np.array_equal(got, want, equal_nan=True), f"{int((got != want).sum())} of {want.size} differ"


@pytest.mark.parametrize("kind,fmt,group,zeros", [("bf16", "int4", 32, True), ("f8block", "fp4", 32, False), ("f16", "int4", 32, False)])
def test_many_rows_on_a_wide_weight_with_long_rows(kind, fmt, group, zeros):
    """As above with more groups to a row than are held at a time."""
    import torch
    import dense_linear_algebra_potrf_amd as bl
    from tests.test_gpu_layer import make_x
    m, n, k = 34, 16387, 256 * group + 33
    announce("weight_matvec wide, many and long", kind, fmt, group, zeros, m, n, k)
    codes, sc, z, cuda = make_weights(1, n, k, fmt, group, zeros, exact=True)
    x64, x, xs = make_x(2, m, k, kind, exact=True)
    y = bl.weight_matvec(x, *cuda, format=fmt, group=group, x_scales=xs, out_dtype=torch.float32)
    got = ref.f64(y)
    for at in range(0, n, 2048):                    # a part of W at a time in 64 bits
        rows = slice(at, at + 2048)
        W = ref.held(codes[rows], sc[rows], None if z is None else z[rows], fmt, group, k)
        assert np.array_equal(got[:, rows], x64 @ W.T)
