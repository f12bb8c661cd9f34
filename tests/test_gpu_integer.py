"""The 8-bit-integer layer operators on the GPU against their definitions in 64 bits
(tests/_integer_ref.py, which derives how far 32 bits may be from them): every
type, odd sizes, strides, masks, extreme values, streams, graphs, and the
operators together."""
from __future__ import annotations

import numpy as np
import pytest

from tests import _integer_ref as ref
from tests._gpu import announce

pytestmark = pytest.mark.gpu

TYPES = ("f32", "f16", "bf16")


def dtype(name):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def rand(seed, *shape):
    import torch
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed))


def held(rows, n, fill=0x55):
    """Codes of n columns in rows of whole 16 bytes and 16 more, all bytes set."""
    import torch
    return torch.full((rows, (n + 15) // 16 * 16 + 16), fill, dtype=torch.int8, device="cuda")


def codes(seed, rows, k, lo=-127, hi=127):
    """Random codes in padded rows, the padding random too."""
    import torch
    g = torch.Generator().manual_seed(seed)
    t = torch.randint(lo, hi + 1, (rows, (k + 15) // 16 * 16), generator=g, dtype=torch.int16).to(torch.int8)
    return t.cuda()[:, :k]


def close(got, want, off, what):
    """got within `off` of want and the rounding of its type; not finite where want is not."""
    import torch
    t = got.dtype
    g = ref.f64(got)
    most = torch.finfo(t).max
    fine = np.isfinite(want) & (np.abs(want) * (1 + ref.half_step(t)) + off < most)
    assert (np.isnan(g) == np.isnan(want)).all(), f"{what}: NaN in other places"
    bound = off + ref.half_step(t) * (np.abs(want) + off) + ref.smallest(t)
    with np.errstate(all="ignore"):
        bad = fine & ~(np.abs(g - want) <= bound)
    assert not bad.any(), f"{what}: {bad.sum()} values, first at {np.argwhere(bad)[0]}: {g[bad][0]} for {want[bad][0]}, {bound[bad][0]} allowed"


# ---------------------------------------------------------------- rounding

def check_quant(x, given=None, values=True, strided=False):
    import torch
    import dense_linear_algebra_potrf_amd as bl
    rows, n = x.shape
    dev = x.cuda()
    if strided:
        wide = torch.full((rows, n + 3), 9.0, dtype=x.dtype, device="cuda")
        wide[:, 1:n + 1] = dev
        dev = wide[:, 1:n + 1]
    out = held(rows, n)
    g = None if given is None else torch.from_numpy(given).cuda()
    q, s, v = bl.int8_quant(dev, given=g, values=values, out=out[:, :n])
    wq, ws = ref.quant(x.float().numpy(), given)
    assert np.array_equal(s.cpu().numpy(), ws, equal_nan=True)
    got = q.cpu().numpy()
    bad = got != wq
    assert not bad.any(), f"{bad.sum()} codes, first at {np.argwhere(bad)[0]}"
    assert bool((out[:, n:] == 0x55).all())
    if values:
        with np.errstate(all="ignore"):
            want = torch.from_numpy(wq.astype(np.float32) * ws[:, None]).to(x.dtype)
        assert torch.equal(torch.nan_to_num(v.cpu(), nan=-7.0), torch.nan_to_num(want, nan=-7.0))
    else:
        assert v is None


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("rows,n", [(1, 1), (3, 7), (70, 100), (9, 250), (33, 500), (5, 1000), (4, 1999), (3, 4099), (2, 6001),
                                    (2, 8192), (3, 12000), (2, 16001), (1, 32768), (3, 40001)])
def test_quant(t, rows, n):
    announce("int8_quant", t, rows, n)
    x = rand(rows + n, rows, n)
    x[rows // 2] *= 37
    check_quant(x.to(dtype(t)), strided=n % 2 == 1)


@pytest.mark.parametrize("t", TYPES)
def test_quant_halves_and_ranges(t):
    """Quotients on a half and next to one, rows of zeros, of one value, subnormal and huge."""
    import torch
    announce("int8_quant halves", t)
    n = 300
    x = torch.zeros(14, n)
    half = torch.arange(n) % 254 - 127 + 0.5
    x[0], x[0, 5] = half, 127.0                     # scale 1, every quotient on a half
    x[1], x[1, 7] = half * 2.0 ** -20, 127 * 2.0 ** -20
    x[2], x[2, 0] = half * (1 + 2.0 ** -20), 127.0  # next to a half
    x[3], x[3, 0] = half * 3, 381.0
    x[5] = -3.0
    x[6] = 2.0 ** -24
    x[7], x[7, 1] = half * 1e-43, 3e-42             # below the smallest scale
    x[8], x[8, 0] = half * 256, 60000.0
    x[9, 17] = 1.0
    x[10] = rand(1, n) * 1e-7
    x[11], x[11, 0] = half * 1.1, 127 * 1.1
    x[12], x[12, 3] = half * 2.0 ** -130, 127 * 2.0 ** -130
    x[13] = rand(2, n) * 1e30 if t != "f16" else rand(2, n) * 1e4
    check_quant(x.to(dtype(t)))


@pytest.mark.parametrize("t", TYPES)
def test_quant_what_is_not_finite(t):
    import torch
    announce("int8_quant not finite", t)
    for n in (65, 3001, 33000):
        x = rand(n, 5, n)
        x[1, n - 1], x[3, 0], x[4, n // 2] = float("nan"), float("inf"), -float("inf")
        check_quant(x.to(dtype(t)))


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("rows,n", [(1, 1), (5, 33), (700, 32), (3, 1001), (2, 40000)])
def test_quant_under_given_scales(t, rows, n):
    announce("int8_quant given", t, rows, n)
    x = rand(n, rows, n)
    given = (0.01 * np.exp(np.random.default_rng(n).standard_normal(rows))).astype(np.float32)
    check_quant(x.to(dtype(t)), given)
    if rows > 4:
        for i, bad in enumerate((0.0, -1.0, np.nan, np.inf, 1e-40)):
            given[i] = bad
        x[5 % rows:, 0], x[5 % rows:, 1], x[5 % rows:, 2] = float("nan"), float("inf"), -float("inf")
        check_quant(x.to(dtype(t)), given, values=False)
    given[:] = 3e38
    check_quant((x.nan_to_num(0, 1, -1) * 60000).to(dtype(t)), given)


def test_quant_refuses():
    import torch
    import dense_linear_algebra_potrf_amd as bl
    announce("int8_quant refusals")
    x = torch.zeros(4, 40, device="cuda")
    with pytest.raises(ValueError, match="given or computed"):
        bl.int8_quant(x, given=torch.ones(4, device="cuda"), scales=torch.ones(4, device="cuda"))
    with pytest.raises(ValueError, match="out must be 4 x 40"):
        bl.int8_quant(x, out=torch.zeros(4, 48, dtype=torch.int8, device="cuda"))
    with pytest.raises(ValueError, match="multiples of 16"):
        bl.int8_quant(x, out=torch.zeros(4, 40, dtype=torch.int8, device="cuda"))
    with pytest.raises(ValueError, match="one device"):
        bl.int8_quant(x, given=torch.ones(4))
    q, s, v = bl.int8_quant(x[:0])
    assert q.shape == (0, 40) and s.shape == (0,) and v is None
    q, _, _ = bl.int8_quant(torch.ones(2, 3, 40, device="cuda"))
    assert q.shape == (2, 3, 40) and bool((q == 127).all())


# ---------------------------------------------------------------- products

def check_matmul(x, w, xs, ws, t, strided=False):
    """y in 32 bits is off by three roundings (the sum's, the scales' product's and their product's); in other
    types by theirs too."""
    import torch
    import dense_linear_algebra_potrf_amd as bl
    m, n = x.shape[0], w.shape[0]
    wide = torch.full((m + 1, n + 5), 7.0, dtype=t, device="cuda")
    y = wide[:m, :n] if strided else torch.full((m, n), 7.0, dtype=t, device="cuda")
    got = bl.int8_matmul(x, w, xs, ws, out=y)
    assert got is y
    want = ref.product(x.cpu().numpy(), w.cpu().numpy()) * ref.f64(xs)[:, None] * ref.f64(ws)
    close(y, want, 3.001 * ref.U * np.abs(want) + 2.0 ** -149, "y")
    assert bool((wide[:m, n:] == 7).all()) and bool((wide[m:] == 7).all())


def scales(seed, m, n):
    import torch
    return 0.01 * torch.exp(rand(seed, m)).cuda(), 0.01 * torch.exp(rand(seed + 1, n)).cuda()


@pytest.mark.parametrize("m", [1, 2, 7, 15, 16, 17, 31, 33, 50, 64, 65, 100, 128, 200, 300])
@pytest.mark.parametrize("n,k", [(1, 1), (3, 15), (33, 16), (40, 129), (70, 1000), (130, 64), (257, 4100), (300, 383), (700, 2500)])
def test_matmul(m, n, k):
    announce("int8_matmul", m, n, k)
    t = dtype(TYPES[(m + n) % 3])
    xs, ws = scales(m, m, n)
    check_matmul(codes(m + k, m, k), codes(n + k + 1, n, k), xs, ws, t, strided=(m + k) % 2 == 1)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("m,n,k", [(1, 9000, 520), (16, 8300, 260), (31, 9000, 130), (60, 9001, 257), (3600, 3700, 200),
                                   (257, 16500, 129), (4097, 2049, 65), (1000, 515, 16384 + 48)])
def test_matmul_large(t, m, n, k):
    announce("int8_matmul large", t, m, n, k)
    xs, ws = scales(m, m, n)
    check_matmul(codes(m, m, k), codes(n, n, k), xs, ws, dtype(t))


@pytest.mark.parametrize("m", [1, 40, 70, 300])
def test_matmul_sums_are_exact(m):
    """Every code -128 in the longest rows that are served: sums of 2^31 - 2^14, and with one code more
    or less each bit of 24; out in 32 bits with scales of one."""
    import torch
    import dense_linear_algebra_potrf_amd as bl
    announce("int8_matmul extreme sums", m)
    k, n = (1 << 17) - 1, 20
    x = torch.full((m, k + 1), -128, dtype=torch.int8, device="cuda")[:, :k]
    w = torch.full((n, k + 1), -128, dtype=torch.int8, device="cuda")[:, :k]
    one = lambda c: torch.ones(c, device="cuda")  # noqa: E731
    y = bl.int8_matmul(x, w, one(m), one(n), out_dtype=torch.float32)
    assert bool((y == float(k * 16384)).all())
    w[1::2] = 127
    y = bl.int8_matmul(x, w, one(m), one(n), out_dtype=torch.float32)
    assert bool((y[:, 1::2] == float(np.float32(-k * 128 * 127))).all()) and bool((y[:, ::2] == float(k * 16384)).all())
    x, w = codes(1, m, 1024, -128, 127), codes(2, n, 1024, -128, 127)   # below 2^24: no rounding
    y = bl.int8_matmul(x, w, one(m), one(n), out_dtype=torch.float32)
    assert np.array_equal(ref.f64(y), ref.product(x.cpu().numpy(), w.cpu().numpy()))


@pytest.mark.parametrize("m", [3, 40, 150])
@pytest.mark.parametrize("t", TYPES)
def test_matmul_scales_of_any_kind(m, t):
    """Scales that are zero, not finite, subnormal or whose product leaves the range of 32 bits: y is what the
    definition says; rows of zeros stay zero under every finite scale."""
    import torch
    announce("int8_matmul scales", m, t)
    n, k = 50, 70
    x, w = codes(5, m, k), codes(6, n, k)
    x[2] = 0
    xs, ws = scales(7, m, n)
    for i, v in enumerate((0.0, 1e-40, 1e30, 1e-30, float("nan"), float("inf"), 3e38, 1e-20, -2.0, 1e-38)):
        ws[3 * i] = v
    xs[0], xs[1], xs[2] = 1e-30, 1e20, 3e38
    import dense_linear_algebra_potrf_amd as bl
    y = bl.int8_matmul(x, w, xs, ws, out_dtype=dtype(t))
    with np.errstate(all="ignore"):
        sums = ref.product(x.cpu().numpy(), w.cpu().numpy())
        want = sums * ref.f64(xs)[:, None] * ref.f64(ws)
    fine = np.isfinite(want)
    g = ref.f64(y)
    assert (np.isnan(g) == np.isnan(want)).all()
    top = torch.finfo(dtype(t)).max
    over = np.abs(want) > top * (1 + torch.finfo(dtype(t)).eps)
    assert (np.abs(g[over]) == np.inf).all() and (np.sign(g[over]) == np.sign(want[over])).all()
    inside = fine & (np.abs(want) < top * (1 - torch.finfo(dtype(t)).eps))
    e = 3.001 * ref.U + ref.half_step(dtype(t))
    assert (np.abs(g - want)[inside] <= (e * 1.001 * np.abs(want) + 2.0 ** -149 + ref.smallest(dtype(t)))[inside]).all()
    assert (g[2][np.isfinite(ref.f64(ws))] == 0).all()


def test_matmul_padding_may_hold_anything():
    import torch
    import dense_linear_algebra_potrf_amd as bl
    announce("int8_matmul padding")
    for m in (1, 16, 33, 64, 65, 300):
        for k in (1, 17, 127, 130, 1000):
            kp = (k + 15) // 16 * 16
            x = torch.full((m, kp + 16), 99, dtype=torch.int8, device="cuda")
            w = torch.full((45, kp), -77, dtype=torch.int8, device="cuda")
            x[:, :k], w[:, :k] = codes(m, m, k), codes(k, 45, k)
            xs, ws = scales(m, m, 45)
            check_matmul(x[:, :k], w[:, :k], xs, ws, torch.bfloat16)
    y = bl.int8_matmul(x[:0, :k], w[:, :k], xs[:0], ws)
    assert y.shape == (0, 45)


def test_matmul_offsets_beyond_32_bits():
    """W past 2^31 bytes and y past 2^32 elements."""
    import torch
    import dense_linear_algebra_potrf_amd as bl
    announce("int8_matmul beyond 2^32")
    n, k = 20000, 131056
    w = torch.zeros(n, k, dtype=torch.int8, device="cuda")
    w[-40:] = codes(1, 40, k)
    x = codes(2, 70, k)
    xs, ws = scales(3, 70, n)
    for m in (1, 20, 64, 70):
        y = bl.int8_matmul(x[:m], w, xs[:m], ws, out_dtype=torch.float32)
        want = ref.product(x[:m].cpu().numpy(), w[-40:].cpu().numpy()) * ref.f64(xs[:m])[:, None] * ref.f64(ws[-40:])
        close(y[:, -40:], want, 3.001 * ref.U * np.abs(want), "y")
        assert not y[:, :-40].any()
    del w
    m = n = 66000
    x, w = codes(4, m, 16), codes(5, n, 16)
    xs, ws = scales(6, m, n)
    y = bl.int8_matmul(x, w, xs, ws)
    for rows in (slice(0, 3), slice(m - 3, m), slice(33000, 33002)):
        want = ref.product(x[rows].cpu().numpy(), w.cpu().numpy()) * ref.f64(xs[rows])[:, None] * ref.f64(ws)
        close(y[rows], want, 3.001 * ref.U * np.abs(want), "y")


def test_matmul_refuses():
    import torch
    import dense_linear_algebra_potrf_amd as bl
    announce("int8_matmul refusals")
    x, w, s = codes(1, 4, 32), codes(2, 5, 48), torch.ones(5, device="cuda")
    with pytest.raises(ValueError, match="x has 32 columns and w 48"):
        bl.int8_matmul(x, w, s[:4], s)
    with pytest.raises(ValueError, match="x_scales must be"):
        bl.int8_matmul(x, w[:, :32], s, s)
    with pytest.raises(TypeError, match="w_scales must be"):
        bl.int8_matmul(x, w[:, :32], s[:4], s.half())
    with pytest.raises(TypeError, match="out must be"):
        bl.int8_matmul(x, w[:, :32], s[:4], s, out_dtype=torch.float64)
    with pytest.raises(ValueError, match="out must be 4 x 5"):
        bl.int8_matmul(x, w[:, :32], s[:4], s, out=torch.zeros(4, 6, device="cuda"))
    with pytest.raises(ValueError, match="one device"):
        bl.int8_matmul(x, w[:, :32].cpu(), s[:4], s)
    with pytest.raises(bl.BatchlasError, match="2\\^17"):
        t = torch.zeros(2, 1 << 17, dtype=torch.int8, device="cuda")
        bl.int8_matmul(t, t, s[:2], s[:2])


# ---------------------------------------------------------------- norms around a block

WIDTHS = [(1, 1), (6, 7), (40, 100), (12, 250), (18, 500), (6, 1000), (6, 2047), (4, 4096), (6, 5001), (4, 8192), (2, 12000),
          (4, 16384), (2, 20001), (1, 32768)]


def norm_inputs(seed, t, rows, n, post, gates, flat=False):
    w = (1 + 0.2 * rand(seed + 2, n)).to(t).cuda()
    p = (1 + 0.2 * rand(seed + 3, n)).to(t).cuda() if post else None
    g = rand(seed + 4, gates, n).to(t).cuda() if gates else None
    return rand(seed, rows, n).to(t).cuda(), (2 * rand(seed + 1, rows, n)).to(t).cuda(), w, p, g[0] if gates and flat else g


def f64s(*ts):
    return [None if t is None else ref.f64(t) for t in ts]


def check_norm(y, x, w, p, g, c, eps, int8, h, v, s, rows=None):
    with np.errstate(all="ignore"):
        wh, wv, eh, ev = ref.block_norm(*f64s(y, x, w, p, g), c, eps)
    if rows is not None:
        wh, wv, eh, ev, h, v = wh[rows], wv[rows], eh[rows], ev[rows], h[rows], v[rows]
        s = None if s is None else s[rows]
    close(h, wh, eh, "h")
    if not int8:
        close(v, wv, ev, "v")
        return
    q, s = ref.f64(v), ref.f64(s)
    top = np.abs(wv).max(1)
    assert (np.abs(s - np.maximum(top / 127, 2.0 ** -126)) <= ev.max(1) / 127 + ref.U * s).all()
    # half a step, and what v and the scale may be off
    off = s[:, None] / 2 * (1 + 1e-6) + ev + (np.abs(q) * ev.max(1, keepdims=True)) / 127
    assert (np.abs(q * s[:, None] - wv) <= off).all()
    assert (np.abs(q).max(1) == np.where(top > 2.0 ** -126, 127, np.abs(q).max(1))).all()


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("rows,n", WIDTHS)
@pytest.mark.parametrize("post,int8", [(True, False), (True, True), (False, False), (False, True)])
def test_block_norm(t, rows, n, post, int8):
    import torch
    import dense_linear_algebra_potrf_amd as bl
    announce("block_norm", t, rows, n, post, int8)
    gates = {0: 0, 1: 1, 2: rows, 3: rows // 2 if rows % 2 == 0 else 1}[(n + rows + post) % 4]
    y, x, w, p, g = norm_inputs(n, dtype(t), rows, n, post, gates, flat=gates == 1)
    out = held(rows, n) if int8 else torch.full((rows, n + 3), 7.0, dtype=dtype(t), device="cuda")
    v, s, h = bl.block_norm(y, x, w, p, g, residual_scale=0.7, eps=1e-5, int8=int8, out=out[:, :n])
    check_norm(y, x, w, p, g, float(np.float32(0.7)), 1e-5, int8, h, v, s)
    assert bool((out[:, n:] == (0x55 if int8 else 7)).all())
    if not int8:
        assert s is None


@pytest.mark.parametrize("t", TYPES)
def test_block_norm_in_place_and_strided(t):
    import torch
    import dense_linear_algebra_potrf_amd as bl
    announce("block_norm in place", t)
    rows, n = 12, 333
    y, x, w, p, g = norm_inputs(1, dtype(t), rows, n, True, 3)
    want = bl.block_norm(y, x, w, p, g)
    for name in ("x", "y"):
        a, b = y.clone(), x.clone()
        v, _, h = bl.block_norm(a, b, w, p, g, residual_out=b if name == "x" else a)
        assert torch.equal(h, want[2]) and torch.equal(v, want[0])
        assert torch.equal(b if name == "x" else a, want[2])
    wide = lambda m: torch.cat([m, m, m], 1)[:, n:2 * n]  # noqa: E731
    v, _, h = bl.block_norm(wide(y), wide(x), w, p, wide(g), out=torch.zeros_like(wide(y)), residual_out=torch.zeros_like(wide(y)))
    assert torch.equal(h, want[2]) and torch.equal(v, want[0])
    v, _, h = bl.block_norm(y.view(3, 4, n), x.view(3, 4, n), w, p, g.view(3, 1, n))
    assert v.shape == (3, 4, n) and torch.equal(h.view(rows, n), want[2]) and torch.equal(v.view(rows, n), want[0])


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("n", [60, 700, 5000, 30000])
def test_block_norm_masks_and_ranges(t, n):
    """Rows of zeros, of tiny and of huge values next to others; what is not finite stays in its row."""
    import torch
    import dense_linear_algebra_potrf_amd as bl
    announce("block_norm ranges", t, n)
    rows = 9
    small, big = (1e-6, 200.0) if t == "f16" else (1e-30, 1e25)
    y, x, w, p, _ = norm_inputs(3, dtype(t), rows, n, True, 0)
    y[0] = x[0] = 0
    y[1], x[1] = y[1] * small, x[1] * small
    y[2], x[2] = y[2] * big, x[2] * big
    y[3], x[3] = y[3] * small, x[3] * big
    y[4] = 0
    x[5] = 0
    x[6, n // 2] = float("nan")
    y[7, n - 1] = float("inf")
    for int8 in (False, True):
        for post in (p, None):
            v, s, h = bl.block_norm(y, x, w, post, eps=1e-6, int8=int8)
            check_norm(y, x, w, post, None, 1.0, 1e-6, int8, h, v, s, rows=[0, 1, 2, 3, 4, 5, 8])
            if int8:
                assert bool(torch.isnan(s[6:8]).all()) and not v[6:8].any() and bool(torch.isfinite(s[[0, 1, 2, 8]]).all())
            else:
                assert bool(torch.isnan(v[6]).all()) and bool(torch.isnan(v[7]).any())
    # no eps: unit rows from any finite values but zero
    v, _, h = bl.block_norm(y[1:4], x[1:4], w, p, eps=0.0)
    check_norm(y[1:4], x[1:4], w, p, None, 1.0, 0.0, False, h, v, None)


def test_block_norm_refuses():
    import torch
    import dense_linear_algebra_potrf_amd as bl
    announce("block_norm refusals")
    y, x, w, p, g = norm_inputs(1, torch.float16, 6, 50, True, 4)
    with pytest.raises(ValueError, match="gate must have 50 columns"):
        bl.block_norm(y, x, w, p, g)
    with pytest.raises(ValueError, match="gate must have 50 columns"):
        bl.block_norm(y, x, w, p, g[:3, :49])
    with pytest.raises(TypeError, match="gate must be"):
        bl.block_norm(y, x, w, p, g[:3].float())
    with pytest.raises(TypeError, match="weight must be"):
        bl.block_norm(y, x, w.float())
    with pytest.raises(ValueError, match="residual must be"):
        bl.block_norm(y, x[:5], w)
    with pytest.raises(ValueError, match="scales are for int8"):
        bl.block_norm(y, x, w, scales=torch.ones(6, device="cuda"))
    with pytest.raises(bl.BatchlasError, match="eps must be"):
        bl.block_norm(y, x, w, eps=-1.0)
    with pytest.raises(bl.BatchlasError, match="residual_scale"):
        bl.block_norm(y, x, w, residual_scale=float("inf"))
    with pytest.raises(ValueError, match="dgate needs a gate"):
        bl.block_norm_grad(y, y, x, w, dgate=w)
    with pytest.raises(ValueError, match="dpost_weight needs"):
        bl.block_norm_grad(y, y, x, w, dpost_weight=w.float())
    with pytest.raises(TypeError, match="dgate must be"):
        bl.block_norm_grad(y, y, x, w, p, g[:3], dgate=g[:3].bfloat16())
    with pytest.raises(bl.BatchlasError, match="workspace_bytes"):
        bl.block_norm_grad(y, y, x, w, p, g[:3], workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    v, _, h = bl.block_norm(y[:0], x[:0], w, p, g)
    assert v.shape == h.shape == (0, 50)


# ---------------------------------------------------------------- their gradient

GRAD_WIDTHS = [(1, 1), (6, 7), (48, 100), (30, 250), (30, 500), (36, 1000), (30, 2047), (12, 4096), (6, 5001), (6, 8192),
               (6, 12000), (4, 16384)]


def grad_inputs(seed, t, rows, n, post, gates, dh, flat=False):
    y, h, w, p, g = norm_inputs(seed, t, rows, n, post, gates, flat)
    dv = rand(seed + 5, rows, n).to(t).cuda()
    return dv, y, h, w, p, g, rand(seed + 6, rows, n).to(t).cuda() if dh else None


NAMES = ("dy", "dx", "dgate", "dweight", "dpost_weight")


def check_grad(inputs, c, eps, got, rows=None):
    dv, y, h, w, p, g, dh = f64s(*inputs)
    with np.errstate(all="ignore"):
        want = ref.block_norm_grad(dv, y, h, w, p, g, dh, c, eps)
    for name, t in zip(NAMES, got):
        if name not in want:
            assert t is None, name
        elif rows is None:
            close(t, *want[name], name)
        elif name in ("dy", "dx"):
            close(t[rows], want[name][0][rows], want[name][1][rows], name)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("rows,n", GRAD_WIDTHS)
@pytest.mark.parametrize("gate", ["none", "channel", "sequence", "token"])
def test_block_norm_grad(t, rows, n, gate):
    import torch
    import dense_linear_algebra_potrf_amd as bl
    announce("block_norm_grad", t, rows, n, gate)
    gates = {"none": 0, "channel": 1, "sequence": max(1, rows // 3) if rows % 3 == 0 else 1, "token": rows}[gate]
    post, dh = (n + rows) % 3 != 0 or gate == "token", (n + len(gate)) % 2 == 0
    inputs = grad_inputs(n, dtype(t), rows, n, post, gates, dh, flat=gate == "channel")
    got = bl.block_norm_grad(*inputs, residual_scale=0.7, eps=1e-5)
    check_grad(inputs, float(np.float32(0.7)), 1e-5, got)
    if gate == "channel":
        assert got[2].dtype is torch.float32 and got[2].shape == (n,)
    elif gate != "none":
        assert got[2].dtype is dtype(t)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("rows,n,gates", [(1700, 65, 17), (1700, 65, 1), (1700, 65, 425), (1700, 65, 1700), (1700, 65, 340),
                                          (6000, 130, 4), (2100, 1100, 3), (2100, 1100, 700), (9000, 40, 2), (2060, 4100, 2),
                                          (2060, 2300, 1030), (2060, 2300, 0), (4200, 9000, 2), (40000, 24, 8)])
@pytest.mark.parametrize("post", [True, False])
def test_block_norm_grad_long(t, rows, n, gates, post):
    """Runs within a gate and of several gates, the last ones shorter, in all shapes."""
    import dense_linear_algebra_potrf_amd as bl
    announce("block_norm_grad long", t, rows, n, gates, post)
    inputs = grad_inputs(rows, dtype(t), rows, n, post, gates, gates % 2 == 0)
    got = bl.block_norm_grad(*inputs, eps=1e-6)
    check_grad(inputs, 1.0, 1e-6, got)


def test_block_norm_grad_what_is_asked_for():
    import torch
    import dense_linear_algebra_potrf_amd as bl
    announce("block_norm_grad parts")
    for rows, n, gates in ((700, 96, 2), (700, 96, 350), (40, 5000, 1), (40, 16000, 40)):
        inputs = grad_inputs(3, torch.bfloat16, rows, n, True, gates, True)
        want = bl.block_norm_grad(*inputs)
        for mask in range(8):
            asked = dict(zip(("dgate", "dweight", "dpost_weight"), (None if mask >> i & 1 else False for i in range(3))))
            got = bl.block_norm_grad(*inputs, **asked)
            for name, a, b in zip(NAMES, got, want):
                if name in asked and asked[name] is False:
                    assert a is None
                else:
                    assert torch.equal(a, b), (name, mask)
        f = bl.block_norm_grad(*inputs, dgate=torch.empty(gates, n, device="cuda"))[2]
        assert f.dtype is torch.float32 and torch.equal(f.bfloat16(), want[2])
    # no rows: sums of nothing
    dv, y, h, w, p, g, dh = grad_inputs(3, torch.bfloat16, 4, 100, True, 2, True)
    dy, dx, dg, dw, dp = bl.block_norm_grad(dv[:0], y[:0], h[:0], w, p, g, dh[:0])
    assert dy.shape == dx.shape == (0, 100) and not dg.any() and not dw.any() and not dp.any() and dg.shape == (2, 100)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("n", [100, 101, 3000, 3003, 5005, 16000, 16003])
def test_block_norm_grad_in_place_and_strided(t, n):
    import torch
    import dense_linear_algebra_potrf_amd as bl
    announce("block_norm_grad in place", t, n)
    rows = 12
    inputs = grad_inputs(5, dtype(t), rows, n, True, 3, True)
    want = bl.block_norm_grad(*inputs)
    places = {"dv": 0, "y": 1, "h": 2, "dh": 6}
    for a in places:
        for b in places:
            if a == b:
                continue
            ins = [i.clone() for i in inputs]
            got = bl.block_norm_grad(*ins, dy=ins[places[a]], dx=ins[places[b]])
            assert got[0] is ins[places[a]] and all(torch.equal(x, y) for x, y in zip(got, want)), (a, b)
    wide = lambda m: torch.cat([m, m, m], 1)[:, n:2 * n]  # noqa: E731
    dv, y, h, w, p, g, dh = inputs
    got = bl.block_norm_grad(wide(dv), wide(y), wide(h), w, p, wide(g), wide(dh), dy=wide(y), dx=wide(y), dgate=wide(g))
    assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("n", [60, 700, 5000, 16000])
def test_block_norm_grad_masks_and_ranges(t, n):
    import torch
    import dense_linear_algebra_potrf_amd as bl
    announce("block_norm_grad ranges", t, n)
    rows = 8
    small, big = (1e-6, 200.0) if t == "f16" else (1e-30, 1e25)
    for post in (True, False):
        dv, y, h, w, p, g, dh = grad_inputs(7, dtype(t), rows, n, post, 2, True)
        y[0] = h[0] = 0
        y[1], h[1] = y[1] * small, h[1] * small
        y[2], h[2] = y[2] * big, h[2] * big
        dv[3] = dh[3] = 0
        got = bl.block_norm_grad(dv, y, h, w, p, g, dh, eps=1e-6)
        check_grad((dv, y, h, w, p, g, dh), 1.0, 1e-6, got, rows=[0, 1, 2, 3, 4, 5, 6, 7] if t == "f16" else [0, 3, 4, 5, 6, 7])
        assert not got[1][3].any()
        for m in (1, 2):
            with np.errstate(all="ignore"):
                want = ref.block_norm_grad(*f64s(dv, y, h, w, p, g, dh), 1.0, 1e-6)
            close(got[1][m:m + 1], want["dx"][0][m:m + 1], want["dx"][1][m:m + 1], "dx")
        # what is not finite stays in its row and in the sums it goes into
        dv[5, n // 2], y[6, 0] = float("nan"), float("inf")
        bad = bl.block_norm_grad(dv, y, h, w, p, g, dh, eps=1e-6)
        for a, b in zip(bad[:2], got[:2]):
            assert torch.equal(a[[0, 1, 2, 3, 4, 7]], b[[0, 1, 2, 3, 4, 7]])
        assert torch.equal(bad[2][0], got[2][0])
        assert bool(torch.isnan(bad[1][5]).all())


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("n", [60, 700, 5000, 16000])
@pytest.mark.parametrize("of_rows,of_gradients", [(1e12, 1e27), (1e-12, 1e-27)])
def test_block_norm_grad_products_leave_the_range(t, n, of_rows, of_gradients):
    """Neither the rows' squares, the gradients nor the results leave 32 bits, but the rows' products with the gradients."""
    import dense_linear_algebra_potrf_amd as bl
    announce("block_norm_grad products", t, n, of_rows)
    dv, y, h, w, p, g, dh = grad_inputs(11, dtype(t), 6, n, True, 2, True)
    inputs = dv * of_gradients, y * of_rows, h * of_rows, w, p, g, dh * of_gradients
    check_grad(inputs, 1.0, 0.0, bl.block_norm_grad(*inputs, eps=0.0))


# ---------------------------------------------------------------- together

def layer_state(seed, m=37, n=200, k=1000):
    import torch
    b = torch.bfloat16
    s = {key: rand(seed + i, m, k).to(b).cuda() for i, key in enumerate(("y", "x", "dv", "dh"))}
    s["w"], s["p"] = rand(seed + 8, k).to(b).cuda(), rand(seed + 9, k).to(b).cuda()
    s["g"], s["W"] = rand(seed + 10, 1, k)[0].to(b).cuda(), rand(seed + 11, n, k).to(b).cuda()
    return s


def layer_step(bl, s, stream=None, buffers=None):
    """Between two blocks: the norms, the product with rounded weights, and the gradient of the norms."""
    kw = dict(stream=stream)
    wq, ws, _ = bl.int8_quant(s["W"], **kw)
    q, qs, h = bl.block_norm(s["y"], s["x"], s["w"], s["p"], s["g"], residual_scale=0.5, int8=True, **kw)
    out = bl.int8_matmul(q, wq, qs, ws, **kw)
    return [wq, ws, q, qs, h, out, *bl.block_norm_grad(s["dv"], s["y"], h, s["w"], s["p"], s["g"], s["dh"], residual_scale=0.5, **kw)]


def raw(ts):
    import torch
    return [t.contiguous().view(torch.uint8).clone() for t in ts]


@pytest.mark.parametrize("m,n,k", [(1, 200, 1000), (37, 200, 1000), (300, 130, 520)])
def test_layer_together(m, n, k):
    """A block's norms, its product and its gradient as they would be used: the product against 64 bits
    from the codes, each other part against its definition."""
    import torch
    import dense_linear_algebra_potrf_amd as bl
    announce("integer layer", m, n, k)
    s = layer_state(m, m, n, k)
    wq, ws, q, qs, h, out, *grads = layer_step(bl, s)
    check_norm(s["y"], s["x"], s["w"], s["p"], s["g"], 0.5, 1e-6, True, h, q, qs)
    want = ref.product(q.cpu().numpy(), wq.cpu().numpy()) * ref.f64(qs)[:, None] * ref.f64(ws)
    close(out, want, 3.001 * ref.U * np.abs(want), "y")
    check_grad((s["dv"], s["y"], h, s["w"], s["p"], s["g"], s["dh"]), 0.5, 1e-6, grads)
    # what the layer stands for: its two roundings move an output by at most half a step of each factor
    v = ref.block_norm(*f64s(s["y"], s["x"], s["w"], s["p"], s["g"]), 0.5, 1e-6)[1]
    W = ref.f64(s["W"])
    step = 0.51 * (ref.f64(qs)[:, None] * np.abs(W).sum(1) + ref.f64(ws) * np.abs(v).sum(1)[:, None]) \
        + 0.26 * k * ref.f64(qs)[:, None] * ref.f64(ws)
    assert (np.abs(ref.f64(out) - v @ W.T) <= step + 2.0 ** -8 * np.abs(v @ W.T)).all()


def test_runs_alike_on_another_stream_and_in_a_graph():
    """Two runs, a run on another stream and every replay of a graph (with eager work between the replays)
    give the same bits."""
    import torch
    import dense_linear_algebra_potrf_amd as bl
    announce("integer layer: streams and graph")
    for m, n, k in ((37, 200, 1000), (400, 140, 700)):
        s = layer_state(0, m, n, k)
        want = raw(layer_step(bl, s))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, raw(layer_step(bl, s))))
        side = torch.cuda.Stream()
        late = torch.zeros(1 << 22, device="cuda")
        other = layer_state(0, m, n, k)
        for t in (other["x"], other["y"]):
            t.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):               # inputs written on the side stream, after a delay
            for _ in range(20):
                late.add_(1)
            other["x"].copy_(s["x"])
            other["y"].copy_(s["y"])
        got = layer_step(bl, other, stream=side)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, raw(got)))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = layer_step(bl, other)
        for rep in range(4):
            fresh = layer_state(10 * rep, m, n, k)
            for key in other:
                other[key].copy_(fresh[key])
            for t in out:
                t.zero_()
            torch.cuda.synchronize()
            eager = raw(layer_step(bl, fresh))
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(eager, raw(out))), f"replay {rep}"


def test_what_a_call_on_a_stream_allocates_belongs_to_it():
    """Workspaces and outputs of calls that wait on a side stream are not handed out again to work that
    runs meanwhile on the current one."""
    import torch
    import dense_linear_algebra_potrf_amd as bl
    announce("integer layer: allocations on a side stream")
    s = layer_state(5)
    want = raw(layer_step(bl, s))
    late, side = torch.zeros(1 << 24, device="cuda"), torch.cuda.Stream()
    sizes = sorted({t.numel() for t in want} | {bl.block_norm_grad_workspace(torch.bfloat16, 37, 1000, 1)})
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(100):
            late.add_(1)
    got = layer_step(bl, s, stream=side)
    keep = [torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda") for size in sizes for _ in range(8)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, raw(got)))
    assert all(bool((t == 0xFF).all()) for t in keep)


def test_norm_offsets_beyond_32_bits():
    """The last rows of arrays past 2^32 bytes, and a gate past 2^31."""
    import torch
    import dense_linear_algebra_potrf_amd as bl
    announce("integer layer beyond 2^32 bytes")
    n, rows = 16384, (1 << 17) + 6                  # 2^31 elements and some
    tall = torch.zeros(rows, n, dtype=torch.bfloat16, device="cuda")
    y, x, w, p, g = norm_inputs(1, torch.bfloat16, 6, n, True, 6)
    tall[-6:] = y
    q, s, _ = bl.int8_quant(tall)
    wq, _ = ref.quant(y.float().cpu().numpy())
    assert np.array_equal(q[-6:].cpu().numpy(), wq) and not q[:-6].view(torch.int32).any()
    del q
    gate = torch.zeros_like(tall)
    gate[-6:] = g
    v, _, h = bl.block_norm(tall, tall, w, p, gate)
    check_norm(y, y, w, p, g, 1.0, 1e-6, False, h[-6:], v[-6:], None)
    assert not v[:-6].view(torch.int32).any()
    del h
    dv = v                                           # zeros above
    got = bl.block_norm_grad(dv, tall, tall, w, p, gate, eps=1e-2)
    want = bl.block_norm_grad(dv[-6:], y, y, w, p, g, eps=1e-2)
    for a, b in zip(got[:3], want[:3]):
        assert torch.equal(a[-6:], b)
        assert not a[:-6].view(torch.int32).any()


@pytest.mark.parametrize("n", [40, 1030])
def test_more_rows_than_a_launch_has_groups(n):
    """Rows beyond 2^20 workgroups are those of a call on them alone."""
    import torch
    import dense_linear_algebra_potrf_amd as bl
    announce("integer layer, many rows", n)
    rows = (1 << 20) * (16 if n == 40 else 1) + 21
    parts = [slice(0, 40), slice(rows - 40, rows)]
    y = torch.randn(rows, n, device="cuda", dtype=torch.float16)
    w, p, g = (torch.randn(n, device="cuda", dtype=torch.float16) for _ in range(3))
    q, s, _ = bl.int8_quant(y)
    again = bl.int8_quant(y, given=s)[0]
    assert torch.equal(again, q)
    v, _, h = bl.block_norm(y, y, w, p, g, residual_scale=0.5)
    c, cs, _ = bl.block_norm(y, y, w, p, g, residual_scale=0.5, int8=True, residual_out=h.clone())
    for part in parts:
        for a, b in zip((q, s), bl.int8_quant(y[part])):
            assert torch.equal(a[part], b)
        for a, b in zip((v, None, h), bl.block_norm(y[part], y[part], w, p, g, residual_scale=0.5)):
            assert b is None or torch.equal(a[part], b)
        for a, b in zip((c, cs), bl.block_norm(y[part], y[part], w, p, g, residual_scale=0.5, int8=True)):
            assert torch.equal(a[part], b)
    dy, dx = bl.block_norm_grad(v, y, h, w, p, g, dgate=False, dweight=False, dpost_weight=False)[:2]
    for part in parts:
        for a, b in zip((dy, dx), bl.block_norm_grad(v[part], y[part], h[part], w, p, g)):
            assert torch.equal(a[part], b)


def test_calls_at_once_on_two_streams():
    """Steps that run beside each other on two streams, each with what it allocates, give the bits of one alone."""
    import torch
    import dense_linear_algebra_potrf_amd as bl
    announce("integer layer: two streams at once")
    states = [layer_state(40 + i, m=700 + 13 * i, n=900, k=2000) for i in range(2)]
    want = [raw(layer_step(bl, s)) for s in states]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = [layer_step(bl, s, stream=stream) for s, stream in zip(states, streams)]
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(x, y) for x, y in zip(a, raw(b)))


@pytest.mark.parametrize("shape", [(1000,), (3, 1000), (2, 5, 1000), (0, 1000), (2, 0, 1000)])
def test_any_number_of_dimensions(shape):
    """Rows of any shape, of a width that leaves padding, through the whole layer."""
    import torch
    import dense_linear_algebra_potrf_amd as bl
    announce("integer layer: dimensions", shape)
    rows, k = int(np.prod(shape[:-1])), shape[-1]
    s = layer_state(60, m=max(rows, 1), n=48, k=k)
    flat = {key: s[key][:rows] for key in ("y", "x", "dv", "dh")}
    wq, ws, _ = bl.int8_quant(s["W"])
    q, qs, h = bl.block_norm(flat["y"].view(shape), flat["x"].view(shape), s["w"], s["p"], s["g"], int8=True)
    z = bl.int8_matmul(q, wq, qs, ws)
    assert q.shape == h.shape == shape and qs.shape == (rows,) and z.shape == (*shape[:-1], 48)
    q2, qs2, h2 = bl.block_norm(flat["y"], flat["x"], s["w"], s["p"], s["g"], int8=True)
    assert torch.equal(q.reshape(rows, k), q2) and torch.equal(qs, qs2) and torch.equal(h.view(rows, k), h2)
    assert torch.equal(z.view(rows, 48), bl.int8_matmul(q2, wq, qs2, ws))
    got = bl.block_norm_grad(*(flat[key].view(shape) for key in ("dv", "y")), h, s["w"], s["p"], s["g"], flat["dh"].view(shape))
    want = bl.block_norm_grad(flat["dv"], flat["y"], h2, s["w"], s["p"], s["g"], flat["dh"])
    assert got[0].shape == got[1].shape == shape
    assert all(torch.equal(a.reshape(b.shape), b) for a, b in zip(got, want))
    c, cs, values = bl.int8_quant(flat["x"].view(shape), values=True)
    assert c.shape == values.shape == shape and cs.shape == (rows,)
