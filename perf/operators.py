"""The cases on which the low-bit layer operators are measured, with their plain forms.

Four operators serve a layer whose weights are held in 4 bits (calibrated with
the library's batched positive-definite solves) and whose activations are
handed over in 8 bits:

  rmsnorm_quant   root-mean-square norm of x + residual, written in 8 bits with scales
  rmsnorm_grad    its gradient: of the inputs and of the norm's weights
  weight_quant    weights to 4-bit codes with group scales, and the values they stand for
  weight_matvec   products of a few tokens with such weights

`run` computes a case in elementary 32-bit torch operations, or, where `own` is
set, calls the library's operators on the same inputs.  `exact` gives the
outputs from the definitions in 64 bits, from one formula per operator.
"""
import math

import torch

own = False

EPS = 1e-6                       # the norm's epsilon
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
E4M3_MAX, E2M1_MAX = 448.0, 6.0  # largest magnitudes of the 8-bit and 4-bit floats
TINY = 2.0 ** -126               # smallest scale that is stored
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one token of a decoding step, residual added, scales per 32 columns: latency
        dict(name="norm_token", op="rmsnorm_quant", rows=1, n=4096, dtype="bf16", scale="block", residual=True),
        # a long prompt through a wide model's norm
        dict(name="norm_prompt", op="rmsnorm_quant", rows=8192, n=8192, dtype="bf16", scale="block", residual=True),
        # an odd width without residual, one scale a row (row-scaled 8-bit products follow)
        dict(name="norm_odd", op="rmsnorm_quant", rows=1023, n=5001, dtype="f16", scale="row", residual=False),
        # a training step's norm gradient, the residual path's gradient added
        dict(name="grad_batch", op="rmsnorm_grad", rows=8192, n=4096, dtype="bf16", dh=True),
        # the same in 32 bits at an odd width, first norm of a stack: no other path
        dict(name="grad_odd", op="rmsnorm_grad", rows=517, n=1537, dtype="f32", dh=False),
        # a square projection to 4-bit integers with zero points, as the calibration rounds it
        dict(name="quant_int", op="weight_quant", n=4096, k=4096, dtype="f32", format="int4", group=128, zeros=True),
        # a wide projection to 4-bit floats with power-of-two scales
        dict(name="quant_float", op="weight_quant", n=16384, k=8192, dtype="bf16", format="fp4", group=32, zeros=False),
        # one token against a square projection: the smallest product of a decoding step
        dict(name="matvec_token", op="weight_matvec", m=1, n=4096, k=4096, x="bf16", format="int4", group=128, zeros=False),
        # one token against a wide projection with zero points
        dict(name="matvec_wide", op="weight_matvec", m=1, n=28672, k=8192, x="f16", format="int4", group=64, zeros=True),
        # a few sequences, 8-bit activations from the norm, 4-bit float weights
        dict(name="matvec_floats", op="weight_matvec", m=4, n=16384, k=4096, x="f8block", format="fp4", group=32, zeros=False),
        # a batch of sequences decoding together, small groups
        dict(name="matvec_batch", op="weight_matvec", m=64, n=8192, k=8192, x="bf16", format="int4", group=32, zeros=False),
        # odd sizes, row-scaled 8-bit activations
        dict(name="matvec_odd", op="weight_matvec", m=7, n=5003, k=2500, x="f8row", format="int4", group=128, zeros=True),
    ]


def _log(rng, lo, hi, most=None):
    """A size from lo to hi, spread over its logarithm, at most `most`; every other one a multiple of 64."""
    hi = hi if most is None else max(lo, min(hi, most))
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5 and v > 64:
        v -= v % 64
    return v + 1 if v == 3072 else max(lo, v)


def draw(rng):
    op = rng.choice(("rmsnorm_quant", "rmsnorm_grad", "weight_quant", "weight_matvec", "weight_matvec"))
    if op == "rmsnorm_quant":
        n = _log(rng, 64, 16384)
        return dict(op=op, rows=_log(rng, 1, 8192, (1 << 26) // n), n=n, dtype=rng.choice(("bf16", "f16", "f32")),
                    scale=rng.choice(("block", "row")), residual=rng.random() < 0.7)
    if op == "rmsnorm_grad":
        n = _log(rng, 64, 16384)
        return dict(op=op, rows=_log(rng, 1, 8192, (1 << 25) // n), n=n, dtype=rng.choice(("bf16", "f16", "f32")),
                    dh=rng.random() < 0.6)
    form = rng.choice(("int4", "int4", "fp4"))
    group = rng.choice((32, 64, 128)) if form == "int4" else 32
    zeros = form == "int4" and rng.random() < 0.5
    k = _log(rng, 256, 16384)
    if op == "weight_quant":
        return dict(op=op, n=_log(rng, 64, 16384, (1 << 27) // k), k=k, dtype=rng.choice(("bf16", "f16", "f32")),
                    format=form, group=group, zeros=zeros)
    return dict(op=op, m=_log(rng, 1, 64), n=_log(rng, 64, 28672, (1 << 27) // k), k=k,
                x=rng.choice(("bf16", "f16", "f8block", "f8row")), format=form, group=group, zeros=zeros)


def _size(name):
    return 4 if name == "f32" else 2


def work(case):
    if case["op"] == "rmsnorm_quant":
        e = case["rows"] * case["n"]
        s = _size(case["dtype"])
        scales = case["rows"] * (-(-case["n"] // 32) if case["scale"] == "block" else 4)
        return {"bytes": e * (s * (3 if case["residual"] else 1) + 1) + scales + case["n"] * s, "flops": 6 * e}
    if case["op"] == "rmsnorm_grad":
        e = case["rows"] * case["n"]
        s = _size(case["dtype"])
        return {"bytes": e * s * (4 if case["dh"] else 3) + case["n"] * (s + 4), "flops": 12 * e}
    groups = case["n"] * -(-case["k"] // case["group"])
    held = case["n"] * -(-case["k"] // 2) + groups * ((1 if case["format"] == "fp4" else 2) + (1 if case["zeros"] else 0))
    if case["op"] == "weight_quant":
        return {"bytes": 2 * case["n"] * case["k"] * _size(case["dtype"]) + held, "flops": 5 * case["n"] * case["k"]}
    x = case["m"] * case["k"] * (1 if case["x"].startswith("f8") else 2)
    return {"bytes": held + x + 2 * case["m"] * case["n"], "flops": 2 * case["m"] * case["n"] * case["k"]}


# ---------------------------------------------------------------- inputs

def _activations(g, rows, n, dev):
    """Hidden states: most columns near 1, a few in two hundred an order of magnitude larger."""
    x = torch.randn(rows, n, generator=g, device=dev)
    outlier = torch.rand(n, generator=g, device=dev) < 0.005
    return x * torch.where(outlier, 12.0, 1.0)


def _weights(g, n, k, dev):
    """Projection weights: normal, rows of different gain, a little off centre."""
    gain = torch.exp(0.3 * torch.randn(n, 1, generator=g, device=dev)) * 0.02
    return (torch.randn(n, k, generator=g, device=dev) + 0.05) * gain


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    s = dict(case)
    if case["op"] in ("rmsnorm_quant", "rmsnorm_grad"):
        rows, n, dt = case["rows"], case["n"], TYPES[case["dtype"]]
        s["w"] = (1 + 0.2 * torch.randn(n, generator=g, device=dev)).to(dt)
        if case["op"] == "rmsnorm_quant":
            s["x"] = _activations(g, rows, n, dev).to(dt)
            if rows > 4:
                s["x"][rows // 2] = 0        # a padding token
            s["r"] = s["hout"] = None
            if case["residual"]:
                s["r"] = (2 * _activations(g, rows, n, dev)).to(dt)
                if rows > 4:
                    s["r"][rows // 2] = 0
                s["hout"] = torch.empty(rows, n, dtype=dt, device=dev)
            # the buffers that a serving loop keeps
            s["q"] = torch.empty(rows, n, dtype=torch.float8_e4m3fn, device=dev)
            s["qs"] = torch.empty(rows, -(-n // 32), dtype=torch.float8_e8m0fnu, device=dev) if case["scale"] == "block" \
                else torch.empty(rows, dtype=torch.float32, device=dev)
        else:
            s["h"] = _activations(g, rows, n, dev).to(dt)
            s["dy"] = (0.01 * torch.randn(rows, n, generator=g, device=dev)).to(dt)
            s["dh"] = (0.01 * torch.randn(rows, n, generator=g, device=dev)).to(dt) if case["dh"] else None
        return s
    n, k, group = case["n"], case["k"], case["group"]
    if case["op"] == "weight_quant":
        s["W"] = _weights(g, n, k, dev).to(TYPES[case["dtype"]])
        return s
    m, groups = case["m"], -(-k // group)
    # codes as rounding normal weights gives them, two a byte, rows padded to 16 bytes
    row = -(-(-(-k // 2)) // 16) * 16
    if case["format"] == "int4":
        nib = lambda: (torch.randn(n, row, generator=g, device=dev) * 2.4 + 8).round_().clamp_(0, 15).to(torch.uint8)  # noqa: E731
        s["scales"] = (0.006 * torch.exp(0.3 * torch.randn(n, groups, generator=g, device=dev))).to(torch.bfloat16)
    else:
        nib = lambda: torch.randint(0, 16, (n, row), generator=g, device=dev, dtype=torch.uint8)  # noqa: E731
        s["scales"] = (torch.randint(118, 122, (n, groups), generator=g, device=dev, dtype=torch.uint8)).view(torch.float8_e8m0fnu)
    s["codes"] = nib() | (nib() << 4)
    s["z"] = torch.randint(5, 11, (n, groups), generator=g, device=dev, dtype=torch.uint8) if case["zeros"] else None
    x = _activations(g, m, k, dev)
    s["xs"] = None
    if case["x"] == "f8block":
        e = torch.randint(117, 122, (m, -(-k // 32)), generator=g, device=dev, dtype=torch.uint8)
        s["xs"] = e.view(torch.float8_e8m0fnu)
        x = (x * 30).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    elif case["x"] == "f8row":
        s["xs"] = 0.02 * (1 + torch.rand(m, generator=g, device=dev))
        x = (x * 30).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    else:
        x = x.to(TYPES[case["x"]])
    s["act"] = x
    s["y"] = torch.empty(m, n, dtype=torch.float16 if case["x"] == "f16" else torch.bfloat16, device=dev)
    return s


# ---------------------------------------------------------------- plain forms, in 32 bits

def _pieces(v, size):
    """[rows, n] -> [rows, pieces, size], the last piece filled up with zeros."""
    rows, n = v.shape
    pad = -n % size
    if pad:
        v = torch.nn.functional.pad(v, (0, pad))
    return v.view(rows, -1, size)


def _exponent(big, most):
    """The least e with big <= most * 2^e, from -127 to 127."""
    frac, e = torch.frexp(big)                       # big = frac 2^e, 1/2 <= frac < 1
    top, te = math.frexp(most)
    e = e - te + (frac > top).int()
    return torch.where(big == 0, torch.full_like(e, -127), e.clamp(-127, 127))


def _plain_norm(s):
    x = s["x"].float()
    h = x if s["r"] is None else x + s["r"].float()
    v = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * s["w"].float()
    out = {}
    if s["scale"] == "block":
        b = _pieces(v, 32)
        e = _exponent(b.abs().amax(2), E4M3_MAX)
        q = torch.ldexp(b, -e[:, :, None]).reshape(v.shape[0], -1)[:, :v.shape[1]]
        out["scales"] = (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
    else:
        scale = (v.abs().amax(1) / E4M3_MAX).clamp(min=TINY)
        q = v / scale[:, None]
        out["scales"] = scale
    out["q"] = q.to(torch.float8_e4m3fn)
    if s["r"] is not None:
        out["h"] = h.to(s["x"].dtype)
    return out


def _plain_grad(s):
    h, g = s["h"].float(), s["dy"].float()
    gw = g * s["w"].float()
    rs = torch.rsqrt((h * h).mean(1, keepdim=True) + EPS)
    dx = rs * (gw - h * (rs * rs * (gw * h).mean(1, keepdim=True)))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return {"dx": dx.to(s["h"].dtype), "dweight": (g * h * rs).sum(0)}


def _plain_quant(s):
    W = s["W"].float()
    b = _pieces(W, s["group"])
    out = {}
    if s["format"] == "fp4":
        e = _exponent(b.abs().amax(2), E2M1_MAX)
        t = torch.ldexp(b, -e[:, :, None])
        a = t.abs()
        step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
        val = torch.ldexp(torch.copysign(torch.round(a / step) * step, t), e[:, :, None])
        out["scales"] = (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
    else:
        if s["zeros"]:
            lo, hi = b.amin(2).clamp(max=0), b.amax(2).clamp(min=0)
            scale = ((hi - lo) / torch.full_like(hi, 15)).to(torch.bfloat16).float().clamp(min=TINY)
            z = torch.round(-lo / scale).clamp(0, 15)
            out["zeros"] = z.to(torch.uint8)
            z = z[:, :, None]
            q = (torch.round(b / scale[:, :, None]) + z).clamp(0, 15) - z
        else:
            big = b.abs().amax(2)
            scale = (big / torch.full_like(big, 7)).to(torch.bfloat16).float().clamp(min=TINY)
            q = torch.round(b / scale[:, :, None]).clamp(-8, 7)
        val = q * scale[:, :, None]
        out["scales"] = scale.to(torch.bfloat16)
    out["values"] = val.reshape(W.shape[0], -1)[:, :W.shape[1]].to(s["W"].dtype)
    return out


def _held(s, dtype):
    """The weights that the codes stand for, [n, k]."""
    c, k = s["codes"], s["k"]
    nib = torch.stack((c & 15, c >> 4), 2).view(c.shape[0], -1)[:, :k]
    per = lambda t: t.to(dtype).repeat_interleave(s["group"], 1)[:, :k]  # noqa: E731
    if s["format"] == "fp4":
        table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=dtype, device=c.device)
        return table[nib.int()] * per(s["scales"])
    return (nib.to(dtype) - (8 if s["z"] is None else per(s["z"]))) * per(s["scales"])


def _active(s, dtype):
    """The activations that x stands for, [m, k]."""
    x = s["act"].to(dtype)
    if s["x"] == "f8block":
        return x * s["xs"].to(dtype).repeat_interleave(32, 1)[:, :s["k"]]
    return x * s["xs"].to(dtype)[:, None] if s["x"] == "f8row" else x


def _plain_matvec(s):
    return (_active(s, torch.float32) @ _held(s, torch.float32).t()).to(s["y"].dtype)


def run(s):
    op = s["op"]
    if not own:
        return {"rmsnorm_quant": _plain_norm, "rmsnorm_grad": _plain_grad, "weight_quant": _plain_quant,
                "weight_matvec": _plain_matvec}[op](s)
    import dense_linear_algebra_potrf_amd as bl
    if op == "weight_matvec":
        return bl.weight_matvec(s["act"], s["codes"], s["scales"], s["z"], format=s["format"], group=s["group"],
                                x_scales=s["xs"], out=s["y"])
    if op == "rmsnorm_quant":
        q, scales, h = bl.rmsnorm_quant(s["x"], s["w"], s["r"], eps=EPS, scale=s["scale"], out=s["q"], scales=s["qs"],
                                        residual_out=s["hout"])
        return {"q": q, "scales": scales} if h is None else {"q": q, "scales": scales, "h": h}
    if op == "rmsnorm_grad":
        dx, dweight = bl.rmsnorm_grad(s["dy"], s["h"], s["w"], s["dh"], eps=EPS)
        return {"dx": dx, "dweight": dweight}
    codes, scales, zeros, values = bl.weight_quant(s["W"], format=s["format"], group=s["group"], zeros=s["zeros"], values=True)
    out = {"scales": scales, "values": values}
    if zeros is not None:
        out["zeros"] = zeros
    return out


# ---------------------------------------------------------------- the definitions in 64 bits

def _least_power(big, most):
    e = torch.ceil(torch.log2(big / most))
    e = e + (big > most * torch.exp2(e)).double()                 # log2's rounding, either way
    e = e - (big <= most * torch.exp2(e - 1)).double()
    return torch.where(big == 0, torch.full_like(e, -127.0), e.clamp(-127, 127))


def _nearest(v, mantissa, lowest):
    """v rounded to a float with that many mantissa bits and that lowest exponent, ties to even."""
    _, e = torch.frexp(v)
    step = torch.exp2(((e - 1).clamp(min=lowest) - mantissa).double())
    return torch.round(v / step) * step


def _by_group(v, size, f):
    """f of each piece of `size` columns, as one value a piece."""
    return torch.stack([f(p) for p in v.split(size, 1)], 1)


def _spread(v, size, n):
    return v.repeat_interleave(size, 1)[:, :n]


def exact(case, seed):
    s = prepare(case, seed)
    d = torch.float64
    if case["op"] == "weight_matvec":
        return _active(s, d) @ _held(s, d).t()
    if case["op"] == "rmsnorm_quant":
        h = s["x"].to(d) + (0 if s["r"] is None else s["r"].to(d))
        v = h / torch.sqrt(h.pow(2).sum(1, keepdim=True) / case["n"] + EPS) * s["w"].to(d)
        if case["scale"] == "block":
            scale = torch.exp2(_least_power(_by_group(v, 32, lambda p: p.abs().amax(1)), E4M3_MAX))
            q = v / _spread(scale, 32, case["n"])
        else:
            scale = (v.abs().amax(1) / E4M3_MAX).clamp(min=TINY)
            q = v / scale[:, None]
        out = {"q": _nearest(q, 3, -6), "scales": scale}
        if s["r"] is not None:
            out["h"] = h
        return out
    if case["op"] == "rmsnorm_grad":
        h, g, w, n = s["h"].to(d), s["dy"].to(d), s["w"].to(d), case["n"]
        mean = h.pow(2).sum(1, keepdim=True) / n + EPS
        dot = (g * w * h).sum(1, keepdim=True)
        dx = g * w / mean.sqrt() - h * dot / (n * mean ** 1.5)
        return {"dx": dx if s["dh"] is None else dx + s["dh"].to(d), "dweight": (g * h / mean.sqrt()).sum(0)}
    W, k, group = s["W"].to(d), case["k"], case["group"]
    if case["format"] == "fp4":
        scale = torch.exp2(_least_power(_by_group(W, group, lambda p: p.abs().amax(1)), E2M1_MAX))
        wide = _spread(scale, group, k)
        return {"scales": scale, "values": _nearest(W / wide, 1, 0) * wide}
    # the scale is stored in 16 bits and the codes go by the stored one, so the definition rounds it too
    if case["zeros"]:
        lo = _by_group(W, group, lambda p: p.amin(1).clamp(max=0))
        hi = _by_group(W, group, lambda p: p.amax(1).clamp(min=0))
        scale = _nearest((hi - lo) / 15, 7, -126).clamp(min=TINY)
        zero = torch.round(-lo / scale).clamp(0, 15)
        wide, z = _spread(scale, group, k), _spread(zero, group, k)
        code = (torch.round(W / wide) + z).clamp(0, 15)
        return {"scales": scale, "values": (code - z) * wide, "zeros": zero}
    scale = _nearest(_by_group(W, group, lambda p: p.abs().amax(1)) / 7, 7, -126).clamp(min=TINY)
    wide = _spread(scale, group, k)
    return {"scales": scale, "values": torch.round(W / wide).clamp(-8, 7) * wide}
