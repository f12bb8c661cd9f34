"""Calibration of 4-bit and 8-bit weights with the batched positive-definite solve.

Rounding a group g of a layer's columns changes the layer's output on
its inputs X by E H_gg E^T, E = W_g - Q_g and H = X^T X.  The columns F that are
not rounded yet can take up most of it: with the change of W_g fixed, the change
of W_F that makes the output's squared error least is E (H_FF^-1 H_Fg)^T.  The
columns are cut into blocks of at most a few hundred, H is taken block by block
(its off-diagonal blocks are left out), and one step rounds the same group of
every block (weight_quant, or int8_quant under the channels' scales) and solves
for every block at once (posv: order of F, `group` right-hand sides).

    python -m dense_linear_algebra_potrf_amd.calibrate

runs the low-bit layer from end to end on seeded inputs: the norm that writes
the activations in 8 bits, weights rounded with and without calibration, the
products with them, and the gradient of the norm's weights; then the same with
8-bit integers, between two blocks of a network.
"""
from __future__ import annotations

import argparse
import functools
import sys

import torch

import dense_linear_algebra_potrf_amd as bl


def second_moments(X, block: int, damping: float = 0.01):
    """H of each block of columns, [blocks, block, block] in float32, from inputs X [samples, k]; damping times
    the mean of its diagonal is added to the diagonal."""
    samples, k = X.shape
    if k % block:
        raise ValueError("k must be a multiple of block")
    x = X.float().view(samples, k // block, block).permute(1, 2, 0).contiguous()
    H = torch.bmm(x, x.transpose(1, 2).contiguous())
    diagonal = H.diagonal(dim1=1, dim2=2)
    diagonal += damping * diagonal.mean(1, keepdim=True).clamp(min=1e-30)
    return H


def calibrate_weights(W, H, *, format: str = "int4", group: int | None = None, zeros: bool = False):
    """Round W [n, k] to 4 bits against the second moments H [blocks, block, block] of its inputs.

    Returns what weight_quant(..., values=True) returns, the values in float32.
    block is k / blocks, a multiple of group, and at most 512 + group.
    """
    if group is None:
        group = 128 if format == "int4" else 32
    round_to = functools.partial(bl.weight_quant, format=format, group=group, zeros=zeros, values=True)
    return round_to(_compensated(W, H, group, lambda part: round_to(part)[3]))


@torch.no_grad()
def calibrate_channels(W, H, *, group: int = 64):
    """Round W [n, k] to 8-bit integers with a scale for each channel (row) against the second moments H of its inputs.

    Returns what int8_quant(..., values=True) returns, the values in float32; the
    scales are those of W's own rows.  H and group are as in calibrate_weights.
    """
    scales = bl.int8_quant(W)[1]
    of_blocks = scales.repeat_interleave(H.shape[0])
    Wc = _compensated(W, H, group, lambda part: bl.int8_quant(part, given=of_blocks, values=True)[2])
    return bl.int8_quant(Wc, given=scales, values=True)


def _compensated(W, H, group: int, rounded):
    """W in float32, each group but its block's first moved to take up the rounding of those before it;
    rounded(part) is what the codes of [n blocks, group] columns stand for."""
    n, k = W.shape
    blocks, block = H.shape[0], H.shape[1]
    if blocks * block != k or block % group:
        raise ValueError("H must be blocks of k / blocks columns, a multiple of the group")
    Wc = W.float().clone()
    rows, view = Wc.view(n * blocks, block), Wc.view(n, blocks, block)
    failed = torch.zeros(blocks, dtype=torch.int32, device=W.device)
    for c in range(0, block - group, group):
        part = rows[:, c:c + group]
        E = (part - rounded(part)).view(n, blocks, group).transpose(0, 1).contiguous()
        A = H[:, c + group:, c + group:].contiguous()
        X = H[:, c:c + group, c + group:].contiguous()        # H_Fg, column-major; becomes H_FF^-1 H_Fg
        failed |= bl.posv(A, X, "L")
        view[:, :, c + group:] += torch.bmm(E, X).transpose(0, 1)
    if bool(failed.any()):
        raise ValueError("H is not positive definite")
    return Wc


def output_error(W, values, X) -> float:
    """Relative error of the layer's output on X."""
    want = X.float() @ W.float().t()
    return float(torch.linalg.norm(X.float() @ values.float().t() - want) / torch.linalg.norm(want))


def demo(n: int = 512, k: int = 1024, samples: int = 4096, tokens: int = 4, block: int = 256, seed: int = 0) -> dict:
    """The layer from end to end; returns the errors and outputs that main() prints."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    mix = rand(k, k) / k ** 0.5 + 0.5 * torch.eye(k, device="cuda")        # inputs whose columns are correlated
    W, w = 0.02 * rand(n, k), (1 + 0.1 * rand(k)).bfloat16()
    hidden, residual = (rand(samples, k) @ mix).bfloat16(), rand(samples, k).bfloat16()
    q, scales, h = bl.rmsnorm_quant(hidden, w, residual)
    X = q.float() * scales.float().repeat_interleave(32, 1)[:, :k]         # what the products will see
    H = second_moments(X, block)
    out = {}
    for format, group in (("int4", 64), ("fp4", 32)):
        plain = bl.weight_quant(W, format=format, group=group, values=True)
        tuned = calibrate_weights(W, H, format=format, group=group)
        y = bl.weight_matvec(q[:tokens], *tuned[:3], format=format, group=group, x_scales=scales[:tokens])
        out[format] = {"rounded": output_error(W, plain[3], X), "calibrated": output_error(W, tuned[3], X),
                       "y": y, "want": X[:tokens] @ W.t()}
    # tuning the norm's weights afterwards: the gradient of half the squared error of the 4-bit float layer
    values = tuned[3]
    dv = ((X @ values.t() - X @ W.t()) @ values).bfloat16()
    out["dx"], out["dw"] = bl.rmsnorm_grad(dv, h, w)
    # in 8-bit integers, after a block whose output is normed, gated and added to the scaled residual
    post, gate = (1 + 0.1 * rand(k)).bfloat16(), (0.5 + 0.1 * rand(k)).bfloat16()
    q, scales, h = bl.block_norm(hidden, residual, w, post, gate, residual_scale=0.9, int8=True)
    X = q.float() * scales[:, None]
    plain, tuned = bl.int8_quant(W, values=True), calibrate_channels(W, second_moments(X, block))
    y = bl.int8_matmul(q[:tokens], tuned[0], scales[:tokens], tuned[1])
    out["int8"] = {"rounded": output_error(W, plain[2], X), "calibrated": output_error(W, tuned[2], X),
                   "y": y, "want": X[:tokens] @ W.t()}
    dv = ((X @ tuned[2].t() - X @ W.t()) @ tuned[2]).bfloat16()
    out["block_norm"] = dict(zip(("dy", "dx", "dgate", "dweight", "dpost_weight"),
                                 bl.block_norm_grad(dv, hidden, h, w, post, gate, residual_scale=0.9)))
    return out


def main(argv=None) -> int:
    ap = argparse.ArgumentParser(description="the low-bit layer from end to end on seeded inputs")
    ap.add_argument("--rows", type=int, default=512, help="rows of the weights")
    ap.add_argument("--columns", type=int, default=1024, help="columns of the weights")
    ap.add_argument("--block", type=int, default=256, help="columns whose second moments are kept together")
    a = ap.parse_args(argv)
    out = demo(a.rows, a.columns, block=a.block)
    for format, operator in (("int4", "weight_matvec"), ("fp4", "weight_matvec"), ("int8", "int8_matmul")):
        o = out[format]
        far = float(torch.linalg.norm(o["y"].float() - o["want"]) / torch.linalg.norm(o["want"]))
        print(f"{format}: output error {o['rounded']:.4f} rounded, {o['calibrated']:.4f} calibrated; "
              f"4 tokens through {operator} {far:.4f}", flush=True)
    print(f"norm gradient: |dw| = {float(out['dw'].norm()):.4g}", flush=True)
    print("norms around the block: " + ", ".join(f"|{name}| = {float(out['block_norm'][name].norm()):.4g}"
                                                 for name in ("dweight", "dpost_weight", "dgate")), flush=True)
    return 0


if __name__ == "__main__":
    sys.exit(main())
