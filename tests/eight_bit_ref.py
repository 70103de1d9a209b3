"""Reference forms of the operators around the mixers, in 64 bits (numpy), and their bounds.

Bounds count roundings, each at most half a step (U = 2^-24 in fp32, 2^-8 in bf16, relative to
the value).  A norm's value takes at most: one rounding each for the residual's sum, the
weight's offset and two products; half of the relative error of the sum of squares, which goes
through at most 32 + 10 additions and a product with a rounded 1 / D; an inverse square root
good to two units in the last place, 4 U.  NORM = 40 U is above their sum (31 U).  A gate adds e^-z (a few units of U; from the base-2 hardware
exponential and the fast division in bf16, 2^-21 and the exponent's own rounding), a sum, a
division and a product: GATED = 64 U in fp32, 2^-17 in bf16.
"""
import numpy as np
import torch

U = 2.0 ** -24
NORM = 40 * U
GATED = {torch.float32: 64 * U, torch.bfloat16: 2.0 ** -17}
HALF_STEP = {torch.float32: U, torch.bfloat16: 2.0 ** -8}
TINY = 127 * 2.0 ** -126


def f64(t):
    return t.detach().cpu().double().numpy()


def add_rmsnorm(x, w, residual, eps, offset):
    h = f64(x) if residual is None else f64(x) + f64(residual)
    y = h * (offset + f64(w)) / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    return y, h


def gated_rmsnorm(x, z, w, eps):
    a, b = f64(x), f64(z)
    y = a * f64(w) / np.sqrt((a * a).mean(-1, keepdims=True) + eps)
    with np.errstate(over="ignore"):
        y = y * b / (1 + np.exp(-b))
    return y.reshape(a.shape[0], -1)


def quotients(y):
    """(127 y / max|y|, scale) of the rows; a row of zeros has the smallest scale."""
    largest = np.maximum(np.abs(y).max(-1, keepdims=True), TINY)
    return 127 * y / largest, largest[:, 0] / 127


def assert_close(got, want, rel, dtype):
    """Every element within its type's half step and `rel` of itself (values under the normal
    range: of the smallest normal)."""
    err = np.abs(f64(got) - want)
    bound = (HALF_STEP[dtype] * (1 + rel) + rel) * np.maximum(np.abs(want), 2.0 ** -126)
    assert np.isfinite(f64(got)).all()
    assert (err <= bound).all(), float((err / bound).max())


def assert_codes(q, scale, y, rel):
    """Codes are the nearest to 127 y / max|y|, but for the error of both: 254 rel."""
    want, s = quotients(y)
    off = np.abs(f64(q) - want)
    assert (off <= 0.5 + 254 * rel + 2.0 ** -15).all(), float(off.max())
    assert (np.abs(f64(scale) - s) <= (rel + 4 * U) * s).all()


def product(a, a_scale, w, w_scale, bias, dtype):
    """The exact sum, then fp32 steps in the documented order: bits, not a bound."""
    sums = (a.cpu().double() @ w.cpu().double().t()).float()        # < 2^53: exact, one rounding
    out = sums * a_scale.cpu()[:, None] * w_scale.cpu()
    if bias is not None:
        out = out + bias.cpu().float()
    return out.to(dtype)
