"""Plain fp64 forms of the q/k normalisation with rotation and of its gradients, with the rounding
error that fp32 arithmetic may bring (test infrastructure, like the rest of this package).

Bounds, in units of U = 2^-24.  The norm: squares and sums of at most 8 values in a thread and 5 or
6 joins (14, halved by the square root), root, quotient and two products (6): 16 with the weight.
cos and sin: the angle is reduced in 64 bits, its fraction of a turn rounded to 32 bits (2 pi 2^-26)
and the functions are good to 2 ulp: 4 U each.  A turned value: two products and a sum (2).
The weights' gradients: as if all rows were added one after another, which holds for any order and is far
above the sums that are made; the tests of many rows count those.
"""
import numpy as np

U = 2.0 ** -24
NORM, TRIG = 16, 8


def turn(x, angle, interleaved, back=False):
    """x (..., d); angle (..., rot/2).  Also the sums of magnitudes each result is made of."""
    half = angle.shape[-1]
    c, s = np.cos(angle), np.sin(angle) * (-1 if back else 1)
    y, m = x.copy(), np.abs(x)
    one, two = ((slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else
                (slice(0, half), slice(half, 2 * half)))
    a, b = x[..., one], x[..., two]
    y[..., one], y[..., two] = a * c - b * s, a * s + b * c
    m[..., one] = m[..., two] = np.abs(a) + np.abs(b)
    return y, m


def _unit(x, norm, eps):
    c = {"rms": 1.0 / x.shape[-1], "l2": 1.0, None: 0.0}[norm]
    m = c * (x * x).sum(-1, keepdims=True) + eps
    if norm is None:
        return np.ones_like(m), c
    with np.errstate(divide="ignore"):
        return np.where(m > 0, 1 / np.sqrt(m), 0.0), c


def fwd(x, pos, inv_freq, norm, w, eps, interleaved):
    """x (B, T, H, d), pos (B, T).  Returns (y, its fp32 error bound)."""
    angle = pos[:, :, None, None] * inv_freq
    r, _ = _unit(x, norm, eps)
    y, m = turn(x * r * w, angle, interleaved)
    return y, U * (NORM + TRIG + 2) * m


def bwd(x, dy, pos, inv_freq, norm, w, eps, interleaved):
    """Returns ((dx, dw), (their bounds))."""
    angle = pos[:, :, None, None] * inv_freq
    r, c = _unit(x, norm, eps)
    u, m = turn(dy, angle, interleaved, back=True)
    eu = U * (TRIG + 2) * m
    xn = x * r
    dot = (w * u * xn).sum(-1, keepdims=True)
    edot = (np.abs(w * xn) * (eu + U * (NORM + 16) * np.abs(u))).sum(-1, keepdims=True)
    dx = r * (w * u - c * xn * dot)
    edx = r * (np.abs(w) * eu + c * np.abs(xn) * edot +
               U * (NORM + 4) * (np.abs(w * u) + 2 * c * np.abs(xn * dot)))
    rows = x.shape[0] * x.shape[1] * x.shape[2]
    axes = (0, 1, 2)
    edw = (np.abs(xn) * eu + U * (NORM + 2 + rows) * np.abs(u * xn)).sum(axes)
    return (dx, (u * xn).sum(axes)), (edx, edw)
