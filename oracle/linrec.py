"""Plain fp64 forms of the gated linear recurrence and its gradients, token by token, with the
rounding error that fp32 arithmetic may bring (test infrastructure, like the rest of this package).

Each value comes with a bound of the form (accumulated magnitude) x 2^-24: a companion recurrence
counts, for every term that reaches a result, the fp32 operations on its way.
  M_t = a_t M_{t-1} + w_t |x_t|                        (the sum of the terms' magnitudes)
  C_t = a_t (C_{t-1} + k_t M_{t-1}) + k_t w_t |x_t|    (the same, each times its operations)
k_t = 12 + 4 |g_t| per token: the factor exp(g) (2 ulp of the exponential of a base-2 argument whose
rounding is |g| log2(e) half-ulps: 4 + 2 |g| half-ulps, twice where the products of several factors
are formed apart from the terms), the write strength (4), the product, the sum, and the joins of
partial results (4).
"""
import numpy as np

U = 2.0 ** -24


def _k(g):
    return 12 + 4 * np.abs(np.where(np.isfinite(g), g, 0.0))


def segments(B, T, cu=None):
    return [(b * T, (b + 1) * T) for b in range(B)] if cu is None else list(zip(cu[:-1], cu[1:]))


def fwd(x, g, h0, segs, complement=False):
    """x, g: (tokens, D); h0: (N, D).  Returns (o, hT, before, err_o, err_hT, err_before): the
    outputs, the states entering each token, and their fp32 error bounds."""
    a = np.exp(g)
    w = -np.expm1(g) if complement else np.ones_like(g)
    k = _k(g)
    o, before, eo, eb = (np.zeros_like(x) for _ in range(4))
    hT, ehT = h0.copy(), np.zeros_like(h0)
    for n, (t0, t1) in enumerate(segs):
        h, M, C = h0[n].copy(), np.abs(h0[n]), np.zeros_like(h0[n])
        for t in range(t0, t1):
            before[t], eb[t] = h, U * C
            put = w[t] * x[t]
            h = a[t] * h + put
            C = a[t] * (C + k[t] * M) + k[t] * np.abs(put)
            M = a[t] * M + np.abs(put)
            o[t], eo[t] = h, U * C
        hT[n], ehT[n] = h, U * C
    return o, hT, before, eo, ehT, eb


def bwd(x, g, h0, do, dhT, segs, complement=False):
    """Returns ((dx, dg, dh0), (their fp32 error bounds))."""
    _, _, before, _, _, eb = fwd(x, g, h0, segs, complement)
    a = np.exp(g)
    w = -np.expm1(g) if complement else np.ones_like(g)
    k = _k(g)
    if complement:
        eb = eb + U * (np.abs(before) + np.abs(x))
        before = before - x
    dx, dg, edx, edg = (np.zeros_like(x) for _ in range(4))
    dh0, edh0 = dhT.copy(), np.zeros_like(dhT)
    for n, (t0, t1) in enumerate(segs):
        c, M, C = dhT[n].copy(), np.abs(dhT[n]), np.zeros_like(dhT[n])
        for t in range(t1 - 1, t0 - 1, -1):
            e = do[t] + c
            Me = np.abs(do[t]) + M
            Ce = C + 2 * Me
            dx[t], edx[t] = w[t] * e, np.abs(w[t]) * U * (Ce + k[t] * Me)
            c, M, C = a[t] * e, a[t] * Me, a[t] * (Ce + k[t] * Me)
            dg[t] = c * before[t]
            edg[t] = np.abs(before[t]) * U * (C + 4 * M) + np.abs(c) * eb[t]
        dh0[n], edh0[n] = c, U * C
    return (dx, dg, dh0), (edx, edg, edh0)
