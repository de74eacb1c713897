"""Plain 64-bit forms of the selective scan and the residual norm in numpy, token by token, with componentwise error
scales in units of 2^-24: the same computation on absolute values, each 32-bit operation adding what it may be off by.  No
code is shared with the library."""
import numpy as np

from mixer_reference import f64, sigmoid, within  # noqa: F401


def softplus(v):
    return np.maximum(v, 0) + np.log1p(np.exp(-np.abs(v)))


def silu(z):
    """silu(z), silu'(z)."""
    s, r = sigmoid(z), sigmoid(-z)
    return z * s, s * (1 + z * r)


def spread(v, D):
    """[T, G, S] beside the D channels."""
    return np.repeat(v, D // v.shape[1], 1)


def by_group(v, G):
    """[D, S] summed over each group's channels."""
    return v.reshape(G, v.shape[0] // G, -1).sum(1)


def ssm(x, dt, a, b, c, lens, skip=None, z=None, bias=None, use_softplus=False, s0=None, dy=None, dfin=None):
    """(y, fin), or (y, fin, dx, ddt, da, db, dc, dskip, dz, dbias, ds0) with dy; all [.., G, S] for b, c."""
    T, D = x.shape
    G, S = b.shape[1:]
    N = len(lens)
    raw = dt + (0.0 if bias is None else bias)
    step = softplus(raw) if use_softplus else raw
    fb, fc = spread(b, D), spread(c, D)
    h, prev, fin = np.zeros((T, D, S)), np.zeros((T, D, S)), np.zeros((N, D, S))
    t0 = 0
    for i, L in enumerate(lens):
        st = np.zeros((D, S)) if s0 is None else s0[i].copy()
        for t in range(t0, t0 + L):
            prev[t] = st
            st = np.exp(step[t][:, None] * a) * st + (step[t] * x[t])[:, None] * fb[t]
            h[t] = st
        fin[i] = st
        t0 += L
    p = (h * fc).sum(2) + (0.0 if skip is None else skip * x)
    f, df = (1.0, None) if z is None else silu(z)
    y = p * f
    if dy is None:
        return y, fin
    dp = dy * f
    dx, ddt = np.zeros_like(x), np.zeros_like(x)
    da, db, dc, ds0 = np.zeros((D, S)), np.zeros((T, G, S)), np.zeros((T, G, S)), np.zeros((N, D, S))
    end = T
    for i in range(N - 1, -1, -1):
        g = np.zeros((D, S)) if dfin is None else dfin[i].copy()
        for t in range(end - 1, end - 1 - lens[i], -1):
            e = fc[t] * dp[t][:, None] + g
            dc[t] = by_group(dp[t][:, None] * h[t], G)
            db[t] = by_group(e * (step[t] * x[t])[:, None], G)
            du = (e * fb[t]).sum(1)
            g = np.exp(step[t][:, None] * a) * e
            w = g * prev[t]
            da += w * step[t][:, None]
            dx[t] = du * step[t]
            ddt[t] = du * x[t] + (w * a).sum(1)
        ds0[i] = g
        end -= lens[i]
    if skip is not None:
        dx += dp * skip
    if use_softplus:
        ddt *= sigmoid(raw)
    return (y, fin, dx, ddt, da, db, dc, None if skip is None else (dp * x).sum(0), None if z is None else dy * p * df,
            None if bias is None else ddt.sum(0), ds0)


def ssm_scales(x, dt, a, b, c, lens, skip=None, z=None, bias=None, use_softplus=False, s0=None, dy=None, dfin=None):
    """How far the results of ssm() may be off, in units of 2^-24, by first-order bounds:

      raw     1 rounding of the sum
      step    softplus: its derivative times raw's, and 8 of its value (an exponential and a log1p of two last places each)
      decay   |a| times the step's error, the roundings of a log2(e), of the product and of the block's sum (4 of |step a|),
              and 8 for ex2 (2^-22 and the result's rounding)
      others  1 for each product and sum, a sum of n terms n of their absolute sum (a gate's sigmoid 8 + 2 |z|, at most 2 |z|
              for the argument of its exponential)."""
    T, D = x.shape
    G, S = b.shape[1:]
    N = len(lens)
    raw = dt + (0.0 if bias is None else bias)
    step = softplus(raw) if use_softplus else raw
    e_raw = 0.0 * raw if bias is None else np.abs(dt) + np.abs(bias)
    e_step = sigmoid(raw) * e_raw + 8 * step if use_softplus else e_raw
    step = np.abs(step)
    ax, fb, fc = np.abs(x), np.abs(spread(b, D)), np.abs(spread(c, D))
    u, e_u = step * ax, (e_step + step) * ax
    h, eh, prev, e_prev = (np.zeros((T, D, S)) for _ in range(4))
    fin = np.zeros((N, D, S))
    signed = softplus(raw) if use_softplus else raw

    def decay(t):
        d = np.exp(signed[t][:, None] * a)
        return d, np.abs(a) * e_step[t][:, None] + 4 * step[t][:, None] * np.abs(a) + 8

    t0 = 0
    for i, L in enumerate(lens):
        st = np.zeros((D, S)) if s0 is None else np.abs(s0[i])
        er = np.zeros((D, S))
        for t in range(t0, t0 + L):
            prev[t], e_prev[t] = st, er
            d, ed = decay(t)
            er = d * (er + (ed + 1) * st) + (e_u[t] + u[t])[:, None] * fb[t]
            st = d * st + u[t][:, None] * fb[t]
            er = er + st
            h[t], eh[t] = st, er
        fin[i] = er
        t0 += L
    sk = 0.0 if skip is None else np.abs(skip) * ax
    p, e_p = (h * fc).sum(2) + sk, (eh * fc).sum(2) + (S + 2) * ((h * fc).sum(2) + sk)
    if z is None:
        f, df, e_f = 1.0, 0.0, 0.0
    else:
        f, df = (np.abs(v) for v in silu(z))
        e_f = (8 + 2 * np.abs(z)) * f
        s = sigmoid(z)
        df = s * (1 + np.abs(z) * sigmoid(-z))  # a bound: the terms' absolute values
    y = e_p * f + p * e_f + p * f
    if dy is None:
        return y, fin
    ady = np.abs(dy)
    dp, e_dp = ady * f, ady * (e_f + (0.0 if z is None else f))
    e_dz = None if z is None else ady * (e_p * df + p * df * (12 + 4 * np.abs(z)) + 2 * p * df)
    dx, ddt = np.zeros_like(x), np.zeros_like(x)
    db, dc, ds0, da, abs_da = np.zeros((T, G, S)), np.zeros((T, G, S)), np.zeros((N, D, S)), np.zeros((D, S)), np.zeros((D, S))
    terms = 16 + D
    end = T
    abs_ddt = np.zeros_like(x)
    for i in range(N - 1, -1, -1):
        g, eg = (np.zeros((D, S)) if dfin is None else np.abs(dfin[i])), np.zeros((D, S))
        for t in range(end - 1, end - 1 - lens[i], -1):
            q, e_q = dp[t][:, None], (0.0 * dp[t] + e_dp[t])[:, None] if np.ndim(e_dp) else 0.0
            e = fc[t] * q + g
            ee = eg + fc[t] * e_q + e
            dc[t] = by_group(q * eh[t] + e_q * h[t] + terms * q * h[t], G)
            ut, e_ut = u[t][:, None], e_u[t][:, None]
            db[t] = by_group(ee * ut + e * e_ut + terms * e * ut, G)
            du, e_du = (e * fb[t]).sum(1), (ee * fb[t]).sum(1) + S * (e * fb[t]).sum(1)
            d, ed = decay(t)
            g, eg = d * e, d * (ee + (ed + 1) * e)
            w, ew = g * prev[t], eg * prev[t] + g * e_prev[t] + g * prev[t]
            st, e_st = step[t][:, None], e_step[t][:, None]
            da += ew * st + w * e_st + w * st
            abs_da += w * st
            dx[t] = e_du * step[t] + du * e_step[t] + 2 * du * step[t]
            wa, e_wa = (w * np.abs(a)).sum(1), (ew * np.abs(a)).sum(1) + (S + 3) * (w * np.abs(a)).sum(1)
            ddt[t] = e_du * ax[t] + e_wa + 2 * (du * ax[t] + wa)
            abs_ddt[t] = du * ax[t] + wa
        ds0[i] = eg
        end -= lens[i]
    da = da + T * abs_da
    if skip is not None:
        dx = dx + (e_dp + 2 * dp) * np.abs(skip)
    if use_softplus:
        s = sigmoid(raw)
        ddt = s * (ddt + abs_ddt * (10 + 2 * np.abs(raw) + e_raw))
        abs_ddt = abs_ddt * s
    e_skip = None if skip is None else ((e_dp + dp) * ax).sum(0) + T * (dp * ax).sum(0)
    e_bias = None if bias is None else ddt.sum(0) + T * abs_ddt.sum(0)
    return y, fin, dx, ddt, da, db, dc, e_skip, e_dz, e_bias, ds0


# ------------------------------------------------------------------ residual norm
def rn(s, w, eps=1e-5, dy=None, d_res=None):
    """y of the rows s, or (y, ds, dw)."""
    r = 1 / np.sqrt((s * s).mean(1, keepdims=True) + eps)
    n = s * r
    y = n * w
    if dy is None:
        return y
    dn = dy * w
    ds = r * (dn - n * (dn * n).mean(1, keepdims=True)) + (0.0 if d_res is None else d_res)
    return y, ds, (dy * n).sum(0)


def rn_scales(s, w, eps=1e-5, dy=None, d_res=None):
    """In units of 2^-24: the sum of V squares in registers, lanes and warps (at most 32 + 5 + 16 additions of a term) moves
    r by half of its relative error, which with the reciprocal square root is below 40."""
    T = s.shape[0]
    r = 1 / np.sqrt((s * s).mean(1, keepdims=True) + eps)
    n, w = np.abs(s) * r, np.abs(w)
    y = 44 * n * w
    if dy is None:
        return y
    dn = np.abs(dy) * w
    ds = r * (44 * dn + n * 240 * (dn * n).mean(1, keepdims=True)) + (0.0 if d_res is None else np.abs(d_res))
    ds = ds + r * (dn + n * (dn * n).mean(1, keepdims=True))
    return y, ds, (44 + T) * (np.abs(dy) * n).sum(0)
