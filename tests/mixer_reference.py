"""Plain 64-bit forms of the token-mixer operators, token by token in numpy, with componentwise scales for
rounding bounds: the same computation on absolute values, which bounds how far a chain of correctly ordered
32-bit operations can be off per unit of relative rounding.  No code is shared with the library."""
import numpy as np


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def half_step(dtype):
    import torch
    return torch.finfo(dtype).eps / 2


def sigmoid(x):
    e = np.exp(-np.abs(x))
    return np.where(x >= 0, 1 / (1 + e), e / (1 + e))


def act(kind, p):
    """(act(p), act'(p))."""
    if kind in (None, "none"):
        return p, np.ones_like(p)
    s, r = sigmoid(p), sigmoid(-p)
    return (s, s * r) if kind == "sigmoid" else (p * s, s * (1 + p * r))


# ------------------------------------------------------------------ gated linear recurrence
def glr_gate(g, logsigmoid=False, lower_bound=None, complement=False):
    """(a, m, dlog a / dg)."""
    if logsigmoid:
        a, rest, slope = sigmoid(g), sigmoid(-g), sigmoid(-g)
    elif lower_bound is not None:
        lg = lower_bound * sigmoid(g)
        a, rest, slope = np.exp(lg), -np.expm1(lg), lower_bound * sigmoid(g) * sigmoid(-g)
    else:
        a, rest, slope = np.exp(g), -np.expm1(g), np.ones_like(g)
    return a, (rest if complement else np.ones_like(g)), slope


def glr_fwd(x, g, lens, s0=None, **gate):
    a, m, _ = glr_gate(g, **gate)
    D = x.shape[1]
    h, fin, t = np.zeros_like(x), np.zeros((len(lens), D)), 0
    for i, L in enumerate(lens):
        st = np.zeros(D) if s0 is None else s0[i].copy()
        for t in range(t, t + L):
            with np.errstate(invalid="ignore"):
                st = a[t] * st + m[t] * x[t]
            h[t] = st
        t = sum(lens[:i + 1])
        fin[i] = st
    return h, fin


def glr_bwd(x, g, lens, dh, s0=None, dfin=None, complement=False, **gate):
    """(dx, dg, ds0)."""
    a, m, slope = glr_gate(g, complement=complement, **gate)
    D, N = x.shape[1], len(lens)
    prev, dx, dg, ds0 = np.zeros_like(x), np.zeros_like(x), np.zeros_like(x), np.zeros((N, D))
    for i, L in enumerate(lens):
        t0 = sum(lens[:i])
        st = np.zeros(D) if s0 is None else s0[i].copy()
        for t in range(t0, t0 + L):
            prev[t] = st
            st = a[t] * st + m[t] * x[t]
        e = np.zeros(D) if dfin is None else dfin[i].copy()
        for t in range(t0 + L - 1, t0 - 1, -1):
            e = e + dh[t]
            dx[t] = m[t] * e
            e = a[t] * e
            dg[t] = e * (prev[t] - x[t] if complement else prev[t]) * slope[t]
        ds0[i] = e
    return dx, dg, ds0


def glr_scales(x, g, lens, s0=None, dh=None, dfin=None, complement=False, **gate):
    """Running error scales of (h, fin), and of (dx, dg, ds0) with dh: every step adds one unit of its absolute
    value to the error, which decays along with the state, E_t = a_t E_{t-1} + |h|_t."""
    a, m, slope = glr_gate(g, complement=complement, **gate)
    x, slope = np.abs(x), np.abs(slope)
    D, N = x.shape[1], len(lens)
    H, fin = np.zeros_like(x), np.zeros((N, D))
    dx, dg, ds0 = np.zeros_like(x), np.zeros_like(x), np.zeros((N, D))
    for i, L in enumerate(lens):
        t0 = sum(lens[:i])
        v = np.zeros(D) if s0 is None else np.abs(s0[i])
        E, prev, Eprev = np.zeros(D), np.zeros((L, D)), np.zeros((L, D))
        for k in range(L):
            prev[k], Eprev[k] = v, E
            v = a[t0 + k] * v + m[t0 + k] * x[t0 + k]
            E = a[t0 + k] * E + v
            H[t0 + k] = E
        fin[i] = E
        if dh is None:
            continue
        e, E = np.zeros(D) if dfin is None else np.abs(dfin[i]), np.zeros(D)
        for k in range(L - 1, -1, -1):
            t = t0 + k
            e = e + np.abs(dh[t])
            E = E + e
            dx[t] = m[t] * E
            e, E = a[t] * e, a[t] * (E + e)
            inner = prev[k] + (x[t] if complement else 0.0)
            dg[t] = (E * inner + e * Eprev[k] + e * inner) * slope[t]
        ds0[i] = E
    return (H, fin) if dh is None else (H, fin, dx, dg, ds0)


# ------------------------------------------------------------------ group norm
def gn(x, w, b, z, dy=None, center=True, activation="silu", eps=1e-5):
    """y, or (y, dx, dw, db, dz) with dy.  w, b [V] or [H, V]."""
    mu = x.mean(-1, keepdims=True) if center else 0.0
    c = x - mu
    r = 1 / np.sqrt((c * c).mean(-1, keepdims=True) + eps)
    n = c * r
    p = n * w + (0.0 if b is None else b)
    if z is None:
        y, da = act(activation, p)
    else:
        f, df = act(activation, z)
        y = p * f
    if dy is None:
        return y
    dp, dz = (dy * da, None) if z is None else (dy * f, dy * p * df)
    over = (0, 1) if w.ndim == 1 else (0,)
    dw, db = (dp * n).sum(over), dp.sum(over)
    dn = dp * w
    dx = dn - n * (dn * n).mean(-1, keepdims=True)
    if center:
        dx = dx - dn.mean(-1, keepdims=True)
    return y, r * dx, dw, (None if b is None else db), dz


def gn_scales(x, w, b, z, dy, center=True, activation="silu", eps=1e-5):
    """Scales of (y, dx, dw, db, dz): each intermediate replaced by a bound of its terms' absolute values.  An
    activation changes an error by at most 1.1 times it (silu' <= 1.1), its derivative by half of it."""
    V = x.shape[-1]
    mu = x.mean(-1, keepdims=True) if center else 0.0
    r = 1 / np.sqrt(((x - mu) ** 2).mean(-1, keepdims=True) + eps)
    # the mean of V terms is off by their absolute mean per unit of rounding, and r with the square of the row's size
    size = np.abs(x) + (np.abs(x).mean(-1, keepdims=True) if center else 0.0)
    cond = 1 + (size * size).mean(-1, keepdims=True) * r * r if center else 1.0
    n = size * r * cond
    p = n * np.abs(w) + (0.0 if b is None else np.abs(b))
    if z is None:
        y = 1.1 * p
        dp, dz = np.abs(dy) * (1.1 + 0.5 * p), None
    else:
        f = np.abs(act(activation, z)[0]) + (1.0 if activation == "none" else 0.1)
        y = p * f
        dp, dz = np.abs(dy) * f, np.abs(dy) * p * 1.1
    over = (0, 1) if w.ndim == 1 else (0,)
    dn = dp * np.abs(w)
    dx = dn + n * (dn * n).mean(-1, keepdims=True) + dn.mean(-1, keepdims=True)
    return y, r * cond * dx, (dp * n).sum(over), dp.sum(over), dz


# ------------------------------------------------------------------ short convolution
def sconv(x, w, b, lens, s0=None, dy=None, dfin=None, activation="silu", absolute=False):
    """(y, fin), or (y, fin, dx, dw, db, ds0) with dy; absolute: their scales."""
    D, W = w.shape
    N = len(lens)
    s0 = np.zeros((N, W - 1, D)) if s0 is None else s0
    y, fin = np.zeros_like(x), np.zeros((N, W - 1, D))
    dx, ds0, dw, db = np.zeros_like(x), np.zeros((N, W - 1, D)), np.zeros((D, W)), np.zeros(D)
    for i, L in enumerate(lens):
        t0 = sum(lens[:i])
        line = np.concatenate([s0[i], x[t0:t0 + L]])
        fin[i] = line[L:]
        dline = np.zeros_like(line)
        if dy is not None and dfin is not None:
            dline[L:] += np.abs(dfin[i]) if absolute else dfin[i]
        for t in range(L):
            win = line[t:t + W].T  # [D, W]
            if absolute:
                p = (np.abs(w) * np.abs(win)).sum(1) + (0.0 if b is None else np.abs(b))
                y[t0 + t], da = 1.1 * p, 1.1 + 0.5 * p
                d = None if dy is None else np.abs(dy[t0 + t]) * da
                wt, win = np.abs(w), np.abs(win)
            else:
                p = (w * win).sum(1) + (0.0 if b is None else b)
                y[t0 + t], da = act(activation, p)
                d = None if dy is None else dy[t0 + t] * da
                wt = w
            if d is None:
                continue
            dline[t:t + W] += (wt * d[:, None]).T
            dw += win * d[:, None]
            db += d
        ds0[i], dx[t0:t0 + L] = dline[:W - 1], dline[W - 1:]
    if dy is None:
        return y, fin
    return y, fin, dx, dw, (None if b is None else db), ds0


def within(name, got, ref, dtype, units, scale):
    """got is ref rounded once to dtype, after 32-bit operations that may be off by units * 2^-24 of scale; a value
    below bf16's and fp32's normal range may flush."""
    if ref is None:
        assert got is None, name
        return
    got = f64(got)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    bad = ~np.isfinite(ref)
    assert np.array_equal(np.isnan(got), np.isnan(ref)) and np.array_equal(got[bad & ~np.isnan(ref)], ref[bad & ~np.isnan(ref)]), name
    off = np.abs(np.where(bad, 0.0, got) - np.where(bad, 0.0, ref))
    h = half_step(dtype)
    fp32 = units * 2.0 ** -24 * np.where(bad, 0.0, scale)
    most = h * np.abs(np.where(bad, 0.0, ref)) + (1 + h) * fp32 + 2.0 ** -126
    worst = np.max(off / most) if off.size else 0.0
    assert worst <= 1.0, f"{name}: {worst:.3f} of the bound"
