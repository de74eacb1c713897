"""The 64-bit forms that the GPU tests compare with: against central differences and closed values (CPU)."""
import numpy as np
import pytest

import block_reference as R


def _draw(lens, D, S, G, seed, **opts):
    rng = np.random.default_rng(seed)
    T, N = sum(lens), len(lens)
    v = dict(x=rng.normal(size=(T, D)), dt=rng.normal(size=(T, D)), a=-np.exp(rng.normal(size=(D, S))),
             b=rng.normal(size=(T, G, S)), c=rng.normal(size=(T, G, S)), s0=rng.normal(size=(N, D, S)))
    if opts.get("skip", True):
        v["skip"] = rng.normal(size=D)
    if opts.get("z", True):
        v["z"] = rng.normal(size=(T, D))
    if opts.get("bias", True):
        v["bias"] = rng.normal(size=D)
    if not opts.get("use_softplus", True):
        v["dt"] = np.abs(v["dt"])
    return v, rng.normal(size=(T, D)), rng.normal(size=(N, D, S))


@pytest.mark.parametrize("opts", [{}, {"z": False}, {"skip": False, "bias": False}, {"use_softplus": False}],
                         ids=["all", "no gate", "plain", "steps"])
def test_scan_gradients_against_differences(opts):
    lens, D, S, G = [5, 0, 1, 4], 6, 3, 2
    v, dy, dfin = _draw(lens, D, S, G, 1, **opts)
    sp = opts.get("use_softplus", True)

    def loss(**over):
        y, fin = R.ssm(**{**v, **over}, lens=lens, use_softplus=sp)
        return (dy * y).sum() + (dfin * fin).sum()

    names = ["x", "dt", "a", "b", "c", "skip", "z", "bias", "s0"]
    grads = dict(zip(names, R.ssm(**v, lens=lens, use_softplus=sp, dy=dy, dfin=dfin)[2:]))
    rng = np.random.default_rng(2)
    for name in names:
        if name not in v:
            assert grads[name] is None or name == "s0"
            continue
        d = rng.normal(size=v[name].shape)
        h = 1e-5
        num = (loss(**{name: v[name] + h * d}) - loss(**{name: v[name] - h * d})) / (2 * h)
        assert abs(num - (grads[name] * d).sum()) <= 1e-7 * (1 + np.abs(grads[name] * d).sum()), name


def test_scan_closed_values():
    """Constant decay and input: h_t = u (1 - q^t) / (1 - q); a closed gate passes nothing, a step of 0 keeps the state."""
    T = 6
    one = np.ones((T, 1))
    y, fin = R.ssm(one, 0.5 * one, np.array([[-2.0]]), one[:, None], one[:, None], [T])
    q = np.exp(-1.0)
    assert np.allclose(y[:, 0], 0.5 * (1 - q ** np.arange(1, T + 1)) / (1 - q), rtol=1e-14)
    assert np.allclose(fin[0, 0, 0], y[-1, 0])
    y, _ = R.ssm(one, one, np.array([[-2.0]]), one[:, None], one[:, None], [T], z=-800 * one)
    assert np.all(y == 0)
    s0 = np.full((1, 1, 1), 3.0)
    y, fin = R.ssm(one, 0 * one, np.array([[-2.0]]), one[:, None], one[:, None], [T], s0=s0)
    assert np.all(y == 3) and np.all(fin == 3)
    # the step of a bias alone: softplus(ln(e - 1)) = 1
    y, _ = R.ssm(one, 0 * one, np.array([[-1.0]]), one[:, None], one[:, None], [T], bias=np.log(np.expm1(np.ones(1))), use_softplus=True)
    assert np.allclose(y[0, 0], 1.0, rtol=1e-14) and np.allclose(y[1, 0], 1 + np.exp(-1.0), rtol=1e-14)


def test_norm_gradients_against_differences():
    rng = np.random.default_rng(3)
    s, w, dy, dr = rng.normal(size=(4, 7)), rng.normal(size=7), rng.normal(size=(4, 7)), rng.normal(size=(4, 7))
    y, ds, dw = R.rn(s, w, dy=dy, d_res=dr)
    for name, at, g in (("s", s, ds), ("w", w, dw)):
        d, h = rng.normal(size=at.shape), 1e-6

        def loss(v):
            q = dict(s=s, w=w)
            q[name] = v
            return (dy * R.rn(**q)).sum() + (dr * q["s"]).sum()

        assert abs((loss(at + h * d) - loss(at - h * d)) / (2 * h) - (g * d).sum()) <= 1e-7
    assert np.allclose(R.rn(np.full((1, 4), 5.0), np.ones(4), eps=1e-300), 1.0)
