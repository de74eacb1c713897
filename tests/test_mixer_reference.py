"""The 64-bit forms that the token-mixer GPU tests compare with, pinned by central differences of their own forward
and by closed values (CPU)."""
import numpy as np
import pytest

import mixer_reference as R

LENS = [3, 0, 1, 6]


def differences(f, v, cot, step=1e-6):
    """d sum(cot * f(v)) / dv by central differences."""
    out = np.zeros_like(v)
    for k in np.ndindex(v.shape):
        hi, lo = v.copy(), v.copy()
        hi[k] += step
        lo[k] -= step
        out[k] = sum(((a - b) * c).sum() for a, b, c in zip(f(hi), f(lo), cot)) / (2 * step)
    return out


@pytest.mark.parametrize("gate", [{}, {"logsigmoid": True}, {"lower_bound": -0.7}])
@pytest.mark.parametrize("complement", [False, True])
def test_glr_gradients(gate, complement):
    rng = np.random.default_rng(1)
    x, dh, g = rng.normal(size=(10, 2)), rng.normal(size=(10, 2)), -np.abs(rng.normal(size=(10, 2)))
    s0, dfin = rng.normal(size=(4, 2)), rng.normal(size=(4, 2))
    f = lambda x_, g_, s_: R.glr_fwd(x_, g_, LENS, s_, complement=complement, **gate)  # noqa: E731
    dx, dg, ds0 = R.glr_bwd(x, g, LENS, dh, s0, dfin, complement=complement, **gate)
    assert np.allclose(dx, differences(lambda v: f(v, g, s0), x, (dh, dfin)), atol=1e-7)
    assert np.allclose(dg, differences(lambda v: f(x, v, s0), g, (dh, dfin)), atol=1e-7)
    assert np.allclose(ds0, differences(lambda v: f(x, g, v), s0, (dh, dfin)), atol=1e-7)


def test_glr_closed_values():
    # constant decay 1/2 and unit inputs: 1, 3/2, 7/4; with the complement 1/2, 3/4, 7/8
    x, g = np.ones((3, 1)), np.full((3, 1), np.log(0.5))
    assert np.allclose(R.glr_fwd(x, g, [3])[0][:, 0], [1, 1.5, 1.75])
    assert np.allclose(R.glr_fwd(x, g, [3], complement=True)[0][:, 0], [0.5, 0.75, 0.875])
    assert np.allclose(R.glr_fwd(x, np.zeros((3, 1)), [3], logsigmoid=True)[0][:, 0], [1, 1.5, 1.75])


@pytest.mark.parametrize("center", [False, True])
@pytest.mark.parametrize("activation,gated", [("none", False), ("silu", False), ("sigmoid", False), ("silu", True),
                                              ("sigmoid", True)])
@pytest.mark.parametrize("per_head", [False, True])
def test_gn_gradients(center, activation, gated, per_head):
    rng = np.random.default_rng(2)
    x, dy = rng.normal(size=(3, 2, 5)), rng.normal(size=(3, 2, 5))
    z = rng.normal(size=(3, 2, 5)) if gated else None
    w, b = rng.normal(size=(2, 5) if per_head else 5), rng.normal(size=(2, 5) if per_head else 5)
    opts = dict(center=center, activation=activation)
    _, dx, dw, db, dz = R.gn(x, w, b, z, dy, **opts)
    assert np.allclose(dx, differences(lambda v: (R.gn(v, w, b, z, **opts),), x, (dy,)), atol=1e-7)
    assert np.allclose(dw, differences(lambda v: (R.gn(x, v, b, z, **opts),), w, (dy,)), atol=1e-7)
    assert np.allclose(db, differences(lambda v: (R.gn(x, w, v, z, **opts),), b, (dy,)), atol=1e-7)
    if gated:
        assert np.allclose(dz, differences(lambda v: (R.gn(x, w, b, v, **opts),), z, (dy,)), atol=1e-7)


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("activation", ["none", "silu"])
def test_sconv_gradients(W, activation):
    rng = np.random.default_rng(3)
    x, dy, w, b = rng.normal(size=(10, 2)), rng.normal(size=(10, 2)), rng.normal(size=(2, W)), rng.normal(size=2)
    s0, dfin = rng.normal(size=(4, W - 1, 2)), rng.normal(size=(4, W - 1, 2))
    f = lambda x_, w_, b_, s_: R.sconv(x_, w_, b_, LENS, s_, activation=activation)  # noqa: E731
    _, fin, dx, dw, db, ds0 = R.sconv(x, w, b, LENS, s0, dy, dfin, activation=activation)
    cot = (dy, dfin)
    assert np.allclose(dx, differences(lambda v: f(v, w, b, s0), x, cot), atol=1e-7)
    assert np.allclose(dw, differences(lambda v: f(x, v, b, s0), w, cot), atol=1e-7)
    assert np.allclose(db, differences(lambda v: f(x, w, v, s0), b, cot), atol=1e-7)
    assert np.allclose(ds0, differences(lambda v: f(x, w, b, v), s0, cot), atol=1e-7)
    assert np.array_equal(fin[1], s0[1]) and np.array_equal(fin[3], x[10 - (W - 1):])


def test_planted_mistakes_are_seen():
    """The comparison rejects a wrong value in one place and a NaN that the reference has not."""
    import torch
    ref = np.array([[1.0, 2.0], [3.0, 4.0]])
    R.within("same", torch.tensor(ref, dtype=torch.float32), ref, torch.float32, 4, np.abs(ref))
    for bad in (4.001, float("nan"), float("inf")):
        got = torch.tensor(ref, dtype=torch.float32)
        got[1, 1] = bad
        with pytest.raises(AssertionError):
            R.within("planted", got, ref, torch.float32, 4, np.abs(ref))
