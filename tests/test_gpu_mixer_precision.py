"""Where 32 bits cancel: the token-mixer operators at values whose results are small differences in a naive form, against
the 64-bit forms, with bounds that follow the result's own size (fixed before the first run).

Units are 2^-24 of the value.  An exponential of v is off by 1.5 |v| units for its argument's roundings and 3 for
ex2.approx (2^-22.5), a reciprocal by 2 (rcp.approx, one unit in the last place), a sum or product by 1.  An
intermediate below 2^-126 is 0, which is 2^-126 times what it would have been multiplied by."""
import numpy as np
import pytest
import torch

import gated_delta_rule_29_gb300 as la
import mixer_reference as R
import test_gpu_glr as glr

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return torch.device("cuda:0")


def far(shape, seed, lo=-20.0, hi=20.0):
    gen = torch.Generator().manual_seed(seed)
    return lo + (hi - lo) * torch.rand(shape, generator=gen)


def act_units(v):
    """An activation's derivative at |v| <= 20: the exponential, its sum with 1, the reciprocal and three products."""
    return 1.5 * np.abs(v) + 10


@pytest.mark.parametrize("act", ["silu", "sigmoid"])
@pytest.mark.parametrize("V", [64, 100])
def test_gate_gradient_far_from_zero(act, V):
    """dz = dy p act'(z) for gates in [-20, 20] and beyond the exponential's range, where it is 0."""
    T, H = 40, 2
    gen = torch.Generator().manual_seed(V)
    x, dy = (torch.randn(T, H, V, generator=gen).to(dev()) for _ in range(2))
    z, w = far((T, H, V), V + 1).to(dev()), (1 + 0.1 * torch.randn(V, generator=gen)).to(dev())
    z[0, 0, :8] = torch.tensor([-1e4, -200.0, -89.0, -88.0, 88.0, 89.0, 200.0, 1e4])
    dz = la.gn_bwd(x, w, dy, z=z, center=False, activation=act)[3]
    xs, ws, zs, ds = (R.f64(t) for t in (x, w, z, dy))
    ref = R.gn(xs, ws, None, zs, ds, center=False, activation=act)[4]
    r = 1 / np.sqrt((xs * xs).mean(-1, keepdims=True) + 1e-5)
    da = R.act(act, zs)[1]
    # silu' = s (1 + z r) passes through 0 at z = -1.28: its terms there are as large as s
    size = np.abs(da) if act == "sigmoid" else np.maximum(np.abs(da), R.sigmoid(zs) * np.where(zs < 0, 1 - zs, 1.0))
    p, units = np.abs(ds * xs * r * ws), 2 * V + 64 + act_units(np.clip(zs, -20, 20))
    R.within("dz", dz, ref, F32, 1, p * (units * size + 2.0 ** (24 - 126) * (1 + np.abs(zs))))


@pytest.mark.parametrize("act", ["silu", "sigmoid"])
def test_activation_gradient_far_from_zero(act):
    """db = dy act'(p) of a single row, p from a bias in [4, 20]."""
    V = 512
    gen = torch.Generator().manual_seed(3)
    x, dy = (torch.randn(1, 1, V, generator=gen).to(dev()) for _ in range(2))
    w, b = (0.1 * torch.randn(V, generator=gen)).to(dev()), far((V,), 4, lo=4.0).to(dev())
    db = la.gn_bwd(x, w, dy, b, center=True, activation=act)[2]
    xs, ws, bs, ds = (R.f64(t) for t in (x, w, b, dy))
    ref = R.gn(xs, ws, bs, None, ds, center=True, activation=act)[3]
    c = xs - xs.mean(-1, keepdims=True)
    p = (c / np.sqrt((c * c).mean(-1, keepdims=True) + 1e-5) * ws + bs)[0, 0]
    # p is off by 2 V + 64 units of the norm's part and one of its sum; act' goes with e^-p
    n = np.abs(xs[0, 0]) + np.abs(xs).mean()
    units = (2 * V + 64) * 2 * n * np.abs(ws) + np.abs(p) + act_units(p)
    R.within("db", db, ref, F32, units, np.abs(ds[0, 0]) * R.act(act, p)[1])


@pytest.mark.parametrize("act", ["silu", "sigmoid"])
@pytest.mark.parametrize("W", [2, 3, 4])
def test_convolution_gradient_far_from_zero(act, W):
    """dx of sequences of one token: w_{W-1} dy act'(p), p from a bias in [4, 20]."""
    N, D = 50, 96
    gen = torch.Generator().manual_seed(W)
    x, dy = (torch.randn(N, D, generator=gen).to(dev()) for _ in range(2))
    w, b = (0.5 * torch.randn(D, W, generator=gen)).to(dev()), far((D,), W, lo=4.0).to(dev())
    cu = torch.arange(N + 1, dtype=torch.int32, device=dev())
    dx = la.sconv_bwd(x, w, cu, dy, b, activation=act)[0]
    xs, ws, bs, ds = (R.f64(t) for t in (x, w, b, dy))
    ref = R.sconv(xs, ws, bs, [1] * N, None, ds, activation=act)[2]
    p = xs * ws[:, -1] + bs
    size = np.abs(xs * ws[:, -1]) + np.abs(bs)
    R.within("dx", dx, ref, F32, (W + 1) * size + act_units(p) + 2, np.abs(ds * ws[:, -1]) * R.act(act, p)[1])


@pytest.mark.parametrize("gt", [BF, F32])
@pytest.mark.parametrize("gate,complement", [("logsigmoid", False), ("logsigmoid", True), ("bound", False)])
def test_closed_gates(gt, gate, complement):
    """Logits from where the sigmoid is small to the type's lowest value and minus infinity: a closed gate leaves nothing
    of the state before it (h is 0 where no input follows), and the gradients through it are the formula's."""
    logits = [-20.0, -50.0, -80.0, -86.0, -100.0, -1e4, torch.finfo(gt).min, float("-inf")]
    lens, D = [40, 300], 8 * len(logits)
    t = glr.draw(lens, D, F32, gt, "logsigmoid", seed=31)
    for at in (20, 150, 330):
        t["g"][at] = torch.tensor(logits).repeat_interleave(8).to(gt)
        t["x"][at:at + 5] = 0.0
    glr.check(t, lens, gate, complement)


@pytest.mark.parametrize("bound", [-0.5, -5.0])
def test_slow_bounded_gates(bound):
    """Decays a = exp(bound s(g)) just below 1, one token against a state of ones: their errors add up over 1 / |log a|
    tokens, by their mean where gates vary.  A value is off by at most 4 units of 2^-24 (ex2.approx 3, the rest at
    most |log a| of its own units and the rounding of the argument), and the mean of many by 1/4 (a rounding to nearest
    has none)."""
    g = torch.linspace(-11, 8, 1 << 18, device=dev())
    a = la.glr_decode(torch.zeros(1, g.numel(), device=dev()), g[None].contiguous(),
                      state := torch.ones(1, g.numel(), device=dev()), gate_lower_bound=bound)
    assert torch.equal(a, state) and bool((a <= 1).all())
    log_a = bound * R.sigmoid(R.f64(g))
    off = (R.f64(a)[0] / np.exp(log_a) - 1) * 2.0 ** 24
    for lo, hi in ((1e-5, 1e-4), (1e-4, 1e-3), (1e-3, 1e-2), (1e-2, 1 / 16), (1 / 16, 1 / 8), (1 / 8, 1 / 4), (1 / 4, 1 / 2)):
        at = (-log_a >= lo) & (-log_a < hi)
        assert at.sum() > 2000 and np.abs(off[at]).max() <= 4 and abs(off[at].mean()) <= 0.25, (lo, off[at].mean())


@pytest.mark.parametrize("repeat", [False, True])
def test_states_of_slow_bounded_gates(repeat):
    """Final states of 20000 tokens whose gates stay the same, or vary, around decays of 0.99 and 0.999."""
    T, D = 20000, 64
    gen = torch.Generator().manual_seed(11)
    mid = torch.where(torch.arange(D) % 2 == 0, -3.9, -6.2)
    g = mid + 0.7 * torch.randn(1 if repeat else T, D, generator=gen)
    g = g.expand(T, D).contiguous().to(dev())
    x = torch.rand(T, D, generator=gen).to(dev())
    cu = torch.tensor([0, T], dtype=torch.int32, device=dev())
    fin = la.glr_fwd(x, g, cu, gate_lower_bound=-0.5)[1]
    args = (R.f64(x), R.f64(g), [T])
    ref, scale = R.glr_fwd(*args, lower_bound=-0.5)[1], R.glr_scales(*args, lower_bound=-0.5)[1]
    # every step within 4 units for its decay, 1 for its sum, and 1 for the joining of spans, warps and blocks
    R.within("final_state", fin, ref, F32, 6, scale)
