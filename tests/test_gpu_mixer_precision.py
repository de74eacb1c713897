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
