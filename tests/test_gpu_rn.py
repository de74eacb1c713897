"""The residual norm on the GPU against its 64-bit form.

Bounds (fixed before the first run): y, the gradients: one rounding to the type after at most twice the units of rn_scales
(block_reference.py).  In 8 bits a value is y / scale rounded to e4m3: off by half a step, 2^-4 of it or 2^-10 of the
scale below the normal range, and by what y itself may be off."""
import numpy as np
import pytest
import torch

import block_reference as R
import gated_delta_rule_29_gb300 as la
from gated_delta_rule_29_gb300 import binding as B

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
UNITS = 2
WIDTHS = [1, 2, 7, 31, 32, 33, 127, 128, 129, 256, 264, 512, 1001, 2048, 4096, 5000, 8192, 8200, 16384]


def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return torch.device("cuda:0")


def draw(T, V, xt=BF, rt=BF, wt=F32, seed=1):
    gen = torch.Generator().manual_seed(seed)
    t = dict(x=torch.randn(T, V, generator=gen).to(xt), w=(1 + 0.1 * torch.randn(V, generator=gen)).to(wt),
             dy=torch.randn(T, V, generator=gen).to(xt))
    if rt is not None:
        t["r"], t["dr"] = (2 * torch.randn(T, V, generator=gen)).to(rt), torch.randn(T, V, generator=gen).to(rt)
    return {k: v.to(dev()) for k, v in t.items()}


def check(t, **kw):
    y, s, none = la.rn_fwd(t["x"], t["w"], t.get("r"), **kw)
    assert none is None
    if "r" in t:
        assert torch.equal(s, (t["x"].float() + t["r"].float()).to(t["r"].dtype))
    else:
        assert s is t["x"]
    dx, dw, ds = la.rn_bwd(s, t["w"], t["dy"], d_residual=t.get("dr"), **kw)
    v = dict(s=R.f64(s), w=R.f64(t["w"]), dy=R.f64(t["dy"]), d_res=R.f64(t.get("dr")))
    ref, scale = R.rn(**v, **kw), R.rn_scales(**v, **kw)
    R.within("y", y, ref[0], y.dtype, UNITS, scale[0])
    R.within("dx", dx, ref[1], t["x"].dtype, UNITS, scale[1])
    R.within("ds", ds, ref[1], s.dtype, UNITS, scale[1])
    R.within("dw", dw, ref[2], t["w"].dtype, UNITS, scale[2])
    assert (ds is dx) == (s.dtype == dx.dtype)
    return y, s, dx, dw, ds


@pytest.mark.parametrize("V", WIDTHS)
@pytest.mark.parametrize("xt,rt", [(BF, None), (BF, BF), (BF, F32), (F32, F32)])
def test_widths_and_types(V, xt, rt):
    check(draw(13, V, xt, rt, BF if V % 2 else F32, seed=V))


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 700, 5003])
@pytest.mark.parametrize("V", [96, 4096])
def test_rows(T, V):
    check(draw(T, V, seed=T))


def expect_8bit(y, scales, s, w, kind, eps=1e-5):
    ref, units = R.rn(R.f64(s), R.f64(w), eps), R.rn_scales(R.f64(s), R.f64(w), eps)
    T, V = ref.shape
    width = {"row": V, "block": 128, "mx": 32}[kind]
    pad = np.zeros((T, -(-V // width) * width))
    pad[:, :V] = np.abs(ref)
    most = np.maximum(pad.reshape(T, -1, width).max(2), 2.0 ** -100) / 448
    got = scales.float().cpu().numpy().astype(np.float64)
    assert got.shape == most.shape
    # y's relative error is at most 2 * 44 units, and the scale's two more roundings
    if kind == "mx":
        want = 2.0 ** np.ceil(np.log2(most))
        near = np.abs(most / 2.0 ** np.round(np.log2(most)) - 1) < 100 * 2.0 ** -24  # either power is right there
        assert np.all((got == want) | (near & ((got == 2 * want) | (got == want / 2))))
    else:
        assert np.all(np.abs(got / most - 1) <= 100 * 2.0 ** -24)
    each = np.repeat(got, width, 1)[:, :V]
    val = y.float().cpu().numpy().astype(np.float64) * each
    off = np.abs(val - ref)
    assert np.all(off <= 2.0 ** -4 * np.abs(ref) * (1 + 1e-4) + 2.0 ** -10 * each * (1 + 1e-4) + UNITS * 2.0 ** -24 * units)


@pytest.mark.parametrize("kind", ["row", "block", "mx"])
@pytest.mark.parametrize("V", WIDTHS)
@pytest.mark.parametrize("xt,rt", [(BF, BF), (BF, F32), (F32, None)])
def test_eight_bits(V, kind, xt, rt):
    t = draw(9, V, xt, rt, seed=V)
    t["x"][3] *= 100
    t["x"][:, V // 2] *= 30
    t["w"][V // 3] *= 0.001
    y, s, scales = la.rn_fwd(t["x"], t["w"], t.get("r"), quantize=kind)
    assert y.dtype == torch.float8_e4m3fn and scales.dtype == (torch.float8_e8m0fnu if kind == "mx" else F32)
    expect_8bit(y, scales, s, t["w"], kind)


@pytest.mark.parametrize("kind", ["row", "block", "mx"])
def test_eight_bits_are_rounded_to_nearest(kind):
    """The values are those that a conversion of y / scale gives, but for y next to a border."""
    t = draw(50, 512, seed=4)
    full, s, _ = la.rn_fwd(t["x"].float(), t["w"], t["r"].float())
    q, _, scales = la.rn_fwd(t["x"].float(), t["w"], t["r"].float(), quantize=kind)
    each = scales.float().repeat_interleave({"row": 512, "block": 128, "mx": 32}[kind], 1)
    assert float((q.float() != (full / each).to(torch.float8_e4m3fn).float()).float().mean()) < 1e-3


@pytest.mark.parametrize("kind", [None, "row", "block", "mx"])
def test_zero_tiny_and_infinite_rows(kind):
    t = draw(6, 256, F32, None, seed=5)
    t["x"][0] = 0
    t["x"][1] = 1e-30
    t["x"][2, 7] = float("nan")
    t["x"][3, 9] = float("inf")
    t["x"][4] *= 1e15
    y, _, scales = la.rn_fwd(t["x"], t["w"], quantize=kind)
    y = y.float()
    assert not y[0].any() and bool(torch.isnan(y[2]).all()) and bool(torch.isnan(y[3, 9]))
    assert bool(torch.isfinite(y[[0, 1, 4, 5]]).all())
    if kind is None:
        ref = R.rn(R.f64(t["x"][[1, 4, 5]]), R.f64(t["w"]))
        R.within("y", y[[1, 4, 5]], ref, F32, UNITS, R.rn_scales(R.f64(t["x"][[1, 4, 5]]), R.f64(t["w"])))
    else:
        assert bool(torch.isfinite(scales.float()[[0, 1, 4, 5]]).all()) and bool(torch.isnan(scales.float()[2]).all())
        expect_8bit(y[[0, 1, 4, 5]], scales.float()[[0, 1, 4, 5]], t["x"][[0, 1, 4, 5]], t["w"], kind)


@pytest.mark.parametrize("V", [512, 500, 37])
def test_views_and_in_place(V):
    t = draw(33, V, seed=V)
    want = check(t)
    wide = torch.full((33, 3 * V + 5), float("nan"), dtype=BF, device=dev())
    v = {}
    for i, k in enumerate(("x", "r", "dy")):
        wide[:, 1 + i * V:1 + (i + 1) * V] = t[k]
        v[k] = wide[:, 1 + i * V:1 + (i + 1) * V]
    buf = torch.full((33, V + 3), 7.0, dtype=BF, device=dev())
    # widths of vectors and of single elements sum in other orders: results within a rounding of each other
    y, s, _ = la.rn_fwd(v["x"], t["w"], v["r"], y=buf[:, 2:2 + V])
    assert torch.equal(s, want[1]) and bool((buf[:, :2] == 7).all()) and bool((buf[:, 2 + V:] == 7).all())
    assert float((y.float() - want[0].float()).abs().max()) <= 2.0 ** -7 * float(want[0].float().abs().max())
    res = t["r"].clone()
    y, s, _ = la.rn_fwd(t["x"], t["w"], res, residual_out=res)
    assert s is res and torch.equal(res, want[1]) and torch.equal(y, want[0])
    x = t["x"].clone()
    _, s, _ = la.rn_fwd(x, t["w"], t["r"], residual_out=x)
    assert s is x and torch.equal(x, want[1])
    for k in ("dy", "dr"):
        u = {n: a.clone() for n, a in t.items()}
        dx, dw, _ = la.rn_bwd(want[1], t["w"], u["dy"], d_residual=u["dr"], dx=u[k])
        assert dx is u[k] and torch.equal(dx, want[2]) and torch.equal(dw, want[3])
    one = t["dy"][:1].expand(33, V)
    t["dy"] = one
    check(t)


def test_refusals_and_nothing_to_do():
    t = draw(4, 64, seed=3)
    for call, error in ((lambda: la.rn_fwd(t["x"], t["w"][:32]), ValueError), (lambda: la.rn_fwd(t["x"], t["w"], t["r"][:2]), ValueError),
                        (lambda: la.rn_fwd(t["x"], t["w"], quantize="int4"), ValueError), (lambda: la.rn_fwd(t["x"].half(), t["w"]), TypeError),
                        (lambda: la.rn_fwd(t["x"], t["w"], residual_out=t["r"]), ValueError),
                        (lambda: la.rn_fwd(t["x"], t["w"], scales=t["w"]), ValueError),
                        (lambda: la.rn_fwd(t["x"], t["w"], y=t["x"], quantize="row"), TypeError),
                        (lambda: la.rn_fwd(t["x"].float(), t["w"], t["r"]), B.LinAttnError),
                        (lambda: la.rn_fwd(t["x"], t["w"], eps=0.0), B.LinAttnError),
                        (lambda: la.rn_bwd(t["x"], t["w"], t["dy"].float()), B.LinAttnError),
                        (lambda: la.rn_bwd(t["x"], t["w"], t["dy"], d_residual=t["dr"].float()), TypeError),
                        (lambda: la.rn_bwd(t["x"], t["w"], t["dy"], ds=t["dr"]), ValueError)):
        with pytest.raises(error):
            call()
    y, s, sc = la.rn_fwd(t["x"][:0], t["w"], t["r"][:0], quantize="block")
    assert y.shape == (0, 64) and sc.shape == (0, 1)
    dx, dw, _ = la.rn_bwd(s, t["w"], t["dy"][:0])
    assert dx.shape == (0, 64) and not dw.any()


def test_rows_beyond_32_bits():
    T, V = 40, 256
    t = draw(T, V, seed=21)
    want = check(t)
    stride = (1 << 31) // 32 + 8
    big = torch.empty(T * stride, dtype=BF, device=dev())
    v = {}
    for i, k in enumerate(("x", "r", "dy", "dr", "y", "s")):
        v[k] = big.as_strided((T, V), (stride, 1), i * V)
        if k in t:
            v[k].copy_(t[k])
    y, s, _ = la.rn_fwd(v["x"], t["w"], v["r"], y=v["y"], residual_out=v["s"])
    assert torch.equal(y, want[0]) and torch.equal(s, want[1])
    dx, dw, _ = la.rn_bwd(v["s"], t["w"], v["dy"], d_residual=v["dr"], dx=v["x"])
    assert torch.equal(dx, want[2]) and torch.equal(dw, want[3])
