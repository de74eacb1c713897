"""Eight-bit results of the residual norm where its factors leave the 32-bit range: a small eps beside rows or blocks of
zeros and tiny rows, and results that are not finite.  Bounds as in test_gpu_rn.py."""
import pytest
import torch

import gated_delta_rule_29_gb300 as la
from test_gpu_rn import BF, F32, dev, draw, expect_8bit

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("eps", [3e-12, 1e-12, 1e-20, 1e-30])
@pytest.mark.parametrize("kind", ["row", "block", "mx"])
@pytest.mark.parametrize("V,xt,rt", [(256, F32, None), (512, BF, BF), (333, F32, F32), (8448, BF, None)])
def test_small_eps(V, xt, rt, kind, eps):
    """A padding row, blocks of zeros in a row, rows whose mean square is eps's and far below it, and an ordinary one."""
    t = draw(7, V, xt, rt, seed=V)
    r = t.get("r")
    if r is not None:
        r.zero_()  # the stream is x
    t["x"][0] = 0
    t["x"][1] *= 1e-6
    t["x"][2] *= 1e-6
    t["x"][2, 96:] = 0
    t["x"][3] *= 1e-15
    t["x"][4] *= 1e-18
    t["x"][4, :130] = 0
    t["x"][5, 32:] = 0
    y, s, scales = la.rn_fwd(t["x"], t["w"], r, quantize=kind, eps=eps)
    assert bool(torch.isfinite(y.float()).all()) and bool(torch.isfinite(scales.float()).all())
    assert not y.float()[0].any()
    expect_8bit(y, scales, s, t["w"], kind, eps)


@pytest.mark.parametrize("kind", ["row", "block", "mx"])
def test_tiny_rows_are_scaled(kind):
    """Rows so small that the inverse of their values leaves the range, which a small eps brings back into it."""
    t = draw(5, 512, F32, None, seed=3)
    t["x"] *= torch.tensor([1e-37, 1e-36, 1e-33, 1e-30, 1.0], device=dev())[:, None]
    y, s, scales = la.rn_fwd(t["x"], t["w"], quantize=kind, eps=1e-30)
    expect_8bit(y, scales, s, t["w"], kind, 1e-30)


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("kind,width", [("row", 512), ("block", 128), ("mx", 32)])
def test_blocks_that_are_not_finite(kind, width, value):
    """A weight that is not finite beside finite rows: the scales and values of its block are NaN, the others' as they are."""
    t = draw(6, 512, F32, F32, seed=3)
    want, _, want_scales = la.rn_fwd(t["x"], t["w"], t["r"], quantize=kind)
    w = t["w"].clone()
    w[200] = value
    y, _, scales = la.rn_fwd(t["x"], w, t["r"], quantize=kind)
    bad = torch.arange(512, device=dev()) // width == 200 // width
    assert bool(torch.isnan(scales.float()[:, 200 // width]).all()) and bool(torch.isnan(y.float()[:, bad]).all())
    assert torch.equal(y.float()[:, ~bad], want.float()[:, ~bad])
    assert int(torch.isnan(scales.float()).sum()) == 6
    other = torch.arange(want_scales.shape[1], device=dev()) != 200 // width
    assert torch.equal(scales.float()[:, other], want_scales.float()[:, other])
