"""A row's bits of the residual norm, alone and among others."""
import pytest
import torch

import gated_delta_rule_29_gb300 as la
from test_gpu_rn import BF, F32, dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("stride", [4096, 4099, 4104, 4098])
@pytest.mark.parametrize("xt", [BF, F32])
def test_a_row_alone_and_among_others(xt, stride):
    """Every row of a view, at all alignments that its stride gives, by itself: y, 8-bit values with their scales, dx."""
    T, V = 40, 4096
    gen = torch.Generator().manual_seed(stride)
    x, r, dy = (torch.randn(T * stride, generator=gen).to(xt).to(dev()).as_strided((T, V), (stride, 1)) for _ in range(3))
    w = (1 + 0.1 * torch.randn(V, generator=gen)).to(dev())
    y, s, _ = la.rn_fwd(x, w, r)
    s = s.as_strided((T, V), (V, 1))
    q, _, scales = la.rn_fwd(x, w, r, quantize="block")
    dx = la.rn_bwd(x, w, dy, d_residual=r)[0]
    for t in range(T):
        at = slice(t, t + 1)
        y1, s1, _ = la.rn_fwd(x[at], w, r[at])
        q1, _, scales1 = la.rn_fwd(x[at], w, r[at], quantize="block")
        assert torch.equal(y1, y[at]) and torch.equal(s1, s[at]), t
        assert torch.equal(q1.view(torch.uint8), q[at].view(torch.uint8)) and torch.equal(scales1, scales[at]), t
        assert torch.equal(la.rn_bwd(x[at], w, dy[at], d_residual=r[at])[0], dx[at]), t
