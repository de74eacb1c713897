"""The norm's weight gradient over many rows."""
import pytest
import torch

import gated_delta_rule_29_gb300 as la
from test_gpu_rn import BF, F32, dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,V,rt", [(1 << 18, 4096, F32), (1 << 18, 4096, BF), (1 << 19, 1001, BF)])
def test_weight_gradient_over_many_rows(T, V, rt):
    """Equal rows, so that every row adds the same and a running sum is off by the same rounding again and again.  A row's term goes
    through 64 additions of its part, the parts of a CTA (T / (152 CTAs x 64) at most), 8 groups, 15 CTAs and 32 warps, half a unit of
    2^-23 each; the term itself is off by 44 units at most (rn_scales)."""
    gen = torch.Generator().manual_seed(2)
    s, dy = torch.randn(1, V, generator=gen).to(rt).to(dev()), (1 + torch.rand(1, V, generator=gen)).to(BF).to(dev())
    w = torch.ones(V, device=dev())
    _, dw, _ = la.rn_bwd(s.expand(T, V), w, dy.expand(T, V))
    v = s.double()[0]
    want = T * dy.double()[0] * v / (v.square().mean() + 1e-5).sqrt()
    off = (dw.double() / want - 1).abs() * 2.0 ** 24
    assert float(off.max()) <= 64 + T / (152 * 64) + 8 + 15 + 32 + 44
