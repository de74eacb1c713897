"""The norm's backward takes one wave of CTAs of whatever form the operands ask for, and its partial sums fit the workspace
that the shape alone determines."""
import pytest
import torch

import gated_delta_rule_29_gb300 as la
from gated_delta_rule_29_gb300 import binding as B

SMS, MOST = 152, 3


@pytest.mark.parametrize("H,V", [(32, 128), (4, 64), (1, 8)])
def test_workspace_is_one_wave_at_most(H, V):
    """Bytes grow with the rows, to the wave of three CTAs an SM and no further (fp32 sums of a weight and a bias)."""
    size = B.load().la_gn_bwd_workspace_bytes
    sizes = [size(T, H, V, 0) for T in (0, 1, 100, 1000, 2000, 3600, 4000, 8000, 65536, 1 << 22)]
    wave = SMS * MOST * V * 2 * 4
    assert sizes == sorted(sizes) and sizes[-1] == (wave + 255) // 256 * 256
    assert size(3600, 32, 128, 0) == SMS * MOST * 128 * 2 * 4


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,V", [(1, 1, 1), (3600, 32, 128), (2500, 7, 128), (4099, 10, 100), (900, 3, 600), (70, 2, 4096), (5, 300, 16)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("per_head,bias", [(False, False), (True, False), (False, True), (True, True)])
def test_partial_sums_stay_in_the_workspace(T, H, V, dtype, per_head, bias):
    gen = torch.Generator().manual_seed(T + V)
    x, dy = (torch.randn(T, H, V, generator=gen).to(dtype).cuda() for _ in range(2))
    w = torch.randn((H, V) if per_head else (V,), generator=gen).cuda()
    b = torch.randn(w.shape, generator=gen).cuda() if bias else None
    need = B.load().la_gn_bwd_workspace_bytes(T, H, V, int(per_head))
    whole = torch.full((need + 65536,), 0x5A, dtype=torch.uint8, device="cuda")
    got = la.gn_bwd(x, w, dy, b, workspace=whole[:need])
    assert bool((whole[need:] == 0x5A).all())
    want = la.gn_bwd(x, w, dy, b)
    assert all(torch.equal(p, q) for p, q in zip(got, want) if p is not None)
    if bias:  # db of an identity activation is the sum of dy
        db = la.gn_bwd(x, w, dy, b, activation="none")[2]
        ref = dy.double().sum(0 if per_head else (0, 1))
        rows = T if per_head else T * H
        assert bool(((db.double() - ref).abs() <= (rows + 2) * 2.0 ** -24 * dy.double().abs().sum(0 if per_head else (0, 1))).all())
