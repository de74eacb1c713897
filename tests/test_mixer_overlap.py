"""Results over what the call still reads, or over each other, are refused: on the host with fake pointers (the library
returns before any CUDA call), and on a GPU that what only looks like it is taken."""
import ctypes

import pytest
import torch

import gated_delta_rule_29_gb300 as la
from gated_delta_rule_29_gb300 import binding as B
from test_mixer_abi import FAKE, INV, VALID

BF = torch.bfloat16


def code(fn, **over):
    cls, fields = VALID[fn]
    p = cls()
    for k, v in {**fields, **over}.items():
        setattr(p, k, v)
    return getattr(B.load(), fn)(ctypes.byref(p), None)


FAR = FAKE + (1 << 30)
OVER = [("sconv_fwd", dict(y=FAKE)),                                       # the same rows
        ("sconv_fwd", dict(y=FAKE + 2 * 63)),                              # the last channel of a row
        ("sconv_fwd", dict(y=FAKE + 128 * 255)),                           # the last row
        ("sconv_fwd", dict(x=FAKE + 128 * 255, y=FAKE)),
        ("sconv_fwd", dict(x_stride_t=100, y_stride_t=100, y=FAKE + 2 * (1000 - 63))),
        ("sconv_fwd", dict(y_stride_t=80, y=FAKE + 2 * 10)),               # the first rows, other strides
        ("sconv_fwd", dict(T=1, N=1, y=FAKE + 2 * 32)),
        ("sconv_fwd", dict(x_dtype=1, y=FAKE + 4 * 63)),
        ("sconv_bwd", dict(x=FAR, dx=FAKE)), ("sconv_bwd", dict(dy=FAR, dx=FAKE + 128 * 100)),
        ("sconv_bwd", dict(dy=FAR, dx=FAKE - 128 * 100))]


@pytest.mark.parametrize("fn,over", OVER, ids=lambda v: "-".join(f"{k}_{x:x}" for k, x in v.items()) if isinstance(v, dict) else v)
def test_convolution_over_its_inputs(fn, over):
    assert code(fn, **over) == INV


# 8 tokens x 2 heads of 64 channels
ROWS_MEET = [(64, 64), (96, 64), (64, 448), (128, 190), (256, 450), (100, 700), (128, 64 + 2)]


@pytest.mark.parametrize("st,sh", ROWS_MEET)
def test_norm_rows_over_each_other(st, sh):
    assert code("gn_fwd", y_stride_t=st, y_stride_h=sh) == INV
    assert code("gn_bwd", dx_stride_t=st, dx_stride_h=sh) == INV
    z = dict(z=FAKE, z_stride_t=128, z_stride_h=64, dz=FAKE)
    assert code("gn_bwd", **z, dz_stride_t=st, dz_stride_h=sh) == INV


@pytest.mark.gpu
@pytest.mark.parametrize("st,sh", [(128, 64), (200, 70), (64, 512), (70, 600), (192, 64), (128, 960), (256, 64 * 3), (128, 192), (256, 448), (64 * 3, 64 * 2)])
def test_norm_rows_beside_each_other(st, sh):
    """Results by token or by head, with gaps, and interleaved."""
    T, H, V = (8, 2, 64) if (st, sh) != (64 * 3, 64 * 2) else (2, 2, 64)
    gen = torch.Generator().manual_seed(2)
    x, dy = (torch.randn(T, H, V, generator=gen).to(BF).cuda() for _ in range(2))
    w = torch.randn(V, generator=gen).cuda()
    buf = torch.full((T * st + H * sh + V,), 7.0, dtype=BF, device="cuda")
    out = buf.as_strided((T, H, V), (st, sh, 1))
    assert torch.equal(la.gn_fwd(x, w, y=out), la.gn_fwd(x, w))
    assert int((buf != 7).sum()) <= T * H * V
    assert torch.equal(la.gn_bwd(x, w, dy, dx=out)[0], la.gn_bwd(x, w, dy)[0])


@pytest.mark.gpu
def test_convolution_beside_its_inputs():
    """Interleaved column slices of one buffer, the halves of one buffer, and rows of other strides share no memory."""
    T, D = 300, 64
    gen = torch.Generator().manual_seed(1)
    x, dy = (torch.randn(T, D, generator=gen).to(BF).cuda() for _ in range(2))
    w = torch.randn(D, 4, generator=gen).cuda()
    cu = torch.tensor([0, 100, T], dtype=torch.int32, device="cuda")
    y, dx = la.sconv_fwd(x, w, cu)[0], la.sconv_bwd(x, w, cu, dy)[0]
    wide = torch.zeros(T, 3 * D, dtype=BF, device="cuda")
    tall = torch.zeros(3 * T, D, dtype=BF, device="cuda")
    for a, b, c in (wide.split(D, 1), tall.split(T)):
        a.copy_(x)
        c.copy_(dy)
        assert torch.equal(la.sconv_fwd(a, w, cu, y=b)[0], y)
        assert torch.equal(la.sconv_bwd(a, w, cu, c, dx=b)[0], dx)
        for over in (lambda: la.sconv_fwd(a, w, cu, y=a), lambda: la.sconv_bwd(a, w, cu, c, dx=c),
                     lambda: la.sconv_bwd(a, w, cu, c, dx=a)):
            with pytest.raises(B.LinAttnError):
                over()
        assert torch.equal(a, x) and torch.equal(c, dy)
