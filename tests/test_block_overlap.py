"""Results of the scan and the norm that share memory with an operand of another row stride, anywhere, with the scan's
vectors or the norm's parameters, on the host with fake pointers (the library returns before any CUDA call), and on a GPU that what only looks like it is
taken."""
import ctypes

import pytest
import torch

import gated_delta_rule_29_gb300 as la
from gated_delta_rule_29_gb300 import binding as B
from test_block_abi import FAR, VALID
from test_mixer_abi import FAKE, INV

# rows are 128 bytes of bf16; the scans have 256 of them, single tokens 2, the norms 8
OVER = [("ssm_fwd", dict(x=FAR + 128 * 5, x_stride_t=0)),                       # a broadcast row in the middle of the result
        ("ssm_fwd", dict(z=FAR + 128 * 255, z_stride_t=0)),                     # the last row
        ("ssm_fwd", dict(dt=FAR + 64, dt_stride_t=0)),
        ("ssm_fwd", dict(x=FAR + 128 * 200, x_stride_t=128)),                   # behind the first rows, twice the stride
        ("ssm_fwd", dict(x=FAR - 256 * 100, x_stride_t=128)),                   # row 100 of it is the result's first
        ("ssm_fwd", dict(y_stride_t=128, dt=FAR + 256 * 3, dt_stride_t=64)),
        ("ssm_fwd", dict(y_stride_t=100, z=FAR + 200 * 7 - 128 * 9 + 2, z_stride_t=64)),
        ("ssm_decode", dict(y_stride_n=128, x=FAR + 256, x_stride_n=0)),
        ("ssm_decode", dict(y_stride_n=128, dt=FAR + 128, dt_stride_n=64)),
        ("ssm_bwd", dict(x=FAR + 128 * 9, x_stride_t=0)), ("ssm_bwd", dict(dy=FAR + 128 * 100, dy_stride_t=70)),
        ("ssm_bwd", dict(ddt=FAR + 128 * 200, ddt_stride_t=65)),
        ("rn_fwd", dict(x=FAR + 128 * 7, x_stride_t=0)), ("rn_fwd", dict(x=FAR + 128 * 3, x_stride_t=100)),
        ("rn_fwd", dict(residual=FAKE + (1 << 20), residual_stride_t=64, residual_out=FAR + 128 * 6, residual_out_stride_t=80)),
        ("rn_fwd", dict(quantize=1, scales=FAKE, x=FAR + 64 * 5, x_stride_t=100)),
        ("rn_bwd", dict(s=FAR + 128 * 7, s_stride_t=0)), ("rn_bwd", dict(dy=FAR + 128 * 7 + 126, dy_stride_t=900)),
        ("rn_bwd", dict(ds=FAR + 128 * 7, ds_stride_t=65))]
# two vectors of 32 bytes a row
OVER_VECTORS = [("ssm_fwd", dict(b=FAR)), ("ssm_fwd", dict(c=FAR + 128 * 255)), ("ssm_fwd", dict(b=FAR + 128 * 5, b_stride_t=0)),
                ("ssm_fwd", dict(y_stride_t=128, c=FAR + 96, b_stride_t=128, c_stride_t=128)),
                ("ssm_fwd", dict(b=FAR - (1 << 20) + 64, b_stride_t=128, b_stride_g=1 << 19)), ("ssm_decode", dict(c=FAR + 128)),
                ("ssm_bwd", dict(b=FAR)), ("ssm_bwd", dict(c=FAR + (1 << 20))), ("ssm_bwd", dict(z=FAKE, z_stride_t=64, dz=FAKE + (1 << 21),
                 dz_stride_t=64, b=FAKE + (1 << 21) + 128 * 30))]
# the norm's weight (128 bytes), its gradient and the scales
EIGHT = dict(quantize=2, scales=FAR + (1 << 20))
OVER_PARAMETERS = [("rn_fwd", dict(weight=FAR + 128 * 7)), ("rn_fwd", dict(weight=FAR - 126, weight_dtype=0)),
                   ("rn_fwd", dict(residual=FAKE + (1 << 20), residual_stride_t=64, residual_out=FAKE + (1 << 21), residual_out_stride_t=64,
                                   weight=FAKE + (1 << 21) + 1000)),
                   ("rn_fwd", dict(EIGHT, scales=FAR)), ("rn_fwd", dict(EIGHT, scales=FAR + 64 * 8 - 4)), ("rn_fwd", dict(EIGHT, scales=FAKE + 128 * 8 - 4)),
                   ("rn_fwd", dict(EIGHT, weight=FAR + (1 << 20) + 28)),
                   ("rn_fwd", dict(EIGHT, residual=FAR + (1 << 20) - 1020, residual_stride_t=64, residual_out=FAKE + (1 << 21), residual_out_stride_t=64)),
                   ("rn_fwd", dict(EIGHT, residual=FAKE + (1 << 20), residual_stride_t=64, residual_out=FAR + (1 << 20) - 1020, residual_out_stride_t=64)),
                   ("rn_bwd", dict(d_weight=FAR + 128 * 7)), ("rn_bwd", dict(weight=FAR + 64, d_weight=FAKE + (1 << 22))),
                   ("rn_bwd", dict(ds=FAKE + (1 << 21), ds_stride_t=64, d_weight=FAKE + (1 << 21) + 512))]


def code(fn, over):
    cls, fields = VALID[fn]
    p = cls()
    for k, v in {**fields, **over}.items():
        setattr(p, k, v)
    return getattr(B.load(), fn)(ctypes.byref(p), None)


@pytest.mark.parametrize("fn,over", OVER + OVER_VECTORS + OVER_PARAMETERS, ids=lambda v: "-".join(f"{k}_{x:x}" for k, x in v.items()) if isinstance(v, dict) else v)
def test_rows_of_another_stride(fn, over):
    assert code(fn, over) == INV


@pytest.mark.gpu
def test_rows_beside_each_other():
    """Results between the rows and columns of a buffer that their operands lie in, with other strides."""
    T, D, S = 60, 64, 16
    gen = torch.Generator().manual_seed(1)
    cu = torch.tensor([0, 25, T], dtype=torch.int32, device="cuda")

    def randn(*shape):
        return torch.randn(*shape, generator=gen).to(torch.bfloat16).cuda()

    # every row of buf: x dt z b c in 3 D + 4 S columns, then D more of which every second row takes one of y
    wide = 4 * D + 4 * S
    buf = torch.zeros(2 * T, wide, dtype=torch.bfloat16, device="cuda")
    x, dt, z = (buf[:T, i * D:(i + 1) * D] for i in range(3))
    b, c = (buf[:T, 3 * D + i * 2 * S:3 * D + (i + 1) * 2 * S].unflatten(1, (2, S)) for i in range(2))
    y = buf[::2, 3 * D + 4 * S:]
    for v in (x, dt, z, b, c):
        v.copy_(randn(*v.shape))
    a = -torch.rand(D, S, generator=gen).cuda()
    ops, opts = (x, dt, a, b, c), dict(z=z, dt_softplus=True)
    want = la.ssm_fwd(*(v.clone() for v in ops), cu, **opts)[0]
    assert torch.equal(la.ssm_fwd(*ops, cu, y=y, **opts)[0], want)
    grads = la.ssm_bwd(*ops, cu, x, **opts)
    assert torch.equal(la.ssm_bwd(*ops, cu, x, dx=y, **opts)[0], grads[0])
    pool = torch.zeros(T, D, S, device="cuda")
    want = la.ssm_decode(*ops, pool.clone(), **opts)
    assert torch.equal(la.ssm_decode(*ops, pool, y=y, **opts), want)
    w = torch.randn(D, generator=gen).cuda()
    want, s, _ = la.rn_fwd(x, w, dt)
    assert torch.equal(la.rn_fwd(x, w, dt, y=y)[0], want)
    assert torch.equal(la.rn_bwd(x, w, z, dx=y)[0], la.rn_bwd(x, w, z)[0])
    for call in (lambda: la.ssm_fwd(*ops, cu, y=buf[::2, :D], **opts), lambda: la.ssm_decode(*ops, pool, y=buf[::2, 2 * D:3 * D], **opts),
                 lambda: la.ssm_decode(*ops, pool, y=buf[::2, 3 * D:4 * D], **opts), lambda: la.ssm_bwd(*ops, cu, x, ddt=buf[::2, 3 * D:4 * D], **opts),
                 lambda: la.rn_fwd(x, w, dt, y=buf[::2, D:2 * D])):
        with pytest.raises(B.LinAttnError):
            call()
