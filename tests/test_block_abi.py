"""The entry points of the selective scan and the residual norm on the host: struct layout, sizes and refusals (no GPU
needed; the library returns before any CUDA call, so the fake pointers are never read)."""
import ctypes

import pytest
import torch

import gated_delta_rule_29_gb300 as la
from gated_delta_rule_29_gb300 import binding as B
from test_abi import FAKE, _c_layout
from test_mixer_abi import INV, OK_WS, SEQ, SEQ_BAD, UNS, WS


@pytest.mark.parametrize("cls,cname", [
    (B.SsmFwdParams, "la_ssm_fwd_params"), (B.SsmBwdParams, "la_ssm_bwd_params"),
    (B.SsmDecodeParams, "la_ssm_decode_params"), (B.RnFwdParams, "la_rn_fwd_params"), (B.RnBwdParams, "la_rn_bwd_params")])
def test_ctypes_mirror_matches_c_layout(cls, cname):
    names = [f[0] for f in cls._fields_]
    size, offs = _c_layout(cname, names)
    assert ctypes.sizeof(cls) == size
    for name, off in zip(names, offs):
        assert getattr(cls, name).offset == off, name


FAR = FAKE + (1 << 30)
SSM = dict(x=FAKE, dt=FAKE, b=FAKE, c=FAKE, a=FAKE, D=64, N=2, S=16, G=2, b_stride_g=16, c_stride_g=16)
ROWS = dict(x_stride_t=64, dt_stride_t=64, z_stride_t=64, b_stride_t=32, c_stride_t=32)
WORK = dict(workspace=FAKE, workspace_bytes=OK_WS)
RN = dict(weight=FAKE, T=8, V=64, eps=1e-5)
VALID = {
    "ssm_fwd": (B.SsmFwdParams, dict(SSM, **SEQ, **ROWS, **WORK, y=FAR, y_stride_t=64)),
    "ssm_bwd": (B.SsmBwdParams, dict(SSM, **SEQ, **ROWS, **WORK, dy=FAKE, dy_stride_t=64, dx=FAR, dx_stride_t=64, ddt=FAR + (1 << 20),
                                     ddt_stride_t=64, db=FAR, dc=FAR, da=FAR)),
    "ssm_decode": (B.SsmDecodeParams, dict(SSM, x_stride_n=64, dt_stride_n=64, b_stride_n=32, c_stride_n=32, state_pool=FAKE,
                                           state_dtype=1, state_pool_size=4, y=FAR, y_stride_n=64)),
    "rn_fwd": (B.RnFwdParams, dict(RN, x=FAKE, x_stride_t=64, y=FAR, y_stride_t=64)),
    "rn_bwd": (B.RnBwdParams, dict(RN, s=FAKE, s_stride_t=64, dy=FAKE, dy_stride_t=64, dx=FAR, dx_stride_t=64, d_weight=FAR, **WORK)),
}
SSM_BAD = [(dict(x=None), INV), (dict(x=FAKE + 1), INV), (dict(dt=None), INV), (dict(b=None), INV), (dict(c=None), INV),
           (dict(b=FAKE + 1), INV), (dict(b_stride_g=-1), INV), (dict(a=None), INV), (dict(a=FAKE + 2), INV), (dict(skip=FAKE + 2), INV),
           (dict(dt_bias=FAKE + 2), INV), (dict(D=0), INV), (dict(S=0), INV), (dict(G=0), INV), (dict(G=3), INV), (dict(S=65), UNS),
           (dict(x_dtype=5), UNS), (dict(z=FAKE + 1), INV)]
REFUSALS = {
    "ssm_fwd": SEQ_BAD + SSM_BAD + [
        (dict(y=None), INV), (dict(y_stride_t=63), INV), (dict(initial_state=FAKE, initial_state_dtype=5), UNS),
        (dict(initial_state=FAKE + 2, initial_state_dtype=1), INV), (dict(state_indices=FAKE, state_pool_size=2), INV),
        (dict(state_indices=FAKE, initial_state=FAKE, state_pool_size=0), INV),
        (dict(state_indices=FAKE, initial_state=FAKE, state_pool_size=2, final_state=FAKE), INV), (dict(checkpoints=FAKE + 2), INV),
        (dict(time_block=-64), INV), (dict(time_block=32), INV), (dict(time_block=96), INV), (dict(workspace=None, time_block=64), WS),
        (dict(workspace_bytes=64, time_block=64), WS), (dict(workspace=FAKE + 16, time_block=64), WS),
        (dict(y=FAKE + 128), INV), (dict(y=FAKE, y_stride_t=128), INV)],
    "ssm_bwd": SEQ_BAD + SSM_BAD + [
        (dict(dy=None), INV), (dict(dx=None), INV), (dict(ddt=None), INV), (dict(dx_stride_t=1), INV), (dict(db=None), INV),
        (dict(dc=None), INV), (dict(da=None), INV), (dict(z=FAKE), INV), (dict(skip=FAKE), INV), (dict(dt_bias=FAKE), INV),
        (dict(d_final_state=FAKE + 1), INV), (dict(workspace=None), WS), (dict(workspace_bytes=64), WS), (dict(workspace=FAKE + 16), WS)],
    "ssm_decode": SSM_BAD + [
        (dict(N=-1), INV), (dict(state_pool=None), INV), (dict(state_pool_size=1), INV), (dict(state_dtype=4), UNS),
        (dict(state_indices=FAKE + 2), INV), (dict(y=None), INV), (dict(y_stride_n=10), INV)],
    "rn_fwd": [
        (dict(T=-1), INV), (dict(V=0), INV), (dict(V=16385), UNS), (dict(x=None), INV), (dict(x=FAKE + 1), INV), (dict(x_dtype=2), UNS),
        (dict(weight=None), INV), (dict(weight_dtype=2), UNS), (dict(eps=0.0), INV), (dict(eps=float("inf")), INV),
        (dict(x_stride_t=-1), INV), (dict(y=None), INV), (dict(y_stride_t=63), INV), (dict(y=FAR + 1), INV), (dict(quantize=4), INV),
        (dict(quantize=-1), INV), (dict(quantize=1), INV), (dict(quantize=1, scales=FAKE + 2), INV), (dict(quantize=3), INV),
        (dict(residual=FAKE, residual_stride_t=64), INV),
        (dict(residual=FAKE, residual_stride_t=64, residual_out=FAR, residual_out_stride_t=10), INV),
        (dict(x_dtype=1, residual=FAKE, residual_stride_t=64, residual_out=FAR, residual_out_stride_t=64), UNS)],
    "rn_bwd": [
        (dict(T=-1), INV), (dict(V=0), INV), (dict(V=16385), UNS), (dict(s=None), INV), (dict(dy=None), INV), (dict(dx=None), INV),
        (dict(x_dtype=1), UNS), (dict(s_dtype=3), UNS), (dict(d_weight=None), INV), (dict(eps=-1.0), INV), (dict(d_residual=FAKE + 1), INV),
        (dict(ds=FAKE + 1, ds_stride_t=64), INV), (dict(dx_stride_t=10), INV), (dict(workspace=None), WS), (dict(workspace_bytes=8), WS),
        (dict(workspace=FAKE + 128), WS)],
}


@pytest.mark.parametrize("fn,over,code", [(f, o, c) for f, cases in REFUSALS.items() for o, c in cases],
                         ids=lambda v: "-".join(f"{k}_{x}" for k, x in v.items()) if isinstance(v, dict) else None)
def test_refusals(fn, over, code):
    cls, fields = VALID[fn]
    p = cls()
    for k, v in {**fields, **over}.items():
        setattr(p, k, v)
    assert getattr(B.load(), fn)(ctypes.byref(p), None) == code
    assert getattr(B.load(), fn)(None, None) == INV


NEAR = FAKE + 64  # a row is 128 bytes of bf16
SHARED = {
    "ssm_decode": [dict(y=NEAR), dict(y=FAKE, y_stride_n=128), dict(y=FAKE + 128), dict(z=FAR + 128, z_stride_n=64)],
    "ssm_bwd": [dict(dx=FAKE), dict(dx=NEAR), dict(ddt=FAKE + 128), dict(ddt=FAR), dict(ddt=FAR + 64),
                dict(z=FAKE, z_stride_t=64, dz=FAKE, dz_stride_t=64), dict(z=FAKE, z_stride_t=64, dz=FAR, dz_stride_t=64),
                dict(dy=FAR + 128)],
    "rn_fwd": [dict(y=NEAR), dict(y=FAKE, y_stride_t=128), dict(y=FAKE, quantize=1, scales=FAR),
               dict(residual=FAKE, residual_stride_t=64, residual_out=FAR, residual_out_stride_t=64),  # y
               dict(residual=FAKE, residual_stride_t=64, residual_out=NEAR, residual_out_stride_t=64),
               dict(residual=FAKE, residual_stride_t=64, residual_out=FAKE, residual_out_stride_t=128),
               dict(residual=FAR + 128, residual_stride_t=64, residual_out=FAR + (1 << 20), residual_out_stride_t=64),  # y
               dict(residual=FAR + (1 << 20), residual_dtype=1, residual_stride_t=64, residual_out=FAKE, residual_out_stride_t=64)],
    "rn_bwd": [dict(dx=NEAR), dict(dx=FAKE, dx_stride_t=128), dict(dx=FAKE, s_dtype=1), dict(ds=FAR, ds_stride_t=64),
               dict(ds=FAR + 64, ds_stride_t=64), dict(ds=NEAR, ds_stride_t=64), dict(d_residual=FAR + 128, d_residual_stride_t=64)],
}


@pytest.mark.parametrize("fn,over", [(f, o) for f, cases in SHARED.items() for o in cases],
                         ids=lambda v: "-".join(f"{k}_{x}" for k, x in v.items()) if isinstance(v, dict) else None)
def test_results_over_other_operands_are_refused(fn, over):
    """Results that lie over an input other than element by element, or over each other."""
    cls, fields = VALID[fn]
    p = cls()
    for k, v in {**fields, **over}.items():
        setattr(p, k, v)
    assert getattr(B.load(), fn)(ctypes.byref(p), None) == INV


def test_sizes():
    lib = B.load()
    assert la.ssm_checkpoint_rows(0, 3) == 3 and la.ssm_checkpoint_rows(1000, 3) == 65
    assert lib.la_ssm_checkpoint_rows(-1, 3) == 0
    assert lib.la_ssm_fwd_workspace_bytes(128, 3, 70, 16, 1, 64) == 0
    assert lib.la_ssm_fwd_workspace_bytes(129, 3, 70, 16, 1, 64) >= 5 * 70 * 17 * 4
    assert lib.la_ssm_fwd_workspace_bytes(1000, 3, 70, 16, 1, 0) >= lib.la_ssm_fwd_workspace_bytes(1000, 3, 70, 16, 1, 512)
    for bad in ((-1, 3, 70, 16, 1), (10, 3, 70, 65, 1), (10, 3, 70, 16, 3)):
        assert lib.la_ssm_fwd_workspace_bytes(*bad, 64) == 0 and lib.la_ssm_bwd_workspace_bytes(*bad, 0) == 0
    assert lib.la_ssm_bwd_workspace_bytes(1000, 3, 70, 16, 1, 0) >= lib.la_ssm_bwd_workspace_bytes(1000, 3, 70, 16, 1, 1) + 65 * 70 * 16 * 4
    assert [lib.la_rn_scale_blocks(V, q) for V, q in ((4096, 0), (4096, 1), (4096, 2), (4097, 2), (33, 3), (0, 3), (5, 9))] == [0, 1, 32, 33, 2, 0, 0]
    assert lib.la_rn_bwd_workspace_bytes(10, 64) > 0 and lib.la_rn_bwd_workspace_bytes(10, 16385) == 0


def test_wrappers_refuse_cpu_tensors():
    x, cu, v = torch.zeros(4, 8), torch.tensor([0, 4], dtype=torch.int32), torch.zeros(4, 2)
    a = torch.zeros(8, 2)
    for call in (lambda: la.ssm_fwd(x, x, a, v, v, cu), lambda: la.ssm_bwd(x, x, a, v, v, cu, x), lambda: la.ssm_decode(x, x, a, v, v, x[None]),
                 lambda: la.rn_fwd(x, x[0]), lambda: la.rn_bwd(x, x[0], x)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()


def test_a_stream_of_another_device_is_refused_by_keyword():
    """Also where the first operand is not called x."""
    import types

    from test_mixer_device import CudaOperand
    s = torch.zeros(4, 8).as_subclass(CudaOperand)
    with pytest.raises(ValueError, match="stream must be on cuda:0"):
        la.rn_bwd(s=s, weight=s[0], dy=s, stream=types.SimpleNamespace(device=torch.device("cuda", 1)))
