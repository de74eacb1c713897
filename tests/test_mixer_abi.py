"""The token-mixer entry points on the host: struct layout, workspace sizes and refusals (no GPU needed; the library
returns before any CUDA call, so the fake pointers are never read)."""
import ctypes

import pytest
import torch

import gated_delta_rule_29_gb300 as la
from gated_delta_rule_29_gb300 import binding as B
from test_abi import FAKE, _c_layout

OK_WS = 1 << 40


@pytest.mark.parametrize("cls,cname", [
    (B.GlrFwdParams, "la_glr_fwd_params"), (B.GlrBwdParams, "la_glr_bwd_params"),
    (B.GlrDecodeParams, "la_glr_decode_params"), (B.GnFwdParams, "la_gn_fwd_params"),
    (B.GnBwdParams, "la_gn_bwd_params"), (B.SconvFwdParams, "la_sconv_fwd_params"),
    (B.SconvBwdParams, "la_sconv_bwd_params"), (B.SconvDecodeParams, "la_sconv_decode_params")])
def test_ctypes_mirror_matches_c_layout(cls, cname):
    names = [f[0] for f in cls._fields_]
    size, offs = _c_layout(cname, names)
    assert ctypes.sizeof(cls) == size
    for name, off in zip(names, offs):
        assert getattr(cls, name).offset == off, name


GLR = dict(x=FAKE, x_stride_t=64, g=FAKE, g_stride_t=64, D=64, N=2, x_dtype=0, g_dtype=1)
SEQ = dict(cu_seqlens=FAKE, cu_seqlens_bits=32, T=256)
GN = dict(x=FAKE, x_stride_t=128, x_stride_h=64, weight=FAKE, T=8, H=2, V=64, eps=1e-5)
CONV = dict(x=FAKE, weight=FAKE, D=64, N=2, W=4)
VALID = {
    "glr_fwd": (B.GlrFwdParams, dict(GLR, **SEQ, h=FAKE, h_stride_t=64, workspace=FAKE, workspace_bytes=OK_WS)),
    "glr_bwd": (B.GlrBwdParams, dict(GLR, **SEQ, d_h=FAKE, d_h_stride_t=64, dx=FAKE, dx_stride_t=64, dg=FAKE,
                                     dg_stride_t=64, workspace=FAKE, workspace_bytes=OK_WS)),
    "glr_decode": (B.GlrDecodeParams, dict(x=FAKE, x_stride_n=64, g=FAKE, g_stride_n=64, g_dtype=1, D=64, N=2, state_pool=FAKE,
                                           state_dtype=1, state_pool_size=4, h=FAKE, h_stride_n=64)),
    "gn_fwd": (B.GnFwdParams, dict(GN, y=FAKE, y_stride_t=128, y_stride_h=64)),
    "gn_bwd": (B.GnBwdParams, dict(GN, dy=FAKE, dy_stride_t=128, dy_stride_h=64, dx=FAKE, dx_stride_t=128,
                                   dx_stride_h=64, d_weight=FAKE, workspace=FAKE, workspace_bytes=OK_WS)),
    "sconv_fwd": (B.SconvFwdParams, dict(CONV, **SEQ, x_stride_t=64, y=FAKE, y_stride_t=64)),
    "sconv_bwd": (B.SconvBwdParams, dict(CONV, **SEQ, x_stride_t=64, dy=FAKE, dy_stride_t=64, dx=FAKE, dx_stride_t=64,
                                         d_weight=FAKE, workspace=FAKE, workspace_bytes=OK_WS)),
    "sconv_decode": (B.SconvDecodeParams, dict(CONV, x_stride_n=64, state_pool=FAKE, state_pool_size=4, y=FAKE,
                                               y_stride_n=64)),
}
INV, UNS, WS = B.LA_ERR_INVALID_ARG, B.LA_ERR_UNSUPPORTED, B.LA_ERR_WORKSPACE
SEQ_BAD = [(dict(T=-1), INV), (dict(N=-1), INV), (dict(N=0), INV), (dict(cu_seqlens=None), INV),
           (dict(cu_seqlens_bits=16), INV), (dict(cu_seqlens=FAKE + 4, cu_seqlens_bits=64), INV), (dict(T=1 << 41), UNS)]
X_BAD = [(dict(x=None), INV), (dict(x=FAKE + 1), INV), (dict(D=0), INV), (dict(x_dtype=7), UNS)]
GATE_BAD = [(dict(gate_mode=1), UNS), (dict(gate_mode=9), INV), (dict(gate_mode=2, gate_lower_bound=0.0), INV),
            (dict(gate_mode=2, gate_lower_bound=float("-inf")), INV), (dict(g=None), INV), (dict(g=FAKE + 2), INV),
            (dict(g_dtype=2), UNS)]
GN_BAD = [(dict(T=-1), INV), (dict(H=0), INV), (dict(V=0), INV), (dict(V=8193), UNS), (dict(x=None), INV),
          (dict(x_dtype=2), UNS), (dict(weight_dtype=2), UNS), (dict(weight=None), INV), (dict(bias=FAKE + 1), INV),
          (dict(activation=3), INV), (dict(eps=0.0), INV), (dict(eps=float("nan")), INV), (dict(x_stride_t=-1), INV),
          (dict(z=FAKE + 1, z_stride_t=128, z_stride_h=64), INV)]
CONV_BAD = [(dict(W=1), UNS), (dict(W=5), UNS), (dict(weight=None), INV), (dict(weight_dtype=3), UNS),
            (dict(activation=-1), INV), (dict(bias=FAKE + 1), INV)]
REFUSALS = {
    "glr_fwd": SEQ_BAD + X_BAD + GATE_BAD + [
        (dict(h=None), INV), (dict(h_stride_t=63), INV), (dict(initial_state=FAKE, initial_state_dtype=5), UNS),
        (dict(initial_state=FAKE + 2, initial_state_dtype=1), INV), (dict(state_indices=FAKE, state_pool_size=2), INV),
        (dict(state_indices=FAKE, initial_state=FAKE, state_pool_size=0), INV),
        (dict(state_indices=FAKE, initial_state=FAKE, state_pool_size=2, final_state=FAKE), INV),
        (dict(checkpoints=FAKE + 2), INV)],
    "glr_bwd": SEQ_BAD + X_BAD + GATE_BAD + [
        (dict(d_h=None), INV), (dict(dx=None), INV), (dict(dg=None), INV), (dict(dx_stride_t=1), INV),
        (dict(d_final_state=FAKE + 1), INV), (dict(workspace=None), WS), (dict(workspace_bytes=64), WS),
        (dict(workspace=FAKE + 16), WS)],
    "glr_decode": X_BAD + GATE_BAD + [
        (dict(N=-1), INV), (dict(state_pool=None), INV), (dict(state_pool_size=1), INV), (dict(state_dtype=4), UNS),
        (dict(state_indices=FAKE + 2), INV), (dict(h=None), INV), (dict(h_stride_n=10), INV)],
    "gn_fwd": GN_BAD + [(dict(y=None), INV), (dict(y_stride_t=32), INV), (dict(y_stride_h=63), INV)],
    "gn_bwd": GN_BAD + [
        (dict(dy=None), INV), (dict(dx=None), INV), (dict(d_weight=None), INV), (dict(bias=FAKE), INV),
        (dict(z=FAKE, z_stride_t=128, z_stride_h=64), INV), (dict(workspace=None), WS), (dict(workspace_bytes=8), WS),
        (dict(workspace=FAKE + 128), WS)],
    "sconv_fwd": SEQ_BAD + X_BAD + CONV_BAD + [
        (dict(y=None), INV), (dict(y_stride_t=3), INV), (dict(initial_state=FAKE + 1), INV),
        (dict(state_indices=FAKE, state_pool_size=2), INV),
        (dict(state_indices=FAKE, initial_state=FAKE, state_pool_size=2, final_state=FAKE), INV)],
    "sconv_bwd": SEQ_BAD + X_BAD + CONV_BAD + [
        (dict(dy=None), INV), (dict(dx=None), INV), (dict(d_weight=None), INV), (dict(bias=FAKE), INV),
        (dict(workspace=None), WS), (dict(workspace_bytes=0), WS), (dict(workspace=FAKE + 64), WS)],
    "sconv_decode": X_BAD + CONV_BAD + [
        (dict(N=-1), INV), (dict(state_pool=None), INV), (dict(state_pool_size=1), INV), (dict(y=None), INV),
        (dict(state_indices=FAKE + 1), INV)],
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


def test_sizes():
    lib = B.load()
    assert la.glr_checkpoint_rows(0, 3) == 3 and la.glr_checkpoint_rows(1000, 3) == 10
    assert lib.la_glr_checkpoint_rows(-1, 3) == 0
    assert lib.la_glr_workspace_bytes(1000, 3, 70, 1, 0) >= 10 * 70 * 4
    assert lib.la_glr_workspace_bytes(1000, 3, 70, 1, 0) > lib.la_glr_workspace_bytes(1000, 3, 70, 1, 1)
    assert lib.la_glr_workspace_bytes(-1, 3, 70, 1, 0) == 0
    assert lib.la_gn_bwd_workspace_bytes(10, 2, 64, 0) > 0 and lib.la_gn_bwd_workspace_bytes(10, 2, 8193, 0) == 0
    assert lib.la_sconv_bwd_workspace_bytes(300, 2, 64, 4) > 0 and lib.la_sconv_bwd_workspace_bytes(300, 2, 64, 5) == 0


def test_wrappers_refuse_cpu_tensors():
    x, cu = torch.zeros(4, 8), torch.tensor([0, 4], dtype=torch.int32)
    for call in (lambda: la.glr_fwd(x, x, cu), lambda: la.glr_bwd(x, x, cu, x), lambda: la.glr_decode(x, x, x),
                 lambda: la.gn_fwd(x[None], x[0]), lambda: la.gn_bwd(x[None], x[0], x[None]),
                 lambda: la.sconv_fwd(x, torch.zeros(8, 4), cu), lambda: la.sconv_bwd(x, torch.zeros(8, 4), cu, x),
                 lambda: la.sconv_decode(x, torch.zeros(8, 4), x[None])):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()
