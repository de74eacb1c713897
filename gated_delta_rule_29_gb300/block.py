"""Torch-facing wrappers of the operators of a state-space block: the selective state space scan (ssm_*) and the
root-mean-square norm with the residual's addition (rn_*), and their autograd forms.

As in mixer.py, PyTorch only supplies device memory and the stream; every step runs in the library's CUDA kernels.
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch

from . import binding as B
from .mixer import (_DTYPES, _FP32, _STATE_DTYPES, _call, _cotangent, _dtype, _indices, _on_stream, _packed, _result, _rows,
                    _sequences, _state_dest, _status, _workspace)


# ------------------------------------------------------------------ selective state space scan
def ssm_checkpoint_rows(T: int, N: int) -> int:
    """Rows of ssm_fwd's checkpoints for T tokens in N sequences."""
    return int(B.load().la_ssm_checkpoint_rows(int(T), int(N)))


def _like(name: str, v, like: torch.Tensor) -> int:
    """Row stride of an operand of the shape, type and device of `like`, rank 2."""
    if isinstance(v, torch.Tensor) and v.dtype is like.dtype and v.shape == like.shape and v.get_device() == like.get_device():
        row, last = v.stride()
        if last == 1:
            return row
    row = _rows(name, v, 2, like)[0]
    if v.dtype != like.dtype:
        raise TypeError(f"{name} must be {like.dtype}, got {v.dtype}")
    return row


def _vectors(name: str, v, rows: int, like: torch.Tensor) -> tuple:
    """Strides (row, group) and shape (G, S) of [rows, S] or [rows, G, S] vectors of the type of `like`."""
    shape = getattr(v, "shape", ())
    strides = _rows(name, v, 2 if len(shape) == 2 else 3)
    if v.dtype != like.dtype:
        raise TypeError(f"{name} must be {like.dtype}, got {v.dtype}")
    if shape[0] != rows or v.get_device() != like.get_device():
        raise ValueError(f"{name} must have {rows} rows on {like.device}, got {tuple(shape)} on {v.device}")
    return (strides[0], 0, 1, shape[1]) if len(shape) == 2 else (strides[0], strides[1], shape[1], shape[2])


def _ssm_inputs(cls, x, dt, a, b, c, skip, z, dt_bias, dt_softplus) -> tuple:
    """The call's parameters with the operands, which are the first fields of every ssm_* struct in the same order, filled
    in; and (rows, D, S, G)."""
    x_row = _rows("x", x, 2)[0]
    _dtype("x", x)
    rows, D = x.shape
    dt_row = _like("dt", dt, x)
    z_row, z_at = (0, None) if z is None else (_like("z", z, x), z.data_ptr())
    b_row, b_group, G, S = _vectors("b", b, rows, x)
    c_row, c_group, c_G, c_S = _vectors("c", c, rows, x)
    if (c_G, c_S) != (G, S):
        raise ValueError(f"b and c must have the same shape, got {tuple(b.shape)} and {tuple(c.shape)}")
    if G < 1 or D % G:
        raise ValueError(f"the {D} channels must be a multiple of the {G} groups of b and c")
    p = cls(x.data_ptr(), x_row, dt.data_ptr(), dt_row, z_at, z_row, b.data_ptr(), b_row, b_group, c.data_ptr(), c_row, c_group,
            _packed("a", a, (D, S), _FP32, x), None if skip is None else _packed("skip", skip, (D,), _FP32, x),
            None if dt_bias is None else _packed("dt_bias", dt_bias, (D,), _FP32, x), bool(dt_softplus))
    p.D, p.S, p.G, p.x_dtype = D, S, G, _DTYPES[x.dtype]
    return p, rows, D, S, G


@_on_stream
def ssm_fwd(x: torch.Tensor, dt: torch.Tensor, a: torch.Tensor, b: torch.Tensor, c: torch.Tensor,
            cu_seqlens: torch.Tensor, *, skip: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
            dt_bias: Optional[torch.Tensor] = None, dt_softplus: bool = False,
            initial_state: Optional[torch.Tensor] = None, output_final_state: bool = True,
            output_checkpoints: bool = False, state_indices: Optional[torch.Tensor] = None, time_block: int = 0,
            y: Optional[torch.Tensor] = None, final_state: Optional[torch.Tensor] = None,
            checkpoints: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
            status: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None
            ) -> Tuple[torch.Tensor, Optional[torch.Tensor], Optional[torch.Tensor]]:
    """Selective state space scan: h_t = exp(dt_t a) h_{t-1} + dt_t x_t b_t for S states a channel of every sequence,
    y_t = c_t h_t + skip x_t, times silu(z_t) with the gate z.  Returns (y [T, D] in x's dtype, final_state [N, D, S]
    fp32 or None, checkpoints or None).  Asynchronous on the current stream.

    x, dt, z [T, D] and b, c [T, S] or [T, G, S] (channels in G groups) are of one dtype, bf16 or fp32; a [D, S]
    (rates, <= 0 for states that decay), skip, dt_bias [D] are fp32.  dt_t is dt + dt_bias, or softplus of that with
    dt_softplus.

    output_checkpoints keeps the fp32 state entering every 16 tokens for ssm_bwd.  state_indices ([N] int32):
    initial_state is then a pool [P, D, S] and each sequence's end state is written back to its slot.  time_block (0, or a
    power of two from 64 on): sequences longer than two such blocks are split along time; 0 chooses by T, D, S and the groups, a
    given one makes a sequence's bits independent of the batch around it."""
    p, T, D, S, G = _ssm_inputs(B.SsmFwdParams, x, dt, a, b, c, skip, z, dt_bias, dt_softplus)
    p.T = T
    N = _sequences(p, cu_seqlens, x)
    if time_block < 0 or time_block & (time_block - 1) or 0 < time_block < 64 or time_block > 1 << 30:
        raise ValueError(f"time_block must be 0 or a power of two from 64 to 2^30, got {time_block}")
    p.time_block = time_block
    if state_indices is not None:
        if initial_state is None or initial_state.dim() != 3:
            raise ValueError("state_indices needs initial_state as a contiguous pool [P, D, S]")
        if final_state is not None:
            raise ValueError("state_indices and final_state are exclusive")
        _indices(p, state_indices, N, x)
        p.state_pool_size = initial_state.shape[0]
        output_final_state = False
    if initial_state is not None:
        rows = N if state_indices is None else initial_state.shape[0]
        p.initial_state = _packed("initial_state", initial_state, (rows, D, S), _STATE_DTYPES, x)
        p.initial_state_dtype = _DTYPES[initial_state.dtype]
    y, strides = _result("y", y, x)
    p.y, p.y_stride_t = y.data_ptr(), strides[0]
    if output_final_state:
        final_state, p.final_state = _state_dest("final_state", final_state, (N, D, S), torch.float32, x)
    else:
        final_state = None
    if output_checkpoints or checkpoints is not None:
        checkpoints, p.checkpoints = _state_dest("checkpoints", checkpoints, (ssm_checkpoint_rows(T, N), D, S),
                                                 torch.float32, x)
    need = B.load().la_ssm_fwd_workspace_bytes(T, N, D, S, G, time_block)
    ws = _workspace(p, workspace, need, x)  # noqa: F841
    if status is not None:
        _status(p, status, x)
    _call("ssm_fwd", p, x)
    return y, final_state, checkpoints


@_on_stream
def ssm_bwd(x: torch.Tensor, dt: torch.Tensor, a: torch.Tensor, b: torch.Tensor, c: torch.Tensor,
            cu_seqlens: torch.Tensor, dy: torch.Tensor, *, skip: Optional[torch.Tensor] = None,
            z: Optional[torch.Tensor] = None, dt_bias: Optional[torch.Tensor] = None, dt_softplus: bool = False,
            initial_state: Optional[torch.Tensor] = None, d_final_state: Optional[torch.Tensor] = None,
            checkpoints: Optional[torch.Tensor] = None, dx: Optional[torch.Tensor] = None,
            ddt: Optional[torch.Tensor] = None, dz: Optional[torch.Tensor] = None,
            workspace: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
            stream: Optional[torch.cuda.Stream] = None) -> tuple:
    """Gradients of sum(dy * y) + sum(d_final_state * final_state) for ssm_fwd with the same inputs: (dx, ddt, da, db,
    dc, d_skip or None, dz or None, d_dt_bias or None, d_initial_state [N, D, S] fp32), each in its input's dtype.
    checkpoints: the forward's; without them the states are recomputed (one more forward pass)."""
    p, T, D, S, G = _ssm_inputs(B.SsmBwdParams, x, dt, a, b, c, skip, z, dt_bias, dt_softplus)
    p.T = T
    N = _sequences(p, cu_seqlens, x)
    p.dy, p.dy_stride_t = dy.data_ptr() if isinstance(dy, torch.Tensor) else None, _like("dy", dy, x)
    if initial_state is not None:
        p.initial_state = _packed("initial_state", initial_state, (N, D, S), _STATE_DTYPES, x)
        p.initial_state_dtype = _DTYPES[initial_state.dtype]
    if d_final_state is not None:
        p.d_final_state = _packed("d_final_state", d_final_state, (N, D, S), _FP32, x)
    if checkpoints is not None:
        p.checkpoints = _packed("checkpoints", checkpoints, (ssm_checkpoint_rows(T, N), D, S), _FP32, x)
    dx, strides = _result("dx", dx, x)
    p.dx, p.dx_stride_t = dx.data_ptr(), strides[0]
    ddt, strides = _result("ddt", ddt, x)
    p.ddt, p.ddt_stride_t = ddt.data_ptr(), strides[0]
    if z is not None:
        dz, strides = _result("dz", dz, x)
        p.dz, p.dz_stride_t = dz.data_ptr(), strides[0]
    else:
        dz = None
    db, dc, da = (torch.empty_like(v, memory_format=torch.contiguous_format) for v in (b, c, a))
    p.db, p.dc, p.da = db.data_ptr(), dc.data_ptr(), da.data_ptr()
    d_skip = d_bias = None
    if skip is not None:
        d_skip = torch.empty_like(skip)
        p.d_skip = d_skip.data_ptr()
    if dt_bias is not None:
        d_bias = torch.empty_like(dt_bias)
        p.d_dt_bias = d_bias.data_ptr()
    d_initial, p.d_initial_state = _state_dest("d_initial_state", None, (N, D, S), torch.float32, x)
    need = B.load().la_ssm_bwd_workspace_bytes(T, N, D, S, G, checkpoints is not None)
    ws = _workspace(p, workspace, need, x)  # noqa: F841
    if status is not None:
        _status(p, status, x)
    _call("ssm_bwd", p, x)
    return dx, ddt, da, db, dc, d_skip, dz, d_bias, d_initial


@_on_stream
def ssm_decode(x: torch.Tensor, dt: torch.Tensor, a: torch.Tensor, b: torch.Tensor, c: torch.Tensor,
               state_pool: torch.Tensor, *, state_indices: Optional[torch.Tensor] = None,
               skip: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
               dt_bias: Optional[torch.Tensor] = None, dt_softplus: bool = False, y: Optional[torch.Tensor] = None,
               status: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """One scan step for each of N sequences: x, dt, z [N, D], b, c [N, S] or [N, G, S]; sequence i steps
    pool[state_indices[i]] (pool[i] without indices) of state_pool [P, D, S] (fp32 or bf16) in place.  Returns y [N, D]
    in x's dtype."""
    p, N, D, S, _ = _ssm_inputs(B.SsmDecodeParams, x, dt, a, b, c, skip, z, dt_bias, dt_softplus)
    p.N = N
    if not isinstance(state_pool, torch.Tensor) or state_pool.dim() != 3:
        raise ValueError("state_pool must be a contiguous [P, D, S] tensor")
    p.state_pool_size = P = state_pool.shape[0]
    p.state_pool = _packed("state_pool", state_pool, (P, D, S), _STATE_DTYPES, x)
    p.state_dtype = _DTYPES[state_pool.dtype]
    if state_indices is not None:
        _indices(p, state_indices, N, x)
    y, strides = _result("y", y, x)
    p.y, p.y_stride_n = y.data_ptr(), strides[0]
    if status is not None:
        _status(p, status, x)
    _call("ssm_decode", p, x)
    return y


# ------------------------------------------------------------------ residual norm
_QUANTIZE = {None: B.LA_QUANT_NONE, "row": B.LA_QUANT_ROW, "block": B.LA_QUANT_BLOCK, "mx": B.LA_QUANT_MX}


def _rn_weight(p, weight, like: torch.Tensor, eps: float) -> None:
    p.weight, p.weight_dtype = _packed("weight", weight, (like.shape[1],), _STATE_DTYPES, like), _DTYPES[weight.dtype]
    p.eps = eps


@_on_stream
def rn_fwd(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None, *, eps: float = 1e-5,
           quantize: Optional[str] = None, y: Optional[torch.Tensor] = None,
           residual_out: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None,
           stream: Optional[torch.cuda.Stream] = None
           ) -> Tuple[torch.Tensor, torch.Tensor, Optional[torch.Tensor]]:
    """Root-mean-square norm of every row of s = x + residual (x [T, V], bf16 or fp32; residual in x's dtype or fp32),
    times weight [V].  Returns (y, s, scales): s in the residual's dtype (x itself without a residual), y in x's dtype
    and scales None, or with quantize

      "row"    y float8_e4m3fn, scales [T, 1] fp32, one for each row
      "block"  the same, one for each block of 128 columns
      "mx"     one for each block of 32 columns, a power of two (float8_e8m0fnu, as block-scaled products take them).

    residual_out may be the residual (or x): the stream is then updated in place."""
    p = B.RnFwdParams()
    p.x_stride_t = _rows("x", x, 2)[0]
    p.x, p.x_dtype = x.data_ptr(), _dtype("x", x)
    p.T, p.V = T, V = x.shape
    _rn_weight(p, weight, x, eps)
    if residual is not None:
        p.residual_stride_t = _rows("residual", residual, 2, x)[0]
        p.residual, p.residual_dtype = residual.data_ptr(), _dtype("residual", residual)
        residual_out, strides = _result("residual_out", residual_out, residual)
        p.residual_out, p.residual_out_stride_t = residual_out.data_ptr(), strides[0]
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    try:
        p.quantize = kind = _QUANTIZE[quantize]
    except KeyError:
        raise ValueError(f"quantize must be None, 'row', 'block' or 'mx', got {quantize!r}") from None
    if kind == B.LA_QUANT_NONE:
        if scales is not None:
            raise ValueError("scales needs quantize")
        y, strides = _result("y", y, x)
    else:
        if y is None:
            y = torch.empty((T, V), dtype=torch.float8_e4m3fn, device=x.device)
        strides = _rows("y", y, 2, x)
        if y.dtype != torch.float8_e4m3fn:
            raise TypeError(f"y must be {torch.float8_e4m3fn}, got {y.dtype}")
        shape = (T, B.load().la_rn_scale_blocks(V, kind))
        scales, p.scales = _state_dest("scales", scales, shape, torch.float8_e8m0fnu if quantize == "mx" else torch.float32, x)
    p.y, p.y_stride_t = y.data_ptr(), strides[0]
    _call("rn_fwd", p, x)
    return y, (x if residual is None else residual_out), scales


@_on_stream
def rn_bwd(s: torch.Tensor, weight: torch.Tensor, dy: torch.Tensor, *, d_residual: Optional[torch.Tensor] = None,
           eps: float = 1e-5, dx: Optional[torch.Tensor] = None, ds: Optional[torch.Tensor] = None,
           workspace: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None
           ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Gradients of sum(dy * y) + sum(d_residual * s) for rn_fwd that returned s (an 8-bit result counts as y itself):
    (dx in dy's dtype, d_weight, ds in s's dtype: the residual's gradient, and dx itself where the dtypes are one)."""
    p = B.RnBwdParams()
    p.s_stride_t = _rows("s", s, 2)[0]
    p.s, p.s_dtype = s.data_ptr(), _dtype("s", s)
    p.T, p.V = T, V = s.shape
    p.dy_stride_t = _rows("dy", dy, 2, s)[0]
    p.dy, p.x_dtype = dy.data_ptr(), _dtype("dy", dy)
    if d_residual is not None:
        p.d_residual_stride_t = _like("d_residual", d_residual, s)
        p.d_residual = d_residual.data_ptr()
    _rn_weight(p, weight, s, eps)
    dx, strides = _result("dx", dx, dy)
    p.dx, p.dx_stride_t = dx.data_ptr(), strides[0]
    if s.dtype != dy.dtype:
        ds, strides = _result("ds", ds, s)
        p.ds, p.ds_stride_t = ds.data_ptr(), strides[0]
    elif ds is not None:
        raise ValueError("ds is dx where s and dy have one dtype")
    else:
        ds = dx
    d_weight = torch.empty_like(weight)
    p.d_weight = d_weight.data_ptr()
    ws = _workspace(p, workspace, B.load().la_rn_bwd_workspace_bytes(T, V), s)  # noqa: F841
    _call("rn_bwd", p, s)
    return dx, d_weight, ds


# ------------------------------------------------------------------ autograd
class _SelectiveScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, dt, a, b, c, cu_seqlens, skip, z, dt_bias, initial_state, dt_softplus, save_checkpoints, time_block):
        y, fin, ck = ssm_fwd(x, dt, a, b, c, cu_seqlens, skip=skip, z=z, dt_bias=dt_bias, dt_softplus=dt_softplus,
                             initial_state=initial_state, output_checkpoints=save_checkpoints, time_block=time_block)
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(x, dt, a, b, c, cu_seqlens, skip, z, dt_bias, initial_state, ck)
        ctx.dt_softplus = dt_softplus
        return y, fin

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, d_fin):
        x, dt, a, b, c, cu, skip, z, dt_bias, s0, ck = ctx.saved_tensors
        if d_fin is not None:
            d_fin = d_fin.float().contiguous()
        dx, ddt, da, db, dc, d_skip, dz, d_bias, ds0 = ssm_bwd(
            x, dt, a, b, c, cu, _cotangent(dy, x), skip=skip, z=z, dt_bias=dt_bias, dt_softplus=ctx.dt_softplus,
            initial_state=s0, d_final_state=d_fin, checkpoints=ck)
        return dx, ddt, da, db, dc, None, d_skip, dz, d_bias, None if s0 is None else ds0.to(s0.dtype), None, None, None


def selective_scan(x: torch.Tensor, dt: torch.Tensor, a: torch.Tensor, b: torch.Tensor, c: torch.Tensor,
                   cu_seqlens: torch.Tensor, *, skip: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
                   dt_bias: Optional[torch.Tensor] = None, dt_softplus: bool = False,
                   initial_state: Optional[torch.Tensor] = None, save_checkpoints: bool = True, time_block: int = 0
                   ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Differentiable ssm_fwd: returns (y, final_state); gradients flow to x, dt, a, b, c, skip, z, dt_bias and
    initial_state.  save_checkpoints keeps the state entering every 16 tokens (D * S * 4 bytes each) for the backward, where
    there will be one; without them it recomputes them (in the blocks of time_block 0)."""
    save_checkpoints = save_checkpoints and torch.is_grad_enabled() and any(
        getattr(v, "requires_grad", False) for v in (x, dt, a, b, c, skip, z, dt_bias, initial_state))
    return _SelectiveScan.apply(x, dt, a, b, c, cu_seqlens, skip, z, dt_bias, initial_state, dt_softplus, save_checkpoints,
                                time_block)


class _ResidualNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        y, s, _ = rn_fwd(x, weight, residual, eps=eps)
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(s, weight)
        ctx.eps, ctx.dtype, ctx.added = eps, x.dtype, residual is not None
        return (y, s) if ctx.added else y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, d_s=None):
        s, weight = ctx.saved_tensors
        dy = torch.zeros_like(s, dtype=ctx.dtype) if dy is None else _cotangent(dy, dy)  # the type of y, which is x's
        dx, dw, ds = rn_bwd(s, weight, dy, d_residual=None if d_s is None else _cotangent(d_s, s), eps=ctx.eps)
        return dx, dw, (ds if ctx.added else None), None


def residual_norm(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None, *, eps: float = 1e-5):
    """Differentiable rn_fwd without quantize: (y, x + residual), or y alone without a residual; gradients flow to x,
    weight and residual."""
    return _ResidualNorm.apply(x, weight, residual, eps)
