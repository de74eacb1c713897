"""Torch-facing wrappers of the token-mixer operators: the gated linear recurrence (glr_*), the
per-head group norm with an activation or gate (gn_*), the short causal convolution (sconv_*), and
their autograd forms.

As in api.py, PyTorch only supplies device memory and the stream; every step runs in the library's
CUDA kernels.  Outputs and workspaces are allocated on the stream the call runs on.
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional, Tuple

import torch

from . import binding as B
from .api import _cu_bits

_DTYPES = {torch.bfloat16: B.LA_DTYPE_BF16, torch.float32: B.LA_DTYPE_F32}
_ACTIVATIONS = {None: B.LA_ACT_NONE, "none": B.LA_ACT_NONE, "silu": B.LA_ACT_SILU, "sigmoid": B.LA_ACT_SIGMOID}


def _dtype(name: str, x: torch.Tensor) -> int:
    d = _DTYPES.get(x.dtype)
    if d is None:
        raise TypeError(f"{name} must be bfloat16 or float32, got {x.dtype} (dtypes are strict)")
    return d


def _activation(name) -> int:
    try:
        return _ACTIVATIONS[name]
    except KeyError:
        raise ValueError(f"activation must be one of 'none', 'silu', 'sigmoid', got {name!r}") from None


def _rows(name: str, x, rank: int, like: Optional[torch.Tensor] = None) -> tuple:
    """Strides of a rank-2 or rank-3 CUDA operand with a contiguous innermost axis; `like`: the operand whose
    shape and device it must have."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    strides = x.stride()
    if len(strides) != rank:
        raise ValueError(f"{name} must be rank {rank}, got shape {tuple(x.shape)}")
    if strides[-1] != 1 and x.shape[-1] > 1:
        raise ValueError(f"{name} must have a contiguous innermost axis")
    if like is not None and (x.shape != like.shape or x.get_device() != like.get_device()):
        raise ValueError(f"{name} must have shape {tuple(like.shape)} on {like.device}, got {tuple(x.shape)} on {x.device}")
    return strides


def _packed(name: str, x, shape: tuple, dtypes: tuple, like: torch.Tensor) -> int:
    """Address of a contiguous operand of a known shape (a parameter, a state) on the device of `like`."""
    if not isinstance(x, torch.Tensor) or x.get_device() != like.get_device():
        raise ValueError(f"{name} must be a tensor on {like.device}")
    if x.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {x.dtype}")
    if x.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(x.shape)}")
    if not x.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return x.data_ptr()


def _result(name: str, x: Optional[torch.Tensor], like: torch.Tensor) -> tuple:
    """A caller's output with the shape and dtype of `like`, or a new contiguous one, and its strides."""
    if x is None:
        x = torch.empty_like(like, memory_format=torch.contiguous_format)
        return x, x.stride()
    strides = _rows(name, x, like.dim(), like)
    if x.dtype != like.dtype:
        raise TypeError(f"{name} must be {like.dtype}, got {x.dtype}")
    return x, strides


def _state_dest(name: str, x: Optional[torch.Tensor], shape: tuple, dtype: torch.dtype, like: torch.Tensor) -> tuple:
    if x is None:
        x = torch.empty(shape, dtype=dtype, device=like.device)
        return x, x.data_ptr()
    return x, _packed(name, x, shape, (dtype,), like)


def _sequences(p, cu_seqlens: torch.Tensor, like: torch.Tensor) -> int:
    if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.get_device() != like.get_device():
        raise ValueError(f"cu_seqlens must be a tensor on {like.device}")
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1 or not cu_seqlens.is_contiguous():
        raise ValueError("cu_seqlens must be a contiguous [N + 1] vector")
    p.cu_seqlens, p.cu_seqlens_bits = cu_seqlens.data_ptr(), _cu_bits(cu_seqlens)
    p.N = N = cu_seqlens.numel() - 1
    return N


def _indices(p, state_indices, N: int, like: torch.Tensor) -> None:
    if state_indices.dtype != torch.int32 or state_indices.shape != (N,) \
            or state_indices.get_device() != like.get_device() or not state_indices.is_contiguous():
        raise ValueError(f"state_indices must be a contiguous int32 [{N}] vector on {like.device}")
    p.state_indices = state_indices.data_ptr()


def _workspace(p, workspace: Optional[torch.Tensor], need: int, like: torch.Tensor) -> Optional[torch.Tensor]:
    if workspace is None:
        if need == 0:
            return None
        workspace = torch.empty(need, dtype=torch.uint8, device=like.device)
    elif workspace.get_device() != like.get_device() or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous on {like.device}")
    p.workspace, p.workspace_bytes = workspace.data_ptr(), workspace.nbytes
    return workspace


def _status(p, status: torch.Tensor, like: torch.Tensor) -> None:
    if status.dtype != torch.int32 or status.numel() < 1 or status.get_device() != like.get_device():
        raise ValueError(f"status must be int32 on {like.device}")
    p.status = status.data_ptr()


def _on_stream(fn):
    """Makes a wrapper's `stream` argument, which must be on the device of its first operand, the current stream while
    it runs, so that what it allocates belongs to that stream."""
    @functools.wraps(fn)
    def call(*args, **kwargs):
        stream = kwargs.get("stream")
        if stream is None:
            return fn(*args, **kwargs)
        x = args[0] if args else kwargs.get("x", kwargs.get("s"))
        if isinstance(x, torch.Tensor) and x.is_cuda and stream.device != x.device:
            raise ValueError(f"stream must be on {x.device}, got one on {stream.device}")
        with torch.cuda.stream(stream):
            return fn(*args, **kwargs)
    return call


_functions = {}


def _call(name: str, p, like: torch.Tensor) -> None:
    """One library call on the operands' device, which the library takes from the thread, and its current stream."""
    fn = _functions.get(name)
    if fn is None:
        fn = _functions[name] = getattr(B.load(), name)
    device = like.get_device()
    if device == _current_device():
        code = fn(ctypes.byref(p), _raw_stream(device))
    else:
        with torch.cuda.device(device):
            code = fn(ctypes.byref(p), _raw_stream(device))
    if code:
        B.check(code, name)


def _raw_stream(device: int) -> int:
    return torch.cuda.current_stream(device).cuda_stream


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _raw_stream)  # the same without a Python Stream object
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


# ------------------------------------------------------------------ gated linear recurrence
def _gate(p, gate_logsigmoid: bool, gate_lower_bound: Optional[float], complement_input: bool) -> None:
    if gate_logsigmoid and gate_lower_bound is not None:
        raise ValueError("choose one gate transform: gate_logsigmoid or gate_lower_bound")
    if gate_lower_bound is not None:
        p.gate_mode, p.gate_lower_bound = B.LA_GATE_SIGMOID_BOUND, float(gate_lower_bound)
    elif gate_logsigmoid:
        p.gate_mode = B.LA_GATE_LOGSIGMOID
    p.complement_input = int(bool(complement_input))


_STATE_DTYPES = (torch.float32, torch.bfloat16)
_FP32 = (torch.float32,)


def glr_checkpoint_rows(T: int, N: int) -> int:
    """Rows of glr_fwd's checkpoints for T tokens in N sequences."""
    return int(B.load().la_glr_checkpoint_rows(int(T), int(N)))


def _glr_inputs(p, x, g, gate_logsigmoid, gate_lower_bound, complement_input) -> tuple:
    xs, gs = _rows("x", x, 2), _rows("g", g, 2, x)
    p.x, p.x_dtype, p.g, p.g_dtype = x.data_ptr(), _dtype("x", x), g.data_ptr(), _dtype("g", g)
    if gate_logsigmoid or gate_lower_bound is not None or complement_input:
        _gate(p, gate_logsigmoid, gate_lower_bound, complement_input)
    return xs[0], gs[0]


@_on_stream
def glr_fwd(x: torch.Tensor, g: torch.Tensor, cu_seqlens: torch.Tensor, *,
            initial_state: Optional[torch.Tensor] = None, output_final_state: bool = True,
            gate_logsigmoid: bool = False, gate_lower_bound: Optional[float] = None,
            complement_input: bool = False, output_checkpoints: bool = False,
            state_indices: Optional[torch.Tensor] = None, h: Optional[torch.Tensor] = None,
            final_state: Optional[torch.Tensor] = None, checkpoints: Optional[torch.Tensor] = None,
            workspace: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
            stream: Optional[torch.cuda.Stream] = None
            ) -> Tuple[torch.Tensor, Optional[torch.Tensor], Optional[torch.Tensor]]:
    """Gated linear recurrence h_t = a_t h_{t-1} + m_t x_t per channel of every sequence.  Returns (h [T, D] in
    x's dtype, final_state [N, D] fp32 or None, checkpoints or None).  Asynchronous on the current stream.

    x, g [T, D] (bf16 or fp32 each).  g is the natural-log decay, a = exp(g) with g <= 0, unless gate_logsigmoid
    (a = sigmoid(g)) or gate_lower_bound < 0 (a = exp(gate_lower_bound * sigmoid(g))) is given.  m = 1, or 1 - a
    with complement_input.

    output_checkpoints keeps the fp32 state entering every 128-token block for glr_bwd.  state_indices ([N]
    int32): initial_state is then a pool [P, D] and each sequence's end state is written back to its slot."""
    p = B.GlrFwdParams()
    p.x_stride_t, p.g_stride_t = _glr_inputs(p, x, g, gate_logsigmoid, gate_lower_bound, complement_input)
    p.T, p.D = T, D = x.shape
    N = _sequences(p, cu_seqlens, x)
    if state_indices is not None:
        if initial_state is None or initial_state.dim() != 2:
            raise ValueError("state_indices needs initial_state as a contiguous pool [P, D]")
        if final_state is not None:
            raise ValueError("state_indices and final_state are exclusive")
        _indices(p, state_indices, N, x)
        p.state_pool_size = initial_state.shape[0]
        output_final_state = False
    if initial_state is not None:
        rows = N if state_indices is None else initial_state.shape[0]
        p.initial_state = _packed("initial_state", initial_state, (rows, D), _STATE_DTYPES, x)
        p.initial_state_dtype = _DTYPES[initial_state.dtype]
    h, strides = _result("h", h, x)
    p.h, p.h_stride_t = h.data_ptr(), strides[0]
    if output_final_state:
        final_state, p.final_state = _state_dest("final_state", final_state, (N, D), torch.float32, x)
    else:
        final_state = None
    if output_checkpoints or checkpoints is not None:
        checkpoints, p.checkpoints = _state_dest("checkpoints", checkpoints, (glr_checkpoint_rows(T, N), D),
                                                 torch.float32, x)
    ws = _workspace(p, workspace, B.load().la_glr_workspace_bytes(T, N, D, 0, 0), x)  # noqa: F841
    if status is not None:
        _status(p, status, x)
    _call("glr_fwd", p, x)
    return h, final_state, checkpoints


@_on_stream
def glr_bwd(x: torch.Tensor, g: torch.Tensor, cu_seqlens: torch.Tensor, d_h: torch.Tensor, *,
            initial_state: Optional[torch.Tensor] = None, d_final_state: Optional[torch.Tensor] = None,
            checkpoints: Optional[torch.Tensor] = None, gate_logsigmoid: bool = False,
            gate_lower_bound: Optional[float] = None, complement_input: bool = False,
            dx: Optional[torch.Tensor] = None, dg: Optional[torch.Tensor] = None,
            d_initial_state: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
            status: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None
            ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Gradients of sum(d_h * h) + sum(d_final_state * final_state) for glr_fwd with the same inputs.  Returns (dx
    in x's dtype, dg of g as given in g's dtype, d_initial_state [N, D] fp32).  checkpoints: the forward's; without
    them the states are recomputed (one more forward pass)."""
    p = B.GlrBwdParams()
    p.x_stride_t, p.g_stride_t = _glr_inputs(p, x, g, gate_logsigmoid, gate_lower_bound, complement_input)
    p.T, p.D = T, D = x.shape
    N = _sequences(p, cu_seqlens, x)
    p.d_h_stride_t = _rows("d_h", d_h, 2, x)[0]
    if d_h.dtype != x.dtype:
        raise TypeError(f"d_h must be {x.dtype}, got {d_h.dtype}")
    p.d_h = d_h.data_ptr()
    if initial_state is not None:
        p.initial_state = _packed("initial_state", initial_state, (N, D), _STATE_DTYPES, x)
        p.initial_state_dtype = _DTYPES[initial_state.dtype]
    if d_final_state is not None:
        p.d_final_state = _packed("d_final_state", d_final_state, (N, D), _FP32, x)
    if checkpoints is not None:
        p.checkpoints = _packed("checkpoints", checkpoints, (glr_checkpoint_rows(T, N), D), _FP32, x)
    dx, strides = _result("dx", dx, x)
    p.dx, p.dx_stride_t = dx.data_ptr(), strides[0]
    dg, strides = _result("dg", dg, g)
    p.dg, p.dg_stride_t = dg.data_ptr(), strides[0]
    d_initial_state, p.d_initial_state = _state_dest("d_initial_state", d_initial_state, (N, D), torch.float32, x)
    need = B.load().la_glr_workspace_bytes(T, N, D, 1, checkpoints is not None)
    ws = _workspace(p, workspace, need, x)  # noqa: F841
    if status is not None:
        _status(p, status, x)
    _call("glr_bwd", p, x)
    return dx, dg, d_initial_state


@_on_stream
def glr_decode(x: torch.Tensor, g: torch.Tensor, state_pool: torch.Tensor, *,
               state_indices: Optional[torch.Tensor] = None, gate_logsigmoid: bool = False,
               gate_lower_bound: Optional[float] = None, complement_input: bool = False,
               h: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """One recurrence step for each of N sequences: x, g [N, D]; sequence i steps pool[state_indices[i]] (pool[i]
    without indices) of state_pool [P, D] (fp32 or bf16) in place.  Returns h [N, D] in x's dtype."""
    p = B.GlrDecodeParams()
    p.x_stride_n, p.g_stride_n = _glr_inputs(p, x, g, gate_logsigmoid, gate_lower_bound, complement_input)
    p.N, p.D = N, D = x.shape
    if not isinstance(state_pool, torch.Tensor) or state_pool.dim() != 2:
        raise ValueError("state_pool must be a contiguous [P, D] tensor")
    p.state_pool_size = P = state_pool.shape[0]
    p.state_pool = _packed("state_pool", state_pool, (P, D), _STATE_DTYPES, x)
    p.state_dtype = _DTYPES[state_pool.dtype]
    if state_indices is not None:
        _indices(p, state_indices, N, x)
    h, strides = _result("h", h, x)
    p.h, p.h_stride_n = h.data_ptr(), strides[0]
    if status is not None:
        _status(p, status, x)
    _call("glr_decode", p, x)
    return h


# ------------------------------------------------------------------ group norm
def _gn_inputs(p, x, weight, bias, z, center, activation, eps) -> None:
    _, p.x_stride_h, _ = strides = _rows("x", x, 3)
    p.x, p.x_stride_t, p.x_dtype = x.data_ptr(), strides[0], _dtype("x", x)
    p.T, p.H, p.V = _, H, V = x.shape
    if not isinstance(weight, torch.Tensor) or weight.dim() not in (1, 2):
        raise ValueError("weight must be [V] or [H, V]")
    per_head = weight.dim() == 2
    shape = (H, V) if per_head else (V,)
    p.weight, p.per_head = _packed("weight", weight, shape, _STATE_DTYPES, x), per_head
    p.weight_dtype = _DTYPES[weight.dtype]
    if bias is not None:
        p.bias = _packed("bias", bias, shape, (weight.dtype,), x)
    if z is not None:
        strides = _rows("z", z, 3, x)
        if z.dtype != x.dtype:
            raise TypeError(f"z must be {x.dtype}, got {z.dtype}")
        p.z, p.z_stride_t, p.z_stride_h = z.data_ptr(), strides[0], strides[1]
    p.center, p.activation, p.eps = bool(center), _activation(activation), eps


@_on_stream
def gn_fwd(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None, *,
           z: Optional[torch.Tensor] = None, center: bool = True, activation: Optional[str] = "silu",
           eps: float = 1e-5, y: Optional[torch.Tensor] = None,
           stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Group norm of every head's V channels of every token, x [T, H, V] (bf16 or fp32), with an activation:
    p = n weight + bias, y = activation(p) without z, y = p * activation(z) with the gate z [T, H, V].
    weight and bias are [V] (shared by the heads) or [H, V]; center=False leaves the mean in (RMS norm)."""
    p = B.GnFwdParams()
    _gn_inputs(p, x, weight, bias, z, center, activation, eps)
    y, strides = _result("y", y, x)
    p.y, p.y_stride_t, p.y_stride_h = y.data_ptr(), strides[0], strides[1]
    _call("gn_fwd", p, x)
    return y


@_on_stream
def gn_bwd(x: torch.Tensor, weight: torch.Tensor, dy: torch.Tensor, bias: Optional[torch.Tensor] = None, *,
           z: Optional[torch.Tensor] = None, center: bool = True, activation: Optional[str] = "silu",
           eps: float = 1e-5, dx: Optional[torch.Tensor] = None, dz: Optional[torch.Tensor] = None,
           workspace: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None
           ) -> Tuple[torch.Tensor, torch.Tensor, Optional[torch.Tensor], Optional[torch.Tensor]]:
    """Gradients of sum(dy * y) for gn_fwd with the same inputs: (dx, d_weight, d_bias or None, dz or None)."""
    p = B.GnBwdParams()
    _gn_inputs(p, x, weight, bias, z, center, activation, eps)
    strides = _rows("dy", dy, 3, x)
    if dy.dtype != x.dtype:
        raise TypeError(f"dy must be {x.dtype}, got {dy.dtype}")
    p.dy, p.dy_stride_t, p.dy_stride_h = dy.data_ptr(), strides[0], strides[1]
    dx, strides = _result("dx", dx, x)
    p.dx, p.dx_stride_t, p.dx_stride_h = dx.data_ptr(), strides[0], strides[1]
    if z is not None:
        dz, strides = _result("dz", dz, x)
        p.dz, p.dz_stride_t, p.dz_stride_h = dz.data_ptr(), strides[0], strides[1]
    else:
        dz = None
    d_weight = torch.empty_like(weight)
    p.d_weight = d_weight.data_ptr()
    d_bias = None
    if bias is not None:
        d_bias = torch.empty_like(bias)
        p.d_bias = d_bias.data_ptr()
    ws = _workspace(p, workspace, B.load().la_gn_bwd_workspace_bytes(p.T, p.H, p.V, p.per_head), x)  # noqa: F841
    _call("gn_bwd", p, x)
    return dx, d_weight, d_bias, dz


# ------------------------------------------------------------------ short convolution
def _sconv_inputs(p, x, weight, bias, activation) -> int:
    """Fills in the operands; returns x's row stride."""
    strides = _rows("x", x, 2)
    D = x.shape[1]
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be [D, W]")
    W = weight.shape[1]
    p.weight, p.weight_dtype = _packed("weight", weight, (D, W), _STATE_DTYPES, x), _DTYPES[weight.dtype]
    if bias is not None:
        p.bias = _packed("bias", bias, (D,), (weight.dtype,), x)
    p.x, p.x_dtype = x.data_ptr(), _dtype("x", x)
    p.D, p.W, p.activation = D, W, _activation(activation)
    return strides[0]


@_on_stream
def sconv_fwd(x: torch.Tensor, weight: torch.Tensor, cu_seqlens: torch.Tensor, bias: Optional[torch.Tensor] = None, *,
              activation: Optional[str] = "silu", initial_state: Optional[torch.Tensor] = None,
              output_final_state: bool = True, state_indices: Optional[torch.Tensor] = None,
              y: Optional[torch.Tensor] = None, final_state: Optional[torch.Tensor] = None,
              status: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None
              ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Causal depthwise convolution over W = 2, 3 or 4 tokens along each sequence, with an activation:
    y_t = act(bias + sum_j weight[:, j] x_{t - (W - 1) + j}), x [T, D] (bf16 or fp32), weight [D, W].
    Returns (y, final_state [N, W - 1, D] in x's dtype: the last W - 1 inputs, or None).

    initial_state [N, W - 1, D]: the tokens before each sequence's first (zeros without one).  state_indices ([N]
    int32): initial_state is then a pool [P, W - 1, D], updated in place, and no final_state is returned."""
    p = B.SconvFwdParams()
    p.x_stride_t = _sconv_inputs(p, x, weight, bias, activation)
    p.T, D = x.shape
    rows = weight.shape[1] - 1
    N = _sequences(p, cu_seqlens, x)
    states = N
    if state_indices is not None:
        if initial_state is None or initial_state.dim() != 3:
            raise ValueError("state_indices needs initial_state as a contiguous pool [P, W - 1, D]")
        if final_state is not None:
            raise ValueError("state_indices and final_state are exclusive")
        _indices(p, state_indices, N, x)
        p.state_pool_size = states = initial_state.shape[0]
        output_final_state = False
    if initial_state is not None:
        p.initial_state = _packed("initial_state", initial_state, (states, rows, D), (x.dtype,), x)
    y, strides = _result("y", y, x)
    p.y, p.y_stride_t = y.data_ptr(), strides[0]
    if output_final_state:
        final_state, p.final_state = _state_dest("final_state", final_state, (N, max(rows, 0), D), x.dtype, x)
    else:
        final_state = None
    if status is not None:
        _status(p, status, x)
    _call("sconv_fwd", p, x)
    return y, final_state


@_on_stream
def sconv_bwd(x: torch.Tensor, weight: torch.Tensor, cu_seqlens: torch.Tensor, dy: torch.Tensor,
              bias: Optional[torch.Tensor] = None, *, activation: Optional[str] = "silu",
              initial_state: Optional[torch.Tensor] = None, d_final_state: Optional[torch.Tensor] = None,
              dx: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
              status: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None
              ) -> Tuple[torch.Tensor, torch.Tensor, Optional[torch.Tensor], torch.Tensor]:
    """Gradients of sum(dy * y) + sum(d_final_state * final_state) for sconv_fwd with the same inputs: (dx, d_weight,
    d_bias or None, d_initial_state [N, W - 1, D] in x's dtype)."""
    p = B.SconvBwdParams()
    p.x_stride_t = _sconv_inputs(p, x, weight, bias, activation)
    p.T, D = T, _ = x.shape
    W = weight.shape[1]
    N = _sequences(p, cu_seqlens, x)
    p.dy_stride_t = _rows("dy", dy, 2, x)[0]
    if dy.dtype != x.dtype:
        raise TypeError(f"dy must be {x.dtype}, got {dy.dtype}")
    p.dy = dy.data_ptr()
    if initial_state is not None:
        p.initial_state = _packed("initial_state", initial_state, (N, W - 1, D), (x.dtype,), x)
    if d_final_state is not None:
        p.d_final_state = _packed("d_final_state", d_final_state, (N, W - 1, D), (x.dtype,), x)
    dx, strides = _result("dx", dx, x)
    p.dx, p.dx_stride_t = dx.data_ptr(), strides[0]
    d_weight = torch.empty_like(weight)
    p.d_weight = d_weight.data_ptr()
    d_bias = None
    if bias is not None:
        d_bias = torch.empty_like(bias)
        p.d_bias = d_bias.data_ptr()
    d_initial_state = torch.empty((N, max(W - 1, 0), D), dtype=x.dtype, device=x.device)
    p.d_initial_state = d_initial_state.data_ptr()
    ws = _workspace(p, workspace, B.load().la_sconv_bwd_workspace_bytes(T, N, D, W), x)  # noqa: F841
    if status is not None:
        _status(p, status, x)
    _call("sconv_bwd", p, x)
    return dx, d_weight, d_bias, d_initial_state


@_on_stream
def sconv_decode(x: torch.Tensor, weight: torch.Tensor, state_pool: torch.Tensor, bias: Optional[torch.Tensor] = None, *,
                 state_indices: Optional[torch.Tensor] = None, activation: Optional[str] = "silu",
                 y: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                 stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """One new token for each of N sequences: x [N, D]; sequence i's last W - 1 inputs are pool[state_indices[i]]
    (pool[i] without indices) of state_pool [P, W - 1, D] in x's dtype, moved on in place.  Returns y [N, D]."""
    p = B.SconvDecodeParams()
    p.x_stride_n = _sconv_inputs(p, x, weight, bias, activation)
    p.N, D = N, _ = x.shape
    if not isinstance(state_pool, torch.Tensor) or state_pool.dim() != 3:
        raise ValueError("state_pool must be a contiguous [P, W - 1, D] tensor")
    p.state_pool_size = P = state_pool.shape[0]
    p.state_pool = _packed("state_pool", state_pool, (P, weight.shape[1] - 1, D), (x.dtype,), x)
    if state_indices is not None:
        _indices(p, state_indices, N, x)
    y, strides = _result("y", y, x)
    p.y, p.y_stride_n = y.data_ptr(), strides[0]
    if status is not None:
        _status(p, status, x)
    _call("sconv_decode", p, x)
    return y


# ------------------------------------------------------------------ autograd
def _cotangent(d, like: torch.Tensor) -> torch.Tensor:
    """An output's cotangent as the kernels read it (an expanded one is laid out)."""
    if d is None:
        return torch.zeros_like(like)
    d = d.to(like.dtype)
    return d if d.shape[-1] <= 1 or d.stride(-1) == 1 else d.contiguous()


class _GLR(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, g, cu_seqlens, initial_state, save_checkpoints, gate):
        h, fin, ck = glr_fwd(x, g, cu_seqlens, initial_state=initial_state, output_checkpoints=save_checkpoints, **gate)
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(x, g, cu_seqlens, initial_state, ck)
        ctx.gate = gate
        return h, fin

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, d_h, d_fin):
        x, g, cu, s0, ck = ctx.saved_tensors
        if d_fin is not None:
            d_fin = d_fin.float().contiguous()
        dx, dg, ds0 = glr_bwd(x, g, cu, _cotangent(d_h, x), initial_state=s0, d_final_state=d_fin, checkpoints=ck,
                              **ctx.gate)
        return dx, dg, None, None if s0 is None else ds0.to(s0.dtype), None, None


def gated_linear_recurrence(x: torch.Tensor, g: torch.Tensor, cu_seqlens: torch.Tensor, *,
                            initial_state: Optional[torch.Tensor] = None, gate_logsigmoid: bool = False,
                            gate_lower_bound: Optional[float] = None, complement_input: bool = False,
                            save_checkpoints: bool = True) -> Tuple[torch.Tensor, torch.Tensor]:
    """Differentiable glr_fwd: returns (h, final_state); gradients flow to x, g and initial_state.
    save_checkpoints keeps the state entering every 128 tokens (D * 4 bytes each) for the backward; without them
    it recomputes them."""
    gate = {"gate_logsigmoid": gate_logsigmoid, "gate_lower_bound": gate_lower_bound,
            "complement_input": complement_input}
    return _GLR.apply(x, g, cu_seqlens, initial_state, save_checkpoints, gate)


class _GroupNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, z, opts):
        ctx.save_for_backward(x, weight, bias, z)
        ctx.opts = opts
        return gn_fwd(x, weight, bias, z=z, **opts)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, weight, bias, z = ctx.saved_tensors
        dx, dw, db, dz = gn_bwd(x, weight, _cotangent(dy, x), bias, z=z, **ctx.opts)
        return dx, dw, db, dz, None


def group_norm(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None, *,
               z: Optional[torch.Tensor] = None, center: bool = True, activation: Optional[str] = "silu",
               eps: float = 1e-5) -> torch.Tensor:
    """Differentiable gn_fwd: gradients flow to x, weight, bias and z."""
    return _GroupNorm.apply(x, weight, bias, z, {"center": center, "activation": activation, "eps": eps})


class _ShortConv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, cu_seqlens, initial_state, activation):
        y, fin = sconv_fwd(x, weight, cu_seqlens, bias, activation=activation, initial_state=initial_state)
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(x, weight, bias, cu_seqlens, initial_state)
        ctx.activation = activation
        return y, fin

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, d_fin):
        x, weight, bias, cu, s0 = ctx.saved_tensors
        if d_fin is not None:
            d_fin = d_fin.to(x.dtype).contiguous()
        dx, dw, db, ds0 = sconv_bwd(x, weight, cu, _cotangent(dy, x), bias, activation=ctx.activation,
                                    initial_state=s0, d_final_state=d_fin)
        return dx, dw, db, None, None if s0 is None else ds0, None


def short_conv(x: torch.Tensor, weight: torch.Tensor, cu_seqlens: torch.Tensor, bias: Optional[torch.Tensor] = None, *,
               activation: Optional[str] = "silu", initial_state: Optional[torch.Tensor] = None
               ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Differentiable sconv_fwd: returns (y, final_state); gradients flow to x, weight, bias and initial_state."""
    return _ShortConv.apply(x, weight, bias, cu_seqlens, initial_state, activation)
